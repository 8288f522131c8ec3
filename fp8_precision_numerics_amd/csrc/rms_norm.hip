// Root-mean-square norm that adds the residual and leaves in 8 bits, and its
// gradient.
//
//   h = round_to_xtype(x + residual)      (x itself without a residual)
//   r = 1 / sqrt(mean_n h^2 + eps)
//   y = h * r * weight,  q = round_to_fp8(y * scale)
//
// with one scale for the tensor (delayed scaling) or one per 128 values of a row
// (current scaling, s_b = MAX / max|y| over the block, as the per-block
// quantiser).  Gradient, with g = dy * weight:
//
//   dx = r (g - h r^2 mean_n(g h)) + dresidual,   dweight_n = sum_m dy h r
//
// HBM-bound; measured on MI355X (bf16, residual): 8192 x 4096 with amax 43 us (235 MB,
// 5.5 TB/s, a copy's rate), 1777 x 7168 with block scales 19.7 us (90 MB, 4.6 TB/s), the
// gradient of 8192 x 4096 with dweight 54 us (268 MB, 5.0 TB/s); one row of 4096 3 us.
// The forward reads x (and the residual) once and writes the sum and
// the codes once, because a row stays in registers between the sum of squares
// and the encode.  A row of up to 1024 values belongs to a wavefront (its sum takes
// shuffles only), one of up to 16384 to a workgroup just large enough for two groups
// of eight consecutive values ("octets") a thread.  The grid walks the
// rows, so the weight is loaded once per workgroup and the gradient's dweight
// stays in registers: one fp32 partial row per workgroup goes to the workspace,
// and a second kernel adds them in a fixed order.  Rows too long for the
// registers are read twice (the second time mostly from the caches).
// Sums of squares and of products are fp32: per lane over its octets, then across
// lanes, so a term of a row of up to 16384 values passes through at most about 40 roundings.
#include "device_common.hpp"
#include "launch.hpp"
#include "row_octets.hpp"
#include "stats.hpp"

namespace fp8mi {
namespace {

struct NormArgs {
  const void* x;
  const void* residual;  // null: none
  const void* weight;
  void* sum_out;         // null without a residual; may be null, x or the residual
  uint8_t* q;
  const float* scale;    // one scale for the tensor
  float* scale_inv;      // blocks: one per 128 values of a row
  float* rstd;           // may be null
  uint32_t* amax_bits;
  unsigned long long* sat;
  uint4* partials;
  int64_t rows, cols;
  float eps;
};

// What a norm's epilogue does: codes with the given scale, the same with amax and
// saturation count, or codes and inverse scales per 128 values.
enum : int { kNormScaled = 0, kNormStats = 1, kNormBlocks = 2 };

template <int XT, int FMT, int KIND>
__device__ __forceinline__ void norm_encode(const NormArgs& a, const Octet<XT>& h, const Octet<XT>& wt, float r,
                                            float scale, int64_t row, int64_t o, int64_t octets, bool valid,
                                            LaneStats& st) {
  float y[8], w[8];
  h.widen(y);
  wt.widen(w);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
  if constexpr (KIND == kNormBlocks) {
    // The 16 lanes of a block hold consecutive octets; a lane past the row's end
    // takes part with zeros.
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = f2u(y[e]) & 0x7FFFFFFFu;
      m = m > b ? m : b;
    }
    if (!valid) m = 0u;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const uint32_t other = (uint32_t)__shfl_xor((int)m, off, 64);
      m = m > other ? m : other;
    }
    float si = 1.0f;
    scale = 1.0f;
    scale_from_amax_bits<FMT>(m, &scale, &si);
    if (valid && (o & 15) == 0) a.scale_inv[row * ((octets + 15) / 16) + (o >> 4)] = si;
  }
  if (valid) {
    const uint2 c = encode8<FMT>(y, scale, KIND == kNormStats, KIND == kNormStats && a.sat, st);
    *reinterpret_cast<uint2*>(a.q + row * a.cols + o * 8) = c;
  }
}

// WG: a row per workgroup, whose size fits the row; otherwise a row per wavefront, four
// side by side.
template <int XT, int FMT, int KIND, bool WG, int VPT>
__global__ __launch_bounds__(WG ? 1024 : 256) void rmsnorm_kernel(NormArgs a) {
  __shared__ float buf[2][kMaxWaves];
  const int TPR = WG ? blockDim.x : 64, RPB = WG ? 1 : 4;
  const int t = WG ? threadIdx.x : threadIdx.x & 63;
  const int64_t octets = a.cols / 8;
  const float scale = KIND == kNormBlocks ? 1.0f : *a.scale;
  const float inv_n = 1.0f / (float)a.cols;
  Octet<XT> wt[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    wt[v].clear();
    if (t + v * TPR < octets) wt[v].load(a.weight, t + v * TPR);
  }
  LaneStats st;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + (WG ? 0 : threadIdx.x >> 6); row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const int64_t base = row * octets;
    Octet<XT> h[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      h[v].clear();
      if (t + v * TPR < octets) h[v].load_nt(a.x, base + t + v * TPR);
    }
    if (a.residual) {
      Octet<XT> res[VPT];
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        res[v].clear();
        if (t + v * TPR < octets) res[v].load_nt(a.residual, base + t + v * TPR);
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float f[8], g[8];
        h[v].widen(f);
        res[v].widen(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += g[e];
        h[v].narrow(f);
        if (a.sum_out && t + v * TPR < octets) h[v].store_nt(a.sum_out, base + t + v * TPR);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float f[8];
      h[v].widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
    }
    ss = row_sum<WG>(ss, buf, turn++);
    const float r = 1.0f / __builtin_sqrtf(ss * inv_n + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = r;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int64_t o = t + v * TPR;
      norm_encode<XT, FMT, KIND>(a, h[v], wt[v], r, scale, row, o, octets, o < octets, st);
    }
  }
  if constexpr (KIND == kNormStats) block_finish(st.amax(), wave_sum_u32(st.sat), a.amax_bits, a.sat, a.partials);
}

// Rows of any length: a workgroup per row, two passes over it.  The second pass
// reads the stored sum where there is one (each lane what it stored itself),
// since x or the residual may be the buffer that the sum has overwritten.
template <int XT, int FMT, int KIND, int NT>
__global__ __launch_bounds__(NT) void rmsnorm_long_kernel(NormArgs a) {
  __shared__ float buf[2][kMaxWaves];
  const int t = threadIdx.x;
  const int64_t octets = a.cols / 8;
  const float scale = KIND == kNormBlocks ? 1.0f : *a.scale;
  LaneStats st;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * octets;
    auto added = [&](int64_t o) {
      Octet<XT> h;
      h.load(a.x, base + o);
      if (a.residual) {
        Octet<XT> res;
        res.load(a.residual, base + o);
        float f[8], g[8];
        h.widen(f);
        res.widen(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += g[e];
        h.narrow(f);
      }
      return h;
    };
    float ss = 0.0f;
    for (int64_t o = t; o < octets; o += NT) {
      const Octet<XT> h = added(o);
      if (a.sum_out) h.store(a.sum_out, base + o);
      float f[8], part = 0.0f;
      h.widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) part = __builtin_fmaf(f[e], f[e], part);
      ss += part;
    }
    ss = row_sum<true>(ss, buf, turn++);
    const float r = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = r;
    // whole workgroup passes, so that the 16 lanes of a block meet in its shuffles
    for (int64_t o0 = 0; o0 < octets; o0 += NT) {
      const int64_t o = o0 + t;
      Octet<XT> h, wt;
      h.clear();
      wt.clear();
      if (o < octets) {
        if (a.sum_out) h.load(a.sum_out, base + o);
        else h = added(o);
        wt.load(a.weight, o);
      }
      norm_encode<XT, FMT, KIND>(a, h, wt, r, scale, row, o, octets, o < octets, st);
    }
  }
  if constexpr (KIND == kNormStats) block_finish(st.amax(), wave_sum_u32(st.sat), a.amax_bits, a.sat, a.partials);
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
struct NormBackArgs {
  const void* dy;
  const void* h;
  const float* rstd;
  const void* weight;
  const void* dres;  // may be null
  void* dx;
  float* partials;   // [workgroups x cols] fp32, null: no dweight
  int64_t rows, cols;
};

template <int XT, bool WG, int VPT>
__global__ __launch_bounds__(WG ? 1024 : 256) void rmsnorm_backward_kernel(NormBackArgs a) {
  __shared__ float buf[2][kMaxWaves];
  const int TPR = WG ? blockDim.x : 64, RPB = WG ? 1 : 4;
  const int t = WG ? threadIdx.x : threadIdx.x & 63;
  const int64_t octets = a.cols / 8;
  const float inv_n = 1.0f / (float)a.cols;
  float w[VPT][8], dw[VPT][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    Octet<XT> wt;
    wt.clear();
    if (t + v * TPR < octets) wt.load(a.weight, t + v * TPR);
    wt.widen(w[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + (WG ? 0 : threadIdx.x >> 6); row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const int64_t base = row * octets;
    Octet<XT> dy[VPT], h[VPT], dr[VPT];
    const float r = a.rstd[row];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      dy[v].clear();
      h[v].clear();
      dr[v].clear();
      if (t + v * TPR < octets) {
        dy[v].load(a.dy, base + t + v * TPR);
        h[v].load(a.h, base + t + v * TPR);
        if (a.dres) dr[v].load(a.dres, base + t + v * TPR);
      }
    }
    float gh = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float d[8], f[8];
      dy[v].widen(d);
      h[v].widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        gh = __builtin_fmaf(d[e] * w[v][e], f[e], gh);
        dw[v][e] = __builtin_fmaf(d[e], f[e] * r, dw[v][e]);
      }
    }
    gh = row_sum<WG>(gh, buf, turn++);
    const float k = gh * inv_n * r * r;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (t + v * TPR >= octets) continue;
      float d[8], f[8], s[8];
      dy[v].widen(d);
      h[v].widen(f);
      dr[v].widen(s);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += r * (d[e] * w[v][e] - f[e] * k);
      Octet<XT> out;
      out.narrow(s);
      out.store_nt(a.dx, base + t + v * TPR);
    }
  }
  if (!a.partials) return;
  if constexpr (!WG) {
    // the rows side by side add up in LDS, in a fixed order
    __shared__ float sum[4][64 * VPT * 8];
    float* mine = sum[threadIdx.x >> 6];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[(v * 8 + e) * 64 + t] = dw[v][e];
    __syncthreads();
    if (threadIdx.x >= 64) return;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int g = 1; g < 4; ++g) dw[v][e] += sum[g][(v * 8 + e) * 64 + t];
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (t + v * TPR >= octets) continue;
    float4* dst = reinterpret_cast<float4*>(a.partials + (int64_t)blockIdx.x * a.cols + (t + v * TPR) * 8);
    dst[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
    dst[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
  }
}

// Rows of any length: two passes, dweight added up in the workgroup's own partial
// row (each lane its own columns, so no two lanes meet at an address).
template <int XT, int NT>
__global__ __launch_bounds__(NT) void rmsnorm_backward_long_kernel(NormBackArgs a) {
  __shared__ float buf[2][kMaxWaves];
  const int t = threadIdx.x;
  const int64_t octets = a.cols / 8;
  float* part = a.partials ? a.partials + (int64_t)blockIdx.x * a.cols : nullptr;
  int turn = 0;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * octets;
    const float r = a.rstd[row];
    float gh = 0.0f;
    for (int64_t o = t; o < octets; o += NT) {
      Octet<XT> dy, h, wt;
      dy.load(a.dy, base + o);
      h.load(a.h, base + o);
      wt.load(a.weight, o);
      float d[8], f[8], w[8], acc = 0.0f;
      dy.widen(d);
      h.widen(f);
      wt.widen(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = __builtin_fmaf(d[e] * w[e], f[e], acc);
      gh += acc;
    }
    gh = row_sum<true>(gh, buf, turn++);
    const float k = gh / (float)a.cols * r * r;
    for (int64_t o = t; o < octets; o += NT) {
      Octet<XT> dy, h, wt, dr, out;
      dy.load(a.dy, base + o);
      h.load(a.h, base + o);
      wt.load(a.weight, o);
      dr.clear();
      if (a.dres) dr.load(a.dres, base + o);
      float d[8], f[8], w[8], s[8];
      dy.widen(d);
      h.widen(f);
      wt.widen(w);
      dr.widen(s);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += r * (d[e] * w[e] - f[e] * k);
      out.narrow(s);
      out.store(a.dx, base + o);
      if (part) {
        float4* p = reinterpret_cast<float4*>(part + o * 8);
        float4 lo = first ? make_float4(0.f, 0.f, 0.f, 0.f) : p[0], hi = first ? make_float4(0.f, 0.f, 0.f, 0.f) : p[1];
        lo.x = __builtin_fmaf(d[0], f[0] * r, lo.x);
        lo.y = __builtin_fmaf(d[1], f[1] * r, lo.y);
        lo.z = __builtin_fmaf(d[2], f[2] * r, lo.z);
        lo.w = __builtin_fmaf(d[3], f[3] * r, lo.w);
        hi.x = __builtin_fmaf(d[4], f[4] * r, hi.x);
        hi.y = __builtin_fmaf(d[5], f[5] * r, hi.y);
        hi.z = __builtin_fmaf(d[6], f[6] * r, hi.z);
        hi.w = __builtin_fmaf(d[7], f[7] * r, hi.w);
        p[0] = lo;
        p[1] = hi;
      }
    }
    first = false;
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
// Workgroups of the forward.  Threads a compute unit: 2048, or 1024 where every
// workgroup costs a partial of the statistics (8192 x 4096: 42.9 against 44.0 us;
// without them 40.3 and 42.3, but 1777 x 7168 19.0 and 18.2 us).  With statistics, up to
// four rows a wavefront or workgroup stay in one workgroup, which writes them itself:
// the second launch costs 3 us, a further row about one.
int norm_groups(int64_t rows, int64_t octets, int kind) {
  const bool stats = kind == kNormStats;
  const int rpb = octets <= 128 ? 4 : 1;
  if (stats && rows <= 4 * rpb) return 1;
  if (octets <= 128) return row_groups(rows, rpb, 8, 0);
  if (octets <= 2048) return row_groups(rows, rpb, (stats ? 1024 : 2048) / row_threads(octets), 0);
  return row_groups(rows, rpb, 2, 0);
}

template <int XT, int FMT, int KIND>
void norm_run(const NormArgs& a, int g, hipStream_t st) {
  const int64_t o = a.cols / 8;
  const dim3 grid((unsigned)g);
  if (o <= 64) hipLaunchKernelGGL((rmsnorm_kernel<XT, FMT, KIND, false, 1>), grid, dim3(256), 0, st, a);
  else if (o <= 128) hipLaunchKernelGGL((rmsnorm_kernel<XT, FMT, KIND, false, 2>), grid, dim3(256), 0, st, a);
  else if (o <= 2048) hipLaunchKernelGGL((rmsnorm_kernel<XT, FMT, KIND, true, 2>), grid, dim3(row_threads(o)), 0, st, a);
  else hipLaunchKernelGGL((rmsnorm_long_kernel<XT, FMT, KIND, 1024>), grid, dim3(1024), 0, st, a);
}

template <int XT, int FMT>
void norm_kind(const NormArgs& a, int kind, int g, hipStream_t st) {
  if (kind == kNormBlocks) norm_run<XT, FMT, kNormBlocks>(a, g, st);
  else if (kind == kNormStats) norm_run<XT, FMT, kNormStats>(a, g, st);
  else norm_run<XT, FMT, kNormScaled>(a, g, st);
}

void norm_launch(const NormArgs& a, int xtype, int fmt, int kind, int g, hipStream_t st) {
  if (xtype == kBF16) {
    if (fmt == kE4M3) norm_kind<kBF16, kE4M3>(a, kind, g, st);
    else norm_kind<kBF16, kE5M2>(a, kind, g, st);
  } else {
    if (fmt == kE4M3) norm_kind<kF32, kE4M3>(a, kind, g, st);
    else norm_kind<kF32, kE5M2>(a, kind, g, st);
  }
}

// Workgroups of the gradient's kernel: up to 1024 threads a compute unit for rows of a
// wavefront; two workgroups for rows up to 8192 (4096: 46.1 us against 52.1 with four,
// whose partials cost more than they gain), one beyond.
int norm_back_groups(int64_t rows, int64_t octets, int64_t slots) {
  if (octets <= 128) return row_groups(rows, 4, 4, slots);
  return row_groups(rows, 1, octets <= 1024 ? 2 : 1, slots);
}

template <int XT>
void norm_back_run(const NormBackArgs& a, int g, hipStream_t st) {
  const int64_t o = a.cols / 8;
  const dim3 grid((unsigned)g);
  if (o <= 64) hipLaunchKernelGGL((rmsnorm_backward_kernel<XT, false, 1>), grid, dim3(256), 0, st, a);
  else if (o <= 128) hipLaunchKernelGGL((rmsnorm_backward_kernel<XT, false, 2>), grid, dim3(256), 0, st, a);
  else if (o <= 2048) hipLaunchKernelGGL((rmsnorm_backward_kernel<XT, true, 2>), grid, dim3(row_threads(o)), 0, st, a);
  else hipLaunchKernelGGL((rmsnorm_backward_long_kernel<XT, 1024>), grid, dim3(1024), 0, st, a);
}

}  // namespace

hipError_t launch_rmsnorm_quantize(const void* x, const void* residual, const void* weight, int xtype, int64_t rows,
                                   int64_t cols, float eps, int fmt, const float* scale, void* sum_out, uint8_t* q,
                                   float* rstd, float* amax, unsigned long long* sat, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  const bool stats = amax || sat, empty = rows * cols == 0;
  const int kind = stats ? kNormStats : kNormScaled;
  const int g = empty ? 0 : norm_groups(rows, cols / 8, kind);
  const bool gather = stats && g != 1;  // a single workgroup writes the statistics itself
  // A slot for every workgroup, or none: a grid cut to the slots there are would leave
  // the device idle (8192 x 4096 on one workgroup: 15 ms against 38 us with atomics).
  const bool fits = workspace && workspace_bytes >= (size_t)g * sizeof(uint4);
  NormArgs a{x, residual, weight, sum_out, q, scale, nullptr, rstd, reinterpret_cast<uint32_t*>(amax), sat,
             gather && fits ? reinterpret_cast<uint4*>(workspace) : nullptr, rows, cols, eps};
  if (gather && !a.partials) {
    const hipError_t e = launch_clear_stats(amax, sat, stream);
    if (e != hipSuccess) return e;
  }
  if (!empty) norm_launch(a, xtype, fmt, kind, g, stream);
  if (a.partials) return launch_reduce_stats(a.partials, g, amax, sat, stream);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_quantize_blockwise(const void* x, const void* residual, const void* weight, int xtype,
                                             int64_t rows, int64_t cols, float eps, int fmt, void* sum_out, uint8_t* q,
                                             float* scale_inv, float* rstd, hipStream_t stream) {
  if (rows * cols == 0) return hipSuccess;
  const NormArgs a{x, residual, weight, sum_out, q, nullptr, scale_inv, rstd, nullptr, nullptr, nullptr, rows, cols, eps};
  norm_launch(a, xtype, fmt, kNormBlocks, norm_groups(rows, cols / 8, kNormBlocks), stream);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_backward(const void* dy, const void* h, const float* rstd, const void* weight,
                                   const void* dres, int xtype, int64_t rows, int64_t cols, void* dx, float* dweight,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int g = 0;
  float* partials = nullptr;
  if (rows * cols > 0) {
    g = norm_back_groups(rows, cols / 8, dweight ? (int64_t)(workspace_bytes / (cols * sizeof(float))) : 0);
    if (dweight) partials = g == 1 ? dweight : reinterpret_cast<float*>(workspace);  // a single partial row is the result
    const NormBackArgs a{dy, h, rstd, weight, dres, dx, partials, rows, cols};
    if (xtype == kBF16) norm_back_run<kBF16>(a, g, stream);
    else norm_back_run<kF32>(a, g, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dweight && g != 1) return launch_column_sums(partials, g, cols, dweight, nullptr, 0, nullptr, nullptr, stream);
  return hipGetLastError();
}

}  // namespace fp8mi
