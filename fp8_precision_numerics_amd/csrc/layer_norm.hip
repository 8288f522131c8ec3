// Layer norm that drops values of a branch, adds the residual and leaves in 8 bits,
// and its gradient.
//
//   h = round_to_xtype(drop(x) + residual)
//   m = mean_n h,  r = 1 / sqrt(mean_n (h - m)^2 + eps)
//   y = (h - m) * r * weight + bias,  q = round_to_fp8(y * scale)
//
// Gradient, with g = dy * weight and a = (h - m) r:
//
//   dh = r (g - mean_n g - a mean_n(g a)) + dresidual
//   dx = round(dh),  dbranch = round(drop'(dh)),  dweight_n = sum_m dy a,  dbias_n = sum_m dy
//
// HBM-bound; measured on MI355X (bf16, residual, dropout): 8192 x 4096 with amax 44-45.5 us (235 MB, 5.2-5.3 TB/s, a copy's
// rate), its gradient with both sums and the branch's 65.4 us (336 MB, 5.1 TB/s); 1777 x 1040 fp32 gradient 12 us, of which
// the second launch takes 4; one row of 4096 4.0 us a call.
// The arrangement is the root-mean-square norm's (rms_norm.hip): a row
// stays in registers from the load to the encode, so x and the residual are read
// once and the variance is the sum of (h - m)^2 of values that are there, not a
// difference of two large sums.  A row of up to 1024 values belongs to a wavefront,
// one of up to 16384 to a workgroup just large enough for two octets a thread; the
// grid walks the rows, so weight and bias are loaded once and the gradient's sums
// over the rows stay in registers until one partial row a workgroup goes to the
// workspace.  Longer rows are read three times (gradient: twice), the later times
// mostly from the caches.
// The dropped values are drawn anew in the backward pass (philox.hpp), which costs no
// memory traffic.
// Sums are fp32: per lane over its octets, then across lanes, so a term of a row of
// up to 16384 values passes through at most about 40 roundings.
#include <type_traits>

#include "column_sums.hpp"
#include "launch.hpp"
#include "model_ends.hpp"
#include "philox.hpp"
#include "row_octets.hpp"
#include "stats.hpp"

namespace fp8mi {
namespace {

struct LayerArgs {
  const void* x;
  const void* residual;  // null: none
  const void* weight;
  const void* bias;      // null: none
  void* sum_out;         // may be null, x or the residual
  uint8_t* q;
  const float* scale;
  float* mean;           // may be null
  float* rstd;           // may be null
  uint32_t* amax_bits;
  unsigned long long* sat;
  uint4* partials;
  int64_t rows, cols;
  float eps;
  Dropout drop;
};

// Octet `o` of the tensor (flat): x, dropped and added to the residual `res` (zero
// without one).  Two fp32 roundings, then the type's.
template <int XT>
__device__ __forceinline__ void join_branch(Octet<XT>& h, const Octet<XT>& res, bool add, const Dropper& drop, int64_t o) {
#pragma clang fp contract(off)  // the sum is not fused with the scaling before it
  float f[8];
  h.widen(f);
  if (drop.cut) drop.apply(f, o);
  if (add) {
    float g[8];
    res.widen(g);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += g[e];
  }
  h.narrow(f);
}

template <int XT, int FMT, bool STATS>
__device__ __forceinline__ void layer_encode(const LayerArgs& a, const Octet<XT>& h, const Octet<XT>& wt,
                                             const Octet<XT>& bs, float m, float r, float scale, int64_t octet,
                                             LaneStats& st) {
  float y[8], w[8], b[8];
  h.widen(y);
  wt.widen(w);
  bs.widen(b);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf((y[e] - m) * r, w[e], b[e]);
  const uint2 c = encode8<FMT>(y, scale, STATS, STATS && a.sat, st);
  *reinterpret_cast<uint2*>(a.q + octet * 8) = c;
}

// WG: a row per workgroup, whose size fits the row; otherwise a row per wavefront, four
// side by side.  PRE: a row is requested while the one before it is worked on.
template <int XT, int FMT, bool STATS, bool WG, int VPT, bool PRE>
__global__ __launch_bounds__(WG ? (PRE ? 512 : 1024) : 256) void layernorm_kernel(LayerArgs a) {
  __shared__ float buf[2][kMaxWaves];
  const int TPR = WG ? blockDim.x : 64, RPB = WG ? 1 : 4;
  const int t = WG ? threadIdx.x : threadIdx.x & 63;
  const int64_t octets = a.cols / 8;
  const float scale = *a.scale;
  const float inv_n = 1.0f / (float)a.cols;
  const Dropper drop(a.drop);
  const bool join = a.residual || drop.cut;
  Octet<XT> wt[VPT], bs[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    wt[v].clear();
    bs[v].clear();
    if (t + v * TPR < octets) {
      wt[v].load(a.weight, t + v * TPR);
      if (a.bias) bs[v].load(a.bias, t + v * TPR);
    }
  }
  auto request = [&](int64_t row, Octet<XT>* h, Octet<XT>* res) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      h[v].clear();
      res[v].clear();
      if (row < a.rows && t + v * TPR < octets) {
        h[v].load_nt(a.x, row * octets + t + v * TPR);
        if (a.residual) res[v].load_nt(a.residual, row * octets + t + v * TPR);
      }
    }
  };
  LaneStats st;
  int turn = 0;
  Octet<XT> nh[VPT], nres[VPT];
  if constexpr (PRE) request((int64_t)blockIdx.x * RPB + (WG ? 0 : threadIdx.x >> 6), nh, nres);
  for (int64_t row = (int64_t)blockIdx.x * RPB + (WG ? 0 : threadIdx.x >> 6); row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const int64_t base = row * octets;
    Octet<XT> h[VPT], res[VPT];
    if constexpr (PRE) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        h[v] = nh[v];
        res[v] = nres[v];
      }
      request(row + (int64_t)gridDim.x * RPB, nh, nres);
    } else {
      request(row, h, res);
    }
    if (join) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) join_branch<XT>(h[v], res[v], a.residual != nullptr, drop, base + t + v * TPR);
    }
    if (a.sum_out) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (t + v * TPR < octets) h[v].store_nt(a.sum_out, base + t + v * TPR);
    }
    // A lane past the row's end holds zeros: right for the sum, left out of the squares.
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float f[8];
      h[v].widen(f);
      s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    const float m = row_sum<WG>(s, buf, turn++) * inv_n;
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float f[8];
      h[v].widen(f);
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) part = __builtin_fmaf(f[e] - m, f[e] - m, part);
      ss += t + v * TPR < octets ? part : 0.0f;
    }
    ss = row_sum<WG>(ss, buf, turn++);
    const float r = 1.0f / __builtin_sqrtf(ss * inv_n + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (t + v * TPR < octets) layer_encode<XT, FMT, STATS>(a, h[v], wt[v], bs[v], m, r, scale, base + t + v * TPR, st);
  }
  if constexpr (STATS) block_finish(st.amax(), wave_sum_u32(st.sat), a.amax_bits, a.sat, a.partials);
}

// Rows of any length: a workgroup per row, three passes over it.  The later ones read
// the stored sum where there is one (each lane what it stored itself), since x or the
// residual may be the buffer that the sum has overwritten.
template <int XT, int FMT, bool STATS, int NT>
__global__ __launch_bounds__(NT) void layernorm_long_kernel(LayerArgs a) {
  __shared__ float buf[2][kMaxWaves];
  const int t = threadIdx.x;
  const int64_t octets = a.cols / 8;
  const float scale = *a.scale;
  const Dropper drop(a.drop);
  const bool join = a.residual || drop.cut;
  LaneStats st;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * octets;
    auto joined = [&](int64_t o) {
      Octet<XT> h, res;
      h.load(a.x, base + o);
      if (join) {
        res.clear();
        if (a.residual) res.load(a.residual, base + o);
        join_branch<XT>(h, res, a.residual != nullptr, drop, base + o);
      }
      return h;
    };
    auto again = [&](int64_t o) {
      if (!a.sum_out) return joined(o);
      Octet<XT> h;
      h.load(a.sum_out, base + o);
      return h;
    };
    float s = 0.0f;
    for (int64_t o = t; o < octets; o += NT) {
      const Octet<XT> h = joined(o);
      if (a.sum_out) h.store(a.sum_out, base + o);
      float f[8];
      h.widen(f);
      s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    const float m = row_sum<true>(s, buf, turn++) / (float)a.cols;
    float ss = 0.0f;
    for (int64_t o = t; o < octets; o += NT) {
      const Octet<XT> h = again(o);
      float f[8], part = 0.0f;
      h.widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) part = __builtin_fmaf(f[e] - m, f[e] - m, part);
      ss += part;
    }
    ss = row_sum<true>(ss, buf, turn++);
    const float r = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
    }
    for (int64_t o = t; o < octets; o += NT) {
      const Octet<XT> h = again(o);
      Octet<XT> wt, bs;
      wt.load(a.weight, o);
      bs.clear();
      if (a.bias) bs.load(a.bias, o);
      layer_encode<XT, FMT, STATS>(a, h, wt, bs, m, r, scale, base + o, st);
    }
  }
  if constexpr (STATS) block_finish(st.amax(), wave_sum_u32(st.sat), a.amax_bits, a.sat, a.partials);
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
struct LayerBackArgs {
  const void* dy;
  const void* h;
  const float* mean;
  const float* rstd;
  const void* weight;
  const void* dres;   // may be null
  void* dx;
  void* dbranch;      // may be null
  // One partial row a workgroup of either sum, `pitch` apart; null: not asked for.
  float* dw;
  float* db;
  int64_t pitch;
  int64_t rows, cols;
  Dropout drop;
  int lanes;          // threads a row: 64, or a multiple of it; a workgroup has blockDim.x / lanes rows side by side
};

// Two sums over the lanes of a row at once; as row_sum, of the row's `waves` waves from wave `w0` of the workgroup on.
template <bool WG>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 (*buf)[kMaxWaves], int turn, int w0, int waves) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    v.x += __shfl_xor(v.x, off, 64);
    v.y += __shfl_xor(v.y, off, 64);
  }
  if constexpr (WG) {
    if ((threadIdx.x & 63) == 0) buf[turn & 1][threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[turn & 1][w0];
    for (int w = 1; w < waves; ++w) {
      v.x += buf[turn & 1][w0 + w].x;
      v.y += buf[turn & 1][w0 + w].y;
    }
  }
  return v;
}

// dh of an octet and its two roundings; `octet`: flat.
template <int XT>
__device__ __forceinline__ void layer_gradient(const LayerBackArgs& a, const Dropper& drop, const Octet<XT>& dy,
                                               const Octet<XT>& h, const Octet<XT>& dr, const float* w, float m,
                                               float r, float2 means, int64_t octet) {
  float d[8], f[8], s[8];
  dy.widen(d);
  h.widen(f);
  dr.widen(s);
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] += r * (d[e] * w[e] - means.x - (f[e] - m) * r * means.y);
  Octet<XT> out;
  out.narrow(s);
  out.store_nt(a.dx, octet);
  if (a.dbranch) {
    if (drop.cut) drop.apply(s, octet);
    out.narrow(s);
    out.store_nt(a.dbranch, octet);
  }
}

// One row as loaded.
template <int XT, int VPT>
struct BackRow {
  Octet<XT> dy[VPT], h[VPT], dr[VPT];
  float m, r;
  __device__ __forceinline__ void load(const LayerBackArgs& a, int64_t row, int64_t octets, int t, int TPR) {
    const bool here = row < a.rows;
    m = r = 0.0f;
    if (here) {
      m = a.mean[row];
      r = a.rstd[row];
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      dy[v].clear();
      h[v].clear();
      dr[v].clear();
      if (here && t + v * TPR < octets) {
        const int64_t o = row * octets + t + v * TPR;
        dy[v].load(a.dy, o);
        h[v].load(a.h, o);
        if (a.dres) dr[v].load(a.dres, o);
      }
    }
  }
};

// NT: the largest workgroup.  PRE: a row is requested while the one before it is worked on, which takes the place of
// more workgroups.  Rows side by side in a workgroup add their sums up in LDS at the end: a partial row a
// workgroup, not a row.  Rows of more than 8192 values have workgroups of up to 1024
// threads, whose 128 registers do not hold another row, nor all of one: 28 bytes a lane spill (fp32: 52).  2000 x 16384 bf16 with a
// residual 76 us (3.4 TB/s), with the branch's 90; with 512 threads of four octets and the row requested ahead, which spills more, 112.
// WG: a row is several waves', otherwise one's.
template <int XT, bool WG, int VPT, int NT, bool PRE>
__global__ __launch_bounds__(NT) void layernorm_backward_kernel(LayerBackArgs a) {
  __shared__ float2 buf[2][kMaxWaves];
  const int TPR = WG ? a.lanes : 64, RPB = blockDim.x / TPR;
  const int side = threadIdx.x / TPR, t = threadIdx.x - side * TPR;
  const int64_t octets = a.cols / 8;
  const float inv_n = 1.0f / (float)a.cols;
  const Dropper drop(a.drop);
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + side;
  BackRow<XT, VPT> next;
  if constexpr (PRE) next.load(a, row, octets, t, TPR);
  Octet<XT> wt[VPT];
  float dw[VPT][8], db[VPT][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    wt[v].clear();
    if (t + v * TPR < octets) wt[v].load(a.weight, t + v * TPR);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
  }
  int turn = 0;
  // WG: the rows side by side meet at barriers, so all go on until the first of them is past the end; a row
  // past it has loaded zeros.
  for (; row - (WG ? side : 0) < a.rows; row += step) {
    const int64_t base = row * octets;
    BackRow<XT, VPT> now;
    if constexpr (PRE) {
      now = next;
      next.load(a, row + step, octets, t, TPR);
    } else {
      now.load(a, row, octets, t, TPR);
    }
    const float m = now.m, r = now.r;
    float2 sum = make_float2(0.0f, 0.0f);  // a lane past the row's end holds dy = 0
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float d[8], f[8], w[8];
      now.dy[v].widen(d);
      now.h[v].widen(f);
      wt[v].widen(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float at = (f[e] - m) * r, g = d[e] * w[e];
        sum.x += g;
        sum.y = __builtin_fmaf(g, at, sum.y);
        dw[v][e] = __builtin_fmaf(d[e], at, dw[v][e]);
        db[v][e] += d[e];
      }
    }
    sum = row_sum2<WG>(sum, buf, turn++, side * (TPR >> 6), TPR >> 6);
    if (WG && row >= a.rows) continue;
    const float2 means = make_float2(sum.x * inv_n, sum.y * inv_n);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (t + v * TPR >= octets) continue;
      float w[8];
      wt[v].widen(w);
      layer_gradient<XT>(a, drop, now.dy[v], now.h[v], now.dr[v], w, m, r, means, base + t + v * TPR);
    }
  }
  if (!a.dw && !a.db) return;
  if (RPB > 1) {
    // the rows side by side add up in LDS, in a fixed order, one sum after the other
    __shared__ float sums[NT < 1024 ? NT * VPT * 8 : 1];  // workgroups of more than 512 threads hold one row
    auto meet = [&](float (*v8)[8]) {
      if constexpr (NT < 1024) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) sums[(v * 8 + e) * blockDim.x + threadIdx.x] = v8[v][e];
        __syncthreads();
        if (side == 0) {
          for (int g = 1; g < RPB; ++g)
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
              for (int e = 0; e < 8; ++e) v8[v][e] += sums[(v * 8 + e) * blockDim.x + g * TPR + t];
        }
      }
    };
    if (a.dw) meet(dw);
    if (a.db) meet(db);
    if (side != 0) return;
  }
  auto put = [&](float* to, float (*v8)[8]) {
    if (!to) return;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (t + v * TPR >= octets) continue;
      float4* dst = reinterpret_cast<float4*>(to + (int64_t)blockIdx.x * a.pitch + (int64_t)(t + v * TPR) * 8);
      dst[0] = make_float4(v8[v][0], v8[v][1], v8[v][2], v8[v][3]);
      dst[1] = make_float4(v8[v][4], v8[v][5], v8[v][6], v8[v][7]);
    }
  };
  put(a.dw, dw);
  put(a.db, db);
}

// Rows of any length: two passes, the sums over the rows added up in the workgroup's
// own partial rows (each lane its own columns, so no two lanes meet at an address).
template <int XT, int NT>
__global__ __launch_bounds__(NT) void layernorm_backward_long_kernel(LayerBackArgs a) {
  __shared__ float2 buf[2][kMaxWaves];
  const int t = threadIdx.x;
  const int64_t octets = a.cols / 8;
  const Dropper drop(a.drop);
  float* dw = a.dw ? a.dw + (int64_t)blockIdx.x * a.pitch : nullptr;
  float* db = a.db ? a.db + (int64_t)blockIdx.x * a.pitch : nullptr;
  int turn = 0;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * octets;
    const float m = a.mean[row], r = a.rstd[row];
    float2 sum = make_float2(0.0f, 0.0f);
    for (int64_t o = t; o < octets; o += NT) {
      Octet<XT> dy, h, wt;
      dy.load(a.dy, base + o);
      h.load(a.h, base + o);
      wt.load(a.weight, o);
      float d[8], f[8], w[8];
      float2 part = make_float2(0.0f, 0.0f);
      dy.widen(d);
      h.widen(f);
      wt.widen(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = d[e] * w[e];
        part.x += g;
        part.y = __builtin_fmaf(g, (f[e] - m) * r, part.y);
      }
      sum.x += part.x;
      sum.y += part.y;
    }
    sum = row_sum2<true>(sum, buf, turn++, 0, NT / 64);
    const float2 means = make_float2(sum.x / (float)a.cols, sum.y / (float)a.cols);
    for (int64_t o = t; o < octets; o += NT) {
      Octet<XT> dy, h, wt, dr;
      dy.load(a.dy, base + o);
      h.load(a.h, base + o);
      wt.load(a.weight, o);
      dr.clear();
      if (a.dres) dr.load(a.dres, base + o);
      float d[8], f[8], w[8];
      dy.widen(d);
      h.widen(f);
      wt.widen(w);
      layer_gradient<XT>(a, drop, dy, h, dr, w, m, r, means, base + o);
      auto add = [&](float* to, bool times) {
        if (!to) return;
        float4* p = reinterpret_cast<float4*>(to + o * 8);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (!first) {
          const float4 lo = p[0], hi = p[1];
          v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = times ? __builtin_fmaf(d[e], (f[e] - m) * r, v[e]) : v[e] + d[e];
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
      };
      add(dw, true);
      add(db, false);
    }
    first = false;
  }
}

// The partial rows' sums: 16 columns a workgroup, dweight's columns first, then dbias's; `first`: the launch's first of those.
__global__ __launch_bounds__(16 * kSumLanes) void layer_sums_kernel(const float* dw, const float* db, int64_t pitch,
                                                                   int count, int64_t cols, float* dweight,
                                                                   float* dbias, int64_t first) {
  const int64_t groups = cols / 16;  // cols is a multiple of 16
  const int64_t block = first + blockIdx.x;
  const bool second = !dw || block >= groups;
  const int64_t c = (block - (dw && second ? groups : 0)) * 16 + (threadIdx.x & 15);
  const float v = column_sum(second ? db : dw, count, pitch, c, true);
  if (threadIdx.x < 16) (second ? dbias : dweight)[c] = v;
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
// Workgroups of the forward: 1024 threads a compute unit, each with a row requested ahead (8192 x 4096 with dropout and
// statistics: 45.5 us, with 768 threads 45.1, with 512 49.7, with 2048 47.6).  With statistics, up to four rows a wavefront or
// workgroup stay in one workgroup, which writes them itself.
int layer_groups(int64_t rows, int64_t octets, bool stats) {
  const int rpb = octets <= 128 ? 4 : 1;
  if (stats && rows <= 4 * rpb) return 1;
  if (octets <= 128) return row_groups(rows, rpb, 4, 0);
  if (octets <= 2048) return row_groups(rows, rpb, 1024 / row_threads(octets), 0);
  return row_groups(rows, rpb, 2, 0);
}

// A row is requested ahead where a workgroup has more than one (8192 x 4096, dropout: 45.5 us against 48.7,
// without dropout 43.2 and 45.8; 1777 x 1040 fp32 with a residual and statistics, a row each: 13.7 and 11.8).  Rows of more than 8192 values need workgroups whose
// registers do not hold another.
template <int XT, int FMT, bool STATS>
void layer_run(const LayerArgs& a, int g, hipStream_t st) {
  const int64_t o = a.cols / 8;
  const dim3 grid((unsigned)g);
  const bool pre = a.rows > (int64_t)g * (o <= 128 ? 4 : 1);
  auto run = [&](auto ahead) {
    constexpr bool PRE = decltype(ahead)::value;
    if (o <= 64) hipLaunchKernelGGL((layernorm_kernel<XT, FMT, STATS, false, 1, PRE>), grid, dim3(256), 0, st, a);
    else if (o <= 128) hipLaunchKernelGGL((layernorm_kernel<XT, FMT, STATS, false, 2, PRE>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((layernorm_kernel<XT, FMT, STATS, true, 2, PRE>), grid, dim3(row_threads(o)), 0, st, a);
  };
  if (o > 2048) hipLaunchKernelGGL((layernorm_long_kernel<XT, FMT, STATS, 1024>), grid, dim3(1024), 0, st, a);
  else if (pre && o <= 1024) run(std::true_type{});
  else run(std::false_type{});
}

template <int XT, int FMT>
void layer_stats(const LayerArgs& a, bool stats, int g, hipStream_t st) {
  if (stats) layer_run<XT, FMT, true>(a, g, st);
  else layer_run<XT, FMT, false>(a, g, st);
}

// Threads of a workgroup of the gradient's kernel: rows of less than 4096 values stand side by side in as many as 512 threads
// hold (bf16 with a residual, 4096 x 2048: 18.3 us, with a row each 21.0; 8192 x 1536: 22.5, 26.2; but 8192 x 4096 with dropout 67.6, 65.9).
int layer_back_threads(int64_t octets) {
  if (octets <= 128) return 256;
  if (octets >= 512) return row_threads(octets);
  return 512 / row_threads(octets) * row_threads(octets);
}

// Its workgroups: one a compute unit, which has a row requested ahead (8192 x 4096 with dropout: 66 us, with two, whose partial
// rows cost more than they gain, 74; with one that requests none ahead 96, with two 71); two of
// four wavefront rows (8192 x 1024: 17.5, with one 17.9, with four 20.9).
int layer_back_groups(int64_t rows, int64_t octets, int64_t slots) {
  const int rpb = octets <= 128 ? 4 : layer_back_threads(octets) / row_threads(octets);
  return row_groups(rows, rpb, octets <= 128 ? 2 : 1, slots);
}

template <int XT>
void layer_back_run(LayerBackArgs a, int g, hipStream_t st) {
  const int64_t o = a.cols / 8;
  const dim3 grid((unsigned)g);
  a.lanes = o <= 128 ? 64 : row_threads(o);
  if (o <= 64) hipLaunchKernelGGL((layernorm_backward_kernel<XT, false, 1, 256, true>), grid, dim3(256), 0, st, a);
  else if (o <= 128) hipLaunchKernelGGL((layernorm_backward_kernel<XT, false, 2, 256, true>), grid, dim3(256), 0, st, a);
  else if (o <= 1024) hipLaunchKernelGGL((layernorm_backward_kernel<XT, true, 2, 512, true>), grid, dim3(layer_back_threads(o)), 0, st, a);
  else if (o <= 2048) hipLaunchKernelGGL((layernorm_backward_kernel<XT, true, 2, 1024, false>), grid, dim3(row_threads(o)), 0, st, a);
  else hipLaunchKernelGGL((layernorm_backward_long_kernel<XT, 1024>), grid, dim3(1024), 0, st, a);
}

}  // namespace

hipError_t launch_layernorm_quantize(const void* x, const void* residual, const void* weight, const void* bias, int xtype,
                                     int64_t rows, int64_t cols, float eps, const Dropout& drop, int fmt,
                                     const float* scale, void* sum_out, uint8_t* q, float* mean, float* rstd,
                                     float* amax, unsigned long long* sat, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream) {
  const bool stats = amax || sat, empty = rows * cols == 0;
  const int g = empty ? 0 : layer_groups(rows, cols / 8, stats);
  const bool gather = stats && g != 1;  // a single workgroup writes the statistics itself
  const bool fits = workspace && workspace_bytes >= (size_t)g * sizeof(uint4);  // a slot for every workgroup, or none
  const LayerArgs a{x, residual, weight, bias, sum_out, q, scale, mean, rstd, reinterpret_cast<uint32_t*>(amax), sat,
                    gather && fits ? reinterpret_cast<uint4*>(workspace) : nullptr, rows, cols, eps, drop};
  if (gather && !a.partials) {
    const hipError_t e = launch_clear_stats(amax, sat, stream);
    if (e != hipSuccess) return e;
  }
  if (!empty) {
    if (xtype == kBF16) {
      if (fmt == kE4M3) layer_stats<kBF16, kE4M3>(a, stats, g, stream);
      else layer_stats<kBF16, kE5M2>(a, stats, g, stream);
    } else {
      if (fmt == kE4M3) layer_stats<kF32, kE4M3>(a, stats, g, stream);
      else layer_stats<kF32, kE5M2>(a, stats, g, stream);
    }
  }
  if (a.partials) return launch_reduce_stats(a.partials, g, amax, sat, stream);
  return hipGetLastError();
}

hipError_t launch_layernorm_backward(const void* dy, const void* h, const float* mean, const float* rstd,
                                     const void* weight, const void* dres, int xtype, int64_t rows, int64_t cols,
                                     const Dropout& drop, void* dx, void* dbranch, float* dweight, float* dbias,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (cols == 0) return hipSuccess;
  const int sums = (dweight ? 1 : 0) + (dbias ? 1 : 0);
  LayerBackArgs a{dy, h, mean, rstd, weight, dres, dx, dbranch, dweight, dbias, 0, rows, cols, drop, 0};
  int g = 0;
  if (rows > 0) {
    g = layer_back_groups(rows, cols / 8, sums ? (int64_t)(workspace_bytes / (sums * cols * sizeof(float))) : 0);
    if (sums && g != 1) {  // a single partial row is the result
      float* ws = reinterpret_cast<float*>(workspace);
      a.pitch = sums * cols;
      a.dw = dweight ? ws : nullptr;
      a.db = dbias ? ws + (dweight ? cols : 0) : nullptr;
    }
    if (xtype == kBF16) layer_back_run<kBF16>(a, g, stream);
    else layer_back_run<kF32>(a, g, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (sums && g != 1) {
    // (a launch has fewer than 2^32 threads)
    const int64_t blocks = sums * (cols / 16), most = int64_t(1) << 21;
    for (int64_t first = 0; first < blocks; first += most)
      hipLaunchKernelGGL(layer_sums_kernel, dim3((unsigned)(blocks - first < most ? blocks - first : most)), dim3(16 * kSumLanes),
                         0, stream, a.dw, a.db, a.pitch, g, cols, dweight, dbias, first);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace fp8mi
