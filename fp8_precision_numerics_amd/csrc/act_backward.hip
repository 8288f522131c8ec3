// Gradients through an activation, cast to FP8 in both orientations.
//
//   fp8_act_backward    d = dy act'(z)                         [M x N]
//   fp8_gated_backward  d = [ dh u act'(g) | dh act(g) ]       [M x 2F], gu = [g | u]
//
//   q = round_to_fp8(d * scale), q_t its transpose (what the weight gradient's
//   GEMM takes as its K-contiguous operand), amax = max |d|, and for the first
//   dbias_n = sum_m d.
//
// HBM-bound: one read of the inputs, one write of each orientation.  Measured on
// MI355X: gated, 8192 x 2 x 16384, 233 us (1.34 GB, 5.8 TB/s); with bias gradient and
// GELU, 4096 x 16384, 77 us (0.40 GB, 5.2 TB/s).  A workgroup
// takes 128 x 128 tiles of d (gated: the gate's and the up projection's tile of
// the same 128 x 128 of dh, so that dh is read once); codes go out row-major
// straight from the registers and column-major through LDS with 4 x 4 byte
// transposes.  A workgroup walks down one strip of 128 columns, so the bias
// gradient's column sums stay in its registers over the strip: one fp32 partial
// row per walk goes to the workspace, added up in a fixed order by
// column_sums_kernel.
#include <type_traits>

#include "activation.hpp"
#include "column_sums.hpp"
#include "launch.hpp"
#include "stats.hpp"
#include "transpose.hpp"

namespace fp8mi {
namespace {

constexpr int kNT = 256;

struct BackArgs {
  const void* dy;        // [M x N] (gated: dh)
  const uint16_t* z;     // [M x N] bf16 (gated: [M x 2N]); null where the activation is none
  const float* scale;
  uint8_t* q;            // may be null
  uint8_t* q_t;          // may be null
  uint32_t* amax_bits;
  unsigned long long* sat;
  uint4* stat_slots;     // one per workgroup, or null
  float* col_partials;   // [walks x N] fp32, or null
  int64_t M, N;
  int walks;             // workgroups per column strip
};

// Eight consecutive values of a row-major matrix as loaded (nontemporal: read once).
template <int XT>
struct Raw8 {
  typedef unsigned int vec4 __attribute__((ext_vector_type(4)));
  vec4 v[XT == kBF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, uint32_t elem) {
    const vec4* src = reinterpret_cast<const vec4*>(reinterpret_cast<const uint8_t*>(p) + elem * (XT == kBF16 ? 2u : 4u));
    v[0] = __builtin_nontemporal_load(src);
    if constexpr (XT == kF32) v[1] = __builtin_nontemporal_load(src + 1);
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (XT == kBF16) return (k & 1) ? bf16_hi(v[0][k >> 1]) : bf16_lo(v[0][k >> 1]);
    else return u2f(v[k >> 2][k & 3]);
  }
};

// Tile 0 of LDS holds the codes of d (gated: of the gate's part), tile 1 those of
// the up projection's part.
template <int XT, int FMT, int ACT, bool GATED, bool STATS>
__global__ __launch_bounds__(kNT, 4) void act_backward_kernel(BackArgs a) {
  constexpr int TILES = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t tile[TILES][kTile * kPitch];
  const int t = threadIdx.x;
  const int vi = t & 15, rr0 = t >> 4;  // the lane's 8 columns and first row (of 16 passes 16 rows apart: 8)
  const int64_t strips = (a.N + kTile - 1) / kTile;
  // Rows that are no multiple of 128 bytes: neighbouring strips share lines, so they go
  // to one XCD (workgroups are dealt to the 8 XCDs in turn), whose L2 reads such a line
  // once and writes it whole (gated 5760 x 2 x 14768: 230 against 248 us).  Whole rows
  // stay dealt out, which spreads them over the channels (2864 x 16320: 56 against 74 us).
  const unsigned xcd = blockIdx.x & 7u, each = gridDim.x >> 3, more = gridDim.x & 7u;
  const unsigned place = (a.N & 63) ? xcd * each + (xcd < more ? xcd : more) + (blockIdx.x >> 3) : blockIdx.x;
  const int64_t strip = place % strips, walk = place / strips;
  const int64_t col0 = strip * kTile, c = col0 + vi * 8;
  const int64_t ldq = GATED ? 2 * a.N : a.N;
  const int64_t row_tiles = (a.M + kTile - 1) / kTile;
  const uint32_t off_n = (uint32_t)(rr0 * a.N + vi * 8), off_q = (uint32_t)(rr0 * ldq + vi * 8);
  const float s = *a.scale;
  LaneStats st;
  float db[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t rt = walk; rt < row_tiles; rt += a.walks) {
    const int64_t row0 = rt * kTile;
    // Pass i covers rows row0 + 16 i + rr0.  Addresses: a uniform base per pass plus the
    // lane's 32-bit offset, the same for every pass.  Four passes' loads are issued
    // before the first is used, held as they were loaded: widened, they took 256
    // registers and left one wave a SIMD (416 us against 233 us for 8192 x 2 x 16384).
    auto passes = [&](int i0, auto whole) {
      Raw8<XT> dy[4];
      Raw8<kBF16> z[4], u[GATED ? 4 : 1];
      auto inside = [&](int i) { return decltype(whole)::value || (row0 + i * 16 + rr0 < a.M && c < a.N); };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t base = row0 + (i0 + i) * 16;
        if (inside(i0 + i)) {
          dy[i].load(reinterpret_cast<const uint8_t*>(a.dy) + (base * a.N + col0) * (XT == kBF16 ? 2 : 4), off_n);
          if constexpr (GATED) {
            z[i].load(a.z + base * ldq + col0, off_q);
            u[i].load(a.z + base * ldq + a.N + col0, off_q);
          } else if constexpr (ACT != kActNone) {
            z[i].load(a.z + base * a.N + col0, off_n);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t base = row0 + (i0 + i) * 16;
        if (inside(i0 + i)) {
          float d[8], e[GATED ? 8 : 1];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float val, slope;
            const float g = dy[i].get(k);
            if constexpr (GATED) {
              act_value_slope<ACT>(z[i].get(k), &val, &slope);
              d[k] = g * u[i].get(k) * slope;
              e[k] = g * val;
            } else if constexpr (ACT != kActNone) {
              act_value_slope<ACT>(z[i].get(k), &val, &slope);
              d[k] = g * slope;
            } else {
              d[k] = g;
            }
            if constexpr (!GATED) db[k] += d[k];
          }
          auto put = [&](const float* f, int h) {
            const uint2 cd = encode8<FMT>(f, s, STATS, STATS && a.sat, st);
            if (a.q) *reinterpret_cast<uint2*>(a.q + base * ldq + h * a.N + col0 + off_q) = cd;
            if (a.q_t) {
              uint32_t* dst = reinterpret_cast<uint32_t*>(tile[h] + ((i0 + i) * 16 + rr0) * kPitch + vi * 8);
              dst[0] = cd.x;
              dst[1] = cd.y;
            }
          };
          put(d, 0);
          if constexpr (GATED) put(e, TILES - 1);
        }
        __builtin_amdgcn_sched_barrier(0);  // one pass's values at a time: mixed, the passes spill
      }
    };
    const bool interior = row0 + kTile <= a.M && col0 + kTile <= a.N;
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += 4) {
      if (interior) passes(i0, std::true_type{});
      else passes(i0, std::false_type{});
    }
    if (a.q_t) {  // M and N are multiples of 16 here
      __syncthreads();
#pragma unroll
      for (int h = 0; h < TILES; ++h)
        transposed_store(tile[h], a.q_t + (int64_t)h * a.N * a.M, a.M, a.N, row0, col0, t);
      __syncthreads();
    }
  }
  if constexpr (!GATED) {
    if (a.col_partials) {
      // the 16 lanes of each column group add up in LDS (the tile's space), in a fixed order
      __syncthreads();
      float* sum = reinterpret_cast<float*>(tile[0]);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[rr0 * kTile + vi * 8 + k] = db[k];
      __syncthreads();
      if (t < kTile && col0 + t < a.N) {
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < 16; ++g) v += sum[g * kTile + t];
        a.col_partials[walk * a.N + col0 + t] = v;
      }
    }
  }
  if constexpr (STATS) block_finish<kNT / 64>(st.amax(), wave_sum_u32(st.sat), a.amax_bits, a.sat, a.stat_slots);
}

// out[n] = sum over the rows of partials [count x cols] (column_sums.hpp).  With statistics'
// slots, one more workgroup (the last) reduces those, which saves a launch (3 us of a small call).
__global__ __launch_bounds__(16 * kSumLanes) void column_sums_kernel(const float* __restrict__ partials, int count,
                                                                    int64_t cols, float* __restrict__ out,
                                                                    const uint4* __restrict__ slots, int nslots,
                                                                    uint32_t* amax_bits, unsigned long long* sat) {
  if (slots && blockIdx.x == gridDim.x - 1) {
    __shared__ uint32_t s_max[kSumLanes / 4];
    __shared__ unsigned long long s_cnt[kSumLanes / 4];
    uint32_t m = 0u;
    unsigned long long c = 0ull;
    for (int i = threadIdx.x; i < nslots; i += 16 * kSumLanes) {
      const uint4 p = slots[i];
      m = m > p.x ? m : p.x;
      c += (unsigned long long)p.z | ((unsigned long long)p.w << 32);
    }
    m = wave_max_u32(m);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) c += __shfl_xor(c, off, 64);
    if ((threadIdx.x & 63) == 0) {
      s_max[threadIdx.x >> 6] = m;
      s_cnt[threadIdx.x >> 6] = c;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kSumLanes / 4; ++w) {
        m = m > s_max[w] ? m : s_max[w];
        c += s_cnt[w];
      }
      if (amax_bits) *amax_bits = m;
      if (sat) *sat = c;
    }
    return;
  }
  const int64_t c = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
  const float v = column_sum(partials, count, cols, c, c < cols);
  if (threadIdx.x < 16 && c < cols) out[c] = v;
}

template <int XT, int FMT, int ACT, bool GATED>
void back_run(const BackArgs& a, bool stats, unsigned grid, hipStream_t st) {
  if (stats) hipLaunchKernelGGL((act_backward_kernel<XT, FMT, ACT, GATED, true>), dim3(grid), dim3(kNT), 0, st, a);
  else hipLaunchKernelGGL((act_backward_kernel<XT, FMT, ACT, GATED, false>), dim3(grid), dim3(kNT), 0, st, a);
}

template <int XT, int FMT, bool GATED>
void back_act(const BackArgs& a, int act, bool stats, unsigned grid, hipStream_t st) {
  if (act == kActRelu) back_run<XT, FMT, kActRelu, GATED>(a, stats, grid, st);
  else if (act == kActSilu) back_run<XT, FMT, kActSilu, GATED>(a, stats, grid, st);
  else if (act == kActGelu) back_run<XT, FMT, kActGelu, GATED>(a, stats, grid, st);
  else back_run<XT, FMT, kActNone, GATED>(a, stats, grid, st);
}

template <bool GATED>
hipError_t back_launch(BackArgs a, int xtype, int fmt, int act, float* dbias, float* amax, void* workspace,
                       size_t workspace_bytes, hipStream_t st) {
  const bool stats = amax || a.sat;
  const int64_t strips = (a.N + kTile - 1) / kTile, row_tiles = (a.M + kTile - 1) / kTile;
  const bool empty = a.M * a.N == 0;
  // As many walks a strip as fill the device with 8 workgroups a compute unit.
  int64_t walks = empty ? 0 : persistent_groups(8) / strips;
  if (!empty) walks = walks < 1 ? 1 : (walks > row_tiles ? row_tiles : walks);
  // The workspace holds the bias gradient's partial rows (a single one goes straight to
  // dbias), then the statistics' slots.
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  if (dbias && !empty) {
    const int64_t fit = (int64_t)(workspace_bytes / (a.N * sizeof(float)));  // >= 1: checked by the entry point
    if (walks > fit) walks = fit;
    a.col_partials = walks == 1 ? dbias : reinterpret_cast<float*>(ws);
    const size_t used = walks == 1 ? 0 : ((size_t)walks * a.N * sizeof(float) + 15) & ~size_t(15);
    ws = used < workspace_bytes ? ws + used : nullptr;
    workspace_bytes = ws ? workspace_bytes - used : 0;
  }
  const int64_t groups = walks * strips;
  const bool gather = stats && groups != 1;  // a single workgroup writes the statistics itself
  if (gather && ws && workspace_bytes >= (size_t)groups * sizeof(uint4)) a.stat_slots = reinterpret_cast<uint4*>(ws);
  if (gather && !a.stat_slots) {
    const hipError_t e = launch_clear_stats(amax, a.sat, st);
    if (e != hipSuccess) return e;
  }
  a.walks = (int)walks;
  if (!empty) {
    if (xtype == kBF16) {
      if (fmt == kE4M3) back_act<kBF16, kE4M3, GATED>(a, act, stats, (unsigned)groups, st);
      else back_act<kBF16, kE5M2, GATED>(a, act, stats, (unsigned)groups, st);
    } else {
      if (fmt == kE4M3) back_act<kF32, kE4M3, GATED>(a, act, stats, (unsigned)groups, st);
      else back_act<kF32, kE5M2, GATED>(a, act, stats, (unsigned)groups, st);
    }
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dbias && walks != 1)
    return launch_column_sums(a.col_partials, (int)walks, a.N, dbias, a.stat_slots, (int)groups, amax, a.sat, st);
  if (a.stat_slots) return launch_reduce_stats(a.stat_slots, (int)groups, amax, a.sat, st);
  return hipSuccess;
}

}  // namespace

hipError_t launch_column_sums(const float* partials, int count, int64_t cols, float* out, const void* slots, int nslots,
                              float* amax, unsigned long long* sat, hipStream_t stream) {
  const unsigned groups = (unsigned)((cols + 15) / 16) + (slots ? 1u : 0u);
  if (groups == 0) return hipSuccess;
  hipLaunchKernelGGL(column_sums_kernel, dim3(groups), dim3(16 * kSumLanes), 0, stream, partials, count, cols, out,
                     reinterpret_cast<const uint4*>(slots), nslots, reinterpret_cast<uint32_t*>(amax), sat);
  return hipGetLastError();
}

hipError_t launch_act_backward(const void* dy, int xtype, const uint16_t* z, int act, int64_t M, int64_t N, int fmt,
                               const float* scale, uint8_t* q, uint8_t* q_t, float* dbias, float* amax,
                               unsigned long long* sat, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const BackArgs a{dy, z, scale, q, q_t, reinterpret_cast<uint32_t*>(amax), sat, nullptr, nullptr, M, N, 0};
  return back_launch<false>(a, xtype, fmt, act, dbias, amax, workspace, workspace_bytes, stream);
}

hipError_t launch_gated_backward(const void* dh, int xtype, const uint16_t* gu, int act, int64_t M, int64_t F, int fmt,
                                 const float* scale, uint8_t* q, uint8_t* q_t, float* amax, unsigned long long* sat,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const BackArgs a{dh, gu, scale, q, q_t, reinterpret_cast<uint32_t*>(amax), sat, nullptr, nullptr, M, F, 0};
  return back_launch<true>(a, xtype, fmt, act, nullptr, amax, workspace, workspace_bytes, stream);
}

}  // namespace fp8mi
