// The amax (as fp32 bits) and saturation count of an FP8 output, gathered over
// a grid: lanes to workgroup here, workgroups to the outputs either through one
// 16-byte partial per workgroup, reduced afterwards by reduce_partials_kernel
// (quantize.hip), or by device-scope atomics.  Both are a maximum and an integer
// sum, so the result does not depend on the order.
#pragma once

#include "device_common.hpp"

namespace fp8mi {

// Fold (per-lane amax bits, per-wave saturation count) into the global outputs:
// either one partial per workgroup (`partials` non-null: slot blockIdx.x gets
// {amax bits, 0, count lo, count hi}, reduced afterwards by
// reduce_partials_kernel) or device-scope atomics on the outputs.  The atomics
// on one address are serialised across the chip (about 4 ns each on MI355X,
// ~4 us for a 512-workgroup grid); the partials cost one tiny extra kernel.
template <int MAX_WAVES = 16>
__device__ __forceinline__ void block_finish(uint32_t amx, uint32_t wave_cnt, uint32_t* amax_bits,
                                             unsigned long long* sat, uint4* partials) {
  __shared__ uint32_t s_max[MAX_WAVES];
  __shared__ uint32_t s_cnt[MAX_WAVES];
  amx = wave_max_u32(amx);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;  // at most MAX_WAVES of them
  if (lane == 0) {
    s_max[wave] = amx;
    s_cnt[wave] = wave_cnt;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t m = s_max[0];
    unsigned long long c = s_cnt[0];
    const int waves = MAX_WAVES < (int)(blockDim.x >> 6) ? MAX_WAVES : (int)(blockDim.x >> 6);
    for (int w = 1; w < waves; ++w) {
      m = m > s_max[w] ? m : s_max[w];
      c += s_cnt[w];
    }
    if (partials) {
      partials[blockIdx.x] = make_uint4(m, 0u, (uint32_t)c, (uint32_t)(c >> 32));
    } else if (gridDim.x == 1) {  // the only one: no clearing needed beforehand
      if (amax_bits) *amax_bits = m;
      if (sat) *sat = c;
    } else {
      // The output only grows, so an older value of it is a safe bound: the atomic is
      // skipped where it would change nothing.
      if (amax_bits && m > __hip_atomic_load(amax_bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
        atomicMax(amax_bits, m);
      if (sat && c) atomicAdd(sat, c);
    }
  }
}

// One lane's running amax and saturation count over the values it encodes.
struct LaneStats {
  float max = 0.0f;  // IEEE maximum of |y|: a NaN stays
  uint32_t sat = 0u;
  // Non-negative floats order as their bit patterns, NaN above Inf.
  __device__ __forceinline__ uint32_t amax() const { return f2u(max) & 0x7FFFFFFFu; }
};

// Codes of eight values y times `scale` (byte i of the pair = value i); max |y| and the
// count of |y * scale| > max are folded into `st` where asked for.
// The eight magnitudes' maximum (V_MAXIMUM3_F32, which keeps a NaN) decides the way:
// rounding is monotone, so where fp32(max |y| * scale) <= max no product saturates and
// none is NaN, and the conversion instruction alone is the rule.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* y, float scale, bool amax, bool sat, LaneStats& st) {
  float m = __builtin_elementwise_maximum(__builtin_fabsf(y[0]), __builtin_fabsf(y[1]));
#pragma unroll
  for (int e = 2; e < 8; e += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(y[e]), __builtin_fabsf(y[e + 1])), m);
  if (amax) st.max = __builtin_elementwise_maximum(st.max, m);
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = y[e] * scale;
  uint2 c;
  if (__builtin_expect(__builtin_fabsf(m * scale) <= Fp8Traits<FMT>::max_value, 1)) {
    c.x = cvt_pk<FMT, true>(p[2], p[3], cvt_pk<FMT, false>(p[0], p[1], 0u));
    c.y = cvt_pk<FMT, true>(p[6], p[7], cvt_pk<FMT, false>(p[4], p[5], 0u));
  } else {
    c.x = encode4<FMT>(p[0], p[1], p[2], p[3]);
    c.y = encode4<FMT>(p[4], p[5], p[6], p[7]);
    if (sat) {
#pragma unroll
      for (int e = 0; e < 8; ++e) st.sat += __builtin_fabsf(p[e]) > Fp8Traits<FMT>::max_value ? 1u : 0u;
    }
  }
  return c;
}

}  // namespace fp8mi
