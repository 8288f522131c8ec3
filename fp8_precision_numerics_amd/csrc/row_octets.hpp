// What the row norms (rms_norm.hip, layer_norm.hip) share: a row of values in
// groups of eight ("octets") over the lanes of a wavefront or of a workgroup.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace fp8mi {

// Eight consecutive values as loaded: one 16-B vector (bf16) or two (fp32).
template <int XT>
struct Octet {
  typedef unsigned int vec4 __attribute__((ext_vector_type(4)));
  static constexpr int NV = XT == kBF16 ? 1 : 2;
  uint4 v[NV];
  __device__ __forceinline__ void load(const void* p, int64_t octet) {
    const uint4* src = reinterpret_cast<const uint4*>(p) + octet * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = src[i];
  }
  // Data that is read once, streamed past the caches.
  __device__ __forceinline__ void load_nt(const void* p, int64_t octet) {
    const vec4* src = reinterpret_cast<const vec4*>(p) + octet * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const vec4 r = __builtin_nontemporal_load(src + i);
      v[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t octet) const {
    uint4* dst = reinterpret_cast<uint4*>(p) + octet * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) dst[i] = v[i];
  }
  __device__ __forceinline__ void store_nt(void* p, int64_t octet) const {
    vec4* dst = reinterpret_cast<vec4*>(p) + octet * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) __builtin_nontemporal_store((vec4){v[i].x, v[i].y, v[i].z, v[i].w}, dst + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void widen(float* f) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (XT == kBF16) {
          f[2 * k] = bf16_lo(w[k]);
          f[2 * k + 1] = bf16_hi(w[k]);
        } else {
          f[4 * i + k] = u2f(w[k]);
        }
      }
    }
  }
  // Rounded to the nearest value of the type (ties to even).
  __device__ __forceinline__ void narrow(const float* f) {
    if constexpr (XT == kBF16) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * k], f[2 * k + 1]}, v2bf));
      v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      v[0] = make_uint4(f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3]));
      v[1] = make_uint4(f2u(f[4]), f2u(f[5]), f2u(f[6]), f2u(f[7]));
    }
  }
};

// Sum over the lanes of a row; every lane gets it.  WG: the row is the whole
// workgroup's: through LDS, in two buffers used in turn, so that one barrier a row
// is enough (a wave that is a row ahead writes the other buffer).  Otherwise it is
// one wave's.
constexpr int kMaxWaves = 16;
template <bool WG>
__device__ __forceinline__ float row_sum(float v, float (*buf)[kMaxWaves], int turn) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if constexpr (WG) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[turn & 1][threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[turn & 1][0];
    for (int w = 1; w < waves; ++w) v += buf[turn & 1][w];
  }
  return v;
}

// Workgroups for `rows` rows, `rpb` at a time, at most `per_cu` per compute unit
// and (with one slot each) no more than there are slots.
inline int row_groups(int64_t rows, int rpb, int per_cu, int64_t slots) {
  int64_t g = (rows + rpb - 1) / rpb;
  const int cap = persistent_groups(per_cu);
  if (g > cap) g = cap;
  if (slots > 0 && g > slots) g = slots;
  return g < 1 ? 1 : (int)g;
}

// Threads of a workgroup that holds a row in two octets a thread.
inline int row_threads(int64_t octets) { return (int)((octets + 127) / 128 * 64); }

}  // namespace fp8mi
