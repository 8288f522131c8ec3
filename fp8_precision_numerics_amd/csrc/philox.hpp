// Dropout from a counter-based generator: no mask is stored, the backward pass
// draws the same bits again.
//
// The generator is Philox4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011): a bijection of a
// 128-bit counter under a 64-bit key, two 32 x 32 -> 64 bit products a round.  The
// key is the seed, the counter's upper half the offset, its lower half the number of
// an octet (eight consecutive values of the tensor, flat).  Each value of the octet
// takes 16 of the 128 bits, so a call of 10 rounds serves eight values: with 32 bits
// a value the draws would take twice the instructions, while a probability in
// steps of 2^-16 is off by at most 8e-6; kept values are divided by the
// probability that is really used, so the expectation is exact.
#pragma once

#include "device_common.hpp"

namespace fp8mi {

__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint2 k) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k.x, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k.y, (uint32_t)a);
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

// Host argument: a value is dropped where its 16 bits are below `cut` (0: no dropout), and
// multiplied with `scale` = 65536 / (65536 - cut) otherwise.
struct Dropout {
  const unsigned long long* rng;  // device: {seed, offset}
  uint32_t cut;
  float scale;
};

// The same with the seed and the offset read.
struct Dropper {
  uint2 seed, offset;
  uint32_t cut;
  float scale;
  __device__ __forceinline__ explicit Dropper(const Dropout& d) : cut(d.cut), scale(d.scale) {
    seed = offset = make_uint2(0u, 0u);
    if (cut) {
      const unsigned long long s = d.rng[0], o = d.rng[1];
      seed = make_uint2((uint32_t)s, (uint32_t)(s >> 32));
      offset = make_uint2((uint32_t)o, (uint32_t)(o >> 32));
    }
  }
  // The eight values of octet `g`: kept ones scaled, dropped ones 0 whatever they were.
  __device__ __forceinline__ void apply(float* f, int64_t g) const {
    const uint4 r = philox4x32_10(make_uint4((uint32_t)g, (uint32_t)((uint64_t)g >> 32), offset.x, offset.y), seed);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = ((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) < cut ? 0.0f : f[e] * scale;
  }
};

}  // namespace fp8mi
