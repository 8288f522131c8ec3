// The feed-forward GEMMs for few rows (decoding): M up to 64.
//
// Bound by the weights' bytes: every code of B is read once and contracted with
// all rows of A at once, so the kernel is a stream over B.  A workgroup of 8
// wavefronts takes 16 output columns (gated: the 16 gate rows and the 16 up rows
// of B) over the whole K: K steps of 128 are dealt to the waves in turn, each
// wave keeps U steps of B in flight (2 KiB a step and 16 rows, straight from HBM
// to registers: no other wave needs them), and A's codes come from L2.  The
// waves' partial sums meet in LDS, and the epilogue follows there.
//
// Both accumulation modes use the exact arithmetic here (codes widened to bf16,
// V_MFMA_F32_16X16X32_BF16, fp32 sums): the widening hides behind the stream.
//
// Operand lanes of 16x16x32: lane l supplies row l % 16 and eight K values; any
// assignment of K values works as long as both operands use the same one, so
// lane group l / 16 takes the 32-byte slice l / 16 of a 128-byte step and
// sub-step s its bytes [8s, 8s + 8).  B goes first, so lane l holds row l % 16 of
// A and columns 4 (l / 16) .. + 3.
#include "gemm_few_rows.hpp"
#include "gemm_tile.hpp"

namespace fp8mi {
namespace {

constexpr int kWavesFew = 8;

struct Slice {
  uint4 v[2];  // 32 bytes of K
};

__device__ __forceinline__ Slice load_slice(const uint8_t* p) {
  Slice s;
  s.v[0] = reinterpret_cast<const uint4*>(p)[0];
  s.v[1] = reinterpret_cast<const uint4*>(p)[1];
  return s;
}
// The ragged last step: `left` bytes of K remain at p (K is a multiple of 16).
__device__ __forceinline__ Slice load_slice_tail(const uint8_t* p, int left) {
  Slice s;
  s.v[0] = s.v[1] = make_uint4(0u, 0u, 0u, 0u);
  if (left > 0) s.v[0] = reinterpret_cast<const uint4*>(p)[0];
  if (left > 16) s.v[1] = reinterpret_cast<const uint4*>(p)[1];
  return s;
}

template <int F>
__device__ __forceinline__ v8bf widen_part(const Slice& s, int i) {
  const uint4 g = s.v[i >> 1];
  return (i & 1) ? widen8_scaled_bf16<F>(g.z, g.w, 1.0f) : widen8_scaled_bf16<F>(g.x, g.y, 1.0f);
}

template <int MB, int U, int FA, int FB, bool GATED>
__global__ __launch_bounds__(64 * kWavesFew) void gemm_few_rows_kernel(const uint8_t* __restrict__ A,
                                                                      const uint8_t* __restrict__ B, int M, int N,
                                                                      int K, const float* __restrict__ sinv_a,
                                                                      const float* __restrict__ sinv_b, EpiArgs epi) {
  constexpr int NB = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float red[kWavesFew][NB][MB * 16][16];
  const int lane = threadIdx.x & 63, rl = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  // Rows past the edge repeat the last one: they only feed outputs that are not stored.
  const int64_t nrow = n0 + rl < N ? n0 + rl : N - 1;
  const uint8_t* bp[NB];
  bp[0] = B + nrow * K + kq * 32;
  if constexpr (GATED) bp[1] = B + (nrow + N) * K + kq * 32;
  const uint8_t* ap[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = i * 16 + rl;
    ap[i] = A + (int64_t)(m < M ? m : M - 1) * K + kq * 32;
  }
  v4f acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = (v4f){0.f, 0.f, 0.f, 0.f};

  auto contract = [&](const Slice* b, const Slice* a) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v8bf bh[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) bh[j] = widen_part<FB>(b[j], s);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const v8bf ah = widen_part<FA>(a[i], s);
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bh[j], ah, acc[j][i], 0, 0, 0);
      }
    }
  };

  const int full = K / kBK;
  int s = w;
  for (; s + (U - 1) * kWavesFew < full; s += U * kWavesFew) {
    Slice b[U][NB], a[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (int64_t)(s + u * kWavesFew) * kBK;
#pragma unroll
      for (int j = 0; j < NB; ++j) b[u][j] = load_slice(bp[j] + k);
#pragma unroll
      for (int i = 0; i < MB; ++i) a[u][i] = load_slice(ap[i] + k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) contract(b[u], a[u]);
  }
  for (; s * kBK < K; s += kWavesFew) {
    const int64_t k = (int64_t)s * kBK;
    const int left = K - (int)k - kq * 32;
    Slice b[NB], a[MB];
#pragma unroll
    for (int j = 0; j < NB; ++j) b[j] = load_slice_tail(bp[j] + k, left);
#pragma unroll
    for (int i = 0; i < MB; ++i) a[i] = load_slice_tail(ap[i] + k, left);
    contract(b, a);
  }

#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) *reinterpret_cast<v4f*>(&red[w][j][i * 16 + rl][4 * kq]) = acc[j][i];
  __syncthreads();

  // 8 columns a thread: rows 0 .. 16 MB - 1, two chunks each.
  const int t = threadIdx.x;
  if (t >= (MB > 1 ? MB * 32 : 64)) return;  // whole waves (MB = 1: the second half of one has no row)
  const int m = t >> 1;
  const int64_t n = n0 + (t & 1) * 8;
  const int left = n < N ? (int)(N - n < 8 ? N - n : 8) : 0;
  const bool vec = (N & 7) == 0;
  LaneStats st;
  if (m < M && left) {
    const float sc = sinv_a[0] * sinv_b[0];
    float v[NB][8], bias[8], res[8];
    uint4 bb = make_uint4(0u, 0u, 0u, 0u), rr = bb;
    if constexpr (!GATED) {
      if (epi.bias) bb = load_bf16x8(epi.bias + n, vec, left);
      if (epi.residual) rr = load_bf16x8(epi.residual + (int64_t)m * N + n, vec, left);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
#pragma unroll
      for (int q = 0; q < kWavesFew; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4f p = *reinterpret_cast<const v4f*>(&red[q][j][m][(t & 1) * 8 + 4 * h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][4 * h + e] += p[e];
        }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= sc;
    }
    unpack_bf16x8(bb, bias);
    unpack_bf16x8(rr, res);
    const float scale = (epi.out == kYE4M3 || epi.out == kYE5M2) ? *epi.out_scale : 1.0f;
    epilogue8<GATED>(epi, v[0], v[NB - 1], bias, res, m, n, N, vec, left, scale, st);
  }
  if (epi.amax_bits || epi.sat) publish_epilogue_stats(epi, st, 0u, threadIdx.x & 63);
}

template <int FA, int FB, bool GATED>
hipError_t few_run(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                   const float* sb, const EpiArgs& epi, hipStream_t st) {
  const dim3 grid((unsigned)((N + 15) / 16)), block(64 * kWavesFew);
  if (M <= 16)
    hipLaunchKernelGGL((gemm_few_rows_kernel<1, 4, FA, FB, GATED>), grid, block, 0, st, A, B, (int)M, (int)N, (int)K, sa, sb, epi);
  else if (M <= 32)
    hipLaunchKernelGGL((gemm_few_rows_kernel<2, 2, FA, FB, GATED>), grid, block, 0, st, A, B, (int)M, (int)N, (int)K, sa, sb, epi);
  else
    hipLaunchKernelGGL((gemm_few_rows_kernel<4, 2, FA, FB, GATED>), grid, block, 0, st, A, B, (int)M, (int)N, (int)K, sa, sb, epi);
  return hipGetLastError();
}

template <bool GATED>
hipError_t few_fmt(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                   const float* sa, const float* sb, const EpiArgs& epi, hipStream_t st) {
  if (fa == kE4M3 && fb == kE4M3) return few_run<kE4M3, kE4M3, GATED>(A, B, M, N, K, sa, sb, epi, st);
  if (fa == kE5M2 && fb == kE4M3) return few_run<kE5M2, kE4M3, GATED>(A, B, M, N, K, sa, sb, epi, st);
  if (fa == kE4M3 && fb == kE5M2) return few_run<kE4M3, kE5M2, GATED>(A, B, M, N, K, sa, sb, epi, st);
  return few_run<kE5M2, kE5M2, GATED>(A, B, M, N, K, sa, sb, epi, st);
}

}  // namespace

hipError_t launch_gemm_few_rows(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const EpiArgs& epi, bool gated,
                                hipStream_t stream) {
  if (gated) return few_fmt<true>(A, fa, B, fb, M, N, K, sinv_a, sinv_b, epi, stream);
  return few_fmt<false>(A, fa, B, fb, M, N, K, sinv_a, sinv_b, epi, stream);
}

}  // namespace fp8mi
