// The feed-forward GEMMs for few rows (decoding): M up to 16.
//
// Bound by the weights' bytes: every code of B is read once and contracted with
// all rows of A at once, so the kernel is a stream over B.  A tile is 16 output
// columns (gated: the 16 gate rows and the 16 up rows of B); `split` waves of a
// workgroup of 8 share a tile's K, in chunks of U steps of 128 dealt to them in
// turn, and a workgroup takes 8 / split tiles.  A wave requests its next chunk
// before it contracts the present one (straight from HBM to registers: no other
// wave needs it); A's codes come from L2.  The waves' partial sums meet in LDS,
// and the epilogue follows there.
//
// Each tile begins its K at another chunk (the tile's number, round the end): rows
// of B are often a power of two apart, and with every wave of the chip at the same
// K their reads fell on few of the memory's channels.  Measured on MI355X, cold
// weights: gated 2 x 16384 x 4096, 8 rows, 24.0 us (5.6 TB/s) against 28.5 us
// without the turn; 4096 x 16384 16.1 against 19.3 us (14.9 us in a run of its own); a plain
// read of the same bytes takes 21.5 and 11.4 us.  Waves: a split that gives the chip about 2048
// waves (8 a compute unit) is best; with 1 wave a tile 41.3 us, with 8 33.3 us,
// with 2 28.2 us (gated shape, before the turn).
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
#include "launch.hpp"

namespace fp8mi {
namespace {

constexpr int kWavesFew = 8;

// Bytes [16 i, 16 i + 16) and [64 + 16 i, 64 + 16 i + 16) of a 128-byte K step (i: lane
// group), so that the four lanes of a row read 64 contiguous bytes.
struct Slice {
  uint4 v[2];
};

__device__ __forceinline__ Slice load_slice(const uint8_t* p) {
  Slice s;
  s.v[0] = reinterpret_cast<const uint4*>(p)[0];
  s.v[1] = reinterpret_cast<const uint4*>(p)[4];
  return s;
}
// The ragged last step: `left` bytes of K remain at p (K is a multiple of 16).
__device__ __forceinline__ Slice load_slice_tail(const uint8_t* p, int left) {
  Slice s;
  s.v[0] = s.v[1] = make_uint4(0u, 0u, 0u, 0u);
  if (left > 0) s.v[0] = reinterpret_cast<const uint4*>(p)[0];
  if (left > 64) s.v[1] = reinterpret_cast<const uint4*>(p)[4];
  return s;
}

template <int F>
__device__ __forceinline__ v8bf widen_part(const Slice& s, int i) {
  const uint4 g = s.v[i >> 1];
  return (i & 1) ? widen8_scaled_bf16<F>(g.z, g.w, 1.0f) : widen8_scaled_bf16<F>(g.x, g.y, 1.0f);
}

template <int FA, int FB, bool GATED>
__global__ __launch_bounds__(64 * kWavesFew) void gemm_few_rows_kernel(const uint8_t* __restrict__ A,
                                                                      const uint8_t* __restrict__ B, int M, int N,
                                                                      int K, const float* __restrict__ sinv_a,
                                                                      const float* __restrict__ sinv_b, EpiArgs epi,
                                                                      int split) {
  constexpr int NW = kWavesFew;
  constexpr int NB = GATED ? 2 : 1;
  constexpr int U = 2;
  __shared__ __attribute__((aligned(16))) float red[NW][NB][16][16];
  const int lane = threadIdx.x & 63, rl = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_wg = NW / split, part = w & (split - 1);
  const int64_t tile = (int64_t)blockIdx.x * tiles_wg + w / split;
  const int64_t n0 = tile * 16;
  // Rows past the edge repeat the last one: they only feed outputs that are not stored.
  const int64_t nrow = n0 + rl < N ? n0 + rl : N - 1;
  const uint8_t* bp[NB];
  bp[0] = B + nrow * K + kq * 16;
  if constexpr (GATED) bp[1] = B + (nrow + N) * K + kq * 16;
  const uint8_t* ap = A + (int64_t)(rl < M ? rl : M - 1) * K + kq * 16;
  v4f acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = (v4f){0.f, 0.f, 0.f, 0.f};

  auto contract = [&](const Slice* b, const Slice& a) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const v8bf ah = widen_part<FA>(a, s);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_part<FB>(b[j], s), ah, acc[j], 0, 0, 0);
    }
  };

  const int chunks = K / (U * kBK);
  struct Chunk {
    Slice b[U][NB], a[U];
  };
  const int first = chunks > 0 ? (int)(tile % chunks) : 0;
  auto fetch = [&](Chunk& f, int c) {
    c += first;
    const int64_t k = (int64_t)(c < chunks ? c : c - chunks) * (U * kBK);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < NB; ++j) f.b[u][j] = load_slice(bp[j] + k + u * kBK);
      f.a[u] = load_slice(ap + k + u * kBK);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto use = [&](const Chunk& f) {
#pragma unroll
    for (int u = 0; u < U; ++u) contract(f.b[u], f.a[u]);
    __builtin_amdgcn_sched_barrier(0);
  };
  Chunk f0, f1;
  int c = part;
  if (c < chunks) fetch(f0, c);
  while (c < chunks) {
    if (c + split < chunks) fetch(f1, c + split);
    use(f0);
    c += split;
    if (c >= chunks) break;
    if (c + split < chunks) fetch(f0, c + split);
    use(f1);
    c += split;
  }
  // The steps that fill no chunk, one a wave in turn, the last of them ragged.
  for (int s = chunks * U + part; s * kBK < K; s += split) {
    const int64_t k = (int64_t)s * kBK;
    const int left = K - (int)k - kq * 16;
    Slice b[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) b[j] = load_slice_tail(bp[j] + k, left);
    contract(b, load_slice_tail(ap + k, left));
  }

#pragma unroll
  for (int j = 0; j < NB; ++j) *reinterpret_cast<v4f*>(&red[w][j][rl][4 * kq]) = acc[j];
  __syncthreads();

  // 8 columns a thread: of each tile, 16 rows of two chunks.
  LaneStats st;
  for (int t = threadIdx.x; t < tiles_wg * 32; t += 64 * NW) {
    const int slot = t / 32, m = (t >> 1) & 15;
    const int64_t n = ((int64_t)blockIdx.x * tiles_wg + slot) * 16 + (t & 1) * 8;
    const int left = n < N ? (int)(N - n < 8 ? N - n : 8) : 0;
    const bool vec = (N & 7) == 0;
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
        for (int q = slot * split; q < (slot + 1) * split; ++q)
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
  }
  if (epi.amax_bits || epi.sat) publish_epilogue_stats(epi, st, reinterpret_cast<uint32_t*>(red));
}

template <int FA, int FB, bool GATED>
hipError_t few_run(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                   const float* sb, const EpiArgs& epi, hipStream_t st) {
  const int64_t tiles = (N + 15) / 16;
  int split = 1;
  while (split < kWavesFew && tiles * split < persistent_groups(8)) split *= 2;
  const int tiles_wg = kWavesFew / split;
  hipLaunchKernelGGL((gemm_few_rows_kernel<FA, FB, GATED>), dim3((unsigned)((tiles + tiles_wg - 1) / tiles_wg)),
                     dim3(64 * kWavesFew), 0, st, A, B, (int)M, (int)N, (int)K, sa, sb, epi, split);
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
