// The gradient products of the vocabulary's cross entropy: the dense kernel
// (gemm_kernel.hpp) on a first operand whose rows are padded with zeros to whole steps, so that the
// number of tokens and of the vocabulary's columns, which are their K, may be any and no step
// is loaded in another way, with the fp32 sum of earlier pieces added in the epilogue.
// Bound by the matrix cores from some 1000 rows on: 8192 x 4096 x 16384 on the FP8 cores 412 us (2.67 PFLOP/s), the cores 63 % busy by the counters, LDS reads of the
// transposed operand 40 % in conflict.
#include "gemm_few_rows.hpp"
#include "gemm_epi_dispatch.hpp"
#include "launch.hpp"
#include "vocab.hpp"

namespace fp8mi {
namespace {

constexpr int64_t kShortK = 4 * kBK;

template <int FA, int FB, int MODE>
hipError_t product_shape(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa, const float* sb,
                         const ProductEpi& epi, size_t workspace_bytes, hipStream_t st) {
  TileChoice c = choose_tile(M, N, K, MODE == kAccumMfma8, workspace_bytes, persistent_groups(1));
  // A K of up to four steps is over soon after its output begins to be written: smaller tiles, several workgroups a compute unit, store
  // and load side by side, which the estimate does not know; and on the FP8 cores, whose steps are half as long, the traffic of 128 x 128 tiles
  // shows from three steps on, where there are rounds enough of the large ones to hide their ends.  dw with the logits before it, in us on
  // 64 x 128, 128 x 128 and 256 x 256 tiles, all of one run (65536 x 4096: 16 rounds of 256 x 256 tiles on 256 compute units; 32000 x 4096: 7.8;
  // 50021 x 2048: 6.1; 50021 x 1024: 3.1):
  //   exact      rows   65536 x 4096    32000 x 4096    50021 x 2048    50021 x 1024
  //                64   222 218 225     115 115 121      89  92  96      52  54  59
  //               200   328 311 314     174 167 171     139 134 142      80  80  88
  //               300   458 437 437     248 237 241     195 186 195     108 105 114
  //               500   549 512 511     277 260 262     240 228 234     135 132 142
  //   FP8 cores    64   176 180 188     102 106 111      77  83  86      46  49  53
  //               200   236 227 226     131 127 129     103 105 108      63  64  68
  //               300   315 300 291     162 154 154     152 152 154      91  91  95
  //               500   367 347 335     188 178 176     166 161 161     101  99 102
  if (K <= kShortK && c.split == 1) {
    const bool rounds = ((M + 255) / 256) * ((N + 255) / 256) > 7 * (int64_t)persistent_groups(1);
    c.shape = K <= kBK ? 2 : MODE == kAccumMfma8 && K > 2 * kBK && rounds ? 0 : 1;
  }
  if (c.shape == 0) {
    if constexpr (MODE == kAccumExact) return epi_run<256, 256, 2, 4, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
    else return epi_run<256, 256, 4, 2, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
  }
  if (c.shape == 1) return epi_run<128, 128, 2, 2, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
  if (c.shape == 2) return epi_run<64, 128, 2, 2, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
  return epi_run<64, 128, 2, 2, FA, FB, MODE, ProductEpi, 3, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
}

template <int MODE>
hipError_t product_fmt(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K, const float* sa,
                       const float* sb, const ProductEpi& epi, size_t workspace_bytes, hipStream_t st) {
  if (fa == kE4M3 && fb == kE4M3) return product_shape<kE4M3, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  if (fa == kE5M2 && fb == kE4M3) return product_shape<kE5M2, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  if (fa == kE4M3 && fb == kE5M2) return product_shape<kE4M3, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  return product_shape<kE5M2, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
}

}  // namespace

hipError_t launch_vocab_product(const uint8_t* A, int64_t lda, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const float* add, void* y, int ytype, int accum,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ProductEpi epi{};
  epi.act = kActNone;
  epi.out = ytype;
  epi.partials = reinterpret_cast<float*>(workspace);
  epi.split = 1;
  epi.lda = (int)lda;
  auto rows = [&](int64_t from, int64_t count) {
    epi.y = reinterpret_cast<uint8_t*>(y) + from * N * (ytype == kF32 ? 4 : 2);
    epi.add = add ? add + from * N : nullptr;
    const uint8_t* a = A + from * lda;
    if (accum == kAccumMfma8) return product_fmt<kAccumMfma8>(a, fa, B, fb, count, N, K, sinv_a, sinv_b, epi, workspace_bytes, stream);
    return product_fmt<kAccumExact>(a, fa, B, fb, count, N, K, sinv_a, sinv_b, epi, workspace_bytes, stream);
  };
  // The rows may be cut (the large tiles are square, so the sides may be named in either order).
  const int64_t first = K <= kShortK ? M : plan_rounds(N, M, K, accum == kAccumMfma8, workspace_bytes, persistent_groups(1)).first;
  const hipError_t e = rows(0, first);
  return e != hipSuccess || first == M ? e : rows(first, M - first);
}

}  // namespace fp8mi
