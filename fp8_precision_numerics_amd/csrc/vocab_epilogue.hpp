// What becomes of a tile of logits z = (A B^T) sinv_a sinv_b, so that no logit is
// ever stored: the loss keeps two numbers a row and tile, the gradient one code a
// logit, both ways round.
//
//   loss      m = max z,  s = sum exp(z - m) over the tile's columns of a row, and z of the target
//   gradient  d = dloss (exp(z - lse) - [column = target]),  q = round_to_fp8(fp32(d * scale))
//
// Both take the accumulators as they are.  A lane holds one row of each matrix-core block and
// runs of four consecutive columns, so the row's maximum and sum are taken in registers, two (32 x 32
// blocks) or four lanes meet by shuffles and the tile's waves in LDS; nothing of the
// tile is staged.  The gradient's codes are packed four columns to a dword for the row-major tile
// in LDS, and transposed between the four lanes of four consecutive rows for the other one.
//
// exp(z - m) is 2^(c s - m log2 e) (V_EXP_F32) with c the accumulator and s = sinv_a sinv_b log2 e:
// one multiply-add, exact until its rounding.  s and m log2 e are rounded before it, so the exponent is off by up to
// 2^-24 (|z| + |m|), where z rounded and then the difference would be off by 2^-24 |z|: at logits of 20, 2.4e-6 against 1.2e-6, both
// inside what the product's own bound allows z (1e-5 of its sum of magnitudes).  An infinite or NaN logit makes its row's loss NaN; a
// row whose target lies outside the vocabulary has no gradient, whatever its logits are.
#pragma once

#include "epilogue.hpp"
#include "stats.hpp"

namespace fp8mi {

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// exp(v * sc - m), where s = sc log2 e and t = -m log2 e.
__device__ __forceinline__ float exp_of(float v, float s, float t) { return __builtin_amdgcn_exp2f(__builtin_fmaf(v, s, t)); }

// Targets of the rows, int64 or int32.
struct Targets {
  const void* p;
  bool wide;
  // Target of row m relative to column `from`; -1 where it lies before it, or 2^31 and more behind.
  __device__ __forceinline__ int at(int64_t m, int64_t from) const {
    const int64_t t = (wide ? reinterpret_cast<const int64_t*>(p)[m] : (int64_t)reinterpret_cast<const int32_t*>(p)[m]);
    const int64_t rel = (int64_t)((uint64_t)t - (uint64_t)from);
    return rel >= 0 && rel == (int64_t)(int)rel ? (int)rel : -1;
  }
  __device__ __forceinline__ bool inside(int64_t m, int64_t vocab) const {
    const int64_t t = wide ? reinterpret_cast<const int64_t*>(p)[m] : (int64_t)reinterpret_cast<const int32_t*>(p)[m];
    return t >= 0 && t < vocab;
  }
};

// The four consecutive columns that registers hold of a matrix-core block: group g of a 32 x 32
// block (columns 8 g + 4 (lane / 32) ..), or a 16 x 16 block (columns 4 (lane / 16) ..).
template <int BLK, class V>
__device__ __forceinline__ v4f block_quad(const V& acc, int g) {
  if constexpr (BLK == 32) return (v4f){acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
  else return acc;
}
template <int BLK>
__device__ __forceinline__ int block_col(int lane, int g) {
  return BLK == 32 ? 8 * g + 4 * (lane >> 5) : 4 * (lane >> 4);
}
template <int BLK>
constexpr int kBlockGroups = BLK == 32 ? 4 : 1;

struct LossEpi {
  float2* partials;  // [tiles of columns x M]: {m, s}
  float* mine;       // [M]: the target's logit, written where the target is in these columns
  Targets targets;
  int64_t col0;      // column 0 of this product in the vocabulary

  // The sum of exp(x - top) and top itself over the lanes of a row (the lanes `step` and more apart).
  template <int BLK>
  static __device__ __forceinline__ float lanes_max(float v) {
    if constexpr (BLK == 16) v = __builtin_fmaxf(v, __shfl_xor(v, 16, 64));
    return __builtin_fmaxf(v, __shfl_xor(v, 32, 64));
  }
  template <int BLK>
  static __device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (BLK == 16) v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
  }
  // exp(x - m) is taken from 0 where a part has no column (m = -inf): it is 0 then, not NaN.
  static __device__ __forceinline__ float reference(float m) { return m == -__builtin_inff() ? 0.0f : m; }

  template <int BM, int BN, int WM, int WN, int BLK, class ACC>
  __device__ __forceinline__ void finish_tile(const ACC& acc, float sc, uint8_t* smem, int64_t M, int64_t N,
                                              int64_t m_base, int64_t n_base, int tn, int w, int lane) const {
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / BLK, FN = WTN / BLK, G = kBlockGroups<BLK>;
    const int wm = w / WN, wn = w % WN;
    const int cols_left = (int)(N - n_base < BN ? N - n_base : BN);
    float2* part = reinterpret_cast<float2*>(smem);  // [WN][BM]
    int want[FM];  // the row's target, as a column of the tile
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = m_base + wm * WTM + i * BLK + (lane & (BLK - 1));
      want[i] = m < M ? targets.at(m, col0 + n_base) : -1;
    }
    __syncthreads();  // the LDS is free
    // `edge`: the tile crosses the last column; `neg`: sc is negative (or NaN), so that the largest logit is
    // not the largest accumulator's.
    auto rows = [&](auto edge, auto neg) {
      const float s = sc * kLog2e;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = wm * WTM + i * BLK + (lane & (BLK - 1));
        auto each = [&](auto&& f) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const int c = wn * WTN + j * BLK + block_col<BLK>(lane, g);
              const v4f v = block_quad<BLK>(acc[i][j], g);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (decltype(edge)::value && c + e >= cols_left) continue;
                f(v[e], c + e);
              }
            }
        };
        float top = -__builtin_inff();
        if constexpr (decltype(neg)::value) {
          each([&](float v, int) { top = __builtin_fmaxf(top, v * sc); });
        } else {
          each([&](float v, int) { top = __builtin_fmaxf(top, v); });
          // -inf where the wave has no column, whatever sc is
          top = top == -__builtin_inff() ? top : top * sc;
        }
        top = lanes_max<BLK>(top);
        const float t = -reference(top) * kLog2e;
        float sum = 0.0f;
        each([&](float v, int) { sum += exp_of(v, s, t); });
        sum = lanes_sum<BLK>(sum);
        if (lane < BLK) part[wn * BM + r] = make_float2(top, sum);
        // few waves hold the target of any of their rows
        const int w0 = want[i];
        const bool here = w0 >= wn * WTN && w0 < (wn + 1) * WTN && w0 < cols_left;
        if (__any(here)) {
          each([&](float v, int c) {
            if (here && c == w0) mine[m_base + r] = v * sc;
          });
        }
      }
    };
    auto with_edge = [&](auto neg) {
      if (cols_left == BN) rows(std::false_type{}, neg);
      else rows(std::true_type{}, neg);
    };
    if (__builtin_expect(sc >= 0.0f, 1)) with_edge(std::false_type{});
    else with_edge(std::true_type{});
    __syncthreads();
    const int t = threadIdx.x;
    if (t < BM && m_base + t < M) {
      float2 v[WN];
      float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
      for (int k = 0; k < WN; ++k) {
        v[k] = part[k * BM + t];
        top = __builtin_fmaxf(top, v[k].x);
      }
      const float ref = reference(top);
#pragma unroll
      for (int k = 0; k < WN; ++k) sum += v[k].y * exp_of(v[k].x - ref);
      partials[(int64_t)tn * M + m_base + t] = make_float2(top, sum);
    }
  }

  // The few-row kernel's sums: red[wave][row][column] of a 16 x 16 tile each, `split` waves a tile,
  // tiles_wg tiles a workgroup of NW waves.  32 lanes a row, four columns a lane.
  template <int NW>
  __device__ __forceinline__ void finish_rows(const float (*red)[16][16], int split, int tiles_wg, float sc, int M,
                                              int N) const {
    const int m = threadIdx.x >> 5, c4 = threadIdx.x & 31, slot = c4 >> 2;
    const int64_t n = ((int64_t)blockIdx.x * tiles_wg + slot) * 16 + (c4 & 3) * 4;
    v4f x = (v4f){0.f, 0.f, 0.f, 0.f};
    if (slot < tiles_wg) {
      for (int k = slot * split; k < (slot + 1) * split; ++k) x += *reinterpret_cast<const v4f*>(&red[k][m][(c4 & 3) * 4]);
    }
    x *= sc;
    float top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (slot >= tiles_wg || n + e >= N) x[e] = -__builtin_inff();
      top = __builtin_fmaxf(top, x[e]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off, 64));
    const float ref = reference(top);
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += exp_of(x[e] - ref);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (m >= M) return;
    if (c4 == 0) partials[(int64_t)blockIdx.x * M + m] = make_float2(top, sum);
    if (slot < tiles_wg) {
      const int t = targets.at(m, col0 + n);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t == e && n + e < N) mine[m] = x[e];
    }
  }
};
template <>
struct is_tile_epilogue<LossEpi> {
  static constexpr bool value = true;
};

// A tile of codes in LDS, ROWS x COLS bytes: the 16-byte granule g of row r sits at position
// g ^ (r mod granules a row), so that lanes on consecutive rows meet different banks.
template <int COLS>
struct CodeTile {
  static constexpr int GR = COLS / 16;
  uint8_t* lds;
  __device__ __forceinline__ uint8_t* at(int r, int byte) const {
    return lds + r * COLS + ((((byte >> 4) ^ r) & (GR - 1)) << 4) + (byte & 15);
  }
};

// Lane l of each four consecutive lanes holds four codes (columns 0 .. 3) of its row; it gets those
// of column l & 3 of the four rows (byte = row).
__device__ __forceinline__ uint32_t transpose_quad(uint32_t w, uint32_t pair) {
  const uint32_t w0 = __builtin_amdgcn_mov_dpp((int)w, 0x00, 0xF, 0xF, true);  // quad_perm: lane 0's, 1's, 2's, 3's
  const uint32_t w1 = __builtin_amdgcn_mov_dpp((int)w, 0x55, 0xF, 0xF, true);
  const uint32_t w2 = __builtin_amdgcn_mov_dpp((int)w, 0xAA, 0xF, 0xF, true);
  const uint32_t w3 = __builtin_amdgcn_mov_dpp((int)w, 0xFF, 0xF, 0xF, true);
  // `pair` selects byte (lane & 3) of the second source (0 .. 3), then that of the first (4 .. 7)
  const uint32_t lo = __builtin_amdgcn_perm(w1, w0, pair), hi = __builtin_amdgcn_perm(w3, w2, pair);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

struct LogitGradEpi {
  const float* lse;    // [M]
  const float* dloss;  // [M]
  const float* scale;
  uint8_t* q;          // [M x ldq] codes of d, zeros from column N to the next multiple of 128; or null
  uint8_t* q_t;        // [N x ldt] of its transpose, zeros from M to ldt; or null
  uint32_t* amax_bits; // cleared beforehand; may be null
  unsigned long long* sat;
  Targets targets;
  int64_t vocab;       // a row whose target lies outside has no gradient
  int64_t col0;
  int64_t ldq, ldt;    // multiples of 128; ldt less than 128 above M
  int fmt;

  template <int BM, int BN, int WM, int WN, int BLK, class ACC>
  __device__ __forceinline__ void finish_tile(const ACC& acc, float sc, uint8_t* smem, int64_t M, int64_t N,
                                              int64_t m_base, int64_t n_base, int tn, int w, int lane) const {
    if (fmt == kE4M3) codes<kE4M3, BM, BN, WM, WN, BLK>(acc, sc, smem, M, N, m_base, n_base, w, lane);
    else codes<kE5M2, BM, BN, WM, WN, BLK>(acc, sc, smem, M, N, m_base, n_base, w, lane);
  }

  template <int FMT, int BM, int BN, int WM, int WN, int BLK, class ACC>
  __device__ __forceinline__ void codes(const ACC& acc, float sc, uint8_t* smem, int64_t M, int64_t N, int64_t m_base,
                                        int64_t n_base, int w, int lane) const {
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / BLK, FN = WTN / BLK, G = kBlockGroups<BLK>;
    constexpr int NT = 64 * WM * WN;
    const int wm = w / WN, wn = w % WN;
    const int cols_left = (int)(N - n_base < BN ? N - n_base : BN);
    const CodeTile<BN> rows_tile{smem};
    const CodeTile<BM> cols_tile{smem + BM * BN};
    const uint32_t pair = 0x0C0C0400u + 0x0101u * (lane & 3);  // bytes 2 and 3 are not used (constant 0)
    const float out = *scale, s = sc * kLog2e;
    constexpr float kMax = Fp8Traits<FMT>::max_value;
    // A row without a gradient (past the edge, or its target outside) has its codes masked and takes no part
    // in the statistics: a factor of 0 would not do, since its logits may be NaN.
    int want[FM];
    float t[FM], grad[FM];  // -lse log2 e, and dloss
    bool live[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = m_base + wm * WTM + i * BLK + (lane & (BLK - 1));
      live[i] = m < M && targets.inside(m, vocab);
      want[i] = live[i] ? targets.at(m, col0 + n_base) : -1;
      t[i] = live[i] ? lse[m] * -kLog2e : 0.0f;
      grad[i] = live[i] ? dloss[m] : 0.0f;
    }
    __syncthreads();  // the LDS is free
    LaneStats st;
    const bool count = sat != nullptr;
    auto rows = [&](auto edge) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = wm * WTM + i * BLK + (lane & (BLK - 1));
        const uint32_t mask = live[i] ? 0xFFFFFFFFu : 0u;
        const bool here = want[i] >= wn * WTN && want[i] < (wn + 1) * WTN;
        const bool any = __any(here);
        float top = 0.0f;  // the largest |exp(z - lse) - [target]| of the row's values
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const int c = wn * WTN + j * BLK + block_col<BLK>(lane, g);
            const v4f v = block_quad<BLK>(acc[i][j], g);
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = exp_of(v[e], s, t[i]);
            if (any) {
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] -= c + e == want[i] ? 1.0f : 0.0f;
            }
            if constexpr (decltype(edge)::value) {
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] = c + e >= cols_left ? 0.0f : p[e];
            }
            float m = __builtin_elementwise_maximum(__builtin_fabsf(p[0]), __builtin_fabsf(p[1]));
            m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(p[2]), __builtin_fabsf(p[3])), m);
            top = __builtin_elementwise_maximum(top, m);
            // Roundings are monotone: where the largest stays inside, all do, and none is NaN.
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = p[e] * grad[i] * out;
            uint32_t word;
            if (__builtin_expect(__builtin_fabsf(m * grad[i] * out) <= kMax, 1)) {
              word = cvt_pk<FMT, true>(d[2], d[3], cvt_pk<FMT, false>(d[0], d[1], 0u));
            } else {
              // Each for itself: with an infinite dloss or scale a p of 0 gives NaN, but not in the padding.
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const bool past = decltype(edge)::value && c + e >= cols_left;
                d[e] = past ? 0.0f : d[e];
                if (live[i] && !past) {
                  st.max = __builtin_elementwise_maximum(st.max, __builtin_fabsf(p[e] * grad[i]));
                  if (count) st.sat += __builtin_fabsf(d[e]) > kMax ? 1u : 0u;
                }
              }
              word = encode4<FMT>(d[0], d[1], d[2], d[3]);
            }
            word &= mask;
            if (q) *reinterpret_cast<uint32_t*>(rows_tile.at(r, c)) = word;
            if (q_t) *reinterpret_cast<uint32_t*>(cols_tile.at(c + (lane & 3), r & ~3)) = transpose_quad(word, pair);
          }
        // (A top of 0 may be the padding's; a p of 0 with an infinite dloss has been seen to above.)
        if (live[i] && top != 0.0f) st.max = __builtin_elementwise_maximum(st.max, __builtin_fabsf(top * grad[i]));
      }
    };
    if (cols_left == BN) rows(std::false_type{});
    else rows(std::true_type{});
    __syncthreads();
    const int tid = threadIdx.x;
    if (q) {
      constexpr int GR = BN / 16;
      for (int idx = tid; idx < BM * GR; idx += NT) {
        const int r = idx / GR, byte = idx % GR * 16;
        if (m_base + r >= M) break;  // rows are visited in order
        if (n_base + byte < ((N + 127) & ~int64_t(127)))
          *reinterpret_cast<uint4*>(q + (m_base + r) * ldq + n_base + byte) = *reinterpret_cast<const uint4*>(rows_tile.at(r, byte));
      }
    }
    if (q_t) {
      constexpr int GR = BM / 16;
      for (int idx = tid; idx < BN * GR; idx += NT) {
        const int r = idx / GR, byte = idx % GR * 16;
        if (r >= cols_left) break;
        if (m_base + byte < ldt)
          *reinterpret_cast<uint4*>(q_t + (n_base + r) * ldt + m_base + byte) = *reinterpret_cast<const uint4*>(cols_tile.at(r, byte));
      }
      if constexpr (BM < 128) {  // rows' padding past the last tile
        static_assert(BM == 64, "half a step");
        if (m_base + 2 * BM == ldt && m_base + BM >= M) {
          for (int idx = tid; idx < cols_left * GR; idx += NT)
            *reinterpret_cast<uint4*>(q_t + (n_base + idx / GR) * ldt + m_base + BM + idx % GR * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    if (amax_bits || sat) {
      __syncthreads();
      EpiArgs stats{};
      stats.amax_bits = amax_bits;
      stats.sat = sat;
      publish_epilogue_stats(stats, st, reinterpret_cast<uint32_t*>(smem));
    }
  }
};
template <>
struct is_tile_epilogue<LogitGradEpi> {
  static constexpr bool value = true;
};

}  // namespace fp8mi
