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
// exp(z - m) is 2^((z - m) log2 e) (V_EXP_F32): the difference first, so its error is relative
// to the difference, not to the logits.  An infinite or NaN logit makes its row's loss NaN; a
// row whose target lies outside the vocabulary has no gradient, whatever its logits are.
#pragma once

#include "epilogue.hpp"
#include "stats.hpp"

namespace fp8mi {


__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

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
    auto rows = [&](auto edge) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = wm * WTM + i * BLK + (lane & (BLK - 1));
        auto each = [&](auto&& f) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const int c = wn * WTN + j * BLK + block_col<BLK>(lane, g);
              const v4f v = block_quad<BLK>(acc[i][j], g) * sc;
#pragma unroll
              for (int e = 0; e < 4; ++e) f((decltype(edge)::value && c + e >= cols_left) ? -__builtin_inff() : v[e], c + e);
            }
        };
        float top = -__builtin_inff();
        each([&](float x, int) { top = __builtin_fmaxf(top, x); });
        top = lanes_max<BLK>(top);
        const float ref = reference(top);
        float sum = 0.0f;
        each([&](float x, int) { sum += exp_of(x - ref); });
        sum = lanes_sum<BLK>(sum);
        if (lane < BLK) part[wn * BM + r] = make_float2(top, sum);
        // few waves hold the target of any of their rows
        const int t = want[i];
        const bool here = t >= wn * WTN && t < (wn + 1) * WTN && t < cols_left;
        if (__any(here)) {
          each([&](float x, int c) {
            if (here && c == t) mine[m_base + r] = x;
          });
        }
      }
    };
    if (cols_left == BN) rows(std::false_type{});
    else rows(std::true_type{});
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
  uint8_t* q;          // [M x ldq] codes of d, zeros from column N to ldq; or null
  uint8_t* q_t;        // [N x ldt] of its transpose, zeros from M to ldt; or null
  uint32_t* amax_bits; // cleared beforehand; may be null
  unsigned long long* sat;
  Targets targets;
  int64_t vocab;       // a row whose target lies outside has no gradient
  int64_t col0;
  int64_t ldq, ldt;    // multiples of 16, less than 16 above N and M
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
    const float out = *scale;
    const uint32_t pair = 0x0C0C0400u + 0x0101u * (lane & 3);  // bytes 2 and 3 are not used (constant 0)
    constexpr int kDead = -2;  // a row without a gradient: selected, not multiplied away, since its logits may be NaN
    int want[FM];
    float top[FM], grad[FM];   // lse and dloss
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = m_base + wm * WTM + i * BLK + (lane & (BLK - 1));
      const bool live = m < M && targets.inside(m, vocab);
      want[i] = live ? targets.at(m, col0 + n_base) : kDead;
      top[i] = live ? lse[m] : 0.0f;
      grad[i] = live ? dloss[m] : 0.0f;
    }
    __syncthreads();  // the LDS is free
    LaneStats st;
    const bool with_sat = sat != nullptr;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * WTM + i * BLK + (lane & (BLK - 1));
      const bool dead = want[i] == kDead;
      const bool here = want[i] >= wn * WTN && want[i] < (wn + 1) * WTN;
      const bool any = __any(here);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int c = wn * WTN + j * BLK + block_col<BLK>(lane, g);
          const v4f v = block_quad<BLK>(acc[i][j], g) * sc;
          float d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = exp_of(v[e] - top[i]);
          if (any) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] -= c + e == want[i] ? 1.0f : 0.0f;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = (dead || c + e >= cols_left) ? 0.0f : d[e] * grad[i];
          const uint32_t word = encode4_stats<FMT>(d, out, with_sat, st);
          if (q) *reinterpret_cast<uint32_t*>(rows_tile.at(r, c)) = word;
          if (q_t) *reinterpret_cast<uint32_t*>(cols_tile.at(c + (lane & 3), r & ~3)) = transpose_quad(word, pair);
        }
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (q) {
      constexpr int GR = BN / 16;
      for (int idx = t; idx < BM * GR; idx += NT) {
        const int r = idx / GR, byte = idx % GR * 16;
        if (m_base + r >= M) break;  // rows are visited in order
        if (n_base + byte < ldq)
          *reinterpret_cast<uint4*>(q + (m_base + r) * ldq + n_base + byte) = *reinterpret_cast<const uint4*>(rows_tile.at(r, byte));
      }
    }
    if (q_t) {
      constexpr int GR = BM / 16;
      for (int idx = t; idx < BN * GR; idx += NT) {
        const int r = idx / GR, byte = idx % GR * 16;
        if (r >= cols_left) break;
        if (m_base + byte < ldt)
          *reinterpret_cast<uint4*>(q_t + (n_base + r) * ldt + m_base + byte) = *reinterpret_cast<const uint4*>(cols_tile.at(r, byte));
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

  // encode8 (stats.hpp) on four values.
  template <int FMT>
  static __device__ __forceinline__ uint32_t encode4_stats(const float* d, float scale, bool count, LaneStats& st) {
    float m = __builtin_elementwise_maximum(__builtin_fabsf(d[0]), __builtin_fabsf(d[1]));
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(d[2]), __builtin_fabsf(d[3])), m);
    st.max = __builtin_elementwise_maximum(st.max, m);
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = d[e] * scale;
    if (__builtin_expect(__builtin_fabsf(m * scale) <= Fp8Traits<FMT>::max_value, 1))
      return cvt_pk<FMT, true>(p[2], p[3], cvt_pk<FMT, false>(p[0], p[1], 0u));
    if (count) {
#pragma unroll
      for (int e = 0; e < 4; ++e) st.sat += __builtin_fabsf(p[e]) > Fp8Traits<FMT>::max_value ? 1u : 0u;
    }
    return encode4<FMT>(p[0], p[1], p[2], p[3]);
  }
};
template <>
struct is_tile_epilogue<LogitGradEpi> {
  static constexpr bool value = true;
};

}  // namespace fp8mi
