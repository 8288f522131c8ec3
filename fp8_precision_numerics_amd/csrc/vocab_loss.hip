// Softmax cross entropy over a vocabulary without its logits: the head's product
// with the loss behind it (vocab_epilogue.hpp), forward.
//
//   z = (x W^T) sinv_x sinv_w [M x V],  lse = log sum_v exp z,  loss = lse - z[target]
//
// Matrix-core-bound for many rows (2 M V K operations), bound by the weight's V K bytes
// for a few, which take the streaming kernel of gemm_few_rows.hip.  A tile leaves the maximum and
// the sum of each of its rows (8 bytes a row and 256 columns: 1/64 of bf16 logits), a second kernel joins
// them; a workspace too small for the whole vocabulary's is served in pieces, the joined
// pair of each row carried from one to the next.
// Measured on MI355X: 8192 x 65536 x 4096 exact 2.77-2.95 ms (1.49-1.58 PFLOP/s, the clock under the power limit), 1003 x 50021 x 4096
// 0.305 ms (1.35), a row of 131072 x 4096 93 us (5.8 TB/s of the weight), 64 rows 121 us (FP8 cores 111); the joining kernel 5-6 us of each.
#include "gemm_few_rows.hpp"
#include "launch.hpp"
#include "model_ends.hpp"
#include "vocab_dispatch.hpp"

namespace fp8mi {
namespace {

struct JoinArgs {
  const float2* partials;  // [tiles x M]
  float2* state;           // [M]: the columns before these
  const float* mine;
  Targets targets;
  float* loss;
  float* lse;
  int64_t M, vocab;
  int tiles;
  bool first, last;
};

// {m, s} of two sets of columns together.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = __builtin_fmaxf(a.x, b.x), ref = LossEpi::reference(m);
  return make_float2(m, a.y * exp_of(a.x - ref) + b.y * exp_of(b.x - ref));
}

// R rows a workgroup of 256, 256 / R lanes down the tiles of each.
template <int R>
__global__ __launch_bounds__(256) void vocab_join_kernel(JoinArgs a) {
  constexpr int L = 256 / R;
  __shared__ float2 buf[256];
  const int t = threadIdx.x, l = t / R;
  const int64_t row = (int64_t)blockIdx.x * R + t % R;
  const bool here = row < a.M;
  constexpr int U = 8;
  const float2 none = make_float2(-__builtin_inff(), 0.0f);
  float2 v = none;
  if (here) {
    for (int k = l; k < a.tiles; k += U * L) {
      float2 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) p[u] = k + u * L < a.tiles ? a.partials[(int64_t)(k + u * L) * a.M + row] : none;
#pragma unroll
      for (int u = 0; u < U; ++u) v = join(v, p[u]);
    }
  }
  buf[t] = v;
  __syncthreads();
#pragma unroll
  for (int half = L / 2; half > 0; half >>= 1) {
    if (l < half) buf[t] = join(buf[t], buf[t + half * R]);
    __syncthreads();
  }
  if (l != 0 || !here) return;
  v = buf[t];
  if (!a.first) v = join(a.state[row], v);
  if (!a.last) {
    a.state[row] = v;
    return;
  }
  const float lse = v.x + logf(v.y);
  if (a.lse) a.lse[row] = lse;
  if (a.loss) a.loss[row] = a.targets.inside(row, a.vocab) ? lse - a.mine[row] : 0.0f;
}

// As many rows a workgroup (up to a line of the partials) as leave one for about every second compute unit.
void join_launch(const JoinArgs& a, hipStream_t st) {
  if (a.M >= 2048) hipLaunchKernelGGL(vocab_join_kernel<16>, dim3((unsigned)((a.M + 15) / 16)), dim3(256), 0, st, a);
  else if (a.M >= 512) hipLaunchKernelGGL(vocab_join_kernel<4>, dim3((unsigned)((a.M + 3) / 4)), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(vocab_join_kernel<1>, dim3((unsigned)a.M), dim3(256), 0, st, a);
}

}  // namespace

hipError_t launch_vocab_logits(const VocabOperands& o, int64_t col, int64_t N, const LossEpi& epi, int accum, int* tiles,
                               hipStream_t stream) {
  const int64_t first = plan_rounds(o.M, N, o.K, accum == kAccumMfma8, 0, persistent_groups(1)).first;
  LossEpi e = epi;
  *tiles = 0;
  for (int64_t at = 0; at < N;) {
    const int64_t n = at == 0 ? first : N - first, wide = vocab_shape(o, n, accum) == 0 ? 256 : 128;
    e.col0 = epi.col0 + at;
    e.partials = epi.partials + (int64_t)*tiles * o.M;
    const hipError_t status = vocab_launch(o, col + at, n, e, accum, stream);
    if (status != hipSuccess) return status;
    *tiles += (int)((n + wide - 1) / wide);
    at += n;
  }
  return hipSuccess;
}

hipError_t launch_vocab_cross_entropy(const VocabOperands& o, int64_t V, const Targets& targets, float* loss, float* lse,
                                      int accum, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  JoinArgs j{nullptr, nullptr, reinterpret_cast<float*>(ws), targets, loss, lse, o.M, V, 0, true, true};
  LossEpi epi{nullptr, reinterpret_cast<float*>(ws), targets, 0};
  ws += up16(o.M * 4);
  j.state = reinterpret_cast<float2*>(ws);
  ws += up16(o.M * 8);
  j.partials = epi.partials = reinterpret_cast<float2*>(ws);
  // slots for the pairs of so many tiles
  const int64_t slots = (int64_t)(workspace_bytes - (size_t)(ws - reinterpret_cast<uint8_t*>(workspace))) / (o.M * 8);
  // The streaming kernel reads and widens the rows anew for every 16 columns, which from about 9 rows on takes longer than the tiles'
  // padding to 64 rows does, if there is a tile for every compute unit: 16 rows, 131072 x 4096 123 us against 110, 50021 x 1024 23 against
  // 18, but 32000 x 4096 (250 tiles) 38 both; 8 rows 108 against 110.
  const bool few = o.M <= kFewRows / 2 || (o.M <= kFewRows && (V + 127) / 128 < persistent_groups(1));
  const int64_t longest = few ? kFewColumns : launch_columns(o.M);
  for (int64_t col = 0; col < V;) {
    int64_t n = V - col;
    hipError_t e;
    const int64_t fit = slots * 128;  // the narrower tiles', and the streaming kernel's with a wave a tile
    if (n > fit) n = fit / kPieceCols * kPieceCols;
    if (n > longest) n = longest;
    epi.col0 = col;
    if (few) {
      e = launch_loss_few_rows(o.a, o.fa, o.b + col * o.K, o.fb, o.M, n, o.K, o.sinv_a, o.sinv_b, epi, slots, &j.tiles, stream);
    } else {
      e = launch_vocab_logits(o, col, n, epi, logits_mode(o.M, accum), &j.tiles, stream);
    }
    if (e != hipSuccess) return e;
    j.first = col == 0;
    col += n;
    j.last = col >= V;
    join_launch(j, stream);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8mi
