// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = round(scale * table[id_t])              (zeros where the id lies outside the table)
//   dtable[v] = round(base[v] + scale * sum over { t : id_t = v } of dy[t])
//
// Both are bound by memory.  The lookup is a gather of whole rows: a lane moves octets
// (eight values: 16 bytes of bf16, 8 of codes), consecutive lanes consecutive ones.
//
// The gradient adds rows in an order that is fixed (t ascending, joined in pieces), so
// that its bits repeat: tokens are sorted by (id, t), stably and without atomics.
//   rank_tokens_kernel   blocks of kSortBlock tokens: a token's place is the number of tokens of
//                        its block that come before it, counted by comparing it with all of them
//                        (LDS broadcasts, half a wave per thirty-second of the block): one launch, no
//                        passes over digits.  8192 tokens are 67 M comparisons.
//   merge_tokens_kernel  more blocks than one: a token's place in the whole is its place in its
//                        block plus its rank in every other block, by bisection.
//   token_rows_kernel    the sorted list in chunks of equal length, so that a common token costs
//                        no workgroup more than a rare one: runs of one id that lie inside a
//                        chunk are written, those that cross its ends leave partial rows.  The
//                        workgroups behind those write base (or zeros) to the rows of ids that do not
//                        occur, which they look up in the list: every row is written once, and the sums
//                        run beside that stream.
//   token_joins_kernel   adds the partial rows of each run that crosses.
// Measured on MI355X: lookup of 8192 rows of 4096 bf16 20.5 us (134 MB, 6.5 TB/s); gradient of a 65536 x 4096 bf16
// table added to a base, 8192 tokens of a skewed distribution, 235 us (1.14 GB, 4.85 TB/s: a copy's rate), of which the
// sort 10.8 and the joins 7 (with a kernel of its own that first filled every row: 318 us).
#include "launch.hpp"
#include "model_ends.hpp"
#include "row_octets.hpp"
#include "token_chunks.hpp"

namespace fp8mi {
namespace {

constexpr uint32_t kNoToken = 0x80000000u;  // sorts behind every id
constexpr int kLookNT = 256;

__device__ __forceinline__ int64_t token_at(const void* tokens, bool wide, int64_t t) {
  return wide ? reinterpret_cast<const int64_t*>(tokens)[t] : reinterpret_cast<const int32_t*>(tokens)[t];
}

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
struct LookupArgs {
  const void* tokens;
  const void* table;
  const float* sinv;  // of codes
  void* out;
  int64_t rows, vocab, octets;
  float scale;
  int lanes;          // lanes a row, a power of two up to kLookNT
  int slices;         // workgroups a row
  bool wide;          // int64 tokens
};

// Table types: kF32, kBF16, and codes.
enum : int { kTableE4M3 = 2, kTableE5M2 = 3 };

// Eight codes (bytes of w.x, then w.y), exactly.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float* f) {
  const uint32_t p[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v2f lo, hi;
    if constexpr (FMT == kE4M3) {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)p[i], true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)p[i], false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)p[i], true);
    }
    f[4 * i] = lo[0];
    f[4 * i + 1] = lo[1];
    f[4 * i + 2] = hi[0];
    f[4 * i + 3] = hi[1];
  }
}

template <int TT, int OT>
__global__ __launch_bounds__(kLookNT) void lookup_kernel(LookupArgs a) {
  const int block = blockIdx.x / a.slices, blocks = gridDim.x / a.slices;
  const int slice = blockIdx.x - block * a.slices;
  const int lane = threadIdx.x & (a.lanes - 1), side = kLookNT / a.lanes;  // rows side by side
  float inv = 1.0f;
  if constexpr (TT == kTableE4M3 || TT == kTableE5M2) inv = *a.sinv;
  for (int64_t t = (int64_t)block * side + threadIdx.x / a.lanes; t < a.rows; t += (int64_t)blocks * side) {
    const int64_t id = token_at(a.tokens, a.wide, t);
    const bool inside = id >= 0 && id < a.vocab;
    for (int64_t o = lane + (int64_t)slice * a.lanes; o < a.octets; o += (int64_t)a.lanes * a.slices) {
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (inside) {
        if constexpr (TT == kF32 || TT == kBF16) {
          Octet<TT> v;
          v.load(a.table, id * a.octets + o);
          v.widen(f);
        } else {
          decode8<TT == kTableE4M3 ? kE4M3 : kE5M2>(reinterpret_cast<const uint2*>(a.table)[id * a.octets + o], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= inv;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= a.scale;
      }
      Octet<OT> r;
      r.narrow(f);
      r.store_nt(a.out, t * a.octets + o);
    }
  }
}

// Lanes of a row: the smallest power of two that holds its octets, up to a workgroup.
int row_lanes(int64_t octets) {
  int lanes = 2;
  while (lanes < kLookNT && lanes < octets) lanes *= 2;
  return lanes;
}

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kSortGroup = 32;                             // tokens a workgroup ranks
constexpr int kSortPart = kSortBlock / (2 * kSortWaves);   // ids a half wave compares with
constexpr int kSortPitch = kSortPart + 4;                  // of parts in LDS, so that the halves' reads meet other banks

struct SortArgs {
  const void* tokens;
  uint32_t* keys;   // sorted within blocks
  int32_t* places;  // the tokens' numbers, likewise
  int64_t rows, vocab;
  bool wide;
};

// Lane l holds token l % 32 of the group and compares it with the ids of part 2 w + l / 32.
__global__ __launch_bounds__(64 * kSortWaves) void rank_tokens_kernel(SortArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t ids[2 * kSortWaves * kSortPitch];
  __shared__ int counts[2 * kSortWaves][kSortGroup];
  const int64_t first = (int64_t)blockIdx.y * kSortBlock;
  const int n = (int)(a.rows - first < kSortBlock ? a.rows - first : kSortBlock);
  auto slot = [](int j) { return j + j / kSortPart * (kSortPitch - kSortPart); };
#pragma unroll
  for (int i = 0; i < kSortBlock / (64 * kSortWaves); ++i) {
    const int j = threadIdx.x + i * 64 * kSortWaves;
    uint32_t key = 0xFFFFFFFFu;  // past the end: below nothing
    if (j < n) {
      const int64_t id = token_at(a.tokens, a.wide, first + j);
      key = id >= 0 && id < a.vocab ? (uint32_t)id : kNoToken;
    }
    ids[slot(j)] = key;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, part = 2 * w + (lane >> 5);
  const int group = blockIdx.x * kSortGroup, mine = group + (lane & 31);
  const uint32_t key = ids[slot(mine)];
  int count = 0;
  if (2 * w * kSortPart < n) {
    // 32 ids before the group count where they are not above, that is below the next number; those of the group
    // itself and behind it where they are below.
    for (int j0 = 0; j0 < kSortPart; j0 += kSortGroup) {
      const uint32_t limit = part * kSortPart + j0 < group ? key + 1u : key;
#pragma unroll
      for (int j = 0; j < kSortGroup; j += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(&ids[part * kSortPitch + j0 + j]);
        count += (v.x < limit) + (v.y < limit) + (v.z < limit) + (v.w < limit);
      }
    }
  }
  if (part == 0) {  // equal ids of the group before this one
    for (int j = group; j < mine; ++j) count += ids[slot(j)] == key ? 1 : 0;
  }
  counts[part][lane & 31] = count;
  __syncthreads();
  if (threadIdx.x < kSortGroup && mine < n) {
    int place = 0;
#pragma unroll
    for (int p = 0; p < 2 * kSortWaves; ++p) place += counts[p][threadIdx.x];
    a.keys[first + place] = key;
    a.places[first + place] = (int32_t)(first + mine);
  }
}

// Number of keys of keys[0 .. n) that are below `limit` (equal: they count too).
__device__ __forceinline__ int count_below(const uint32_t* keys, int n, uint32_t limit, bool equal) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    const uint32_t k = keys[mid];
    if (k < limit || (equal && k == limit)) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(256) void merge_tokens_kernel(const uint32_t* keys, const int32_t* places, int64_t rows,
                                                          uint32_t* out_keys, int32_t* out_places) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows) return;
  const int64_t own = i / kSortBlock, blocks = (rows + kSortBlock - 1) / kSortBlock;
  const uint32_t key = keys[i];
  int64_t place = i - own * kSortBlock;
  for (int64_t b = 0; b < blocks; ++b) {
    if (b == own) continue;
    const int64_t first = b * kSortBlock;
    const int n = (int)(rows - first < kSortBlock ? rows - first : kSortBlock);
    place += count_below(keys + first, n, key, b < own);
  }
  out_keys[place] = key;
  out_places[place] = places[i];
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------
struct SumArgs {
  const uint32_t* keys;
  const int32_t* places;
  const void* dy;
  const void* base;  // null: zeros
  void* dtable;
  float* partials;   // [chunks x 2 x cols]: a chunk's sum of the run that enters it, of the one that leaves it
  int64_t rows, octets;
  float scale;
  int chunk;         // sorted tokens a chunk
  int chunks;
  int lanes, slices; // as in LookupArgs; lanes x slices cover a row
  int sum_groups;    // workgroups of the sums; those behind them fill
  int64_t vocab;
  int words;         // 16-byte words of a table row
  int band;          // rows that a filling workgroup takes together
};

template <int OT>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, int64_t o, const float* acc) {
  const int64_t at = (int64_t)key * a.octets + o;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.base) {
    Octet<OT> b;
    b.load(a.base, at);
    b.widen(f);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(acc[e], a.scale, f[e]);
  Octet<OT> r;
  r.narrow(f);
  r.store(a.dtable, at);
}

__device__ __forceinline__ void write_partial(const SumArgs& a, int64_t chunk, int side, int64_t o, const float* acc) {
  float4* p = reinterpret_cast<float4*>(a.partials + ((chunk * 2 + side) * a.octets + o) * 8);
  p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// The chunk and the octet of a thread; false where it has none.
__device__ __forceinline__ bool chunk_of(const SumArgs& a, int64_t* chunk, int64_t* o) {
  const int64_t block = blockIdx.x / a.slices;
  *chunk = block * (kLookNT / a.lanes) + threadIdx.x / a.lanes;
  *o = (threadIdx.x & (a.lanes - 1)) + (int64_t)(blockIdx.x - block * a.slices) * a.lanes;
  return *chunk < a.chunks && *o < a.octets;
}

// base or zeros to the rows whose id does not occur.  A workgroup takes bands of `band` rows, as many bands apart
// as there are workgroups, 256 rows at a time: a thread looks one row up, then all stream the
// rows that are left, flat.
__device__ __forceinline__ void fill_absent(const SumArgs& a) {
  typedef unsigned int vec4 __attribute__((ext_vector_type(4)));
  __shared__ uint32_t absent[kLookNT];
  __shared__ int before[kLookNT / 64 + 1];
  const int t = threadIdx.x, w = t >> 6;
  const int64_t me = blockIdx.x - a.sum_groups, groups = gridDim.x - a.sum_groups;
  const int bands = kLookNT / a.band;
  const uint32_t d = a.words, magic = 0xFFFFFFFFu / d + 1u;  // d = 1 wraps to 0: not used then (a row has two words at least)
  const vec4* src = reinterpret_cast<const vec4*>(a.base);
  vec4* dst = reinterpret_cast<vec4*>(a.dtable);
  for (int64_t s = 0; (s * groups + me) * a.band < a.vocab; s += bands) {
    const int64_t row = ((s + t / a.band) * groups + me) * a.band + t % a.band;
    bool take = false;
    if (row < a.vocab) {
      const int at = count_below(a.keys, (int)a.rows, (uint32_t)row, false);
      take = at == a.rows || a.keys[at] != (uint32_t)row;
    }
    const unsigned long long votes = __ballot(take);
    if ((t & 63) == 0) before[w + 1] = __popcll(votes);
    if (t == 0) before[0] = 0;
    __syncthreads();
    if (t == 0) {
#pragma unroll
      for (int k = 1; k <= kLookNT / 64; ++k) before[k] += before[k - 1];
    }
    __syncthreads();
    if (take) absent[before[w] + __popcll(votes & ((1ull << (t & 63)) - 1ull))] = (uint32_t)row;
    __syncthreads();
    const uint32_t total = (uint32_t)before[kLookNT / 64] * d;  // at most 256 x 2^18
    constexpr int U = 4;
    for (uint32_t f = t; f < total; f += U * kLookNT) {
      int64_t at[U];
      vec4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t x = f + u * kLookNT < total ? f + u * kLookNT : f;
        uint32_t q = __umulhi(x, magic);  // x / d, or one more
        q -= q * d > x ? 1u : 0u;
        at[u] = (int64_t)absent[q] * d + (x - q * d);
        v[u] = a.base ? __builtin_nontemporal_load(src + at[u]) : (vec4){0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (f + u * kLookNT < total) __builtin_nontemporal_store(v[u], dst + at[u]);
    }
    __syncthreads();  // the list is free
  }
}

template <int DT, int OT>
__global__ __launch_bounds__(kLookNT) void token_rows_kernel(SumArgs a) {
  if ((int)blockIdx.x >= a.sum_groups) {
    fill_absent(a);
    return;
  }
  int64_t chunk, o;
  if (!chunk_of(a, &chunk, &o)) return;
  const int64_t first = chunk * a.chunk;
  const int n = (int)(a.rows - first < a.chunk ? a.rows - first : a.chunk);
  uint32_t key = a.keys[first];
  const bool enters = first > 0 && a.keys[first - 1] == key;
  const bool leaves = first + n < a.rows && a.keys[first + n - 1] == a.keys[first + n];
  bool head = enters;  // the present run came in from the chunk before
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;  // rows requested at once
  for (int i = 0; i < n; i += U) {
    Octet<DT> v[U];
    uint32_t ks[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ks[u] = kNoToken;
      v[u].clear();
      if (i + u < n) {
        ks[u] = a.keys[first + i + u];
        if (ks[u] != kNoToken) v[u].load_nt(a.dy, (int64_t)a.places[first + i + u] * a.octets + o);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < n) {
        if (ks[u] != key) {
          if (head) write_partial(a, chunk, 0, o, acc);
          else write_row<OT>(a, key, o, acc);  // keys ascend, so the one that ends here is a token's
          head = false;
          key = ks[u];
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        }
        float f[8];
        v[u].widen(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[e];
      }
    }
  }
  if (key == kNoToken) return;
  if (head) write_partial(a, chunk, 0, o, acc);
  else if (leaves) write_partial(a, chunk, 1, o, acc);
  else write_row<OT>(a, key, o, acc);
}

constexpr int kJoinLanes = 64, kJoinSides = kLookNT / kJoinLanes;
// Octet `o` of the run that begins in `chunk` and leaves it: partial row 0 is what leaves this chunk, partial row i what
// enters chunk + i, up to the one that holds the run's last token.
template <int OT>
__device__ __forceinline__ void join_run(const SumArgs& a, int64_t chunk, int64_t o, int lane, int side,
                                         float (*sums)[8][kJoinLanes]) {
  const int64_t end = (chunk + 1) * a.chunk, mine = end + (int64_t)lane * a.chunk;
  const uint32_t key = a.keys[end];
  // the chunks that begin with the token: a lane looks at each of 64, and a longer run is measured by bisection
  int count = 1 + __popcll(__ballot(mine < a.rows && a.keys[mine < a.rows ? mine : end] == key));
  if (count == 65) {
    const int64_t last = end + count_below(a.keys + end, (int)(a.rows - end), key, true) - 1;
    count = (int)(last / a.chunk - chunk) + 1;
  }
  const int quarter = (count + kJoinSides - 1) / kJoinSides;
  const int from = side * quarter, to = from + quarter < count ? from + quarter : count;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (o < a.octets) {
    constexpr int U = 8;
    for (int i = from; i < to; i += U) {
      float4 v[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + u < to) {
          const float4* p = reinterpret_cast<const float4*>(a.partials + (((chunk + i + u) * 2 + (i + u == 0 ? 1 : 0)) * a.octets + o) * 8);
          v[u][0] = p[0];
          v[u][1] = p[1];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[side][e][lane] = acc[e];
  __syncthreads();
  if (side != 0 || o >= a.octets) return;
#pragma unroll
  for (int s = 1; s < kJoinSides; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += sums[s][e][lane];
  write_row<OT>(a, key, o, acc);
}

// A run that leaves the chunk in which it begins: its partial rows, in order.  A workgroup has 64 octets of the
// row, each of its waves a quarter of the partial rows, eight of them requested at once: the run of a
// token that pads a batch is as long as the list (gradient of 8192 tokens of 4096 bf16 columns added in place, all of one token:
// 51 us, with a lane down all partial rows 81; half of 65536 tokens of one: 344, 540).  It looks at `joins`
// chunks at once, a lane each, and takes the runs that begin there one after the other: most chunks have none.
template <int OT>
__global__ __launch_bounds__(kLookNT) void token_joins_kernel(SumArgs a, int joins) {
  __shared__ float sums[kJoinSides][8][kJoinLanes];
  const int64_t slices = (a.octets + kJoinLanes - 1) / kJoinLanes, group = blockIdx.x / slices;
  const int lane = threadIdx.x & (kJoinLanes - 1), side = threadIdx.x / kJoinLanes;
  const int64_t o = lane + (blockIdx.x - group * slices) * kJoinLanes;
  bool begins = false;
  if (lane < joins) {
    const int64_t first = (group * joins + lane) * a.chunk, end = first + a.chunk;
    if (end < a.rows) {
      const uint32_t key = a.keys[end];
      begins = key != kNoToken && a.keys[end - 1] == key &&                      // it leaves
               !(first > 0 && a.keys[first] == key && a.keys[first - 1] == key); // and did not begin earlier
    }
  }
  // the same in every wave
  for (unsigned long long left = __ballot(begins); left; left &= left - 1) {
    const int64_t chunk = group * joins + __builtin_ctzll(left);
    join_run<OT>(a, chunk, o, lane, side, sums);
    __syncthreads();  // the sums are free
  }
}

// base, or zeros without one, into the whole table: 16 bytes a lane and turn.
__global__ __launch_bounds__(256) void fill_rows_kernel(const uint4* base, uint4* to, int64_t count) {
  typedef unsigned int vec4 __attribute__((ext_vector_type(4)));
  constexpr int U = 4;
  const int64_t step = (int64_t)gridDim.x * 256;
  const vec4* src = reinterpret_cast<const vec4*>(base);
  vec4* dst = reinterpret_cast<vec4*>(to);
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (; i + (U - 1) * step < count; i += U * step) {
    vec4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = base ? __builtin_nontemporal_load(src + i + u * step) : (vec4){0u, 0u, 0u, 0u};
#pragma unroll
    for (int u = 0; u < U; ++u) __builtin_nontemporal_store(v[u], dst + i + u * step);
  }
  for (; i < count; i += step) dst[i] = base ? src[i] : (vec4){0u, 0u, 0u, 0u};
}

template <int TT>
hipError_t lookup_run(const LookupArgs& a, int otype, unsigned grid, hipStream_t st) {
  if (otype == kBF16) hipLaunchKernelGGL((lookup_kernel<TT, kBF16>), dim3(grid), dim3(kLookNT), 0, st, a);
  else hipLaunchKernelGGL((lookup_kernel<TT, kF32>), dim3(grid), dim3(kLookNT), 0, st, a);
  return hipGetLastError();
}

template <int OT>
hipError_t sums_run(const SumArgs& a, int dytype, unsigned fill_groups, hipStream_t st) {
  const dim3 all((unsigned)a.sum_groups + fill_groups);
  if (dytype == kBF16) hipLaunchKernelGGL((token_rows_kernel<kBF16, OT>), all, dim3(kLookNT), 0, st, a);
  else hipLaunchKernelGGL((token_rows_kernel<kF32, OT>), all, dim3(kLookNT), 0, st, a);
  if (a.chunks > 1) {
    // As many chunks a workgroup as leave 16 workgroups a compute unit, and no more than a wave has lanes.
    const int64_t slices = (a.octets + kJoinLanes - 1) / kJoinLanes;
    int64_t joins = (slices * a.chunks + persistent_groups(16) - 1) / persistent_groups(16);
    if (joins > kJoinLanes) joins = kJoinLanes;
    hipLaunchKernelGGL(token_joins_kernel<OT>, dim3((unsigned)((a.chunks + joins - 1) / joins * slices)), dim3(kLookNT), 0, st, a, (int)joins);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fill_rows(const void* base, void* to, int64_t words, hipStream_t stream) {
  int64_t groups = (words + 1023) / 1024;
  if (groups > persistent_groups(8)) groups = persistent_groups(8);
  if (groups == 0) return hipSuccess;
  hipLaunchKernelGGL(fill_rows_kernel, dim3((unsigned)groups), dim3(256), 0, stream, reinterpret_cast<const uint4*>(base),
                     reinterpret_cast<uint4*>(to), words);
  return hipGetLastError();
}

hipError_t launch_embedding(const void* tokens, bool wide, int64_t rows, const void* table, int ttype, int64_t vocab,
                            int64_t cols, const float* sinv, float scale, void* out, int otype, hipStream_t stream) {
  LookupArgs a{tokens, table, sinv, out, rows, vocab, cols / 8, scale, 0, 1, wide};
  a.lanes = row_lanes(a.octets);
  int64_t blocks = (rows * a.lanes + kLookNT - 1) / kLookNT;
  if (blocks > persistent_groups(32)) blocks = persistent_groups(32);
  // A row over several workgroups only where there are too few rows to fill the device.
  while (a.slices * a.lanes < a.octets && blocks * a.slices < persistent_groups(2)) ++a.slices;
  const unsigned grid = (unsigned)(blocks * a.slices);
  if (ttype == kF32) return lookup_run<kF32>(a, otype, grid, stream);
  if (ttype == kBF16) return lookup_run<kBF16>(a, otype, grid, stream);
  if (ttype == kTableE4M3) return lookup_run<kTableE4M3>(a, otype, grid, stream);
  return lookup_run<kTableE5M2>(a, otype, grid, stream);
}

hipError_t launch_embedding_backward(const void* tokens, bool wide, int64_t rows, const void* dy, int dytype,
                                     int64_t vocab, int64_t cols, float scale, const void* base, void* dtable,
                                     int ttype, void* workspace, hipStream_t stream) {
  const int64_t words = cols / 8 * (ttype == kBF16 ? 1 : 2);  // of a table row
  if (rows == 0) return base != dtable ? launch_fill_rows(base, dtable, vocab * words, stream) : hipSuccess;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  auto take = [&]() {
    void* p = ws;
    ws += token_words(rows);
    return p;
  };
  SortArgs s{tokens, reinterpret_cast<uint32_t*>(take()), nullptr, rows, vocab, wide};
  s.places = reinterpret_cast<int32_t*>(take());
  const int64_t blocks = (rows + kSortBlock - 1) / kSortBlock;
  const int64_t in_block = rows < kSortBlock ? rows : kSortBlock;
  hipLaunchKernelGGL(rank_tokens_kernel, dim3((unsigned)((in_block + kSortGroup - 1) / kSortGroup), (unsigned)blocks), dim3(64 * kSortWaves), 0,
                     stream, s);
  SumArgs a{s.keys, s.places, dy, base, dtable, nullptr, rows, cols / 8, scale, (int)chunk_size(rows), 0, 0, 0, 0,
            vocab, (int)words, 1};
  if (blocks > 1) {
    uint32_t* keys = reinterpret_cast<uint32_t*>(take());
    int32_t* places = reinterpret_cast<int32_t*>(take());
    hipLaunchKernelGGL(merge_tokens_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, stream, s.keys, s.places,
                       rows, keys, places);
    a.keys = keys;
    a.places = places;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.partials = reinterpret_cast<float*>(ws);
  a.chunks = (int)chunk_count(rows);
  a.lanes = row_lanes(a.octets);
  a.slices = (int)((a.octets + a.lanes - 1) / a.lanes);
  a.sum_groups = (int)(((int64_t)a.chunks * a.lanes + kLookNT - 1) / kLookNT * a.slices);
  // Bands of about 32 KiB; eight filling workgroups a compute unit, if there is a band for each.
  while (a.band < 32 && a.band * words * 16 < 32768) a.band *= 2;
  int64_t fill = base != dtable ? (vocab + a.band - 1) / a.band : 0;
  if (fill > persistent_groups(8)) fill = persistent_groups(8);
  return ttype == kBF16 ? sums_run<kBF16>(a, dytype, (unsigned)fill, stream) : sums_run<kF32>(a, dytype, (unsigned)fill, stream);
}

}  // namespace fp8mi
