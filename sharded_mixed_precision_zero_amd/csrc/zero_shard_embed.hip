// zero_shard_embed.hip -- the embedding of tokens and the gradient of its
// table, on MI355X (gfx950) (declarations and the contract:
// include/zero_shard.h).
//
//   forward   y[t] = scale table[row(t)],  row(t) = ids[t] - first (zeros where
//             that is no row of this table)
//   backward  dtable[v] = scale sum of dy[t] over the tokens t of row v
//
// Both are HBM-bound.  The backward pass sorts the tokens by row (stably, so
// every row's sum runs over its tokens in order), then streams dy once in that
// order: a thread holds eight columns of a row's sum in registers.  No atomics:
// the same inputs give the same bits.
//
//   sort   tiles of tokens by counting: a token's place is the number of
//          tokens of its tile that come before it.  One launch, no passes over
//          digits that wait for each other.  Longer lists merge up to eight runs
//          at a time, each token finding its place by binary search in the other runs.
//   sum    pieces of kPiece sorted tokens.  A row is cut every `run` tokens, and
//          each part, or the whole of a shorter row, belongs to the piece that it
//          begins in, so that no piece does much more than its share however
//          the tokens are distributed.
//   join   the parts of those long rows, in order.
//
// A few tokens are one launch that sorts nothing (embed_few_kernel).

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "zero_shard.h"
#include "zs_rows.h"

namespace {

using namespace zs_dev;

constexpr int kThreads = 256;
// Tokens sorted by counting: up to kTile as one tile (whole passes: 8192 x 64 27 us, 30 as
// four tiles and a merge, 4097 x 64 23 and 29, 8192 x 5120 94 and 96), up to kOneMerge in
// tiles that one merge joins (16384 x 64: 35 us, 41 with smaller ones and two merges),
// beyond in small ones, since a tile costs the square of its length (65536 x 64: 66 us for
// 72, 300000 x 64: 197 for 237).
constexpr int kTile = 8192, kMiddleTile = 2048, kSmallTile = 1024;
constexpr int64_t kOneMerge = 8 * kMiddleTile;  // kRuns of them
constexpr int kPlaced = 32;       // of them, that a workgroup places
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRuns = 8;          // runs merged at a time
// Tokens of a long row's part: 8 where there are few tokens, 32 where the parts' traffic
// counts.  Between 1100 and 2048 tokens, which are sorted, both are as fast (19 to 73 us
// from 64 to 5120 columns, within 1 us of each other), but for one row of all tokens
// (2048 x 1024: 33 us with 8, 29 with 32); the order of sums that the border makes is stated.
constexpr int kRun = 32, kShortRun = 8;
constexpr int64_t kFew = 2048;
// Tokens that are not sorted, and the workgroups up to which that pays: each looks through
// all tokens (700 x 4096, 5600 of them: 13 us for 16; 512 x 8192, 8192 of them: 18 for
// 18; 300 x 16384, 9600: 22 for 18).
constexpr int kFewest = 1024;
constexpr int64_t kFewestGroups = 6000;
constexpr int kPiece = 8;         // tokens of a piece, and rows of dy in flight
// Waves that share a long row's parts: most workgroups find no such row, so few
// (65536 x 5120: 16 us with 4 waves, 24 with 8; one row of 8192 tokens 24 and 16).
constexpr int kJoinWaves = 4;
constexpr unsigned kWide = 48;    // pieces of eight columns from which a wave has one row's
constexpr int kEach = 4;          // pieces of eight columns of a forward thread
constexpr unsigned kNone = 0xffffffffu;  // sorts behind every row

struct Ids {
  const void *p;
  int64_t first, vocab, padding;
  int32_t bytes;    // of an id
  int32_t pad_set;  // an id that does not count
  __device__ __forceinline__ int64_t id(int64_t t) const {
    return bytes == 8 ? static_cast<const int64_t *>(p)[t]
                      : int64_t(static_cast<const int32_t *>(p)[t]);
  }
  // The table's row of an id, or -1.
  __device__ __forceinline__ int64_t row(int64_t i) const {
    // any two 64-bit numbers have a difference modulo 2^64
    const uint64_t r = uint64_t(i) - uint64_t(first);
    return r < uint64_t(vocab) ? int64_t(r) : -1;
  }
  // The same for the gradient's sorting: vocab for what counts nowhere.
  __device__ __forceinline__ unsigned key(int64_t t) const {
    const int64_t i = id(t), r = pad_set && i == padding ? -1 : row(i);
    return r < 0 ? unsigned(vocab) : unsigned(r);
  }
};

// Eight columns from `col` on of rows of `cols`, as they are loaded: where a row ends
// inside of them, its last eight, of which `skip` are not these; left: 8 or, of a row of
// fewer, all of it.  Nothing then waits for single elements on the way (8192 x 511
// bf16: 34 us for 46 backward).
template <bool TAIL>
struct Span {
  unsigned i;
  int skip = 0;
  int64_t left;
  __device__ __forceinline__ Span(unsigned col, int64_t cols) : i(col), left(cols - col) {
    if (TAIL && left > 0 && left < 8 && cols >= 8) {
      skip = 8 - int(left);
      i -= unsigned(skip);
      left = 8;
    }
  }
  template <bool ONCE, class T>
  __device__ __forceinline__ void get(Eight<T> &v, const void *row, bool in = true) const {
    v.template load<TAIL, ONCE>(row, i, in ? left : 0);
  }
  template <bool ONCE, class T>
  __device__ __forceinline__ void put(const Eight<T> &v, void *row) const {
    if (!TAIL || skip == 0) v.template store<TAIL, ONCE>(row, i, left);
    else store_last(v, row, i, skip);
  }
};

struct FwdArgs {
  Ids ids;
  int64_t tokens, cols, ld_table, ld_y;
  const void *table;
  void *y;
  float scale;
  unsigned per;  // pieces of eight columns
};

// A workgroup takes kEach * kThreads pieces of eight columns one after another,
// whatever token they belong to.
template <class TW, class TY, bool TAIL>
__global__ void __launch_bounds__(kThreads) embed_kernel(const FwdArgs A) {
  const unsigned base = blockIdx.x * (kThreads * kEach), t0 = base / A.per;  // below 2^31
  const unsigned c0 = base - t0 * A.per;
  int64_t token[kEach], row[kEach];
  unsigned col[kEach];
  Eight<TW> w[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const unsigned q = c0 + unsigned(k * kThreads) + threadIdx.x;
    const unsigned up = q / A.per;
    token[k] = int64_t(t0) + up;
    col[k] = (q - up * A.per) * 8;
    row[k] = token[k] < A.tokens ? A.ids.row(A.ids.id(token[k])) : -1;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    Span<TAIL>(col[k], A.cols)
        .template get<false>(w[k], row_of<TW>(A.table, row[k], A.ld_table), row[k] >= 0);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (token[k] >= A.tokens) break;
    float v[8];
    Eight<TY> y;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = w[k].get(e) * A.scale;
      // a binary32 number, not the first half of an instruction that rounds the
      // exact product to binary16
      asm volatile("" : "+v"(v[e]));
    }
    y.set(v);
    // past the caches, which the table should stay in (65536 x 5120: 189 us for 195)
    Span<TAIL>(col[k], A.cols).template put<!TAIL>(y, row_of<TY>(A.y, token[k], A.ld_y));
  }
}

struct SortArgs {
  Ids ids;
  int64_t tokens;
  int32_t tile, groups;  // of kPlaced tokens, of a workgroup
  unsigned *keys;  // rows, sorted; vocab: no row of this table
  int *order;      // their tokens
};

// A workgroup places `groups` times kPlaced tokens.  Its waves share the tile's tokens
// in chunks of 64; in each wave two lanes take a token, one for either half of a
// chunk (with 64 tokens a wave, half of the CUs had nothing to do with 8192 of them
// and each of the others read all keys out of LDS twice as often: 17 us for 10).
// Of equal rows the earlier token comes first: tokens of earlier chunks count up to
// the same row, those of later ones below it.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs A) {
  __shared__ __align__(16) unsigned keys[kTile];
  __shared__ unsigned counts[kSortWaves][kPlaced];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned blocks = unsigned(A.tile / (kPlaced * A.groups));  // of a tile
  const int64_t tile = int64_t(blockIdx.x / blocks) * A.tile;
  const int64_t left = A.tokens - tile;
  const int n = left < A.tile ? int(left) : A.tile, chunks = (n + 63) / 64;
#pragma unroll
  for (int i = 0; i < kTile / kSortThreads; ++i) {
    const int s = i * kSortThreads + int(threadIdx.x);
    if (s < chunks * 64) keys[s] = s < n ? A.ids.key(tile + s) : kNone;
  }
  __syncthreads();
  for (int g = 0; g < A.groups; ++g) {
    const int own = (int(blockIdx.x % blocks) * A.groups + g) * kPlaced;  // in the tile
    if (own >= n) break;
    const int at = own + lane % kPlaced, half = lane / kPlaced * 32;
    const unsigned mine = keys[at];
    unsigned count = 0;
    for (int c = wave; c < chunks; c += kSortWaves) {
      const u32x4 *from = reinterpret_cast<const u32x4 *>(keys + c * 64 + half);
      if (c != own / 64) {
        const unsigned below = c < own / 64 ? mine + 1 : mine;  // of kNone: anything
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u32x4 k = from[j];
#pragma unroll
          for (int e = 0; e < 4; ++e) count += k[e] < below ? 1u : 0u;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u32x4 k = from[j];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            count += k[e] < mine || (k[e] == mine && half + j * 4 + e < at % 64) ? 1u : 0u;
        }
      }
    }
    count += __shfl_xor(count, 32, 64);
    if (lane < kPlaced) counts[wave][lane] = count;
    __syncthreads();
    if (wave == 0 && lane < kPlaced && at < n) {
      unsigned place = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) place += counts[w][lane];
      A.keys[tile + place] = mine;
      A.order[tile + place] = int(tile + at);
    }
    __syncthreads();  // before the counts of the next group
  }
}

struct MergeArgs {
  int32_t tokens, run;  // sorted runs of this length
  const unsigned *keys;
  const int *order;
  unsigned *keys_out;
  int *order_out;
};

// A token's place among up to kRuns runs: its place in its own and, in each
// other, the number of tokens that come before it.  The searches run side by side, all
// loads of a step in flight (with branches around them 16000 tokens took 21 us for 8).
__global__ void __launch_bounds__(kThreads) embed_merge_kernel(const MergeArgs A) {
  const int i = int(blockIdx.x) * kThreads + int(threadIdx.x);
  if (i >= A.tokens) return;
  const int group = i / (A.run * kRuns) * (A.run * kRuns), own = (i - group) / A.run;
  const unsigned key = A.keys[i];
  int lo[kRuns], hi[kRuns];
#pragma unroll
  for (int q = 0; q < kRuns; ++q) {
    const int from = group + q * A.run, to = from + A.run;
    lo[q] = from < A.tokens ? from : A.tokens;
    hi[q] = to < A.tokens ? to : A.tokens;
    if (q == own) hi[q] = lo[q];
  }
  for (int span = A.run; span > 0; span >>= 1) {
    unsigned k[kRuns];
#pragma unroll
    for (int q = 0; q < kRuns; ++q) {
      const int mid = (lo[q] + hi[q]) >> 1;
      k[q] = A.keys[mid < A.tokens ? mid : i];  // all of them before any is looked at
    }
#pragma unroll
    for (int q = 0; q < kRuns; ++q) {
      const int mid = (lo[q] + hi[q]) >> 1;
      // an earlier run's equals come first
      const bool before = q < own ? k[q] <= key : k[q] < key;
      const bool open = lo[q] < hi[q];
      lo[q] = open && before ? mid + 1 : lo[q];
      hi[q] = open && !before ? mid : hi[q];
    }
  }
  int place = i - own * A.run;  // its place in its run, behind the group's start
#pragma unroll
  for (int q = 0; q < kRuns; ++q) {
    const int from = group + q * A.run;
    if (q != own && from < A.tokens) place += lo[q] - from;
  }
  A.keys_out[place] = key;
  A.order_out[place] = A.order[i];
}

struct SumArgs {
  int64_t tokens, vocab, cols, ld_dy, ld_out;
  const unsigned *keys;
  const int *order;
  const void *dy;
  void *out;
  float *part;  // [2 tokens / run][per * 8], see part_of
  int32_t run;  // tokens of a long row's part
  float scale;
  int32_t add;        // to what is there
  unsigned per;       // pieces of eight columns
  unsigned waves;     // of a piece of tokens
  int64_t sum_blocks; // workgroups that sum; the others clear
  int32_t rows;       // that a workgroup clears
  int32_t flat;       // 1: they are one stretch of whole sixteen bytes
};

// The first of keys[lo, hi) that is not below `key`, hi if none: eight looks side by
// side, each time an eighth is left.
__device__ __forceinline__ int64_t first_not_below(const unsigned *keys, int64_t lo, int64_t hi,
                                                   unsigned key) {
  while (lo < hi) {
    const int64_t span = hi - lo;
    int below = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) below += keys[lo + (span * q >> 3)] < key ? 1 : 0;
    if (below == 0) return lo;
    if (below < 8) hi = lo + (span * below >> 3);
    lo += (span * (below - 1) >> 3) + 1;
  }
  return lo;
}

// Where the part of a long row that begins at sorted token `at` is kept.  Of the parts
// that begin within `run` tokens one at most is its row's first (its row goes on
// for all of them) and one at most is not.
__device__ __forceinline__ int64_t part_of(const SumArgs &A, int64_t at, bool first) {
  return (A.run == kRun ? at / kRun : at / kShortRun) * 2 + (first ? 1 : 0);
}

// A row's sum, scaled and joined with what is there, into the table's gradient.
template <class TG, bool TAIL>
__device__ __forceinline__ void put_row(const SumArgs &A, unsigned row, unsigned col,
                                        float (&v)[8]) {
  void *to = row_of<TG>(A.out, row, A.ld_out);
  const Span<TAIL> span(col, A.cols);
  Eight<TG> w;
  if (A.add) {
    span.template get<false>(w, to);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(A.scale, v[e], w.get(e));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= A.scale;
  }
  w.set(v);
  span.template put<false>(w, to);
}

// Rows without tokens become zeros: A.rows of them from `block` times that on.
// mark(row, rows, used) says which have some.  ONCE: past the caches, where dy streams
// as well (8192 x 5120: 93 us for 98; with few tokens 14 us for 17 the other way).
template <class TG, bool TAIL, bool ONCE, class F>
__device__ __forceinline__ void clear_rows(const SumArgs &A, int64_t block, F mark) {
  __shared__ int used[kThreads];
  const int64_t r0 = block * A.rows;
  const int rows = int(A.vocab - r0 < A.rows ? A.vocab - r0 : A.rows);
  mark(r0, rows, used);
  using raw = typename TG::raw;
  if (A.flat && !__syncthreads_or(int(threadIdx.x) < rows && used[threadIdx.x])) {
    // one stretch of memory, from a multiple of sixteen bytes on
    char *to = static_cast<char *>(A.out) + r0 * A.cols * int64_t(sizeof(raw));
    const int64_t bytes = rows * A.cols * int64_t(sizeof(raw));
#pragma unroll 4
    for (int64_t i = threadIdx.x * 16; i + 16 <= bytes; i += kThreads * 16) {
      if constexpr (ONCE)
        __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4 *>(to + i));
      else
        *reinterpret_cast<u32x4 *>(to + i) = u32x4{0, 0, 0, 0};
    }
    const int64_t rest = bytes / 16 * 16 + threadIdx.x * int64_t(sizeof(raw));
    if (rest < bytes) *reinterpret_cast<raw *>(to + rest) = raw(0);
    return;
  }
  // in elements, or in sixteen bytes side by side
  constexpr int64_t kUnit = TAIL ? 1 : 16 / sizeof(raw);
  const int64_t units = A.cols / kUnit;
  // `across` threads a row, several rows at a time where rows are short
  const unsigned across = units < kThreads ? unsigned(units) : kThreads;
  const unsigned sub = threadIdx.x / across, subs = kThreads / across;
  if (sub >= subs) return;
  for (int r = int(sub); r < rows; r += int(subs)) {
    if (used[r]) continue;
    raw *to = static_cast<raw *>(row_of<TG>(A.out, r0 + r, A.ld_out));
    for (int64_t c = threadIdx.x - sub * across; c < units; c += across) {
      if constexpr (TAIL) to[c] = raw(0);
      else if constexpr (ONCE)
        __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4 *>(to) + c);
      else reinterpret_cast<u32x4 *>(to)[c] = u32x4{0, 0, 0, 0};
    }
  }
}

// A few tokens are not sorted: a workgroup for each token and 64 pieces of
// eight columns looks through all ids, and if none before it is the same it sums that
// row, by the same parts as below, a stretch of them a wave (333 x 1601: one launch of
// 7.0 us for three that took 18).
template <class TY, class TG, bool TAIL>
__global__ void __launch_bounds__(kThreads) embed_few_kernel(const SumArgs A, const Ids ids) {
  const int n = int(A.tokens), lane = threadIdx.x & 63;
  if (int64_t(blockIdx.x) >= A.sum_blocks) {
    clear_rows<TG, TAIL, false>(A, int64_t(blockIdx.x) - A.sum_blocks,
                         [&](int64_t r0, int rows, int *used) {
                           used[threadIdx.x] = 0;
                           __syncthreads();
                           for (int i = threadIdx.x; i < n; i += kThreads) {
                             const int64_t r = int64_t(ids.key(i)) - r0;
                             if (r >= 0 && r < rows) used[r] = 1;
                           }
                           __syncthreads();
                         });
    return;
  }
  __shared__ uint16_t lists[kJoinWaves][kFewest];
  __shared__ float sums[kJoinWaves][8][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t *list = lists[wave];  // every wave its own: no barrier
  const int token = int(blockIdx.x / A.waves);
  const unsigned c = (blockIdx.x - unsigned(token) * A.waves) * 64 + lane, col = c * 8;
  const int64_t mine = ids.id(token), columns = A.cols - col;
  int64_t all[kFewest / 64];
#pragma unroll
  for (int q = 0; q < kFewest / 64; ++q) {
    const int i = q * 64 + lane;
    all[q] = i < n ? ids.id(i) : 0;
  }
  const unsigned key = ids.key(token);
  if (key >= unsigned(A.vocab)) return;
  int total = 0;
#pragma unroll
  for (int q = 0; q < kFewest / 64; ++q) {
    const int i = q * 64 + lane;
    const bool same = i < n && all[q] == mine;
    const uint64_t mask = __ballot(same);
    if (same) list[total + __popcll(mask & ((uint64_t(1) << lane) - 1))] = uint16_t(i);
    total += __popcll(mask);
  }
  // LDS of this wave alone
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  if (list[0] != token) return;  // the row is an earlier one's
  const int parts = (total + kShortRun - 1) / kShortRun;
  const int each = (parts + kJoinWaves - 1) / kJoinWaves;
  const int lo = wave * each, hi = lo + each < parts ? lo + each : parts;
  const Span<TAIL> span(col, A.cols);
  float acc[8] = {};
  for (int p = lo; p < hi; ++p) {
    Eight<TY> v[kShortRun];
#pragma unroll
    for (int j = 0; j < kShortRun; ++j) {
      const int at = p * kShortRun + j;
      const int t = __builtin_amdgcn_readfirstlane(int(list[at < total ? at : 0]));
      span.template get<!TAIL>(v[j], row_of<TY>(A.dy, t, A.ld_dy), at < total);
    }
    float part[8] = {};
#pragma unroll
    for (int j = 0; j < kShortRun; ++j)
      if (p * kShortRun + j < total)
#pragma unroll
        for (int e = 0; e < 8; ++e) part[e] += v[j].get(e);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += part[e];
  }
  if (parts > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wave][e][lane] = acc[e];
    __syncthreads();
  }
  if (wave != 0 || columns <= 0) return;
  if (parts > 1)
    for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += sums[w][e][lane];
  put_row<TG, TAIL>(A, key, col, acc);
}

// The sorted lists are not written while they are read here: the scalar units may
// load from them where the place is the whole wave's.
template <class T>
__device__ __forceinline__ const T __attribute__((address_space(4))) *sorted(const void *p) {
  return (const T __attribute__((address_space(4))) *)uintptr_t(p);
}

// kPiece sorted places from `at` on, a multiple of kPiece: their tokens, and a bit for each
// that is of another row than the place before it (`prev`: the first one's) or of
// the row `key`; the first `live` of them are of rows of the table.
struct Places {
  int token[kPiece];
  unsigned begins, same, first, last;
  int live;
  __device__ __forceinline__ void load(const SumArgs &A, int64_t at) {
    if (at + kPiece <= A.tokens) {
#pragma unroll
      for (int q = 0; q < kPiece / 4; ++q) {
        const u32x4 k = *sorted<u32x4>(A.keys + at + q * 4);
        const u32x4 t = *sorted<u32x4>(A.order + at + q * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          row[q * 4 + e] = k[e];
          token[q * 4 + e] = int(t[e]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        row[e] = at + e < A.tokens ? *sorted<unsigned>(A.keys + at + e) : kNone;
        token[e] = at + e < A.tokens ? *sorted<int>(A.order + at + e) : 0;
      }
    }
  }
  __device__ __forceinline__ void look(const SumArgs &A, unsigned prev, unsigned key) {
    begins = same = 0;
    live = 0;
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      begins |= row[e] != (e ? row[e - 1] : prev) ? 1u << e : 0u;
      same |= row[e] == key ? 1u << e : 0u;
      live += row[e] < unsigned(A.vocab) ? 1 : 0;
    }
    first = row[0];
    last = row[kPiece - 1];
  }
  unsigned row[kPiece];  // until look
};

// WAVES: a wave has one piece, and what concerns its rows is the scalar units' work; a
// piece has A.waves of them (65536 x 5120: 205 us for 319 with each thread on its own).
// Rows of too few columns to fill a wave share waves: a thread is any piece's.
template <class TY, class TG, bool TAIL, bool WAVES>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const SumArgs A) {
  if (int64_t(blockIdx.x) >= A.sum_blocks) {
    clear_rows<TG, TAIL, true>(A, int64_t(blockIdx.x) - A.sum_blocks,
                         [&](int64_t r0, int rows, int *used) {
                           if (int(threadIdx.x) < rows) {
                             const unsigned key = unsigned(r0 + threadIdx.x);
                             const int64_t at = first_not_below(A.keys, 0, A.tokens, key);
                             used[threadIdx.x] = at < A.tokens && A.keys[at] == key;
                           }
                           __syncthreads();
                         });
    return;
  }
  unsigned piece, col;
  if constexpr (WAVES) {
    const unsigned wave =
        __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
    piece = wave / A.waves;
    col = ((wave - piece * A.waves) * 64 + (threadIdx.x & 63)) * 8;
  } else {
    const unsigned id = blockIdx.x * kThreads + threadIdx.x;  // below 2^31
    piece = id / A.per;
    col = (id - piece * A.per) * 8;
  }
  const int64_t width = int64_t(A.per) * 8, columns = A.cols - col;
  const Span<TAIL> span(col, A.cols);
  const int64_t from = int64_t(piece) * kPiece, to = from + kPiece;
  if (from >= A.tokens) return;
  // this piece's places, the next one's, and how many of the kRun before it (a multiple
  // of any run) are of its first row: loads side by side
  Places now, next;
  now.load(A, from);
  next.load(A, to);
  int before = 0;
#pragma unroll
  for (int k = kPiece; k <= kRun; k += kPiece)
    if (from >= k) {
#pragma unroll
      for (int h = 0; h < kPiece / 4; ++h) {
        const u32x4 v = *sorted<u32x4>(A.keys + from - k + h * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) before += v[e] == now.row[0] ? 1 : 0;
      }
    }
  now.look(A, before ? now.row[0] : kNone, now.row[0]);
  next.look(A, now.last, now.last);
  // Where a part may begin: at a row's first place, and where the next part of a row that
  // began before this piece does, if that row is still there.
  unsigned starts = now.begins, mine = now.begins ? ~0u << __builtin_ctz(now.begins) : 0u;
  if (before) {
    const int64_t row0 =
        before < kRun ? from - before : first_not_below(A.keys, 0, from - kRun, now.first);
    const int64_t part = row0 + ((from - row0 + A.run - 1) & -int64_t(A.run));
    if (part < to && (now.same >> (part - from) & 1)) {
      starts |= 1u << (part - from);
      mine = ~0u << (part - from);
    }
  }
  mine &= (1u << now.live) - 1u;  // places that are summed here
  if (!mine) return;
  int64_t start = 0;                   // of the part being summed
  bool active = false, whole = false;  // whole: at its row's first place
  float acc[8];
  for (int64_t at = from;; at += kPiece) {
    Eight<TY> v[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const bool take = mine >> j & 1;
      span.template get<!TAIL>(v[j], row_of<TY>(A.dy, take ? now.token[j] : 0, A.ld_dy), take);
    }
    int cur = 0;
    for (;;) {
      if (!active) {
        const unsigned left = at == from ? starts & mine & ~0u << cur : 0u;
        if (!left) return;
        cur = __builtin_ctz(left);
        start = at + cur;
        whole = now.begins >> cur & 1;
        active = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
      }
      // to the next row, behind the table's rows, or to the part's end
      int end = now.live;
      const unsigned row = start == at + cur ? now.begins & ~1u << cur : now.begins & ~0u << cur;
      if (row && __builtin_ctz(row) < end) end = __builtin_ctz(row);
      if (start + A.run - at < end) end = int(start + A.run - at);
#pragma unroll
      for (int j = 0; j < kPiece; ++j)
        if (j >= cur && j < end) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[j].get(e);
        }
      if (end == kPiece) break;
      const unsigned key = *sorted<unsigned>(A.keys + start);
      if (columns <= 0) {
        // no columns of this thread
      } else if (whole && (end == now.live || (row >> end & 1))) {
        put_row<TG, TAIL>(A, key, col, acc);
      } else {
        Eight<F32> part;
        part.set(acc);
        part.template store<false>(A.part + part_of(A, start, whole) * width, col, 8);
      }
      active = false;
      cur = end;
      if (at != from || end == now.live) return;
    }
    // the part goes on, or ends with these places
    now = next;
    const int64_t left = start + A.run - (at + kPiece);
    mine = now.same & (now.begins & 1 ? 0u : ~0u);
    if (now.begins >> 1) mine &= (1u << __builtin_ctz(now.begins & ~1u)) - 1u;
    if (left < kPiece) mine &= (1u << left) - 1u;
    if (left >= kPiece) {  // also to see whether the row ends with its part
      next.load(A, at + 2 * kPiece);
      next.look(A, now.last, now.last);
    }
  }
}

// The parts of the row that begins among the `run` places from blockIdx.x run on and
// goes on for more than `run`, if there is one: each wave adds a stretch of them, then
// the waves' sums are added in order.
template <class TG, bool TAIL>
__global__ void __launch_bounds__(64 * kJoinWaves) embed_join_kernel(const SumArgs A) {
  __shared__ float sums[kJoinWaves][8][64];
  const int run = A.run;
  const int64_t from = int64_t(blockIdx.x) * run, to = from + run;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (to >= A.tokens) return;
  // lanes: the place before, the run's places, the one behind
  const int64_t look = from - 1 + lane;
  const unsigned near = lane < run + 2 && look >= 0 ? A.keys[look] : kNone;
  const unsigned key = __builtin_amdgcn_readlane(near, run);
  if (key >= unsigned(A.vocab)) return;
  const uint64_t same = __ballot(near == key);
  if (!(same >> (run + 1) & 1) || (same & 1)) return;  // ends in here, or began before
  const int64_t start = from - 1 + __builtin_ctzll(same);
  if (start + run >= A.tokens || A.keys[start + run] != key) return;
  // a part a lane: how many begin within the row
  int64_t parts = 1;
  for (;;) {
    const int64_t at = start + (parts + lane) * run;
    const uint64_t more = __ballot(at < A.tokens && A.keys[at < A.tokens ? at : start] == key);
    parts += __builtin_popcountll(more);
    if (more != ~uint64_t(0)) break;
  }
  const unsigned c = blockIdx.y * 64 + lane, col = c * 8;
  const int64_t width = int64_t(A.per) * 8, each = (parts + kJoinWaves - 1) / kJoinWaves;
  float acc[8] = {};
  if (c < A.per) {
    const int64_t lo = wave * each, hi = lo + each < parts ? lo + each : parts;
#pragma unroll 8
    for (int64_t j = lo; j < hi; ++j) {
      Eight<F32> v;
      v.template load<false>(A.part + part_of(A, start + j * run, j == 0) * width, col, 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v.get(e);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[wave][e][lane] = acc[e];
  __syncthreads();
  if (wave != 0 || c >= A.per) return;
  for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += sums[w][e][lane];
  put_row<TG, TAIL>(A, key, col, acc);
}

// ------------------------------------------------------------------- host

bool desc_ok(const zs_embedding_desc *d) {
  if (!d || d->tokens < 0 || d->tokens > ZS_EMBEDDING_MAX_TOKENS) return false;
  if (d->vocab < 1 || d->vocab > ZS_EMBEDDING_MAX_VOCAB) return false;
  if (d->first > INT64_MAX - (d->vocab - 1)) return false;  // its last id
  if (d->cols < 1 || d->cols > (INT64_C(1) << 20) || d->pad_set < 0 || d->pad_set > 1)
    return false;
  // what the kernels count in 32 bits, and the threads that a launch takes
  if (d->tokens * up(d->cols, 8) >= INT64_C(1) << 34) return false;
  if (d->vocab * d->cols > INT64_C(1) << 37) return false;
  if (d->id_bytes != 4 && d->id_bytes != 8) return false;
  if (!dtype_size(d->dtype) || d->accumulate < 0 || d->accumulate > 1) return false;
  for (const int32_t t : {d->table_dtype, d->grad_dtype})
    if (t != ZS_F32 && t != d->dtype) return false;
  if (!std::isfinite(d->scale)) return false;
  for (const int64_t ld : {d->ld_table, d->ld_y, d->ld_dy, d->ld_dtable})
    if (ld != 0 && (ld < d->cols || ld > (INT64_C(1) << 31))) return false;
  return true;
}

unsigned per_of(const zs_embedding_desc &d) { return unsigned((d.cols + 7) / 8); }
bool unsorted(const zs_embedding_desc &d) {
  return d.tokens <= kFewest && d.tokens * ((per_of(d) + 63) / 64) <= kFewestGroups;
}
int run_of(const zs_embedding_desc &d) { return d.tokens <= kFew ? kShortRun : kRun; }

// Workspace: the sorted rows and tokens (twice where runs are merged), the
// parts of long rows.
struct Plan {
  int64_t keys[2] = {}, order[2] = {}, part = 0, bytes = 0;
  bool merged = false;
  explicit Plan(const zs_embedding_desc &d) {
    if (unsorted(d)) return;
    const int64_t list = up(d.tokens * 4, 256), runs = (d.tokens + run_of(d) - 1) / run_of(d);
    merged = d.tokens > kTile;
    keys[0] = 0;
    order[0] = list;
    keys[1] = merged ? 2 * list : 0;
    order[1] = merged ? 3 * list : list;
    part = merged ? 4 * list : 2 * list;
    bytes = part + (runs > 1 ? runs * 2 * per_of(d) * 8 * 4 : 0);
  }
};

template <class F>
int by_type(int32_t narrow, int32_t other, F f) {
  if (narrow == ZS_F32) return f(F32{}, F32{});
  if (narrow == ZS_BF16) return other == ZS_F32 ? f(Bf16{}, F32{}) : f(Bf16{}, Bf16{});
  return other == ZS_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
}

template <class F>
int by_tail(bool tail, F f) {
  return tail ? f(std::true_type{}) : f(std::false_type{});
}

Ids ids_of(const zs_embedding_desc &d, const void *ids) {
  return Ids{ids, d.first, d.vocab, d.padding, d.id_bytes, d.pad_set};
}

int sort(const zs_embedding_desc &d, const Plan &p, const void *ids, char *ws, hipStream_t st,
         int &turn) {
  const auto keys = [&](int k) { return reinterpret_cast<unsigned *>(ws + p.keys[k]); };
  const auto order = [&](int k) { return reinterpret_cast<int *>(ws + p.order[k]); };
  turn = 0;
  const int32_t tile = d.tokens <= kTile       ? kTile
                       : d.tokens <= kOneMerge ? kMiddleTile
                                               : kSmallTile;
  // a workgroup or two for each CU, at most a tile's
  int32_t groups = 1;
  while (d.tokens > int64_t(512) * kPlaced * groups && groups < tile / kPlaced) groups *= 2;
  const int64_t blocks = (d.tokens + kPlaced * groups - 1) / (kPlaced * groups);
  hipLaunchKernelGGL(embed_sort_kernel, dim3(unsigned(blocks)), dim3(kSortThreads), 0, st,
                     SortArgs{ids_of(d, ids), d.tokens, tile, groups, keys(0), order(0)});
  for (int64_t run = tile; run < d.tokens; run *= kRuns, turn ^= 1) {
    hipLaunchKernelGGL(embed_merge_kernel, dim3(unsigned((d.tokens + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, st,
                       MergeArgs{int32_t(d.tokens), int32_t(run), keys(turn), order(turn), keys(turn ^ 1),
                                 order(turn ^ 1)});
  }
  return launched();
}

}  // namespace

extern "C" {

int zero_shard_embedding(const zs_embedding_desc *d, const void *ids, const void *table, void *y) {
  if (!desc_ok(d)) return ZS_EINVAL;
  if (d->tokens == 0) return ZS_OK;
  if (!ids || !table || !y) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), tsize = dtype_size(d->table_dtype);
  if (!aligned(ids, d->id_bytes) || !aligned(table, tsize) || !aligned(y, size)) return ZS_EALIGN;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  const FwdArgs A{ids_of(*d, ids), d->tokens, d->cols, ld(d->ld_table), ld(d->ld_y), table, y,
                  d->scale, per_of(*d)};
  const int64_t blocks = (A.tokens * A.per + kThreads * kEach - 1) / (kThreads * kEach);
  if (const int rc = device_is_gfx950()) return rc;
  return by_type(d->dtype, d->table_dtype, [&](auto ty, auto tw) {
    return by_tail(d->cols % 8 != 0, [&](auto tail) {
      hipLaunchKernelGGL((embed_kernel<decltype(tw), decltype(ty), tail.value>),
                         dim3(unsigned(blocks)), dim3(kThreads), 0,
                         static_cast<hipStream_t>(d->stream), A);
      return launched();
    });
  });
}

int64_t zero_shard_embedding_workspace(const zs_embedding_desc *d) {
  return desc_ok(d) ? Plan(*d).bytes : -1;
}

int zero_shard_embedding_bwd(const zs_embedding_desc *d, const void *ids, const void *dy,
                             void *dtable, void *workspace, int64_t workspace_bytes) {
  if (!desc_ok(d)) return ZS_EINVAL;
  if (d->tokens == 0 && d->accumulate) return ZS_OK;
  if (!dtable) return ZS_EINVAL;
  const Plan p(*d);
  if (d->tokens > 0 && (!ids || !dy)) return ZS_EINVAL;
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), gsize = dtype_size(d->grad_dtype);
  if (!aligned(ids, d->id_bytes) || !aligned(dy, size) || !aligned(dtable, gsize) ||
      !aligned(workspace, 256))
    return ZS_EALIGN;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  const int run = run_of(*d);
  const int64_t pieces = (d->tokens + kPiece - 1) / kPiece, runs = (d->tokens + run - 1) / run;
  SumArgs A{};
  A.tokens = d->tokens;
  A.vocab = d->vocab;
  A.cols = d->cols;
  A.ld_dy = ld(d->ld_dy);
  A.ld_out = ld(d->ld_dtable);
  A.dy = dy;
  A.out = dtable;
  A.run = run;
  A.scale = d->scale;
  A.add = d->accumulate;
  A.per = per_of(*d);
  A.waves = (A.per + 63) / 64;
  const bool wide = A.per >= kWide, few = unsorted(*d);
  const int64_t threads = wide ? int64_t(A.waves) * 64 : A.per;
  A.sum_blocks = few ? d->tokens * A.waves : (pieces * threads + kThreads - 1) / kThreads;
  // A workgroup clears about 32 KiB, to which its searches are little, or 16 where they are
  // quick (333 x 1601 64 KiB: 8.2 us for 7.0; 8192 x 5120 the same from 16 to 256).
  const int64_t stretch = few ? 16384 : 32768;
  A.rows = int32_t((stretch + d->cols * gsize - 1) / (d->cols * gsize));
  while (d->vocab > (INT64_C(1) << 22) * A.rows) A.rows *= 2;  // what a launch takes
  if (A.rows > kThreads) A.rows = kThreads;
  if (d->cols * gsize % 16) A.rows = int32_t(up(A.rows, 16 / gsize));
  A.flat = A.ld_out == d->cols && aligned(dtable, 16);
  const int64_t clear = d->accumulate ? 0 : (d->vocab + A.rows - 1) / A.rows;
  if (const int rc = device_is_gfx950()) return rc;
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  char *ws = static_cast<char *>(workspace);
  if (!few) {
    int turn = 0;
    if (const int rc = sort(*d, p, ids, ws, st, turn)) return rc;
    A.keys = reinterpret_cast<const unsigned *>(ws + p.keys[turn]);
    A.order = reinterpret_cast<const int *>(ws + p.order[turn]);
    A.part = reinterpret_cast<float *>(ws + p.part);
  }
  const bool even = rows_even(dy, A.ld_dy, size) && rows_even(dtable, A.ld_out, gsize);
  return by_type(d->dtype, d->grad_dtype, [&](auto ty, auto tg) {
    using TG = decltype(tg);
    return by_tail(d->cols % 8 != 0 || !even, [&](auto tail) {
      const dim3 grid(unsigned(A.sum_blocks + clear));
      if (few) {
        hipLaunchKernelGGL((embed_few_kernel<decltype(ty), TG, tail.value>), grid, dim3(kThreads),
                           0, st, A, ids_of(*d, ids));
        return launched();
      }
      if (wide)
        hipLaunchKernelGGL((embed_sum_kernel<decltype(ty), TG, tail.value, true>), grid,
                           dim3(kThreads), 0, st, A);
      else
        hipLaunchKernelGGL((embed_sum_kernel<decltype(ty), TG, tail.value, false>), grid,
                           dim3(kThreads), 0, st, A);
      if (runs > 1)
        hipLaunchKernelGGL((embed_join_kernel<TG, tail.value>),
                           dim3(unsigned(runs), (A.per + 63) / 64), dim3(64 * kJoinWaves), 0, st,
                           A);
      return launched();
    });
  });
}

}  // extern "C"
