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
//   sort   tiles of kTile tokens by counting: a token's place is the number of
//          tokens of its tile that come before it.  One launch, no passes over
//          digits that wait for each other.  Longer lists merge up to eight runs
//          at a time, each token finding its place by binary search in the other runs.
//   sum    pieces of kPiece sorted tokens.  A row is cut every kRun tokens, and
//          each part, or the whole of a shorter row, belongs to the piece that it
//          begins in, so that no piece does much more than its share however
//          the tokens are distributed.
//   join   the parts of those long rows, in order.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "zero_shard.h"
#include "zs_rows.h"

namespace {

using namespace zs_dev;

constexpr int kThreads = 256;
// Tokens sorted by counting: up to kTile as one tile (8192: 10 us, 6 and 11 as four
// tiles and a merge), more in tiles of kSmallTile, whose cost does not grow with the
// square of their length (65536: 371 us the whole pass, 418 with long tiles).
constexpr int kTile = 8192, kSmallTile = 2048;
constexpr int kPlaced = 32;       // of them, that a workgroup places
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRuns = 8;          // runs merged at a time
constexpr int kRun = 32;          // tokens of a long row's part
constexpr int kPiece = 8;         // tokens of a piece, and rows of dy in flight
constexpr int kJoinWaves = 8;
constexpr int kEach = 4;          // pieces of eight columns of a forward thread
constexpr unsigned kNone = 0xffffffffu;  // sorts behind every row
constexpr int64_t kMaxGrid = 0x7fffffff;

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
  const int64_t total = A.tokens * A.per;
  const int64_t base = int64_t(blockIdx.x) * (kThreads * kEach);
  const int64_t t0 = base / A.per;
  const unsigned c0 = unsigned(base - t0 * A.per);
  int64_t token[kEach], row[kEach];
  unsigned col[kEach];
  Eight<TW> w[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const unsigned q = c0 + unsigned(k * kThreads) + threadIdx.x;
    const unsigned up = q / A.per;
    token[k] = t0 + up;
    col[k] = (q - up * A.per) * 8;
    row[k] = token[k] < A.tokens ? A.ids.row(A.ids.id(token[k])) : -1;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    w[k].template load<TAIL>(row_of<TW>(A.table, row[k], A.ld_table), col[k],
                             row[k] >= 0 ? A.cols - col[k] : 0);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (base + k * kThreads + threadIdx.x >= total) break;
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
    y.template store<TAIL, !TAIL>(row_of<TY>(A.y, token[k], A.ld_y), col[k], A.cols - col[k]);
  }
}

struct SortArgs {
  Ids ids;
  int64_t tokens;
  int32_t tile;
  unsigned *keys;  // rows, sorted; vocab: no row of this table
  int *order;      // their tokens
};

// A workgroup places kPlaced tokens.  Its waves share the tile's tokens in chunks of 64;
// in each wave two lanes take a token, one for either half of a chunk (with 64
// tokens a wave, half of the CUs had nothing to do and each of the others
// read all keys out of LDS twice as often: 17 us for SORTUS).  Of equal rows the
// earlier token comes first: tokens of earlier chunks count up to the same row,
// those of later ones below it.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs A) {
  __shared__ __align__(16) unsigned keys[kTile];
  __shared__ unsigned counts[kSortWaves][kPlaced];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned blocks = unsigned(A.tile) / kPlaced;  // of a tile
  const int64_t tile = int64_t(blockIdx.x / blocks) * A.tile;
  const int own = int(blockIdx.x % blocks) * kPlaced;  // in the tile
  const int64_t left = A.tokens - tile;
  const int n = left < A.tile ? int(left) : A.tile, chunks = (n + 63) / 64;
#pragma unroll
  for (int i = 0; i < kTile / kSortThreads; ++i) {
    const int s = i * kSortThreads + int(threadIdx.x);
    if (s < chunks * 64) keys[s] = s < n ? A.ids.key(tile + s) : kNone;
  }
  __syncthreads();
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
}

struct MergeArgs {
  int32_t tokens, run;  // sorted runs of this length
  const unsigned *keys;
  const int *order;
  unsigned *keys_out;
  int *order_out;
};

// A token's place among up to kRuns runs: its place in its own and, in each
// other, the number of tokens that come before it.  The searches run side by side.
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
#pragma unroll
    for (int q = 0; q < kRuns; ++q)
      if (lo[q] < hi[q]) {
        const int mid = (lo[q] + hi[q]) >> 1;
        const unsigned k = A.keys[mid];
        // an earlier run's equals come first
        if (q < own ? k <= key : k < key) lo[q] = mid + 1;
        else hi[q] = mid;
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
  float *part;  // [2 tokens / kRun][per * 8], see part_of
  float scale;
  int32_t add;        // to what is there
  unsigned per;       // pieces of eight columns
  int64_t sum_blocks; // workgroups that sum; the others clear
  int32_t rows;       // that a workgroup clears
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
// that begin within kRun tokens one at most is its row's first (its row goes on
// for all of them) and one at most is not.
__device__ __forceinline__ int64_t part_of(int64_t at, bool first) {
  return at / kRun * 2 + (first ? 1 : 0);
}

// A row's sum, scaled and joined with what is there, into the table's gradient.
template <class TG, bool TAIL>
__device__ __forceinline__ void put_row(const SumArgs &A, unsigned row, unsigned col,
                                        float (&v)[8]) {
  void *to = row_of<TG>(A.out, row, A.ld_out);
  Eight<TG> w;
  if (A.add) {
    w.template load<TAIL>(to, col, A.cols - col);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(A.scale, v[e], w.get(e));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= A.scale;
  }
  w.set(v);
  w.template store<TAIL>(to, col, A.cols - col);
}

// Rows without tokens become zeros.
template <class TG, bool TAIL>
__device__ __forceinline__ void clear_rows(const SumArgs &A, int64_t block) {
  __shared__ int used[kThreads];
  const int64_t r0 = block * A.rows;
  const int rows = int(A.vocab - r0 < A.rows ? A.vocab - r0 : A.rows);
  if (int(threadIdx.x) < rows) {
    const unsigned key = unsigned(r0 + threadIdx.x);
    const int64_t at = first_not_below(A.keys, 0, A.tokens, key);
    used[threadIdx.x] = at < A.tokens && A.keys[at] == key;
  }
  __syncthreads();
  // in elements, or in sixteen bytes side by side
  using raw = typename TG::raw;
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
      else __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4 *>(to) + c);
    }
  }
}

// Keys and tokens of kPiece sorted places from `at` on, a multiple of kPiece.
struct Places {
  unsigned key[kPiece];
  int token[kPiece];
  __device__ __forceinline__ void load(const SumArgs &A, int64_t at) {
    if (at + kPiece <= A.tokens) {
#pragma unroll
      for (int q = 0; q < kPiece / 4; ++q) {
        const u32x4 k = *reinterpret_cast<const u32x4 *>(A.keys + at + q * 4);
        const u32x4 t = *reinterpret_cast<const u32x4 *>(A.order + at + q * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          key[q * 4 + e] = k[e];
          token[q * 4 + e] = int(t[e]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        key[e] = at + e < A.tokens ? A.keys[at + e] : kNone;
        token[e] = at + e < A.tokens ? A.order[at + e] : 0;
      }
    }
  }
};

template <class TY, class TG, bool TAIL>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const SumArgs A) {
  if (int64_t(blockIdx.x) >= A.sum_blocks) {
    clear_rows<TG, TAIL>(A, int64_t(blockIdx.x) - A.sum_blocks);
    return;
  }
  const int64_t base = int64_t(blockIdx.x) * kThreads;
  const int64_t p0 = base / A.per;
  const unsigned q = unsigned(base - p0 * A.per) + threadIdx.x, up = q / A.per;
  const unsigned col = (q - up * A.per) * 8;
  const int64_t from = (p0 + up) * kPiece;
  if (from >= A.tokens) return;
  // this piece's places, the next one's, and how many of the kRun before it are of its
  // first row: three loads side by side
  Places now, next;
  now.load(A, from);
  next.load(A, from + kPiece);
  int before = 0;
#pragma unroll
  for (int k = kPiece; k <= kRun; k += kPiece)
    if (from >= k) {
#pragma unroll
      for (int h = 0; h < kPiece / 4; ++h) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(A.keys + from - k + h * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) before += v[e] == now.key[0] ? 1 : 0;
      }
    }
  // a row that began before this piece: its next part may begin in here
  const unsigned first = now.key[0], last = now.key[kPiece - 1];
  int64_t part = from;
  if (before) {
    const int64_t row0 =
        before < kRun ? from - before : first_not_below(A.keys, 0, from - kRun, first);
    part = row0 + (from - row0 + kRun - 1) / kRun * kRun;
  }
  const int64_t to = from + kPiece;
  unsigned key = kNone;  // of the row being summed
  int64_t start = 0;     // its part's first place
  bool active = false, whole = false;  // whole: that is the row's first place too
  float acc[8];
  const auto flush = [&](bool ended) {
    if (whole && ended) {
      put_row<TG, TAIL>(A, key, col, acc);
    } else {
      Eight<F32> v;
      v.set(acc);
      v.template store<false>(A.part + part_of(start, whole) * (int64_t(A.per) * 8), col, 8);
    }
  };
  for (int64_t at = from;; at += kPiece) {
    Eight<TY> v[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const unsigned k = now.key[j];
      const bool mine = at == from ? !(before && k == first && at + j < part)
                                   : k == last && at + j - start < kRun;
      const bool take = mine && k < unsigned(A.vocab);
      v[j].template load<TAIL, !TAIL>(row_of<TY>(A.dy, take ? now.token[j] : 0, A.ld_dy), col,
                                      take ? A.cols - col : 0);
    }
    Places after;
    after.load(A, at + 2 * kPiece);
    bool done = false;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const unsigned k = now.key[j];
      const int64_t i = at + j;
      const bool row = j ? k != now.key[j - 1] : at == from ? !before : k != key;
      const bool none = k >= unsigned(A.vocab);  // and so are all places behind
      if (active && (row || none || i - start == kRun)) {
        flush(row || none);
        active = false;
      }
      if (none || (i >= to && !active)) {
        done = true;
        break;
      }
      if (row || (before && i == part && k == first)) {
        key = k;
        start = i;
        whole = row;
        active = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
      }
      if (active) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[j].get(e);
      }
    }
    if (done || !active) break;
    now = next;
    next = after;
  }
}

// The parts of the row that begins among the kRun places from blockIdx.x kRun on and
// goes on for more than kRun, if there is one: each wave adds a stretch of them, then
// the waves' sums are added in order.
template <class TG, bool TAIL>
__global__ void __launch_bounds__(64 * kJoinWaves) embed_join_kernel(const SumArgs A) {
  __shared__ float sums[kJoinWaves][8][64];
  const int64_t from = int64_t(blockIdx.x) * kRun, to = from + kRun;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (to >= A.tokens) return;
  // lanes: the place before, the kRun places, the one behind
  const int64_t look = from - 1 + lane;
  const unsigned near = lane < kRun + 2 && look >= 0 ? A.keys[look] : kNone;
  const unsigned key = __builtin_amdgcn_readlane(near, kRun);
  if (key >= unsigned(A.vocab)) return;
  const uint64_t same = __ballot(near == key);
  if (!(same >> (kRun + 1) & 1) || (same & 1)) return;  // ends in here, or began before
  const int64_t start = from - 1 + __builtin_ctzll(same);
  if (start + kRun >= A.tokens || A.keys[start + kRun] != key) return;
  // a part a lane: how many begin within the row
  int64_t parts = 1;
  for (;;) {
    const int64_t at = start + (parts + lane) * kRun;
    const uint64_t more = __ballot(at < A.tokens && A.keys[at < A.tokens ? at : start] == key);
    parts += __builtin_popcountll(more);
    if (more != ~uint64_t(0)) break;
  }
  const unsigned c = blockIdx.y * 64 + lane, col = c * 8;
  const int64_t width = int64_t(A.per) * 8, each = (parts + kJoinWaves - 1) / kJoinWaves;
  float acc[8] = {};
  if (c < A.per) {
    const int64_t lo = wave * each, hi = lo + each < parts ? lo + each : parts;
#pragma unroll 4
    for (int64_t j = lo; j < hi; ++j) {
      Eight<F32> v;
      v.template load<false>(A.part + part_of(start + j * kRun, j == 0) * width, col, 8);
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

// Workspace: the sorted rows and tokens (twice where runs are merged), the
// parts of long rows.
struct Plan {
  int64_t keys[2], order[2], part, bytes;
  bool merged;
  explicit Plan(const zs_embedding_desc &d) {
    const int64_t list = up(d.tokens * 4, 256), runs = (d.tokens + kRun - 1) / kRun;
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
  const int64_t blocks = (d.tokens + kPlaced - 1) / kPlaced;
  const int32_t tile = d.tokens <= kTile ? kTile : kSmallTile;
  hipLaunchKernelGGL(embed_sort_kernel, dim3(unsigned(blocks)), dim3(kSortThreads), 0, st,
                     SortArgs{ids_of(d, ids), d.tokens, tile, keys(0), order(0)});
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
  if (blocks > kMaxGrid / kThreads) return ZS_EINVAL;
  if (const int rc = device_is_gfx950()) return rc;
  const bool even = rows_even(table, A.ld_table, tsize) && rows_even(y, A.ld_y, size);
  return by_type(d->dtype, d->table_dtype, [&](auto ty, auto tw) {
    return by_tail(d->cols % 8 != 0 || !even, [&](auto tail) {
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
  if (d->tokens > 0 && (!ids || !dy || !workspace || workspace_bytes < p.bytes)) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), gsize = dtype_size(d->grad_dtype);
  if (!aligned(ids, d->id_bytes) || !aligned(dy, size) || !aligned(dtable, gsize) ||
      !aligned(workspace, 256))
    return ZS_EALIGN;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  const int64_t pieces = (d->tokens + kPiece - 1) / kPiece, runs = (d->tokens + kRun - 1) / kRun;
  SumArgs A{d->tokens, d->vocab, d->cols, ld(d->ld_dy), ld(d->ld_dtable), nullptr, nullptr, dy,
            dtable, nullptr, d->scale, d->accumulate, per_of(*d), 0, 0};
  A.sum_blocks = (pieces * A.per + kThreads - 1) / kThreads;
  // about 64 KiB a workgroup clears, so that its searches are hidden
  A.rows = int32_t((65536 + d->cols * gsize - 1) / (d->cols * gsize));
  if (A.rows > kThreads) A.rows = kThreads;
  const int64_t clear = d->accumulate ? 0 : (d->vocab + A.rows - 1) / A.rows;
  if (A.sum_blocks + clear > kMaxGrid / kThreads) return ZS_EINVAL;
  if (const int rc = device_is_gfx950()) return rc;
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  char *ws = static_cast<char *>(workspace);
  if (d->tokens > 0) {
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
      hipLaunchKernelGGL((embed_sum_kernel<decltype(ty), TG, tail.value>),
                         dim3(unsigned(A.sum_blocks + clear)), dim3(kThreads), 0, st, A);
      if (runs > 1)
        hipLaunchKernelGGL((embed_join_kernel<TG, tail.value>),
                           dim3(unsigned(runs), (A.per + 63) / 64), dim3(64 * kJoinWaves), 0, st,
                           A);
      return launched();
    });
  });
}

}  // extern "C"
