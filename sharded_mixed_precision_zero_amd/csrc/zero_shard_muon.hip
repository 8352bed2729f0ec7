// zero_shard_muon.hip -- the Muon update of a rank's weight matrices on MI355X
// (gfx950): momentum over the averaged contributions, orthogonalisation by
// Newton-Schulz products, weight update (declarations and the contract:
// include/zero_shard.h).
//
// momentum and apply are HBM-bound elementwise passes over a flat range, in
// binary64 with one rounding to binary32 per value, as the shard step's update;
// bf16 values (the update matrix, the weights' copy) are rounded from those, so
// that they are the same whether the binary32 value is stored as well or not.
//
// ortho: with m = min(rows, cols), n = max(rows, cols) and X the m x n matrix
// (the transpose of a tall one), X0 = G / (|G|_F + eps) and, `steps` times,
//   A = X X^T;   B = a I + b A + c A A;   X = B X
// (a X is folded into B's diagonal).  The products run on the matrix cores
// with binary32 accumulation.  Between products X, A and B are held in
// binary16, scaled by 2^11: with coefficients that keep the singular values
// near 1 every entry is bounded (|X|, |A| below 1.5, |B| below 4), so binary16
// has the range, entries down to 2^-25 keep all 11 bits, and the rounding is 8
// times finer than bf16's, at the same rate: against binary64 the result is
// off by 1.2e-3 of its norm before its own rounding to bf16 (2.1e-3 after it)
// where bf16 in between gives 1.0e-2 (Gaussian matrices, 64 x 64 to
// 1024 x 1024).
//
// All three products are C[i][j] = sum_k P[i][k] Q[j][k] over rows of
// contiguous k: X X^T and A A^T (A is symmetric) as they stand, and B X with
// X kept transposed as well, which each update's epilogue writes next to X.
// A and B are symmetric, so only the tiles on and below the diagonal are
// computed and each is stored twice: m^2 n + m^3 + 2 m^2 n operations a step
// in place of 2 m^2 n + 2 m^3 + 2 m^2 n.
//
// Of a matrix much longer than wide the products with X are most of that, and
// two steps are taken with one of each: A and the polynomials in it commute, so
// after B the next A is B A B, and with its polynomial B' the two steps are
// X = (B' B) X: 3 m^2 n + 6 m^3 for two steps (the three extra products are
// symmetric) in place of 6 m^2 n + 2 m^3.  Rounding leaves A with eigenvalues a
// little below 0 and B A B multiplies those by a^2, so it is done once and then
// A is made anew from X: in two steps the result is as far off as before
// (Gaussian 512 x 1382, without the rests of the diagonals: 1.26e-3 for 1.19e-3;
// ill-conditioned and rank-8 ones: less than before), in three it diverges where A is singular.
//
// What bounds the large ones is the card's power: with the operands' bits at
// random the clock falls to 1.9-2.1 GHz at 60% of the matrix cores' cycles, and
// a variant that needs fewer cycles (32 x 32 x 16 instructions: 10% fewer) takes
// the same time.  5120 x 5120 in five steps: 2.4 ms, 1.1 PFLOP/s of the
// operations counted above, where a library product of that size reaches 1.0
// and of 8192 1.4; 13824 x 5120 4.1 ms, 1.5 PFLOP/s of the single steps' count.
// X is laid out padded to multiples of 64 with zeros, which the iteration keeps
// zero; tiles reach past that, loads there are dropped by the hardware's bounds
// and stores checked.  Matrices of up to 128 rows take ways of their own.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "zero_shard.h"
#include "zs_args.h"
#include "zs_device.h"

namespace {

using namespace zs_dev;

using half8 = _Float16 __attribute__((ext_vector_type(8)));
using half4 = _Float16 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr unsigned kFew = 256;  // workgroups: one a CU, too few for HBM to bound them
// Elements of a launch of momentum or apply, a thread for eight: it takes below
// 2^32 threads.
constexpr int64_t kPiece = INT64_C(1) << 34;

// ------------------------------------------------- momentum and apply

struct Rows {
  const uint16_t *p[ZS_MAX_ND];
};

struct MomentumArgs {
  Rows rows;
  int64_t n;
  int32_t n_d, nesterov;
  double mu;
  const float *m_in;
  float *m_out;
  void *update;
};

// A wave takes 512 elements, a lane two fours of them 256 apart, so that each
// access of the wave covers one stretch; all of them go past the caches (the
// whole Muon step takes the same time with the update kept there).  Eight rows
// are in flight while the binary64 sum keeps the rank order, of short ranges two
// times eight.  Out of no cache: 16 rows of 5120 x 5120 190 us, 5.8 TB/s, 3 rows
// of 9.4 million 29 us (eight consecutive elements a lane, momentum and update
// through the caches: 220 and 37 us); 64 rows of 40000 11 us (14 with eight rows
// in flight).  The last n % 512 elements have a lane each (60 rows of 3001: 11
// us; one lane for eight of them, element by element, 20).
struct Fours {
  u32x2 w[2];
  __device__ __forceinline__ float get(int e) const {
    const unsigned v = w[e / 4][e % 4 / 2];
    return __uint_as_float(e % 2 ? v & 0xffff0000u : v << 16);
  }
};

template <class T>  // of a row: Fours, or one element
__device__ __forceinline__ T row_at(const uint16_t *row, int64_t e0) {
  T v;
  if constexpr (sizeof(T) == 2) {
    v = row[e0];
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v.w[h] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(row + e0 + h * 256));
  }
  return v;
}

// DEEP: the next eight rows' loads are issued before these are added.
template <bool DEEP, int N, class T, class F>
__device__ __forceinline__ void sum_rows(const MomentumArgs &A, int64_t e0, double (&s)[N], F get) {
  const auto load = [&](T (&r)[8], int k) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < A.n_d) r[i] = row_at<T>(A.rows.p[k + i], e0);
  };
  const auto add = [&](const T (&r)[8], int k) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < A.n_d) {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] += double(get(r[i], e));
      }
  };
  const auto load8 = [&](T (&r)[8], int k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = row_at<T>(A.rows.p[k + i], e0);
  };
  const auto add8 = [&](const T (&r)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] += double(get(r[i], e));
  };
  T r[8], q[8];
  int k = 0;
  if constexpr (DEEP) {
    if (A.n_d >= 8) load8(r, 0);
    for (; k + 24 <= A.n_d; k += 16) {
      load8(q, k + 8);
      add8(r);
      load8(r, k + 16);
      add8(q);
    }
    if (k + 16 <= A.n_d) {
      load8(q, k + 8);
      add8(r);
      load(r, k + 16);
      add8(q);
      add(r, k + 16);
    } else if (k + 8 <= A.n_d) {
      load(q, k + 8);
      add8(r);
      add(q, k + 8);
    } else {
      load(q, k);
      add(q, k);
    }
  } else {
    for (; k + 8 <= A.n_d; k += 8) {
      load8(r, k);
      add8(r);
    }
    if (k < A.n_d) {
      load(q, k);
      add(q, k);
    }
  }
}

// g = the average; the new momentum; the update
__device__ __forceinline__ void momentum_of(const MomentumArgs &A, double sum, float &m, float &u) {
  const float g = float(sum / double(A.n_d));
  const double mm = A.mu * double(m) + double(g);
  m = float(mm);
  u = A.nesterov ? float(double(g) + A.mu * mm) : float(mm);
}

template <class TU, bool DEEP>
__global__ void __launch_bounds__(kThreads) momentum_kernel(const MomentumArgs A) {
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x, whole = A.n / 512 * 512;
  if (at < whole / 8) {
    const int64_t e0 = at / 64 * 512 + at % 64 * 4;
    f32x4 m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      m[h] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(A.m_in + e0 + h * 256));
    double s[8] = {};
    sum_rows<DEEP, 8, Fours>(A, e0, s, [](const Fours &r, int e) { return r.get(e); });
    struct Out {
      typename TU::raw e[4];
    };
    using Words = std::conditional_t<sizeof(Out) == 16, u32x4, u32x2>;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Out out;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = m[h][e], u;
        momentum_of(A, s[h * 4 + e], v, u);
        m[h][e] = v;
        out.e[e] = TU::store(u);
      }
      __builtin_nontemporal_store(m[h], reinterpret_cast<f32x4 *>(A.m_out + e0 + h * 256));
      __builtin_nontemporal_store(
          __builtin_bit_cast(Words, out),
          reinterpret_cast<Words *>(static_cast<typename TU::raw *>(A.update) + e0 + h * 256));
    }
  } else {
    const int64_t e0 = whole + (at - whole / 8);
    if (e0 >= A.n) return;
    float m = A.m_in[e0], u;
    double s[1] = {};
    sum_rows<true, 1, uint16_t>(A, e0, s, [](uint16_t r, int) { return Bf16::load(r); });
    momentum_of(A, s[0], m, u);
    A.m_out[e0] = m;
    static_cast<typename TU::raw *>(A.update)[e0] = TU::store(u);
  }
}

struct ApplyArgs {
  int64_t n;
  const uint16_t *o;
  const float *in;
  float *out;
  uint16_t *p;
  double decay, step;  // lr * weight_decay, lr * scale
};

// A wave takes 512 elements, a lane two fours of them 256 apart, so that each
// access of the wave covers one stretch; the state is read and written once a
// step and goes past the caches.  13824 x 5120: 134 us, 6.3 TB/s (eight
// consecutive elements a lane, through the caches: 152 us).
__global__ void __launch_bounds__(kThreads) apply_kernel(const ApplyArgs A) {
  using u16x4 = uint16_t __attribute__((ext_vector_type(4)));
  const int64_t wave = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t e0 = wave * 512 + (threadIdx.x & 63) * 4;
  const auto next = [&](float w, uint16_t o) {
    const double x = double(w);
    return float((x - A.decay * x) - A.step * double(Bf16::load(o)));
  };
  f32x4 w[2];
  u16x4 o[2], p[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (e0 + h * 256 + 4 <= A.n) {
      w[h] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(A.in + e0 + h * 256));
      o[h] = __builtin_nontemporal_load(reinterpret_cast<const u16x4 *>(A.o + e0 + h * 256));
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t e1 = e0 + h * 256;
    if (e1 + 4 <= A.n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[h][e] = next(w[h][e], o[h][e]);
        p[h][e] = Bf16::store(w[h][e]);
      }
      __builtin_nontemporal_store(w[h], reinterpret_cast<f32x4 *>(A.out + e1));
      __builtin_nontemporal_store(p[h], reinterpret_cast<u16x4 *>(A.p + e1));
    } else {
      for (int64_t e = e1; e < A.n; ++e) {
        const float v = next(A.in[e], A.o[e]);
        A.out[e] = v;
        A.p[e] = Bf16::store(v);
      }
    }
  }
}

// --------------------------------------------------- ortho: norm and layout

constexpr float kScale = 2048.0f;  // 2^11: X, A and B are held times this
constexpr int kNormBlocks = 1024;  // most partial sums of squares per matrix
constexpr int kNormRun = 2048;     // consecutive elements a workgroup sums at a time
constexpr int kStrip = 256;        // columns of 64 rows that a workgroup lays out
constexpr int kCutTiles = kThreads;  // most tiles of a product that are cut along k

struct InArgs {
  const void *g;
  int64_t rows, cols, ld, stride;  // of the input, elements
  double *partials;                // [batch][blocks]
  int32_t *arrived;                // [kCutTiles], zeroed
  _Float16 *x, *xt;                // [batch][mp][np] and [batch][np][mp]
  int64_t mp, np;
  double eps;
  int32_t blocks;
  int32_t tall;  // rows > cols: X is the transpose of G
};

// Sum over the workgroup's 256 threads (the result in thread 0).
__device__ __forceinline__ double block_sum(double v, double *lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v += lds[w];
  return v;
}

// Partial sums of squares, 8 elements a thread and run.
template <class TG>
__global__ void __launch_bounds__(kThreads) ortho_norm_kernel(const InArgs A) {
  __shared__ double lds[kThreads / 64];
  if (blockIdx.x + blockIdx.y == 0) A.arrived[threadIdx.x] = 0;
  const typename TG::raw *g =
      static_cast<const typename TG::raw *>(A.g) + int64_t(blockIdx.y) * A.stride;
  const unsigned runs = unsigned((A.cols + kNormRun - 1) / kNormRun);
  const int64_t all = A.rows * runs;
  double s = 0.0;
#pragma unroll 2
  for (int64_t w = blockIdx.x; w < all; w += A.blocks) {
    // all < 2^20 * 2^9
    const unsigned r = unsigned(w) / runs;
    const int64_t c = int64_t(unsigned(w) - r * runs) * kNormRun + threadIdx.x * 8;
    Eight<TG> v;
    v.load(g + r * A.ld, c, A.cols - c);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma(double(v.get(e)), double(v.get(e)), s);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) A.partials[int64_t(blockIdx.y) * A.blocks + blockIdx.x] = s;
}

// 64 x 64 tiles of X and of its transpose, scaled and padded with zeros, a
// strip of 64 rows after another.
template <class TG>
__global__ void __launch_bounds__(kThreads) ortho_layout_kernel(const InArgs A) {
  __shared__ double lds[kThreads / 64];
  __shared__ __align__(16) _Float16 tile[64][68];
  const int64_t b = blockIdx.z;
  double sum = 0.0;
  for (int i = threadIdx.x; i < A.blocks; i += kThreads) sum += A.partials[b * A.blocks + i];
  sum = block_sum(sum, lds);
  const double scale = double(kScale) / (sqrt(sum) + A.eps);
  const typename TG::raw *g = static_cast<const typename TG::raw *>(A.g) + b * A.stride;
  // in the input's orientation, padded to rp x cp
  const int64_t rp = A.tall ? A.np : A.mp, cp = A.tall ? A.mp : A.np;
  const int64_t r0 = int64_t(blockIdx.y) * 64, c1 = int64_t(blockIdx.x + 1) * kStrip;
  _Float16 *same = (A.tall ? A.xt : A.x) + b * A.mp * A.np;
  _Float16 *turned = (A.tall ? A.x : A.xt) + b * A.mp * A.np;
  const int row = threadIdx.x >> 3, piece = (threadIdx.x & 7) * 8;
  for (int64_t c0 = c1 - kStrip; c0 < c1 && c0 < cp; c0 += 64) {
    half8 out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = r0 + row + i * 32, c = c0 + piece, left = r < A.rows ? A.cols - c : 0;
      Eight<TG> v;
      v.load(g + r * A.ld, c, left);
#pragma unroll
      for (int e = 0; e < 8; ++e) out[i][e] = _Float16(float(double(v.get(e)) * scale));
      *reinterpret_cast<half8 *>(same + r * cp + c) = out[i];
    }
    __syncthreads();  // the last tile has been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<half4 *>(&tile[row + i * 32][piece]) = out[i].lo;
      *reinterpret_cast<half4 *>(&tile[row + i * 32][piece + 4]) = out[i].hi;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) out[i][e] = tile[piece + e][row + i * 32];
      *reinterpret_cast<half8 *>(turned + (c0 + row + i * 32) * rp + r0 + piece) = out[i];
    }
  }
}

// ------------------------------------------------------- ortho: products

enum Product {
  kGram,  // A = X X^T                  symmetric
  kPoly,  // B = a I + b A + c A A      symmetric
  kNext,  // X = B X, and X^T
  kLast   // O = B X, in the caller's orientation and bf16
};

struct MulArgs {
  const _Float16 *p, *q;       // [batch][rows][k], [batch][cols][k]
  int64_t stride_p, stride_q;  // elements per matrix
  int32_t k;                   // a multiple of 64
  int32_t rows, cols;          // of C, multiples of 64
  int32_t tiles_r, tiles_c;    // of C
  int32_t per, one;            // tiles computed per matrix; whether there is one matrix
  int32_t cut, groups;         // all `cut` tiles are cut between `groups` workgroups; or 0
  float *parts;                // [2 groups][tile] partial sums of cut tiles
  int32_t *arrived;            // [cut] workgroups done with a cut tile; 0 between launches
  _Float16 *c, *ct;            // C (row length cols) and C^T (row length rows)
  int64_t stride_c;
  // The rests of P's, Q's and C's diagonals, [batch][rows], where they are no X;
  // or null
  const float *rest_p, *rest_q;
  float *rest_c;
  float a, b, cc;              // kPoly's coefficients
  int32_t past;                // C^T goes past the caches
  // kLast
  uint16_t *o;
  int64_t out_rows, out_cols, ld_o, stride_o;
  int32_t tall, wide;          // wide: 16 bytes of a row at a time
};

// What rounding to binary16 took off an element v of a diagonal, relative to
// what is left.  The diagonals of A and B are much the largest elements there
// and much alike, so their rounding scales whole rows of X; where the singular
// values lie together on a steep part of the polynomial, the next steps make
// that larger: the result of a random 32 x 13824 came out 2.3 times as far off as
// the rounding of a right one to bf16, 430 x 13824 1.7, 256 x 256 1.26 times.  So
// it is kept.  Rows of B X are multiplied by 1 + rest, which is right for the
// diagonal's share and for the others no more than their own rounding; in
// products of A and B it is made good on the diagonal alone.  With it those are
// 1.03, 1.03 and 1.17 times; it costs 0.5% at 5120 x 13824, 3% at 300 x 700.
// Below binary16's normal range nothing is kept, so that the rest is never more
// than 2^-11.
__device__ __forceinline__ float rest_in(float v) {
  const float h = float(_Float16(v));
  return __builtin_fabsf(h) < 0x1p-14f ? 0.0f : (v - h) * __builtin_amdgcn_rcpf(h);
}

#define ZS_LDS(p) ((__attribute__((address_space(3))) void *)(p))

// All waves of the workgroup; accesses to memory stay on their side of it.
[[maybe_unused]] __device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// At most N of this wave's loads and stores outstanding.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt has 6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}

template <int V>
using Const = std::integral_constant<int, V>;

// The order of a turn's instructions: G times EACH matrix instructions, the
// share of N loads that falls to it, one read.
template <int I, int G, int N, int EACH>
__device__ __forceinline__ void order() {
  if constexpr (I < G) {
    __builtin_amdgcn_sched_group_barrier(0x8, EACH, 0);
    constexpr int LOADS = (I + 1) * N / G - I * N / G;
    if constexpr (LOADS > 0) __builtin_amdgcn_sched_group_barrier(0x10, LOADS, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    order<I + 1, G, N, EACH>();
  }
}

// How many tiles of tile row tr lie on or below the diagonal.
__host__ __device__ inline int below(int tr, int TR, int TC, int tiles_c) {
  const int n = ((tr + 1) * TR - 1) / TC + 1;
  return n < tiles_c ? n : tiles_c;
}

// Tile t of a matrix, in bands of 4 tile rows, column by column within the
// band, so that neighbours share both operands in L2; of symmetric products
// the tiles on and below the diagonal.
template <bool SYM, int TR, int TC>
__device__ __forceinline__ void tile_of(int t, int tiles_r, int tiles_c, int &tr, int &tc) {
  if constexpr (SYM) {
    int row = 0, rows = 0, least = 0;
    for (;; row += 4) {
      rows = tiles_r - row < 4 ? tiles_r - row : 4;
      least = below(row, TR, TC, tiles_c);
      int all = 0;
      for (int i = 0; i < rows; ++i) all += below(row + i, TR, TC, tiles_c);
      if (t < all || row + 4 >= tiles_r) break;
      t -= all;
    }
    if (t < rows * least) {
      tc = rows == 4 ? t >> 2 : t / rows;
      tr = row + t - tc * rows;
      return;
    }
    t -= rows * least;  // the columns that only the band's later rows have
    for (int i = 1; i < rows; ++i) {
      const int extra = below(row + i, TR, TC, tiles_c) - least;
      tr = row + i;
      tc = least + t;
      if (t < extra) return;
      t -= extra;
    }
  } else {
    const int band = t / (4 * tiles_c), in = t - band * 4 * tiles_c;
    const int rows = tiles_r - band * 4 < 4 ? tiles_r - band * 4 : 4;
    tc = rows == 4 ? in >> 2 : in / rows;
    tr = band * 4 + in - tc * rows;
  }
}

// TR x TC tiles of C, WR x WC waves, S buffers of 64 of k.  The operands go
// from global memory straight into LDS, S - 1 buffers ahead of their use, so a
// buffer costs one barrier; a row of 64 is eight pieces of 16 bytes, piece c
// of row r at position c ^ (r & 7), so the rows that one read instruction
// serves together lie in different banks.  The registers of the next 32 of k
// are read while the matrix cores work on the present ones.
template <int KIND, bool CUT, int TR, int TC, int WR, int WC, int S>
__global__ void __launch_bounds__(WR *WC * 64) ortho_mul_kernel(const MulArgs A) {
#ifdef __HIP_DEVICE_COMPILE__  // the buffer resources' type is known to the device pass only
  constexpr bool SYM = KIND == kGram || KIND == kPoly;
  constexpr int NW = WR * WC, TM = TR / WR / 16, TN = TC / WC / 16;
  // load instructions (8 rows of 64) per wave and buffer, of P and of both;
  // P's rows in LDS are filled up to a multiple of 8 NW
  constexpr int LP = (TR + 8 * NW - 1) / (8 * NW), L = LP + TC / (8 * NW);
  constexpr int PITCH = TC + 8, PITCH_T = TR + 8;  // of the tile and its transpose on their way out
  constexpr int QAT = LP * 8 * NW * 64, BUF = QAT + TC * 64;
  constexpr int STAGE = S * BUF, EPI = TR * PITCH > TC * PITCH_T ? TR * PITCH : TC * PITCH_T;
  __shared__ __align__(16) _Float16 lds[STAGE > EPI ? STAGE : EPI];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const auto uniform = [](unsigned v) { return int(__builtin_amdgcn_readfirstlane(v)); };

  // Workgroups go to the 8 XCDs in turn: each gets a contiguous run of tiles.
  const unsigned total = gridDim.x, id = blockIdx.x, xcd = id & 7;
  const unsigned each = total / 8, more = total % 8;
  const int at = int(xcd * each + (xcd < more ? xcd : more) + id / 8);
  const int nk = A.k / 64;

  // One whole tile, or this workgroup's share of the cut ones in 64s of k.
  [[maybe_unused]] const unsigned steps = unsigned(A.cut) * nk, groups = A.groups;
  int s0 = 0, s1 = nk;
  if constexpr (CUT) {  // groups * steps < 2^32
    s0 = uniform(at * steps / groups);
    s1 = uniform((at + 1) * steps / groups);
  }
  do {
    int tile = at, k0 = 0, k1 = nk;
    if constexpr (CUT) {
      tile = uniform(unsigned(s0) / unsigned(nk));
      k0 = s0 - tile * nk;
      k1 = s1 - s0 < nk - k0 ? k0 + s1 - s0 : nk;
      s0 += k1 - k0;
    }
    // Opaque, so that no address is computed ahead of this loop and kept: the
    // registers are full.
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63;
    const int64_t mat = A.one ? 0 : uniform(unsigned(tile) / unsigned(A.per));
    int tr, tc;
    tile_of<SYM, TR, TC>(tile - int(mat) * A.per, A.tiles_r, A.tiles_c, tr, tc);
    tr = uniform(tr);
    tc = uniform(tc);
    const int row0 = tr * TR, col0 = tc * TC;  // of the tile in C

    // A lane's offset in bytes, below 256 rows of 2^20; loads of rows past the
    // operand's end are dropped by the bounds of its buffer resource.
    const int in = wave * 8 + (lane >> 3);
    const int off = (in * A.k + ((lane & 7) ^ (lane >> 3)) * 8) * 2;
    const auto operand = [&](const _Float16 *p, int left, int T) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16 *>(p), 0,
                                               (left < T ? left : T) * A.k * 2, 0x00020000);
    };
    const auto pg = operand(A.p + mat * A.stride_p + int64_t(row0) * A.k, A.rows - row0, TR);
    const auto qg = operand(A.q + mat * A.stride_q + int64_t(col0) * A.k, A.cols - col0, TC);
    // The buffers go round: `rd` is read next and `wr_` written next (offsets
    // into lds), `from` is the k that is loaded next; past the end the last
    // buffer is loaded once more, so that as many loads are outstanding in
    // every turn.
    int rd = 0, wr_ = 0, from = k0 * 64;
    const int end = k1 * 64;
    const auto load = [&](int i) {  // the i-th of a buffer's loads
      const int j = i < LP ? i : i - LP;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          i < LP ? pg : qg, ZS_LDS(lds + wr_ + (i < LP ? 0 : QAT) + (j * NW + wave) * 512), 16, off,
          (from + j * NW * 8 * A.k) * 2, 0, 0);
      if (i == L - 1) {
        wr_ = wr_ == (S - 1) * BUF ? 0 : wr_ + BUF;
        from = from + 64 < end ? from + 64 : from;
      }
    };
    // the buffer at rd is there for all waves, and all have read the one before
    const auto advance = [&] {
      __builtin_amdgcn_sched_barrier(0);
      wait_loads<(S - 2) * L>();
      barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    half8 regs[2][TM + TN];
    // where this lane's pieces of a buffer's first and second 32 of k are
    int pos[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int piece = (lane & 15) * 64 + ((h * 4 + (lane >> 4)) ^ (lane & 7)) * 8;
      pos[h][0] = piece + wr * TM * 1024;
      pos[h][1] = piece + QAT + wc * TN * 1024;
    }
    const auto fetch = [&](auto half, int i) {  // the i-th block of that half of the buffer at rd
      const int p = i < TM ? pos[half.value][0] + i * 1024 : pos[half.value][1] + (i - TM) * 1024;
      regs[half.value][i] = *reinterpret_cast<const half8 *>(lds + rd + p);
      if (half.value && i == TM + TN - 1) rd = rd == (S - 1) * BUF ? 0 : rd + BUF;
    };
    f32x4 acc[TM][TN] = {};
    // 32 of k, while the next 32 are read and, in the turn after the barrier,
    // the loads of the buffer that it freed are issued, evenly between the
    // matrix instructions: all loads at once fill the queue that the reads
    // need, and the matrix cores wait.
    const auto turn = [&](auto half) {
      constexpr int G = TM + TN, N = half.value ? L : 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int i = g * N / G; i < (g + 1) * N / G; ++i) load(i);
        fetch(Const<1 - half.value>{}, g);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              regs[half.value][i], regs[half.value][TM + j], acc[i][j], 0, 0, 0);
      constexpr int EACH = TM * TN / G > 0 ? TM * TN / G : 1;
      order<0, G, N, EACH>();
    };

    if constexpr (CUT) barrier();  // the previous tile's epilogue is done with the buffers
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
#pragma unroll
      for (int i = 0; i < L; ++i) load(i);
    advance();
#pragma unroll
    for (int i = 0; i < L; ++i) load(i);
#pragma unroll
    for (int i = 0; i < TM + TN; ++i) fetch(Const<0>{}, i);
    for (int u = k0; u < k1; ++u) {
      turn(Const<0>{});
      advance();
      turn(Const<1>{});  // after the last 64 it reads some buffer, not used
    }
    wait_loads<0>();

    // A cut tile: the last of its workgroups to arrive adds the parts, in the
    // order of k whoever that is, and goes on; the others have done theirs.
    if (CUT && k1 - k0 < nk) {
      constexpr int N = TM * TN;
      const auto part = [&](int w, int which, int i) {
        char *p = reinterpret_cast<char *>(A.parts + (int64_t(w) * 2 + which) * (TR * TC));
        return reinterpret_cast<f32x4 *>(p + i * NW * 1024 + unsigned(tid) * 16);
      };
#pragma unroll
      for (int i = 0; i < N; ++i) *part(at, k0 == 0, i) = acc[i / TN][i % TN];
      // Each wave waits for its own stores: the barrier waits for LDS only and the
      // release below for the stores of the first wave.  They are in this XCD's L2
      // then, which the release writes back.
      wait_loads<0>();
      const int w0 = uniform(((tile * nk + 1u) * groups - 1) / steps);
      const int w1 = uniform(((tile + 1u) * nk * groups - 1) / steps);
      int *flag = reinterpret_cast<int *>(lds);
      __syncthreads();
      if (tid == 0) {
        const int before = __hip_atomic_fetch_add(A.arrived + tile, 1, __ATOMIC_ACQ_REL,
                                                  __HIP_MEMORY_SCOPE_AGENT);
        if (before == w1 - w0)
          __hip_atomic_store(A.arrived + tile, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = before == w1 - w0;
      }
      __syncthreads();
      if (!uniform(*flag)) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i / TN][i % TN] = f32x4{};
      for (int w = w0; w <= w1; ++w) {
        // all under way at once: one after the other A of 1000 x 13000 took 48 us
        // for 41 (38 on another card)
        f32x4 got[N];
#pragma unroll
        for (int i = 0; i < N; ++i) got[i] = *part(w, w == w0, i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i / TN][i % TN] += got[i];
      }
    }

    // Lane l of a 16 x 16 block holds rows 4 (l / 16) + 0..3 of column l % 16.
    const int br = wr * TM * 16 + (lane >> 4) * 4, bc = wc * TN * 16 + (lane & 15);
    constexpr float kBack = KIND == kLast ? 1.0f / (kScale * kScale) : 1.0f / kScale;
    const auto narrow = [](float v) -> unsigned {
      if constexpr (KIND == kLast) return Bf16::store(v);
      else return F16::store(v);
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = row0 + br + i * 16;
      f32x4 row = f32x4{} + kBack;  // of B X
      if (!SYM && r < A.rows)
        row += kBack * *reinterpret_cast<const f32x4 *>(A.rest_p + mat * A.rows + r);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if constexpr (KIND == kPoly) {
          // A is symmetric: column c's four rows are four neighbours of row c
          const int c = col0 + bc + j * 16;
          half4 s = {};
          if (r < A.rows && c < A.cols)
            s = *reinterpret_cast<const half4 *>(A.p + mat * A.stride_p + int64_t(c) * A.k + r);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[i][j][e] = A.b * float(s[e]) + A.cc * (acc[i][j][e] * kBack);
            if (r + e == c) acc[i][j][e] += A.a * kScale;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] *= row[e];
        }
      }
    }
    // On the diagonal, of which a lane in four holds an element of a 16 x 16
    // block: what the rests add, and the rest of this one.  All is read first.
    const int wr0 = row0 + wr * TM * 16, wc0 = col0 + wc * TN * 16;
    if (SYM && wr0 < wc0 + TN * 16 && wc0 < wr0 + TM * 16) {
      const int e0 = (lane & 15) - (lane >> 4) * 4;
      float more[TM] = {};
      if (A.rest_p) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int d = wr0 + i * 16 + (lane & 15), c = d < A.cols ? d : 0;
          const int64_t at_c = int64_t(c) * A.k + c, rest = mat * A.rows + c;
          const float p = float(A.p[mat * A.stride_p + at_c]), dp = A.rest_p[rest];
          const float q = float(A.q[mat * A.stride_q + at_c]), dq = A.rest_q[rest];
          more[i] = (dp + dq) * p * q * kBack;
          if (KIND == kPoly) more[i] = A.cc * more[i] + A.b * dp * p;
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int c = wc0 + j * 16 + (lane & 15);
          if (wr0 + i * 16 != wc0 + j * 16 || unsigned(e0) >= 4 || c >= A.cols) continue;
          float v = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[i][j][e] += e0 == e ? more[i] : 0.0f;
            v = e0 == e ? acc[i][j][e] : v;
          }
          A.rest_c[mat * A.rows + c] = rest_in(v);
        }
    }
    u32x2 out[TM][TN];  // a lane's four rows in 16 bits
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          out[i][j][e] = narrow(acc[i][j][2 * e]) | narrow(acc[i][j][2 * e + 1]) << 16;

    uint16_t *epi = reinterpret_cast<uint16_t *>(lds);
    // the tile through LDS, as C (turned = false) or as its transpose
    const auto gather = [&](bool turned) {
      barrier();
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int r = br + i * 16, c = bc + j * 16;
          if (turned) {
            *reinterpret_cast<u32x2 *>(epi + c * PITCH_T + r) = out[i][j];
          } else {
            // Two lanes of neighbouring columns swap a row of each pair, so
            // that each writes two columns of two rows.
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const unsigned v = out[i][j][e];
              const unsigned o = __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);
              const unsigned both =
                  lane & 1 ? (o >> 16) | (v & 0xffff0000u) : (v & 0xffffu) | o << 16;
              *reinterpret_cast<unsigned *>(epi + (r + 2 * e + (lane & 1)) * PITCH + (c & ~1)) =
                  both;
            }
          }
        }
      barrier();
    };
    // Its pieces of 8 to memory, where `want` says so.
    const auto put = [&](auto turned, auto past, auto *dst, int64_t ld, auto want) {
      constexpr int H = turned.value ? TC : TR, W = turned.value ? TR : TC;
      const int r0 = turned.value ? col0 : row0, c0 = turned.value ? row0 : col0;
#pragma unroll 4
      for (int v = tid; v < H * W / 8; v += NW * 64) {
        const int r = v / (W / 8), c = v % (W / 8) * 8;
        if (want(r0 + r, c0 + c)) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(epi + r * (W + 8) + c);
          u32x4 *to = reinterpret_cast<u32x4 *>(dst + int64_t(r0 + r) * ld + c0 + c);
          if (past.value) __builtin_nontemporal_store(v, to);
          else *to = v;
        }
      }
    };
    if constexpr (KIND == kLast) {
      uint16_t *o = A.o + mat * A.stride_o;
      const auto inside = [&](int r, int c) { return r < A.out_rows && c < A.out_cols; };
      gather(A.tall);
      if (A.wide && A.tall) {
        put(Const<1>{}, Const<0>{}, o, A.ld_o, inside);
      } else if (A.wide) {
        put(Const<0>{}, Const<0>{}, o, A.ld_o, inside);
      } else {
        const int H = A.tall ? TC : TR, W = A.tall ? TR : TC;
        const int r0 = A.tall ? col0 : row0, c0 = A.tall ? row0 : col0;
        for (int r = wave; r < H; r += NW)
          for (int c = lane; c < W; c += 64)
            if (inside(r0 + r, c0 + c))
              o[(r0 + r) * A.ld_o + c0 + c] = epi[r * (W + 8) + c];
      }
    } else {
      gather(false);
      put(Const<0>{}, Const<0>{}, A.c + mat * A.stride_c, A.cols,
          [&](int r, int c) { return r < A.rows && c < A.cols; });
      if constexpr (KIND == kNext) {
        gather(true);
        const auto inside = [&](int r, int c) { return r < A.cols && c < A.rows; };
        if (A.past) put(Const<1>{}, Const<1>{}, A.ct + mat * A.stride_c, A.rows, inside);
        else put(Const<1>{}, Const<0>{}, A.ct + mat * A.stride_c, A.rows, inside);
      } else if (TR != TC || tr != tc) {
        // what no tile on or below the diagonal holds
        gather(true);
        put(Const<1>{}, Const<0>{}, A.c + mat * A.stride_c, A.rows, [&](int r, int c) {
          return r < A.cols && c < A.rows && c / TC * TC > r / TR * TR + TR - 1;
        });
      }
    }
  } while (CUT && s0 < s1);
#endif
}

// ---------------------------------------------- ortho: matrices of up to 128

// Short matrices are worked on in the LDS of a CU, 16 waves of 32 x 32 blocks:
// at up to 128 rows the products are so small that a launch for each costs more
// than the work.  Rows of k elements lie k + 8 apart, so that the 16 rows one
// read instruction serves lie in different banks.
constexpr int kSmallThreads = 1024;
constexpr int kSmallWaves = kSmallThreads / 64;
constexpr int kSmallLds = 81920;   // 16-bit elements: 160 KB
constexpr int kSmallPacks = 5;     // of 8 elements that a thread brings in
constexpr int kSmallBlocks = 3;    // of 32 x 32 that a wave computes
constexpr float kBack1 = 1.0f / kScale, kBack2 = kBack1 * kBack1;

using Block = f32x4[2][2];

struct BlockRegs {
  half8 p[2], q[2];
  // 32 of k at p and q (this lane's pieces)
  __device__ __forceinline__ void read(const _Float16 *pp, const _Float16 *qq, int pitch) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      p[e] = *reinterpret_cast<const half8 *>(pp + e * 16 * pitch);
      q[e] = *reinterpret_cast<const half8 *>(qq + e * 16 * pitch);
    }
  }
  __device__ __forceinline__ void add(Block &acc) const {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc[e][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(p[e], q[h], acc[e][h], 0, 0, 0);
  }
};

__device__ __forceinline__ const _Float16 *block_at(const _Float16 *p, int i, int pitch, int lane) {
  return p + (i * 32 + (lane & 15)) * pitch + (lane >> 4) * 8;
}

// Block i, j of P Q^T over K 32s of k.
template <int K>
__device__ __forceinline__ void block_mul(const _Float16 *P, const _Float16 *Q, int i, int j,
                                          int lane, Block &acc) {
  constexpr int pitch = K * 32 + 8;
  const _Float16 *p = block_at(P, i, pitch, lane), *q = block_at(Q, j, pitch, lane);
  BlockRegs f[K];
#pragma unroll
  for (int k = 0; k < K; ++k) f[k].read(p + k * 32, q + k * 32, pitch);
#pragma unroll
  for (int k = 0; k < K; ++k) f[k].add(acc);
}

// f(r, c, rows r..r+3 of column c), for each of the block's four parts
template <class F>
__device__ __forceinline__ void block_each(int i, int j, int lane, const Block &acc, F f) {
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      f(i * 32 + e * 16 + (lane >> 4) * 4, j * 32 + h * 16 + (lane & 15), acc[e][h]);
}

__device__ __forceinline__ half4 narrow4(const f32x4 &v) {
  half4 h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = _Float16(v[e]);
  return h;
}

// A symmetric matrix of mp rows in LDS is followed by the rests of its diagonal
// (96 x 128: 22.3 us, without them 21.8; 64 x 13824 36 and 33).
constexpr int64_t short_size(int64_t mp) { return mp * (mp + 8) + 2 * mp; }

template <int MB>
__device__ __forceinline__ float *rest_of(_Float16 *M) {
  return reinterpret_cast<float *>(M + MB * 32 * (MB * 32 + 8));
}
template <int MB>
__device__ __forceinline__ const float *rest_of(const _Float16 *M) {
  return rest_of<MB>(const_cast<_Float16 *>(M));
}

// What the rests add to a block of a symmetric product, where its sums start: to
// the diagonal's elements, of which a lane in four holds one in each of two parts.
template <int MB>
__device__ __forceinline__ void block_start(const _Float16 *P, const _Float16 *Q, int i, int j,
                                            int lane, Block &acc) {
#pragma unroll
  for (int p = 0; p < 4; ++p) acc[p / 2][p % 2] = f32x4{};
  if (i != j) return;
  const float *dp = rest_of<MB>(P), *dq = rest_of<MB>(Q);
  const int at = (lane & 15) - (lane >> 4) * 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int c = i * 32 + t * 16 + (lane & 15), to = c * (MB * 32 + 8) + c;
    const float more = (dp[c] + dq[c]) * float(P[to]) * float(Q[to]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][t][e] = at == e ? more : 0.0f;
  }
}

// The wave's block of a symmetric MB x MB one.  Of the larger ones, which the
// reading of LDS bounds, those on and below the diagonal are computed and
// written twice (128 x 128, without the rests: 31.0 -> 28.2 us); of the smaller
// all, which the latency bounds (64 x 512: 31.3 us, with half of them 31.9).
template <int MB>
struct Lower {
  static constexpr bool kHalf = MB > 2;
  static constexpr int kBlocks = kHalf ? MB * (MB + 1) / 2 : MB * MB;
  static_assert(kBlocks <= kSmallWaves, "a wave has one block");
  int i, j;
  __device__ __forceinline__ explicit Lower(int wave)
      : i(!kHalf ? wave / MB : wave < 1 ? 0 : wave < 3 ? 1 : wave < 6 ? 2 : 3),
        j(kHalf ? wave - i * (i + 1) / 2 : wave % MB) {}
  // f(r, c, rows r..r+3 of column c) to C.  They are neighbours in row c too.
  template <class F>
  __device__ __forceinline__ void put(_Float16 *C, int lane, const Block &acc, F f) const {
    constexpr int pm = MB * 32 + 8;
    // Of the two parts on the diagonal a lane in four holds an element each.
    float rest[2];
    const int at = (lane & 15) - (lane >> 4) * 4;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = i * 32 + p / 2 * 16 + (lane >> 4) * 4, c = j * 32 + p % 2 * 16 + (lane & 15);
      const f32x4 v = f(r, c, acc[p / 2][p % 2]);
      const half4 h = narrow4(v);
      *reinterpret_cast<half4 *>(C + c * pm + r) = h;
      if (kHalf && i != j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) C[(r + e) * pm + c] = h[e];
      }
      if (p / 2 == p % 2) {
        rest[p / 2] = v[0];
#pragma unroll
        for (int e = 1; e < 4; ++e) rest[p / 2] = at == e ? v[e] : rest[p / 2];
      }
    }
    if (i == j && at >= 0 && at < 4) {
      float *to = rest_of<MB>(C) + i * 32 + (lane & 15);
      to[0] = rest_in(rest[0]);
      to[16] = rest_in(rest[1]);
    }
  }
};

// C = P Q of symmetric matrices that commute.  All waves; a barrier follows.
template <int MB>
__device__ __forceinline__ void short_mul(const _Float16 *P, const _Float16 *Q, _Float16 *C,
                                          int wave, int lane) {
  if (wave < Lower<MB>::kBlocks) {
    const Lower<MB> at(wave);
    Block acc;
    block_start<MB>(P, Q, at.i, at.j, lane, acc);
    block_mul<MB>(P, Q, at.i, at.j, lane, acc);
    at.put(C, lane, acc, [](int, int, const f32x4 &v) { return v * kBack1; });
  }
  __syncthreads();
}

// B = a I + b A + c A A.
template <int MB>
__device__ __forceinline__ void short_poly(const float *k, const _Float16 *A, _Float16 *B, int wave,
                                           int lane) {
  constexpr int pm = MB * 32 + 8;
  if (wave < Lower<MB>::kBlocks) {
    const Lower<MB> at(wave);
    const float *d = rest_of<MB>(A);
    Block acc;
    block_start<MB>(A, A, at.i, at.j, lane, acc);
    block_mul<MB>(A, A, at.i, at.j, lane, acc);
    at.put(B, lane, acc, [&](int r, int c, f32x4 v) {
      const half4 old = *reinterpret_cast<const half4 *>(A + c * pm + r);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = __builtin_fmaf(k[1], float(old[e]), (k[2] * kBack1) * v[e]);
      if (at.i == at.j) {
        const float more = k[0] * kScale + k[1] * d[c] * float(A[c * pm + c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += r + e == c ? more : 0.0f;
      }
      return v;
    });
  }
  __syncthreads();
}

// Block i, j of B X.
template <int MB>
__device__ __forceinline__ void times(const _Float16 *B, const _Float16 *xt, int i, int j, int lane,
                                      Block &acc) {
  const float *rest = rest_of<MB>(B) + i * 32 + (lane >> 4) * 4;
  f32x4 d[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) d[e] = *reinterpret_cast<const f32x4 *>(rest + e * 16) + 1.0f;
  acc[0][0] = acc[0][1] = acc[1][0] = acc[1][1] = f32x4{};
  block_mul<MB>(B, xt, i, j, lane, acc);
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[p / 2][p % 2][n] *= d[p / 2][n];
}

// A matrix's (or a strip's) rp x cp elements in LDS, in the caller's
// orientation, and from there turned; rows of the caller's matrix past `rows`
// and columns past `cols` are zeros.  A barrier follows.
template <class TG>
struct Brought {
  Eight<TG> v[kSmallPacks];
  int per, packs;
  __device__ __forceinline__ void load(const typename TG::raw *g, int64_t ld, int rp, int cp,
                                       int rows, int cols) {
    per = cp / 8;
    packs = rp * per;
#pragma unroll
    for (int i = 0; i < kSmallPacks; ++i) {
      const int p = int(threadIdx.x) + i * kSmallThreads;
      if (p >= packs) break;
      const int r = p / per, c = (p - r * per) * 8;
      v[i].load(g + r * ld, c, r < rows ? cols - c : 0);
    }
  }
  __device__ __forceinline__ double squares() const {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kSmallPacks; ++i) {
      if (int(threadIdx.x) + i * kSmallThreads >= packs) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fma(double(v[i].get(e)), double(v[i].get(e)), sum);
    }
    return sum;
  }
  __device__ __forceinline__ void place(double scale, _Float16 *same, _Float16 *turned) const {
    const int cp = per * 8, rp = packs / per;
#pragma unroll
    for (int i = 0; i < kSmallPacks; ++i) {
      const int p = int(threadIdx.x) + i * kSmallThreads;
      if (p >= packs) break;
      const int r = p / per, c = (p - r * per) * 8;
      half8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = _Float16(float(double(v[i].get(e)) * scale));
      *reinterpret_cast<half8 *>(same + r * (cp + 8) + c) = h;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < packs; p += kSmallThreads) {
      const int r = p / cp * 8, c = p % cp;
      half8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = same[(r + e) * (cp + 8) + c];
      *reinterpret_cast<half8 *>(turned + c * (rp + 8) + r) = h;
    }
    __syncthreads();
  }
};

// Sum over the workgroup's 1024 threads, in all of them.
__device__ __forceinline__ double small_sum(double v, double *lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kSmallWaves; ++w) v += lds[w];
  return v;
}

// What an update leaves: X or X^T (whichever are given) from the blocks of B X,
// in binary16, or the result in bf16.
template <int MB, bool LAST>
__device__ __forceinline__ void short_put(const Block *acc, int blocks, _Float16 *x, int pn,
                                          _Float16 *xt, int wave, int lane) {
  constexpr int pm = MB * 32 + 8;
#pragma unroll
  for (int u = 0; u < kSmallBlocks; ++u) {
    const int t = wave + u * kSmallWaves;
    if (t < blocks)
      block_each(t % MB, t / MB, lane, acc[u], [&](int r, int c, f32x4 v) {
        half4 h;
        if constexpr (LAST) {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = __builtin_bit_cast(_Float16, Bf16::store(v[e] * kBack2));
        } else {
          h = narrow4(v * kBack1);
        }
        if (xt) *reinterpret_cast<half4 *>(xt + c * pm + r) = h;
        if (x) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[(r + e) * pn + c] = h[e];
        }
      });
  }
}

// The bf16 result from LDS, rp x cp of pitch cp + 8, to rows x cols of o.
__device__ __forceinline__ void short_out(const _Float16 *from, int rp, int cp, uint16_t *o,
                                          int64_t ld, int rows, int cols) {
  struct __attribute__((packed, aligned(2))) Vec {
    half8 h;
  };
  const int per = cp / 8;
  for (int p = threadIdx.x; p < rp * per; p += kSmallThreads) {
    const int r = p / per, c = (p - r * per) * 8;
    if (r >= rows) break;
    uint16_t *to = o + r * ld + c;
    const _Float16 *h = from + r * (cp + 8) + c;
    if (c + 8 <= cols) {
      reinterpret_cast<Vec *>(to)->h = *reinterpret_cast<const half8 *>(h);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < cols) to[e] = reinterpret_cast<const uint16_t *>(h)[e];
    }
  }
}

struct SmallArgs {
  const void *g;
  uint16_t *o;
  int64_t ld_in, stride_in, ld_o, stride_o;
  double eps;
  int32_t rows, cols, mp, np, tall, steps;
  float coeffs[3 * ZS_ORTHO_MAX_STEPS];
};

int64_t small_lds(int64_t mp, int64_t np) {
  return mp * (np + 8) + np * (mp + 8) + 2 * short_size(mp);
}

// A matrix whose X, X^T, A and B fit in the LDS of one CU: one workgroup, one
// launch (96 x 128: 17 launches take 67 us, this 22 us; 64 x 512 68 and 32 us).
template <class TG, int MB>
__global__ void __launch_bounds__(kSmallThreads) ortho_small_kernel(const SmallArgs A) {
  __shared__ __align__(16) _Float16 lds[kSmallLds];
  int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int mp = MB * 32, pm = mp + 8;
  const int np = A.np, pn = np + 8, nb = np / 32;
  _Float16 *x = lds, *xt = x + mp * pn, *a = xt + np * pm, *b = a + short_size(mp);
  // the input's and output's orientation
  const int rp = A.tall ? np : mp, cp = A.tall ? mp : np;
  _Float16 *same = A.tall ? xt : x, *turned = A.tall ? x : xt;
  {
    Brought<TG> in;
    in.load(static_cast<const typename TG::raw *>(A.g) + int64_t(blockIdx.x) * A.stride_in, A.ld_in,
            rp, cp, A.rows, A.cols);
    // the sums' places are B's
    const double sum = small_sum(in.squares(), reinterpret_cast<double *>(b));
    in.place(double(kScale) / (sqrt(sum) + A.eps), same, turned);
  }
  for (int s = 0; s < A.steps; ++s) {
    // Opaque, so that no address is computed ahead of the loop and kept.
    asm volatile("" : "+v"(lane));
    if (wave < Lower<MB>::kBlocks) {
      const Lower<MB> at(wave);
      Block acc = {};
      const _Float16 *p = block_at(x, at.i, pn, lane), *q = block_at(x, at.j, pn, lane);
      BlockRegs f0, f1;
      f0.read(p, q, pn);
      for (int k = 1; k < nb; k += 2) {
        f1.read(p + k * 32, q + k * 32, pn);
        f0.add(acc);
        const int next = k + 1 < nb ? k + 1 : k;
        f0.read(p + next * 32, q + next * 32, pn);
        f1.add(acc);
      }
      if (nb & 1) f0.add(acc);
      at.put(a, lane, acc, [](int, int, const f32x4 &v) { return v * kBack1; });
    }
    __syncthreads();
    short_poly<MB>(A.coeffs + 3 * s, a, b, wave, lane);
    Block acc[kSmallBlocks];
#pragma unroll
    for (int u = 0; u < kSmallBlocks; ++u) {
      const int t = wave + u * kSmallWaves;
      if (t < MB * nb) times<MB>(b, xt, t % MB, t / MB, lane, acc[u]);
    }
    __syncthreads();  // X^T has been read
    if (s + 1 < A.steps)
      short_put<MB, false>(acc, MB * nb, x, pn, xt, wave, lane);
    else
      short_put<MB, true>(acc, MB * nb, A.tall ? nullptr : x, pn, A.tall ? xt : nullptr, wave, lane);
    __syncthreads();
  }
  short_out(same, rp, cp, A.o + int64_t(blockIdx.x) * A.stride_o, A.ld_o, A.rows, A.cols);
}

// Longer ones in strips of 128 columns of X, a workgroup each.  Between two
// updates of X only A is needed of all strips together: each leaves its part of
// X X^T, one launch adds them, and the next update's workgroups all work out
// the polynomials in A again, two steps of them where the coefficients allow
// it, and apply them to their strip.  64 x 13824: 8 launches, 36 us, in place of
// 19, 105 us.  What is left is launches and waiting: at 128 rows a product of 128^3
// takes 1.5 us, of which one CU's matrix cores work 0.2.  (Of the one-workgroup
// kernel's time, 96 x 128 to 128 x 160, the LDS is busy 43-57%, a third of that with
// bank conflicts, the matrix cores 11-18%; its waves wait 49-63%.)
constexpr int kStripCols = 128, kStripRows = 128;

struct StripArgs {
  const void *g;
  uint16_t *o;
  int64_t ld_in, stride_in, ld_o, stride_o;
  const double *partials;  // of the norm, [batch][blocks]
  double eps;
  _Float16 *xt;   // [batch][strips * kStripCols][mp]
  float *parts;   // [batch][strips][mp][mp] of X X^T, times 2^22
  _Float16 *a;    // [batch][short_size(mp)], as it lies in LDS
  int32_t blocks, rows, cols, tall, strips, pair;
  float k[6];     // this update's coefficients
};

// This strip's part of X X^T, and its X^T for the next update.
template <int MB>
__device__ __forceinline__ void strip_leave(const StripArgs &A, const _Float16 *x,
                                            const _Float16 *xt, int wave, int lane) {
  constexpr int mp = MB * 32, pm = mp + 8;
  const int64_t strip = int64_t(blockIdx.y) * A.strips + blockIdx.x;
  if (wave < MB * MB) {
    Block acc = {};
    block_mul<kStripCols / 32>(x, x, wave / MB, wave % MB, lane, acc);
    float *out = A.parts + strip * (mp * mp);
    block_each(wave / MB, wave % MB, lane, acc, [&](int r, int c, f32x4 v) {
      *reinterpret_cast<f32x4 *>(out + c * mp + r) = v;
    });
  }
  _Float16 *to = A.xt + strip * (kStripCols * mp);
  for (int p = threadIdx.x; p < kStripCols * mp / 8; p += kSmallThreads) {
    const int r = p / (mp / 8), c = p % (mp / 8) * 8;
    *reinterpret_cast<half8 *>(to + p * 8) = *reinterpret_cast<const half8 *>(xt + r * pm + c);
  }
}

template <class TG, int MB>
__global__ void __launch_bounds__(kSmallThreads) ortho_strip_in_kernel(const StripArgs A) {
  constexpr int mp = MB * 32, pm = mp + 8, W = kStripCols;
  __shared__ __align__(16) _Float16 lds[mp * (W + 8) + W * pm];
  __shared__ double sums[kSmallWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  _Float16 *x = lds, *xt = lds + mp * (W + 8);
  const int64_t first = int64_t(blockIdx.x) * W;  // column of X
  const typename TG::raw *g = static_cast<const typename TG::raw *>(A.g) +
                              blockIdx.y * A.stride_in + first * (A.tall ? A.ld_in : 1);
  const int rows = A.tall ? int(A.rows - first) : A.rows;
  const int cols = A.tall ? A.cols : int(A.cols - first);
  Brought<TG> in;
  in.load(g, A.ld_in, A.tall ? W : mp, A.tall ? mp : W, rows, cols);
  double sum = 0.0;
  for (int i = threadIdx.x; i < A.blocks; i += kSmallThreads)
    sum += A.partials[int64_t(blockIdx.y) * A.blocks + i];
  sum = small_sum(sum, sums);
  in.place(double(kScale) / (sqrt(sum) + A.eps), A.tall ? xt : x, A.tall ? x : xt);
  strip_leave<MB>(A, x, xt, wave, lane);
}

// A from the strips' parts, in their order within each of 64 interleaved
// groups, the groups then in order.
__global__ void __launch_bounds__(1024) ortho_strip_sum_kernel(const StripArgs A, int mp) {
  __shared__ float lds[64][68];
  const int64_t b = blockIdx.y, square = mp * mp;
  const int at = blockIdx.x * 64;
  const float *p = A.parts + b * A.strips * square + at + threadIdx.x * 4;
  f32x4 s = {};
#pragma unroll 4
  for (int k = threadIdx.y; k < A.strips; k += 64)
    s += *reinterpret_cast<const f32x4 *>(p + int64_t(k) * square);
  *reinterpret_cast<f32x4 *>(&lds[threadIdx.y][threadIdx.x * 4]) = s;
  __syncthreads();
  const int t = threadIdx.y * 16 + threadIdx.x;
  if (t >= 64) return;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 64; ++k) sum += lds[k][t];
  const int r = (at + t) / mp, c = (at + t) - r * mp;
  _Float16 *to = A.a + b * short_size(mp);
  to[r * (mp + 8) + c] = _Float16(sum * kBack1);
  if (r == c) reinterpret_cast<float *>(to + mp * (mp + 8))[r] = rest_in(sum * kBack1);
}

template <int MB, bool LAST>
__global__ void __launch_bounds__(kSmallThreads) ortho_strip_step_kernel(const StripArgs A) {
  constexpr int mp = MB * 32, pm = mp + 8, W = kStripCols, square = short_size(mp);
  // X lies over B and C, which are done with by then, where LDS is full
  constexpr int xat = MB == 4 ? square : 3 * square;
  static_assert(MB < 4 || mp * (W + 8) <= 2 * square, "X in B and C's place");
  __shared__ __align__(16) _Float16 lds[W * pm + (MB == 4 ? 3 * square : 3 * square + mp * (W + 8))];
  int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  _Float16 *xt = lds, *a = xt + W * pm, *b = a + square, *c = b + square, *x = a + xat;
  const int64_t strip = int64_t(blockIdx.y) * A.strips + blockIdx.x;
  for (int p = threadIdx.x; p < square / 8; p += kSmallThreads)
    reinterpret_cast<half8 *>(a)[p] =
        reinterpret_cast<const half8 *>(A.a + int64_t(blockIdx.y) * square)[p];
  for (int p = threadIdx.x; p < W * mp / 8; p += kSmallThreads)
    *reinterpret_cast<half8 *>(xt + p / (mp / 8) * pm + p % (mp / 8) * 8) =
        *reinterpret_cast<const half8 *>(A.xt + strip * (W * mp) + p * 8);
  __syncthreads();
  short_poly<MB>(A.k, a, b, wave, lane);
  const _Float16 *by = b;
  if (A.pair) {
    // A of the next step is B A B; its B times this one's is applied to X
    short_mul<MB>(b, a, c, wave, lane);
    short_mul<MB>(c, b, a, wave, lane);
    short_poly<MB>(A.k + 3, a, c, wave, lane);
    short_mul<MB>(c, b, a, wave, lane);
    by = a;
  }
  constexpr int blocks = MB * W / 32;
  static_assert(blocks <= kSmallWaves * kSmallBlocks, "a wave's blocks");
  Block acc[kSmallBlocks];
#pragma unroll
  for (int u = 0; u < kSmallBlocks; ++u) {
    const int t = wave + u * kSmallWaves;
    if (t < blocks) times<MB>(by, xt, t % MB, t / MB, lane, acc[u]);
  }
  __syncthreads();  // X^T, B and C have been read
  short_put<MB, LAST>(acc, blocks, LAST && A.tall ? nullptr : x, W + 8,
                      LAST && !A.tall ? nullptr : xt, wave, lane);
  __syncthreads();
  if constexpr (LAST) {
    const int64_t first = int64_t(blockIdx.x) * W;
    uint16_t *o = A.o + blockIdx.y * A.stride_o + first * (A.tall ? A.ld_o : 1);
    if (A.tall) short_out(xt, W, mp, o, A.ld_o, int(A.rows - first), A.cols);
    else short_out(x, mp, W, o, A.ld_o, A.rows, int(A.cols - first));
  } else {
    strip_leave<MB>(A, x, xt, wave, lane);
  }
}

// ------------------------------------------------------------------- host

constexpr float kCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr float kPairMost = 16.0f;
constexpr int64_t kCacheBytes = INT64_C(256) << 20;

// Whether two steps may be taken together: rounding in A comes out of the pair
// a a' times as large.
bool pairs(const float *k, const float *k2) {
  return k[0] * k2[0] > 0.0f && k[0] * k2[0] <= kPairMost;
}

constexpr int64_t kMaxSide = INT64_C(1) << 20;

bool muon_ok(const zs_muon_desc *d) {
  return d && d->n >= 0 && d->n_d >= 1 && d->n_d <= ZS_MAX_ND && d->mu >= 0.0f && d->mu < 1.0f &&
         (d->nesterov == 0 || d->nesterov == 1) && (d->dtype == ZS_F32 || d->dtype == ZS_BF16) &&
         d->weight_decay >= 0.0f && std::isfinite(d->weight_decay) &&
         d->n <= INT64_C(0x7fffffff) * kThreads * 8;
}

bool ortho_ok(const zs_ortho_desc *d) {
  if (!d || d->batch < 0 || d->rows < 0 || d->cols < 0) return false;
  if (d->rows > kMaxSide || d->cols > kMaxSide || d->batch > 65535) return false;
  if (!dtype_size(d->dtype)) return false;
  if (d->steps < 1 || d->steps > ZS_ORTHO_MAX_STEPS) return false;
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return false;
  const int64_t big = INT64_C(1) << 40;
  if (d->ld_in != 0 && (d->ld_in < d->cols || d->ld_in > big)) return false;
  if (d->ld_out != 0 && (d->ld_out < d->cols || d->ld_out > big)) return false;
  if (d->stride_in < 0 || d->stride_in > big || d->stride_out < 0 || d->stride_out > big)
    return false;
  // the output's matrices must not overlap
  const int64_t ld_out = d->ld_out ? d->ld_out : d->cols;
  if (d->batch > 1 && d->rows > 0 && d->stride_out != 0 &&
      d->stride_out < (d->rows - 1) * ld_out + d->cols)
    return false;
  if (d->coeffs)
    for (int i = 0; i < 3 * d->steps; ++i)
      if (!std::isfinite(d->coeffs[i])) return false;
  return true;
}

// The tile shapes, how many workgroups the card holds at once, and what a tile
// costs in microseconds (measured): 64 of k when few workgroups run and when
// the card is full of them (then the clock is lower and L2 is shared), the
// rest of a tile, and each part of a cut one.
// The shapes between 256 x 256 and 128 x 256 fill the last turn of the card
// better: 5120 x 5120 is 400 tiles of 256 x 256 (two turns of 256, 279 us) or
// 460 of 224 x 256 (253 us); its lower triangle 210 (144 us) or 251 (128 us).
// (Over many products, when the clock has fallen, idle CUs leave it higher and
// the two differ by 1%.)
// Smaller tiles give more workgroups but read more: 4 of 1024 x 1024 take
// 30 us as 64 tiles of 256 x 256, 16 us as 256 of 128 x 128, 21 us as 1024 of
// 64 x 64.
struct Shape {
  int TR, TC, cap;
  double alone, full, rest, part;
};
constexpr Shape kShapes[] = {
    {256, 256, 256, 1.05, 1.74, 12.5, 0.0},  {224, 256, 256, 0.95, 1.49, 11.5, 0.0},
    {192, 256, 256, 0.86, 1.29, 10.8, 0.0},  {128, 256, 256, 0.58, 0.82, 9.6, 4.2},
    {128, 128, 256, 0.33, 0.467, 8.0, 1.15}, {64, 64, 512, 0.22, 0.39, 5.5, 1.5},
};
constexpr int kNumShapes = sizeof kShapes / sizeof kShapes[0];
constexpr int kFirstCut = 3, kMostParts = 8;
constexpr int64_t kMostTiles = 0xffffffff / 512;  // of a launch: it takes below 2^32 threads

// How one product is spread over the card: its tile shape, and whether the
// tiles are cut along k.
struct Way {
  int shape, tiles_r, tiles_c, per, grid, cut;
  double us;
};

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// r x c of `batch` matrices (half of it when symmetric) over k.
Way way_with(int64_t batch, int64_t r, int64_t c, int64_t k, bool symmetric, int shape) {
  const Shape &S = kShapes[shape];
  Way w = {};
  w.shape = shape;
  w.tiles_r = int(up(r, S.TR) / S.TR);
  w.tiles_c = int(up(c, S.TC) / S.TC);
  int64_t per = 0;
  if (symmetric)
    for (int i = 0; i < w.tiles_r; ++i) per += below(i, S.TR, S.TC, w.tiles_c);
  else
    per = int64_t(w.tiles_r) * w.tiles_c;
  const int64_t tiles = batch * per, nk = k / 64;
  if (tiles > kMostTiles) {
    w.us = INFINITY;
    return w;
  }
  w.per = int(per);
  w.grid = int(tiles);
  // n workgroups at once, each over `steps` 64s of k
  const auto turn = [&](int64_t n, double steps) {
    return steps * (S.alone + (S.full - S.alone) * double(n) / S.cap) + S.rest;
  };
  w.us = double(tiles / S.cap) * turn(S.cap, double(nk)) +
         (tiles % S.cap ? turn(tiles % S.cap, double(nk)) : 0.0);
  // few tiles over a long k: cut along it (larger tiles: parts cost too much)
  for (int64_t parts = shape < kFirstCut ? kMostParts + 1 : 2; parts <= kMostParts && parts * tiles <= S.cap && parts <= nk; ++parts) {
    const double us = turn(parts * tiles, double(nk) / double(parts)) + double(parts) * S.part;
    if (tiles <= kCutTiles && us < w.us) {
      w.us = us;
      w.cut = int(tiles);
      w.grid = int(tiles * parts);
    }
  }
  return w;
}

Way way_of(int64_t batch, int64_t r, int64_t c, int64_t k, bool symmetric) {
  Way best = way_with(batch, r, c, k, symmetric, 0);
  for (int i = 1; i < kNumShapes; ++i) {
    const Way w = way_with(batch, r, c, k, symmetric, i);
    if (w.us < best.us) best = w;
  }
  return best;
}

struct Plan {
  int64_t m, n, mp, np;
  Way gram, poly, next;
  int blocks;   // that sum the squares of a matrix
  bool small;   // one workgroup per matrix, padded to 32
  int strips;   // of kStripCols columns of X, a workgroup each, padded to 32 rows; or 0
  bool paired;  // two steps at a time where the coefficients allow it
  bool tall;
  int64_t partials, arrived, parts, x, xt, y, yt, a, b, c, rests, bytes;  // offsets into the workspace
};

Plan plan_of(const zs_ortho_desc &d) {
  Plan p = {};
  p.tall = d.rows > d.cols;
  p.m = p.tall ? d.cols : d.rows;
  p.n = p.tall ? d.rows : d.cols;
  p.mp = up(p.m, 32);
  p.np = up(p.n, 32);
  p.small = small_lds(p.mp, p.np) <= kSmallLds;
  if (p.small) {
    p.bytes = 256;  // not used: every plan asks for a workspace
    return p;
  }
  const int64_t runs = d.rows * (up(d.cols, kNormRun) / kNormRun);
  p.blocks = int(runs < kNormBlocks ? runs : kNormBlocks);
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t was = at;
    at += up(bytes, 256);
    return was;
  };
  p.partials = take(d.batch * p.blocks * 8);
  p.arrived = take(kCutTiles * 4);
  p.strips = p.mp <= kStripRows ? int(up(p.n, kStripCols) / kStripCols) : 0;
  if (p.strips) {
    p.np = int64_t(p.strips) * kStripCols;
    p.xt = take(d.batch * p.np * p.mp * 2);
    p.parts = take(d.batch * p.strips * p.mp * p.mp * 4);
    p.a = take(d.batch * short_size(p.mp) * 2);
    p.bytes = at;
    return p;
  }
  p.mp = up(p.m, 64);
  p.np = up(p.n, 64);
  p.gram = way_of(d.batch, p.mp, p.mp, p.np, true);
  p.poly = way_of(d.batch, p.mp, p.mp, p.mp, true);
  p.next = way_of(d.batch, p.mp, p.np, p.mp, false);
  if (!std::isfinite(p.gram.us) || !std::isfinite(p.next.us)) {
    p.bytes = -1;
    return p;
  }
  p.paired = d.steps > 1 && 3 * p.poly.us < p.gram.us + p.next.us;
  const auto parts = [](const Way &w) {
    return w.cut ? int64_t(w.grid) * 2 * kShapes[w.shape].TR * kShapes[w.shape].TC * 4 : 0;
  };
  int64_t most = parts(p.next);
  if (parts(p.gram) > most) most = parts(p.gram);
  if (parts(p.poly) > most) most = parts(p.poly);
  p.parts = take(most);
  p.x = take(d.batch * p.mp * p.np * 2);
  p.xt = take(d.batch * p.mp * p.np * 2);
  p.y = take(d.batch * p.mp * p.np * 2);
  p.yt = take(d.batch * p.mp * p.np * 2);
  p.a = take(d.batch * p.mp * p.mp * 2);
  p.b = take(d.batch * p.mp * p.mp * 2);
  p.c = p.paired ? take(d.batch * p.mp * p.mp * 2) : 0;
  p.rests = take(3 * d.batch * p.mp * 4);
  p.bytes = at;
  return p;
}

template <int KIND, bool CUT, int I, int WR, int WC, int S>
void launch(const MulArgs &A, int grid, hipStream_t st) {
  hipLaunchKernelGGL((ortho_mul_kernel<KIND, CUT, kShapes[I].TR, kShapes[I].TC, WR, WC, S>), dim3(grid),
                     dim3(WR * WC * 64), 0, st, A);
}

// C (rows x cols) = P Q^T over k.
template <int KIND>
int multiply(MulArgs &A, const Way &w, int64_t rows, int64_t cols, int64_t k, hipStream_t st) {
  A.rows = int(rows);
  A.cols = int(cols);
  A.k = int(k);
  A.tiles_r = w.tiles_r;
  A.tiles_c = w.tiles_c;
  A.per = w.per;
  A.cut = w.cut;
  A.groups = w.grid;
  A.one = w.per == w.grid || (w.cut && w.per == w.cut);
  if (w.cut) {
    switch (w.shape) {
      case 3: launch<KIND, true, 3, 2, 4, 3>(A, w.grid, st); break;
      case 4: launch<KIND, true, 4, 2, 4, 5>(A, w.grid, st); break;
      default: launch<KIND, true, 5, 2, 2, 5>(A, w.grid, st); break;
    }
  } else {
    switch (w.shape) {
      case 0: launch<KIND, false, 0, 2, 4, 2>(A, w.grid, st); break;
      case 1: launch<KIND, false, 1, 2, 4, 2>(A, w.grid, st); break;
      case 2: launch<KIND, false, 2, 2, 4, 2>(A, w.grid, st); break;
      case 3: launch<KIND, false, 3, 2, 4, 3>(A, w.grid, st); break;
      case 4: launch<KIND, false, 4, 2, 4, 5>(A, w.grid, st); break;
      default: launch<KIND, false, 5, 2, 2, 5>(A, w.grid, st); break;
    }
  }
  return launched();
}

template <class TG>
int norm(const InArgs &A, int64_t batch, hipStream_t st) {
  hipLaunchKernelGGL(ortho_norm_kernel<TG>, dim3(A.blocks, unsigned(batch)), dim3(kThreads), 0,
                     st, A);
  return launched();
}

template <class TG>
int start(const InArgs &A, int64_t batch, hipStream_t st) {
  if (const int rc = norm<TG>(A, batch, st)) return rc;
  const int64_t rp = A.tall ? A.np : A.mp, cp = A.tall ? A.mp : A.np;
  hipLaunchKernelGGL(ortho_layout_kernel<TG>,
                     dim3(unsigned(up(cp, kStrip) / kStrip), unsigned(rp / 64), unsigned(batch)),
                     dim3(kThreads), 0, st, A);
  return launched();
}

// `steps` steps in strips.
template <class TG, int MB>
int strips_of(StripArgs &A, const zs_ortho_desc &d, hipStream_t st) {
  const dim3 grid{unsigned(A.strips), unsigned(d.batch)}, block{kSmallThreads};
  hipLaunchKernelGGL((ortho_strip_in_kernel<TG, MB>), grid, block, 0, st, A);
  int rc = launched();
  for (int s = 0; s < d.steps && !rc; s += A.pair + 1) {
    const float *k = d.coeffs ? d.coeffs + 3 * s : kCoeffs;
    const float *k2 = d.coeffs ? k + 3 : kCoeffs;
    A.pair = s + 1 < d.steps && pairs(k, k2);
    for (int i = 0; i < 3; ++i) {
      A.k[i] = k[i];
      A.k[i + 3] = A.pair ? k2[i] : 0.0f;
    }
    hipLaunchKernelGGL(ortho_strip_sum_kernel, dim3(MB * MB * 16, unsigned(d.batch)), dim3(16, 64),
                       0, st, A, MB * 32);
    if (s + A.pair + 1 < d.steps)
      hipLaunchKernelGGL((ortho_strip_step_kernel<MB, false>), grid, block, 0, st, A);
    else
      hipLaunchKernelGGL((ortho_strip_step_kernel<MB, true>), grid, block, 0, st, A);
    rc = launched();
  }
  return rc;
}

template <class TG>
int strips(StripArgs &A, int64_t mp, const zs_ortho_desc &d, hipStream_t st) {
  switch (mp / 32) {
    case 1: return strips_of<TG, 1>(A, d, st);
    case 2: return strips_of<TG, 2>(A, d, st);
    case 3: return strips_of<TG, 3>(A, d, st);
    default: return strips_of<TG, 4>(A, d, st);
  }
}

template <class TG>
int small(const SmallArgs &A, int64_t batch, hipStream_t st) {
  const dim3 grid{unsigned(batch)}, block{kSmallThreads};
  switch (A.mp / 32) {
    case 1: hipLaunchKernelGGL((ortho_small_kernel<TG, 1>), grid, block, 0, st, A); break;
    case 2: hipLaunchKernelGGL((ortho_small_kernel<TG, 2>), grid, block, 0, st, A); break;
    case 3: hipLaunchKernelGGL((ortho_small_kernel<TG, 3>), grid, block, 0, st, A); break;
    default: hipLaunchKernelGGL((ortho_small_kernel<TG, 4>), grid, block, 0, st, A); break;
  }
  return launched();
}

}  // namespace

extern "C" {

int zero_shard_muon_momentum(const zs_muon_desc *d, const zs_bf16 *const *contrib,
                             const float *m_in, float *m_out, void *update) {
  if (!muon_ok(d)) return ZS_EINVAL;
  if (d->n == 0) return ZS_OK;
  if (!contrib || !m_in || !m_out || !update) return ZS_EINVAL;
  MomentumArgs A;
  std::memset(&A, 0, sizeof A);
  for (int k = 0; k < d->n_d; ++k) {
    if (!contrib[k]) return ZS_EINVAL;
    if (!aligned(contrib[k], 16)) return ZS_EALIGN;
  }
  if (!aligned(m_in, 16) || !aligned(m_out, 16) || !aligned(update, 16)) return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  A.n_d = d->n_d;
  A.nesterov = d->nesterov;
  A.mu = double(d->mu);
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  const auto launch = [&](auto t) {
    using TU = decltype(t);
    for (int64_t from = 0; from < d->n; from += kPiece) {
      A.n = d->n - from < kPiece ? d->n - from : kPiece;
      for (int k = 0; k < d->n_d; ++k) A.rows.p[k] = contrib[k] + from;
      A.m_in = m_in + from;
      A.m_out = m_out + from;
      A.update = static_cast<typename TU::raw *>(update) + from;
      const dim3 grid(unsigned((A.n / 512 * 64 + A.n % 512 + kThreads - 1) / kThreads));
      if (grid.x <= kFew)
        hipLaunchKernelGGL((momentum_kernel<TU, true>), grid, dim3(kThreads), 0, st, A);
      else
        hipLaunchKernelGGL((momentum_kernel<TU, false>), grid, dim3(kThreads), 0, st, A);
      if (const int rc = launched()) return rc;
    }
    return int(ZS_OK);
  };
  return d->dtype == ZS_F32 ? launch(F32{}) : launch(Bf16{});
}

int zero_shard_muon_apply(const zs_muon_desc *d, const zs_bf16 *o, float lr, float scale,
                          const float *master_in, float *master_out, zs_bf16 *param_out) {
  if (!muon_ok(d) || !zs_args::step_ok(lr, 1) || !std::isfinite(scale)) return ZS_EINVAL;
  if (d->n == 0) return ZS_OK;
  if (!o || !master_in || !master_out || !param_out) return ZS_EINVAL;
  if (!aligned(o, 16) || !aligned(master_in, 16) || !aligned(master_out, 16) ||
      !aligned(param_out, 16))
    return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  for (int64_t from = 0; from < d->n; from += kPiece) {
    const int64_t n = d->n - from < kPiece ? d->n - from : kPiece;
    const ApplyArgs A{n, o + from, master_in + from, master_out + from, param_out + from,
                      double(lr) * double(d->weight_decay), double(lr) * double(scale)};
    hipLaunchKernelGGL(apply_kernel, dim3(unsigned((n + kThreads * 8 - 1) / (kThreads * 8))),
                       dim3(kThreads), 0, static_cast<hipStream_t>(d->stream), A);
    if (const int rc = launched()) return rc;
  }
  return ZS_OK;
}

int64_t zero_shard_ortho_workspace(const zs_ortho_desc *d) {
  if (!ortho_ok(d)) return -1;
  if (d->batch == 0 || d->rows == 0 || d->cols == 0) return 0;
  return plan_of(*d).bytes;
}

int zero_shard_ortho(const zs_ortho_desc *d, const void *g, zs_bf16 *o, void *workspace,
                     int64_t workspace_bytes) {
  if (!ortho_ok(d)) return ZS_EINVAL;
  if (d->batch == 0 || d->rows == 0 || d->cols == 0) return ZS_OK;
  const Plan p = plan_of(*d);
  if (!g || !o || !workspace || p.bytes < 0 || workspace_bytes < p.bytes) return ZS_EINVAL;
  if (!aligned(g, dtype_size(d->dtype)) || !aligned(o, 2) || !aligned(workspace, 256))
    return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  char *ws = static_cast<char *>(workspace);
  const auto half = [&](int64_t off) { return reinterpret_cast<_Float16 *>(ws + off); };
  const int64_t ld_in = d->ld_in ? d->ld_in : d->cols, ld_out = d->ld_out ? d->ld_out : d->cols;
  if (p.small) {
    SmallArgs A;
    std::memset(&A, 0, sizeof A);
    A.g = g;
    A.o = o;
    A.ld_in = ld_in;
    A.stride_in = d->stride_in ? d->stride_in : d->rows * ld_in;
    A.ld_o = ld_out;
    A.stride_o = d->stride_out ? d->stride_out : d->rows * ld_out;
    A.eps = double(d->eps);
    A.rows = int32_t(d->rows);
    A.cols = int32_t(d->cols);
    A.mp = int32_t(p.mp);
    A.np = int32_t(p.np);
    A.tall = p.tall;
    A.steps = d->steps;
    for (int i = 0; i < 3 * d->steps; ++i) A.coeffs[i] = d->coeffs ? d->coeffs[i] : kCoeffs[i % 3];
    return d->dtype == ZS_F32    ? small<F32>(A, d->batch, st)
           : d->dtype == ZS_BF16 ? small<Bf16>(A, d->batch, st)
                                 : small<F16>(A, d->batch, st);
  }
  InArgs in;
  std::memset(&in, 0, sizeof in);
  in.g = g;
  in.rows = d->rows;
  in.cols = d->cols;
  in.ld = ld_in;
  in.stride = d->stride_in ? d->stride_in : d->rows * ld_in;
  in.partials = reinterpret_cast<double *>(ws + p.partials);
  in.arrived = reinterpret_cast<int32_t *>(ws + p.arrived);
  in.x = half(p.x);
  in.xt = half(p.xt);
  in.mp = p.mp;
  in.np = p.np;
  in.eps = double(d->eps);
  in.tall = p.tall;
  in.blocks = p.blocks;
  if (p.strips) {
    StripArgs A;
    std::memset(&A, 0, sizeof A);
    A.g = g;
    A.o = o;
    A.ld_in = ld_in;
    A.stride_in = in.stride;
    A.ld_o = ld_out;
    A.stride_o = d->stride_out ? d->stride_out : d->rows * ld_out;
    A.partials = in.partials;
    A.eps = in.eps;
    A.xt = half(p.xt);
    A.parts = reinterpret_cast<float *>(ws + p.parts);
    A.a = half(p.a);
    A.blocks = p.blocks;
    A.rows = int32_t(d->rows);
    A.cols = int32_t(d->cols);
    A.tall = p.tall;
    A.strips = p.strips;
    const auto all = [&](auto t) {
      using TG = decltype(t);
      const int rc = norm<TG>(in, d->batch, st);
      return rc ? rc : strips<TG>(A, p.mp, *d, st);
    };
    return d->dtype == ZS_F32 ? all(F32{}) : d->dtype == ZS_BF16 ? all(Bf16{}) : all(F16{});
  }
  int rc = d->dtype == ZS_F32    ? start<F32>(in, d->batch, st)
           : d->dtype == ZS_BF16 ? start<Bf16>(in, d->batch, st)
                                 : start<F16>(in, d->batch, st);
  _Float16 *x = half(p.x), *xt = half(p.xt), *y = half(p.y), *yt = half(p.yt);
  MulArgs A;
  std::memset(&A, 0, sizeof A);
  A.parts = reinterpret_cast<float *>(ws + p.parts);
  A.arrived = in.arrived;
  A.o = o;
  A.out_rows = d->rows;
  A.out_cols = d->cols;
  A.ld_o = ld_out;
  A.stride_o = d->stride_out ? d->stride_out : d->rows * ld_out;
  A.tall = p.tall;
  A.wide = aligned(o, 16) && d->cols % 8 == 0 && ld_out % 8 == 0 && A.stride_o % 8 == 0;
  const int64_t square = p.mp * p.mp, whole = p.mp * p.np;
  _Float16 *a = half(p.a), *b = half(p.b), *c = half(p.c);
  const auto rest_of = [&](const _Float16 *of) {
    return reinterpret_cast<float *>(ws + p.rests) +
           (of == a ? 0 : of == b ? 1 : 2) * d->batch * p.mp;
  };
  // C = P Q^T of m x m matrices that commute, and poly's combination
  const auto small = [&](auto kind, const _Float16 *pp, const _Float16 *qq, _Float16 *cc) {
    A.p = pp;
    A.q = qq;
    A.rest_p = rest_of(pp);
    A.rest_q = rest_of(qq);
    A.rest_c = rest_of(cc);
    A.stride_p = A.stride_q = A.stride_c = square;
    A.c = cc;
    return multiply<kind.value>(A, p.poly, p.mp, p.mp, p.mp, st);
  };
  const auto poly = [&](const float *k, const _Float16 *from, _Float16 *to) {
    A.a = k[0];
    A.b = k[1];
    A.cc = k[2];
    return small(Const<kPoly>{}, from, from, to);
  };
  // X and X^T are not both held by the card's cache: X, which the next product
  // reads, should be, and X^T not take its place (13824 x 5120: 4.16 -> 4.09 ms;
  // 5120 x 5120, which fits: the same either way, with X past them too +4%).
  A.past = 4 * d->batch * whole > kCacheBytes;
  for (int s = 0; s < d->steps && !rc;) {
    const float *k = d->coeffs ? d->coeffs + 3 * s : kCoeffs;
    const float *k2 = d->coeffs ? k + 3 : kCoeffs;
    A.p = A.q = x;
    A.rest_p = A.rest_q = nullptr;
    A.rest_c = rest_of(a);
    A.stride_p = A.stride_q = whole;
    A.c = a;
    A.stride_c = square;
    if ((rc = multiply<kGram>(A, p.gram, p.mp, p.mp, p.np, st))) break;
    if ((rc = poly(k, a, b))) break;
    const _Float16 *by = b;
    ++s;
    if (p.paired && s < d->steps && pairs(k, k2)) {
      // A of the next step is B A B; its B times this one's is applied to X
      if ((rc = small(Const<kGram>{}, b, a, c)) || (rc = small(Const<kGram>{}, c, b, a)) ||
          (rc = poly(k2, a, c)) || (rc = small(Const<kGram>{}, c, b, a)))
        break;
      by = a;
      ++s;
    }
    A.p = by;
    A.rest_p = rest_of(by);
    A.stride_p = square;
    A.q = xt;
    A.stride_q = whole;
    if (s < d->steps) {
      A.c = y;
      A.ct = yt;
      A.stride_c = whole;
      rc = multiply<kNext>(A, p.next, p.mp, p.np, p.mp, st);
      _Float16 *v = x;
      x = y;
      y = v;
      v = xt;
      xt = yt;
      yt = v;
    } else {
      rc = multiply<kLast>(A, p.next, p.mp, p.np, p.mp, st);
    }
  }
  return rc;
}

}  // extern "C"
