// zero_shard_seam.hip -- the seam between two blocks of a network, forward and
// backward, on MI355X (gfx950) (declarations and the contract:
// include/zero_shard.h).
//
//   forward   n = N0(block) gamma0 + beta0;  s = round(a x + gate n);
//             y = N1(s) gamma + beta
//   backward  D = N1'(dy gamma) + dsum;  dx = a D;  dn = gate D;
//             dblock = N0'(dn gamma0);  the columns' sums of dy h1, dy, dn h0, dn
//
// N0 and N1 are layer or RMS norms (h: their values before gain and bias), N'
// their transposed derivatives: rstd (g - mean(g) - h mean(g h)), without
// mean(g) for RMS.  Everything is binary32 inside, each output rounded once.
//
// Both directions are HBM-bound: a row is read once, stays in registers between
// its two norms (eight columns a thread, sixteen above 8192), and the next row
// is loaded before this one is worked on.  A gate that is one number per column
// factors out of the backward pass's sums: with E = D (or D times the
// element's gate) every gradient of the first norm and the gate follows from
// sum(E h0) and sum(E), so a thread carries four sums a column, whatever is asked
// for.  A workgroup leaves one partial row of each, and a second launch adds them
// in a fixed order: no atomics, so the same inputs give the same bits.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "zero_shard.h"
#include "zs_rows.h"

namespace {

using namespace zs_dev;

constexpr int kThreads = 256;
constexpr int kMaxCols = ZS_BLOCKNORM_MAX_COLS;  // sixteen columns of 1024 threads
constexpr int kCus = 256;
constexpr int kMaxParts = 256;  // partial rows of the columns' sums
constexpr int kResident = 1280;    // threads of the forward pass on a CU
constexpr int kPairThreads = 768;  // most that hold two rows, or sixteen columns, of the
                                  // backward pass without spilling

// A thread's columns: N times eight, `per` threads apart.  Where a row ends inside a
// thread's eight (TAIL), they are the row's last eight, of which the first `skip` are
// the thread's before it: every load is of 16 bytes a piece, and nothing waits for one
// on the way (with the last elements loaded one by one 32768 x 511 bf16 took 67 us
// forward and 127 backward for 33 and 64).  Not with sixteen columns a thread, where the
// registers do not hold what that takes (4096 x 9001 bf16 166 us for 151), nor in
// rows of fewer than eight.  Of sixteen the first eight are always the row's.
template <bool TAIL, int N>
struct Mine : Columns<N> {
  static constexpr bool kShift = TAIL && N == 1;
  int skip = 0;
  bool ends = false;  // whether a thread of this wave skips some
  __device__ __forceinline__ Mine(int t, int per, int cols) : Columns<N>(t, per, cols) {
    if constexpr (kShift) {
      int &left = this->left[0];
      if (left > 0 && left < 8 && cols >= 8) {
        skip = 8 - left;
        this->i[0] -= unsigned(skip);
        left = 8;
      }
      ends = __ballot(skip != 0) != 0;
    }
  }
  // Whether element e is the row's and this thread's, or (not TAIL) all eight.
  __device__ __forceinline__ bool live(int n, int e) const {
    if (n < N - 1) return true;
    return TAIL ? (!kShift || e >= skip) && e < this->left[n] : this->left[n] > 0;
  }
  template <bool ONCE, class T>
  __device__ __forceinline__ void get(Eight<T> &v, const void *row, int n, bool in) const {
    if (n < N - 1) v.template load<false, ONCE>(row, this->i[n], in ? 8 : 0);
    else v.template load<TAIL, ONCE>(row, this->i[n], in ? this->left[n] : 0);
  }
  // Elements that are not become zeros.
  template <class T>
  __device__ __forceinline__ void keep(Eight<T> &v, int n) const {
    if (kShift && ends) {
      int count = skip;
      asm volatile("" : "+v"(count));  // worked out here: there are no registers to keep masks in
      constexpr int kEach = sizeof(typename T::raw) == 4 ? 1 : 2;  // elements of a word
#pragma unroll
      for (int q = 0; q < 8 / kEach; ++q) {
        const unsigned part = kEach == 2 && count == 2 * q + 1 ? 0xffff0000u : ~0u;
        v.w[q] &= count >= kEach * (q + 1) ? 0u : part;
      }
    }
  }
  // The thread's elements.
  template <class T>
  __device__ __forceinline__ void put(const Eight<T> &v, void *row, int n) const {
    if (n < N - 1) v.template store<false>(row, this->i[n], 8);
    else if (!kShift || skip == 0) v.template store<TAIL>(row, this->i[n], this->left[n]);
    else store_last(v, row, this->i[n], skip);
  }
};

// sigmoid and its derivative, from t = exp(-|z|): nothing overflows and 1 - sigmoid
// loses nothing.  exp2 of the product's leading part, the rest to first order (below
// 2^-17 of it); the quotient by one Newton step.  Within 4 half steps of binary32, but 0
// (and the slope too) where they are below its least normal number, z < -87.34: there the
// exponential is 0 (from 87.34 on the slope alone is).
__device__ __forceinline__ float sigmoid(float z, float &slope) {
  constexpr float kLog2e = 1.44269504f, kRest = 1.92596304e-8f;  // of log2 e
  float a = -fabsf(z);
  a = a < -150.0f ? -150.0f : a;  // there t is 0; a NaN stays one
  const float hi = a * kLog2e;
  const float lo = __builtin_fmaf(a, kLog2e, -hi) + a * kRest;
  float t = __builtin_amdgcn_exp2f(hi);
  t = __builtin_fmaf(t, lo * 0.693147181f, t);
  const float y = 1.0f + t;
  float inv = __builtin_amdgcn_rcpf(y);
  inv = __builtin_fmaf(__builtin_fmaf(-y, inv, 1.0f), inv, inv);
  slope = t * inv * inv;
  return z < 0.0f ? t * inv : inv;
}

// Sums of M values (1, 2 or 4) over the wave in one register: afterwards its M
// equal parts hold one each, in order, in every lane.  Exchanging halves lets each
// lane carry on with one value instead of M: 10 instructions for 4 values where one
// after another took 44.
template <int M>
__device__ __forceinline__ float wave_sums(const float (&v)[M]) {
  static_assert(M == 1 || M == 2 || M == 4, "parts of a wave");
  const auto halves = [](float a, float b) {  // lanes 0-31: a, 32-63: b
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const auto rows = [](float a, float b) {  // of sixteen lanes: a, b, a, b
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  float x;
  if constexpr (M == 4) {
    x = rows(halves(v[0], v[2]), halves(v[1], v[3]));
  } else {
    const float h = halves(v[0], v[M - 1]);
    x = rows(h, h);
  }
  return sum16(x);
}

// The waves of a row group, and the LDS they exchange sums through.  One barrier an
// exchange: two buffers take turns, so a buffer is written again only after all have
// passed the next exchange's barrier.
struct Waves {
  float (*lds)[16][8];  // [2][wave of the workgroup][value]
  int first, count;     // of this row group
  int turn = 0;

  __device__ __forceinline__ float (*exchange(float x, int parts, float extra))[8] {
    const int lane = threadIdx.x & 63;
    float (*buf)[8] = lds[turn];
    turn ^= 1;
    float *own = buf[threadIdx.x >> 6];
    if ((lane & (64 / parts - 1)) == 0) own[lane * parts / 64] = x;
    if ((lane & 15) == 1) own[4 + (lane >> 4)] = extra;
    // all of LDS is there; loads from memory stay in flight
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    return buf + first;
  }

  // As wave_sums, over the row group.
  template <int M>
  __device__ __forceinline__ float sums(const float (&v)[M]) {
    const float x = wave_sums(v);
    if (count == 1) return x;
    const int lane = threadIdx.x & 63, w = lane & 15;
    float (*buf)[8] = exchange(x, M, 0.0f);
    return sum16(w < count ? buf[w][lane * M / 64] : 0.0f);
  }
};

// A row's mean and variance with one exchange: each wave centres its own columns,
// and the waves' sums are joined as those of samples with means of their own:
//   mean = sum n_w mean_w / cols;  cols var = sum (sq_w + n_w (mean_w - mean)^2)
// What a wave's mean is off by (off, the sum of its deviations, zero but for
// rounding) is made good, so that rows far from zero keep their digits.
struct Moments {
  float inv;               // 1 / cols
  float inv_own;           // 1 / columns of this wave (0: none)
  float n_lane, inv_lane;  // columns of the row group's wave lane % 16, and their inverse

  // A wave's columns: `per` threads share the row's pieces of eight, N of them each.
  template <int N>
  static __device__ __forceinline__ float columns(int wave, int per, int cols) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int left = cols - (k * per + wave * 64) * 8;
      n += left < 0 ? 0 : left < 512 ? left : 512;
    }
    return float(n);
  }

  // An infinite row keeps its mean.
  static __device__ __forceinline__ float finite(float v) {
    return fabsf(v) < INFINITY ? v : 0.0f;
  }

  // Deviations of R rows from their waves' means, in v's place; afterwards
  // (v + shift) rstd is normalised.
  template <bool TAIL, int N, int R>
  __device__ __forceinline__ void of(float (&v)[R][N][8], Waves &waves, const Mine<TAIL, N> &c,
                                     float eps, float (&mean)[R], float (&rstd)[R],
                                     float (&shift)[R]) {
    const int lane = threadIdx.x & 63;
    float own[R], two[2 * R];
    {
      float sum[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        sum[k] = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[k] += v[k][n][e];
      }
      const float x = wave_sums(sum) * inv_own;
#pragma unroll
      for (int k = 0; k < R; ++k) own[k] = lane_value(x, k * 64 / R);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float sq = 0.0f, off = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        // columns that are not the row's have no deviation from 0
        const float m = c.left[n] > 0 ? own[k] : 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = !TAIL || c.live(n, e) ? v[k][n][e] - m : 0.0f;
          sq = __builtin_fmaf(d, d, sq);
          off += d;
          v[k][n][e] = d;
        }
      }
      two[2 * k] = sq;
      two[2 * k + 1] = off;
    }
    const float x = wave_sums(two);
    // sixteen lanes a row, one a wave
    const int w = lane & 15, k = R == 2 ? lane >> 4 & 1 : 0;
    float m, square;
    if (waves.count == 1) {
      const float sq = R == 2 && k ? lane_value(x, 32) : lane_value(x, 0);
      const float off = R == 2 && k ? lane_value(x, 48) : lane_value(x, 64 / R / 2);
      const float o = finite(off) * inv;
      m = (R == 2 && k ? own[R - 1] : own[0]) + o;
      square = sq - o * o / inv;
    } else {
      float (*buf)[8] = waves.exchange(x, 2 * R, R == 2 && k ? own[R - 1] : own[0]);
      const bool in = w < waves.count;
      const float *from = buf[in ? w : 0];
      const float pivot = buf[0][4 + k];
      const float o = in ? finite(from[2 * k + 1]) * inv_lane : 0.0f;
      const float at = in && n_lane > 0.0f ? from[4 + k] + o : pivot;
      m = pivot + sum16(in ? n_lane * (at - pivot) : 0.0f) * inv;
      const float d = in && n_lane > 0.0f ? at - m : 0.0f;
      square = sum16(in ? (from[2 * k] - o * o * n_lane) + n_lane * d * d : 0.0f);
    }
    // of a constant row a difference of two equal values up to rounding; a NaN stays one
    const float var = square * inv;
    const float r = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean[j] = lane_value(m, j * 16);
      rstd[j] = lane_value(r, j * 16);
      shift[j] = own[j] - mean[j];
    }
  }
};

struct FwdArgs {
  int64_t rows, cols;
  int64_t ld_x, ld_b, ld_z, ld_s, ld_y;  // elements
  const void *x, *block, *z;             // z: gates of elements (before the sigmoid)
  const void *gate, *gamma0, *beta0, *gamma, *beta;
  void *sum, *y;
  float *stats;
  float eps, scale;
  int32_t center, post;
  int32_t per;  // threads of a row
};

// R rows at a time, each over `per` threads (a multiple of 64) of the
// workgroup's blockDim.x / per row groups.  TAIL: the columns are no multiple of 8.
// WIDE: a gate for each element.
template <class TX, class TP, int N, int R, bool TAIL, bool WIDE>
__global__ void __launch_bounds__(1024) seam_fwd_kernel(const FwdArgs A) {
  __shared__ float lds[2][16][8];
  const int per = A.per, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / per);
  const int t = threadIdx.x - sub * per, subs = blockDim.x / per;
  const int wave = __builtin_amdgcn_readfirstlane(t / 64), cols = int(A.cols);
  Waves waves{lds, sub * per / 64, per / 64};
  const float own = Moments::columns<N>(wave, per, cols);
  const float other = Moments::columns<N>(threadIdx.x & 15, per, cols);
  Moments moments{1.0f / float(cols), own > 0.0f ? 1.0f / own : 0.0f, other,
                  other > 0.0f ? 1.0f / other : 0.0f};
  const Mine<TAIL, N> c(t, per, cols);
  const auto live = [&](int n, int e) { return c.live(n, e); };
  // the gate of a column joins the first norm's gain and bias; both are 0 past the
  // row's end, and so is the sum there
  float gain[N][8], bias[N][8];
  {
    Eight<TP> g[N], p[N];
    load_params<TAIL>(g, A.gate, 1.0f, c);
    load_params<TAIL>(p, A.gamma0, 1.0f, c);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) gain[n][e] = live(n, e) ? g[n].get(e) * p[n].get(e) : 0.0f;
    load_params<TAIL>(p, A.beta0, 0.0f, c);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) bias[n][e] = live(n, e) ? g[n].get(e) * p[n].get(e) : 0.0f;
  }
  Eight<TP> gamma[N], beta[N];
  load_params<TAIL>(gamma, A.gamma, 1.0f, c);
  load_params<TAIL>(beta, A.beta, 0.0f, c);
  constexpr bool kOnce = N == 1 && !TAIL && sizeof(typename TX::raw) == 2;
  const int64_t step = int64_t(gridDim.x) * subs * R;
  struct Rows {
    Eight<TX> x[R][N], b[R][N], z[WIDE ? R : 1][WIDE ? N : 1];
  };
  const auto is = [&](int64_t r0, int k) { return r0 + k < A.rows; };
  const auto load = [&](Rows &v, int64_t r0) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const bool in = is(r0, k);
        c.template get<kOnce>(v.x[k][n], row_of<TX>(A.x, r0 + k, A.ld_x), n, in);
        c.template get<kOnce>(v.b[k][n], row_of<TX>(A.block, r0 + k, A.ld_b), n, in && A.block);
        if constexpr (WIDE)
          c.template get<kOnce>(v.z[k][n], row_of<TX>(A.z, r0 + k, A.ld_z), n, in);
      }
  };
  // Rows of values (zeros past their ends) to their normalised ones: v scale + shift.
  float v[R][N][8], mean[R], rstd[R], shift[R];
  const auto statistics = [&]() {
    if (A.center) {
      moments.of<TAIL>(v, waves, c, A.eps, mean, rstd, shift);
#pragma unroll
      for (int k = 0; k < R; ++k) shift[k] *= rstd[k];
    } else {
      float sq[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        sq[k] = shift[k] = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) sq[k] = __builtin_fmaf(v[k][n][e], v[k][n][e], sq[k]);
      }
      const float r = 1.0f / sqrtf(waves.sums(sq) * moments.inv + A.eps);
#pragma unroll
      for (int k = 0; k < R; ++k) rstd[k] = lane_value(r, k * 64 / R);
    }
  };
  const auto keep = [&](int64_t r0, int which) {
    if (t != 0 || !A.stats) return;
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (is(r0, k)) {
        A.stats[which * A.rows + r0 + k] = rstd[k];
        if (A.center) A.stats[(which + 2) * A.rows + r0 + k] = mean[k];
      }
  };
  // The next rows are on their way while these are worked on, where the
  // registers hold both.
  constexpr bool kAhead = N == 1;
  Rows ahead;
  if constexpr (kAhead) load(ahead, (int64_t(blockIdx.x) * subs + sub) * R);
  for (int64_t first = int64_t(blockIdx.x) * subs * R; first < A.rows; first += step) {
    const int64_t r0 = first + sub * R;
    Rows now;
    if constexpr (kAhead) {
      now = ahead;
      if (first + step < A.rows) load(ahead, r0 + step);
    } else {
      load(now, r0);
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        c.keep(now.x[k][n], n);
        c.keep(now.b[k][n], n);
        now.b[k][n].get(v[k][n]);
      }
    if (A.post) {
      statistics();
      keep(r0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        rstd[k] = 1.0f;
        shift[k] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float g = __builtin_fmaf(v[k][n][e], rstd[k], shift[k]);
          g = __builtin_fmaf(g, gain[n][e], bias[n][e]);
          if constexpr (WIDE) {
            float slope;
            g *= sigmoid(now.z[k][n].get(e), slope);
          }
          v[k][n][e] = __builtin_fmaf(A.scale, now.x[k][n].get(e), g);
        }
        if (A.block) {
          now.x[k][n].set(v[k][n]);
          if (is(r0, k))
            c.put(now.x[k][n], row_of<TX>(A.sum, r0 + k, A.ld_s), n);
        }
        now.x[k][n].get(v[k][n]);  // as it was rounded
      }
    statistics();
    keep(r0, 1);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (!is(r0, k)) break;
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float h = __builtin_fmaf(v[k][n][e], rstd[k], shift[k]);
          v[k][n][e] = __builtin_fmaf(h, gamma[n].get(e), beta[n].get(e));
        }
        now.x[k][n].set(v[k][n]);
        c.put(now.x[k][n], row_of<TX>(A.y, r0 + k, A.ld_y), n);
      }
    }
  }
}

struct BwdArgs {
  int64_t rows, cols;
  int64_t ld_dy, ld_ds, ld_s, ld_b, ld_z, ld_dx, ld_db, ld_dz;  // elements
  const void *dy, *dsum, *sum, *block, *z;
  const void *gate, *gamma0, *beta0, *gamma;
  const float *stats;
  void *dx, *dblock, *dz;
  void *dgate, *dgamma0, *dbeta0, *dgamma, *dbeta;  // of the columns
  float *part;  // [4][parts][cols]: sums of dy h1, dy, E h0, E
  float scale;
  int32_t center, post;
  int32_t want;   // 1: the sums of dy h1 and dy, 2: of E h0 and E
  int32_t parts;  // 0: no rows (the gradients are zero)
  int32_t per;    // threads of a row
};

// R rows at a time.  The columns' sums are in LDS, a thread's own places of it, all
// four, or of sixteen columns a thread the first two: with them in registers beside the
// rows 8192 x 5120 bf16 with element gates took 449 us for 183, fp32 349 for 199,
// and two rows at a time did not fit.
template <class TX, class TP, int N, int R, bool TAIL, bool WIDE, int kMost>
__global__ void __launch_bounds__(kMost) seam_bwd_kernel(const BwdArgs A) {
  constexpr int kInLds = N == 2 ? 2 : 4;
  __shared__ float lds[2][16][8];
  __shared__ f32x4 store[kInLds * N * 2 * kMost];
  const int per = A.per, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / per);
  const int t = threadIdx.x - sub * per, subs = blockDim.x / per;
  Waves waves{lds, sub * per / 64, per / 64};
  const Mine<TAIL, N> c(t, per, int(A.cols));
  // past a row's end: whole threads, or (TAIL) single elements
  const auto live = [&](int n, int e) { return !TAIL || c.live(n, e); };
  // Gains and the like stay in registers, or, with sixteen columns a thread, come
  // out of the caches for each row.
  constexpr bool kHeld = N == 1;
  Eight<TP> gamma_held, gamma0_held, beta0_held;
  float gain_held[8];  // gate gamma0, of a column
  const auto fetch = [&](Eight<TP> &v, const void *p, float none, int n) {
    if (p) {
      c.template get<false>(v, p, n, true);
    } else {
      const float all[8] = {none, none, none, none, none, none, none, none};
      v.set(all);
    }
  };
  const auto fetch_gain = [&](float (&v)[8], int n) {
    Eight<TP> g, p;
    fetch(g, A.gate, 1.0f, n);
    fetch(p, A.gamma0, 1.0f, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = g.get(e) * p.get(e);
  };
  if constexpr (kHeld) {
    fetch(gamma_held, A.gamma, 1.0f, 0);
    if constexpr (WIDE) {
      fetch(gamma0_held, A.gamma0, 1.0f, 0);
      fetch(beta0_held, A.beta0, 0.0f, 0);
    } else {
      fetch_gain(gain_held, 0);
    }
  }
  const float inv = 1.0f / float(A.cols);
  float acc[N == 2 ? 2 : 1][N][8] = {};  // what is not in LDS
  // fours of a thread's sums, side by side over the threads
  const auto place = [&](int which, int n, int half) {
    return store + ((which * N + n) * 2 + half) * kMost + threadIdx.x;
  };
  // sum `which` += that
  const auto add = [&](int which, int n, const float (&that)[8]) {
    if (which < kInLds) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 *p = place(which, n, half);
        f32x4 v = *p;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += that[half * 4 + e];
        *p = v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[which - kInLds][n][e] += that[e];
    }
  };
#pragma unroll
  for (int which = 0; which < kInLds; ++which)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      *place(which, n, 0) = f32x4{};
      *place(which, n, 1) = f32x4{};
    }
  constexpr bool kOnce = N == 1 && !TAIL && sizeof(typename TX::raw) == 2;
  const int64_t step = int64_t(gridDim.x) * subs * R;
  struct Rows {
    Eight<TX> dy[R][N], ds[R][N], s[R][N], b[R][N], z[WIDE ? R : 1][WIDE ? N : 1];
    float r0[R], r1[R], m0[R], m1[R];
  };
  const auto is = [&](int64_t first, int k) { return first + k < A.rows; };
  const auto load = [&](Rows &v, int64_t first) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool in = is(first, k);
      const int64_t r = first + k;
      // a block that is not normalised is its own h0
      v.r0[k] = !in ? 0.0f : A.post ? A.stats[r] : 1.0f;
      v.r1[k] = in ? A.stats[A.rows + r] : 0.0f;
      v.m0[k] = in && A.post && A.center ? A.stats[2 * A.rows + r] : 0.0f;
      v.m1[k] = in && A.center ? A.stats[3 * A.rows + r] : 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        c.template get<kOnce>(v.dy[k][n], row_of<TX>(A.dy, r, A.ld_dy), n, in);
        c.template get<kOnce>(v.s[k][n], row_of<TX>(A.sum, r, A.ld_s), n, in);
        c.template get<kOnce>(v.ds[k][n], row_of<TX>(A.dsum, r, A.ld_ds), n, in && A.dsum);
        c.template get<kOnce>(v.b[k][n], row_of<TX>(A.block, r, A.ld_b), n, in && A.block);
        if constexpr (WIDE) c.template get<kOnce>(v.z[k][n], row_of<TX>(A.z, r, A.ld_z), n, in);
      }
    }
  };
  constexpr bool kAhead = N == 1 && sizeof(typename TX::raw) == 2;  // registers hold both
  Rows ahead;
  if constexpr (kAhead) load(ahead, (int64_t(blockIdx.x) * subs + sub) * R);
  for (int64_t at = int64_t(blockIdx.x) * subs * R; at < A.rows; at += step) {
    const int64_t first = at + sub * R;
    Rows now;
    if constexpr (kAhead) {
      now = ahead;
      if (at + step < A.rows) load(ahead, first + step);
    } else {
      load(now, first);
    }
    // Past a row's end the gradients are 0 and so are the factors they meet: rstd is
    // taken as 0 there, since mean rstd may be beyond binary32.  Elements that are
    // another thread's may already be that thread's results where buffers are used in
    // place, whatever these are.
    const auto own = [&](int n, float v) { return c.left[n] > 0 ? v : 0.0f; };
    const auto h1 = [&](int k, int n, int e) {
      const float h = (now.s[k][n].get(e) - now.m1[k]) * own(n, now.r1[k]);
      return live(n, e) ? h : 0.0f;
    };
    const auto h0 = [&](int k, int n, int e) {
      const float h = (now.b[k][n].get(e) - now.m0[k]) * own(n, now.r0[k]);
      return live(n, e) ? h : 0.0f;
    };
    float both[2 * R] = {};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float dh[8] = {}, dd[8] = {};
      if constexpr (!kHeld) fetch(gamma_held, A.gamma, 1.0f, n);
#pragma unroll
      for (int k = 0; k < R; ++k) c.keep(now.dy[k][n], n);
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float h = h1(k, n, e), d = now.dy[k][n].get(e), g = d * gamma_held.get(e);
          both[2 * k] += g;
          both[2 * k + 1] = __builtin_fmaf(g, h, both[2 * k + 1]);
          dh[e] = __builtin_fmaf(d, h, dh[e]);
          dd[e] += d;
        }
      add(0, n, dh);
      add(1, n, dd);
    }
    float total = waves.sums(both) * inv;
    // rstd (g - c1 - h1 c2) = rstd g - rstd c1 - (s - mean) rstd^2 c2
    float c1[R], c2[R], D[R][N][8];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      c1[k] = A.center ? now.r1[k] * lane_value(total, 64 / R * k) : 0.0f;
      c2[k] = now.r1[k] * (now.r1[k] * lane_value(total, 64 / R * k + 32 / R));
      both[2 * k] = both[2 * k + 1] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float dh[8] = {}, dd[8] = {};
      if constexpr (!kHeld) {
        fetch(gamma_held, A.gamma, 1.0f, n);
        if constexpr (WIDE) {
          fetch(gamma0_held, A.gamma0, 1.0f, n);
          fetch(beta0_held, A.beta0, 0.0f, n);
        } else {
          fetch_gain(gain_held, n);
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        now.dy[k][n].forget();
        now.s[k][n].forget();
        float out[8], h[8];
        const float o1 = own(n, c1[k]), o2 = own(n, c2[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float g = now.dy[k][n].get(e) * gamma_held.get(e);
          float d = __builtin_fmaf(-(now.s[k][n].get(e) - now.m1[k]), o2,
                                   now.ds[k][n].get(e) - o1);
          d = __builtin_fmaf(g, now.r1[k], d);
          D[k][n][e] = live(n, e) ? d : 0.0f;
          out[e] = A.scale * d;
          h[e] = h0(k, n, e);
        }
        now.dy[k][n].set(out);
        if (is(first, k))
          c.put(now.dy[k][n], row_of<TX>(A.dx, first + k, A.ld_dx), n);
        if constexpr (WIDE) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float slope;
            const float open = sigmoid(now.z[k][n].get(e), slope);
            float v = h[e];
            if (A.post) v = __builtin_fmaf(v, gamma0_held.get(e), beta0_held.get(e));
            out[e] = D[k][n][e] * v * slope;
            D[k][n][e] *= open;
          }
          now.z[k][n].set(out);
          if (is(first, k) && A.dz)
            c.put(now.z[k][n], row_of<TX>(A.dz, first + k, A.ld_dz), n);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dh[e] = __builtin_fmaf(D[k][n][e], h[e], dh[e]);
          dd[e] += D[k][n][e];
          if constexpr (WIDE) D[k][n][e] *= gamma0_held.get(e);
          else D[k][n][e] *= gain_held[e];
          both[2 * k] += D[k][n][e];
          both[2 * k + 1] = __builtin_fmaf(D[k][n][e], h[e], both[2 * k + 1]);
        }
      }
      add(2, n, dh);
      add(3, n, dd);
    }
    if (!A.block) continue;
#pragma unroll
    for (int k = 0; k < R; ++k) c1[k] = c2[k] = 0.0f;
    if (A.post) {
      total = waves.sums(both) * inv;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        c1[k] = A.center ? now.r0[k] * lane_value(total, 64 / R * k) : 0.0f;
        c2[k] = now.r0[k] * (now.r0[k] * lane_value(total, 64 / R * k + 32 / R));
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (!is(first, k)) break;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        now.b[k][n].forget();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = __builtin_fmaf(-(now.b[k][n].get(e) - now.m0[k]), c2[k], -c1[k]);
          D[k][n][e] = __builtin_fmaf(D[k][n][e], now.r0[k], d);
        }
        now.b[k][n].set(D[k][n]);
        c.put(now.b[k][n], row_of<TX>(A.dblock, first + k, A.ld_db), n);
      }
    }
  }
  if (!A.part) return;
  // the row groups' sums (with sixteen columns a thread there is one), then the
  // workgroup's partial rows
  if (subs > 1) __syncthreads();
  if (sub > 0) return;
#pragma unroll
  for (int which = 0; which < 4; ++which) {
    if (!(A.want & (which < 2 ? 1 : 2))) continue;
    float *out = A.part + (int64_t(which) * A.parts + blockIdx.x) * A.cols;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float sum[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        sum[e] = which < kInLds ? (*place(which, n, e / 4))[e % 4]
                                : acc[N == 2 && which >= 2 ? which - 2 : 0][n][e];
      for (int w = 1; w < subs; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += (*(place(which, n, e / 4) + w * per))[e % 4];
      Eight<F32> v;
      v.set(sum);
      c.put(v, out, n);
    }
  }
}

// The columns' gradients from the sums of the partial rows, which are added in
// the partials' order within each of kSplit interleaved groups, the groups then in
// order.  Four columns a thread; blockIdx.y 0: the second norm's, 1: the
// first's and the gate's:
//   dgamma0 = gate sum(E h0);  dbeta0 = gate sum(E);
//   dgate = sum(D n) = gamma0 sum(E h0) + beta0 sum(E)   (one gate a column)
constexpr int kSplit = 64;
template <class TP>
__global__ void __launch_bounds__(16 * kSplit) seam_join_kernel(const BwdArgs A) {
  __shared__ float lds[2][kSplit][68];
  struct __attribute__((packed, aligned(4))) Four {
    float e[4];
  };
  const int first = blockIdx.y * 2;
  if (!(A.want & (first ? 2 : 1))) return;
  const int64_t c = int64_t(blockIdx.x) * 64 + threadIdx.x * 4;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float *p = A.part + int64_t(first + j) * A.parts * A.cols + c;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= A.cols) {
#pragma unroll 8
      for (int k = threadIdx.y; k < A.parts; k += kSplit) {
        const Four v = *reinterpret_cast<const Four *>(p + k * A.cols);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v.e[e];
      }
    } else {
      for (int k = threadIdx.y; k < A.parts; k += kSplit)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < A.cols) s[e] += p[k * A.cols + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) lds[j][threadIdx.y][threadIdx.x * 4 + e] = s[e];
  }
  __syncthreads();
  const int t = threadIdx.y * 16 + threadIdx.x;
  const int64_t col = int64_t(blockIdx.x) * 64 + t;
  if (t >= 64 || col >= A.cols) return;
  float sh = 0.0f, s1 = 0.0f;
#pragma unroll
  for (int k = 0; k < kSplit; ++k) {
    sh += lds[0][k][t];
    s1 += lds[1][k][t];
  }
  const auto param = [&](const void *p, float none) {
    return p ? TP::load(static_cast<const typename TP::raw *>(p)[col]) : none;
  };
  const auto put = [&](void *p, float v) {
    if (p) static_cast<typename TP::raw *>(p)[col] = TP::store(v);
  };
  if (first == 0) {
    put(A.dgamma, sh);
    put(A.dbeta, s1);
  } else {
    const float gate = param(A.gate, 1.0f);
    put(A.dgamma0, gate * sh);
    put(A.dbeta0, gate * s1);
    put(A.dgate, __builtin_fmaf(param(A.gamma0, 1.0f), sh, param(A.beta0, 0.0f) * s1));
  }
}

// ------------------------------------------------------------------- host

bool desc_ok(const zs_blocknorm_desc *d) {
  if (!d || d->rows < 0 || d->cols < 1 || d->cols > kMaxCols) return false;
  if (d->rows > (INT64_C(1) << 40)) return false;
  if (!dtype_size(d->dtype)) return false;
  if (d->param_dtype != ZS_F32 && d->param_dtype != d->dtype) return false;
  if (d->kind != ZS_NORM_LAYER && d->kind != ZS_NORM_RMS) return false;
  if (d->gate < ZS_GATE_NONE || d->gate > ZS_GATE_SIGMOID || d->post < 0 || d->post > 1)
    return false;
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps) || !std::isfinite(d->residual_scale))
    return false;
  const int64_t lds[] = {d->ld_x, d->ld_block, d->ld_gate, d->ld_sum, d->ld_y, d->ld_dy,
                         d->ld_dsum, d->ld_dx, d->ld_dblock, d->ld_dgate};
  for (int64_t ld : lds)
    if (ld != 0 && (ld < d->cols || ld > (INT64_C(1) << 40))) return false;
  return true;
}

// A row's threads, and the row groups of a workgroup; a workgroup for each row
// where there are few.
struct Way {
  int n, per, subs;
};
Way way_of(const zs_blocknorm_desc &d, int threads) {
  Way w;
  w.n = d.cols <= kMaxCols / 2 ? 1 : 2;
  w.per = int(up(up(d.cols, 8 * w.n) / (8 * w.n), 64));
  w.subs = w.per < threads ? threads / w.per : 1;
  if (d.rows < int64_t(kCus) * w.subs) w.subs = int((d.rows + kCus - 1) / kCus);
  if (w.subs < 1) w.subs = 1;
  return w;
}

// The backward pass takes two rows at a time from 1024 rows on, where the registers hold
// them.  Row groups are counted for one row each, so that of narrow rows some CUs then
// have none (1024 x 512: 128 workgroups of 8 rows), which costs nothing there: the row
// groups' latencies are what takes time (1023 x 512 bf16 13.5 us, 1024 x 512 13.0; x 1024
// 15.3 and 14.9).  Of rows that end inside a thread's eight columns only long ones (8192
// rows, bf16, layer, with two and with one: 2049 columns 71 and 63 us, 3585 107 and 90, 4097
// 123 and 130, 5121 136 and 150, 6143 153 and 165).
bool pairs(const zs_blocknorm_desc &d) {
  return d.rows >= 4 * kCus && d.cols <= 8 * kPairThreads && d.dtype != ZS_F32 &&
         d.gate != ZS_GATE_SIGMOID && (d.cols % 8 == 0 || d.cols > 4096);
}
Way bwd_way_of(const zs_blocknorm_desc &d) { return way_of(d, pairs(d) ? kPairThreads : 1024); }

int64_t parts_of(const zs_blocknorm_desc &d) {
  const int rows = bwd_way_of(d).subs * (pairs(d) ? 2 : 1);
  const int64_t b = (d.rows + rows - 1) / rows;
  return b < kMaxParts ? b : kMaxParts;
}

template <class F>
int by_type(const zs_blocknorm_desc &d, F f) {
  if (d.dtype == ZS_F32) return f(F32{}, F32{});
  if (d.dtype == ZS_BF16)
    return d.param_dtype == ZS_F32 ? f(Bf16{}, F32{}) : f(Bf16{}, Bf16{});
  return d.param_dtype == ZS_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
}

template <class F>
int by_way(int n, bool tail, bool wide, F f) {
  using std::integral_constant;
  const auto gates = [&](auto nn, auto tt) {
    return wide ? f(nn, tt, std::true_type{}) : f(nn, tt, std::false_type{});
  };
  const auto tails = [&](auto nn) {
    return tail ? gates(nn, std::true_type{}) : gates(nn, std::false_type{});
  };
  return n == 1 ? tails(integral_constant<int, 1>{}) : tails(integral_constant<int, 2>{});
}

// Without a block the seam is the second norm of x alone.
bool no_block_ok(const zs_blocknorm_desc &d) {
  return !d.post && d.gate == ZS_GATE_NONE && d.residual_scale == 1.0f;
}

}  // namespace

extern "C" {

int zero_shard_blocknorm(const zs_blocknorm_desc *d, const void *x, const void *block,
                         const void *gate, const void *gamma_post, const void *beta_post,
                         const void *gamma, const void *beta, void *sum, void *y, float *stats) {
  if (!desc_ok(d)) return ZS_EINVAL;
  if (d->rows == 0) return ZS_OK;
  if (!x || !y || !block != !sum || y == sum || !gate != (d->gate == ZS_GATE_NONE))
    return ZS_EINVAL;
  if (!block && !no_block_ok(*d)) return ZS_EINVAL;
  if (!d->post && (gamma_post || beta_post)) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), psize = dtype_size(d->param_dtype);
  const bool wide = d->gate == ZS_GATE_SIGMOID;
  if (!aligned(x, size) || !aligned(block, size) || !aligned(gate, wide ? size : psize) ||
      !aligned(gamma_post, psize) || !aligned(beta_post, psize) || !aligned(gamma, psize) ||
      !aligned(beta, psize) || !aligned(sum, size) || !aligned(y, size) || !aligned(stats, 4))
    return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  const Way w = way_of(*d, kThreads);
  const FwdArgs A{d->rows, d->cols, ld(d->ld_x), ld(d->ld_block), ld(d->ld_gate), ld(d->ld_sum),
                  ld(d->ld_y), x, block, wide ? gate : nullptr, wide ? nullptr : gate, gamma_post,
                  beta_post, gamma, beta, sum, y, stats, d->eps, d->residual_scale,
                  d->kind == ZS_NORM_LAYER, d->post, w.per};
  const int threads = w.per * w.subs;
  return by_type(*d, [&](auto tx, auto tp) {
    using TX = decltype(tx);
    using TP = decltype(tp);
    return by_way(w.n, d->cols % 8 != 0, wide, [&](auto n, auto tail, auto wd) {
      const auto launch = [&](auto r) {
        const int64_t groups = (A.rows + w.subs * r.value - 1) / (w.subs * r.value);
        // about as many as there is room for at once: later ones would run alone
        const int64_t most = int64_t(kCus) * (kResident > threads ? kResident / threads : 1);
        hipLaunchKernelGGL((seam_fwd_kernel<TX, TP, n.value, r.value, tail.value, wd.value>),
                           dim3(unsigned(groups < most ? groups : most)), dim3(threads), 0,
                           static_cast<hipStream_t>(d->stream), A);
        return launched();
      };
      // two rows at a time from 1024 rows on, where the registers hold them and the work
      // on their ends (32768 x 511 bf16: 37 us with two, 33 with one)
      if constexpr (n.value == 1 && sizeof(typename TX::raw) == 2 && !wd.value && !tail.value)
        if (A.rows >= 4 * kCus) return launch(std::integral_constant<int, 2>{});
      return launch(std::integral_constant<int, 1>{});
    });
  });
}

int64_t zero_shard_blocknorm_workspace(const zs_blocknorm_desc *d) {
  if (!desc_ok(d)) return -1;
  return 4 * parts_of(*d) * d->cols * int64_t(sizeof(float));
}

int zero_shard_blocknorm_bwd(const zs_blocknorm_desc *d, const void *dy, const void *dsum,
                             const void *sum, const void *block, const void *gate,
                             const void *gamma_post, const void *beta_post, const void *gamma,
                             const float *stats, void *dx, void *dblock, void *dgate,
                             void *dgamma_post, void *dbeta_post, void *dgamma, void *dbeta,
                             void *workspace, int64_t workspace_bytes) {
  if (!desc_ok(d)) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), psize = dtype_size(d->param_dtype);
  const bool wide = d->gate == ZS_GATE_SIGMOID, column = d->gate == ZS_GATE_COLUMN;
  const int want = (dgamma || dbeta ? 1 : 0) |
                   (dgamma_post || dbeta_post || (column && dgate) ? 2 : 0);
  if (!d->post && (gamma_post || beta_post || dgamma_post || dbeta_post)) return ZS_EINVAL;
  if (d->gate == ZS_GATE_NONE && dgate) return ZS_EINVAL;
  if (d->rows > 0) {
    if (!dy || !sum || !stats || !dx || !block != !dblock || dx == dblock) return ZS_EINVAL;
    if (!gate != (d->gate == ZS_GATE_NONE) || (!block && !no_block_ok(*d))) return ZS_EINVAL;
    if (want && (!workspace || workspace_bytes < zero_shard_blocknorm_workspace(d)))
      return ZS_EINVAL;
  }
  const int gsize = wide ? size : psize;
  if (!aligned(dy, size) || !aligned(dsum, size) || !aligned(sum, size) || !aligned(block, size) ||
      !aligned(gate, gsize) || !aligned(gamma_post, psize) || !aligned(beta_post, psize) ||
      !aligned(gamma, psize) || !aligned(stats, 4) || !aligned(dx, size) ||
      !aligned(dblock, size) || !aligned(dgate, gsize) || !aligned(dgamma_post, psize) ||
      !aligned(dbeta_post, psize) || !aligned(dgamma, psize) || !aligned(dbeta, psize) ||
      !aligned(workspace, 16))
    return ZS_EALIGN;
  if (d->rows == 0 && !want) return ZS_OK;
  if (const int rc = device_is_gfx950()) return rc;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  const Way w = bwd_way_of(*d);
  const BwdArgs A{d->rows, d->cols, ld(d->ld_dy), ld(d->ld_dsum), ld(d->ld_sum), ld(d->ld_block),
                  ld(d->ld_gate), ld(d->ld_dx), ld(d->ld_dblock), ld(d->ld_dgate),
                  dy, dsum, sum, block, wide ? gate : nullptr,
                  wide ? nullptr : gate, gamma_post, beta_post, gamma, stats,
                  dx, dblock, wide ? dgate : nullptr, column ? dgate : nullptr, dgamma_post,
                  dbeta_post, dgamma, dbeta, want ? static_cast<float *>(workspace) : nullptr,
                  d->residual_scale, d->kind == ZS_NORM_LAYER, d->post, want,
                  int32_t(parts_of(*d)), w.per};
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  return by_type(*d, [&](auto tx, auto tp) {
    using TX = decltype(tx);
    using TP = decltype(tp);
    int rc = ZS_OK;
    if (A.rows > 0)
      rc = by_way(w.n, d->cols % 8 != 0, wide, [&](auto n, auto tail, auto wd) {
        using std::integral_constant;
        const auto launch = [&](auto r, auto most) {
          hipLaunchKernelGGL(
              (seam_bwd_kernel<TX, TP, n.value, r.value, tail.value, wd.value, most.value>),
              dim3(unsigned(A.parts)), dim3(w.per * w.subs), 0, st, A);
          return launched();
        };
        if constexpr (n.value == 2) {
          if (w.per <= kPairThreads)  // a third more registers for 12288 columns and fewer
            return launch(integral_constant<int, 1>{}, integral_constant<int, kPairThreads>{});
        } else if constexpr (sizeof(typename TX::raw) == 2 && !wd.value) {
          if (pairs(*d))
            return launch(integral_constant<int, 2>{}, integral_constant<int, kPairThreads>{});
        }
        return launch(integral_constant<int, 1>{}, integral_constant<int, 1024>{});
      });
    if (rc || !want) return rc;
    hipLaunchKernelGGL((seam_join_kernel<TP>), dim3(unsigned((A.cols + 63) / 64), 2),
                       dim3(16, kSplit), 0, st, A);
    return launched();
  });
}

}  // extern "C"
