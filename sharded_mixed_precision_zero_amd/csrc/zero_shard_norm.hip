// zero_shard_norm.hip -- layer norm, forward and backward, on MI355X (gfx950)
// (declarations and the contract: include/zero_shard.h).
//
//   forward   s = round(x + residual) (or x);  mean = sum(s)/D;
//             rstd = 1/sqrt(sum((s - mean)^2)/D + eps);
//             y = (s - mean) rstd gamma + beta
//   backward  h = (x - mean) rstd;  g = dy gamma;
//             dx = rstd (g - sum(g)/D - h sum(g h)/D) + dsum;
//             dgamma = sum_rows dy h;  dbeta = sum_rows dy
//
// Everything is binary32 inside, each output rounded once.  Both directions
// are HBM-bound, so a row is read once and stays in registers as it lay in
// memory, eight elements a thread (sixteen above 8192 columns), and the
// variance is the centred sum of squares over them.  A workgroup takes several
// rows at a time: their loads are in flight together and their sums cross the
// waves together, and it goes on to further rows with gamma and beta (and the
// gradients' sums) in its registers.  The backward pass leaves one partial row
// of dgamma and dbeta per workgroup, and a second launch adds the partials in a
// fixed order: no atomics, so the same inputs give the same bits.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "zero_shard.h"
#include "zs_device.h"

namespace {

using namespace zs_dev;

constexpr int kThreads = 256;
constexpr int kLongThreads = 1024;
constexpr int kMaxRegCols = 16384;  // rows up to here stay in registers
constexpr int kCus = 256;
constexpr int64_t kMaxGrid = 0xffffffff / kLongThreads;  // a launch takes below 2^32 threads
constexpr int kMaxParts = 256;      // partial rows of dgamma / dbeta

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, ROWS, 0xf, false));
}

// Sum over each 16 lanes, in all of them.
__device__ __forceinline__ float sum16(float v) {
  v += dpp<0xb1>(v);   // lanes 1 apart
  v += dpp<0x4e>(v);   // 2 apart
  v += dpp<0x141>(v);  // half row mirrored
  return v + dpp<0x140>(v);  // row mirrored
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Sum over the wave, uniform.
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  v += dpp<0x142, 0xa>(v);  // rows 1 and 3: with the row before
  v += dpp<0x143, 0xc>(v);  // rows 2 and 3: with the first half
  return lane_value(v, 63);
}

// Sums over the waves of a row group, M of them at once, uniform.  One barrier
// each: two buffers take turns, so a buffer is written again only after all
// have passed the next sum's barrier.
struct Sums {
  float (*lds)[16][8];  // [2][wave of the workgroup][sum]
  int first, waves;     // of this row group
  int turn = 0;
  template <int M>
  __device__ __forceinline__ void add(float (&v)[M]) {
    static_assert(M <= 8, "a buffer's row");
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = wave_sum(v[m]);
    if (waves == 1) return;
    const int lane = threadIdx.x & 63;
    float (*buf)[8] = lds[turn];
    turn ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) buf[threadIdx.x >> 6][m] = v[m];
    }
    // all of LDS is there; loads from memory stay in flight
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int m = 0; m < M; m += 4) {
      const int at = m + (lane >> 4), w = lane & 15;
      float s = w < waves && at < M ? buf[first + w][at] : 0.0f;
      s = sum16(s);
#pragma unroll
      for (int k = m; k < m + 4 && k < M; ++k) v[k] = lane_value(s, (k - m) * 16);
    }
  }
};

// The statistics after the centred sweep: off = the sum of (s - mean), zero
// but for the rounding of the mean, becomes what the mean is off by (a row
// far from zero would show it in y); returns rstd.  An infinite row keeps
// its mean.  Of a constant row the variance is a difference of two equal values
// up to rounding, which may fall below 0 by more than eps; a NaN stays one.
__device__ __forceinline__ float finish(float sq, float &off, float inv, float eps, float &mean) {
  off *= inv;
  if (!(fabsf(off) < INFINITY)) off = 0.0f;
  mean += off;
  const float var = sq * inv - off * off;
  return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);
}

struct FwdArgs {
  int64_t rows, cols;
  int64_t ld_x, ld_r, ld_s, ld_y;  // elements
  const void *x, *residual, *gamma, *beta;
  void *sum, *y;
  float *mean, *rstd;
  float eps;
  int32_t per;  // threads of a row
};

template <class T>
__device__ __forceinline__ const void *row_of(const void *p, int64_t r, int64_t ld) {
  return static_cast<const typename T::raw *>(p) + r * ld;
}
template <class T>
__device__ __forceinline__ void *row_of(void *p, int64_t r, int64_t ld) {
  return static_cast<typename T::raw *>(p) + r * ld;
}

// A thread's columns: N times eight, `per` threads apart.
template <int N>
struct Columns {
  unsigned i[N];
  int left[N];
  __device__ __forceinline__ Columns(int t, int per, int cols) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      i[n] = (n * per + t) * 8;
      left[n] = cols - int(i[n]);
    }
  }
};

// gamma or beta at these columns (`none` where the caller gave none)
template <bool TAIL, class TP, int N>
__device__ __forceinline__ void load_params(Eight<TP> (&v)[N], const void *p, float none,
                                            const Columns<N> &c) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (p) {
      v[n].template load<TAIL>(p, c.i[n], c.left[n]);
    } else {
      const float all[8] = {none, none, none, none, none, none, none, none};
      v[n].set(all);
    }
  }
}

// R rows at a time, each over `per` threads (a multiple of 64) of the
// workgroup's blockDim.x / per row groups.  TAIL: the columns are no multiple of 8.
template <class TX, class TP, int N, int R, bool TAIL>
__global__ void __launch_bounds__(1024) ln_fwd_kernel(const FwdArgs A) {
  __shared__ float lds[2][16][8];
  const int per = A.per, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / per);
  const int t = threadIdx.x - sub * per, subs = blockDim.x / per;
  Sums sums{lds, sub * per / 64, per / 64};
  const Columns<N> c(t, per, int(A.cols));
  Eight<TP> gamma[N], beta[N];
  load_params<TAIL>(gamma, A.gamma, 1.0f, c);
  load_params<TAIL>(beta, A.beta, 0.0f, c);
  const float inv = 1.0f / float(A.cols);
  // Past the caches where a lane's accesses are 16 bytes side by side (8192 x 5120
  // bf16 with a residual: 58 us for 67 through them); others leave parts of lines,
  // which should stay (16384 x 511 bf16: 15.4 us for 18.1 past them, 2048 x 1601
  // fp32 11.1 for 14.5; only even rows of fp32 lose by it, 8192 x 4096 102 for 98).
  constexpr bool kOnce = N == 1 && !TAIL && sizeof(typename TX::raw) == 2;
  const int64_t step = int64_t(gridDim.x) * subs * R;
  struct Rows {
    Eight<TX> x[R][N], q[R][N];
  };
  const auto load = [&](Rows &v, int64_t r0) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int left = r0 + k < A.rows ? c.left[n] : 0;
        v.x[k][n].template load<TAIL, kOnce>(row_of<TX>(A.x, r0 + k, A.ld_x), c.i[n], left);
        if (A.residual)
          v.q[k][n].template load<TAIL, kOnce>(row_of<TX>(A.residual, r0 + k, A.ld_r), c.i[n], left);
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
    auto &x = now.x;
    if (A.residual) {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          float s[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = x[k][n].get(e) + now.q[k][n].get(e);
          x[k][n].set(s);
          if (r0 + k < A.rows)
            x[k][n].template store<TAIL>(row_of<TX>(A.sum, r0 + k, A.ld_s), c.i[n], c.left[n]);
        }
    }
    float mean[R], both[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mean[k] = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) mean[k] += x[k][n].get(e);
    }
    sums.add(mean);
    // the deviations; where registers are short, anew from x each time
    constexpr bool kKeep = N == 1;
    float dev[kKeep ? R : 1][kKeep ? N : 1][8];
#pragma unroll
    for (int k = 0; k < R; ++k) {
#pragma unroll
      for (int n = 0; n < N; ++n) x[k][n].forget();
      mean[k] *= inv;
      float sq = 0.0f, off = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = (TAIL ? e : 0) < c.left[n] ? x[k][n].get(e) - mean[k] : 0.0f;
          sq = __builtin_fmaf(d, d, sq);
          off += d;
          if constexpr (kKeep) dev[k][n][e] = d;
        }
      both[2 * k] = sq;
      both[2 * k + 1] = off;
    }
    sums.add(both);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float rough = mean[k];
      float off = both[2 * k + 1];
      const float rstd = finish(both[2 * k], off, inv, A.eps, mean[k]);
      if (r0 + k >= A.rows) break;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float y[8];
        if constexpr (!kKeep) x[k][n].forget();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float d;
          if constexpr (kKeep) d = dev[k][n][e];
          else d = x[k][n].get(e) - rough;
          y[e] = __builtin_fmaf((d - off) * rstd, gamma[n].get(e), beta[n].get(e));
        }
        x[k][n].set(y);
        x[k][n].template store<TAIL>(row_of<TX>(A.y, r0 + k, A.ld_y), c.i[n], c.left[n]);
      }
      if (t == 0) {
        if (A.mean) A.mean[r0 + k] = mean[k];
        if (A.rstd) A.rstd[r0 + k] = rstd;
      }
    }
  }
}

// Rows too long for registers: three sweeps, each thread over its own
// elements (which also makes the sum it wrote the sum it reads back).
template <class TX, class TP>
__global__ void __launch_bounds__(kLongThreads) ln_fwd_long_kernel(const FwdArgs A) {
  __shared__ float lds[2][16][8];
  Sums sums{lds, 0, kLongThreads / 64};
  const float inv = 1.0f / float(A.cols);
  const int64_t i0 = int64_t(threadIdx.x) * 8, step = int64_t(kLongThreads) * 8;
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const void *src = row_of<TX>(A.x, r, A.ld_x);
    float total[1] = {0.0f}, both[2] = {0.0f, 0.0f};
    Eight<TX> x, q;
    if (A.residual) {
      const void *rr = row_of<TX>(A.residual, r, A.ld_r);
      void *sr = row_of<TX>(A.sum, r, A.ld_s);
      for (int64_t i = i0; i < A.cols; i += step) {
        float s[8];
        x.load(src, i, A.cols - i);
        q.load(rr, i, A.cols - i);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = x.get(e) + q.get(e);
        x.set(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) total[0] += x.get(e);
        x.store(sr, i, A.cols - i);
      }
      src = sr;
    } else {
      for (int64_t i = i0; i < A.cols; i += step) {
        x.load(src, i, A.cols - i);
#pragma unroll
        for (int e = 0; e < 8; ++e) total[0] += x.get(e);
      }
    }
    sums.add(total);
    float mean = total[0] * inv;
    const float first = mean;
    for (int64_t i = i0; i < A.cols; i += step) {
      x.load(src, i, A.cols - i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < A.cols - i ? x.get(e) - first : 0.0f;
        both[0] = __builtin_fmaf(d, d, both[0]);
        both[1] += d;
      }
    }
    sums.add(both);
    float off = both[1];
    const float rstd = finish(both[0], off, inv, A.eps, mean);
    void *yr = row_of<TX>(A.y, r, A.ld_y);
    for (int64_t i = i0; i < A.cols; i += step) {
      float y[8];
      Eight<TP> g, b;
      x.load(src, i, A.cols - i);
      if (A.gamma) g.load(A.gamma, i, A.cols - i);
      if (A.beta) b.load(A.beta, i, A.cols - i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = (x.get(e) - first - off) * rstd;
        if (A.gamma) y[e] *= g.get(e);
        if (A.beta) y[e] += b.get(e);
      }
      x.set(y);
      x.store(yr, i, A.cols - i);
    }
    if (threadIdx.x == 0) {
      if (A.mean) A.mean[r] = mean;
      if (A.rstd) A.rstd[r] = rstd;
    }
  }
}

struct BwdArgs {
  int64_t rows, cols;
  int64_t ld_dy, ld_x, ld_ds, ld_dx;  // elements
  const void *dy, *x, *gamma, *dsum;
  const float *mean, *rstd;
  void *dx, *dgamma, *dbeta;
  float *part;    // [parts][cols] of dgamma, then of dbeta
  int32_t parts;  // 0: no rows (the gradients are zero)
  int32_t per;    // threads of a row
};

template <class TX, class TP, int N, int R, bool TAIL>
__global__ void __launch_bounds__(1024) ln_bwd_kernel(const BwdArgs A) {
  __shared__ float lds[2][16][8];
  __shared__ float join[1024 * 8];
  const int per = A.per, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / per);
  const int t = threadIdx.x - sub * per, subs = blockDim.x / per;
  Sums sums{lds, sub * per / 64, per / 64};
  const Columns<N> c(t, per, int(A.cols));
  Eight<TP> gamma[N];
  load_params<TAIL>(gamma, A.gamma, 1.0f, c);
  const float inv = 1.0f / float(A.cols);
  float dg[N][8] = {}, db[N][8] = {};
  // Past the caches as in the forward pass (8192 x 5120 bf16 with a residual: 66 us
  // for 72 through them; 16384 x 511 bf16 through them 29 for 34, 2048 x 1601 fp32
  // 17.7 for 19.7, and 8192 x 4096 fp32 105 for 98).
  constexpr bool kOnce = N == 1 && !TAIL && sizeof(typename TX::raw) == 2;
  const int64_t step = int64_t(gridDim.x) * subs * R;
  struct Rows {
    Eight<TX> x[R][N], dy[R][N], ds[R][N];
    float mean[R], rstd[R];
  };
  const auto load = [&](Rows &v, int64_t r0) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool in = r0 + k < A.rows;
      v.mean[k] = in ? A.mean[r0 + k] : 0.0f;
      v.rstd[k] = in ? A.rstd[r0 + k] : 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int left = in ? c.left[n] : 0;
        v.x[k][n].template load<TAIL, kOnce>(row_of<TX>(A.x, r0 + k, A.ld_x), c.i[n], left);
        v.dy[k][n].template load<TAIL, kOnce>(row_of<TX>(A.dy, r0 + k, A.ld_dy), c.i[n], left);
        if (A.dsum)
          v.ds[k][n].template load<TAIL, kOnce>(row_of<TX>(A.dsum, r0 + k, A.ld_ds), c.i[n], left);
      }
    }
  };
  constexpr bool kAhead = N == 1;  // as in the forward pass
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
    auto &x = now.x, &dy = now.dy, &ds = now.ds;
    auto &mean = now.mean, &rstd = now.rstd;
    float both[2 * R];
    // Past a row's end dy is 0, and so is all that it is a factor of: rstd is taken
    // as 0 there, since -mean rstd may be beyond binary32.
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float scale = (TAIL ? e : 0) < c.left[n] ? rstd[k] : 0.0f;
          const float h = (x[k][n].get(e) - mean[k]) * scale, d = dy[k][n].get(e);
          dg[n][e] = __builtin_fmaf(d, h, dg[n][e]);
          db[n][e] += d;
          const float g = d * gamma[n].get(e);
          c1 += g;
          c2 = __builtin_fmaf(g, h, c2);
        }
      both[2 * k] = c1;
      both[2 * k + 1] = c2;
      __builtin_amdgcn_sched_barrier(0);  // one row's values at a time
    }
    sums.add(both);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (r0 + k >= A.rows) break;
      const float c1 = both[2 * k] * inv, c2 = both[2 * k + 1] * inv;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float v[8];
        x[k][n].forget();
        dy[k][n].forget();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float h = (x[k][n].get(e) - mean[k]) * rstd[k];
          const float g = dy[k][n].get(e) * gamma[n].get(e) - c1;
          v[e] = rstd[k] * __builtin_fmaf(-h, c2, g);
          if (A.dsum) v[e] += ds[k][n].get(e);
        }
        x[k][n].set(v);
        x[k][n].template store<TAIL>(row_of<TX>(A.dx, r0 + k, A.ld_dx), c.i[n], c.left[n]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (!A.part) return;
  // the row groups' sums, then the workgroup's partial row
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float (&acc)[N][8] = which ? db : dg;
    if (which ? !A.dbeta : !A.dgamma) continue;
    float *out = A.part + (int64_t(which) * A.parts + blockIdx.x) * A.cols;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (subs > 1) {
        __syncthreads();
        if (sub > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) join[((sub - 1) * 8 + e) * per + t] = acc[n][e];
        }
        __syncthreads();
        if (sub > 0) continue;
        for (int w = 0; w < subs - 1; ++w)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[n][e] += join[(w * 8 + e) * per + t];
      }
      Eight<F32> v;
      v.set(acc[n]);
      v.template store<TAIL>(out, c.i[n], c.left[n]);
    }
  }
}

// Long rows: column partials over the rows of one slice, then dx by two
// sweeps (in this order: dx may be dy's own buffer).
template <class TX>
__global__ void __launch_bounds__(kThreads) ln_bwd_long_cols_kernel(const BwdArgs A) {
  const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= A.cols) return;
  float dg = 0.0f, db = 0.0f;
  for (int64_t r = blockIdx.y; r < A.rows; r += gridDim.y) {
    const float x = TX::load(static_cast<const typename TX::raw *>(A.x)[r * A.ld_x + c]);
    const float dy = TX::load(static_cast<const typename TX::raw *>(A.dy)[r * A.ld_dy + c]);
    dg = __builtin_fmaf(dy, (x - A.mean[r]) * A.rstd[r], dg);
    db += dy;
  }
  A.part[int64_t(blockIdx.y) * A.cols + c] = dg;
  A.part[(int64_t(A.parts) + blockIdx.y) * A.cols + c] = db;
}

template <class TX, class TP>
__global__ void __launch_bounds__(kLongThreads) ln_bwd_long_dx_kernel(const BwdArgs A) {
  __shared__ float lds[2][16][8];
  Sums sums{lds, 0, kLongThreads / 64};
  const float inv = 1.0f / float(A.cols);
  const int64_t i0 = int64_t(threadIdx.x) * 8, step = int64_t(kLongThreads) * 8;
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const void *xr = row_of<TX>(A.x, r, A.ld_x), *dyr = row_of<TX>(A.dy, r, A.ld_dy);
    const float mean = A.mean[r], rstd = A.rstd[r];
    float both[2] = {0.0f, 0.0f};
    Eight<TX> x, dy, ds;
    Eight<TP> w;
    for (int64_t i = i0; i < A.cols; i += step) {
      x.load(xr, i, A.cols - i);
      dy.load(dyr, i, A.cols - i);
      if (A.gamma) w.load(A.gamma, i, A.cols - i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = A.gamma ? dy.get(e) * w.get(e) : dy.get(e);
        both[0] += g;
        // past the row's end: as in the register kernel
        both[1] = __builtin_fmaf(g, (x.get(e) - mean) * (e < A.cols - i ? rstd : 0.0f), both[1]);
      }
    }
    sums.add(both);
    const float c1 = both[0] * inv, c2 = both[1] * inv;
    void *dxr = row_of<TX>(A.dx, r, A.ld_dx);
    for (int64_t i = i0; i < A.cols; i += step) {
      float v[8];
      x.load(xr, i, A.cols - i);
      dy.load(dyr, i, A.cols - i);
      if (A.gamma) w.load(A.gamma, i, A.cols - i);
      if (A.dsum) ds.load(row_of<TX>(A.dsum, r, A.ld_ds), i, A.cols - i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = A.gamma ? dy.get(e) * w.get(e) : dy.get(e);
        v[e] = rstd * (g - c1 - (x.get(e) - mean) * rstd * c2);
        if (A.dsum) v[e] += ds.get(e);
      }
      x.set(v);
      x.store(dxr, i, A.cols - i);
    }
  }
}

// dgamma / dbeta = the sum of the partial rows, in the partials' order within
// each of kSplit interleaved groups, the groups then in order.  Four columns a
// thread.
constexpr int kSplit = 64;
template <class TP>
__global__ void __launch_bounds__(16 * kSplit) ln_bwd_join_kernel(const BwdArgs A) {
  __shared__ float lds[kSplit][68];
  struct __attribute__((packed, aligned(4))) Four {
    float e[4];
  };
  const int64_t c = int64_t(blockIdx.x) * 64 + threadIdx.x * 4;
  void *out = blockIdx.y ? A.dbeta : A.dgamma;
  if (!out) return;
  const float *p = A.part + int64_t(blockIdx.y) * A.parts * A.cols + c;
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
  for (int e = 0; e < 4; ++e) lds[threadIdx.y][threadIdx.x * 4 + e] = s[e];
  __syncthreads();
  const int t = threadIdx.y * 16 + threadIdx.x;
  if (t >= 64 || int64_t(blockIdx.x) * 64 + t >= A.cols) return;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kSplit; ++k) sum += lds[k][t];
  static_cast<typename TP::raw *>(out)[int64_t(blockIdx.x) * 64 + t] = TP::store(sum);
}

// ------------------------------------------------------------------- host

bool desc_ok(const zs_layernorm_desc *d) {
  if (!d || d->rows < 0 || d->cols < 1 || d->cols > (INT64_C(1) << 31)) return false;
  if (d->rows > (INT64_C(1) << 40)) return false;
  if (!dtype_size(d->dtype)) return false;
  if (d->param_dtype != ZS_F32 && d->param_dtype != d->dtype) return false;
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return false;
  const int64_t lds[] = {d->ld_x, d->ld_residual, d->ld_sum, d->ld_y, d->ld_dy, d->ld_dsum,
                         d->ld_dx};
  for (int64_t ld : lds)
    if (ld != 0 && (ld < d->cols || ld > (INT64_C(1) << 40))) return false;
  return true;
}

// How the register kernels take the rows: N times eight columns a thread, R
// rows at a time, `per` threads a row, `subs` row groups a workgroup.
struct Way {
  int n, r, per, subs;
  bool tail;
  int64_t groups;  // of R rows, workgroups
};

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// `even`: all rows start on 16-byte boundaries.
Way way_of(const zs_layernorm_desc &d, bool forward, bool even = true) {
  Way w;
  w.n = d.cols <= kMaxRegCols / 2 ? 1 : 2;
  w.per = int(up(up(d.cols, 8 * w.n) / (8 * w.n), 64));
  // a workgroup's partial row costs as much whatever it covers
  const int threads = forward ? kThreads : 1024;
  w.subs = w.per < threads ? threads / w.per : 1;
  // few rows: a workgroup for each
  if (d.rows < int64_t(kCus) * w.subs) w.subs = int((d.rows + kCus - 1) / kCus);
  if (w.subs < 1) w.subs = 1;
  w.tail = d.cols % 8 != 0 || !even;
  // two rows at a time once every CU has some, where the registers hold them
  w.r = d.rows >= 4 * kCus && w.n == 1 && (forward || d.dtype != ZS_F32) ? 2 : 1;
  const int64_t rows = int64_t(w.subs) * w.r;
  w.groups = (d.rows + rows - 1) / rows;
  return w;
}

template <bool PAIRS, class F>
int by_way(const Way &w, F f) {
  using std::integral_constant;
  const auto rows = [&](auto n, auto tail) {
    if constexpr (PAIRS && n.value == 1)
      if (w.r == 2) return f(n, integral_constant<int, 2>{}, tail);
    return f(n, integral_constant<int, 1>{}, tail);
  };
  const auto cols = [&](auto n) {
    return w.tail ? rows(n, std::true_type{}) : rows(n, std::false_type{});
  };
  return w.n == 1 ? cols(integral_constant<int, 1>{}) : cols(integral_constant<int, 2>{});
}

template <class F>
int by_type(const zs_layernorm_desc &d, F f) {
  if (d.dtype == ZS_F32) return f(F32{}, F32{});
  if (d.dtype == ZS_BF16)
    return d.param_dtype == ZS_F32 ? f(Bf16{}, F32{}) : f(Bf16{}, Bf16{});
  return d.param_dtype == ZS_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
}

// Every row of p starts on a 16-byte boundary (or p is absent).
bool rows_even(const void *p, int64_t ld, int size) {
  return !p || (aligned(p, 16) && ld * size % 16 == 0);
}

// Workgroups of the backward pass, each of which leaves a partial row.
int64_t parts_of(const zs_layernorm_desc &d) {
  const int64_t b = d.cols > kMaxRegCols ? (d.rows + 3) / 4 : way_of(d, false).groups;
  return b < kMaxParts ? b : kMaxParts;
}

}  // namespace

extern "C" {

int zero_shard_layernorm(const zs_layernorm_desc *d, const void *x, const void *residual,
                         const void *gamma, const void *beta, void *sum, void *y, float *mean,
                         float *rstd) {
  if (!desc_ok(d)) return ZS_EINVAL;
  if (d->rows == 0) return ZS_OK;
  if (!x || !y || !residual != !sum || y == sum) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), psize = dtype_size(d->param_dtype);
  if (!aligned(x, size) || !aligned(residual, size) || !aligned(sum, size) || !aligned(y, size) ||
      !aligned(gamma, psize) || !aligned(beta, psize) || !aligned(mean, 4) || !aligned(rstd, 4))
    return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  FwdArgs A{d->rows, d->cols, ld(d->ld_x), ld(d->ld_residual), ld(d->ld_sum), ld(d->ld_y),
            x, residual, gamma, beta, sum, y, mean, rstd, d->eps, 0};
  const bool even = rows_even(x, A.ld_x, size) && rows_even(residual, A.ld_r, size) &&
                    rows_even(sum, A.ld_s, size) && rows_even(y, A.ld_y, size);
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  return by_type(*d, [&](auto tx, auto tp) {
    using TX = decltype(tx);
    using TP = decltype(tp);
    if (A.cols > kMaxRegCols) {
      hipLaunchKernelGGL((ln_fwd_long_kernel<TX, TP>),
                         dim3(unsigned(A.rows < kMaxGrid ? A.rows : kMaxGrid)),
                         dim3(kLongThreads), 0, st, A);
      return launched();
    }
    const Way w = way_of(*d, true, even);
    A.per = w.per;
    const int threads = w.per * w.subs;
    const int64_t most = int64_t(kCus) * (2048 / threads);
    return by_way<true>(w, [&](auto n, auto r, auto tail) {
      hipLaunchKernelGGL((ln_fwd_kernel<TX, TP, n.value, r.value, tail.value>),
                         dim3(unsigned(w.groups < most ? w.groups : most)), dim3(threads), 0, st,
                         A);
      return launched();
    });
  });
}

int64_t zero_shard_layernorm_workspace(const zs_layernorm_desc *d) {
  if (!desc_ok(d)) return -1;
  return 2 * parts_of(*d) * d->cols * int64_t(sizeof(float));
}

int zero_shard_layernorm_bwd(const zs_layernorm_desc *d, const void *dy, const void *x,
                             const void *gamma, const float *mean, const float *rstd,
                             const void *dsum, void *dx, void *dgamma, void *dbeta,
                             void *workspace, int64_t workspace_bytes) {
  if (!desc_ok(d)) return ZS_EINVAL;
  const int size = dtype_size(d->dtype), psize = dtype_size(d->param_dtype);
  const bool params = dgamma || dbeta;
  if (d->rows > 0) {
    if (!dy || !x || !mean || !rstd || !dx) return ZS_EINVAL;
    if (params && (!workspace || workspace_bytes < zero_shard_layernorm_workspace(d)))
      return ZS_EINVAL;
  }
  if (!aligned(dy, size) || !aligned(x, size) || !aligned(dsum, size) || !aligned(dx, size) ||
      !aligned(gamma, psize) || !aligned(dgamma, psize) || !aligned(dbeta, psize) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
    return ZS_EALIGN;
  if (d->rows == 0 && !params) return ZS_OK;
  if (const int rc = device_is_gfx950()) return rc;
  const auto ld = [&](int64_t v) { return v ? v : d->cols; };
  BwdArgs A{d->rows, d->cols, ld(d->ld_dy), ld(d->ld_x), ld(d->ld_dsum), ld(d->ld_dx),
            dy, x, gamma, dsum, mean, rstd, dx, dgamma, dbeta,
            params ? static_cast<float *>(workspace) : nullptr, int32_t(parts_of(*d)), 0};
  const bool even = rows_even(dy, A.ld_dy, size) && rows_even(x, A.ld_x, size) &&
                    rows_even(dsum, A.ld_ds, size) && rows_even(dx, A.ld_dx, size);
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  return by_type(*d, [&](auto tx, auto tp) {
    using TX = decltype(tx);
    using TP = decltype(tp);
    int rc = ZS_OK;
    if (A.rows > 0 && A.cols > kMaxRegCols) {
      if (A.part)
        hipLaunchKernelGGL((ln_bwd_long_cols_kernel<TX>),
                           dim3(unsigned((A.cols + kThreads - 1) / kThreads), unsigned(A.parts)),
                           dim3(kThreads), 0, st, A);
      hipLaunchKernelGGL((ln_bwd_long_dx_kernel<TX, TP>),
                         dim3(unsigned(A.rows < kMaxGrid ? A.rows : kMaxGrid)),
                         dim3(kLongThreads), 0, st, A);
      rc = launched();
    } else if (A.rows > 0) {
      const Way w = way_of(*d, false, even);
      A.per = w.per;
      rc = by_way<!std::is_same_v<TX, F32>>(w, [&](auto n, auto r, auto tail) {
        hipLaunchKernelGGL((ln_bwd_kernel<TX, TP, n.value, r.value, tail.value>), dim3(unsigned(A.parts)),
                           dim3(w.per * w.subs), 0, st, A);
        return launched();
      });
    }
    if (rc || !params) return rc;
    hipLaunchKernelGGL((ln_bwd_join_kernel<TP>), dim3(unsigned((A.cols + 63) / 64), 2),
                       dim3(16, kSplit), 0, st, A);
    return launched();
  });
}

}  // extern "C"
