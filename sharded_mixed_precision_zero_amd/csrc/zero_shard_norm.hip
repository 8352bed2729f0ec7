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
// are HBM-bound, so a row is read once and stays in registers: one wave per
// row up to 2048 columns, a workgroup per row up to 16384, and the variance is
// the centred sum of squares over the registers.  The backward pass keeps
// dgamma and dbeta of the rows it walks in registers too, one partial row of
// each per workgroup, and a second launch adds the partials in a fixed order:
// no atomics, so the same inputs give the same bits.

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
constexpr int kMaxParts = 512;      // partial rows of dgamma / dbeta

// V consecutive elements of a row: one access of V * sizeof(raw) bytes.
template <class T, int V>
struct Pack {
  using raw = typename T::raw;
  static constexpr int kBytes = V * int(sizeof(raw));
  struct alignas(kBytes < 16 ? kBytes : 16) Vec {
    raw e[V];
  };
  static __device__ __forceinline__ void load(const void *row, int64_t i, float (&out)[V]) {
    const Vec v = *reinterpret_cast<const Vec *>(static_cast<const raw *>(row) + i);
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = T::load(v.e[e]);
  }
  static __device__ __forceinline__ void store(void *row, int64_t i, const float (&in)[V]) {
    Vec v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.e[e] = T::store(in[e]);
    *reinterpret_cast<Vec *>(static_cast<raw *>(row) + i) = v;
  }
};

template <class T>
__device__ __forceinline__ float rounded(float v) {
  return T::load(T::store(v));
}

// Sum of a and b over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*lds)[2]) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __syncthreads();  // the previous sum's readers are done
    if ((threadIdx.x & 63) == 0) {
      lds[threadIdx.x >> 6][0] = a;
      lds[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += lds[w][0];
      b += lds[w][1];
    }
  }
}

// The statistics after the centred sweep: off = the sum of (s - mean), zero
// but for the rounding of the mean, becomes what the mean is off by (a row
// far from zero would show it in y); returns rstd.  An infinite row keeps
// its mean.
__device__ __forceinline__ float finish(float sq, float &off, float inv, float eps, float &mean) {
  off *= inv;
  if (!(fabsf(off) < INFINITY)) off = 0.0f;
  mean += off;
  return 1.0f / sqrtf((sq * inv - off * off) + eps);
}

struct FwdArgs {
  int64_t rows, cols;
  int64_t ld_x, ld_r, ld_s, ld_y;  // elements
  const void *x, *residual, *gamma, *beta;
  void *sum, *y;
  float *mean, *rstd;
  float eps;
};

template <class T>
__device__ __forceinline__ const void *row_of(const void *p, int64_t r, int64_t ld) {
  return static_cast<const typename T::raw *>(p) + r * ld;
}
template <class T>
__device__ __forceinline__ void *row_of(void *p, int64_t r, int64_t ld) {
  return static_cast<typename T::raw *>(p) + r * ld;
}

template <int TPR>
constexpr int kBlock = TPR < kThreads ? kThreads : TPR;

// One row per TPR threads, E elements of it in each thread's registers.
template <class TX, class TP, int TPR, int E, int V>
__global__ void __launch_bounds__(kBlock<TPR>) ln_fwd_kernel(const FwdArgs A) {
  constexpr int N = E / V, RPB = kBlock<TPR> / TPR;
  __shared__ float lds[TPR > 64 ? TPR / 64 : 1][2];
  const int t = threadIdx.x % TPR;
  const float inv = 1.0f / float(A.cols);
  for (int64_t r = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR; r < A.rows;
       r += int64_t(gridDim.x) * RPB) {
    float s[N][V];
    const void *xr = row_of<TX>(A.x, r, A.ld_x);
    float total = 0.0f, sq = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
        Pack<TX, V>::load(xr, i, s[j]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) s[j][e] = 0.0f;
      }
    }
    if (A.residual) {
      const void *rr = row_of<TX>(A.residual, r, A.ld_r);
      void *sr = row_of<TX>(A.sum, r, A.ld_s);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int64_t i = int64_t(j * TPR + t) * V;
        if (i < A.cols) {
          float q[V];
          Pack<TX, V>::load(rr, i, q);
#pragma unroll
          for (int e = 0; e < V; ++e) s[j][e] = rounded<TX>(s[j][e] + q[e]);
          Pack<TX, V>::store(sr, i, s[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) total += s[j][e];
    row_sum2<TPR>(total, sq, lds);
    float mean = total * inv, off = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[j][e] -= mean;
          sq = __builtin_fmaf(s[j][e], s[j][e], sq);
          off += s[j][e];
        }
      }
    }
    row_sum2<TPR>(sq, off, lds);
    const float rstd = finish(sq, off, inv, A.eps, mean);
    void *yr = row_of<TX>(A.y, r, A.ld_y);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
        float g[V], b[V];
        if (A.gamma) Pack<TP, V>::load(A.gamma, i, g);
        if (A.beta) Pack<TP, V>::load(A.beta, i, b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float h = (s[j][e] - off) * rstd;
          if (A.gamma) h *= g[e];
          if (A.beta) h += b[e];
          s[j][e] = h;
        }
        Pack<TX, V>::store(yr, i, s[j]);
      }
    }
    if (t == 0) {
      if (A.mean) A.mean[r] = mean;
      if (A.rstd) A.rstd[r] = rstd;
    }
  }
}

// Rows too long for registers: three sweeps, each thread over its own
// elements (which also makes the sum it wrote the sum it reads back).
template <class TX, class TP, int V>
__global__ void __launch_bounds__(kLongThreads) ln_fwd_long_kernel(const FwdArgs A) {
  __shared__ float lds[kLongThreads / 64][2];
  const float inv = 1.0f / float(A.cols);
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const void *xr = row_of<TX>(A.x, r, A.ld_x);
    const void *src = xr;
    float total = 0.0f, sq = 0.0f, none = 0.0f, s[V];
    if (A.residual) {
      const void *rr = row_of<TX>(A.residual, r, A.ld_r);
      void *sr = row_of<TX>(A.sum, r, A.ld_s);
      for (int64_t i = int64_t(threadIdx.x) * V; i < A.cols; i += int64_t(kLongThreads) * V) {
        float q[V];
        Pack<TX, V>::load(xr, i, s);
        Pack<TX, V>::load(rr, i, q);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[e] = rounded<TX>(s[e] + q[e]);
          total += s[e];
        }
        Pack<TX, V>::store(sr, i, s);
      }
      src = sr;
    } else {
      for (int64_t i = int64_t(threadIdx.x) * V; i < A.cols; i += int64_t(kLongThreads) * V) {
        Pack<TX, V>::load(src, i, s);
#pragma unroll
        for (int e = 0; e < V; ++e) total += s[e];
      }
    }
    row_sum2<kLongThreads>(total, none, lds);
    float mean = total * inv, off = 0.0f;
    const float first = mean;
    for (int64_t i = int64_t(threadIdx.x) * V; i < A.cols; i += int64_t(kLongThreads) * V) {
      Pack<TX, V>::load(src, i, s);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = s[e] - first;
        sq = __builtin_fmaf(c, c, sq);
        off += c;
      }
    }
    row_sum2<kLongThreads>(sq, off, lds);
    const float rstd = finish(sq, off, inv, A.eps, mean);
    void *yr = row_of<TX>(A.y, r, A.ld_y);
    for (int64_t i = int64_t(threadIdx.x) * V; i < A.cols; i += int64_t(kLongThreads) * V) {
      float g[V], b[V];
      Pack<TX, V>::load(src, i, s);
      if (A.gamma) Pack<TP, V>::load(A.gamma, i, g);
      if (A.beta) Pack<TP, V>::load(A.beta, i, b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float h = (s[e] - first - off) * rstd;
        if (A.gamma) h *= g[e];
        if (A.beta) h += b[e];
        s[e] = h;
      }
      Pack<TX, V>::store(yr, i, s);
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
};

template <class TX, class TP, int TPR, int E, int V>
__global__ void __launch_bounds__(kBlock<TPR>) ln_bwd_kernel(const BwdArgs A) {
  constexpr int N = E / V, RPB = kBlock<TPR> / TPR;
  __shared__ float lds[TPR > 64 ? TPR / 64 : 1][2];
  __shared__ float join[RPB > 1 ? (RPB - 1) * TPR * E : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.0f / float(A.cols);
  float dg[N][V], db[N][V];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dg[j][e] = db[j][e] = 0.0f;
  for (int64_t r = int64_t(blockIdx.x) * RPB + sub; r < A.rows; r += int64_t(gridDim.x) * RPB) {
    const void *xr = row_of<TX>(A.x, r, A.ld_x), *dyr = row_of<TX>(A.dy, r, A.ld_dy);
    const float mean = A.mean[r], rstd = A.rstd[r];
    float h[N][V], g[N][V];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
        Pack<TX, V>::load(xr, i, h[j]);
        Pack<TX, V>::load(dyr, i, g[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
        float w[V];
        if (A.gamma) Pack<TP, V>::load(A.gamma, i, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[j][e] = (h[j][e] - mean) * rstd;
          dg[j][e] = __builtin_fmaf(g[j][e], h[j][e], dg[j][e]);
          db[j][e] += g[j][e];
          if (A.gamma) g[j][e] *= w[e];
          c1 += g[j][e];
          c2 = __builtin_fmaf(g[j][e], h[j][e], c2);
        }
      }
    }
    row_sum2<TPR>(c1, c2, lds);
    c1 *= inv;
    c2 *= inv;
    void *dxr = row_of<TX>(A.dx, r, A.ld_dx);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
        float d[V];
        if (A.dsum) Pack<TX, V>::load(row_of<TX>(A.dsum, r, A.ld_ds), i, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float v = rstd * (g[j][e] - c1 - h[j][e] * c2);
          if (A.dsum) v += d[e];
          h[j][e] = v;
        }
        Pack<TX, V>::store(dxr, i, h[j]);
      }
    }
  }
  if (!A.part) return;
  // the rows that the workgroup's waves walked side by side, then its partial
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float (&acc)[N][V] = which ? db : dg;
    if (which ? !A.dbeta : !A.dgamma) continue;
    if constexpr (RPB > 1) {
      __syncthreads();
      if (sub > 0) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) join[((sub - 1) * E + j * V + e) * TPR + t] = acc[j][e];
      }
      __syncthreads();
      if (sub > 0) continue;
#pragma unroll
      for (int w = 0; w < RPB - 1; ++w)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[j][e] += join[(w * E + j * V + e) * TPR + t];
    }
    float *out = A.part + (int64_t(which) * A.parts + blockIdx.x) * A.cols;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = int64_t(j * TPR + t) * V;
      if (i < A.cols) {
#pragma unroll
        for (int e = 0; e < V; ++e) out[i + e] = acc[j][e];
      }
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

template <class TX, class TP, int V>
__global__ void __launch_bounds__(kLongThreads) ln_bwd_long_dx_kernel(const BwdArgs A) {
  __shared__ float lds[kLongThreads / 64][2];
  const float inv = 1.0f / float(A.cols);
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const void *xr = row_of<TX>(A.x, r, A.ld_x), *dyr = row_of<TX>(A.dy, r, A.ld_dy);
    const float mean = A.mean[r], rstd = A.rstd[r];
    float c1 = 0.0f, c2 = 0.0f, h[V], g[V], w[V];
    for (int64_t i = int64_t(threadIdx.x) * V; i < A.cols; i += int64_t(kLongThreads) * V) {
      Pack<TX, V>::load(xr, i, h);
      Pack<TX, V>::load(dyr, i, g);
      if (A.gamma) Pack<TP, V>::load(A.gamma, i, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (A.gamma) g[e] *= w[e];
        c1 += g[e];
        c2 = __builtin_fmaf(g[e], (h[e] - mean) * rstd, c2);
      }
    }
    row_sum2<kLongThreads>(c1, c2, lds);
    c1 *= inv;
    c2 *= inv;
    void *dxr = row_of<TX>(A.dx, r, A.ld_dx);
    for (int64_t i = int64_t(threadIdx.x) * V; i < A.cols; i += int64_t(kLongThreads) * V) {
      float d[V];
      Pack<TX, V>::load(xr, i, h);
      Pack<TX, V>::load(dyr, i, g);
      if (A.gamma) Pack<TP, V>::load(A.gamma, i, w);
      if (A.dsum) Pack<TX, V>::load(row_of<TX>(A.dsum, r, A.ld_ds), i, d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (A.gamma) g[e] *= w[e];
        float v = rstd * (g[e] - c1 - (h[e] - mean) * rstd * c2);
        if (A.dsum) v += d[e];
        h[e] = v;
      }
      Pack<TX, V>::store(dxr, i, h);
    }
  }
}

// dgamma / dbeta = the sum of the partial rows, in the partials' order within
// each of kSplit interleaved groups, the groups then in order.
constexpr int kSplit = 16;
template <class TP>
__global__ void __launch_bounds__(64 * kSplit) ln_bwd_join_kernel(const BwdArgs A) {
  __shared__ float lds[kSplit][64];
  const int64_t c = int64_t(blockIdx.x) * 64 + threadIdx.x;
  void *out = blockIdx.y ? A.dbeta : A.dgamma;
  if (!out) return;
  const float *p = A.part + int64_t(blockIdx.y) * A.parts * A.cols;
  float s = 0.0f;
  if (c < A.cols)
    for (int k = threadIdx.y; k < A.parts; k += kSplit) s += p[int64_t(k) * A.cols + c];
  lds[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y || c >= A.cols) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < kSplit; ++k) s += lds[k][threadIdx.x];
  static_cast<typename TP::raw *>(out)[c] = TP::store(s);
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

// Threads per row and elements per thread of the register kernels.
template <int TPR_, int E_>
struct Shape {
  static constexpr int TPR = TPR_, E = E_;
};

template <class F>
int by_shape(int64_t cols, F f) {
  if (cols <= 512) return f(Shape<64, 8>{});
  if (cols <= 1024) return f(Shape<64, 16>{});
  if (cols <= 2048) return f(Shape<64, 32>{});
  if (cols <= 4096) return f(Shape<256, 16>{});
  if (cols <= 8192) return f(Shape<256, 32>{});
  return f(Shape<1024, 16>{});
}

template <class F>
int by_type(const zs_layernorm_desc &d, F f) {
  if (d.dtype == ZS_F32) return f(F32{}, F32{});
  if (d.dtype == ZS_BF16)
    return d.param_dtype == ZS_F32 ? f(Bf16{}, F32{}) : f(Bf16{}, Bf16{});
  return d.param_dtype == ZS_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
}

template <class F>
int by_vector(bool vec, F f) {
  if (!vec) return f(std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, 8>{});
}

int64_t row_blocks(int64_t rows, int per) {
  const int64_t b = (rows + per - 1) / per;
  return b < 0x7fffffff ? b : 0x7fffffff;
}

int64_t parts_of(const zs_layernorm_desc &d) {
  const int rpb = d.cols <= 2048 ? 4 : 1;
  const int64_t b = row_blocks(d.rows, rpb);
  return b < kMaxParts ? b : kMaxParts;
}

// Every row of p starts on a 16-byte boundary (or p is absent).
bool rows_aligned(const void *p, int64_t ld, int size) {
  return !p || (aligned(p, 16) && ld * size % 16 == 0);
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
            x, residual, gamma, beta, sum, y, mean, rstd, d->eps};
  const bool vec = d->cols % 8 == 0 && rows_aligned(x, A.ld_x, size) &&
                   rows_aligned(residual, A.ld_r, size) && rows_aligned(sum, A.ld_s, size) &&
                   rows_aligned(y, A.ld_y, size) && aligned(gamma, 16) && aligned(beta, 16);
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  return by_type(*d, [&](auto tx, auto tp) {
    using TX = decltype(tx);
    using TP = decltype(tp);
    return by_vector(vec, [&](auto v) {
      constexpr int V = decltype(v)::value;
      if (A.cols > kMaxRegCols) {
        hipLaunchKernelGGL((ln_fwd_long_kernel<TX, TP, V>), dim3(unsigned(row_blocks(A.rows, 1))),
                           dim3(kLongThreads), 0, st, A);
        return launched();
      }
      return by_shape(A.cols, [&](auto s) {
        constexpr int TPR = decltype(s)::TPR, E = decltype(s)::E;
        constexpr int B = kBlock<TPR>;
        hipLaunchKernelGGL((ln_fwd_kernel<TX, TP, TPR, E, V>),
                           dim3(unsigned(row_blocks(A.rows, B / TPR))), dim3(B), 0, st, A);
        return launched();
      });
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
            params ? static_cast<float *>(workspace) : nullptr, int32_t(parts_of(*d))};
  const bool vec = d->cols % 8 == 0 && rows_aligned(dy, A.ld_dy, size) &&
                   rows_aligned(x, A.ld_x, size) && rows_aligned(dsum, A.ld_ds, size) &&
                   rows_aligned(dx, A.ld_dx, size) && aligned(gamma, 16);
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  return by_type(*d, [&](auto tx, auto tp) {
    using TX = decltype(tx);
    using TP = decltype(tp);
    int rc = ZS_OK;
    if (A.rows > 0) {
      rc = by_vector(vec, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (A.cols > kMaxRegCols) {
          if (A.part)
            hipLaunchKernelGGL((ln_bwd_long_cols_kernel<TX>),
                               dim3(unsigned((A.cols + kThreads - 1) / kThreads),
                                    unsigned(A.parts)),
                               dim3(kThreads), 0, st, A);
          hipLaunchKernelGGL((ln_bwd_long_dx_kernel<TX, TP, V>),
                             dim3(unsigned(row_blocks(A.rows, 1))), dim3(kLongThreads), 0, st, A);
          return launched();
        }
        return by_shape(A.cols, [&](auto s) {
          constexpr int TPR = decltype(s)::TPR, E = decltype(s)::E;
          hipLaunchKernelGGL((ln_bwd_kernel<TX, TP, TPR, E, V>), dim3(unsigned(A.parts)),
                             dim3(kBlock<TPR>), 0, st, A);
          return launched();
        });
      });
    }
    if (rc || !params) return rc;
    hipLaunchKernelGGL((ln_bwd_join_kernel<TP>), dim3(unsigned((A.cols + 63) / 64), 2),
                       dim3(64, kSplit), 0, st, A);
    return launched();
  });
}

}  // extern "C"
