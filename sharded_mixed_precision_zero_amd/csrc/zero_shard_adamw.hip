// zero_shard_adamw.hip -- the AdamW step of many tensors at once, with states
// in 32 or in 8 bits, and the sum of squares that clips it, on MI355X (gfx950)
// (declarations and the contract: include/zero_shard.h).
//
// One launch takes every tensor: the tensors are cut into chunks of kChunk
// elements, a workgroup takes one, and a table in device memory names each
// chunk's tensor.  The gradients, which a training program allocates anew, come as
// kernel arguments, up to kGrads of them a launch.
//
// The step is HBM-bound: 28 bytes an element with a 16-bit gradient and copy and
// a 32-bit state, 16.06 with an 8-bit one.  A wave takes 256 elements at a time,
// four consecutive ones a lane, so that each of its accesses covers one stretch and
// so that the 256 elements that share a scale are its own: their largest
// magnitude is a maximum over its lanes.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "zero_shard.h"
#include "zs_args.h"
#include "zs_device.h"

namespace {

using namespace zs_dev;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kBlock = ZS_ADAMW_BLOCK;  // elements that share a scale: a wave's
#ifndef KR
#define KR 4
#endif
constexpr int kRounds = KR;              // blocks of a wave
constexpr int64_t kChunk = int64_t(kBlock) * kWaves * kRounds;
constexpr int kGrads = 440;             // a launch's gradients: 3.4 KiB of arguments
constexpr uint64_t kMagic = 0x31776d6164617a73;  // "szadamw1"

// A tensor of the plan, as the kernels read it.
struct Tensor {
  int64_t n, chunk0;  // chunk0: its first chunk
  const float *master_in;
  float *master_out;
  const void *m_in, *v_in;
  void *m_out, *v_out;
  const float *m_scale_in, *v_scale_in;
  float *m_scale_out, *v_scale_out;
  void *param;
  float weight_decay, lr_scale;
  int32_t state, grad_dtype, param_dtype;
  int32_t number;  // in the caller's list
};
static_assert(sizeof(Tensor) == 128, "a tensor of the plan");

struct Header {
  uint64_t magic;
  int64_t count, chunks, bytes;
  int64_t map, partials;  // offsets: the chunks' tensors (int32), their sums of squares (double)
  int64_t pad[2];
};
static_assert(sizeof(Header) == 64, "the plan's header");

struct Grads {
  const void *p[kGrads];
};

struct Consts {
  double b1, omb1, b2, omb2, bc1, bc2, lr, eps, root;  // root = 1 / sqrt(bc2)
};

struct StepArgs {
  const Tensor *tensors;  // of this launch, [0, ..)
  const int32_t *map;     // of all chunks, tensors counted from the first of all
  int64_t chunk0;         // this launch's first chunk
  int32_t tensor0;        // and tensor
  uint32_t key;
  Consts k;
  const double *dyn;      // iff non-null: lr, bc1, bc2, key
  const double *sumsq;    // iff non-null: clip by it
  double max_norm;
};

struct NormArgs {
  const Tensor *tensors;
  const int32_t *map;
  int64_t chunk0;
  int32_t tensor0;
  double *partials;  // of all chunks
};

// The plan's addresses are all of global memory, which the compiler cannot see
// once they come out of a table.
#define ZS_GLOBAL __attribute__((address_space(1)))
template <class T>
__device__ __forceinline__ const ZS_GLOBAL T *global(const void *p, int64_t i) {
  return (const ZS_GLOBAL T *)(uintptr_t(p) + i * int64_t(sizeof(T)));
}
template <class T>
__device__ __forceinline__ ZS_GLOBAL T *global(void *p, int64_t i) {
  return (ZS_GLOBAL T *)(uintptr_t(p) + i * int64_t(sizeof(T)));
}

// Four consecutive elements of any alignment.  They are touched once a step and
// go past the caches.
template <class T>
struct Four {
  using V = T __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  V v;
  // the first `left` of them where that may be fewer, zeros behind
  template <bool TAIL>
  __device__ __forceinline__ void get(const void *p, int64_t i, int64_t left) {
    if (!TAIL || left >= 4) {
      v = __builtin_nontemporal_load((const ZS_GLOBAL V *)global<T>(p, i));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = e < left ? *global<T>(p, i + e) : T(0);
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void put(void *p, int64_t i, int64_t left) const {
    if (!TAIL || left >= 4) {
      __builtin_nontemporal_store(v, (ZS_GLOBAL V *)global<T>(p, i));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) *global<T>(p, i + e) = v[e];
    }
  }
};

__device__ __forceinline__ double clip_coef(double sumsq, double max_norm) {
  const double c = max_norm / (sqrt(sumsq) + 1e-6);
  if (c != c) return c;  // NaN propagates
  return c < 1.0 ? c : 1.0;
}

// 32 bits, each of which depends on all of x's.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6a09e667u;  // the fractions of sqrt 2 and sqrt 3
  x ^= x >> 15;
  x *= 0xbb67ae85u;
  return x ^ (x >> 16);
}

// ---- states in 8 bits: e4m3 numbers of at most 256, times a scale

// The larger of two magnitudes as bits: a NaN is larger than all else.
__device__ __forceinline__ unsigned larger(unsigned a, unsigned b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ unsigned dpp_larger(unsigned v) {
  return larger(v, __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false));
}

// The largest of the wave's two magnitudes, a's in lanes 0-31, b's in the others:
// after one exchange of halves each lane carries on with one of them.
__device__ __forceinline__ unsigned wave_tops(unsigned a, unsigned b) {
  const auto halves = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  unsigned v = larger(halves[0], halves[1]);
  const auto rows = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = larger(rows[0], rows[1]);
  v = dpp_larger<0xb1>(v);     // lanes 1 apart
  v = dpp_larger<0x4e>(v);     // 2 apart
  v = dpp_larger<0x141>(v);    // half row mirrored
  return dpp_larger<0x140>(v); // row mirrored
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

struct Lane {
  Four<float> w;
  Four<float> g32;      // gradients, of one of the types
  Four<uint16_t> g16;
  Four<float> m32, v32; // states, of one of them
  unsigned m8, v8;
  float ms, vs;
};

template <bool EIGHT, bool TAIL>
__device__ __forceinline__ void load_state(const Tensor &T, Lane &s, int64_t i, int64_t left) {
  s.w.template get<TAIL>(T.master_in, i, left);
  if constexpr (EIGHT) {
    using Word = unsigned __attribute__((aligned(1)));
    if (!TAIL || left >= 4) {
      s.m8 = __builtin_nontemporal_load((const ZS_GLOBAL Word *)global<uint8_t>(T.m_in, i));
      s.v8 = __builtin_nontemporal_load((const ZS_GLOBAL Word *)global<uint8_t>(T.v_in, i));
    } else {
      s.m8 = s.v8 = 0;
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < left) {
          s.m8 |= unsigned(*global<uint8_t>(T.m_in, i + e)) << (8 * e);
          s.v8 |= unsigned(*global<uint8_t>(T.v_in, i + e)) << (8 * e);
        }
    }
    // one for the wave
    const int64_t block = (i - int64_t(threadIdx.x & 63) * 4) / kBlock;
    const bool in = !TAIL || block * kBlock < T.n;
    s.ms = in ? *global<float>(T.m_scale_in, block) : 0.0f;
    s.vs = in ? *global<float>(T.v_scale_in, block) : 0.0f;
  } else {
    s.m32.template get<TAIL>(T.m_in, i, left);
    s.v32.template get<TAIL>(T.v_in, i, left);
  }
}

template <class TG, bool TAIL>
__device__ __forceinline__ void load_grad(const void *g, Lane &s, int64_t i, int64_t left) {
  if constexpr (std::is_same_v<TG, F32>) s.g32.template get<TAIL>(g, i, left);
  else s.g16.template get<TAIL>(g, i, left);
}

template <class TG>
__device__ __forceinline__ float grad_of(const Lane &s, int e) {
  if constexpr (std::is_same_v<TG, F32>) return s.g32.v[e];
  else return TG::load(s.g16.v[e]);
}

// A tensor's constants of the step.
struct Rates {
  double coef, decay, lr;  // lr times the tensor's factor, and that times its weight decay
  // 8 bits, whose roots are held times 2^16 so that squares of small gradients stay
  // normal numbers: b2 and omb2 times 2^32, root = 2^-16 / sqrt(bc2)
  float coef32, b1, omb1, b2, omb2, root, eps;
  double step;                                  // lr / bc1
};

template <class T, bool TAIL>
__device__ __forceinline__ void put_copy(const Tensor &t, const Four<float> &w, int64_t i,
                                         int64_t left) {
  Four<uint16_t> p;
#pragma unroll
  for (int e = 0; e < 4; ++e) p.v[e] = T::store(w.v[e]);
  p.template put<TAIL>(t.param, i, left);
}

template <bool TAIL>
__device__ __forceinline__ void put_weights(const Tensor &T, const Four<float> &w, int64_t i,
                                            int64_t left) {
  w.template put<TAIL>(T.master_out, i, left);
  if (!T.param) return;
  if (T.param_dtype == ZS_BF16) put_copy<Bf16, TAIL>(T, w, i, left);
  else put_copy<F16, TAIL>(T, w, i, left);
}

// AdamW on a lane's four elements: binary64 from the binary32 state, one
// rounding per stored value, in the shard step's order.
template <class TG, bool TAIL>
__device__ __forceinline__ void update32(const Tensor &T, const Consts &k, const Rates &rates,
                                         Lane &s, int64_t i, int64_t left) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double g = rates.coef * double(grad_of<TG>(s, e));
    const double m1 = k.b1 * double(s.m32.v[e]) + k.omb1 * g;
    const double v1 = k.b2 * double(s.v32.v[e]) + k.omb2 * (g * g);
    const double mhat = m1 / k.bc1;
    const double vhat = v1 / k.bc2;
    const double t0 = double(s.w.v[e]);
    const double t1 = t0 - rates.decay * t0 - rates.lr * mhat / (sqrt(vhat) + k.eps);
    s.w.v[e] = float(t1);
    s.m32.v[e] = float(m1);
    s.v32.v[e] = float(v1);
  }
  put_weights<TAIL>(T, s.w, i, left);
  s.m32.template put<TAIL>(T.m_out, i, left);
  s.v32.template put<TAIL>(T.v_out, i, left);
}

// The same with a state in 8 bits.  The moments are binary32 numbers, which
// rounding to 4 significant bits makes little of, with a root and a quotient of an
// instruction or two, within 2^-23 and 2^-22: what the memory leaves time for is some
// 100 instructions an element, and binary64 as above takes more (1034 us for 570 of
// 163.84M elements).  The weights are binary64 as above.
template <class TG, bool TAIL>
__device__ __forceinline__ void update8(const Tensor &T, const Rates &rates, uint32_t base,
                                        Lane &s, int64_t i, int64_t left) {
  float m[4], r[4];
  unsigned mtop = 0, vtop = 0;
  using Two = float __attribute__((ext_vector_type(2)));
  const Two m8[2] = {__builtin_amdgcn_cvt_pk_f32_fp8(s.m8, false),
                     __builtin_amdgcn_cvt_pk_f32_fp8(s.m8, true)};
  const Two v8[2] = {__builtin_amdgcn_cvt_pk_f32_fp8(s.v8, false),
                     __builtin_amdgcn_cvt_pk_f32_fp8(s.v8, true)};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float g = rates.coef32 * grad_of<TG>(s, e);
    const float m0 = m8[e / 2][e % 2] * s.ms, r0 = v8[e / 2][e % 2] * s.vs;
    m[e] = rates.b1 * m0 + rates.omb1 * g;
    r[e] = __builtin_amdgcn_sqrtf((rates.b2 * r0) * r0 + (rates.omb2 * g) * g);
    const double t0 = double(s.w.v[e]);
    const float u = m[e] * __builtin_amdgcn_rcpf(r[e] * rates.root + rates.eps);
    s.w.v[e] = float(t0 - rates.decay * t0 - rates.step * double(u));
    // what is not there counts for nothing: its gradient and state are 0
    mtop = larger(mtop, __float_as_uint(m[e]) & 0x7fffffffu);
    vtop = larger(vtop, __float_as_uint(r[e]) & 0x7fffffffu);
  }
  put_weights<TAIL>(T, s.w, i, left);
  // Scales, and the factors that take magnitudes to [0, 256], m's in the wave's first
  // half, r's in the other.  Blocks of nothing but numbers below 2^-100 are zeros (NaN
  // is not below), so that neither leaves binary32.
  const int lane = threadIdx.x & 63;
  const float held = lane < 32 ? 1.0f : 0x1p-16f;
  const float top = __uint_as_float(wave_tops(mtop, vtop)) * held;
  const bool none = top < 0x1p-100f;
  const float scale = none ? 0.0f : top * 0x1p-8f;
  const float inv = none ? 0.0f : __builtin_amdgcn_rcpf(scale) * held;
  const float minv = lane_value(inv, 0), vinv = lane_value(inv, 32);
  // to e4m3, down or up where 20 bits of dither carry into the number
  unsigned mw = 0, vw = 0;
  const auto encode = [&](auto place) {
    constexpr int e = place.value;
    const uint32_t h = mix(base + uint32_t(i + e));
    const float a = __builtin_amdgcn_fmed3f(m[e] * minv, -256.0f, 256.0f);
    // a root that is there stays above the least number
    const float b = __builtin_amdgcn_fmed3f(r[e] * vinv, r[e] > 0.0f ? 0x1p-9f : 0.0f, 256.0f);
    mw = __builtin_amdgcn_cvt_sr_fp8_f32(a, h << 16 | 0x8000u, mw, e);
    vw = __builtin_amdgcn_cvt_sr_fp8_f32(b, (h & 0xffff0000u) | 0x8000u, vw, e);
  };
  encode(std::integral_constant<int, 0>{});
  encode(std::integral_constant<int, 1>{});
  encode(std::integral_constant<int, 2>{});
  encode(std::integral_constant<int, 3>{});
  if (!TAIL || left >= 4) {
    using Word = unsigned __attribute__((aligned(1)));
    __builtin_nontemporal_store(mw, (ZS_GLOBAL Word *)global<uint8_t>(T.m_out, i));
    __builtin_nontemporal_store(vw, (ZS_GLOBAL Word *)global<uint8_t>(T.v_out, i));
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < left) {
        *global<uint8_t>(T.m_out, i + e) = uint8_t(mw >> (8 * e));
        *global<uint8_t>(T.v_out, i + e) = uint8_t(vw >> (8 * e));
      }
  }
  if ((lane == 0 || lane == 32) && i - lane * 4 < T.n)
    *global<float>(lane ? T.v_scale_out : T.m_scale_out, i / kBlock) = scale;
}

template <bool EIGHT, class TG, bool TAIL>
__device__ __forceinline__ void step_chunk(const Tensor &T, const void *g, const Consts &k,
                                           const Rates &rates, uint32_t key, int64_t from) {
  const int64_t i0 = from + int64_t(threadIdx.x >> 6) * (kBlock * kRounds) + (threadIdx.x & 63) * 4;
  const uint32_t base = mix(key + 0x9e3779b9u * uint32_t(T.number + 1)) +
                        mix(uint32_t(uint64_t(from) >> 32)) * 0x9e3779b9u;
  Lane s[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = i0 + r * kBlock;
    load_state<EIGHT, TAIL>(T, s[r], i, T.n - i);
    load_grad<TG, TAIL>(g, s[r], i, T.n - i);
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = i0 + r * kBlock;
    if constexpr (EIGHT) update8<TG, TAIL>(T, rates, base, s[r], i, T.n - i);
    else update32<TG, TAIL>(T, k, rates, s[r], i, T.n - i);
  }
}

template <bool EIGHT, class TG>
__device__ __forceinline__ void step_any(const Tensor &T, const void *g, const Consts &k,
                                         const Rates &rates, uint32_t key, int64_t from) {
  if (T.n - from < kChunk) step_chunk<EIGHT, TG, true>(T, g, k, rates, key, from);
  else step_chunk<EIGHT, TG, false>(T, g, k, rates, key, from);
}

__global__ void __launch_bounds__(kThreads) adamw_step_kernel(const StepArgs A, const Grads G) {
  const int64_t chunk = A.chunk0 + blockIdx.x;
  const int at = __builtin_amdgcn_readfirstlane(A.map[chunk]) - A.tensor0;
  const Tensor &T = A.tensors[at];
  const void *g = G.p[at];
  Consts k = A.k;
  uint32_t key = A.key;
  if (A.dyn) {
    k.lr = A.dyn[0];
    k.bc1 = A.dyn[1];
    k.bc2 = A.dyn[2];
    k.root = 1.0 / sqrt(k.bc2);
    key = uint32_t(A.dyn[3]);
  }
  Rates rates;
  rates.coef = A.sumsq ? clip_coef(*A.sumsq, A.max_norm) : 1.0;
  rates.lr = k.lr * double(T.lr_scale);
  rates.decay = rates.lr * double(T.weight_decay);
  const int64_t from = (chunk - T.chunk0) * kChunk;
  if (T.state == ZS_STATE_8) {
    rates.coef32 = float(rates.coef);
    rates.b1 = float(k.b1);
    rates.omb1 = float(k.omb1);
    rates.b2 = float(k.b2) * 0x1p32f;
    rates.omb2 = float(k.omb2) * 0x1p32f;
    rates.root = float(k.root) * 0x1p-16f;
    rates.eps = fmaxf(float(k.eps), 0x1p-126f);  // which a quotient by it needs
    rates.step = rates.lr / k.bc1;
    if (T.grad_dtype == ZS_F32) step_any<true, F32>(T, g, k, rates, key, from);
    else if (T.grad_dtype == ZS_BF16) step_any<true, Bf16>(T, g, k, rates, key, from);
    else step_any<true, F16>(T, g, k, rates, key, from);
  } else {
    if (T.grad_dtype == ZS_F32) step_any<false, F32>(T, g, k, rates, key, from);
    else if (T.grad_dtype == ZS_BF16) step_any<false, Bf16>(T, g, k, rates, key, from);
    else step_any<false, F16>(T, g, k, rates, key, from);
  }
}

// A chunk's sum of squares (binary64): a lane's elements in order, a
// butterfly over the wave, the waves in order.
template <class TG>
__device__ __forceinline__ double chunk_squares(const Tensor &T, const void *g, int64_t from) {
  const int64_t i0 = from + int64_t(threadIdx.x >> 6) * (kBlock * kRounds) + (threadIdx.x & 63) * 4;
  Lane s[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    load_grad<TG, true>(g, s[r], i0 + r * kBlock, T.n - i0 - r * kBlock);
  double sum = 0.0;
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double x = double(grad_of<TG>(s[r], e));
      sum += x * x;
    }
  return sum;
}

__global__ void __launch_bounds__(kThreads) adamw_norm_kernel(const NormArgs A, const Grads G) {
  __shared__ double sums[kWaves];
  const int64_t chunk = A.chunk0 + blockIdx.x;
  const int at = __builtin_amdgcn_readfirstlane(A.map[chunk]) - A.tensor0;
  const Tensor &T = A.tensors[at];
  const int64_t from = (chunk - T.chunk0) * kChunk;
  double sum = T.grad_dtype == ZS_F32    ? chunk_squares<F32>(T, G.p[at], from)
               : T.grad_dtype == ZS_BF16 ? chunk_squares<Bf16>(T, G.p[at], from)
                                         : chunk_squares<F16>(T, G.p[at], from);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) sum += sums[w];
    A.partials[chunk] = sum;
  }
}

// The chunks' sums, each thread a strided run of them, then a tree.
constexpr int kFinalThreads = 1024;
__global__ void __launch_bounds__(kFinalThreads) adamw_total_kernel(const double *partials,
                                                                    int64_t n, double *out) {
  __shared__ double sums[kFinalThreads];
  double s = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += kFinalThreads) s += partials[i];
  sums[threadIdx.x] = s;
  __syncthreads();
  for (int half = kFinalThreads / 2; half > 0; half >>= 1) {
    if (int(threadIdx.x) < half) sums[threadIdx.x] += sums[threadIdx.x + half];
    __syncthreads();
  }
  if (threadIdx.x == 0) *out = sums[0];
}

// ------------------------------------------------------------------- host

bool desc_ok(const zs_adamw_desc *d) {
  if (!d || d->count < 0 || d->count > ZS_ADAMW_MAX_TENSORS) return false;
  if (!(d->beta1 >= 0.0f && d->beta1 < 1.0f && d->beta2 >= 0.0f && d->beta2 < 1.0f)) return false;
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return false;
  if (d->bias_correction != 0 && d->bias_correction != 1) return false;
  return std::isfinite(d->max_norm);
}

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// One tensor's fields and pointers.
int tensor_ok(const zs_adamw_tensor &t) {
  if (t.n < 0 || t.n > ZS_ADAMW_MAX_ELEMENTS) return ZS_EINVAL;
  if (t.state != ZS_STATE_32 && t.state != ZS_STATE_8) return ZS_EINVAL;
  if (!dtype_size(t.grad_dtype)) return ZS_EINVAL;
  if (t.param_out && t.param_dtype != ZS_BF16 && t.param_dtype != ZS_F16) return ZS_EINVAL;
  if (!(t.weight_decay >= 0.0f) || !std::isfinite(t.weight_decay)) return ZS_EINVAL;
  if (!(t.lr_scale >= 0.0f) || !std::isfinite(t.lr_scale)) return ZS_EINVAL;
  if (t.n == 0) return ZS_OK;
  if (!t.master_in || !t.master_out || !t.m_in || !t.m_out || !t.v_in || !t.v_out) return ZS_EINVAL;
  const bool eight = t.state == ZS_STATE_8;
  for (const void *p : {static_cast<const void *>(t.m_scale_in),
                        static_cast<const void *>(t.m_scale_out),
                        static_cast<const void *>(t.v_scale_in),
                        static_cast<const void *>(t.v_scale_out)}) {
    if (!p != !eight) return ZS_EINVAL;
    if (!aligned(p, 4)) return ZS_EALIGN;
  }
  const uintptr_t state = eight ? 1 : 4;
  if (!aligned(t.master_in, 4) || !aligned(t.master_out, 4) || !aligned(t.m_in, state) ||
      !aligned(t.m_out, state) || !aligned(t.v_in, state) || !aligned(t.v_out, state) ||
      !aligned(t.param_out, 2))
    return ZS_EALIGN;
  return ZS_OK;
}

// What the step writes overlaps nothing else that it writes: the same tensor
// given twice, or two that share memory, would be updated in no order.
int outputs_apart(const zs_adamw_tensor *t, int64_t count) {
  try {
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;
    const auto add = [&](const void *p, int64_t bytes) {
      if (p && bytes) spans.emplace_back(uintptr_t(p), uintptr_t(p) + uintptr_t(bytes));
    };
    for (int64_t k = 0; k < count; ++k) {
      const int64_t n = t[k].n, size = t[k].state == ZS_STATE_8 ? 1 : 4;
      if (n == 0) continue;
      add(t[k].master_out, 4 * n);
      add(t[k].m_out, size * n);
      add(t[k].v_out, size * n);
      add(t[k].param_out, 2 * n);
      add(t[k].m_scale_out, 4 * blocks_of(n));
      add(t[k].v_scale_out, 4 * blocks_of(n));
    }
    std::sort(spans.begin(), spans.end());
    for (size_t k = 1; k < spans.size(); ++k)
      if (spans[k].first < spans[k - 1].second) return ZS_EINVAL;
  } catch (const std::bad_alloc &) {
    return ZS_ENOMEM;
  }
  return ZS_OK;
}

struct Layout {
  int64_t chunks = 0, map = 0, partials = 0, bytes = -1;
  Layout(const zs_adamw_desc *d, const zs_adamw_tensor *t) {
    if (!desc_ok(d) || (d->count && !t)) return;
    for (int64_t k = 0; k < d->count; ++k) {
      if (t[k].n < 0 || t[k].n > ZS_ADAMW_MAX_ELEMENTS) return;
      chunks += chunks_of(t[k].n);
    }
    if (chunks > INT32_MAX / kThreads) return;  // a launch takes them all
    const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    map = up(int64_t(sizeof(Header)) + d->count * int64_t(sizeof(Tensor)));
    partials = map + up(chunks * 4);
    bytes = partials + up(chunks * 8);
  }
};

const Header *header_of(const void *plan, const zs_adamw_desc *d) {
  const Header *h = static_cast<const Header *>(plan);
  return h && aligned(h, 16) && h->magic == kMagic && h->count == d->count ? h : nullptr;
}
const Tensor *tensors_of(const void *plan) {
  return reinterpret_cast<const Tensor *>(static_cast<const char *>(plan) + sizeof(Header));
}

// The checks of the step and the norm alike: the plan's two copies and the gradients.
int call_ok(const zs_adamw_desc *d, const void *plan, const void *plan_dev,
            const void *const *grads) {
  if (!desc_ok(d)) return ZS_EINVAL;
  const Header *h = header_of(plan, d);
  if (!h || (h->count && !grads)) return ZS_EINVAL;
  if (h->chunks && !plan_dev) return ZS_EINVAL;
  if (!aligned(plan_dev, 256)) return ZS_EALIGN;
  const Tensor *t = tensors_of(plan);
  for (int64_t k = 0; k < h->count; ++k) {
    if (t[k].n && !grads[k]) return ZS_EINVAL;
    if (t[k].n && !aligned(grads[k], dtype_size(t[k].grad_dtype))) return ZS_EALIGN;
  }
  return ZS_OK;
}

// One launch for every kGrads tensors that have elements among them.
template <class F>
int by_launch(const void *plan, const void *const *grads, F f) {
  const Header *h = static_cast<const Header *>(plan);
  const Tensor *t = tensors_of(plan);
  for (int64_t k = 0; k < h->count; k += kGrads) {
    const int64_t to = k + kGrads < h->count ? k + kGrads : h->count;
    const int64_t from_chunk = t[k].chunk0;
    const int64_t chunks = (to < h->count ? t[to].chunk0 : h->chunks) - from_chunk;
    if (chunks == 0) continue;
    Grads G;
    for (int64_t j = k; j < to; ++j) G.p[j - k] = grads[j];
    f(k, from_chunk, unsigned(chunks), G);
    if (const int rc = launched()) return rc;
  }
  return ZS_OK;
}

int step(const zs_adamw_desc *d, const void *plan, void *plan_dev, const void *const *grads,
         double lr, int64_t t, uint32_t key, const double *dyn, const double *sumsq) {
  if (const int rc = call_ok(d, plan, plan_dev, grads)) return rc;
  if ((d->max_norm > 0.0f) != (sumsq != nullptr)) return ZS_EINVAL;
  if (!aligned(sumsq, 8) || !aligned(dyn, 8)) return ZS_EALIGN;
  const Header *h = static_cast<const Header *>(plan);
  if (h->chunks == 0) return ZS_OK;
  if (const int rc = device_is_gfx950()) return rc;
  const double b1 = double(d->beta1), b2 = double(d->beta2);
  Consts k{b1, 1.0 - b1, b2, 1.0 - b2, 1.0, 1.0, lr, double(d->eps), 1.0};
  if (d->bias_correction) {
    k.bc1 = 1.0 - std::pow(b1, double(t));
    k.bc2 = 1.0 - std::pow(b2, double(t));
    k.root = 1.0 / std::sqrt(k.bc2);
  }
  const char *dev = static_cast<const char *>(plan_dev);
  return by_launch(plan, grads, [&](int64_t tensor0, int64_t chunk0, unsigned chunks,
                                    const Grads &G) {
    const StepArgs A{tensors_of(plan_dev) + tensor0,
                     reinterpret_cast<const int32_t *>(dev + h->map), chunk0, int32_t(tensor0), key,
                     k, dyn, sumsq, double(d->max_norm)};
    hipLaunchKernelGGL(adamw_step_kernel, dim3(chunks), dim3(kThreads), 0,
                       static_cast<hipStream_t>(d->stream), A, G);
  });
}

}  // namespace

extern "C" {

int64_t zero_shard_adamw_plan_bytes(const zs_adamw_desc *d, const zs_adamw_tensor *tensors) {
  return Layout(d, tensors).bytes;
}

int zero_shard_adamw_plan(const zs_adamw_desc *d, const zs_adamw_tensor *tensors, void *plan,
                          int64_t plan_bytes) {
  const Layout l(d, tensors);
  if (l.bytes < 0 || !plan || plan_bytes < l.bytes) return ZS_EINVAL;
  if (!aligned(plan, 16)) return ZS_EALIGN;
  for (int64_t k = 0; k < d->count; ++k)
    if (const int rc = tensor_ok(tensors[k])) return rc;
  if (const int rc = outputs_apart(tensors, d->count)) return rc;
  char *at = static_cast<char *>(plan);
  std::memset(at, 0, size_t(l.bytes));
  Header h{};
  h.magic = kMagic;
  h.count = d->count;
  h.chunks = l.chunks;
  h.bytes = l.bytes;
  h.map = l.map;
  h.partials = l.partials;
  std::memcpy(at, &h, sizeof h);
  Tensor *out = reinterpret_cast<Tensor *>(at + sizeof h);
  int32_t *map = reinterpret_cast<int32_t *>(at + l.map);
  int64_t chunk = 0;
  for (int64_t k = 0; k < d->count; ++k) {
    const zs_adamw_tensor &t = tensors[k];
    out[k] = Tensor{t.n, chunk, t.master_in, t.master_out, t.m_in, t.v_in, t.m_out, t.v_out,
                    t.m_scale_in, t.v_scale_in, t.m_scale_out, t.v_scale_out, t.param_out,
                    t.weight_decay, t.lr_scale, t.state, t.grad_dtype, t.param_dtype, int32_t(k)};
    for (int64_t c = chunks_of(t.n); c > 0; --c) map[chunk++] = int32_t(k);
  }
  return ZS_OK;
}

int zero_shard_adamw_gnorm(const zs_adamw_desc *d, const void *plan, void *plan_dev,
                           const void *const *grads, double *sumsq_dev) {
  if (const int rc = call_ok(d, plan, plan_dev, grads)) return rc;
  if (!sumsq_dev) return ZS_EINVAL;
  if (!aligned(sumsq_dev, 8)) return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  const Header *h = static_cast<const Header *>(plan);
  char *dev = static_cast<char *>(plan_dev);
  double *partials = reinterpret_cast<double *>(dev + h->partials);
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  if (const int rc = by_launch(plan, grads, [&](int64_t tensor0, int64_t chunk0, unsigned chunks,
                                                const Grads &G) {
        const NormArgs A{tensors_of(plan_dev) + tensor0,
                         reinterpret_cast<const int32_t *>(dev + h->map), chunk0,
                         int32_t(tensor0), partials};
        hipLaunchKernelGGL(adamw_norm_kernel, dim3(chunks), dim3(kThreads), 0, st, A, G);
      }))
    return rc;
  hipLaunchKernelGGL(adamw_total_kernel, dim3(1), dim3(kFinalThreads), 0, st, partials, h->chunks,
                     sumsq_dev);
  return launched();
}

int zero_shard_adamw(const zs_adamw_desc *d, const void *plan, void *plan_dev,
                     const void *const *grads, float lr, int64_t t, uint32_t key,
                     const double *global_sumsq_dev) {
  if (!zs_args::step_ok(lr, t)) return ZS_EINVAL;
  return step(d, plan, plan_dev, grads, double(lr), t, key, nullptr, global_sumsq_dev);
}

int zero_shard_adamw_consts(const zs_adamw_desc *d, float lr, int64_t t, uint32_t key,
                            double *out) {
  if (!desc_ok(d) || !out || !zs_args::step_ok(lr, t)) return ZS_EINVAL;
  out[0] = double(lr);
  out[1] = d->bias_correction ? 1.0 - std::pow(double(d->beta1), double(t)) : 1.0;
  out[2] = d->bias_correction ? 1.0 - std::pow(double(d->beta2), double(t)) : 1.0;
  out[3] = double(key);
  return ZS_OK;
}

int zero_shard_adamw_dev(const zs_adamw_desc *d, const void *plan, void *plan_dev,
                         const void *const *grads, const double *consts_dev,
                         const double *global_sumsq_dev) {
  if (!consts_dev) return ZS_EINVAL;
  return step(d, plan, plan_dev, grads, 0.0, 1, 0, consts_dev, global_sumsq_dev);
}

}  // extern "C"
