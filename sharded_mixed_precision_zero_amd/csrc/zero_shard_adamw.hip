// zero_shard_adamw.hip -- the AdamW step of many tensors at once, with states
// in 32 or in 8 bits, and the sum of squares that clips it, on MI355X (gfx950)
// (declarations and the contract: include/zero_shard.h).
//
// One launch takes all tensors of a kind of state: they are cut into chunks, a
// workgroup takes one, and a table in device memory names each chunk's tensor.  The
// gradients, which a training program allocates anew, come as kernel arguments,
// up to kGrads of them a launch.  The kinds have a launch each because the
// registers of one (binary64 in the shard step's order) would leave the other too few
// waves (163.84M elements in 8 bits, then: 543 us in one launch, 485 in its own).
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
// Blocks of a wave, in flight together, and elements of a workgroup.  A 32-bit state
// has bytes enough in flight with one block, and short chains of work a wave (160
// tensors of 5120: 6.0 us for 8.4 with two; 163.84M elements 778 for 811); an 8-bit
// one was a little faster with two (513 for 527).
template <bool EIGHT>
constexpr int kRounds = EIGHT ? 2 : 1;
template <bool EIGHT>
constexpr int64_t kChunk = int64_t(kBlock) * kWaves * kRounds<EIGHT>;
// Chunks of a wave of the norm: 8, or 1 where the waves would be few (160 tensors of
// 5120: 10 us for 14).
constexpr int kNormChunks = 8;
constexpr int64_t kFewChunks = 8192;
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
  int64_t map, partials;  // offsets: the chunks' tensors (int32), sums of squares (double)
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
  int64_t chunk0, chunks;  // this launch's
  int32_t tensor0, each;   // each: chunks of a wave
  double *partials;        // a workgroup's each, of this launch
};

// The plan's addresses are all of global memory, which the compiler cannot see
// once they come out of a table.
#define ZS_GLOBAL __attribute__((address_space(1)))
template <class T>
__device__ __forceinline__ const ZS_GLOBAL T *global(const void *p, int64_t i) {
  return (const ZS_GLOBAL T *)(uintptr_t(p) + i * int64_t(sizeof(T)));
}

// Where a lane is in its tensor: element `from`, the same for the workgroup, and
// `at` behind it, which an access adds by itself.  `left`: elements from there on.
struct Place {
  int64_t from;
  unsigned at;
  int64_t left;
  template <class T>
  __device__ __forceinline__ const ZS_GLOBAL T *of(const void *p, unsigned e = 0) const {
    return (const ZS_GLOBAL T *)((const ZS_GLOBAL char *)(uintptr_t(p) + from * int64_t(sizeof(T))) +
                                 (at + e) * unsigned(sizeof(T)));
  }
  template <class T>
  __device__ __forceinline__ ZS_GLOBAL T *of(void *p, unsigned e = 0) const {
    return (ZS_GLOBAL T *)((ZS_GLOBAL char *)(uintptr_t(p) + from * int64_t(sizeof(T))) +
                           (at + e) * unsigned(sizeof(T)));
  }
};

// Four consecutive elements of any alignment.  They are touched once a step and
// go past the caches.
template <class T>
struct Four {
  using V = T __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  V v;
  // the first `left` of them where that may be fewer, zeros behind
  template <bool TAIL>
  __device__ __forceinline__ void get(const void *p, const Place &i) {
    if (!TAIL || i.left >= 4) {
      v = __builtin_nontemporal_load((const ZS_GLOBAL V *)i.of<T>(p));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = e < i.left ? *i.of<T>(p, e) : T(0);
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void put(void *p, const Place &i) const {
    if (!TAIL || i.left >= 4) {
      __builtin_nontemporal_store(v, (ZS_GLOBAL V *)i.of<T>(p));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < i.left) *i.of<T>(p, e) = v[e];
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
__device__ __forceinline__ void load_state(const Tensor &T, Lane &s, const Place &i) {
  s.w.template get<TAIL>(T.master_in, i);
  if constexpr (EIGHT) {
    using Word = unsigned __attribute__((aligned(1)));
    if (!TAIL || i.left >= 4) {
      s.m8 = __builtin_nontemporal_load((const ZS_GLOBAL Word *)i.of<uint8_t>(T.m_in));
      s.v8 = __builtin_nontemporal_load((const ZS_GLOBAL Word *)i.of<uint8_t>(T.v_in));
    } else {
      s.m8 = s.v8 = 0;
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < i.left) {
          s.m8 |= unsigned(*i.of<uint8_t>(T.m_in, e)) << (8 * e);
          s.v8 |= unsigned(*i.of<uint8_t>(T.v_in, e)) << (8 * e);
        }
    }
    // one for the wave
    const int64_t block = i.from / kBlock + __builtin_amdgcn_readfirstlane(i.at / kBlock);
    const bool in = !TAIL || block * kBlock < T.n;
    s.ms = in ? *global<float>(T.m_scale_in, block) : 0.0f;
    s.vs = in ? *global<float>(T.v_scale_in, block) : 0.0f;
  } else {
    s.m32.template get<TAIL>(T.m_in, i);
    s.v32.template get<TAIL>(T.v_in, i);
  }
}

template <class TG, bool TAIL>
__device__ __forceinline__ void load_grad(const void *g, Lane &s, const Place &i) {
  if constexpr (std::is_same_v<TG, F32>) s.g32.template get<TAIL>(g, i);
  else s.g16.template get<TAIL>(g, i);
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
__device__ __forceinline__ void put_copy(const Tensor &t, const Four<float> &w, const Place &i) {
  Four<uint16_t> p;
#pragma unroll
  for (int e = 0; e < 4; ++e) p.v[e] = T::store(w.v[e]);
  p.template put<TAIL>(t.param, i);
}

template <bool TAIL>
__device__ __forceinline__ void put_weights(const Tensor &T, const Four<float> &w,
                                            const Place &i) {
  w.template put<TAIL>(T.master_out, i);
  if (!T.param) return;
  if (T.param_dtype == ZS_BF16) put_copy<Bf16, TAIL>(T, w, i);
  else put_copy<F16, TAIL>(T, w, i);
}

// The root, rounded, of a number from 2^-96 on (below, differences of products are no
// normal numbers).  The instruction's is within a step; a neighbour is nearer where the
// number lies beyond the product of the two: the square of what lies halfway between
// them is that and a quarter of a step's square, and no number lies in between.
__device__ __forceinline__ float root_of(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);
  const float below = __uint_as_float(__float_as_uint(s) - 1);
  const float above = __uint_as_float(__float_as_uint(s) + 1);
  const float r = __builtin_fmaf(-below, s, x) <= 0.0f ? below : s;
  return __builtin_fmaf(-above, s, x) > 0.0f ? above : r;
}

// AdamW on a lane's four elements: binary64 from the binary32 state, one
// rounding per stored value, in the shard step's order.
template <class TG, bool TAIL>
__device__ __forceinline__ void update32(const Tensor &T, const Consts &k, const Rates &rates,
                                         Lane &s, const Place &i) {
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
  put_weights<TAIL>(T, s.w, i);
  s.m32.template put<TAIL>(T.m_out, i);
  s.v32.template put<TAIL>(T.v_out, i);
}

// The same with a state in 8 bits.  The moments are binary32 numbers, which
// rounding to 4 significant bits makes little of: what the memory leaves time for is some
// 100 instructions an element, and binary64 as above takes more (1034 us for 570 of
// 163.84M elements).  What is stored is the definition's number for number: its root and
// its scale's inverse are rounded (461 us for 449 with the instructions' own, within a
// step, which put one of v's scales in 60 a step off; 467 with a root that takes every
// number everywhere).  u's quotient, which only the weights see, is the instruction's,
// within 2^-22; they are binary64 as above.
template <class TG, bool TAIL>
__device__ __forceinline__ void update8(const Tensor &T, const Rates &rates, uint32_t base,
                                        Lane &s, const Place &i) {
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
    r[e] = (rates.b2 * r0) * r0 + (rates.omb2 * g) * g;
  }
  if (__all(fminf(fminf(r[0], r[1]), fminf(r[2], r[3])) >= 0x1p-96f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = root_of(r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = sqrtf(r[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double t0 = double(s.w.v[e]);
    const float u = m[e] * __builtin_amdgcn_rcpf(r[e] * rates.root + rates.eps);
    s.w.v[e] = float(t0 - rates.decay * t0 - rates.step * double(u));
    // what is not there counts for nothing: its gradient and state are 0
    mtop = larger(mtop, __float_as_uint(m[e]) & 0x7fffffffu);
    vtop = larger(vtop, __float_as_uint(r[e]) & 0x7fffffffu);
  }
  put_weights<TAIL>(T, s.w, i);
  // Scales, and the factors that take magnitudes to [0, 256], m's in the wave's first
  // half, r's in the other.  Blocks of nothing but numbers below 2^-100 are zeros (NaN
  // is not below), so that neither leaves binary32.
  const int lane = threadIdx.x & 63;
  const float held = lane < 32 ? 1.0f : 0x1p-16f;
  const float top = __uint_as_float(wave_tops(mtop, vtop)) * held;
  const bool none = top < 0x1p-100f;
  const float scale = none ? 0.0f : top * 0x1p-8f;
  const float inv = none ? 0.0f : 1.0f / scale * held;
  const float minv = lane_value(inv, 0), vinv = lane_value(inv, 32);
  // to e4m3, down or up where 20 bits of dither carry into the number
  unsigned mw = 0, vw = 0;
  const auto encode = [&](auto place) {
    constexpr int e = place.value;
    const uint32_t h = mix(base + uint32_t(i.from) + i.at + unsigned(e));
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
  if (!TAIL || i.left >= 4) {
    using Word = unsigned __attribute__((aligned(1)));
    __builtin_nontemporal_store(mw, (ZS_GLOBAL Word *)i.of<uint8_t>(T.m_out));
    __builtin_nontemporal_store(vw, (ZS_GLOBAL Word *)i.of<uint8_t>(T.v_out));
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < i.left) {
        *i.of<uint8_t>(T.m_out, e) = uint8_t(mw >> (8 * e));
        *i.of<uint8_t>(T.v_out, e) = uint8_t(vw >> (8 * e));
      }
  }
  const int64_t block = i.from / kBlock + __builtin_amdgcn_readfirstlane(i.at / kBlock);
  if ((lane == 0 || lane == 32) && (!TAIL || block * kBlock < T.n))
    Place{block, 0, 1}.of<float>(lane ? T.v_scale_out : T.m_scale_out)[0] = scale;
}

template <bool EIGHT, class TG, bool TAIL>
__device__ __forceinline__ void step_chunk(const Tensor &T, const void *g, const Consts &k,
                                           const Rates &rates, uint32_t key, int64_t from) {
  const unsigned at = (threadIdx.x >> 6) * (kBlock * kRounds<EIGHT>) + (threadIdx.x & 63) * 4;
  const uint32_t base = mix(key + 0x9e3779b9u * uint32_t(T.number + 1)) +
                        mix(uint32_t(uint64_t(from) >> 32)) * 0x9e3779b9u;
  const auto place = [&](int r) {
    const unsigned i = at + unsigned(r * kBlock);
    return Place{from, i, T.n - from - int64_t(i)};
  };
  Lane s[kRounds<EIGHT>];
#pragma unroll
  for (int r = 0; r < kRounds<EIGHT>; ++r) {
    load_state<EIGHT, TAIL>(T, s[r], place(r));
    load_grad<TG, TAIL>(g, s[r], place(r));
  }
#pragma unroll
  for (int r = 0; r < kRounds<EIGHT>; ++r) {
    if constexpr (EIGHT) update8<TG, TAIL>(T, rates, base, s[r], place(r));
    else update32<TG, TAIL>(T, k, rates, s[r], place(r));
  }
}

template <bool EIGHT, class TG>
__device__ __forceinline__ void step_any(const Tensor &T, const void *g, const Consts &k,
                                         const Rates &rates, uint32_t key, int64_t from) {
  if (T.n - from < kChunk<EIGHT>) step_chunk<EIGHT, TG, true>(T, g, k, rates, key, from);
  else step_chunk<EIGHT, TG, false>(T, g, k, rates, key, from);
}

template <bool EIGHT>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(6)))
    adamw_step_kernel(const StepArgs A, const Grads G) {
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
  if constexpr (EIGHT) {
    rates.coef32 = float(rates.coef);
    rates.b1 = float(k.b1);
    rates.omb1 = float(k.omb1);
    rates.b2 = float(k.b2) * 0x1p32f;
    rates.omb2 = float(k.omb2) * 0x1p32f;
    rates.root = float(k.root) * 0x1p-16f;
    rates.eps = fmaxf(float(k.eps), 0x1p-126f);  // which a quotient by it needs
    rates.step = rates.lr / k.bc1;
  }
  const int64_t from = (chunk - T.chunk0) * kChunk<EIGHT>;
  if (T.grad_dtype == ZS_F32) step_any<EIGHT, F32>(T, g, k, rates, key, from);
  else if (T.grad_dtype == ZS_BF16) step_any<EIGHT, Bf16>(T, g, k, rates, key, from);
  else step_any<EIGHT, F16>(T, g, k, rates, key, from);
}

// A lane's part of the sum of squares (binary64) of elements [from, n): sixteen bytes
// at a time, 64 lanes side by side, up to 16 of them in flight.
template <class TG>
__device__ __forceinline__ double squares(const void *g, int64_t from, int64_t n) {
  using raw = typename TG::raw;
  constexpr int kVec = 16 / sizeof(raw), kLoads = 16;
  using V = unsigned __attribute__((ext_vector_type(4), aligned(sizeof(raw))));
  double sum = 0.0;
  for (int64_t i0 = from + (threadIdx.x & 63) * kVec; i0 < n; i0 += kLoads * 64 * kVec) {
    V v[kLoads];
#pragma unroll
    for (int r = 0; r < kLoads; ++r) {
      const int64_t i = i0 + r * (64 * kVec);
      v[r] = V{0, 0, 0, 0};
      if (i + kVec <= n) {
        v[r] = __builtin_nontemporal_load((const ZS_GLOBAL V *)global<raw>(g, i));
      } else if (i < n) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (i + e < n) {
            if constexpr (sizeof(raw) == 4) v[r][e] = __float_as_uint(*global<raw>(g, i + e));
            else v[r][e / 2] |= unsigned(*global<raw>(g, i + e)) << (e % 2 * 16);
          }
      }
    }
#pragma unroll
    for (int r = 0; r < kLoads; ++r)
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        float x;
        if constexpr (sizeof(raw) == 4) x = __uint_as_float(v[r][e]);
        else x = TG::load(raw(v[r][e / 2] >> (e % 2 * 16)));
        sum += double(x) * double(x);
      }
  }
  return sum;
}

// A wave takes A.each chunks, those of one tensor together (2048 elements at a
// time: 88 us for 56 over 163.84M bf16 gradients); its lanes' sums, a butterfly over them,
// the waves in order.
__global__ void __launch_bounds__(kThreads) adamw_norm_kernel(const NormArgs A, const Grads G) {
  __shared__ double sums[kWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t chunk = (int64_t(blockIdx.x) * kWaves + wave) * A.each;
  const int64_t end = chunk + A.each < A.chunks ? chunk + A.each : A.chunks;
  double sum = 0.0;
  while (chunk < end) {
    const int at = __builtin_amdgcn_readfirstlane(A.map[A.chunk0 + chunk]) - A.tensor0;
    const Tensor &T = A.tensors[at];
    const int64_t length = T.state == ZS_STATE_8 ? kChunk<true> : kChunk<false>;
    const int64_t first = A.chunk0 + chunk - T.chunk0, from = first * length;
    const int64_t most = from + (end - chunk) * length, n = T.n < most ? T.n : most;
    if (T.grad_dtype == ZS_F32) sum += squares<F32>(G.p[at], from, n);
    else if (T.grad_dtype == ZS_BF16) sum += squares<Bf16>(G.p[at], from, n);
    else sum += squares<F16>(G.p[at], from, n);
    chunk += (n - from + length - 1) / length;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) sums[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) sum += sums[w];
    A.partials[blockIdx.x] = sum;
  }
}

// The workgroups' sums, each thread a strided run of them, then a tree.
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
int64_t chunks_of(int64_t n, int32_t state) {
  const int64_t length = state == ZS_STATE_8 ? kChunk<true> : kChunk<false>;
  return (n + length - 1) / length;
}

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
      chunks += chunks_of(t[k].n, t[k].state);
    }
    if (chunks > int64_t(UINT32_MAX) / kThreads) return;  // a launch takes them all
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

// Each kGrads tensors: their first chunk, how many are of 8-bit states (which
// come first among them) and how many of others.
template <class F>
int by_group(const void *plan, const void *const *grads, F f) {
  const Header *h = static_cast<const Header *>(plan);
  const Tensor *t = tensors_of(plan);
  int64_t chunk = 0;
  for (int64_t k = 0; k < h->count; k += kGrads) {
    const int64_t to = k + kGrads < h->count ? k + kGrads : h->count;
    Grads G;
    int64_t chunks[2] = {0, 0};
    for (int64_t j = k; j < to; ++j) {
      G.p[j - k] = grads[j];
      chunks[t[j].state == ZS_STATE_8 ? 0 : 1] += chunks_of(t[j].n, t[j].state);
    }
    if (const int rc = f(k, chunk, chunks[0], chunks[1], G)) return rc;
    chunk += chunks[0] + chunks[1];
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
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  return by_group(plan, grads, [&](int64_t tensor0, int64_t chunk0, int64_t eights, int64_t others,
                                   const Grads &G) {
    StepArgs A{tensors_of(plan_dev) + tensor0,
               reinterpret_cast<const int32_t *>(dev + h->map), chunk0, int32_t(tensor0), key,
               k, dyn, sumsq, double(d->max_norm)};
    if (eights)
      hipLaunchKernelGGL(adamw_step_kernel<true>, dim3(unsigned(eights)), dim3(kThreads), 0, st, A,
                         G);
    A.chunk0 += eights;
    if (others)
      hipLaunchKernelGGL(adamw_step_kernel<false>, dim3(unsigned(others)), dim3(kThreads), 0, st,
                         A, G);
    return launched();
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
  for (int64_t k = 0; k < d->count; k += kGrads) {
    const int64_t to = k + kGrads < d->count ? k + kGrads : d->count;
    for (const int32_t state : {ZS_STATE_8, ZS_STATE_32})  // see by_group
      for (int64_t j = k; j < to; ++j) {
        const zs_adamw_tensor &t = tensors[j];
        if (t.state != state) continue;
        out[j] = Tensor{t.n, chunk, t.master_in, t.master_out, t.m_in, t.v_in, t.m_out, t.v_out,
                        t.m_scale_in, t.v_scale_in, t.m_scale_out, t.v_scale_out, t.param_out,
                        t.weight_decay, t.lr_scale, t.state, t.grad_dtype, t.param_dtype,
                        int32_t(j)};
        for (int64_t c = chunks_of(t.n, state); c > 0; --c) map[chunk++] = int32_t(j);
      }
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
  int64_t sums = 0;
  if (const int rc = by_group(plan, grads, [&](int64_t tensor0, int64_t chunk0, int64_t eights,
                                               int64_t others, const Grads &G) {
        const int64_t chunks = eights + others, each = chunks <= kFewChunks ? 1 : kNormChunks;
        const int64_t blocks = (chunks + kWaves * each - 1) / (kWaves * each);
        if (blocks == 0) return int(ZS_OK);
        const NormArgs A{tensors_of(plan_dev) + tensor0,
                         reinterpret_cast<const int32_t *>(dev + h->map), chunk0, chunks,
                         int32_t(tensor0), int32_t(each), partials + sums};
        hipLaunchKernelGGL(adamw_norm_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, st, A, G);
        sums += blocks;
        return launched();
      }))
    return rc;
  hipLaunchKernelGGL(adamw_total_kernel, dim3(1), dim3(kFinalThreads), 0, st, partials, sums,
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
