// zs_device.h -- device and launch helpers shared by the layer-norm and Muon
// kernels (internal; the contract is in include/zero_shard.h).
#ifndef ZS_DEVICE_H
#define ZS_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>

#include "zero_shard.h"

namespace zs_dev {

using u32x4 = unsigned int __attribute__((ext_vector_type(4)));
using u32x2 = unsigned int __attribute__((ext_vector_type(2)));
using f32x4 = float __attribute__((ext_vector_type(4)));

inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline int launched() { return hipGetLastError() == hipSuccess ? ZS_OK : ZS_EHIP; }

// The current device is a gfx950 (checked once per device, then cached).
inline int device_is_gfx950() {
  static std::mutex mu;
  static int state[64] = {0};  // 0 unknown, 1 gfx950, -1 other
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return ZS_EDEVICE;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 64 && state[dev]) return state[dev] > 0 ? ZS_OK : ZS_EDEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return ZS_EHIP;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < 64) state[dev] = ok ? 1 : -1;
  return ok ? ZS_OK : ZS_EDEVICE;
}

inline int dtype_size(int32_t t) { return t == ZS_F32 ? 4 : t == ZS_BF16 || t == ZS_F16 ? 2 : 0; }

// Element types in memory, and their binary32 value.  A store rounds to
// nearest even.
struct F32 {
  using raw = float;
  static __device__ __forceinline__ float load(raw v) { return v; }
  static __device__ __forceinline__ raw store(float v) { return v; }
};
struct Bf16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float load(raw v) { return __uint_as_float(unsigned(v) << 16); }
  static __device__ __forceinline__ raw store(float v) {
    return __builtin_bit_cast(raw, static_cast<__bf16>(v));
  }
  static __device__ __forceinline__ unsigned store2(float lo, float hi) {  // one instruction
    using Two = float __attribute__((ext_vector_type(2)));
    using Out = __bf16 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, __builtin_convertvector((Two{lo, hi}), Out));
  }
};
struct F16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float load(raw v) {
    return static_cast<float>(__builtin_bit_cast(_Float16, v));
  }
  static __device__ __forceinline__ raw store(float v) {
    return __builtin_bit_cast(raw, static_cast<_Float16>(v));
  }
  static __device__ __forceinline__ unsigned store2(float lo, float hi) {
    return unsigned(store(lo)) | unsigned(store(hi)) << 16;
  }
};

// Eight consecutive elements as they lie in memory, aligned to one element:
// the memory takes 16-byte accesses at any address, and rows of odd widths and
// strides need no path of their own.
template <class T>
struct Eight {
  using raw = typename T::raw;
  static constexpr int kWords = int(sizeof(raw)) * 2;
  struct __attribute__((packed, aligned(sizeof(raw)))) Words {
    unsigned w[kWords];
  };
  using Four = unsigned __attribute__((ext_vector_type(4), aligned(sizeof(raw))));
  unsigned w[kWords];

  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(raw) == 4) return T::load(__uint_as_float(w[e]));
    else return T::load(raw(w[e / 2] >> (e % 2 * 16)));
  }
  __device__ __forceinline__ void get(float (&out)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = get(e);
  }
  __device__ __forceinline__ void set(const float (&in)[8]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(raw) == 4) w[i] = __float_as_uint(in[i]);
      else w[i] = T::store2(in[2 * i], in[2 * i + 1]);
    }
  }
  // Values taken from here on are converted anew, not kept in registers.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
  }
  // Elements i.. of a row, the first `left` of them (8 or more: all), others
  // 0.  TAIL: `left` may also be between 0 and 8.  A 32-bit index (of a row
  // below 2^32 bytes) is added to the row's address by the access itself.
  // ONCE: no cache need keep it.
  template <bool TAIL = true, bool ONCE = false, class I, class L>
  __device__ __forceinline__ void load(const void *row, I i, L left) {
    const raw *p =
        reinterpret_cast<const raw *>(static_cast<const char *>(row) + I(i * I(sizeof(raw))));
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
    if (left >= 8) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const Four *from = reinterpret_cast<const Four *>(p) + k / 4;
        const Four v = ONCE ? __builtin_nontemporal_load(from) : *from;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k + q] = v[q];
      }
    } else if (TAIL && left > 0) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < left) {
          if constexpr (sizeof(raw) == 4) w[e] = __float_as_uint(p[e]);
          else w[e / 2] |= unsigned(p[e]) << (e % 2 * 16);
        }
    }
  }
  template <bool TAIL = true, bool ONCE = false, class I, class L>
  __device__ __forceinline__ void store(void *row, I i, L left) const {
    raw *p = reinterpret_cast<raw *>(static_cast<char *>(row) + I(i * I(sizeof(raw))));
    if (left >= 8) {
      if constexpr (ONCE) {
#pragma unroll
        for (int k = 0; k < kWords; k += 4)
          __builtin_nontemporal_store(Four{w[k], w[k + 1], w[k + 2], w[k + 3]},
                                      reinterpret_cast<Four *>(p) + k / 4);
        return;
      }
      Words v;
#pragma unroll
      for (int k = 0; k < kWords; ++k) v.w[k] = w[k];
      *reinterpret_cast<Words *>(p) = v;
    } else if (TAIL && left > 0) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < left) {
          if constexpr (sizeof(raw) == 4) p[e] = __uint_as_float(w[e]);
          else p[e] = raw(w[e / 2] >> (e % 2 * 16));
        }
    }
  }
};

}  // namespace zs_dev

#endif  // ZS_DEVICE_H
