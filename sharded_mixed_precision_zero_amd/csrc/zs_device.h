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
};
struct F16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float load(raw v) {
    return static_cast<float>(__builtin_bit_cast(_Float16, v));
  }
  static __device__ __forceinline__ raw store(float v) {
    return __builtin_bit_cast(raw, static_cast<_Float16>(v));
  }
};

// V consecutive elements, aligned to one element: the memory takes 16-byte
// accesses at any address, and rows of odd widths and strides need no path of
// their own.
template <class T, int V>
struct Pack {
  using raw = typename T::raw;
  struct __attribute__((packed, aligned(sizeof(raw)))) Vec {
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
  // The first n < V of them, the others 0.
  static __device__ __forceinline__ void load_some(const void *row, int64_t i, int n,
                                                   float (&out)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      out[e] = e < n ? T::load(static_cast<const raw *>(row)[i + e]) : 0.0f;
  }
  static __device__ __forceinline__ void store_some(void *row, int64_t i, int n,
                                                    const float (&in)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < n) static_cast<raw *>(row)[i + e] = T::store(in[e]);
  }
};

}  // namespace zs_dev

#endif  // ZS_DEVICE_H
