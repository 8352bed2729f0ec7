// zs_rows.h -- what the kernels that keep whole rows in registers share: sums
// over a row's threads, the statistics of a row, a thread's columns (internal;
// the contract is in include/zero_shard.h).
#ifndef ZS_ROWS_H
#define ZS_ROWS_H

#include "zs_device.h"

namespace zs_dev {

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

// The last 8 - skip (1 to 7) of the eight elements i.. of a row: four, two and one of them
// that end where they do, in words of two elements or of one of 32 bits.
template <class T>
__device__ __forceinline__ void store_last(Eight<T> v, void *row, unsigned i, int skip) {
  v.forget();  // registers, which a choice among them is not to index
  using raw = typename T::raw;
  constexpr bool kFull = sizeof(raw) == 4;
  struct __attribute__((packed, aligned(sizeof(raw)))) Word {
    unsigned w;
  };
  raw *p = reinterpret_cast<raw *>(static_cast<char *>(row) + i * unsigned(sizeof(raw)));
  const auto word = [&](int at, unsigned w) { reinterpret_cast<Word *>(p + at)->w = w; };
  const int count = 8 - skip;
  if (count & 4) {
    if constexpr (kFull) {
#pragma unroll
      for (int e = 4; e < 8; ++e) word(e, v.w[e]);
    } else {
      word(4, v.w[2]);
      word(6, v.w[3]);
    }
  }
  if (count & 2) {
    const bool low = count & 4;
    if constexpr (kFull) {
      word(low ? 2 : 6, low ? v.w[2] : v.w[6]);
      word(low ? 3 : 7, low ? v.w[3] : v.w[7]);
    } else {
      word(low ? 2 : 6, low ? v.w[1] : v.w[3]);
    }
  }
  if (count & 1) {  // the first of them, an odd one
    constexpr int kOdd = kFull ? 2 : 1, kFrom = kFull ? 1 : 0;  // where odd elements are
    const unsigned low = skip & 2 ? v.w[kFrom + kOdd] : v.w[kFrom];
    const unsigned high = skip & 2 ? v.w[kFrom + 3 * kOdd] : v.w[kFrom + 2 * kOdd];
    const unsigned w = skip & 4 ? high : low;
    if constexpr (kFull) word(skip, w);
    else p[skip] = raw(w >> 16);
  }
}

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

// Every row of p starts on a 16-byte boundary (or p is absent).
inline bool rows_even(const void *p, int64_t ld, int size) {
  return !p || (aligned(p, 16) && ld * size % 16 == 0);
}

inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace zs_dev

#endif  // ZS_ROWS_H
