// zero_shard_muon.hip -- the Muon update of a rank's weight matrices on MI355X
// (gfx950): momentum over the averaged contributions, orthogonalisation by
// Newton-Schulz products, weight update (declarations and the contract:
// include/zero_shard.h).
//
// momentum and apply are HBM-bound elementwise passes over a flat range, in
// binary64 with one rounding per stored value, as the shard step's update.
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
// computed and each is stored twice: m^2 n + m^3 + 2 m^2 n multiply-adds a step
// in place of 2 m^2 n + 2 m^3 + 2 m^2 n.
// All of it is laid out padded to whole tiles with zeros, which the iteration
// keeps zero, so the products need no bounds.

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

// ------------------------------------------------- momentum and apply

struct Rows {
  const u32x4 *p[ZS_MAX_ND];
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

// 8 elements per lane: one 16-byte load per contribution row, eight rows in
// flight while the binary64 sum keeps the rank order.
template <class TU>
__global__ void __launch_bounds__(kThreads) momentum_kernel(const MomentumArgs A) {
  const int64_t vec = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t e0 = vec * 8;
  if (e0 >= A.n) return;
  const int nvalid = A.n - e0 < 8 ? int(A.n - e0) : 8;
  double s[8] = {};
  float m[8], g[8], u[8];
  if (nvalid == 8) {
    const f32x4 ma = reinterpret_cast<const f32x4 *>(A.m_in)[2 * vec];
    const f32x4 mb = reinterpret_cast<const f32x4 *>(A.m_in)[2 * vec + 1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = ma[e];
      m[e + 4] = mb[e];
    }
    int k = 0;
    for (; k + 8 <= A.n_d; k += 8) {
      u32x4 r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = __builtin_nontemporal_load(A.rows.p[k + i] + vec);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[2 * e] += double(__uint_as_float(r[i][e] << 16));
          s[2 * e + 1] += double(__uint_as_float(r[i][e] & 0xffff0000u));
        }
    }
    for (; k < A.n_d; ++k) {
      const u32x4 r = __builtin_nontemporal_load(A.rows.p[k] + vec);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * e] += double(__uint_as_float(r[e] << 16));
        s[2 * e + 1] += double(__uint_as_float(r[e] & 0xffff0000u));
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      m[e] = e < nvalid ? A.m_in[e0 + e] : 0.0f;
      if (e < nvalid)
        for (int k = 0; k < A.n_d; ++k)
          s[e] += double(Bf16::load(reinterpret_cast<const uint16_t *>(A.rows.p[k])[e0 + e]));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    g[e] = float(s[e] / double(A.n_d));
    const double mm = A.mu * double(m[e]) + double(g[e]);
    m[e] = float(mm);
    u[e] = A.nesterov ? float(double(g[e]) + A.mu * mm) : float(mm);
  }
  typename TU::raw *up = static_cast<typename TU::raw *>(A.update) + e0;
  if (nvalid == 8) {
    f32x4 *mo = reinterpret_cast<f32x4 *>(A.m_out) + 2 * vec;
    mo[0] = f32x4{m[0], m[1], m[2], m[3]};
    mo[1] = f32x4{m[4], m[5], m[6], m[7]};
    struct alignas(16) Out {
      typename TU::raw e[8];
    } o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.e[e] = TU::store(u[e]);
    *reinterpret_cast<Out *>(up) = o;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nvalid) {
        A.m_out[e0 + e] = m[e];
        up[e] = TU::store(u[e]);
      }
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

__global__ void __launch_bounds__(kThreads) apply_kernel(const ApplyArgs A) {
  const int64_t vec = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t e0 = vec * 8;
  if (e0 >= A.n) return;
  const int nvalid = A.n - e0 < 8 ? int(A.n - e0) : 8;
  float w[8], o[8];
  struct alignas(16) Half {
    uint16_t e[8];
  } p;
  if (nvalid == 8) {
    const f32x4 a = reinterpret_cast<const f32x4 *>(A.in)[2 * vec];
    const f32x4 b = reinterpret_cast<const f32x4 *>(A.in)[2 * vec + 1];
    const Half v = *reinterpret_cast<const Half *>(A.o + e0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = e < 4 ? a[e & 3] : b[e & 3];
      o[e] = Bf16::load(v.e[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = e < nvalid ? A.in[e0 + e] : 0.0f;
      o[e] = e < nvalid ? Bf16::load(A.o[e0 + e]) : 0.0f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double x = double(w[e]);
    w[e] = float((x - A.decay * x) - A.step * double(o[e]));
    p.e[e] = Bf16::store(w[e]);
  }
  if (nvalid == 8) {
    f32x4 *out = reinterpret_cast<f32x4 *>(A.out) + 2 * vec;
    out[0] = f32x4{w[0], w[1], w[2], w[3]};
    out[1] = f32x4{w[4], w[5], w[6], w[7]};
    *reinterpret_cast<Half *>(A.p + e0) = p;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nvalid) {
        A.out[e0 + e] = w[e];
        A.p[e0 + e] = p.e[e];
      }
  }
}

// --------------------------------------------------- ortho: norm and layout

constexpr float kScale = 2048.0f;  // 2^11: X, A and B are held times this
constexpr int kNormBlocks = 256;   // partial sums of squares per matrix
constexpr int kNormRun = 2048;     // consecutive elements a workgroup sums

struct InArgs {
  const void *g;
  int64_t rows, cols, ld, stride;  // of the input, elements
  double *partials;                // [batch][kNormBlocks]
  _Float16 *x, *xt;                // [batch][mp][np] and [batch][np][mp]
  int64_t mp, np;
  double eps;
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

template <class TG>
__global__ void __launch_bounds__(kThreads) ortho_norm_kernel(const InArgs A) {
  __shared__ double lds[kThreads / 64];
  const typename TG::raw *g =
      static_cast<const typename TG::raw *>(A.g) + int64_t(blockIdx.y) * A.stride;
  const int64_t runs = (A.cols + kNormRun - 1) / kNormRun;
  double s = 0.0;
  for (int64_t w = blockIdx.x; w < A.rows * runs; w += kNormBlocks) {
    const int64_t r = w / runs, c0 = (w - r * runs) * kNormRun;
    const int64_t c1 = c0 + kNormRun < A.cols ? c0 + kNormRun : A.cols;
    for (int64_t c = c0 + threadIdx.x; c < c1; c += kThreads) {
      const double v = double(TG::load(g[r * A.ld + c]));
      s = __builtin_fma(v, v, s);
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) A.partials[int64_t(blockIdx.y) * kNormBlocks + blockIdx.x] = s;
}

// 64 x 64 tiles of X and of its transpose, scaled and padded with zeros.
template <class TG>
__global__ void __launch_bounds__(kThreads) ortho_layout_kernel(const InArgs A) {
  __shared__ double lds[kThreads / 64];
  __shared__ _Float16 tile[64][66];
  static_assert(kNormBlocks == kThreads, "one partial per thread");
  const int64_t b = blockIdx.y;
  const double sum = block_sum(A.partials[b * kNormBlocks + threadIdx.x], lds);
  const double scale = double(kScale) / (sqrt(sum) + A.eps);
  const typename TG::raw *g = static_cast<const typename TG::raw *>(A.g) + b * A.stride;
  // the tile in the input's orientation: [r0, r0+64) x [c0, c0+64) of G
  const int64_t rp = A.tall ? A.np : A.mp, cp = A.tall ? A.mp : A.np;
  const int64_t tc = cp / 64;
  const int64_t r0 = int64_t(blockIdx.x) / tc * 64, c0 = int64_t(blockIdx.x) % tc * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  _Float16 *same = (A.tall ? A.xt : A.x) + b * A.mp * A.np;
  _Float16 *turned = (A.tall ? A.x : A.xt) + b * A.mp * A.np;
#pragma unroll 4
  for (int i = wave; i < 64; i += 4) {
    const int64_t r = r0 + i, c = c0 + lane;
    _Float16 v = _Float16(0.0f);
    if (r < A.rows && c < A.cols)
      v = _Float16(float(double(TG::load(g[r * A.ld + c])) * scale));
    tile[i][lane] = v;
    same[r * cp + c] = v;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = wave; i < 64; i += 4) turned[(c0 + i) * rp + r0 + lane] = tile[lane][i];
}

// ------------------------------------------------------- ortho: products

enum Product {
  kGram,  // A = X X^T                  symmetric
  kPoly,  // B = a I + b A + c A A      symmetric
  kNext,  // X = B X, and X^T
  kLast   // O = B X, in the caller's orientation and bf16
};

struct MulArgs {
  const _Float16 *p, *q;      // [batch][rows][k], [batch][cols][k]
  int64_t stride_p, stride_q; // elements per matrix
  int64_t k;
  int32_t tiles_r, tiles_c;   // of C; symmetric products: tiles_r == tiles_c
  int32_t per;                // tiles computed per matrix
  _Float16 *c, *ct;           // C (row length ld_c) and C^T (row length ld_ct)
  int64_t ld_c, ld_ct, stride_c;
  float a, b, cc;             // kPoly's coefficients
  // kLast
  uint16_t *o;
  int64_t rows, cols, ld_o, stride_o;
  int32_t tall;
};

#define ZS_LDS(p) ((__attribute__((address_space(3))) void *)(p))
#define ZS_GLOBAL(p) ((__attribute__((address_space(1))) void *)(p))

// All waves of the workgroup; accesses to memory stay on their side of it.
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// At most N of this wave's loads outstanding.
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

// T x T tiles of C, WR x WC waves, S buffers of BK of k.  The operands go from
// global memory straight into LDS, S - 1 buffers ahead of their use, so a
// buffer costs one barrier; a row of BK is BK / 8 pieces of 16 bytes, piece c
// of row r at position c ^ key(r), so the rows that one read instruction
// serves together lie in different banks.  The registers of the next 32 of k
// are read while the matrix cores work on the present ones.
template <int KIND, int T, int WR, int WC, int BK, int S>
__global__ void __launch_bounds__(WR *WC * 64) ortho_mul_kernel(const MulArgs A) {
  constexpr int NW = WR * WC, TM = T / WR / 16, TN = T / WC / 16;
  constexpr int PIECES = BK / 8, RPI = 64 / PIECES;  // per row; rows per load instruction
  constexpr int L = T / RPI / NW;  // load instructions per wave, operand and buffer
  constexpr int PITCH = T + 8;
  constexpr int BUF = 2 * T * BK, STAGE = S * BUF, EPI = T * PITCH;
  __shared__ __align__(16) _Float16 lds[STAGE > EPI ? STAGE : EPI];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;

  // Workgroups go to the 8 XCDs in turn: each gets a contiguous run of tiles.
  const unsigned total = gridDim.x, id = blockIdx.x, xcd = id & 7;
  const unsigned each = total / 8, more = total % 8;
  const unsigned at = xcd * each + (xcd < more ? xcd : more) + id / 8;
  const int64_t mat = at / unsigned(A.per);
  const int t = int(at % unsigned(A.per));
  int tr, tc;
  if constexpr (KIND == kGram || KIND == kPoly) {
    tr = int((sqrtf(8.0f * float(t) + 1.0f) - 1.0f) * 0.5f);
    while (tr * (tr + 1) / 2 > t) --tr;
    while ((tr + 1) * (tr + 2) / 2 <= t) ++tr;
    tc = t - tr * (tr + 1) / 2;
  } else {
    // bands of 4 tile rows, so that neighbours share both operands in L2
    const int band = t / (4 * A.tiles_c), in = t - band * 4 * A.tiles_c;
    const int rows = A.tiles_r - band * 4 < 4 ? A.tiles_r - band * 4 : 4;
    tr = band * 4 + in % rows;
    tc = in / rows;
  }

  const auto key = [](int r) { return BK == 64 ? r & 7 : (r >> 1) & 3; };
  const unsigned row0 = wave * RPI + lane / PIECES;
  const unsigned off = row0 * unsigned(A.k) + ((lane % PIECES) ^ key(lane / PIECES)) * 8;
  const _Float16 *pg = A.p + mat * A.stride_p + int64_t(tr) * T * A.k;
  const _Float16 *qg = A.q + mat * A.stride_q + int64_t(tc) * T * A.k;
  // The buffers go round: `rd` is read next and `wr_` written next (offsets
  // into lds), `from` is the k that is loaded next; past the end the last
  // buffer is loaded once more, so that as many loads are outstanding in
  // every turn.
  int rd = 0, wr_ = 0;
  int64_t from = 0;
  const auto load = [&](int i) {  // the i-th of a buffer's loads
    const int at = i % L;
    __builtin_amdgcn_global_load_lds(
        ZS_GLOBAL((i < L ? pg : qg) + (from + at * NW * RPI * A.k) + off),
        ZS_LDS(lds + wr_ + (i < L ? 0 : T * BK) + (at * NW + wave) * 512), 16, 0, 0);
    if (i == 2 * L - 1) {
      wr_ = wr_ == (S - 1) * BUF ? 0 : wr_ + BUF;
      from = from + BK < A.k ? from + BK : from;
    }
  };
  // the buffer at rd is there for all waves, and all have read the one before
  const auto advance = [&] {
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<(S - 2) * 2 * L>();
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  half8 regs[2][TM + TN];
  // where this lane's pieces of a buffer's first and second 32 of k are
  int pos[BK / 32][2];
#pragma unroll
  for (int h = 0; h < BK / 32; ++h) {
    const int in = (lane & 15) * BK + ((h * 4 + (lane >> 4)) ^ key(lane & 15)) * 8;
    pos[h][0] = in + wr * TM * 16 * BK;
    pos[h][1] = in + (T + wc * TN * 16) * BK;
  }
  const auto fetch = [&](auto odd, int i) {  // the i-th block of the 32 of k at rd
    constexpr int h = odd.value % (BK / 32);
    const int at = i < TM ? pos[h][0] + i * 16 * BK : pos[h][1] + (i - TM) * 16 * BK;
    regs[odd.value][i] = *reinterpret_cast<const half8 *>(lds + rd + at);
    if (i == TM + TN - 1 && h == BK / 32 - 1) rd = rd == (S - 1) * BUF ? 0 : rd + BUF;
  };
  f32x4 acc[TM][TN] = {};
  // 32 of k, while the next 32 are read and, in the first turn after a
  // barrier, the loads of the buffer that it freed are issued, evenly between
  // the matrix instructions: all loads at once fill the queue that the reads
  // need, and the matrix cores wait.
  const auto turn = [&](auto odd, auto loads) {
    constexpr int G = TM + TN, N = loads.value ? 2 * L : 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int i = g * N / G; i < (g + 1) * N / G; ++i) load(i);
      fetch(Const<1 - odd.value>{}, g);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            regs[odd.value][i], regs[odd.value][TM + j], acc[i][j], 0, 0, 0);
    constexpr int EACH = TM * TN / G > 0 ? TM * TN / G : 1;
    order<0, G, N, EACH>();
  };

  // k is a multiple of 64: two turns of 32 at a time
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
#pragma unroll
    for (int i = 0; i < 2 * L; ++i) load(i);
  advance();
#pragma unroll
  for (int i = 0; i < 2 * L; ++i) load(i);
#pragma unroll
  for (int i = 0; i < TM + TN; ++i) fetch(Const<0>{}, i);
  for (int64_t u = 0; u < A.k; u += 64) {
    if constexpr (BK == 32) advance();
    turn(Const<0>{}, Const<BK == 32>{});
    advance();
    turn(Const<1>{}, Const<1>{});  // reads past the end: of some buffer, not used
  }
  wait_loads<0>();

  // Lane l of a 16 x 16 block holds rows 4 (l / 16) + 0..3 of column l % 16.
  const int br = wr * TM * 16 + (lane >> 4) * 4, bc = wc * TN * 16 + (lane & 15);
  constexpr float kBack = KIND == kLast ? 1.0f / (kScale * kScale) : 1.0f / kScale;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (KIND == kPoly) {
        // A is symmetric: column j's four rows are four neighbours of row j
        const int64_t r = int64_t(tr) * T + br + i * 16, c = int64_t(tc) * T + bc + j * 16;
        const half4 s = *reinterpret_cast<const half4 *>(A.p + mat * A.stride_p + c * A.k + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[i][j][e] = A.b * float(s[e]) + A.cc * (acc[i][j][e] * kBack);
          if (r + e == c) acc[i][j][e] += A.a * kScale;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] *= kBack;
      }
    }

  const auto narrow = [](float v) {
    if constexpr (KIND == kLast) return Bf16::store(v);
    else return F16::store(v);
  };
  uint16_t *epi = reinterpret_cast<uint16_t *>(lds);
  // the tile through LDS, as C (turned = false) or as its transpose
  const auto gather = [&](bool turned) {
    barrier();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = br + i * 16 + e, c = bc + j * 16;
          epi[turned ? c * PITCH + r : r * PITCH + c] = narrow(acc[i][j][e]);
        }
    barrier();
  };
  const auto put = [&](_Float16 *dst, int64_t ld, int64_t r0, int64_t c0) {
    for (int v = threadIdx.x; v < T * T / 8; v += NW * 64) {
      const int r = v / (T / 8), c = v % (T / 8) * 8;
      *reinterpret_cast<u32x4 *>(dst + (r0 + r) * ld + c0 + c) =
          *reinterpret_cast<const u32x4 *>(epi + r * PITCH + c);
    }
  };
  if constexpr (KIND == kLast) {
    gather(A.tall);
    const int64_t r0 = int64_t(A.tall ? tc : tr) * T, c0 = int64_t(A.tall ? tr : tc) * T;
    uint16_t *o = A.o + mat * A.stride_o;
    for (int v = threadIdx.x; v < T * T; v += NW * 64) {
      const int r = v / T, c = v % T;
      if (r0 + r < A.rows && c0 + c < A.cols) o[(r0 + r) * A.ld_o + c0 + c] = epi[r * PITCH + c];
    }
  } else {
    _Float16 *c = A.c + mat * A.stride_c;
    gather(false);
    put(c, A.ld_c, int64_t(tr) * T, int64_t(tc) * T);
    if constexpr (KIND == kNext) {
      gather(true);
      put(A.ct + mat * A.stride_c, A.ld_ct, int64_t(tc) * T, int64_t(tr) * T);
    } else if (tr != tc) {
      gather(true);
      put(c, A.ld_c, int64_t(tc) * T, int64_t(tr) * T);
    }
  }
}

// ------------------------------------------------------------------- host

constexpr float kCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};
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

struct Plan {
  int64_t m, n, mp, np;
  int tile;
  bool tall;
  int64_t partials, x, xt, y, yt, a, b, bytes;  // offsets into the workspace
};

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

Plan plan_of(const zs_ortho_desc &d) {
  Plan p;
  p.tall = d.rows > d.cols;
  p.m = p.tall ? d.cols : d.rows;
  p.n = p.tall ? d.rows : d.cols;
  const auto tiles = [&](int64_t t) { return d.batch * (up(p.m, t) / t) * (up(p.n, t) / t); };
  p.tile = tiles(256) >= 192 ? 256 : tiles(128) >= 192 ? 128 : 64;
  p.mp = up(p.m, p.tile);
  p.np = up(p.n, p.tile);
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t was = at;
    at += up(bytes, 256);
    return was;
  };
  p.partials = take(d.batch * kNormBlocks * 8);
  p.x = take(d.batch * p.mp * p.np * 2);
  p.xt = take(d.batch * p.mp * p.np * 2);
  p.y = take(d.batch * p.mp * p.np * 2);
  p.yt = take(d.batch * p.mp * p.np * 2);
  p.a = take(d.batch * p.mp * p.mp * 2);
  p.b = take(d.batch * p.mp * p.mp * 2);
  p.bytes = at;
  return p;
}

template <int KIND>
int multiply(const MulArgs &A, int64_t batch, int tile, hipStream_t st) {
  const dim3 grid(unsigned(batch * A.per));
  switch (tile) {
    case 256:
      hipLaunchKernelGGL((ortho_mul_kernel<KIND, 256, 2, 4, 64, 2>), grid, dim3(512), 0, st, A);
      break;
    case 128:
      hipLaunchKernelGGL((ortho_mul_kernel<KIND, 128, 2, 4, 64, 5>), grid, dim3(512), 0, st, A);
      break;
    default:
      hipLaunchKernelGGL((ortho_mul_kernel<KIND, 64, 2, 2, 64, 5>), grid, dim3(256), 0, st, A);
      break;
  }
  return launched();
}

template <class TG>
int start(const InArgs &A, int64_t batch, hipStream_t st) {
  hipLaunchKernelGGL(ortho_norm_kernel<TG>, dim3(kNormBlocks, unsigned(batch)), dim3(kThreads), 0,
                     st, A);
  hipLaunchKernelGGL(ortho_layout_kernel<TG>, dim3(unsigned(A.mp / 64 * (A.np / 64)),
                     unsigned(batch)), dim3(kThreads), 0, st, A);
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
    A.rows.p[k] = reinterpret_cast<const u32x4 *>(contrib[k]);
  }
  if (!aligned(m_in, 16) || !aligned(m_out, 16) || !aligned(update, 16)) return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  A.n = d->n;
  A.n_d = d->n_d;
  A.nesterov = d->nesterov;
  A.mu = double(d->mu);
  A.m_in = m_in;
  A.m_out = m_out;
  A.update = update;
  const dim3 grid(unsigned((d->n + kThreads * 8 - 1) / (kThreads * 8)));
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  if (d->dtype == ZS_F32)
    hipLaunchKernelGGL(momentum_kernel<F32>, grid, dim3(kThreads), 0, st, A);
  else
    hipLaunchKernelGGL(momentum_kernel<Bf16>, grid, dim3(kThreads), 0, st, A);
  return launched();
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
  const ApplyArgs A{d->n, o, master_in, master_out, param_out,
                    double(lr) * double(d->weight_decay), double(lr) * double(scale)};
  hipLaunchKernelGGL(apply_kernel, dim3(unsigned((d->n + kThreads * 8 - 1) / (kThreads * 8))),
                     dim3(kThreads), 0, static_cast<hipStream_t>(d->stream), A);
  return launched();
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
  if (!g || !o || !workspace || workspace_bytes < p.bytes) return ZS_EINVAL;
  if (p.mp / 64 * (p.np / 64) > 0x7fffffff ||
      d->batch * (p.mp / p.tile) * (p.np / p.tile) > 0x7fffffff)
    return ZS_EINVAL;
  if (!aligned(g, dtype_size(d->dtype)) || !aligned(o, 2) || !aligned(workspace, 256))
    return ZS_EALIGN;
  if (const int rc = device_is_gfx950()) return rc;
  const hipStream_t st = static_cast<hipStream_t>(d->stream);
  char *ws = static_cast<char *>(workspace);
  const auto half = [&](int64_t off) { return reinterpret_cast<_Float16 *>(ws + off); };
  const int64_t ld_in = d->ld_in ? d->ld_in : d->cols, ld_out = d->ld_out ? d->ld_out : d->cols;
  InArgs in;
  std::memset(&in, 0, sizeof in);
  in.g = g;
  in.rows = d->rows;
  in.cols = d->cols;
  in.ld = ld_in;
  in.stride = d->stride_in ? d->stride_in : d->rows * ld_in;
  in.partials = reinterpret_cast<double *>(ws + p.partials);
  in.x = half(p.x);
  in.xt = half(p.xt);
  in.mp = p.mp;
  in.np = p.np;
  in.eps = double(d->eps);
  in.tall = p.tall;
  int rc = d->dtype == ZS_F32    ? start<F32>(in, d->batch, st)
           : d->dtype == ZS_BF16 ? start<Bf16>(in, d->batch, st)
                                 : start<F16>(in, d->batch, st);
  const int tm = int(p.mp / p.tile), tn = int(p.np / p.tile);
  _Float16 *x = half(p.x), *xt = half(p.xt), *y = half(p.y), *yt = half(p.yt);
  for (int s = 0; s < d->steps && !rc; ++s) {
    const float *k = d->coeffs ? d->coeffs + 3 * s : kCoeffs;
    MulArgs A;
    std::memset(&A, 0, sizeof A);
    A.p = A.q = x;
    A.stride_p = A.stride_q = p.mp * p.np;
    A.k = p.np;
    A.tiles_r = A.tiles_c = tm;
    A.per = tm * (tm + 1) / 2;
    A.c = half(p.a);
    A.ld_c = p.mp;
    A.stride_c = p.mp * p.mp;
    if ((rc = multiply<kGram>(A, d->batch, p.tile, st))) break;
    A.p = A.q = half(p.a);
    A.stride_p = A.stride_q = p.mp * p.mp;
    A.k = p.mp;
    A.c = half(p.b);
    A.a = k[0];
    A.b = k[1];
    A.cc = k[2];
    if ((rc = multiply<kPoly>(A, d->batch, p.tile, st))) break;
    A.p = half(p.b);
    A.q = xt;
    A.stride_q = p.mp * p.np;
    A.tiles_c = tn;
    A.per = tm * tn;
    if (s + 1 < d->steps) {
      A.c = y;
      A.ct = yt;
      A.ld_c = p.np;
      A.ld_ct = p.mp;
      A.stride_c = p.mp * p.np;
      rc = multiply<kNext>(A, d->batch, p.tile, st);
      _Float16 *v = x;
      x = y;
      y = v;
      v = xt;
      xt = yt;
      yt = v;
    } else {
      A.o = o;
      A.rows = d->rows;
      A.cols = d->cols;
      A.ld_o = ld_out;
      A.stride_o = d->stride_out ? d->stride_out : d->rows * ld_out;
      A.tall = p.tall;
      rc = multiply<kLast>(A, d->batch, p.tile, st);
    }
  }
  return rc;
}

}  // extern "C"
