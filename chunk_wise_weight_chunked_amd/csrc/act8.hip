// act8.hip -- activations kept in 8 bits, and the weight gradient from them.
//
//   code = round(x 2^-e), x8 = code 2^e,   grad (+)= x8^T dy
//
// with one e for 32 values of a row: the smallest for which all codes are within
// +-127, between -126 and 121 (127 2^121 is the largest that fp32 has; codes beside it end at
// +-127).  A power of two as the scale makes the codes exact (no division), and x8
// exact in bf16 (7 bits and a sign), so that the weight gradient's products on
// the bf16 matrix cores are exact before they are added in fp32.
//
// The codes of 32768 x 2560 bf16 values take 48 us (5.2 TB/s: bound by HBM; 38 us again and again
// on the same 254 MB, which the last-level cache holds).  The gradient of
// 32768 x 2560 x 7680 takes 1092 us: 57 for x's blocks, 11 for the slices' sums, the rest the
// product at 1.25 PFLOP/s, with the matrix pipe at work in 64% of the cycles at the clock that
// the power leaves.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "piece.h"
#include "seq.h"

namespace ttt {
namespace {

constexpr int kBlock = 256;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// exps of a group from the bits of its largest |x| (NaN above infinity above all
// others): e + 127; 255 where it is not finite.  top = (1 + m) 2^(k) is
// above 127 2^(k-6) where m is above 127/64 - 1.
__device__ __forceinline__ uint32_t group_exp(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int k = (int)(top >> 23) - 127;
  const int e = k - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)(min(max(e, -126), 121) + 127);
}

// LPR lanes walk a row, 8 values each at a time; four neighbouring lanes make a
// group of 32.
template <typename T, int LPR>
__global__ __launch_bounds__(kBlock) void act8_store_kernel(const T* __restrict__ x,
                                                            int8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ exps,
                                                            int64_t rows, int64_t d, int64_t xs) {
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * (kBlock / LPR) + threadIdx.x / LPR;
  if (row >= rows) return;  // the lanes of a group leave together
  const int pieces = (int)(d >> 3), groups = (pieces + 3) >> 2;
  for (int c0 = 0; c0 < pieces; c0 += LPR) {
    const int c = c0 + lane;
    Piece<T> p;
    p.zero();
    if (c < pieces) p.load(x + row * xs + 8 * c);
    float f[8];
    p.get(f);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, abs_bits(f[j]));
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    if (c >= pieces) continue;
    const uint32_t e = group_exp(top);
    const float up = e == 255 ? 0.0f : __uint_as_float((254u - e) << 23);  // 2^-e
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int q = e == 255 ? 0 : __float2int_rn(__builtin_amdgcn_fmed3f(f[j] * up, -127.0f, 127.0f));
      w[j >> 2] |= ((uint32_t)q & 0xffu) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(codes + row * d + 8 * c) = make_uint2(w[0], w[1]);
    if ((c & 3) == 0) exps[row * groups + (c >> 2)] = (uint8_t)e;
  }
}

// 8 codes of a group as values; exps = 255 makes every one NaN (its codes are 0, its
// scale infinite).
__device__ __forceinline__ void decode8(uint2 w, uint32_t e, float f[8]) {
  const float scale = __uint_as_float(e << 23);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int32_t q = (int32_t)((j < 4 ? w.x : w.y) << (24 - 8 * (j & 3))) >> 24;
    f[j] = (float)q * scale;
  }
}

template <typename T, int LPR>
__global__ __launch_bounds__(kBlock) void act8_load_kernel(const int8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ exps,
                                                           T* __restrict__ x, int64_t rows,
                                                           int64_t d, int64_t xs) {
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * (kBlock / LPR) + threadIdx.x / LPR;
  if (row >= rows) return;
  const int pieces = (int)(d >> 3), groups = (pieces + 3) >> 2;
#pragma unroll 4
  for (int c = lane; c < pieces; c += LPR) {
    float f[8];
    decode8(*reinterpret_cast<const uint2*>(codes + row * d + 8 * c),
            exps[row * groups + (c >> 2)], f);
    Piece<T>::store(x + row * xs + 8 * c, f);
  }
}

// ------------------------------------------------------------ weight gradient
// Operands for the matrix product come token-major in blocks of 64 tokens, [block][column]
// [64 tokens] bf16 (128-byte rows: a k-tile of the mainloop), zeros behind the last token.
constexpr int kTokens = kRowBytes / 2;

// A lane takes kCols columns (c0 ..) of 8 tokens (t0 ..), of which `live` are there.  The 8
// lanes that share columns are neighbours, so that they write whole 128-byte rows.
template <int kCols>
struct BlockLane {
  int64_t t0, c0, at;  // at: place of the first column's 8 tokens
  int live;
  bool any;
  __device__ __forceinline__ BlockLane(int64_t columns, int64_t rows, int64_t n) {
    const int oct = threadIdx.x & 7;
    c0 = columns * (32 * kCols) + kCols * (threadIdx.x >> 3);
    t0 = blockIdx.x * (int64_t)kTokens + 8 * oct;
    at = (blockIdx.x * n + c0) * kTokens + 8 * oct;
    live = (int)max<int64_t>(0, min<int64_t>(8, rows - t0));
    any = c0 < n;
  }
};

constexpr int kXColumns = 256;
// kXColumns columns of x, out [..][d].
__device__ __forceinline__ void decode_block(const int8_t* __restrict__ codes,
                                             const uint8_t* __restrict__ exps,
                                             uint16_t* __restrict__ out, int64_t rows, int64_t d,
                                             int64_t columns) {
  constexpr int kCols = kXColumns / 32;
  const BlockLane<kCols> l(columns, rows, d);
  if (!l.any) return;
  const int64_t groups = (d + kAct8Group - 1) / kAct8Group;
  uint2 w[8];
  uint32_t e[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    w[t] = make_uint2(0, 0), e[t] = 0;
    if (t < l.live) {
      w[t] = *reinterpret_cast<const uint2*>(codes + (l.t0 + t) * d + l.c0);
      e[t] = exps[(l.t0 + t) * groups + l.c0 / kAct8Group];
    }
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    float v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
      v[t] = (float)((int32_t)((c < 4 ? w[t].x : w[t].y) << (24 - 8 * (c & 3))) >> 24) *
             __uint_as_float(e[t] << 23);
    Piece<uint16_t>::store(out + l.at + c * kTokens, v);
  }
}

// 128 columns of an fp32 dy as three bf16 terms whose sum it is: the leading 8 bits of
// what is left, three times (multiples of 2^-133, bf16's smallest, towards 0); an infinity
// or NaN goes into the first alone.  Terms `part` values apart.
__device__ __forceinline__ void split_block(const float* __restrict__ dy, int64_t dys,
                                            uint16_t* __restrict__ out, int64_t part, int64_t rows,
                                            int64_t n, int64_t columns) {
  const BlockLane<4> l(columns, rows, n);
  if (!l.any) return;
  float v[8][4];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    float4 f = make_float4(0, 0, 0, 0);
    if (t < l.live) f = *reinterpret_cast<const float4*>(dy + (l.t0 + t) * dys + l.c0);
    v[t][0] = f.x, v[t][1] = f.y, v[t][2] = f.z, v[t][3] = f.w;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t top[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const uint32_t u = __float_as_uint(v[t][c]), m = u & 0x7fffffffu;
        // a NaN whose upper bits are an infinity's stays one
        top[t] = m > 0x7f800000u ? 0x7fc00000u : u & 0xffff0000u;
        v[t][c] = m >= 0x7f800000u ? 0.0f : v[t][c] - __uint_as_float(top[t]);
      }
      *reinterpret_cast<uint4*>(out + k * part + l.at + c * kTokens) =
          make_uint4(top[0] >> 16 | top[1], top[2] >> 16 | top[3], top[4] >> 16 | top[5],
                     top[6] >> 16 | top[7]);
    }
}

// Blocks of x (the first x_columns of the grid's rows), and with dy of its terms.
__global__ __launch_bounds__(kBlock) void act8_operands_kernel(
    const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps, uint16_t* __restrict__ x,
    int64_t rows, int64_t d, unsigned x_columns, const float* __restrict__ dy, int64_t dys,
    uint16_t* __restrict__ terms, int64_t part, int64_t n) {
  if (blockIdx.y < x_columns)
    decode_block(codes, exps, x, rows, d, blockIdx.y);
  else
    split_block(dy, dys, terms, part, rows, n, blockIdx.y - x_columns);
}

// Tiles of the gradient: a workgroup a CU, or two with a quarter of it each.  For dy's terms a
// quarter, in whose stages the three terms' k-tiles lie side by side, so that x's are loaded
// once for the three and a stage has three times the products: with two stages, one workgroup a
// CU, or where there are more tiles than CUs with one stage, two workgroups that cover each
// other's loads and results.  us, one term after the other in two workgroups a CU / side by
// side in two stages / in one: 1554 x 1024 x 1536 36 / 32 / 35, 136 x 200 x 2560 17 / 13 / 14,
// 8192 x 2560 x 2560 349 / 317 / 302, 3000 x 2560 x 2560 137 / 132 / 115, 199 x 4096 x 1536 26 /
// 28 / 23; where the operands come from memory wide tiles are faster, 32768 x 2560 x 7680 3574
// and 4060.
using WideTile = TileShape<256, 256, 2, 4>;
using SmallTile = TileShape<128, 128, 2, 2>;
using TermTile = TileShape<128, 128, 2, 4>;

// k-tiles [k0, k0 + n) of an operand, kParts times: of x again and again, of dy's terms
// one after the other (part_stride bytes between them; wide tiles, of whose stages three terms
// would not fit LDS).
template <class Base, int kParts>
struct PartLoader {
  static constexpr int kPer = Base::kPer;
  Base l;
  int64_t n, part_stride;
  __device__ __forceinline__ rsrc_t rsrc(int64_t kt, bool live = true) const {
    if constexpr (kParts == 1) {
      return l.rsrc(kt, live);
    } else {
      const int64_t part = kt / n;
      Base at = l;
      at.base += part * part_stride;
      return at.rsrc(kt - part * n, live);
    }
  }
  __device__ __forceinline__ void issue_one(rsrc_t r, lds_char* stage, int q) const {
    l.issue_one(r, stage, q);
  }
  __device__ __forceinline__ void issue(int64_t kt, lds_char* stage) {
    const rsrc_t r = rsrc(kt);
#pragma unroll
    for (int q = 0; q < kPer; ++q) l.issue_one(r, stage, q);
  }
};
// k-tiles of dy's three terms, side by side in a stage.
template <class S>
struct TermLoader {
  using Base = DirectLoader<S::BN, S::kWaves>;
  static constexpr int kPer = 3 * Base::kPer;
  static constexpr int kBytes = S::BN * kRowBytes;
  Base l;
  int64_t part_stride;
  struct Rsrc {
    rsrc_t term[3];
  };
  __device__ __forceinline__ Rsrc rsrc(int64_t kt, bool live = true) const {
    Rsrc r;
    Base at = l;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      r.term[t] = at.rsrc(kt, live);
      at.base += part_stride;
    }
    return r;
  }
  __device__ __forceinline__ void issue_one(const Rsrc& r, lds_char* stage, int q) const {
    l.issue_one(r.term[q / Base::kPer], stage + q / Base::kPer * kBytes, q % Base::kPer);
  }
  __device__ __forceinline__ void issue(int64_t kt, lds_char* stage) {
    const Rsrc r = rsrc(kt);
#pragma unroll
    for (int q = 0; q < kPer; ++q) issue_one(r, stage, q);
  }
};
// kCols columns from n0 of an operand of N columns in blocks, k-tiles from k0.
template <class S, int kCols>
__device__ __forceinline__ DirectLoader<kCols, S::kWaves> block_loader(const uint16_t* p, int64_t N,
                                                                       int64_t n0, int64_t k0) {
  DirectLoader<kCols, S::kWaves> l;
  l.init(p + (k0 * N + n0) * kTokens, kRowBytes, N * kRowBytes, (N - n0) * kRowBytes, 0);
  return l;
}
// S::BN columns from n0 of rows [rows][ld] of N columns: stage row 64 (c / 64) + t holds
// token t of the k-tile, columns 64 (c / 64) .. (KMajorLoader of gemm_core.h, for any
// number of columns).
template <class S>
struct RowLoader {
  static constexpr int kPer = S::BN / S::kWaves / 8;
  const char* base;
  int64_t kt_stride, valid_bytes;
  uint32_t voff[kPer];
  uint32_t lds_row0;
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int64_t rows, int64_t N,
                                       int64_t n0, int64_t k0) {
    base = reinterpret_cast<const char*>(p + k0 * kTokens * ld + n0);
    kt_stride = kTokens * ld * 2;
    valid_bytes = ((rows - k0 * kTokens - 1) * ld + N - n0) * 2;
    const int lane = threadIdx.x & 63;
    lds_row0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (S::BN / S::kWaves);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int row = (int)lds_row0 + 8 * q + (lane >> 3);
      const int c = (lane & 7) ^ lds_swz_tr(row);
      voff[q] = (uint32_t)((row / kTokens) * kRowBytes + (row % kTokens) * ld * 2 + c * 16);
    }
  }
  __device__ __forceinline__ rsrc_t rsrc(int64_t kt, bool live = true) const {
    return make_rsrc(base + kt * kt_stride, live ? valid_bytes - kt * kt_stride : 0);
  }
  __device__ __forceinline__ void issue_one(rsrc_t r, lds_char* stage, int q) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(stage + (lds_row0 + 8 * q) * kRowBytes), 16,
        voff[q], 0, 0, 0);
  }
};

// A k-tile's products with x's fragments read as rows and dy's transposed from token rows
// (kRows), or both as rows.  Reads for the next 16 tokens are spread between the matrix
// instructions, hook(q) follows instruction q.  The transposing reads are inline assembly,
// each block with its wait: the compiler lets the builtin wait for every direct-to-LDS load
// in flight, also those into the other stage (2560 x 7680 at 32K tokens: 1438 us with it,
// 1118 without).
template <class S, bool kRows>
struct GradMma {
  using Plain = Mma16<S, false, false>;
  static constexpr int kSteps = Plain::kSteps;
  // A lane's addresses in a stage's first 16 token rows: [columns 32 apart][tokens 4 apart]
  // (see read_a_tr in gemm_core.h: a step of 16 tokens adds 16 rows, and only that).
  uint32_t at[2][2];
  __device__ __forceinline__ void init(const LanePos& p) {
    if constexpr (kRows) {
      const int g = p.lane >> 4, j = p.lane & 15;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = p.wave_n0 + 32 * f + 16 * (g & 1) + 4 * (j & 3);
          const int R = (m >> 6) * 64 + 8 * (g >> 1) + (j >> 2) + 4 * h;
          at[f][h] = (uint32_t)R * kRowBytes +
                     (uint32_t)((((m & 63) >> 3) ^ lds_swz_tr(R)) << 4) + (uint32_t)((m & 7) * 2);
        }
    }
  }
  __device__ __forceinline__ void read_rows(bf16x8_t (&b)[2], const lds_char* sB, int s) const {
    const uint32_t base = (uint32_t)(uintptr_t)sB + (uint32_t)(16 * s * kRowBytes);
    u32x2_t x[4];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n\t"
        "ds_read_b64_tr_b16 %1, %5\n\t"
        "ds_read_b64_tr_b16 %2, %6\n\t"
        "ds_read_b64_tr_b16 %3, %7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
        : "v"(base + at[0][0]), "v"(base + at[0][1]), "v"(base + at[1][0]), "v"(base + at[1][1])
        : "memory");
    b[0] = __builtin_bit_cast(bf16x8_t, u32x4_t{x[0][0], x[0][1], x[1][0], x[1][1]});
    b[1] = __builtin_bit_cast(bf16x8_t, u32x4_t{x[2][0], x[2][1], x[3][0], x[3][1]});
  }
  template <class Hook>
  __device__ __forceinline__ void ktile(Accum<S>& acc, const lds_char* sA, const lds_char* sB,
                                        const LanePos& p, Hook&& hook) const {
    if constexpr (!kRows) {
      Plain::ktile_spread(acc, sA, sB, p, hook);
    } else {
      static_assert(S::NB == 2, "the reads below");
      constexpr int kPerStep = 2 * S::MB;
      bf16x8_t a[2][S::MB], b[2][2];
#pragma unroll
      for (int i = 0; i < S::MB; ++i) a[0][i] = Plain::read_a(sA, p, i, 0);
      read_rows(b[0], sB, 0);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < kPerStep; ++m) {
          const int i = m >> 1, j = m & 1;
          acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[s & 1][i], b[s & 1][j],
                                                                acc.v[i][j], 0, 0, 0);
          if (s + 1 < kSteps) {
            if (m < S::MB) a[(s + 1) & 1][m] = Plain::read_a(sA, p, m, s + 1);
            if (m == kPerStep - S::MB + S::MB / 4) read_rows(b[(s + 1) & 1], sB, s + 1);
          }
          hook(kPerStep * s + m);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
};

// A k-tile's products of x with dy's three terms side by side: x's fragments are read once
// for the three.
template <class S>
struct TermMma {
  using Plain = Mma16<S, false, false>;
  static constexpr int kSteps = Plain::kSteps;
  static constexpr int kEach = S::MB * S::NB, kPerStep = 3 * kEach;
  static constexpr int kReads = S::MB + 3 * S::NB;
  static_assert(kReads <= kPerStep, "a read after each matrix instruction at most");
  __device__ __forceinline__ void init(const LanePos&) {}
  struct Frag {
    bf16x8_t a[S::MB], b[3][S::NB];
    __device__ __forceinline__ void read(const lds_char* sA, const lds_char* sB, const LanePos& p,
                                         int s, int m) {
      if (m < S::MB)
        a[m] = Plain::read_a(sA, p, m, s);
      else
        b[(m - S::MB) / S::NB][(m - S::MB) % S::NB] = Plain::read_b(
            sB + (m - S::MB) / S::NB * (S::BN * kRowBytes), p, (m - S::MB) % S::NB, s);
    }
  };
  template <class Hook>
  __device__ __forceinline__ void ktile(Accum<S>& acc, const lds_char* sA, const lds_char* sB,
                                        const LanePos& p, Hook&& hook) const {
    Frag f[2];
#pragma unroll
    for (int m = 0; m < kReads; ++m) f[0].read(sA, sB, p, 0, m);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < kPerStep; ++m) {
        const int t = m / kEach, i = m % kEach / S::NB, j = m % S::NB;
        acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[s & 1].a[i], f[s & 1].b[t][j],
                                                              acc.v[i][j], 0, 0, 0);
        if (s + 1 < kSteps && m < kReads) f[(s + 1) & 1].read(sA, sB, p, s + 1, m);
        hook(kPerStep * s + m);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
};

// The mainloop of gemm_core.h on these fragments: k-tile kt + 1's loads one after each of
// kt's first matrix instructions.  In one stage a k-tile's loads, then its products.
template <class Mma, int kStages, int kStageBytes, class S, class LA, class LB>
__device__ __forceinline__ void grad_mainloop(Accum<S>& acc, LA& la, LB& lb, int64_t nk,
                                              lds_char* smem, const LanePos& p) {
  constexpr int kLoads = LA::kPer + LB::kPer;
  static_assert(kLoads <= Mma::kSteps * S::MB * S::NB, "the loads fit the k-tile's MFMAs");
  Mma mma;
  mma.init(p);
  if constexpr (kStages == 1) {
    for (int64_t kt = 0; kt < nk; ++kt) {
      la.issue(kt, smem);
      lb.issue(kt, smem + S::BM * kRowBytes);
      wait_vmcnt<0>();
      __syncthreads();
      mma.ktile(acc, smem, smem + S::BM * kRowBytes, p, [](int) {});
      __syncthreads();
    }
    return;
  }
  la.issue(0, smem);
  lb.issue(0, smem + S::BM * kRowBytes);
  wait_vmcnt<0>();
  __syncthreads();
  for (int64_t kt = 0; kt < nk; ++kt) {
    const lds_char* cur = smem + (kt & 1) * kStageBytes;
    lds_char* nxt = smem + ((kt + 1) & 1) * kStageBytes;
    const bool more = kt + 1 < nk;
    const auto ra = la.rsrc(kt + 1, more);
    const auto rb = lb.rsrc(kt + 1, more);
    mma.ktile(acc, cur, cur + S::BM * kRowBytes, p, [&](int q) {
      if (q < LA::kPer)
        la.issue_one(ra, nxt, q);
      else if (q < kLoads)
        lb.issue_one(rb, nxt + S::BM * kRowBytes, q - LA::kPer);
    });
    wait_vmcnt<0>();
    __syncthreads();
  }
}

// Tiles of the gradient; the first `whole` by one workgroup each, the others by
// `slices` workgroups, `slice` k-tiles each, that leave their sums in `part`
// [tile][slice][tile's rows and columns].
struct GradArgs {
  const uint16_t* x;   // blocks of [M]
  const uint16_t* dy;  // rows dys apart (bf16), or terms in blocks of [N]
  int64_t rows, M, N, dys, ktiles;
  int64_t dy_part;     // values between dy's terms
  int64_t slice;
  int32_t whole, slices;
  float* part;
  void* out;
  bool accumulate;
};

template <typename TO, class S, bool kTerms, int kStages>
__global__ __launch_bounds__(S::kThreads)
__attribute__((amdgpu_waves_per_eu(kStages == 1 ? 4 : 2))) void
act8_grad_kernel(GradArgs g) {
#ifdef __HIP_DEVICE_COMPILE__  // the host's pass takes the name alone
  constexpr bool kBeside = std::is_same_v<S, TermTile>;
  constexpr int kParts = kTerms && !kBeside ? 3 : 1;
  constexpr int kStageBytes = S::kStageBytes + (kBeside ? 2 * S::BN * kRowBytes : 0);
  constexpr int kEpiCols = 64, kEpiStride = kEpiCols + 8;  // floats per staged row of results
  constexpr int kEpiBytes = S::BM * kEpiStride * 4;
  constexpr int kBytes = kStages * kStageBytes > kEpiBytes ? kStages * kStageBytes : kEpiBytes;
  __shared__ __attribute__((aligned(16))) char smem_raw[kBytes];
  lds_char* smem = (lds_char*)smem_raw;
  const int tiles_m = (int)((g.M + S::BM - 1) / S::BM), tiles_n = (int)((g.N + S::BN - 1) / S::BN);
  int tile, slice = -1;
  int64_t k0 = 0, n = g.ktiles;
  if ((int)blockIdx.x < g.whole) {
    tile = xcd_remap(blockIdx.x, g.whole);
  } else {
    const int rest = tiles_m * tiles_n - g.whole;
    const int u = xcd_remap(blockIdx.x - g.whole, rest * g.slices);
    slice = u / rest, tile = g.whole + u % rest;
    k0 = slice * g.slice, n = min(g.slice, g.ktiles - k0);
  }
  const TileCoord tc = grouped_tile(tile, tiles_m, tiles_n, 8);
  const int64_t m0 = (int64_t)tc.m * S::BM, n0 = (int64_t)tc.n * S::BN;
  Accum<S> acc;
  acc.zero();
  const LanePos p = lane_pos<S>();
  const auto lx = block_loader<S, S::BM>(g.x, g.M, m0, k0);
  PartLoader<DirectLoader<S::BM, S::kWaves>, kParts> la{lx, n, 0};
  if constexpr (kBeside) {
    TermLoader<S> lb{block_loader<S, S::BN>(g.dy, g.N, n0, k0), g.dy_part * 2};
    grad_mainloop<TermMma<S>, kStages, kStageBytes>(acc, la, lb, n, smem, p);
  } else if constexpr (kTerms) {
    const auto ly = block_loader<S, S::BN>(g.dy, g.N, n0, k0);
    PartLoader<DirectLoader<S::BN, S::kWaves>, kParts> lb{ly, n, g.dy_part * 2};
    grad_mainloop<GradMma<S, false>, kStages, kStageBytes>(acc, la, lb, n * kParts, smem, p);
  } else {
    PartLoader<RowLoader<S>, 1> lb;
    lb.l.init(g.dy, g.dys, g.rows, g.N, n0, k0);
    grad_mainloop<GradMma<S, true>, kStages, kStageBytes>(acc, la, lb, n, smem, p);
  }
  if (slice >= 0) {
    // as the accumulators hold them: act8_sum_kernel finds the rows and columns
    float* const part = g.part + ((int64_t)(tile - g.whole) * g.slices + slice) * (S::BM * S::BN) +
                        (threadIdx.x >> 6) * (S::WM * S::WN) + 4 * p.lane;
#pragma unroll
    for (int i = 0; i < S::MB; ++i)
#pragma unroll
      for (int j = 0; j < S::NB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const floatx16_t& v = acc.v[i][j];
          *reinterpret_cast<float4*>(part + ((i * S::NB + j) * 4 + q) * 256) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
    return;
  }
  for (int q = 0; q < S::BN / kEpiCols; ++q) {
    __syncthreads();  // the mainloop's (or the previous pass's) reads of LDS are done
#pragma unroll
    for (int j = 0; j < S::NB; ++j) {
      const int col = p.wave_n0 + 32 * j;
      if (col < kEpiCols * q || col >= kEpiCols * q + kEpiCols) continue;
      const int c = col - kEpiCols * q + (p.lane & 31);
#pragma unroll
      for (int i = 0; i < S::MB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          lds_store<float>(smem + ((uint32_t)p.row(i, r) * kEpiStride + c) * 4, acc.v[i][j][r]);
    }
    __syncthreads();
    const int64_t cb = n0 + kEpiCols * q;
    for (int it = threadIdx.x; it < S::BM * (kEpiCols / 8); it += S::kThreads) {
      const int t = it / (kEpiCols / 8), c = (it % (kEpiCols / 8)) * 8;
      if (m0 + t >= g.M || cb + c >= g.N) continue;
      const floatx4_t lo = lds_load<floatx4_t>(smem + ((uint32_t)t * kEpiStride + c) * 4);
      const floatx4_t hi = lds_load<floatx4_t>(smem + ((uint32_t)t * kEpiStride + c + 4) * 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      TO* const to = static_cast<TO*>(g.out) + (m0 + t) * g.N + cb + c;
      if (g.accumulate) {
        Piece<TO> old;
        old.load(to);
        float f[8];
        old.get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += f[e];
      }
      Piece<TO>::store(to, v);
    }
  }
#endif
}

// The tiles that came in slices, added in order: a lane has 4 rows of a column, as they
// lie in an accumulator.
template <typename TO, class S>
__global__ __launch_bounds__(kBlock) void act8_sum_kernel(GradArgs g) {
  constexpr int kEach = S::BM * S::BN / (4 * kBlock);  // workgroups of a tile
  const int tiles_m = (int)((g.M + S::BM - 1) / S::BM), tiles_n = (int)((g.N + S::BN - 1) / S::BN);
  const int tile = blockIdx.x / kEach;
  const TileCoord tc = grouped_tile(g.whole + tile, tiles_m, tiles_n, 8);
  const int at = (blockIdx.x % kEach) * kBlock + threadIdx.x, lane = at & 63;
  const int q = (at >> 6) & 3, block = at >> 8;
  const int j = block % S::NB, i = block / S::NB % S::MB, wave = block / (S::NB * S::MB);
  const int64_t row = (int64_t)tc.m * S::BM + wave / S::WAVES_N * S::WM + 32 * i + 8 * q +
                      4 * (lane >> 5);
  const int64_t col = (int64_t)tc.n * S::BN + wave % S::WAVES_N * S::WN + 32 * j + (lane & 31);
  if (col >= g.N) return;
  const float* p = g.part + (int64_t)tile * g.slices * (S::BM * S::BN) + 4 * (int64_t)at;
  float4 f = make_float4(0, 0, 0, 0);
#pragma unroll 8
  for (int s = 0; s < g.slices; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)s * (S::BM * S::BN));
    f.x += v.x, f.y += v.y, f.z += v.z, f.w += v.w;
  }
  const float sum[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (row + e >= g.M) break;
    TO* const to = static_cast<TO*>(g.out) + (row + e) * g.N + col;
    Elem<TO>::store(to, g.accumulate ? Elem<TO>::to_f32(*to) + sum[e] : sum[e]);
  }
}

template <typename F>
hipError_t with_rows(Dtype dt, int64_t d, F&& f) {
  const bool narrow = d <= 128;  // 16 lanes a row, of which d / 8 have a piece
  if (dt == Dtype::F32)
    return narrow ? f(float{}, std::integral_constant<int, 16>{})
                  : f(float{}, std::integral_constant<int, 64>{});
  return narrow ? f(uint16_t{}, std::integral_constant<int, 16>{})
                : f(uint16_t{}, std::integral_constant<int, 64>{});
}

// A launch's threads are counted in 32 bits; calls of more rows take several.
template <typename F>
hipError_t in_launches(int64_t rows, int64_t per, F&& f) {
  const int64_t most = per << 23;
  for (int64_t at = 0; at < rows; at += most) {
    const int64_t n = std::min(rows - at, most);
    f(at, n, dim3((unsigned)((n + per - 1) / per)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

int64_t ktiles_of(const Act8Grad& g) { return (g.rows + kTokens - 1) / kTokens; }
int64_t grad_tiles(const Act8Grad& g, int64_t side) {
  return ((g.d_in + side - 1) / side) * ((g.d_out + side - 1) / side);
}

// Whether small tiles take one stage, and so twice as many workgroups a CU, which cover each
// other's loads and results: with dy's terms where there are more tiles than CUs, else where
// there are more tiles than two a CU and the sums are short (us with one stage / two: 200 x 2560 x
// 4096 20 / 23, 300 x 5120 x 7680 51 / 57, 700 x 2568 x 3336 29 / 35, 1776 x 4096 x 1536 44 / 41,
// 2048 x 2560 x 2560 48 / 42).
bool one_stage(const Act8Grad& g) {
  const int64_t tiles = grad_tiles(g, SmallTile::BM);
  return g.dt == Dtype::F32 ? tiles > 256 : tiles > 512 && ktiles_of(g) <= 16;
}

// How the gradient is cut: tiles of 256 or 128, `whole` of them a workgroup's each, the
// others in `slices` of `slice` k-tiles.
struct Cut {
  int side, whole, slices;
  int64_t slice;
};

// The cut that takes the least time by what was measured of its parts: tiles that fill
// whole rounds of the chip (256 workgroups of wide tiles, 512 of small ones) run whole, in
// step with one another along the tokens, so that they share their operands in L2; what is
// left over is cut along the tokens as well, so that the last round is short.  A slice
// more costs a write and a read of its sums.  Calls in us with wide / small tiles (bf16):
//   1 x 1024 x 1536 16 / 12,  200 x 2560 x 4096 26 / 23,  1000 x 1024 x 1536 29 / 22,
//   2048 x 2560 x 2560 62 / 42,  3000 x 5120 x 7680 238 / 255,  8192 x 2560 x 7680 300 / 350,
//   32768 x 1024 x 4096 259 / 330,  32768 x 2560 x 7680 1093 / 1426
Cut cut_of(const Act8Grad& g) {
  const int64_t n = ktiles_of(g);
  const double terms = g.dt == Dtype::F32 ? 3.0 : 1.0;
  // whether the operands stay in the 256 MB last-level cache
  const bool cached = (double)g.rows * (g.d_in + terms * g.d_out) * 2.0 < 256e6;
  Cut best{};
  double least = -1;
  for (const int side : {256, 128}) {
    const bool beside = side == 128 && terms > 1, single = side == 128 && one_stage(g);
    const bool alone = beside && !single;
    const int64_t round = side == 256 || alone ? 256 : single && !beside ? 1024 : 512;
    const int64_t tiles = grad_tiles(g, side);
    // us of a k-tile or of three side by side (small ones take twice the operands for their work: more where those
    // come from memory) and around them, MB of a tile's sums
    const double ktile = beside ? (alone ? 1.0 : 1.9) * (cached ? 1.0 : 1.7)
                                : terms * (side == 256 ? 1.6 : (cached ? 0.9 : 1.1) * (single ? 2 : 1));
    const double around = side == 256 ? 14.0 : alone ? 6.0 : 5.0;
    const double sums = (double)side * side * 8e-6;
    const int64_t rest = tiles % round;
    const double before = (double)(tiles / round) * ((double)n * ktile + around);
    for (int64_t s = 1; s <= 64 && (s == 1 || (rest && n >= 2 * s)); ++s) {
      const int64_t slice = (n + s - 1) / s, used = (n + slice - 1) / slice;
      const double rounds = (double)((rest * used + round - 1) / round);
      const double us = before + rounds * ((double)slice * ktile + around) +
                        (used > 1 ? (double)(rest * used) * sums / 4.0 + 4.0 : 0.0);
      if (least >= 0 && us >= least) continue;
      least = us;
      best = Cut{side, (int)(used == 1 ? tiles : tiles - rest), (int)used, slice};
    }
  }
  return best;
}

// Workspace: x and dy's terms in blocks, the slices' sums.
struct GradPlan {
  size_t dy, part, bytes;
  Cut cut;
};
GradPlan grad_plan(const Act8Grad& g) {
  GradPlan p;
  p.cut = cut_of(g);
  const size_t tokens = (size_t)ktiles_of(g) * kTokens;
  p.dy = align256(tokens * g.d_in * 2);
  p.part = p.dy + (g.dt == Dtype::F32 ? align256(3 * tokens * g.d_out * 2) : 0);
  p.bytes = p.part + (size_t)(grad_tiles(g, p.cut.side) - p.cut.whole) * p.cut.slices *
                         ((size_t)p.cut.side * p.cut.side * sizeof(float));
  return p;
}

template <class S, bool kTerms, int kStages>
hipError_t launch_products(const Act8Grad& g, const GradArgs& a, hipStream_t s) {
  const int64_t rest = grad_tiles(g, S::BM) - a.whole;
  const dim3 grid((unsigned)(a.whole + rest * a.slices));
  const dim3 sums((unsigned)(rest * (S::BM * S::BN / (4 * kBlock))));
  const bool f32 = kTerms || g.grad_dt == Dtype::F32;
  if (f32)
    act8_grad_kernel<float, S, kTerms, kStages><<<grid, S::kThreads, 0, s>>>(a);
  else if constexpr (!kTerms)
    act8_grad_kernel<uint16_t, S, kTerms, kStages><<<grid, S::kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || rest == 0) return e;
  if (f32)
    act8_sum_kernel<float, S><<<sums, kBlock, 0, s>>>(a);
  else if constexpr (!kTerms)
    act8_sum_kernel<uint16_t, S><<<sums, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act8_store(Dtype dt, const void* x, int64_t rows, int64_t d, int64_t xs,
                             int8_t* codes, uint8_t* exps, hipStream_t s) {
  return with_rows(dt, d, [&](auto t, auto lpr) {
    using T = decltype(t);
    constexpr int L = decltype(lpr)::value;
    const int64_t groups = (d + kAct8Group - 1) / kAct8Group;
    return in_launches(rows, kBlock / L, [&](int64_t at, int64_t n, dim3 grid) {
      act8_store_kernel<T, L><<<grid, kBlock, 0, s>>>(static_cast<const T*>(x) + at * xs,
                                                      codes + at * d, exps + at * groups, n, d, xs);
    });
  });
}

hipError_t launch_act8_load(Dtype dt, const int8_t* codes, const uint8_t* exps, int64_t rows,
                            int64_t d, int64_t xs, void* x, hipStream_t s) {
  return with_rows(dt, d, [&](auto t, auto lpr) {
    using T = decltype(t);
    constexpr int L = decltype(lpr)::value;
    const int64_t groups = (d + kAct8Group - 1) / kAct8Group;
    return in_launches(rows, kBlock / L, [&](int64_t at, int64_t n, dim3 grid) {
      act8_load_kernel<T, L><<<grid, kBlock, 0, s>>>(codes + at * d, exps + at * groups,
                                                     static_cast<T*>(x) + at * xs, n, d, xs);
    });
  });
}

size_t act8_weight_grad_bytes(const Act8Grad& g) { return grad_plan(g).bytes; }

hipError_t launch_act8_weight_grad(const Act8Grad& g, const int8_t* codes, const uint8_t* exps,
                                   const void* dy, void* grad, void* ws, hipStream_t s) {
  const GradPlan p = grad_plan(g);
  char* const base = static_cast<char*>(ws);
  const int64_t n = ktiles_of(g);
  GradArgs a{};
  a.x = reinterpret_cast<uint16_t*>(base), a.rows = g.rows, a.M = g.d_in, a.N = g.d_out;
  a.ktiles = n, a.slice = p.cut.slice, a.whole = p.cut.whole, a.slices = p.cut.slices;
  a.part = reinterpret_cast<float*>(base + p.part);
  a.out = grad, a.accumulate = g.accumulate;
  uint16_t *const x = reinterpret_cast<uint16_t*>(base), *terms = nullptr;
  const bool split = g.dt == Dtype::F32;
  if (split) {
    terms = reinterpret_cast<uint16_t*>(base + p.dy);
    a.dy = terms, a.dy_part = n * kTokens * g.d_out;
  } else {
    a.dy = static_cast<const uint16_t*>(dy), a.dys = g.dys;
  }
  const int64_t groups = (g.d_in + kAct8Group - 1) / kAct8Group;
  const unsigned x_columns = (unsigned)((g.d_in + kXColumns - 1) / kXColumns);
  const hipError_t e = in_launches(n, 1, [&](int64_t at, int64_t, dim3 grid) {
    grid.y = x_columns + (split ? (unsigned)((g.d_out + 127) / 128) : 0);
    const int64_t t = at * kTokens;
    act8_operands_kernel<<<grid, kBlock, 0, s>>>(
        codes + t * g.d_in, exps + t * groups, x + t * g.d_in, g.rows - t, g.d_in, x_columns,
        split ? static_cast<const float*>(dy) + t * g.dys : nullptr, g.dys,
        split ? terms + t * g.d_out : nullptr, a.dy_part, g.d_out);
  });
  if (e != hipSuccess) return e;
  if (p.cut.side == 256)
    return split ? launch_products<WideTile, true, 2>(g, a, s)
                 : launch_products<WideTile, false, 2>(g, a, s);
  if (!split)
    return one_stage(g) ? launch_products<SmallTile, false, 1>(g, a, s)
                        : launch_products<SmallTile, false, 2>(g, a, s);
  return one_stage(g) ? launch_products<TermTile, true, 1>(g, a, s)
                      : launch_products<TermTile, true, 2>(g, a, s);
}

}  // namespace ttt
