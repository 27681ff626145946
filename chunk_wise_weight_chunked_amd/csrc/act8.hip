// act8.hip -- activations kept in 8 bits, and the weight gradient from them.
//
//   code = round(x 2^-e), x8 = code 2^e,   grad (+)= x8^T dy
//
// with one e for 32 values of a row: the smallest for which all codes are within
// +-127, between -126 and 121 (127 2^121 is the largest that fp32 has; codes beside it end at
// +-127).  A power of two as the scale makes the codes exact (no division), and x8
// exact in bf16 (7 bits and a sign), so that the weight gradient's products on
// the bf16 matrix cores are exact before they are added in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// A lane takes 4 columns of 8 tokens: load(first token, first column, tokens that are
// there), then out(place of a column's 8 tokens, column).  The 8 lanes that share columns
// are neighbours, so that they write whole 128-byte rows; a workgroup has 128 columns.
template <class Load, class Out>
__device__ __forceinline__ void to_blocks(int64_t rows, int64_t n, Load&& load, Out&& out) {
  const int64_t block = blockIdx.x, c0 = blockIdx.y * (int64_t)128 + 4 * (threadIdx.x >> 3);
  const int oct = threadIdx.x & 7;
  if (c0 >= n) return;
  const int64_t t0 = block * kTokens + 8 * oct;
  load(t0, c0, (int)max<int64_t>(0, min<int64_t>(8, rows - t0)));
#pragma unroll
  for (int c = 0; c < 4; ++c) out((block * n + c0 + c) * kTokens + 8 * oct, c);
}

__global__ __launch_bounds__(kBlock) void act8_blocks_kernel(const int8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ exps,
                                                             uint16_t* __restrict__ x, int64_t rows,
                                                             int64_t d) {
  float v[8][4];
  to_blocks(
      rows, d,
      [&](int64_t t0, int64_t c0, int live) {
        const int64_t groups = (d + kAct8Group - 1) / kAct8Group;
        uint32_t w[8], e[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          w[t] = e[t] = 0;
          if (t < live) {
            w[t] = *reinterpret_cast<const uint32_t*>(codes + (t0 + t) * d + c0);
            e[t] = exps[(t0 + t) * groups + c0 / kAct8Group];
          }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[t][c] = (float)((int32_t)(w[t] << (24 - 8 * c)) >> 24) * __uint_as_float(e[t] << 23);
      },
      [&](int64_t at, int c) {
        *reinterpret_cast<uint4*>(x + at) =
            make_uint4(pack_bf16x2(v[0][c], v[1][c]), pack_bf16x2(v[2][c], v[3][c]),
                       pack_bf16x2(v[4][c], v[5][c]), pack_bf16x2(v[6][c], v[7][c]));
      });
}

// An fp32 dy as three bf16 terms whose sum it is: the leading 8 bits of what is left,
// three times; an infinity or NaN goes into the first alone.  Terms `part` values apart.
__global__ __launch_bounds__(kBlock) void act8_terms_kernel(const float* __restrict__ dy,
                                                            int64_t dys, uint16_t* __restrict__ out,
                                                            int64_t part, int64_t rows, int64_t n) {
  float v[8][4];
  to_blocks(
      rows, n,
      [&](int64_t t0, int64_t c0, int live) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          float4 f = make_float4(0, 0, 0, 0);
          if (t < live) f = *reinterpret_cast<const float4*>(dy + (t0 + t) * dys + c0);
          v[t][0] = f.x, v[t][1] = f.y, v[t][2] = f.z, v[t][3] = f.w;
        }
      },
      [&](int64_t at, int c) {
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
          *reinterpret_cast<uint4*>(out + k * part + at) =
              make_uint4(top[0] >> 16 | top[1], top[2] >> 16 | top[3], top[4] >> 16 | top[5],
                         top[6] >> 16 | top[7]);
        }
      });
}

using WTile = TileShape<256, 256, 2, 4>;
constexpr int kEpiCols = 64;
constexpr int kEpiStride = kEpiCols + 8;  // floats per staged row

// k-tiles [k0, k0 + n) of an operand, kParts times: of x again and again, of dy's terms
// one after the other (part_stride bytes between them).
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
using BlockLoader = DirectLoader<256, WTile::kWaves>;
using RowLoader = KMajorLoader<uint16_t, WTile::kWaves>;
// 256 columns from n0 of an operand of N columns in blocks.
__device__ __forceinline__ BlockLoader block_loader(const uint16_t* p, int64_t N, int64_t n0,
                                                    int64_t k0) {
  BlockLoader l;
  l.init(p + (k0 * N + n0) * kTokens, kRowBytes, N * kRowBytes, (N - n0) * kRowBytes, 0);
  return l;
}
// The same of rows [rows][ld] of N columns.
__device__ __forceinline__ RowLoader row_loader(const uint16_t* p, int64_t ld, int64_t rows,
                                                int64_t N, int64_t n0, int64_t k0) {
  RowLoader l;
  l.init(p + k0 * kTokens * ld + n0, kRowBytes, ld * 2, kTokens * ld * 2,
         ((rows - k0 * kTokens - 1) * ld + N - n0) * 2);
  return l;
}

// A k-tile's products with x's fragments read as rows and dy's transposed from token rows
// (kRows), or both as rows.  Reads for the next 16 tokens are spread between the matrix
// instructions, hook(q) follows instruction q.  The transposing reads are inline assembly,
// each block with its wait: the compiler lets the builtin wait for every direct-to-LDS load
// in flight, also those into the other stage (2560 x 7680 at 32K tokens: 1438 us with it, 1118 without).
template <bool kRows>
struct GradMma {
  using S = WTile;
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
      static_assert(S::MB == 4 && S::NB == 2, "the reads below");
      bf16x8_t a[2][4], b[2][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[0][i] = Plain::read_a(sA, p, i, 0);
      read_rows(b[0], sB, 0);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int i = m >> 1, j = m & 1;
          acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[s & 1][i], b[s & 1][j],
                                                                acc.v[i][j], 0, 0, 0);
          if (s + 1 < kSteps) {
            if (m < 4) a[(s + 1) & 1][m] = Plain::read_a(sA, p, m, s + 1);
            if (m == 5) read_rows(b[(s + 1) & 1], sB, s + 1);
          }
          hook(8 * s + m);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
};

// The mainloop of gemm_core.h on these fragments: k-tile kt + 1's loads one after each of
// kt's first matrix instructions.
template <class Mma, class LA, class LB>
__device__ __forceinline__ void grad_mainloop(Accum<WTile>& acc, LA& la, LB& lb, int64_t nk,
                                              lds_char* smem, const LanePos& p) {
  using S = WTile;
  constexpr int kLoads = LA::kPer + LB::kPer;
  static_assert(kLoads <= Mma::kSteps * S::MB * S::NB, "the loads fit the k-tile's MFMAs");
  Mma mma;
  mma.init(p);
  la.issue(0, smem);
  lb.issue(0, smem + S::BM * kRowBytes);
  wait_vmcnt<0>();
  __syncthreads();
  for (int64_t kt = 0; kt < nk; ++kt) {
    const lds_char* cur = smem + (kt & 1) * S::kStageBytes;
    lds_char* nxt = smem + ((kt + 1) & 1) * S::kStageBytes;
    const bool more = kt + 1 < nk;
    const rsrc_t ra = la.rsrc(kt + 1, more), rb = lb.rsrc(kt + 1, more);
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
// [tile][slice][256][256].
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

template <typename TO, bool kTerms>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void
act8_grad_kernel(GradArgs g) {
  using S = WTile;
  static_assert(S::kLdsBytes >= S::BM * kEpiStride * 4, "epilogue stage fits the pipeline's LDS");
  constexpr int kParts = kTerms ? 3 : 1;
  __shared__ __attribute__((aligned(16))) char smem_raw[S::kLdsBytes];
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
  PartLoader<BlockLoader, kParts> la{block_loader(g.x, g.M, m0, k0), n, 0};
  if constexpr (kTerms) {
    PartLoader<BlockLoader, kParts> lb{block_loader(g.dy, g.N, n0, k0), n, g.dy_part * 2};
    grad_mainloop<GradMma<false>>(acc, la, lb, n * kParts, smem, p);
  } else {
    PartLoader<RowLoader, kParts> lb{row_loader(g.dy, g.dys, g.rows, g.N, n0, k0), n, 0};
    grad_mainloop<GradMma<true>>(acc, la, lb, n, smem, p);
  }
  float* const part =
      slice < 0 ? nullptr
                : g.part + ((int64_t)(tile - g.whole) * g.slices + slice) * (S::BM * S::BN);
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
      if (part) {
        Piece<float>::store(part + t * S::BN + kEpiCols * q + c, v);
        continue;
      }
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
}

// The tiles that came in slices, added in order: 8 rows of a tile a workgroup.
template <typename TO>
__global__ __launch_bounds__(kBlock) void act8_sum_kernel(GradArgs g) {
  using S = WTile;
  constexpr int kEach = S::BM * S::BN / (8 * kBlock);  // workgroups of a tile
  const int tiles_m = (int)((g.M + S::BM - 1) / S::BM), tiles_n = (int)((g.N + S::BN - 1) / S::BN);
  const int tile = blockIdx.x / kEach;
  const TileCoord tc = grouped_tile(g.whole + tile, tiles_m, tiles_n, 8);
  const int at = (blockIdx.x % kEach) * (8 * kBlock) + 8 * threadIdx.x;
  const int64_t row = (int64_t)tc.m * S::BM + at / S::BN, col = (int64_t)tc.n * S::BN + at % S::BN;
  if (row >= g.M || col >= g.N) return;
  const float* p = g.part + (int64_t)tile * g.slices * (S::BM * S::BN) + at;
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < g.slices; ++s) {
    Piece<float> q;
    q.load(p + (int64_t)s * (S::BM * S::BN));
    float v[8];
    q.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += v[j];
  }
  TO* const to = static_cast<TO*>(g.out) + row * g.N + col;
  if (g.accumulate) {
    Piece<TO> old;
    old.load(to);
    float v[8];
    old.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += v[j];
  }
  Piece<TO>::store(to, f);
}

template <typename F>
hipError_t with_rows(Dtype dt, int64_t d, F&& f) {
  const bool narrow = d <= 128;  // 16 lanes a row: at least one piece of 8 for half of them
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
int64_t grad_tiles(const Act8Grad& g) {
  return ((g.d_in + 255) / 256) * ((g.d_out + 255) / 256);
}

// A workgroup owns a CU: tiles that fill whole rounds of 256 CUs are one workgroup's
// each, in step with one another along the tokens (they share their operands in L2); what
// is left over is cut along the tokens, so that the last round is short.  Some 1.6 us for
// 64 tokens of a tile and 10 around it; a slice more costs a write and a read of its
// 256 KB of sums.
struct Slices {
  int whole, slices;
  int64_t slice;  // k-tiles of a slice
};
Slices slices_of(const Act8Grad& g) {
  constexpr int kCus = 256;
  const int64_t tiles = grad_tiles(g), n = ktiles_of(g);
  const double us = g.dt == Dtype::F32 ? 3 * 1.6 : 1.6;
  const int rest = (int)(tiles % kCus);
  Slices best{(int)(tiles - rest), 1, n};
  double least = 0;
  for (int64_t s = 1; s <= 64 && (s == 1 || n >= 2 * s); ++s) {
    const int64_t slice = (n + s - 1) / s, used = (n + slice - 1) / slice;
    const double rounds = (double)((rest * used + kCus - 1) / kCus);
    const double t = rounds * ((double)slice * us + 10.0) +
                     (used > 1 ? (double)(rest * used) * 0.5e6 / 4e6 + 5.0 : 0.0);
    if (s == 1 || t < least) best.slices = (int)used, best.slice = slice, least = t;
  }
  if (best.slices == 1) best.whole = (int)tiles;
  return best;
}

// Workspace: x and dy's terms in blocks, the slices' sums.
struct GradPlan {
  size_t dy, part, bytes;
  Slices s;
};
GradPlan grad_plan(const Act8Grad& g) {
  GradPlan p;
  p.s = slices_of(g);
  const size_t tokens = (size_t)ktiles_of(g) * kTokens;
  p.dy = align256(tokens * g.d_in * 2);
  p.part = p.dy + (g.dt == Dtype::F32 ? align256(3 * tokens * g.d_out * 2) : 0);
  p.bytes = p.part + (size_t)(grad_tiles(g) - p.s.whole) * p.s.slices * (256 * 256 * sizeof(float));
  return p;
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
  a.ktiles = n, a.slice = p.s.slice, a.whole = p.s.whole, a.slices = p.s.slices;
  a.part = reinterpret_cast<float*>(base + p.part);
  a.out = grad, a.accumulate = g.accumulate;
  uint16_t* const x = reinterpret_cast<uint16_t*>(base);
  const int64_t groups = (g.d_in + kAct8Group - 1) / kAct8Group;
  const auto columns = [](int64_t n) { return (unsigned)((n + 127) / 128); };
  hipError_t e = in_launches(n, 1, [&](int64_t at, int64_t, dim3 grid) {
    grid.y = columns(g.d_in);
    const int64_t t = at * kTokens;
    act8_blocks_kernel<<<grid, kBlock, 0, s>>>(codes + t * g.d_in, exps + t * groups,
                                               x + t * g.d_in, g.rows - t, g.d_in);
  });
  if (e != hipSuccess) return e;
  if (g.dt == Dtype::F32) {
    uint16_t* const terms = reinterpret_cast<uint16_t*>(base + p.dy);
    a.dy = terms, a.dy_part = n * kTokens * g.d_out;
    e = in_launches(n, 1, [&](int64_t at, int64_t, dim3 grid) {
      grid.y = columns(g.d_out);
      const int64_t t = at * kTokens;
      act8_terms_kernel<<<grid, kBlock, 0, s>>>(static_cast<const float*>(dy) + t * g.dys, g.dys,
                                                terms + t * g.d_out, a.dy_part, g.rows - t,
                                                g.d_out);
    });
    if (e != hipSuccess) return e;
  } else {
    a.dy = static_cast<const uint16_t*>(dy), a.dys = g.dys;
  }
  const int64_t rest = grad_tiles(g) - a.whole;
  const dim3 grid((unsigned)(a.whole + rest * a.slices)), sums((unsigned)(rest * 32));
  if (g.dt == Dtype::F32)
    act8_grad_kernel<float, true><<<grid, 512, 0, s>>>(a);
  else if (g.grad_dt == Dtype::F32)
    act8_grad_kernel<float, false><<<grid, 512, 0, s>>>(a);
  else
    act8_grad_kernel<uint16_t, false><<<grid, 512, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || rest == 0) return e;
  if (g.grad_dt == Dtype::F32)
    act8_sum_kernel<float><<<sums, kBlock, 0, s>>>(a);
  else
    act8_sum_kernel<uint16_t><<<sums, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttt
