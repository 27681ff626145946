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

// An fp32 dy as three bf16 terms whose sum it is: the leading 8 bits of what is left,
// three times.  parts [3][rows][n]; an infinity or NaN goes into the first alone.
__global__ __launch_bounds__(kBlock) void act8_split_kernel(const float* __restrict__ dy,
                                                            int64_t dys, uint16_t* __restrict__ parts,
                                                            int64_t rows, int64_t n) {
  const int64_t pieces = n >> 3, total = rows * pieces;
  const int64_t step = (int64_t)gridDim.x * kBlock;
  for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < total; i += step) {
    const int64_t row = i / pieces, c = i % pieces;
    Piece<float> p;
    p.load(dy + row * dys + 8 * c);
    float f[8];
    p.get(f);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = __float_as_uint(f[2 * j]), hi = __float_as_uint(f[2 * j + 1]);
        // a NaN whose upper bits are an infinity's stays one
        const uint32_t a = abs_bits(f[2 * j]) > 0x7f800000u ? 0x7fc00000u : lo & 0xffff0000u;
        const uint32_t b = abs_bits(f[2 * j + 1]) > 0x7f800000u ? 0x7fc00000u : hi & 0xffff0000u;
        w[j] = (a >> 16) | b;
        f[2 * j] = abs_bits(f[2 * j]) >= 0x7f800000u ? 0.0f : f[2 * j] - __uint_as_float(a);
        f[2 * j + 1] =
            abs_bits(f[2 * j + 1]) >= 0x7f800000u ? 0.0f : f[2 * j + 1] - __uint_as_float(b);
      }
      *reinterpret_cast<uint4*>(parts + (k * rows + row) * n + 8 * c) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------ weight gradient
using WTile = TileShape<256, 256, 2, 4>;
constexpr int kTokens = kRowBytes / 2;  // tokens of a k-tile
constexpr int kEpiCols = 64;
constexpr int kEpiStride = kEpiCols + 8;  // floats per staged row

// A tokens-by-columns operand whose k-tiles are walked `parts` times (x8), or
// once over parts one after the other (dy's terms).
struct PartLoader {
  using Base = KMajorLoader<uint16_t, WTile::kWaves>;
  static constexpr int kPer = Base::kPer;
  Base l;
  int64_t per_part, part_stride;  // k-tiles of a part, bytes between parts
  const char* base;
  __device__ __forceinline__ rsrc_t rsrc(int64_t kt, bool live = true) const {
    const int64_t part = kt / per_part, k = kt - part * per_part;
    return make_rsrc(base + part * part_stride + k * l.kt_stride,
                     live ? l.valid_bytes - k * l.kt_stride : 0);
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
// Columns from n0 of token rows [0, rows), ld values apart, n values each.
__device__ __forceinline__ PartLoader part_loader(const uint16_t* p, int64_t ld, int64_t rows,
                                                  int64_t n, int64_t n0, int64_t part_stride) {
  PartLoader l;
  l.base = reinterpret_cast<const char*>(p + n0);
  l.l.init(l.base, kRowBytes, ld * 2, kTokens * ld * 2, ((rows - 1) * ld + n - n0) * 2);
  l.per_part = (rows + kTokens - 1) / kTokens;
  l.part_stride = part_stride;
  return l;
}

struct GradArgs {
  const uint16_t* x;   // [rows][M], decoded
  const uint16_t* dy;  // [parts][rows][N], rows dys apart
  int64_t rows, M, N, dys;
  int64_t slice;       // tokens of a slice, a multiple of kTokens
  int64_t dy_part;     // values between dy's parts
  int32_t parts;
  int32_t slices;
  void* out;           // slices > 1: fp32 [slices][M][N]; otherwise the gradient
  bool accumulate;
};

template <typename TO>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void
act8_grad_kernel(GradArgs g) {
  using S = WTile;
  static_assert(S::kLdsBytes >= S::BM * kEpiStride * 4, "epilogue stage fits the pipeline's LDS");
  __shared__ __attribute__((aligned(16))) char smem_raw[S::kLdsBytes];
  lds_char* smem = (lds_char*)smem_raw;
  const int tiles_m = (int)((g.M + S::BM - 1) / S::BM), tiles_n = (int)((g.N + S::BN - 1) / S::BN);
  const int L = xcd_remap(blockIdx.x, (int)gridDim.x);
  const int64_t slice = L / (tiles_m * tiles_n);
  const TileCoord tc = grouped_tile(L % (tiles_m * tiles_n), tiles_m, tiles_n, 8);
  const int64_t m0 = (int64_t)tc.m * S::BM, n0 = (int64_t)tc.n * S::BN;
  const int64_t k0 = slice * g.slice, rows = min(g.slice, g.rows - k0);
  Accum<S> acc;
  acc.zero();
  const LanePos p = lane_pos<S>();
  PartLoader la = part_loader(g.x + k0 * g.M, g.M, rows, g.M, m0, 0);
  PartLoader lb = part_loader(g.dy + k0 * g.dys, g.dys, rows, g.N, n0, g.dy_part * 2);
  mainloop<uint16_t, S, true, true, true, 1>(acc, la, lb, la.per_part * g.parts, smem, p,
                                             [](int64_t) {});
  TO* const out = static_cast<TO*>(g.out) + slice * g.M * g.N;
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
      TO* const to = out + (m0 + t) * g.N + cb + c;
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

// grad (+)= the slices' products, in order.
template <typename TO>
__global__ __launch_bounds__(kBlock) void act8_sum_kernel(const float* __restrict__ part,
                                                          int slices, TO* __restrict__ grad,
                                                          int64_t n, bool accumulate) {
  const int64_t step = (int64_t)gridDim.x * kBlock * 8;
  for (int64_t i = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 8; i < n; i += step) {
    float f[8];
    Piece<float> p;
    p.load(part + i);
    p.get(f);
    for (int s = 1; s < slices; ++s) {
      Piece<float> q;
      q.load(part + s * n + i);
      float v[8];
      q.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += v[j];
    }
    if (accumulate) {
      Piece<TO> old;
      old.load(grad + i);
      float v[8];
      old.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += v[j];
    }
    Piece<TO>::store(grad + i, f);
  }
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

// Token slices: a workgroup owns a CU, so tiles x slices should fill whole rounds
// of 256 CUs, at some 1.7 us for 64 tokens of a tile; a slice more costs a write
// and a read of the fp32 gradient (8 bytes at 4 TB/s) and 10 us.
int slices_of(const Act8Grad& g) {
  const int64_t tiles = ((g.d_in + 255) / 256) * ((g.d_out + 255) / 256);
  const int64_t ktiles = (g.rows + kTokens - 1) / kTokens * (g.dt == Dtype::F32 ? 3 : 1);
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 32 && (s == 1 || g.rows >= (int64_t)s * 4 * kTokens); ++s) {
    const double rounds = (double)((tiles * s + 255) / 256);
    const double us = rounds * ((double)((ktiles + s - 1) / s) * 1.7 + 10.0) +
                      (s > 1 ? s * (double)(g.d_in * g.d_out) * 8e-6 / 4.0 + 10.0 : 0.0);
    if (s == 1 || us < least) best = s, least = us;
  }
  return best;
}

struct GradPlan {
  size_t dy, part, bytes;
  int slices;
};
GradPlan grad_plan(const Act8Grad& g) {
  GradPlan p;
  p.slices = slices_of(g);
  p.dy = align256((size_t)(g.rows * g.d_in) * 2);
  p.part = p.dy + (g.dt == Dtype::F32 ? align256((size_t)(3 * g.rows * g.d_out) * 2) : 0);
  p.bytes = p.part + (p.slices > 1 ? (size_t)p.slices * g.d_in * g.d_out * sizeof(float) : 0);
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
  uint16_t* const x = reinterpret_cast<uint16_t*>(base);
  float* const part = reinterpret_cast<float*>(base + p.part);
  hipError_t e = launch_act8_load(Dtype::BF16, codes, exps, g.rows, g.d_in, g.d_in, x, s);
  if (e != hipSuccess) return e;
  GradArgs a{};
  a.x = x, a.rows = g.rows, a.M = g.d_in, a.N = g.d_out;
  a.slice = (g.rows + p.slices - 1) / p.slices;
  a.slice = (a.slice + kTokens - 1) / kTokens * kTokens;
  a.slices = (int32_t)((g.rows + a.slice - 1) / a.slice);
  if (g.dt == Dtype::F32) {
    uint16_t* const terms = reinterpret_cast<uint16_t*>(base + p.dy);
    const int64_t n = g.rows * (g.d_out / 8);
    act8_split_kernel<<<dim3((unsigned)std::min<int64_t>((n + kBlock - 1) / kBlock, 8192)), kBlock,
                        0, s>>>(static_cast<const float*>(dy), g.dys, terms, g.rows, g.d_out);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.dy = terms, a.dys = g.d_out, a.parts = 3, a.dy_part = g.rows * g.d_out;
  } else {
    a.dy = static_cast<const uint16_t*>(dy), a.dys = g.dys, a.parts = 1, a.dy_part = 0;
  }
  const int64_t tiles = ((g.d_in + 255) / 256) * ((g.d_out + 255) / 256);
  const dim3 grid((unsigned)(tiles * a.slices));
  const bool direct = a.slices == 1;
  a.out = direct ? grad : part;
  a.accumulate = direct && g.accumulate;
  if (direct && g.grad_dt == Dtype::BF16)
    act8_grad_kernel<uint16_t><<<grid, 512, 0, s>>>(a);
  else
    act8_grad_kernel<float><<<grid, 512, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || direct) return e;
  const int64_t n = g.d_in * g.d_out;
  const dim3 sg((unsigned)std::min<int64_t>((n / 8 + kBlock - 1) / kBlock, 16384));
  if (g.grad_dt == Dtype::BF16)
    act8_sum_kernel<uint16_t><<<sg, kBlock, 0, s>>>(part, a.slices, static_cast<uint16_t*>(grad), n,
                                                    g.accumulate);
  else
    act8_sum_kernel<float><<<sg, kBlock, 0, s>>>(part, a.slices, static_cast<float*>(grad), n,
                                                 g.accumulate);
  return hipGetLastError();
}

}  // namespace ttt
