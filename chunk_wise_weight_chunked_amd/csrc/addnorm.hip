// addnorm.hip -- residual addition and root-mean-square norm, and its gradients.
//
//   r = x + res,  y = r rstd w,  rstd = 1 / sqrt(mean r^2 + eps)
//   dr = rstd (w dy - r rstd^2 mean(w dy r)) + dr_out,  dw = sum_rows dy r rstd
//
// Both directions are bound by HBM: every input is read once and every output
// written once, a row stays in registers between the two uses of its values,
// and the only exchange is the sum over a row.  LPR lanes share a row (16 lanes,
// a wave or a workgroup: row_shape below), so that the sum is a few lane
// shuffles; lane l holds the 8-value pieces l, l + LPR, ... of its row (NV of
// them), one or two 16-byte loads each, all issued before the first is used.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "block.h"
#include "gemm_core.h"

namespace ttt {
namespace {

constexpr int kBlock = 256;
constexpr float kFp8Max = 448.0f;  // largest E4M3 value

// 8 consecutive values as loaded.
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float f[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = chunk_value<uint16_t>(v, i);
  }
  __device__ __forceinline__ static void store(uint16_t* p, const float f[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Piece<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float f[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ static void store(float* p, const float f[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// The sum (or maximum) of v over the LPR lanes of a row, in every one of them.
// For a workgroup's row, `s` holds one value per wave; `slot` alternates
// between uses so that one barrier per reduction is enough.
template <int LPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float (*s)[kBlock / 64], int slot) {
  constexpr int kLanes = LPR < 64 ? LPR : 64;
#pragma unroll
  for (int m = kLanes / 2; m >= 1; m >>= 1) {
    const float o = __shfl_xor(v, m, 64);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  if constexpr (LPR > 64) {
    if ((threadIdx.x & 63) == 0) s[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[slot][0];
#pragma unroll
    for (int w = 1; w < kBlock / 64; ++w) v = kMax ? fmaxf(v, s[slot][w]) : v + s[slot][w];
  }
  return v;
}

// E4M3 (OCP) of 8 values, packed.
__device__ __forceinline__ uint2 pack_fp8x8(const float f[8]) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// The scale that takes `top` to the largest 8-bit value; not below 2^-126, from
// where on down a scale has fewer bits and, rounded, could take `top` past it.
__device__ __forceinline__ float fp8_scale(float top) {
  return top > 0.0f ? fmaxf(top / kFp8Max, 0x1p-126f) : 1.0f;
}

template <typename TX, typename TR, bool kFp8, int LPR, int NV>
__global__ __launch_bounds__(kBlock) void addnorm_forward_kernel(
    const TX* x, const TR* res, const TX* __restrict__ w, TR* r, void* y,
    float* __restrict__ y_scale, int64_t rows, int d, int64_t xs, int64_t ys, float eps,
    bool grouped) {
  __shared__ float red[2][kBlock / 64];
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * (kBlock / LPR) + threadIdx.x / LPR;
  // LPR = kBlock: row < rows for the whole workgroup (its barriers are met by
  // all); lanes without a row in the other layouts meet no barrier
  if (row >= rows) return;
  const int pieces = d >> 3;
  Piece<TX> px[NV], pw[NV];
  Piece<TR> pr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LPR;
    px[i].zero();
    pr[i].zero();
    if (c < pieces) {
      px[i].load(x + row * xs + 8 * c);
      if (res) pr[i].load(res + row * (int64_t)d + 8 * c);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LPR;
    if (c < pieces) pw[i].load(w + 8 * c);
  }
  float v[NV][8], ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LPR;
    float f[8];
    px[i].get(v[i]);
    pr[i].get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] += f[j];
      ss += v[i][j] * v[i][j];
    }
    if (r && c < pieces) Piece<TR>::store(r + row * (int64_t)d + 8 * c, v[i]);
  }
  ss = row_reduce<LPR, false>(ss, red, 0);
  const float rstd = rsqrtf(ss / (float)d + eps);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LPR;
    if (c < pieces) {
      float f[8];
      pw[i].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = v[i][j] * rstd * f[j];
        if constexpr (kFp8) top = fmaxf(top, fabsf(v[i][j]));
      }
      if constexpr (!kFp8)
        Piece<TX>::store(static_cast<TX*>(y) + row * ys + 8 * c, v[i]);
    }
  }
  if constexpr (kFp8) {
    // divided, not multiplied by a rounded reciprocal, which moves values beside a
    // tie to the next code (32768 x 2560: 164 us, 163 with the reciprocal)
    const auto put = [&](int i, int c, float scale) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = v[i][j] / scale;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(y) + row * ys + 8 * c) = pack_fp8x8(f);
    };
    if (!grouped) {
      top = row_reduce<LPR, true>(top, red, 1);
      const float scale = fp8_scale(top);
      if (lane == 0) y_scale[row] = scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = lane + i * LPR;
        if (c < pieces) put(i, c, scale);
      }
    } else {
      // a group is the pieces of 16 neighbouring lanes; d is a multiple of the
      // group, so a group's lanes all have a piece or none has
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = lane + i * LPR;
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = fmaxf(t, fabsf(v[i][j]));
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) t = fmaxf(t, __shfl_xor(t, m, 64));
        if (c < pieces) {
          const float scale = fp8_scale(t);
          if ((lane & 15) == 0) y_scale[row * (d / kNormScaleGroup) + (c >> 4)] = scale;
          put(i, c, scale);
        }
      }
    }
  }
}

// Rows in a grid-stride loop; each lane keeps the sum of dy n of its columns
// in registers over all its rows, and the workgroup's row groups then add
// theirs in a fixed order into one row of `part`.
template <typename TX, typename TR, int LPR, int NV>
__global__ __launch_bounds__(kBlock) void addnorm_backward_kernel(
    const TX* __restrict__ dy, const TR* __restrict__ r, const TX* __restrict__ w,
    const TR* dr_out, TR* dr, TX* __restrict__ dx, float* __restrict__ part, int64_t rows, int d,
    int64_t xs, int64_t ys, float eps) {
  constexpr int kGroups = kBlock / LPR;
  __shared__ float red[4][kBlock / 64];
  extern __shared__ float sum[];  // d floats, kGroups > 1 only
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int pieces = d >> 3;
  Piece<TX> pw[NV];
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LPR;
    pw[i].zero();
    if (c < pieces) pw[i].load(w + 8 * c);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kGroups + group; row < rows;
       row += (int64_t)gridDim.x * kGroups) {
    Piece<TX> pd[NV];
    Piece<TR> pr[NV], po[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = lane + i * LPR;
      pd[i].zero();
      pr[i].zero();
      po[i].zero();
      if (c < pieces) {
        pd[i].load(dy + row * xs + 8 * c);
        pr[i].load(r + row * (int64_t)d + 8 * c);
        if (dr_out) po[i].load(dr_out + row * (int64_t)d + 8 * c);
      }
    }
    float ss = 0.0f, gr = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float fd[8], fr[8], fw[8];
      pd[i].get(fd);
      pr[i].get(fr);
      pw[i].get(fw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss += fr[j] * fr[j];
        gr += fd[j] * fw[j] * fr[j];
      }
    }
    ss = row_reduce<LPR, false>(ss, red, slot);
    gr = row_reduce<LPR, false>(gr, red, slot + 1);
    slot ^= 2;  // the next row's first barrier is passed by all before these are rewritten
    const float rstd = rsqrtf(ss / (float)d + eps);
    const float coef = gr / (float)d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = lane + i * LPR;
      if (c < pieces) {
        float fd[8], fr[8], fw[8], fo[8];
        pd[i].get(fd);
        pr[i].get(fr);
        pw[i].get(fw);
        po[i].get(fo);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[i][j] += fd[j] * (fr[j] * rstd);
          fo[j] += rstd * (fd[j] * fw[j] - fr[j] * coef);
        }
        Piece<TR>::store(dr + row * (int64_t)d + 8 * c, fo);
        if (dx) Piece<TX>::store(dx + row * ys + 8 * c, fo);
      }
    }
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * d;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = lane + i * LPR;
      if (c < pieces) Piece<float>::store(out + 8 * c, acc[i]);
    }
  } else {
    for (int g = 0; g < kGroups; ++g) {
      if (group == g) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = lane + i * LPR;
          if (c < pieces) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sum[8 * c + j] = g == 0 ? acc[i][j] : sum[8 * c + j] + acc[i][j];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += kBlock) out[c] = sum[c];
  }
}

// dw[c] = sum over the partial rows: 64 columns per workgroup, 16 row lanes of
// 16 threads with 4 columns each.
__global__ __launch_bounds__(kBlock) void addnorm_dw_kernel(const float* __restrict__ part,
                                                            float* __restrict__ dw, int64_t blocks,
                                                            int d) {
  __shared__ float4 s[16][16];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + cx * 4;
  float4 a = make_float4(0, 0, 0, 0);
  if (c < d) {
#pragma unroll 4
    for (int64_t b = ry; b < blocks; b += 16) {
      const float4 p = *reinterpret_cast<const float4*>(part + b * d + c);
      a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    }
  }
  s[ry][cx] = a;
  __syncthreads();
  if (ry == 0 && c < d) {
    for (int i = 1; i < 16; ++i) {
      const float4 p = s[i][cx];
      a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    }
    *reinterpret_cast<float4*>(dw + c) = a;
  }
}

// Lanes per row and 8-value pieces per lane of a call.
struct RowShape {
  int lpr, nv;
};

// 16 lanes take rows of up to 128 values; rows of up to 512 a wave.  Longer ones
// (bf16, the backward without dr_out, us with a wave a row / with a workgroup a row;
// the small ones are kernel times, a call is 8 us forward and 15 backward):
//   forward   512 x 1024 3.3 / 3.0,  512 x 2560 4.8 / 3.9,  32768 x 1024 41 / 43,
//             32768 x 1536 78 / 72,  32768 x 2560 129 / 120,  32768 x 4096 204 / 187
//   backward  256 x 2560 9.0 / 7.9,  512 x 2560 9.8 / 10.9,  32768 x 1024 37 / 82,
//             32768 x 2560 102 / 132,  4096 x 4096 38 / 25
// and with fp32 residuals 32768 x 1024 80 / 113, 32768 x 2560 199 / 190, 4096 x 4096
// 49 / 38, all in fp32 77 / 104, 192 / 192, 49 / 37.
// The workgroup shortens the chain of a few rows and has fewer values in a
// lane's registers; the wave needs no barrier and, in the backward, adds four
// rows' sums before they leave the workgroup.
RowShape row_shape(const NormArgs& a, bool backward) {
  const int pieces = (int)(a.d / 8);
  const bool wave = pieces <= 64 || (backward ? pieces <= 320 && a.rows >= 384
                                              : pieces <= 128 && a.rows >= 2048);
  const int lpr = pieces <= 16 ? 16 : wave ? 64 : 256;
  const int need = (pieces + lpr - 1) / lpr;
  const int nv = need <= 1 ? 1 : need <= 2 ? 2 : need <= 3 ? 3 : need <= 5 ? 5 : 8;
  return {lpr, nv};
}

// Calls f with the shape as constants: what row_shape gives in the direction.
template <bool kBackward, typename F>
hipError_t with_shape(const RowShape& s, F&& f) {
#define TTT_SHAPE(L, N) \
  if (s.lpr == L && s.nv == N) return f(std::integral_constant<int, L>{}, std::integral_constant<int, N>{});
  TTT_SHAPE(16, 1)
  TTT_SHAPE(64, 1)
  TTT_SHAPE(64, 2)
  if constexpr (kBackward) {
    TTT_SHAPE(64, 3)
    TTT_SHAPE(64, 5)
  }
  TTT_SHAPE(256, 1)
  TTT_SHAPE(256, 2)
  TTT_SHAPE(256, 3)
  TTT_SHAPE(256, 5)
  TTT_SHAPE(256, 8)
#undef TTT_SHAPE
  return hipErrorInvalidValue;
}

template <typename F>
hipError_t with_types(const NormArgs& a, F&& f) {
  if (a.dt == Dtype::F32) return f(float{}, float{});
  return a.res_dt == Dtype::F32 ? f(uint16_t{}, float{}) : f(uint16_t{}, uint16_t{});
}

}  // namespace

// A launch's threads are counted in 32 bits; calls of more rows take several.
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;

hipError_t launch_addnorm_forward(const NormArgs& a, const void* x, const void* res, const void* w,
                                  void* r, void* y, float* y_scale, hipStream_t s) {
  return with_types(a, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return with_shape<false>(row_shape(a, false), [&](auto lpr, auto nv) {
      constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
      const int64_t per = kBlock / L, most = per * kMaxBlocks;
      const int64_t ys = a.y_stride * (a.fp8 ? 1 : (int64_t)sizeof(TX));
      const int64_t scales = a.grouped ? a.d / kNormScaleGroup : 1;
      const auto go = [&](auto kernel) {
        for (int64_t at = 0; at < a.rows; at += most) {
          const int64_t rows = std::min(a.rows - at, most);
          kernel<<<dim3((unsigned)((rows + per - 1) / per)), kBlock, 0, s>>>(
              static_cast<const TX*>(x) + at * a.x_stride,
              res ? static_cast<const TR*>(res) + at * a.d : nullptr, static_cast<const TX*>(w),
              r ? static_cast<TR*>(r) + at * a.d : nullptr, static_cast<char*>(y) + at * ys,
              y_scale ? y_scale + at * scales : nullptr, rows, (int)a.d, a.x_stride, a.y_stride,
              a.eps, a.grouped);
          const hipError_t e = hipGetLastError();
          if (e != hipSuccess) return e;
        }
        return hipSuccess;
      };
      return a.fp8 ? go(addnorm_forward_kernel<TX, TR, true, L, N>)
                   : go(addnorm_forward_kernel<TX, TR, false, L, N>);
    });
  });
}

// Two workgroups for each CU: the partial sums stay small (512 rows of d) and each
// workgroup walks enough rows to hide them.  Rows of five fp32 pieces a lane or of
// eight pieces need more than 256 registers, one wave a SIMD, so that their
// workgroups run in two turns; the bytes still set their time (with dr_out and an fp32
// residual 32768 x 2560 256 us, 16384 x 9728 488, both 5.2 TB/s; all bf16 134 and
// 246, 5.0 and 5.2).
int64_t addnorm_backward_blocks(const NormArgs& a) {
  const int64_t per = kBlock / row_shape(a, true).lpr;
  return std::min<int64_t>((a.rows + per - 1) / per, 512);
}

hipError_t launch_addnorm_backward(const NormArgs& a, const void* dy, const void* r, const void* w,
                                   const void* dr_out, void* dr, void* dx, float* dw, float* part,
                                   hipStream_t s) {
  const int64_t blocks = addnorm_backward_blocks(a);
  hipError_t e = with_types(a, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return with_shape<true>(row_shape(a, true), [&](auto lpr, auto nv) {
      constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
      const size_t lds = L < kBlock ? (size_t)a.d * sizeof(float) : 0;
      addnorm_backward_kernel<TX, TR, L, N><<<dim3((unsigned)blocks), kBlock, lds, s>>>(
          static_cast<const TX*>(dy), static_cast<const TR*>(r), static_cast<const TX*>(w),
          static_cast<const TR*>(dr_out), static_cast<TR*>(dr), static_cast<TX*>(dx),
          dw ? part : nullptr, a.rows, (int)a.d, a.x_stride, a.y_stride, a.eps);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || !dw) return e;
  addnorm_dw_kernel<<<dim3((unsigned)((a.d + 63) / 64)), kBlock, 0, s>>>(part, dw, blocks,
                                                                         (int)a.d);
  return hipGetLastError();
}

}  // namespace ttt
