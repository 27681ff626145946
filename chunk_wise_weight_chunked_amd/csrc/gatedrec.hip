// gatedrec.hip -- gated linear recurrence and its gradients.
//
//   r = sigmoid(decay_gate), i = sigmoid(input_gate), z = -rate r, a = e^z,
//   b = sqrt(1 - a^2),  u = b i x,  h_t = a_t h_{t-1} + u_t
//
// and for the gradients, from the last token, with c the part of the gradient of
// h_t that comes from behind:
//   l_t = dh_t + c_{t+1},  c_t = a_t l_t
//   dx = l b i,  dinput = l u (1 - i),  y = l (a h_{t-1} - u a^2 / b^2)
//   ddecay = y z (1 - r),  drate = -sum y r
//
// A channel is a chain of its own; the tokens of one are cut into tiles of
// kRecTile, and a tile into runs that a lane holds in registers.  A run, a tile
// or a row of tiles maps the state in front of it to that behind it by
// h -> e^Z h + H with Z the sum of its z: two numbers a channel, that compose.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_core.h"
#include "seq.h"

namespace ttt {
namespace {

constexpr int kBlock = 256;
constexpr int kStrip = 64;  // channels of a tile

// A decay as one float: e^z itself (sign bit clear) or, where z > -1/4, e^z - 1
// (sign bit set, -0 for z = 0).  The second keeps what a decay near 1 loses by its
// rounding, which would be repeated for as long as the channel remembers.
// e^z - 1 = z (1 + z/2 (1 + z/3 (...))) to the sixth power: what is left out is
// below z^6 / 5040 = 5e-8 of it.
__device__ __forceinline__ float decay_of(float z) {
  float p = 1.0f + z * (1.0f / 6.0f);
  p = 1.0f + z * (1.0f / 5.0f) * p;
  p = 1.0f + z * (1.0f / 4.0f) * p;
  p = 1.0f + z * (1.0f / 3.0f) * p;
  p = 1.0f + z * (1.0f / 2.0f) * p;
  return z > -0.25f ? __builtin_copysignf(z * p, -1.0f) : __expf(z);
}
__device__ __forceinline__ bool near_one(float dec) { return __float_as_uint(dec) >> 31; }
// a h + u
__device__ __forceinline__ float decayed(float dec, float h, float u) {
  return __builtin_fmaf(dec, h, u) + (near_one(dec) ? h : 0.0f);
}
// 1 - a^2 = (1 - a)(1 + a)
__device__ __forceinline__ float one_minus_square(float dec) {
  return near_one(dec) ? -dec * (2.0f + dec) : (1.0f - dec) * (1.0f + dec);
}
// z is never positive: a rate below 0 counts as NaN.
__device__ __forceinline__ float rate_at(const float* rate, int64_t c) {
  const float r = rate[c];
  return r >= 0.0f ? r : __builtin_nanf("");
}
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

// kPer values of a lane: 16 bytes.
template <typename T>
struct Lane;
template <>
struct Lane<uint16_t> {
  static constexpr int kPer = 8;
  __device__ __forceinline__ static void put(uint16_t* p, const float f[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Lane<float> {
  static constexpr int kPer = 4;
  __device__ __forceinline__ static void put(float* p, const float f[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <typename T>
__device__ __forceinline__ uint4 get16(const T* p) { return *reinterpret_cast<const uint4*>(p); }

// Lane layout of a tile: kLanes lanes across the strip's channels, kRuns runs of
// kRun tokens.
template <typename T>
struct TileShapeOf {
  static constexpr int kPer = Lane<T>::kPer;
  static constexpr int kLanes = kStrip / kPer;
  static constexpr int kRuns = kBlock / kLanes;
  static constexpr int kRun = kRecTile / kRuns;
};

// Where a workgroup's tile is.
struct TileAt {
  int64_t b, j, strip;
};
__device__ __forceinline__ int64_t tokens_of(const RecArgs& a, int64_t b) {
  if (!a.lengths) return a.T;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// z as its decay and u of one token's channels.
template <typename T>
__device__ __forceinline__ void token(const uint4& vx, const uint4& vg, const uint4& vi,
                                      const float* rate, float* z, float* dec, float* u) {
#pragma unroll
  for (int c = 0; c < Lane<T>::kPer; ++c) {
    z[c] = -rate[c] * sigmoid(chunk_value<T>(vg, c));
    dec[c] = decay_of(z[c]);
    u[c] = sqrtf(one_minus_square(dec[c])) * sigmoid(chunk_value<T>(vi, c)) *
           chunk_value<T>(vx, c);
  }
}

// The recurrent form: a lane walks the tokens of its channels.
template <typename T>
__global__ __launch_bounds__(kBlock) void rec_step_kernel(RecArgs a, const float* s_in,
                                                          float* s_out, T* __restrict__ h,
                                                          int64_t hsb, int64_t hst,
                                                          float* __restrict__ saved) {
  constexpr int kPer = Lane<T>::kPer;
  const int64_t per_row = a.d / kPer;
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i >= a.B * per_row) return;
  const int64_t b = i / per_row, c0 = (i % per_row) * kPer;
  const int64_t n = tokens_of(a, b);
  float s[kPer], rate[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    rate[c] = rate_at(a.rate, c0 + c);
    s[c] = s_in ? s_in[b * a.d + c0 + c] : 0.0f;
  }
  if (saved) {
#pragma unroll
    for (int c = 0; c < kPer; ++c) saved[b * a.d + c0 + c] = s[c];
  }
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.sb + c0;
  const T* g = static_cast<const T*>(a.decay.p) + b * a.decay.sb + c0;
  const T* in = static_cast<const T*>(a.input.p) + b * a.input.sb + c0;
  T* out = h + b * hsb + c0;
  for (int64_t t = 0; t < a.T; ++t) {
    float f[kPer];
    if (t < n) {
      float z[kPer], dec[kPer], u[kPer];
      token<T>(get16(x + t * a.x.st), get16(g + t * a.decay.st), get16(in + t * a.input.st), rate,
               z, dec, u);
#pragma unroll
      for (int c = 0; c < kPer; ++c) f[c] = s[c] = decayed(dec[c], s[c], u[c]);
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) f[c] = 0.0f;
    }
    Lane<T>::put(out + t * hst, f);
  }
  if (s_out) {
#pragma unroll
    for (int c = 0; c < kPer; ++c) s_out[b * a.d + c0 + c] = s[c];
  }
}

// The tile of a workgroup, strips of a tile next to each other.
__device__ __forceinline__ TileAt tile_at(const RecArgs& a, int64_t tiles) {
  const int64_t strips = (a.d + kStrip - 1) / kStrip;
  const int64_t w = blockIdx.x;
  return {(w / strips) / tiles, (w / strips) % tiles, w % strips};
}

// What a lane of a tile works on.
template <typename T>
struct LaneAt {
  int64_t b, j, c0, t0;  // t0: its run's first token
  int lane, run;
  int n;                 // tokens of its run that count
  int rows;              // tokens of its run inside T
  bool live;             // channels inside d
  float rate[Lane<T>::kPer];
};
template <typename T>
__device__ __forceinline__ LaneAt<T> lane_at(const RecArgs& a, const TileAt& at) {
  using S = TileShapeOf<T>;
  LaneAt<T> l;
  l.lane = threadIdx.x % S::kLanes, l.run = threadIdx.x / S::kLanes;
  l.b = at.b, l.j = at.j;
  l.c0 = at.strip * kStrip + l.lane * S::kPer;
  l.t0 = at.j * kRecTile + l.run * S::kRun;
  l.live = l.c0 < a.d;
  const int64_t n = tokens_of(a, at.b);
  l.n = l.live ? (int)min<int64_t>(max<int64_t>(n - l.t0, 0), S::kRun) : 0;
  l.rows = l.live ? (int)min<int64_t>(max<int64_t>(a.T - l.t0, 0), S::kRun) : 0;
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) l.rate[c] = l.live ? rate_at(a.rate, l.c0 + c) : 0.0f;
  return l;
}
template <typename T>
__device__ __forceinline__ const T* row_of(const RecOperand& o, const LaneAt<T>& l) {
  return static_cast<const T*>(o.p) + l.b * o.sb + l.t0 * o.st + l.c0;
}

// z sums and states (from 0) of a workgroup's runs, by run and channel.
template <typename T>
struct RunSums {
  float z[TileShapeOf<T>::kRuns][kStrip], h[TileShapeOf<T>::kRuns][kStrip];
};

// A run's decays and u; its sum of z and its state from 0.
template <typename T>
__device__ __forceinline__ void load_run(const RecArgs& a, const LaneAt<T>& l,
                                         float dec[][Lane<T>::kPer], float u[][Lane<T>::kPer],
                                         float* Z, float* H) {
  using S = TileShapeOf<T>;
  uint4 vx[S::kRun], vg[S::kRun], vi[S::kRun];
  const T *x = row_of<T>(a.x, l), *g = row_of<T>(a.decay, l), *in = row_of<T>(a.input, l);
#pragma unroll
  for (int t = 0; t < S::kRun; ++t)
    if (t < l.n) {
      vx[t] = get16(x + t * a.x.st);
      vg[t] = get16(g + t * a.decay.st);
      vi[t] = get16(in + t * a.input.st);
    }
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) Z[c] = -0.0f, H[c] = 0.0f;
#pragma unroll
  for (int t = 0; t < S::kRun; ++t) {
    float z[S::kPer];
    if (t < l.n) {
      token<T>(vx[t], vg[t], vi[t], l.rate, z, dec[t], u[t]);
    } else {
#pragma unroll
      for (int c = 0; c < S::kPer; ++c) z[c] = -0.0f, dec[t][c] = -0.0f, u[t][c] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) {
      Z[c] += z[c];
      H[c] = decayed(dec[t][c], H[c], u[t][c]);
    }
  }
}

// Each tile's sum of z and state from 0: sums [B][tiles][d] of (Z, H).
template <typename T>
__global__ __launch_bounds__(kBlock) void rec_sums_kernel(RecArgs a, int64_t tiles,
                                                          float2* __restrict__ sums) {
  using S = TileShapeOf<T>;
  __shared__ RunSums<T> rs;
  const TileAt at = tile_at(a, tiles);
  const LaneAt<T> l = lane_at<T>(a, at);
  float dec[S::kRun][S::kPer], u[S::kRun][S::kPer], Z[S::kPer], H[S::kPer];
  load_run<T>(a, l, dec, u, Z, H);
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) {
    rs.z[l.run][l.lane * S::kPer + c] = Z[c];
    rs.h[l.run][l.lane * S::kPer + c] = H[c];
  }
  __syncthreads();
  const int64_t ch = at.strip * kStrip + threadIdx.x;
  if (threadIdx.x >= kStrip || ch >= a.d) return;
  float z = -0.0f, h = 0.0f;
  for (int r = 0; r < S::kRuns; ++r) {
    h = decayed(decay_of(rs.z[r][threadIdx.x]), h, rs.h[r][threadIdx.x]);
    z += rs.z[r][threadIdx.x];
  }
  sums[(at.b * tiles + at.j) * a.d + ch] = make_float2(z, h);
}

// The state in front of every tile, and behind the last (backward: the gradient
// that comes from behind every tile, and in front of the first).
__global__ __launch_bounds__(kBlock) void rec_scan_kernel(const float2* __restrict__ sums,
                                                          const float* s_in, float* s_out,
                                                          float* __restrict__ starts, int64_t B,
                                                          int64_t tiles, int64_t d, bool reverse) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i >= B * d) return;
  const int64_t b = i / d, ch = i % d;
  float s = s_in ? s_in[i] : 0.0f;
  for (int64_t k = 0; k < tiles; ++k) {
    const int64_t j = reverse ? tiles - 1 - k : k;
    const int64_t o = (b * tiles + j) * d + ch;
    starts[o] = s;
    const float2 f = sums[o];
    s = decayed(decay_of(f.x), s, f.y);
  }
  if (s_out) s_out[i] = s;
}

// The outputs of a tile from the state in front of it.
template <typename T>
__global__ __launch_bounds__(kBlock) void rec_apply_kernel(RecArgs a, int64_t tiles,
                                                           const float* __restrict__ starts,
                                                           T* __restrict__ h, int64_t hsb,
                                                           int64_t hst) {
  using S = TileShapeOf<T>;
  __shared__ RunSums<T> rs;
  const TileAt at = tile_at(a, tiles);
  const LaneAt<T> l = lane_at<T>(a, at);
  float dec[S::kRun][S::kPer], u[S::kRun][S::kPer], Z[S::kPer], H[S::kPer];
  load_run<T>(a, l, dec, u, Z, H);
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) {
    rs.z[l.run][l.lane * S::kPer + c] = Z[c];
    rs.h[l.run][l.lane * S::kPer + c] = H[c];
  }
  __syncthreads();
  const int64_t ch = at.strip * kStrip + threadIdx.x;
  if (threadIdx.x < kStrip && ch < a.d) {
    float s = starts[(at.b * tiles + at.j) * a.d + ch];
    for (int r = 0; r < S::kRuns; ++r) {
      const float next = decayed(decay_of(rs.z[r][threadIdx.x]), s, rs.h[r][threadIdx.x]);
      rs.h[r][threadIdx.x] = s;  // the state in front of the run
      s = next;
    }
  }
  __syncthreads();
  if (l.rows == 0) return;
  float s[S::kPer];
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) s[c] = rs.h[l.run][l.lane * S::kPer + c];
  T* out = h + l.b * hsb + l.t0 * hst + l.c0;
#pragma unroll
  for (int t = 0; t < S::kRun; ++t) {
    if (t >= l.rows) break;
    float f[S::kPer];
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) {
      s[c] = decayed(dec[t][c], s[c], u[t][c]);
      f[c] = t < l.n ? s[c] : 0.0f;
    }
    Lane<T>::put(out + t * hst, f);
  }
}

// Each tile's sum of z and gradient from behind, from 0, in front of it.
template <typename T>
__global__ __launch_bounds__(kBlock) void rec_back_sums_kernel(RecArgs a, int64_t tiles,
                                                               float2* __restrict__ sums) {
  using S = TileShapeOf<T>;
  __shared__ RunSums<T> rs;
  const TileAt at = tile_at(a, tiles);
  const LaneAt<T> l = lane_at<T>(a, at);
  const T *g = row_of<T>(a.decay, l), *dh = row_of<T>(a.dh, l);
  float Z[S::kPer], C[S::kPer];
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) Z[c] = -0.0f, C[c] = 0.0f;
#pragma unroll
  for (int t = S::kRun - 1; t >= 0; --t) {
    if (t >= l.n) continue;
    const uint4 vg = get16(g + t * a.decay.st), vd = get16(dh + t * a.dh.st);
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) {
      const float z = -l.rate[c] * sigmoid(chunk_value<T>(vg, c));
      Z[c] += z;
      C[c] = decayed(decay_of(z), C[c] + chunk_value<T>(vd, c), 0.0f);
    }
  }
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) {
    rs.z[l.run][l.lane * S::kPer + c] = Z[c];
    rs.h[l.run][l.lane * S::kPer + c] = C[c];
  }
  __syncthreads();
  const int64_t ch = at.strip * kStrip + threadIdx.x;
  if (threadIdx.x >= kStrip || ch >= a.d) return;
  float z = -0.0f, h = 0.0f;
  for (int r = S::kRuns - 1; r >= 0; --r) {
    h = decayed(decay_of(rs.z[r][threadIdx.x]), h, rs.h[r][threadIdx.x]);
    z += rs.z[r][threadIdx.x];
  }
  sums[(at.b * tiles + at.j) * a.d + ch] = make_float2(z, h);
}

// The gradients of a tile, from the saved state in front of it and the gradient
// that comes from behind it; the tile's sums of drate in `part` [B][tiles][d].
template <typename T>
__global__ __launch_bounds__(kBlock) void rec_back_kernel(RecArgs a, int64_t tiles,
                                                          const float* __restrict__ saved,
                                                          const float* __restrict__ behind,
                                                          T* __restrict__ dx, T* __restrict__ dg,
                                                          T* __restrict__ di,
                                                          float* __restrict__ part) {
  using S = TileShapeOf<T>;
  __shared__ RunSums<T> rs;
  __shared__ float back[S::kRuns][kStrip];
  const TileAt at = tile_at(a, tiles);
  const LaneAt<T> l = lane_at<T>(a, at);
  float dec[S::kRun][S::kPer], u[S::kRun][S::kPer], Z[S::kPer], H[S::kPer];
  load_run<T>(a, l, dec, u, Z, H);
  const T *x = row_of<T>(a.x, l), *g = row_of<T>(a.decay, l), *in = row_of<T>(a.input, l),
          *dh = row_of<T>(a.dh, l);
  float C[S::kPer];
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) C[c] = 0.0f;
#pragma unroll
  for (int t = S::kRun - 1; t >= 0; --t) {
    if (t >= l.n) continue;
    const uint4 vd = get16(dh + t * a.dh.st);
#pragma unroll
    for (int c = 0; c < S::kPer; ++c)
      C[c] = decayed(dec[t][c], C[c] + chunk_value<T>(vd, c), 0.0f);
  }
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) {
    const int k = l.lane * S::kPer + c;
    rs.z[l.run][k] = Z[c], rs.h[l.run][k] = H[c], back[l.run][k] = C[c];
  }
  __syncthreads();
  const int64_t ch = at.strip * kStrip + threadIdx.x;
  const int64_t o = (at.b * tiles + at.j) * a.d + ch;
  if (threadIdx.x < kStrip && ch < a.d) {
    float s = saved[o], c = behind[o];
    for (int r = 0; r < S::kRuns; ++r) {
      const float next = decayed(decay_of(rs.z[r][threadIdx.x]), s, rs.h[r][threadIdx.x]);
      rs.h[r][threadIdx.x] = s;
      s = next;
    }
    for (int r = S::kRuns - 1; r >= 0; --r) {
      const float next = decayed(decay_of(rs.z[r][threadIdx.x]), c, back[r][threadIdx.x]);
      back[r][threadIdx.x] = c;
      c = next;
    }
  }
  __syncthreads();
  float s[S::kRun][S::kPer], c[S::kPer], dr[S::kPer];  // s: the state in front of a token
#pragma unroll
  for (int k = 0; k < S::kPer; ++k) {
    float f = rs.h[l.run][l.lane * S::kPer + k];
    c[k] = back[l.run][l.lane * S::kPer + k];
    dr[k] = 0.0f;
#pragma unroll
    for (int t = 0; t < S::kRun; ++t) {
      s[t][k] = f;
      f = decayed(dec[t][k], f, u[t][k]);
    }
  }
  const int64_t row = (l.b * a.T + l.t0) * a.d + l.c0;
#pragma unroll
  for (int t = S::kRun - 1; t >= 0; --t) {
    if (t >= l.rows) continue;
    float fx[S::kPer], fg[S::kPer], fi[S::kPer];
    if (t < l.n) {
      const uint4 vx = get16(x + t * a.x.st), vg = get16(g + t * a.decay.st),
                  vi = get16(in + t * a.input.st), vd = get16(dh + t * a.dh.st);
#pragma unroll
      for (int k = 0; k < S::kPer; ++k) {
        const float r = sigmoid(chunk_value<T>(vg, k)), i = sigmoid(chunk_value<T>(vi, k));
        const float lam = chunk_value<T>(vd, k) + c[k];
        const float bb = one_minus_square(dec[t][k]), bi = sqrtf(bb) * i;
        // y = l (a h - u a^2 / b^2)
        const float al = decayed(dec[t][k], lam, 0.0f);
        const float ua = bb > 0.0f ? decayed(dec[t][k], u[t][k], 0.0f) / bb : 0.0f;
        const float y = al * (s[t][k] - ua);
        fx[k] = lam * bi;
        fi[k] = fx[k] * chunk_value<T>(vx, k) * (1.0f - i);
        fg[k] = -y * l.rate[k] * r * (1.0f - r);
        dr[k] -= y * r;
        c[k] = al;
      }
    } else {
#pragma unroll
      for (int k = 0; k < S::kPer; ++k) fx[k] = fg[k] = fi[k] = 0.0f;
    }
    Lane<T>::put(dx + row + t * a.d, fx);
    Lane<T>::put(dg + row + t * a.d, fg);
    Lane<T>::put(di + row + t * a.d, fi);
  }
  __syncthreads();  // rs.z is read no more
#pragma unroll
  for (int k = 0; k < S::kPer; ++k) rs.z[l.run][l.lane * S::kPer + k] = dr[k];
  __syncthreads();
  if (threadIdx.x < kStrip && ch < a.d) {
    float f = 0.0f;
    for (int r = 0; r < S::kRuns; ++r) f += rs.z[r][threadIdx.x];
    part[o] = f;
  }
}

// out[c] = sum over rows of part [rows][d]: 64 columns a workgroup, 16 lanes of
// rows.
__global__ __launch_bounds__(kBlock) void rec_rate_kernel(const float* __restrict__ part,
                                                          float* __restrict__ out, int64_t rows,
                                                          int64_t d) {
  __shared__ float4 s[16][16];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int64_t c = blockIdx.x * (int64_t)64 + cx * 4;
  float4 a = make_float4(0, 0, 0, 0);
  if (c < d) {
#pragma unroll 4
    for (int64_t r = ry; r < rows; r += 16) {
      const float4 p = *reinterpret_cast<const float4*>(part + r * d + c);
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
    *reinterpret_cast<float4*>(out + c) = a;
  }
}

int64_t tiles_of(const RecArgs& a) { return (a.T + kRecTile - 1) / kRecTile; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <typename F>
hipError_t with_type(Dtype dt, F&& f) {
  return dt == Dtype::F32 ? f(float{}) : f(uint16_t{});
}

}  // namespace

// The tiles' sums, and the states in front of the tiles where they are not saved.
size_t gatedrec_forward_bytes(const RecArgs& a) {
  if (a.T <= kRecStepTokens) return 0;
  const size_t n = (size_t)(a.B * tiles_of(a) * a.d);
  return align256(n * sizeof(float2)) + n * sizeof(float);
}

hipError_t launch_gatedrec_forward(const RecArgs& a, const float* s_in, float* s_out, void* h,
                                   int64_t hsb, int64_t hst, float* saved, void* ws,
                                   hipStream_t s) {
  return with_type(a.dt, [&](auto t) {
    using T = decltype(t);
    T* out = static_cast<T*>(h);
    if (a.T <= kRecStepTokens) {
      const int64_t n = a.B * (a.d / Lane<T>::kPer);
      rec_step_kernel<T><<<dim3((unsigned)((n + kBlock - 1) / kBlock)), kBlock, 0, s>>>(
          a, s_in, s_out, out, hsb, hst, saved);
      return hipGetLastError();
    }
    const int64_t tiles = tiles_of(a), n = a.B * tiles * a.d;
    float2* sums = static_cast<float2*>(ws);
    float* starts = saved ? saved
                          : reinterpret_cast<float*>(static_cast<char*>(ws) +
                                                     align256(n * sizeof(float2)));
    const dim3 grid((unsigned)(a.B * tiles * ((a.d + kStrip - 1) / kStrip)));
    rec_sums_kernel<T><<<grid, kBlock, 0, s>>>(a, tiles, sums);
    rec_scan_kernel<<<dim3((unsigned)((a.B * a.d + kBlock - 1) / kBlock)), kBlock, 0, s>>>(
        sums, s_in, s_out, starts, a.B, tiles, a.d, false);
    rec_apply_kernel<T><<<grid, kBlock, 0, s>>>(a, tiles, starts, out, hsb, hst);
    return hipGetLastError();
  });
}

size_t gatedrec_backward_bytes(const RecArgs& a) {
  const size_t n = (size_t)(a.B * tiles_of(a) * a.d);
  return align256(n * sizeof(float2)) + 2 * align256(n * sizeof(float));
}

hipError_t launch_gatedrec_backward(const RecArgs& a, const float* saved, const float* ds_out,
                                    void* dx, void* ddecay, void* dinput, float* drate,
                                    float* ds_in, void* ws, hipStream_t s) {
  return with_type(a.dt, [&](auto t) {
    using T = decltype(t);
    const int64_t tiles = tiles_of(a), n = a.B * tiles * a.d;
    char* const base = static_cast<char*>(ws);
    float2* sums = reinterpret_cast<float2*>(base);
    float* behind = reinterpret_cast<float*>(base + align256(n * sizeof(float2)));
    float* part = reinterpret_cast<float*>(base + align256(n * sizeof(float2)) +
                                           align256(n * sizeof(float)));
    const dim3 grid((unsigned)(a.B * tiles * ((a.d + kStrip - 1) / kStrip)));
    rec_back_sums_kernel<T><<<grid, kBlock, 0, s>>>(a, tiles, sums);
    rec_scan_kernel<<<dim3((unsigned)((a.B * a.d + kBlock - 1) / kBlock)), kBlock, 0, s>>>(
        sums, ds_out, ds_in, behind, a.B, tiles, a.d, true);
    rec_back_kernel<T><<<grid, kBlock, 0, s>>>(a, tiles, saved, behind, static_cast<T*>(dx),
                                               static_cast<T*>(ddecay), static_cast<T*>(dinput),
                                               part);
    rec_rate_kernel<<<dim3((unsigned)((a.d + 63) / 64)), kBlock, 0, s>>>(part, drate, a.B * tiles,
                                                                         a.d);
    return hipGetLastError();
  });
}

}  // namespace ttt
