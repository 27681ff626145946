// gatedrec.hip -- gated linear recurrence and its gradients.
//
//   r = sigmoid(decay_gate), i = sigmoid(input_gate), z = -rate r, a = e^z,
//   b = sqrt(1 - a^2),  u = b i x,  h_t = a_t h_{t-1} + u_t
//
// and for the gradients, from the last token, with c the part of the gradient of
// h_t that comes from behind:
//   l_t = dh_t + c_{t+1},  c_t = a_t l_t
//   dx = l b i,  dinput = l u (1 - i),  y = l a (h_{t-1} - i x a / b)
//   ddecay = y z (1 - r),  drate = -sum y r
//
// A channel is a chain of its own; the tokens of one are cut into tiles of
// kRecTile, and a tile into runs that a lane holds in registers.  A run, a tile
// or a row of tiles maps the state in front of it to that behind it by
// h -> e^Z h + H with Z the sum of its z: two numbers a channel, that compose.
//
// Both directions are bound by HBM and read their inputs once: a workgroup loads a
// tile, publishes its map, takes the state in front of it from the tiles in front (through
// their maps, from the nearest place whose state is known) and writes the tile's
// results from its registers.  2560 channels in bf16: 131072 tokens 523 us, 5.1 TB/s; 32768
// forward 143 us, backward 252 us, 4.7 TB/s with a vector instruction at work in 79% of the
// SIMDs' cycles; in fp32 240 and 428 us, 5.6 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_core.h"
#include "rec_link.h"
#include "seq.h"

namespace ttt {
namespace {

constexpr int kBlock = 256;
// Channels of a tile.  Rows of 256 bytes are read and written faster than rows of 128: the
// forward takes 128 channels in bf16 where there are more than 64 (131072 tokens of 2560 523 us,
// 580 with 64) and 64 in fp32 (65536 tokens 465 us, 480 with 128).  The backward takes 64: with
// its registers a tile of 128 has a CU for itself (32768 tokens 252 us, 312 with 128; in tiles
// of 64 tokens, of which 128 channels take no more, 260: it is the vector units that bound it).
constexpr int kStrip = 64, kWideStrip = 128, kFewChannels = 64;

// 2^64 (1 - a^2) from a and its z: near a = 1 by the same polynomial of 2 z.  The roots'
// instructions take values below 2^-126 as 0, which 2^64 times the smallest is not: b
// comes as 2^32 b, its inverse as 2^-32 / b.
// floor: what it is at least.
__device__ __forceinline__ float root_arg(float z, float a, float floor) {
  float p = __builtin_fmaf(z, -0x1.2ee444p+59f, -0x1.38ae68p+61f);
  p = __builtin_fmaf(z, p, -0x1.c6947ap+62f);
  p = __builtin_fmaf(z, p, -0x1.ebfb70p+63f);
  p = __builtin_fmaf(z, p, -0x1.62e430p+64f);
  const float near = __builtin_fmaf(z, p, floor), far = __builtin_fmaf(-a, a, 1.0f) * 0x1p64f;
  return z > -0.25f ? near : far;
}

__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}
// b i from z, a and the input gate.  The root's 2^32 is taken off b, which is never below 2^-75,
// and not off i, which may be any normal number (2^-126 at a gate of -87).
__device__ __forceinline__ float gated(float z, float a, float gate) {
  return __builtin_amdgcn_sqrtf(root_arg(z, a, 0.0f)) * 0x1p-32f * sigmoid(gate);
}

// Two values as bf16 (RNE), by one instruction.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{lo, hi}, b2));
}

// kPer values of a lane: 16 bytes.
template <typename T>
struct Lane;
template <>
struct Lane<uint16_t> {
  static constexpr int kPer = 8;
  __device__ __forceinline__ static uint32_t word(const float f[2]) { return pack2(f[0], f[1]); }
  __device__ __forceinline__ static void put(uint16_t* p, const float f[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                                              pack2(f[6], f[7]));
  }
};
template <>
struct Lane<float> {
  static constexpr int kPer = 4;
  __device__ __forceinline__ static uint32_t word(const float f[1]) { return __float_as_uint(f[0]); }
  __device__ __forceinline__ static void put(float* p, const float f[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
// A decay gate of -infinity in every channel: a token that neither decays nor enters.
template <typename T>
__device__ __forceinline__ uint4 no_token() {
  constexpr uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  return make_uint4(w, w, w, w);
}
template <typename T>
__device__ __forceinline__ uint4 get16(const T* p) { return *reinterpret_cast<const uint4*>(p); }

// Lane layout of a tile of kStrip channels on kThreads: kLanes lanes across the channels,
// kRuns runs of kRun tokens.  kRecTile tokens have 4 threads a channel; a call of fewer tokens
// than a half or a quarter of that, one tile a sequence, as many fewer.
template <typename T_, int kStrip_, int kThreads_>
struct TileLayout {
  using T = T_;
  static constexpr int kStrip = kStrip_, kThreads = kThreads_;
  static constexpr int kPer = Lane<T>::kPer;
  static constexpr int kLanes = kStrip / kPer;
  static constexpr int kRuns = kThreads / kLanes;
  static constexpr int kTile = kRecTile * kThreads / (4 * kStrip);  // tokens
  static constexpr int kRun = kTile / kRuns;
  static constexpr int kParts = kThreads / kStrip;  // a thread a channel, each folds kRuns / kParts runs
};

__device__ __forceinline__ int64_t tokens_of(const RecArgs& a, int64_t b) {
  if (!a.lengths) return a.T;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// The recurrent form: a lane walks the tokens of its channels, kStepAhead loaded at a time
// (64 sessions' next token of 2560 channels: 5.5 us, the latency of one load behind another).
constexpr int kStepAhead = 4;
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
    rate[c] = log_rate(a.rate[c0 + c]);
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
  for (int64_t t0 = 0; t0 < a.T; t0 += kStepAhead) {
    uint4 vx[kStepAhead], vg[kStepAhead], vi[kStepAhead];
#pragma unroll
    for (int i = 0; i < kStepAhead; ++i) {
      vx[i] = vg[i] = vi[i] = make_uint4(0, 0, 0, 0);
      if (t0 + i < n) {
        vx[i] = get16(x + (t0 + i) * a.x.st);
        vg[i] = get16(g + (t0 + i) * a.decay.st);
        vi[i] = get16(in + (t0 + i) * a.input.st);
      }
    }
#pragma unroll
    for (int i = 0; i < kStepAhead; ++i) {
      if (t0 + i >= a.T) break;
      if (t0 + i >= n) {
        *reinterpret_cast<uint4*>(out + (t0 + i) * hst) = make_uint4(0, 0, 0, 0);
        continue;
      }
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const float z = rate[c] * sigmoid(chunk_value<T>(vg[i], c));
        const float u = gated(z, __builtin_amdgcn_exp2f(z), chunk_value<T>(vi[i], c));
        s[c] = decayed(decay_of(z), s[c], u * chunk_value<T>(vx[i], c));
      }
      Lane<T>::put(out + (t0 + i) * hst, s);
    }
  }
  if (s_out) {
#pragma unroll
    for (int c = 0; c < kPer; ++c) s_out[b * a.d + c0 + c] = s[c];
  }
}

// ------------------------------------------------- tiles and what links them
// How words come and go between workgroups (rec_link.h).
struct DeviceWords {
  __device__ __forceinline__ static void put(uint64_t* p, uint64_t w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ static uint64_t get(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ static void pause() { __builtin_amdgcn_s_sleep(1); }
};

// Words unset, the counter of begun tiles at 0.
__global__ __launch_bounds__(kBlock) void rec_clear_kernel(uint4* __restrict__ words, int64_t n,
                                                           uint32_t* __restrict__ begun) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *begun = 0;
  const int64_t step = (int64_t)gridDim.x * kBlock;
  for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < n; i += step)
    words[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// The workgroup's tile.  Tiles are handed out in the order in which workgroups begin,
// those of all sequences and strips at one place before those behind it (backward: in
// front of it): every tile that this one waits for is at work already, and the first
// of a sequence waits for none, so that all waits end whatever the order of workgroups.
template <class S>
__device__ __forceinline__ TileAt tile_at(const RecArgs& a, const Links& links, bool reverse) {
  __shared__ uint32_t ticket;
  uint32_t w = blockIdx.x;
  if (links.maps) {
    if (threadIdx.x == 0)
      ticket = __hip_atomic_fetch_add(links.begun, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    w = __builtin_amdgcn_readfirstlane(ticket);  // so that what follows from it is scalar
  }
  const uint32_t strips = (uint32_t)((a.d + S::kStrip - 1) / S::kStrip), row = strips * (uint32_t)a.B;
  w = min(w, gridDim.x - 1);  // whatever happens to the counter, a tile of this call
  TileAt at;
  at.k = w / row;
  at.b = w % row / strips;
  at.strip = w % strips;
  at.j = reverse ? links.tiles - 1 - at.k : at.k;
  return at;
}

// What a lane of a tile works on.
template <class S>
struct LaneAt {
  int64_t b, j, c0, t0;  // t0: its run's first token
  int64_t last;          // the last token that counts (0 if none does), from t0
  int lane, run;
  bool live;             // channels inside d; others work on the first ones' and put nothing
  bool whole;            // the same for the workgroup: all tokens of the tile count
  int n;                 // tokens of its run that count
  int rows;              // tokens of its run inside T
  float rate[S::kPer];   // as given
};
template <class S>
__device__ __forceinline__ LaneAt<S> lane_at(const RecArgs& a, const TileAt& at) {
  LaneAt<S> l;
  l.lane = threadIdx.x % S::kLanes, l.run = threadIdx.x / S::kLanes;
  l.b = at.b, l.j = at.j;
  const int64_t c0 = at.strip * S::kStrip + l.lane * S::kPer;
  l.live = c0 < a.d;
  l.c0 = l.live ? c0 : 0;
  l.t0 = at.j * S::kTile + l.run * S::kRun;
  const int64_t n = tokens_of(a, at.b);
  const auto inside = [&](int64_t end) {
    const int64_t left = end - l.t0;
    return left < 0 ? 0 : left < S::kRun ? (int)left : S::kRun;
  };
  l.whole = (at.j + 1) * S::kTile <= n;
  l.last = (n > 0 ? n - 1 : 0) - l.t0;
  l.n = inside(n), l.rows = inside(a.T);
#pragma unroll
  for (int c = 0; c < S::kPer; c += 4) {
    const float4 r = *reinterpret_cast<const float4*>(a.rate + l.c0 + c);
    l.rate[c] = r.x, l.rate[c + 1] = r.y, l.rate[c + 2] = r.z, l.rate[c + 3] = r.w;
  }
  return l;
}
// f(whole): the code of a tile of which all tokens count, and that of the others.  Each for
// itself up to its sums, so that the work on the first tokens begins when they are there:
// where the two meet behind the loads, the compiler waits for all of them.
template <class S, class F>
__device__ __forceinline__ void on_run(const LaneAt<S>& l, F&& f) {
  if (l.whole)
    f(std::true_type{});
  else
    f(std::false_type{});
}
// load(t, i) for a run's tokens t, of which it reads the i-th from t0, and none(t) for those
// that do not count.  All loads come first, without a branch between them: where a token does
// not count they read the last one that does (or row 0 of a sequence without tokens) for nothing.
template <bool kWhole, class S, class Load, class None>
__device__ __forceinline__ void load_tokens(const LaneAt<S>& l, Load&& load, None&& none) {
#pragma unroll
  for (int t = 0; t < S::kRun; ++t) load(t, kWhole || t < l.last ? t : l.last);
  if constexpr (!kWhole) {
#pragma unroll
    for (int t = 0; t < S::kRun; ++t)
      if (t >= l.n) none(t);
  }
  __builtin_amdgcn_sched_barrier(0);
}
// log_rate of a channel, behind the tokens' loads (and not waited for in front of them).
template <class S>
__device__ __forceinline__ float rate_after(const LaneAt<S>& l, int c) {
  float r = l.rate[c];
  asm volatile("" : "+v"(r));
  return log_rate(r);
}
// put(t) for a run's tokens, none(t) for the rows behind the last token, as far as T.
template <class S, class Put, class None>
__device__ __forceinline__ void put_tokens(const LaneAt<S>& l, Put&& put, None&& none) {
  if (!l.live) return;
  if (l.whole) {
#pragma unroll
    for (int t = 0; t < S::kRun; ++t) put(t);
  } else {
#pragma unroll
    for (int t = 0; t < S::kRun; ++t) {
      if (t < l.n)
        put(t);
      else if (t < l.rows)
        none(t);
    }
  }
}
template <class S>
__device__ __forceinline__ const typename S::T* row_of(const RecOperand& o, const LaneAt<S>& l) {
  return static_cast<const typename S::T*>(o.p) + l.b * o.sb + l.t0 * o.st + l.c0;
}

// The runs of a tile in LDS, by run and channel: decays over a run and states behind
// it from 0, sums of z.  A part of the threads, one a channel, folds kEach.
template <class S>
struct alignas(16) Runs {
  static constexpr int kEach = S::kRuns / S::kParts;
  float z[S::kRuns][S::kStrip], dec[S::kRuns][S::kStrip], h[S::kRuns][S::kStrip];
  float part_z[S::kParts][S::kStrip], part_h[S::kParts][S::kStrip];
};

// A lane's run into LDS.
template <class S>
__device__ __forceinline__ void put_run(Runs<S>& rs, const LaneAt<S>& l, const float* Z,
                                        const float* H) {
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) {
    const int k = l.lane * S::kPer + c;
    rs.z[l.run][k] = Z[c], rs.dec[l.run][k] = decay_of(Z[c]), rs.h[l.run][k] = H[c];
  }
}

// From the runs in LDS to the state in front of each run, which takes the place of its
// h: the parts fold their runs, the first part folds the parts' and links the tile with
// the ones before it, the parts go through their runs once more.  first: the state of
// the channel in front of the first tile; done(channel, state in front of the tile,
// state behind it) in the first part; beside(channel) in the last one, meanwhile if it is another.
template <bool kReverse, class S, class First, class Done, class Beside>
__device__ __forceinline__ void link_tile(Runs<S>& rs, const RecArgs& a, const Links& links,
                                          const TileAt& at, First&& first, Done&& done,
                                          Beside&& beside) {
  constexpr int kParts = S::kParts, kEach = Runs<S>::kEach;
  const int ch = threadIdx.x % S::kStrip, part = threadIdx.x / S::kStrip;
  const auto run = [&](int i) { return kReverse ? S::kRuns - 1 - i : i; };
  __syncthreads();
  float z = -0.0f, h = 0.0f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = run(part * kEach + i);
    h = decayed(rs.dec[r][ch], h, rs.h[r][ch]);
    z += rs.z[r][ch];
  }
  rs.part_z[part][ch] = z, rs.part_h[part][ch] = h;
  __syncthreads();
  const int64_t c = at.strip * S::kStrip + ch;
  if (part == 0 && c < a.d) {
    float dec[kParts], z = -0.0f, ph = 0.0f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const float zp = rs.part_z[p][ch];
      dec[p] = decay_of(zp);
      ph = decayed(dec[p], ph, rs.part_h[p][ch]);
      z += zp;
    }
    const float whole = decay_of(z);
    float s = links.maps ? link<DeviceWords>(links, at, a.d, c, whole, ph, first) : first(c);
    const float before = s;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const float next = decayed(dec[p], s, rs.part_h[p][ch]);
      rs.part_h[p][ch] = s;  // the state in front of the part
      s = next;
    }
    done(c, before, decayed(whole, before, ph));
  }
  if (part == kParts - 1 && c < a.d) beside(c);
  __syncthreads();
  float s = rs.part_h[part][ch];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = run(part * kEach + i);
    const float next = decayed(rs.dec[r][ch], s, rs.h[r][ch]);
    rs.h[r][ch] = s;
    s = next;
  }
  __syncthreads();
}

// A tile's outputs.
template <typename T, int kStrip, int kThreads>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 ? 4 : 3))) void
rec_forward_kernel(RecArgs a, Links links, const float* s_in, float* s_out, T* __restrict__ h,
                   int64_t hsb, int64_t hst, float* __restrict__ saved) {
  using S = TileLayout<T, kStrip, kThreads>;
  __shared__ Runs<S> rs;
  const TileAt at = tile_at<S>(a, links, false);
  const LaneAt<S> l = lane_at<S>(a, at);
  // Inside a run of a few tokens a itself will do; from run to run the sum of z counts.
  float dec[S::kRun][S::kPer], u[S::kRun][S::kPer], Z[S::kPer], H[S::kPer];
  on_run(l, [&](auto whole) {
    uint4 vx[S::kRun], vg[S::kRun], vi[S::kRun];
    const T *x = row_of(a.x, l), *g = row_of(a.decay, l), *in = row_of(a.input, l);
    load_tokens<whole>(l, [&](int t, int64_t i) {
      vg[t] = get16(g + i * a.decay.st);
      vi[t] = get16(in + i * a.input.st);
      vx[t] = get16(x + i * a.x.st);
    }, [&](int t) {
      vg[t] = no_token<T>();
      vx[t] = vi[t] = make_uint4(0, 0, 0, 0);
    });
    float rate[S::kPer];
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) {
      rate[c] = rate_after(l, c);
      Z[c] = -0.0f, H[c] = 0.0f;
    }
#pragma unroll
    for (int t = 0; t < S::kRun; ++t) {
      __builtin_amdgcn_sched_barrier(0);  // one token after the other, as they come
#pragma unroll
      for (int c = 0; c < S::kPer; ++c) {
        const float z = rate[c] * sigmoid(chunk_value<T>(vg[t], c));
        dec[t][c] = __builtin_amdgcn_exp2f(z);
        u[t][c] = gated(z, dec[t][c], chunk_value<T>(vi[t], c)) * chunk_value<T>(vx[t], c);
        Z[c] += z;
        H[c] = __builtin_fmaf(dec[t][c], H[c], u[t][c]);
      }
    }
  });
  put_run(rs, l, Z, H);
  link_tile<false>(
      rs, a, links, at, [&](int64_t c) { return s_in ? s_in[at.b * a.d + c] : 0.0f; },
      [&](int64_t c, float before, float behind) {
        if (saved) saved[(at.b * links.tiles + at.j) * a.d + c] = before;
        if (s_out && at.k + 1 == links.tiles) s_out[at.b * a.d + c] = behind;
      },
      [](int64_t) {});
  float s[S::kPer];
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) s[c] = rs.h[l.run][l.lane * S::kPer + c];
  T* out = h + l.b * hsb + l.t0 * hst + l.c0;
  put_tokens(l, [&](int t) {
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) s[c] = __builtin_fmaf(dec[t][c], s[c], u[t][c]);
    Lane<T>::put(out + t * hst, s);
  }, [&](int t) { *reinterpret_cast<uint4*>(out + t * hst) = make_uint4(0, 0, 0, 0); });
}

// The gradients of a tile, from the saved state in front of it; the tile's sums of
// drate in `part` [B][tiles][d].  A lane holds its tokens' x and dh as loaded, and their
// r and b i; it goes through its channels one after the other at the end, so that
// the states and results of few are in registers beside them.
template <typename T, int kStrip, int kThreads>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 ? 3 : 2))) void
rec_backward_kernel(RecArgs a, Links links, const float* __restrict__ saved, const float* ds_out,
                    float* ds_in, T* __restrict__ dx, T* __restrict__ dg, T* __restrict__ di,
                    float* __restrict__ part) {
  using S = TileLayout<T, kStrip, kThreads>;
  __shared__ Runs<S> rs;
  __shared__ __attribute__((aligned(16))) float hs[S::kRuns][kStrip];
  const TileAt at = tile_at<S>(a, links, true);
  const LaneAt<S> l = lane_at<S>(a, at);
  uint4 vx[S::kRun], vd[S::kRun];
  float r[S::kRun][S::kPer], bi[S::kRun][S::kPer], rate[S::kPer];
  // C: what comes from behind the run, from 0: the sum of its dh, each through the decays
  // up to its token (A)
  float Z[S::kPer], H[S::kPer], C[S::kPer];
  on_run(l, [&](auto whole) {
    uint4 vg[S::kRun], vi[S::kRun];
    const T *x = row_of(a.x, l), *g = row_of(a.decay, l), *in = row_of(a.input, l),
            *dh = row_of(a.dh, l);
    load_tokens<whole>(l, [&](int t, int64_t i) {
      vg[t] = get16(g + i * a.decay.st);
      vi[t] = get16(in + i * a.input.st);
      vx[t] = get16(x + i * a.x.st);
      vd[t] = get16(dh + i * a.dh.st);
    }, [&](int t) {
      vg[t] = no_token<T>();
      vx[t] = vi[t] = vd[t] = make_uint4(0, 0, 0, 0);
    });
    float A[S::kPer];
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) {
      rate[c] = rate_after(l, c);
      Z[c] = -0.0f, H[c] = C[c] = 0.0f, A[c] = 1.0f;
    }
#pragma unroll
    for (int t = 0; t < S::kRun; ++t) {
      __builtin_amdgcn_sched_barrier(0);  // registers: one token at a time
#pragma unroll
      for (int c = 0; c < S::kPer; ++c) {
        r[t][c] = sigmoid(chunk_value<T>(vg[t], c));
        const float z = rate[c] * r[t][c], dec = __builtin_amdgcn_exp2f(z);
        bi[t][c] = gated(z, dec, chunk_value<T>(vi[t], c));
        Z[c] += z;
        H[c] = __builtin_fmaf(dec, H[c], bi[t][c] * chunk_value<T>(vx[t], c));
        A[c] *= dec;
        C[c] = __builtin_fmaf(A[c], chunk_value<T>(vd[t], c), C[c]);
      }
    }
  });
  put_run(rs, l, Z, C);
#pragma unroll
  for (int c = 0; c < S::kPer; ++c) hs[l.run][l.lane * S::kPer + c] = H[c];
  const auto tile_row = [&](int64_t c) { return (at.b * links.tiles + at.j) * a.d + c; };
  link_tile<true>(
      rs, a, links, at, [&](int64_t c) { return ds_out ? ds_out[at.b * a.d + c] : 0.0f; },
      [&](int64_t c, float, float behind) {
        if (ds_in && at.k + 1 == links.tiles) ds_in[at.b * a.d + c] = behind;
      },
      // the states in front of the runs, from the one in front of the tile
      [&](int64_t c) {
        const int ch = threadIdx.x % S::kStrip;
        float s = saved[tile_row(c)];
#pragma unroll 8
        for (int k = 0; k < S::kRuns; ++k) {
          const float next = decayed(rs.dec[k][ch], s, hs[k][ch]);
          hs[k][ch] = s;
          s = next;
        }
      });
  // what is worked out again below must not be kept in registers from above
#pragma unroll
  for (int t = 0; t < S::kRun; ++t) {
    asm("" : "+v"(vx[t].x), "+v"(vx[t].y), "+v"(vx[t].z), "+v"(vx[t].w));
    asm("" : "+v"(vd[t].x), "+v"(vd[t].y), "+v"(vd[t].z), "+v"(vd[t].w));
#pragma unroll
    for (int c = 0; c < S::kPer; ++c) asm("" : "+v"(r[t][c]));
  }
  uint32_t ox[S::kRun][4], og[S::kRun][4], oi[S::kRun][4];  // results as stored
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    __builtin_amdgcn_sched_barrier(0);  // and one word of channels
    constexpr int kIn = S::kPer / 4;  // channels of a 32-bit word
    float fx[S::kRun][kIn], fg[S::kRun][kIn], fi[S::kRun][kIn];
#pragma unroll
    for (int q = 0; q < kIn; ++q) {
      const int k = w * kIn + q, at_k = l.lane * S::kPer + k;
      // decays, and the states in front of the tokens
      float dec[S::kRun], s[S::kRun], f = hs[l.run][at_k];
#pragma unroll
      for (int t = 0; t < S::kRun; ++t) {
        s[t] = f;
        dec[t] = __builtin_amdgcn_exp2f(rate[k] * r[t][k]);
        f = __builtin_fmaf(dec[t], f, bi[t][k] * chunk_value<T>(vx[t], k));
      }
      float c = rs.h[l.run][at_k], dr = 0.0f;
#pragma unroll
      for (int t = S::kRun - 1; t >= 0; --t) {
        const float x = chunk_value<T>(vx[t], k), lam = chunk_value<T>(vd[t], k) + c;
        // y = l a (h - i x a / b), with i = (b i) / b; where b is 0 so is what they stand
        // beside (1 / b counts as 2^94: above all others, and finite)
        const float al = dec[t] * lam;
        const float inv =
            __builtin_amdgcn_rsqf(root_arg(rate[k] * r[t][k], dec[t], 0x1p-124f)) * 0x1p32f;
        const float i = bi[t][k] * inv;
        const float y = al * __builtin_fmaf(-dec[t], i * x * inv, s[t]);
        const float yr = t < l.n ? y * r[t][k] : 0.0f;
        fx[t][q] = lam * bi[t][k];
        const float fxx = fx[t][q] * x, yz = yr * (rate[k] * (1.0f / kLog2e));
        fi[t][q] = __builtin_fmaf(-fxx, i, fxx);
        fg[t][q] = __builtin_fmaf(-yz, r[t][k], yz);
        dr -= yr;
        c = al;
      }
      rs.z[l.run][at_k] = dr;  // read last in front of link_tile's second barrier
    }
#pragma unroll
    for (int t = 0; t < S::kRun; ++t) {
      ox[t][w] = Lane<T>::word(fx[t]);
      og[t][w] = Lane<T>::word(fg[t]);
      oi[t][w] = Lane<T>::word(fi[t]);
      // here, not in front of the stores, up to where all they come from would be kept
      asm volatile("" : "+v"(ox[t][w]), "+v"(og[t][w]), "+v"(oi[t][w]));
    }
  }
  const int64_t row = (l.b * a.T + l.t0) * a.d + l.c0;
  const auto put = [&](T* p, int t, const uint32_t* o) {
    *reinterpret_cast<uint4*>(p + row + t * a.d) = make_uint4(o[0], o[1], o[2], o[3]);
  };
  put_tokens(l, [&](int t) {
    put(dx, t, ox[t]), put(dg, t, og[t]), put(di, t, oi[t]);
  }, [&](int t) {
    const uint32_t none[4] = {0, 0, 0, 0};
    put(dx, t, none), put(dg, t, none), put(di, t, none);
  });
  __syncthreads();
  const int64_t ch = at.strip * (int64_t)kStrip + threadIdx.x;
  if (threadIdx.x < kStrip && ch < a.d) {
    float f = 0.0f;
#pragma unroll 8
    for (int k = 0; k < S::kRuns; ++k) f += rs.z[k][threadIdx.x];
    part[tile_row(ch)] = f;
  }
}

// out[slice][c] = sum over a slice's rows of part [rows][d]: 16 columns a workgroup, 64 lanes
// of rows.
constexpr int64_t kRateSlice = 2048;
constexpr int kRateRows = 64, kRateCols = 4 * kBlock / kRateRows;
__global__ __launch_bounds__(kBlock) void rec_rate_kernel(const float* __restrict__ part,
                                                          float* __restrict__ out, int64_t rows,
                                                          int64_t slice, int64_t d) {
  __shared__ float4 s[kRateRows][kRateCols / 4];
  const int cx = threadIdx.x % (kRateCols / 4), ry = threadIdx.x / (kRateCols / 4);
  const int64_t c = blockIdx.x * (int64_t)kRateCols + cx * 4, r0 = blockIdx.y * slice;
  const int64_t end = rows - r0 < slice ? rows : r0 + slice;
  float4 a = make_float4(0, 0, 0, 0);
  if (c < d) {
#pragma unroll 4
    for (int64_t r = r0 + ry; r < end; r += kRateRows) {
      const float4 p = *reinterpret_cast<const float4*>(part + r * d + c);
      a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    }
  }
  s[ry][cx] = a;
#pragma unroll
  for (int n = kRateRows / 2; n > 0; n /= 2) {
    __syncthreads();
    if (ry < n) {
      const float4 p = s[ry + n][cx];
      a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
      s[ry][cx] = a;
    }
  }
  if (ry == 0 && c < d) *reinterpret_cast<float4*>(out + blockIdx.y * d + c) = a;
}

int64_t tiles_of(const RecArgs& a) { return (a.T + kRecTile - 1) / kRecTile; }
int64_t groups_of(int64_t tiles) { return (tiles + kGroup - 1) / kGroup; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <typename F>
hipError_t with_type(Dtype dt, F&& f) {
  return dt == Dtype::F32 ? f(float{}) : f(uint16_t{});
}
// Whether a call takes the recurrent form.  A lane's tokens take it 0.8 us each, or what
// the memory takes for them; a tile takes 8 us whatever it holds, and many at once 2.5 ns
// each.  us of 2560 channels, recurrent / tiles: 1 sequence of 8 tokens 9.9 / 7.9, 64 of 4 7.8 /
// 9.9, 64 of 6 8.9 / 10.0, 64 of 8 10.5 / 10.1, 64 of 12 14.6 / 10.6, 512 of 8 27 / 48, 512 of
// 16 48 / 49, 512 of 24 69 / 55.
bool steps(const RecArgs& a) { return a.T <= (a.B * a.d >= ((int64_t)1 << 20) ? 16 : 6); }

// f with the threads of a tile of a call (64 sequences of 32 tokens of 2560 channels 11.8
// us, 25.9 in tiles of 128; 64 tokens 17.6 and 26.8; 512 of 32 tokens 68 and 172).
template <int kStrip, typename F>
void with_threads(const RecArgs& a, F&& f) {
  if (a.T * 4 <= kRecTile)
    f(std::integral_constant<int, kStrip>{});
  else if (a.T * 2 <= kRecTile)
    f(std::integral_constant<int, 2 * kStrip>{});
  else
    f(std::integral_constant<int, 4 * kStrip>{});
}

}  // namespace

// The words that link the tiles and groups, and behind them the counter.
size_t link_bytes(const RecArgs& a) {
  const int64_t tiles = tiles_of(a), words = a.B * (tiles + groups_of(tiles)) * a.d;
  return tiles > 1 ? align256((size_t)words * sizeof(uint64_t)) + 256 : 0;
}

namespace {
// The workspace's links, cleared.
hipError_t clear_links(const RecArgs& a, void* ws, Links* links, hipStream_t s) {
  links->tiles = tiles_of(a), links->groups = groups_of(links->tiles);
  links->maps = links->states = nullptr, links->begun = nullptr;
  if (links->tiles == 1) return hipSuccess;
  const size_t bytes = link_bytes(a) - 256;
  links->maps = static_cast<uint64_t*>(ws);
  links->states = links->maps + a.B * links->tiles * a.d;
  links->begun = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + bytes);
  const int64_t n = (int64_t)(bytes / 16);
  rec_clear_kernel<<<dim3((unsigned)std::min<int64_t>((n + kBlock - 1) / kBlock, 2048)), kBlock, 0,
                     s>>>(static_cast<uint4*>(ws), n, links->begun);
  return hipGetLastError();
}
dim3 tile_grid(const RecArgs& a, int strip) {
  return dim3((unsigned)(a.B * tiles_of(a) * ((a.d + strip - 1) / strip)));
}
// Slices of the tiles' sums of drate: more than one, added up by a launch of its own, where
// one workgroup's loads would show.
int64_t rate_slices(const RecArgs& a) {
  const int64_t rows = a.B * tiles_of(a);
  return rows <= kRateSlice ? 1 : (rows + kRateSlice - 1) / kRateSlice;
}
}  // namespace

size_t gatedrec_forward_bytes(const RecArgs& a) { return link_bytes(a); }

hipError_t launch_gatedrec_forward(const RecArgs& a, const float* s_in, float* s_out, void* h,
                                   int64_t hsb, int64_t hst, float* saved, void* ws,
                                   hipStream_t s) {
  return with_type(a.dt, [&](auto t) {
    using T = decltype(t);
    T* out = static_cast<T*>(h);
    if (steps(a)) {
      const int64_t n = a.B * (a.d / Lane<T>::kPer);
      rec_step_kernel<T><<<dim3((unsigned)((n + kBlock - 1) / kBlock)), kBlock, 0, s>>>(
          a, s_in, s_out, out, hsb, hst, saved);
      return hipGetLastError();
    }
    Links links;
    const hipError_t e = clear_links(a, ws, &links, s);
    if (e != hipSuccess) return e;
    const auto go = [&](auto strip) {
      constexpr int kStrip = decltype(strip)::value;
      with_threads<kStrip>(a, [&](auto threads) {
        constexpr int n = decltype(threads)::value;
        rec_forward_kernel<T, kStrip, n><<<tile_grid(a, kStrip), n, 0, s>>>(
            a, links, s_in, s_out, out, hsb, hst, saved);
      });
    };
    if constexpr (sizeof(T) == 2) {
      if (a.d > kFewChannels)
        go(std::integral_constant<int, kWideStrip>{});
      else
        go(std::integral_constant<int, kStrip>{});
    } else {
      go(std::integral_constant<int, kStrip>{});
    }
    return hipGetLastError();
  });
}

// The links, the tiles' sums of drate, and their slices' sums.
size_t gatedrec_backward_bytes(const RecArgs& a) {
  const int64_t rows = a.B * tiles_of(a), slices = rate_slices(a);
  return link_bytes(a) + (size_t)((rows + (slices > 1 ? slices : 0)) * a.d) * sizeof(float);
}

hipError_t launch_gatedrec_backward(const RecArgs& a, const float* saved, const float* ds_out,
                                    void* dx, void* ddecay, void* dinput, float* drate,
                                    float* ds_in, void* ws, hipStream_t s) {
  return with_type(a.dt, [&](auto t) {
    using T = decltype(t);
    Links links;
    const hipError_t e = clear_links(a, ws, &links, s);
    if (e != hipSuccess) return e;
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + link_bytes(a));
    with_threads<kStrip>(a, [&](auto threads) {
      constexpr int n = decltype(threads)::value;
      rec_backward_kernel<T, kStrip, n><<<tile_grid(a, kStrip), n, 0, s>>>(
          a, links, saved, ds_out, ds_in, static_cast<T*>(dx), static_cast<T*>(ddecay),
          static_cast<T*>(dinput), part);
    });
    const unsigned columns = (unsigned)((a.d + kRateCols - 1) / kRateCols);
    const int64_t rows = a.B * links.tiles, slices = rate_slices(a);
    float* const sums = slices > 1 ? part + rows * a.d : drate;
    rec_rate_kernel<<<dim3(columns, (unsigned)slices), kBlock, 0, s>>>(
        part, sums, rows, slices > 1 ? kRateSlice : rows, a.d);
    if (slices > 1)
      rec_rate_kernel<<<dim3(columns), kBlock, 0, s>>>(sums, drate, slices, slices, a.d);
    return hipGetLastError();
  });
}

}  // namespace ttt
