// embed.hip -- embedding lookup with scaling, and the table's gradient by sorted
// tokens.
//
//   out[n] = scale table[ids[n]],   grad[v] (+)= scale sum_{n: ids[n] = v} dout[n]
//
// The lookup copies rows: bound by HBM.  The gradient sorts the tokens by id
// (least significant digit first, stable, so that equal ids keep the order of
// their places), cuts the sorted tokens into pieces of kPiece and lets a wave sum
// a piece's rows in registers: an id whose tokens lie in one piece gets its row
// written at once, the sums of ids that reach over pieces go to the workspace and
// are added in order by a last launch.  No atomic sums: the result does not
// depend on what runs when.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "piece.h"
#include "seq.h"

namespace ttt {
namespace {

constexpr int kBlock = 256;
constexpr int kPiece = 32;       // sorted tokens that a wave sums
constexpr int kWaveCols = 512;   // columns of a wave: 8 a lane
constexpr int kSortBlock = 1024;
constexpr int kSortTile = 4096;  // tokens that a workgroup of the sort orders
constexpr int kSortRounds = kSortTile / kSortBlock;
constexpr int kSortWaves = kSortBlock / 64;
constexpr int kMaxBins = 512;

__device__ __forceinline__ int64_t id_at(const void* ids, bool wide, int64_t n) {
  return wide ? static_cast<const int64_t*>(ids)[n] : static_cast<const int32_t*>(ids)[n];
}

// LPR lanes copy a row, 8 values each at a time.
template <typename T, typename TO, int LPR>
__global__ __launch_bounds__(kBlock) void embed_forward_kernel(
    const void* __restrict__ ids, bool wide, const T* __restrict__ table, TO* __restrict__ out,
    int64_t N, int64_t V, int64_t d, float scale) {
  const int lane = threadIdx.x % LPR;
  const int64_t n = (int64_t)blockIdx.x * (kBlock / LPR) + threadIdx.x / LPR;
  if (n >= N) return;
  const int64_t id = id_at(ids, wide, n);
  const bool live = id >= 0 && id < V;
  const T* row = table + (live ? id : 0) * d;
  const int pieces = (int)(d >> 3);
#pragma unroll 4
  for (int c = lane; c < pieces; c += LPR) {
    Piece<T> p;
    p.load(row + 8 * c);
    float f[8];
    p.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = live ? f[j] * scale : 0.0f;
    Piece<TO>::store(out + n * d + 8 * c, f);
  }
}

// ------------------------------------------------------------------ the sort
// Keys are ids, V for those outside [0, V), which so come last.
struct SortIn {
  const void* ids;      // first pass, null later
  const uint32_t* keys;
  const uint32_t* pos;
  bool wide;
  int64_t N, V;
  __device__ __forceinline__ uint32_t key(int64_t n) const {
    if (!ids) return keys[n];
    const int64_t id = id_at(ids, wide, n);
    return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
  }
};

// hist[bin][tile]: tokens of a tile with this digit.
__global__ __launch_bounds__(kSortBlock) void embed_hist_kernel(SortIn in, int shift, int bins,
                                                                int64_t tiles,
                                                                uint32_t* __restrict__ hist) {
  __shared__ uint32_t count[kMaxBins];
  for (int b = threadIdx.x; b < bins; b += kSortBlock) count[b] = 0;
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * kSortTile;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t n = n0 + r * kSortBlock + threadIdx.x;
    if (n < in.N) atomicAdd(&count[(in.key(n) >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortBlock) hist[b * tiles + blockIdx.x] = count[b];
}

// Exclusive sums of v over the workgroup's threads (kThreads a multiple of 64),
// and the sum of all of them in *total.
template <int kThreads>
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* wave_sum,
                                                    uint32_t* total) {
  constexpr int kWaves = kThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t o = __shfl_up(x, m, 64);
    if (lane >= m) x += o;
  }
  if (lane == 63) wave_sum[wave] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += wave_sum[w];
    all += wave_sum[w];
  }
  __syncthreads();  // wave_sum may be used again
  *total = all;
  return before + x - v;
}

// hist[bin][tile] -> tokens of this digit in the tiles in front; total[bin].
__global__ __launch_bounds__(kBlock) void embed_scan_kernel(uint32_t* __restrict__ hist,
                                                            int64_t tiles,
                                                            uint32_t* __restrict__ total) {
  __shared__ uint32_t wave_sum[kBlock / 64];
  uint32_t run = 0;
  uint32_t* const h = hist + blockIdx.x * tiles;
  for (int64_t t0 = 0; t0 < tiles; t0 += kBlock) {
    const int64_t t = t0 + threadIdx.x;
    const uint32_t v = t < tiles ? h[t] : 0;
    uint32_t sum;
    const uint32_t e = block_exclusive<kBlock>(v, wave_sum, &sum);
    if (t < tiles) h[t] = run + e;
    run += sum;
  }
  if (threadIdx.x == 0) total[blockIdx.x] = run;
}

// The tile's tokens to their places.  Wave w takes the tokens 256 w .. of the
// tile in rounds of 64; a token's rank among those of its digit is the count of
// the wave's earlier rounds and of the lower lanes of its own with that digit,
// found by a ballot for each bit.
__global__ __launch_bounds__(kSortBlock) void embed_scatter_kernel(
    SortIn in, int shift, int bits, int64_t tiles, const uint32_t* __restrict__ hist,
    const uint32_t* __restrict__ total, uint32_t* __restrict__ keys_out,
    uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t count[kSortWaves][kMaxBins];
  __shared__ uint32_t wave_sum[kSortWaves];
  const int bins = 1 << bits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kSortWaves * bins; i += kSortBlock) count[i / bins][i % bins] = 0;
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * kSortTile + wave * (64 * kSortRounds) + lane;
  uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    key[r] = n0 + 64 * r < in.N ? in.key(n0 + 64 * r) : 0;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const bool live = n0 + 64 * r < in.N;
    const uint32_t digit = (key[r] >> shift) & (bins - 1);
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const bool one = (digit >> b) & 1;
      const uint64_t with = __ballot(one);
      same &= one ? with : ~with;
    }
    const uint32_t lower = __popcll(same & ((1ull << lane) - 1));
    uint32_t before = 0;
    if (live) before = count[wave][digit];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (live && lower == 0) count[wave][digit] = before + (uint32_t)__popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    rank[r] = before + lower;
  }
  __syncthreads();
  // places: digits in front, tiles in front, waves in front
  const bool has = threadIdx.x < (unsigned)bins;
  const uint32_t mine = has ? total[threadIdx.x] : 0;
  uint32_t all;
  uint32_t at = block_exclusive<kSortBlock>(mine, wave_sum, &all);
  if (has) {
    at += hist[threadIdx.x * tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = count[w][threadIdx.x];
      count[w][threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t n = n0 + 64 * r;
    if (n >= in.N) continue;
    const uint32_t to = count[wave][(key[r] >> shift) & (bins - 1)] + rank[r];
    keys_out[to] = key[r];
    pos_out[to] = in.pos ? in.pos[n] : (uint32_t)n;
  }
}

// ------------------------------------------------------------------- the sums
__global__ __launch_bounds__(kBlock) void embed_zero_kernel(uint4* __restrict__ p, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * kBlock;
  for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < n; i += step)
    p[i] = make_uint4(0, 0, 0, 0);
}

template <typename TO>
__device__ __forceinline__ void put_row(TO* row, const float sum[8], float scale, bool accumulate) {
  float f[8], old[8];
  if (accumulate) {
    Piece<TO> p;
    p.load(row);
    p.get(old);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = accumulate ? old[j] + scale * sum[j] : scale * sum[j];
  Piece<TO>::store(row, f);
}

// A wave sums kWaveCols columns of a piece of the sorted tokens.  part[2 p] has
// the sum of piece p's first tokens where their id began in front of it or goes
// on behind it without another in the piece, part[2 p + 1] that of its last
// tokens where their id goes on behind it.
template <typename T, typename TO>
__global__ __launch_bounds__(kBlock) void embed_sum_kernel(
    const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos,
    const T* __restrict__ dout, TO* __restrict__ grad, float* __restrict__ part, int64_t N,
    int64_t V, int64_t d, float scale, bool accumulate, int64_t units, int col_parts) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t p = unit / col_parts;
  const int64_t col = (unit % col_parts) * kWaveCols + 8 * lane;
  const int64_t n0 = p * kPiece;
  const int n = (int)min<int64_t>(kPiece, N - n0);
  // lane l: token l of the piece; ids in front of it and behind it (none: V + 1)
  const uint32_t none = (uint32_t)V + 1;
  const uint32_t key = lane < n ? keys[n0 + lane] : none;
  const uint32_t at = lane < n ? pos[n0 + lane] : 0;
  const uint32_t front = n0 > 0 ? keys[n0 - 1] : none;
  const uint32_t behind = n0 + n < N ? keys[n0 + n] : none;
  const bool mine = col < d;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  int first = 0;  // of the current id
  constexpr int kAhead = 8;
  for (int t0 = 0; t0 < n; t0 += kAhead) {
    Piece<T> row[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      row[i].zero();
      const int t = t0 + i;
      const uint32_t where = __builtin_amdgcn_readlane(at, t);
      const uint32_t id = __builtin_amdgcn_readlane(key, t);
      if (t < n && mine && id < (uint32_t)V) row[i].load(dout + (int64_t)where * d + col);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = t0 + i;
      if (t >= n) break;
      float f[8];
      row[i].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
      const uint32_t id = __builtin_amdgcn_readlane(key, t);
      const uint32_t next = t + 1 < n ? __builtin_amdgcn_readlane(key, t + 1) : behind;
      if (t + 1 < n && next == id) continue;
      // the id's last token of the piece
      if (id < (uint32_t)V && mine) {
        const bool whole = (first > 0 || front != id) && (t + 1 < n || next != id);
        if (whole)
          put_row<TO>(grad + (int64_t)id * d + col, sum, scale, accumulate);
        else
          Piece<float>::store(part + (2 * p + (first > 0 ? 1 : 0)) * d + col, sum);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
      first = t + 1;
    }
  }
}

// The rows of ids that reach over pieces: the workgroups of the piece in which
// one begins add its pieces' sums, 4 waves every fourth and then each other's,
// 256 columns each.
template <typename TO>
__global__ __launch_bounds__(kBlock) void embed_join_kernel(
    const uint32_t* __restrict__ keys, const float* __restrict__ part, TO* __restrict__ grad,
    int64_t N, int64_t V, int64_t d, float scale, bool accumulate) {
  __shared__ float s[4][256];
  const int64_t p = blockIdx.x, n0 = p * kPiece;
  const int64_t last = min<int64_t>(n0 + kPiece, N) - 1;
  if (last + 1 >= N) return;
  const uint32_t id = keys[last];
  if (id >= (uint32_t)V || keys[last + 1] != id) return;
  const bool inside = keys[n0] != id;  // begins behind the piece's first token
  if (!inside && n0 > 0 && keys[n0 - 1] == id) return;  // began in an earlier piece
  // the first token behind the id's
  int64_t lo = last + 1, hi = N;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] <= id) lo = mid + 1; else hi = mid;
  }
  const int64_t end = (lo - 1) / kPiece;  // its last piece
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t col = (int64_t)blockIdx.y * 256 + 4 * lane;
  float4 a = make_float4(0, 0, 0, 0);
  if (col < d) {
#pragma unroll 4
    for (int64_t q = p + wave; q <= end; q += 4) {
      const int64_t slot = 2 * q + (q == p && inside ? 1 : 0);
      const float4 v = *reinterpret_cast<const float4*>(part + slot * d + col);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
  *reinterpret_cast<float4*>(&s[wave][4 * lane]) = a;
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.y * 256 + 8 * threadIdx.x;
  if (threadIdx.x >= 32 || c >= d) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int x = 8 * threadIdx.x + j;
    sum[j] = (s[0][x] + s[1][x]) + (s[2][x] + s[3][x]);
  }
  put_row<TO>(grad + (int64_t)id * d + c, sum, scale, accumulate);
}

// ---------------------------------------------------------------- host side
struct SortPlan {
  int passes, bits;  // passes of `bits` bits each
  int64_t tiles;
};
SortPlan sort_plan(const EmbedArgs& a) {
  int bits = 1;
  while (((int64_t)1 << bits) <= a.V) ++bits;  // keys 0 .. V
  SortPlan p;
  p.passes = (bits + 8) / 9;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = (a.N + kSortTile - 1) / kSortTile;
  return p;
}
size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t pieces_of(const EmbedArgs& a) { return (a.N + kPiece - 1) / kPiece; }

// Workspace: two sets of keys and places, the digits' counts, the partial sums.
struct GradPlan {
  size_t keys[2], pos[2], hist, total, part, bytes;
};
GradPlan grad_plan(const EmbedArgs& a) {
  const SortPlan sp = sort_plan(a);
  GradPlan p;
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  for (int i = 0; i < 2; ++i) p.keys[i] = take(a.N * 4), p.pos[i] = take(a.N * 4);
  p.hist = take(((size_t)sp.tiles << sp.bits) * 4);
  p.total = take(((size_t)1 << sp.bits) * 4);
  p.part = take((size_t)(2 * pieces_of(a) * a.d) * sizeof(float));
  p.bytes = at;
  return p;
}

template <typename F>
hipError_t with_types(const EmbedArgs& a, F&& f) {
  if (a.dt == Dtype::F32) return f(float{}, float{});
  return a.out_dt == Dtype::F32 ? f(uint16_t{}, float{}) : f(uint16_t{}, uint16_t{});
}

}  // namespace

hipError_t launch_embed_forward(const EmbedArgs& a, const void* ids, const void* table, void* out,
                                hipStream_t s) {
  return with_types(a, [&](auto t, auto to) {
    using T = decltype(t);
    using TO = decltype(to);
    const auto go = [&](auto lpr) {
      constexpr int L = decltype(lpr)::value;
      // a launch's threads are counted in 32 bits
      const int64_t per = kBlock / L, most = per << 23;
      for (int64_t at = 0; at < a.N; at += most) {
        const int64_t n = std::min(a.N - at, most);
        embed_forward_kernel<T, TO, L><<<dim3((unsigned)((n + per - 1) / per)), kBlock, 0, s>>>(
            static_cast<const char*>(ids) + at * (a.wide_ids ? 8 : 4), a.wide_ids,
            static_cast<const T*>(table), static_cast<TO*>(out) + at * a.d, n, a.V, a.d, a.scale);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    };
    return a.d <= 128 ? go(std::integral_constant<int, 16>{})
                      : go(std::integral_constant<int, 64>{});
  });
}

size_t embed_backward_bytes(const EmbedArgs& a) { return grad_plan(a).bytes; }

hipError_t launch_embed_backward(const EmbedArgs& a, const void* ids, const void* dout, void* grad,
                                 void* ws, hipStream_t s) {
  const SortPlan sp = sort_plan(a);
  const GradPlan p = grad_plan(a);
  char* const base = static_cast<char*>(ws);
  const auto u32 = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
  uint32_t *hist = u32(p.hist), *total = u32(p.total);
  const int bins = 1 << sp.bits;
  int cur = 0;
  for (int i = 0; i < sp.passes; ++i) {
    const int shift = i * sp.bits;
    SortIn in{i ? nullptr : ids, u32(p.keys[cur ^ 1]), i ? u32(p.pos[cur ^ 1]) : nullptr,
              a.wide_ids, a.N, a.V};
    embed_hist_kernel<<<dim3((unsigned)sp.tiles), kSortBlock, 0, s>>>(in, shift, bins, sp.tiles,
                                                                      hist);
    embed_scan_kernel<<<dim3((unsigned)bins), kBlock, 0, s>>>(hist, sp.tiles, total);
    embed_scatter_kernel<<<dim3((unsigned)sp.tiles), kSortBlock, 0, s>>>(
        in, shift, sp.bits, sp.tiles, hist, total, u32(p.keys[cur]), u32(p.pos[cur]));
    cur ^= 1;
  }
  const uint32_t *keys = u32(p.keys[cur ^ 1]), *pos = u32(p.pos[cur ^ 1]);
  float* part = reinterpret_cast<float*>(base + p.part);
  return with_types(a, [&](auto t, auto to) {
    using T = decltype(t);
    using TO = decltype(to);
    if (!a.accumulate) {
      const int64_t n = a.V * a.d * (int64_t)sizeof(TO) / 16;
      embed_zero_kernel<<<dim3((unsigned)std::min<int64_t>((n + kBlock - 1) / kBlock, 4096)),
                          kBlock, 0, s>>>(static_cast<uint4*>(grad), n);
    }
    const int col_parts = (int)((a.d + kWaveCols - 1) / kWaveCols);
    const int64_t units = pieces_of(a) * col_parts;
    // units of 64 threads: fewer than 2^32 threads a launch (checked by the caller)
    embed_sum_kernel<T, TO><<<dim3((unsigned)((units + 3) / 4)), kBlock, 0, s>>>(
        keys, pos, static_cast<const T*>(dout), static_cast<TO*>(grad), part, a.N, a.V, a.d,
        a.scale, a.accumulate, units, col_parts);
    embed_join_kernel<TO><<<dim3((unsigned)pieces_of(a), (unsigned)((a.d + 255) / 256)), kBlock, 0,
                            s>>>(keys, part, static_cast<TO*>(grad), a.N, a.V, a.d, a.scale,
                                 a.accumulate);
    return hipGetLastError();
  });
}

}  // namespace ttt
