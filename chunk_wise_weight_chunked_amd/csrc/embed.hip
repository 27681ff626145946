// embed.hip -- embedding lookup with scaling, and the table's gradient by sorted
// tokens.
//
//   out[n] = scale table[ids[n]],   grad[v] (+)= scale sum_{n: ids[n] = v} dout[n]
//
// The lookup copies rows: bound by memory and caches.  The gradient sorts the tokens by id
// (least significant digit first, stable, so that equal ids keep the order of
// their places), cuts the sorted tokens into pieces of 8 to 32 and lets a wave sum
// a piece's rows in registers: an id whose tokens lie in one piece gets its row
// written at once, the sums of ids that reach over pieces go to the workspace and
// are added in order by a last launch.  No atomic sums: the result does not
// depend on what runs when.  Up to 64 tokens take one launch without a sort.
//
// The lookup of 131072 rows of 2560 bf16 values takes 185 us: 1.34 GB into and out of the L2s
// at 7.3 TB/s, many rows again and again from the last-level cache.  The gradient of 32768
// tokens of 2560 into 50001 fp32 rows takes 181 us: the sort's launches, each some 4 to 8 us
// of waiting for the one before, and 4.2 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "piece.h"
#include "seq.h"

namespace ttt {
namespace {

constexpr int kBlock = 256;
constexpr int kPiece = 32;       // sorted tokens that a wave sums, at most
constexpr int kWaveCols = 512;   // columns of a wave: 8 a lane
constexpr int kSortBlock = 1024;  // tokens that a workgroup of the sort orders, one a lane
constexpr int kSortWaves = kSortBlock / 64;
constexpr int kMaxBins = 512;
constexpr int kFewTiles = 64;    // 31984 tokens 69.5 us, 72.9 with another launch; 65000 139.6, 141.1

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

// A share of a gradient's zeros, written by the workgroups of a launch of the sort that
// come behind its own: the sort leaves most of the chip idle, and the zeros need no more
// than the memory's bandwidth.
struct Zeros {
  uint4* p;
  int64_t n;      // 0: none, and no workgroups behind the launch's own
  int32_t own;    // the launch's own workgroups
  template <int kThreads>
  __device__ __forceinline__ bool fill() const {
    if ((int)blockIdx.x < own) return false;
    const int64_t step = (int64_t)(gridDim.x - own) * kThreads;
    for (int64_t i = (int64_t)(blockIdx.x - own) * kThreads + threadIdx.x; i < n; i += step)
      p[i] = make_uint4(0, 0, 0, 0);
    return true;
  }
};

// hist[tile][bin]: tokens of a tile with this digit.
__global__ __launch_bounds__(kSortBlock) void embed_hist_kernel(SortIn in, int shift, int bins,
                                                                uint32_t* __restrict__ hist,
                                                                Zeros zeros) {
  __shared__ uint32_t count[kMaxBins];
  if (zeros.fill<kSortBlock>()) return;
  const int b = threadIdx.x;
  if (b < bins) count[b] = 0;
  __syncthreads();
  const int64_t n = (int64_t)blockIdx.x * kSortBlock + threadIdx.x;
  if (n < in.N) atomicAdd(&count[(in.key(n) >> shift) & (bins - 1)], 1u);
  __syncthreads();
  if (b < bins) hist[(int64_t)blockIdx.x * bins + b] = count[b];
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

// hist[tile][bin] -> tokens of this digit in the tiles in front; total[bin].  64 digits a
// workgroup, a wave walks its share of the tiles.
__global__ __launch_bounds__(kSortBlock) void embed_scan_kernel(uint32_t* __restrict__ hist,
                                                                int bins, int64_t tiles,
                                                                uint32_t* __restrict__ total) {
  __shared__ uint32_t sum[kSortWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bin = blockIdx.x * 64 + lane;
  const int64_t share = (tiles + kSortWaves - 1) / kSortWaves;
  const int64_t t0 = wave * share, t1 = min(t0 + share, tiles);
  uint32_t n = 0;
  if (bin < bins)
#pragma unroll 8
    for (int64_t t = t0; t < t1; ++t) n += hist[t * bins + bin];
  sum[wave][lane] = n;
  __syncthreads();
  uint32_t at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) at += sum[w][lane];
    all += sum[w][lane];
  }
  if (bin >= bins) return;
  if (wave == 0) total[bin] = all;
#pragma unroll 8
  for (int64_t t = t0; t < t1; ++t) {
    const uint32_t c = hist[t * bins + bin];
    hist[t * bins + bin] = at;
    at += c;
  }
}

// The tile's tokens to their places.  A token's rank among those of its digit is the
// count of the lower lanes of its wave with that digit, found by a ballot for each bit,
// and of the waves and tiles in front.  Without `total`, hist still holds the tiles' own
// counts, and the workgroup adds up those in front of it itself.
__global__ __launch_bounds__(kSortBlock) void embed_scatter_kernel(
    SortIn in, int shift, int bits, int64_t tiles, const uint32_t* __restrict__ hist,
    const uint32_t* __restrict__ total, uint32_t* __restrict__ keys_out,
    uint32_t* __restrict__ pos_out, Zeros zeros) {
  __shared__ uint32_t count[kSortWaves][kMaxBins];
  __shared__ uint32_t wave_sum[kSortWaves];
  if (zeros.fill<kSortBlock>()) return;
  const int bins = 1 << bits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * kSortBlock + threadIdx.x;
  const bool live = n < in.N, has = threadIdx.x < (unsigned)bins;
  const uint32_t key = live ? in.key(n) : 0;
  const uint32_t place = live && in.pos ? in.pos[n] : (uint32_t)n;
  uint32_t mine = 0, tile = 0;
  if (has && total) {
    mine = total[threadIdx.x];
    tile = hist[(int64_t)blockIdx.x * bins + threadIdx.x];
  } else if (has) {
    constexpr int kLoads = 32;  // at a time
    for (int t0 = 0; t0 < (int)tiles; t0 += kLoads) {
      uint32_t c[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        c[i] = hist[min(t0 + i, (int)tiles - 1) * bins + threadIdx.x];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        mine += t0 + i < (int)tiles ? c[i] : 0;
        tile += t0 + i < (int)blockIdx.x ? c[i] : 0;
      }
    }
  }
  for (int i = lane; i < bins; i += 64) count[wave][i] = 0;
  const uint32_t digit = (key >> shift) & (bins - 1);
  uint64_t same = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const bool one = (digit >> b) & 1;
    const uint64_t with = __ballot(one);
    same &= one ? with : ~with;
  }
  const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (live && rank == 0) count[wave][digit] = (uint32_t)__popcll(same);
  __syncthreads();
  uint32_t all;
  uint32_t at = block_exclusive<kSortBlock>(mine, wave_sum, &all) + tile;
  if (has) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = count[w][threadIdx.x];
      count[w][threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  if (!live) return;
  const uint32_t to = count[wave][digit] + rank;
  keys_out[to] = key;
  pos_out[to] = place;
}

// All passes for up to kSmall tokens in one workgroup: tokens in LDS, wave w has the
// tokens w 64 rounds .. of each pass in rounds of 64, and counts a digit's tokens of its
// earlier rounds as well.  (512 columns of 50001 rows added to, one workgroup / the
// launches above: 1000 tokens 15 / 25 us, 4000 22 / 25, 6000 28 / 27, 8192 34 / 29; of 1000
// rows 6000 22 / 25, 8192 27 / 25.)
constexpr int kSmallRounds = 6;
constexpr int kSmall = kSmallRounds * kSortBlock;
__global__ __launch_bounds__(kSortBlock) void embed_sort_kernel(SortIn in, int passes, int bits,
                                                                uint32_t* __restrict__ keys_out,
                                                                uint32_t* __restrict__ pos_out,
                                                                Zeros zeros) {
  __shared__ uint32_t count[kSortWaves][kMaxBins];
  __shared__ uint32_t wave_sum[kSortWaves];
  __shared__ uint2 token[kSmall];  // key, place
  if (zeros.fill<kSortBlock>()) return;
  const int bins = 1 << bits, N = (int)in.N;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rounds = (N + kSortBlock - 1) / kSortBlock;
  const int n0 = wave * 64 * rounds + lane;
  uint2 own[kSmallRounds];
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r) {
    const int n = n0 + 64 * r;
    own[r] = make_uint2(r < rounds && n < N ? in.key(n) : 0, (uint32_t)n);
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits;
    for (int i = lane; i < bins; i += 64) count[wave][i] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint32_t rank[kSmallRounds];
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
      if (r >= rounds) break;
      const bool live = n0 + 64 * r < N;
      const uint32_t digit = (own[r].x >> shift) & (bins - 1);
      uint64_t same = __ballot(live);
      for (int b = 0; b < bits; ++b) {
        const bool one = (digit >> b) & 1;
        const uint64_t with = __ballot(one);
        same &= one ? with : ~with;
      }
      const uint32_t lower = __popcll(same & ((1ull << lane) - 1));
      const uint32_t before = live ? count[wave][digit] : 0;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (live && lower == 0) count[wave][digit] = before + (uint32_t)__popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      rank[r] = before + lower;
    }
    __syncthreads();
    uint32_t mine = 0, all;
    const bool has = threadIdx.x < (unsigned)bins;
    if (has) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) mine += count[w][threadIdx.x];
    }
    uint32_t at = block_exclusive<kSortBlock>(mine, wave_sum, &all);
    if (has) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = count[w][threadIdx.x];
        count[w][threadIdx.x] = at;
        at += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r)
      if (r < rounds && n0 + 64 * r < N)
        token[count[wave][(own[r].x >> shift) & (bins - 1)] + rank[r]] = own[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r)
      if (r < rounds && n0 + 64 * r < N) own[r] = token[n0 + 64 * r];
    __syncthreads();  // counts and tokens are written again
  }
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r) {
    const int n = n0 + 64 * r;
    if (r < rounds && n < N) keys_out[n] = own[r].x, pos_out[n] = own[r].y;
  }
}

// ------------------------------------------------------------------- the sums
// A gradient's row from its sum and, where it is added to, what is there.
template <typename TO, bool kAdd>
__device__ __forceinline__ void put_row(TO* row, const float sum[8], float scale,
                                        const Piece<TO>& there) {
  float f[8];
  there.get(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = kAdd ? f[j] + scale * sum[j] : scale * sum[j];
  Piece<TO>::store(row, f);
}

// Zeros in the rows v0 + i of the bits i of `none`.
template <typename TO>
__device__ __forceinline__ void put_zeros(TO* __restrict__ grad, int64_t d, int64_t v0,
                                          uint64_t none) {
  const int64_t n = d * (int64_t)sizeof(TO) / 16;
  while (none) {
    uint4* const row = reinterpret_cast<uint4*>(grad + (v0 + __builtin_ctzll(none)) * d);
    none &= none - 1;
    for (int64_t i = threadIdx.x & 63; i < n; i += 64) row[i] = make_uint4(0, 0, 0, 0);
  }
}

// Zeros for rows without tokens: a wave takes kZeroRows rows from v0 on and looks each up
// in the sorted tokens' ids.
constexpr int kZeroRows = 16;
template <typename TO>
__device__ __forceinline__ void zero_rows(const uint32_t* __restrict__ keys, TO* __restrict__ grad,
                                          int64_t N, int64_t V, int64_t d, int64_t v0) {
  const int lane = threadIdx.x & 63;
  const int64_t v = v0 + lane;
  int64_t lo = 0, hi = N;  // the first token whose id is not below v
  while (lane < kZeroRows && lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if ((int64_t)keys[mid] < v) lo = mid + 1; else hi = mid;
  }
  put_zeros(grad, d, v0,
            __ballot(lane < kZeroRows && v < V && (lo == N || (int64_t)keys[lo] != v)));
}

// A wave sums kWaveCols columns of a piece of the sorted tokens; behind those waves come
// the ones that write the zeros of rows [zero0, zero1).  part[2 p] has
// the sum of piece p's first tokens where their id began in front of it or goes
// on behind it without another in the piece, part[2 p + 1] that of its last
// tokens where their id goes on behind it.
template <typename T, typename TO, bool kAdd>
__global__ __launch_bounds__(kBlock) void embed_sum_kernel(
    const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos,
    const T* __restrict__ dout, TO* __restrict__ grad, float* __restrict__ part, int64_t N,
    int64_t V, int64_t d, float scale, int piece, int64_t units, int col_parts, int64_t zero0,
    int64_t zero1) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kBlock / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // wave-uniform
  if (unit >= units) {
    const int64_t step = ((int64_t)gridDim.x * (kBlock / 64) - units) * kZeroRows;
    for (int64_t v0 = zero0 + (unit - units) * kZeroRows; v0 < zero1; v0 += step)
      zero_rows(keys, grad, N, zero1, d, v0);
    return;
  }
  const int64_t p = unit / col_parts;
  const int64_t col = (unit % col_parts) * kWaveCols + 8 * lane;
  const int64_t n0 = p * piece;
  const int n = (int)min<int64_t>(piece, N - n0);
  // lane l: token l of the piece; ids in front of it and behind it (none: V + 1)
  const uint32_t none = (uint32_t)V + 1;
  const uint32_t key = lane < n ? keys[n0 + lane] : none;
  const uint32_t at = pos[n0 + min(lane, n - 1)];
  const uint32_t front = n0 > 0 ? keys[n0 - 1] : none;
  const uint32_t behind = n0 + n < N ? keys[n0 + n] : none;
  const bool mine = col < d;
  const T* const from = dout + (mine ? col : 0);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  int first = 0;  // of the current id
  // Rows are loaded ahead, and with kAdd the gradient's row of each token's id beside them
  // (again and again for an id of many tokens, from L2): a call of 31984 tokens of 1024
  // values takes 3 us of 73 more where a wave waits for it at the end of each id.
  constexpr int kAhead = kAdd ? 4 : 8;
  struct Ahead {
    Piece<T> row[kAhead];
    Piece<TO> there[kAhead];
  } ahead[2];
  // what is read for nothing (behind the last token, of no id) is never put anywhere
  const auto load = [&](Ahead& a, int t0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a.row[i].load(from + (int64_t)(uint32_t)__builtin_amdgcn_readlane(at, t0 + i) * d);
      a.there[i].zero();
      if constexpr (kAdd) {
        const uint32_t id = __builtin_amdgcn_readlane(key, t0 + i);
        a.there[i].load(grad + (int64_t)(id < (uint32_t)V ? id : 0) * d + (mine ? col : 0));
      }
      __builtin_amdgcn_sched_barrier(0);  // in the order in which they are used
    }
  };
  const auto add = [&](const Ahead& a, int t0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = t0 + i;
      float f[8];
      a.row[i].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
      const uint32_t id = __builtin_amdgcn_readlane(key, t);
      const uint32_t next = t + 1 < n ? __builtin_amdgcn_readlane(key, t + 1) : behind;
      if (t >= n || (t + 1 < n && next == id)) continue;
      // the id's last token of the piece
      if (id < (uint32_t)V && mine) {
        const bool whole = (first > 0 || front != id) && next != id;
        if (whole)
          put_row<TO, kAdd>(grad + (int64_t)id * d + col, sum, scale, a.there[i]);
        else
          Piece<float>::store(part + (2 * p + (first > 0 ? 1 : 0)) * d + col, sum);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
      first = t + 1;
    }
  };
  load(ahead[0], 0);
  for (int t0 = 0; t0 < n; t0 += 2 * kAhead) {
    if (t0 + kAhead < n) load(ahead[1], t0 + kAhead);
    add(ahead[0], t0);
    if (t0 + 2 * kAhead < n) load(ahead[0], t0 + 2 * kAhead);
    add(ahead[1], t0 + kAhead);
  }
}

// Sums of 64 pieces (from a multiple of 64 on) that hold one id alone, [group][d]: an id
// of very many tokens is then joined from them.
constexpr int kGroup = 64;
__global__ __launch_bounds__(kBlock) void embed_group_kernel(const uint32_t* __restrict__ keys,
                                                             const float* __restrict__ part,
                                                             float* __restrict__ group, int64_t N,
                                                             int64_t d, int piece) {
  __shared__ float4 s[4][64];
  const int64_t p = (int64_t)blockIdx.x * kGroup;
  if ((p + kGroup) * piece > N || keys[p * piece] != keys[(p + kGroup) * piece - 1]) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t col = (int64_t)blockIdx.y * 256 + 4 * lane;
  float4 a = make_float4(0, 0, 0, 0);
  if (col < d) {
#pragma unroll 8
    for (int q = wave; q < kGroup; q += 4) {
      const float4 v = *reinterpret_cast<const float4*>(part + 2 * (p + q) * d + col);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
  s[wave][lane] = a;
  __syncthreads();
  if (wave > 0 || col >= d) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 v = s[w][lane];
    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
  }
  *reinterpret_cast<float4*>(group + blockIdx.x * d + col) = a;
}

// The rows of ids that reach over pieces: the workgroups of the piece in which
// one begins add its pieces' sums, 4 waves every fourth and then each other's,
// 256 columns each; of the whole groups of pieces behind it their groups' (group, or null).
template <typename TO, bool kAdd>
__global__ __launch_bounds__(kBlock) void embed_join_kernel(
    const uint32_t* __restrict__ keys, const float* __restrict__ part, TO* __restrict__ grad,
    const float* __restrict__ group, int64_t N, int64_t V, int64_t d, float scale, int piece,
    unsigned pieces, int64_t zero0) {
  __shared__ float s[4][256];
  if (blockIdx.x >= pieces) {  // the last rows' zeros
    const int64_t v0 = zero0 + kZeroRows * (((int64_t)(blockIdx.x - pieces) * gridDim.y +
                                             blockIdx.y) * (kBlock / 64) + (threadIdx.x >> 6));
    if (v0 < V) zero_rows(keys, grad, N, V, d, v0);
    return;
  }
  const int64_t p = blockIdx.x, n0 = p * piece;
  const int64_t last = min<int64_t>(n0 + piece, N) - 1;
  if (last + 1 >= N) return;
  const uint32_t id = keys[last];
  if (id >= (uint32_t)V || keys[last + 1] != id) return;
  const bool inside = keys[n0] != id;  // begins behind the piece's first token
  if (!inside && n0 > 0 && keys[n0 - 1] == id) return;  // began in an earlier piece
  const int64_t c = (int64_t)blockIdx.y * 256 + 8 * threadIdx.x;  // what a thread puts in the end
  Piece<TO> there;
  there.zero();
  if (kAdd && threadIdx.x < 32 && c < d) there.load(grad + (int64_t)id * d + c);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int64_t end = p;  // the id's last piece: those behind p begin with it
  for (;;) {
    const int64_t n = (end + 1 + lane) * piece;
    const uint64_t other = __ballot(n >= N || keys[n] != id);
    if (other) {
      end += __builtin_ctzll(other);
      break;
    }
    end += 64;
  }
  const int64_t col = (int64_t)blockIdx.y * 256 + 4 * lane;
  float4 a = make_float4(0, 0, 0, 0);
  // pieces p .. head - 1 and tail .. end, groups head / kGroup .. tail / kGroup - 1; the
  // id fills the groups: it begins in front of them and goes on to end, whose last tokens
  // may be another's, so that end is in none
  int64_t head = end + 1, tail = end + 1;
  if (group && end / kGroup > p / kGroup + 1)
    head = (p / kGroup + 1) * kGroup, tail = end / kGroup * kGroup;
  if (col < d) {
    const auto add = [&](const float* from) {
      const float4 v = *reinterpret_cast<const float4*>(from + col);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    };
#pragma unroll 8
    for (int64_t q = p + wave; q < head; q += 4) add(part + (2 * q + (q == p && inside ? 1 : 0)) * d);
#pragma unroll 8
    for (int64_t g = head / kGroup + wave; g < tail / kGroup; g += 4) add(group + g * d);
#pragma unroll 8
    for (int64_t q = tail + wave; q <= end; q += 4) add(part + 2 * q * d);
  }
  *reinterpret_cast<float4*>(&s[wave][4 * lane]) = a;
  __syncthreads();
  if (threadIdx.x >= 32 || c >= d) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int x = 8 * threadIdx.x + j;
    sum[j] = (s[0][x] + s[1][x]) + (s[2][x] + s[3][x]);
  }
  put_row<TO, kAdd>(grad + (int64_t)id * d + c, sum, scale, there);
}

// The whole gradient of up to 64 tokens: every wave has all ids, one a lane.  A wave sums
// kWaveCols columns of one id's tokens in the order of their places; behind those waves come
// the ones for the zeros.  (1024 columns, here / in the launches above: 64 tokens added 5.6 /
// 13.5 us, 64 into 2000 rows 7.8 / 17; 64 of one id into 2000 rows of 2560 7.3 / 13.8, added.)
constexpr int kFew = 64;
template <typename T, typename TO, bool kAdd>
__global__ __launch_bounds__(kBlock) void embed_few_kernel(SortIn in, const T* __restrict__ dout,
                                                           TO* __restrict__ grad, int64_t d,
                                                           float scale, int64_t units,
                                                           int col_parts) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kBlock / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // wave-uniform
  const uint32_t key = lane < (int)in.N ? in.key(lane) : (uint32_t)in.V;
  if (unit >= units) {
    if constexpr (!kAdd) {
      const int64_t step = ((int64_t)gridDim.x * (kBlock / 64) - units) * kZeroRows;
      for (int64_t v0 = (unit - units) * kZeroRows; v0 < in.V; v0 += step) {
        bool has = false;
        for (int t = 0; t < (int)in.N; ++t)
          has |= (int64_t)(uint32_t)__builtin_amdgcn_readlane(key, t) == v0 + lane;
        put_zeros(grad, d, v0, __ballot(lane < kZeroRows && v0 + lane < in.V && !has));
      }
    }
    return;
  }
  const int first = (int)(unit / col_parts);
  const uint32_t id = __builtin_amdgcn_readlane(key, first);
  uint64_t mine = __ballot(key == id);
  if (id >= (uint32_t)in.V || __builtin_ctzll(mine) != first) return;  // none, or another wave's
  const int64_t col = (unit % col_parts) * kWaveCols + 8 * lane;
  if (col >= d) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  Piece<TO> there;
  there.zero();
  TO* const to = grad + (int64_t)id * d + col;
  if constexpr (kAdd) there.load(to);
  constexpr int kAhead = 8;
  while (mine) {
    Piece<T> row[kAhead];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      row[i].zero();
      if (!mine) continue;
      row[i].load(dout + (int64_t)__builtin_ctzll(mine) * d + col);
      mine &= mine - 1;
      n = i + 1;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i >= n) break;
      float f[8];
      row[i].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
    }
  }
  put_row<TO, kAdd>(to, sum, scale, there);
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
  p.tiles = (a.N + kSortBlock - 1) / kSortBlock;
  return p;
}
size_t align256(size_t n) { return (n + 255) / 256 * 256; }
// Tokens of a piece: few make more waves of shorter chains, many fewer sums that the join adds.
// us with pieces of 8 / 16 / 32, added: 3000 tokens of 512 columns 19 / 21 / 26, 10000 31 / 30 /
// 35, 24000 38 / 37 / 36; 3000 of 1024 21 / 23 / 29, 6000 33 / 32 / 35, 32000 75 / 67 / 62.
int piece_of(const EmbedArgs& a) {
  const int64_t waves = a.N * ((a.d + kWaveCols - 1) / kWaveCols);  // with pieces of one
  return waves <= 8192 ? 8 : waves <= 20480 ? 16 : kPiece;
}
int64_t pieces_of(const EmbedArgs& a) { return (a.N + piece_of(a) - 1) / piece_of(a); }

// Whether an id can have so many pieces that adding them one by one shows: with all tokens
// of one id 131072 x 1024 take 101 us in groups and 166 without, 1000000 x 64 348 and 937; a
// launch more costs a call of 131072 different ones 2 of 245 us.
bool grouped(const EmbedArgs& a) { return pieces_of(a) >= 4096; }

// Workspace: two sets of keys and places, the digits' counts, the pieces' and groups' sums.
struct GradPlan {
  size_t keys[2], pos[2], hist, total, part, group, bytes;
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
  p.group = at;
  if (grouped(a)) take((size_t)(pieces_of(a) / kGroup * a.d) * sizeof(float));
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

size_t embed_backward_bytes(const EmbedArgs& a) { return a.N <= kFew ? 0 : grad_plan(a).bytes; }

hipError_t launch_embed_backward(const EmbedArgs& a, const void* ids, const void* dout, void* grad,
                                 void* ws, hipStream_t s) {
  const auto typed = [&](auto&& go) {
    return with_types(a, [&](auto t, auto to) {
      return a.accumulate ? go(t, to, std::true_type{}) : go(t, to, std::false_type{});
    });
  };
  const int col_parts = (int)((a.d + kWaveCols - 1) / kWaveCols);
  // waves for n rows' zeros: a launch's threads are counted in 32 bits, and where 2^22 waves do
  // not take them all, they go on with further ones
  const auto zero_waves = [](int64_t n) {
    return std::min<int64_t>((n + kZeroRows - 1) / kZeroRows, (int64_t)1 << 22);
  };
  if (a.N <= kFew)
    return typed([&](auto t, auto to, auto add) {
      using T = decltype(t);
      using TO = decltype(to);
      const int64_t units = a.N * col_parts, all = units + (add ? 0 : zero_waves(a.V));
      embed_few_kernel<T, TO, add><<<dim3((unsigned)((all + 3) / 4)), kBlock, 0, s>>>(
          SortIn{ids, nullptr, nullptr, a.wide_ids, a.N, a.V}, static_cast<const T*>(dout),
          static_cast<TO*>(grad), a.d, a.scale, units, col_parts);
      return hipGetLastError();
    });
  const SortPlan sp = sort_plan(a);
  const GradPlan p = grad_plan(a);
  char* const base = static_cast<char*>(ws);
  const auto u32 = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
  uint32_t *hist = u32(p.hist), *total = u32(p.total);
  const int bins = 1 << sp.bits;
  // The first rows are zeroed whole beside the sort, as many as its launches have time for
  // (some 4 us each, 16 MB); the launches behind it leave out those that have tokens.
  const int64_t row = a.d * (int64_t)dtype_bytes(a.out_dt) / 16;
  const int64_t share = std::min<int64_t>(((int64_t)1 << 20) / row,
                                          a.V / (2 * sp.passes + 4));  // rows a launch
  int64_t zeroed = a.accumulate ? a.V : 0;
  const auto zeros = [&](int64_t own, int threads, unsigned* grid) {
    const int64_t rows = std::min(share, a.V - zeroed);
    Zeros z{static_cast<uint4*>(grad) + zeroed * row, rows * row, (int32_t)own};
    zeroed += rows;
    *grid = (unsigned)(own + std::min<int64_t>((z.n + threads - 1) / threads, (1 << 20) / threads));
    return z;
  };
  unsigned grid;
  int cur = 0;
  if (a.N <= kSmall) {
    const SortIn in{ids, nullptr, nullptr, a.wide_ids, a.N, a.V};
    const Zeros z = zeros(1, kSortBlock, &grid);
    embed_sort_kernel<<<dim3(grid), kSortBlock, 0, s>>>(in, sp.passes, sp.bits, u32(p.keys[0]),
                                                        u32(p.pos[0]), z);
    cur = 1;
  } else {
    // where a workgroup adds up the counts of all tiles as fast as another launch would
    const bool few = sp.tiles <= kFewTiles;
    for (int i = 0; i < sp.passes; ++i) {
      const int shift = i * sp.bits;
      const SortIn in{i ? nullptr : ids, u32(p.keys[cur ^ 1]), i ? u32(p.pos[cur ^ 1]) : nullptr,
                      a.wide_ids, a.N, a.V};
      Zeros z = zeros(sp.tiles, kSortBlock, &grid);
      embed_hist_kernel<<<dim3(grid), kSortBlock, 0, s>>>(in, shift, bins, hist, z);
      if (!few)
        embed_scan_kernel<<<dim3((unsigned)((bins + 63) / 64)), kSortBlock, 0, s>>>(hist, bins,
                                                                                    sp.tiles, total);
      z = zeros(sp.tiles, kSortBlock, &grid);
      embed_scatter_kernel<<<dim3(grid), kSortBlock, 0, s>>>(
          in, shift, sp.bits, sp.tiles, hist, few ? nullptr : total, u32(p.keys[cur]),
          u32(p.pos[cur]), z);
      cur ^= 1;
    }
  }
  const uint32_t *keys = u32(p.keys[cur ^ 1]), *pos = u32(p.pos[cur ^ 1]);
  float* part = reinterpret_cast<float*>(base + p.part);
  return typed([&](auto t, auto to, auto add) {
    using T = decltype(t);
    using TO = decltype(to);
    constexpr bool kAdd = decltype(add)::value;
    const int64_t units = pieces_of(a) * col_parts;  // 2^25 at most
    const int64_t late = std::min(3 * share, a.V - zeroed), zero1 = a.V - late;
    const int64_t all = units + zero_waves(zero1 - zeroed);
    embed_sum_kernel<T, TO, kAdd><<<dim3((unsigned)((all + 3) / 4)), kBlock, 0, s>>>(
        keys, pos, static_cast<const T*>(dout), static_cast<TO*>(grad), part, a.N, a.V, a.d,
        a.scale, piece_of(a), units, col_parts, zeroed, zero1);
    const unsigned pieces = (unsigned)pieces_of(a), cols = (unsigned)((a.d + 255) / 256);
    const int64_t waves = (late + kZeroRows - 1) / kZeroRows;
    const unsigned extra = (unsigned)((waves + 4 * cols - 1) / (4 * cols));
    float* const group = grouped(a) ? reinterpret_cast<float*>(base + p.group) : nullptr;
    if (group)
      embed_group_kernel<<<dim3(pieces / kGroup, cols), kBlock, 0, s>>>(keys, part, group, a.N, a.d,
                                                                        piece_of(a));
    embed_join_kernel<TO, kAdd><<<dim3(pieces + extra, cols), kBlock, 0, s>>>(
        keys, part, static_cast<TO*>(grad), group, a.N, a.V, a.d, a.scale, piece_of(a),
        pieces, zero1);
    return hipGetLastError();
  });
}

}  // namespace ttt
