// linattn.hip -- linear attention with a decay for each head.
//
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
//
// Chunked form, for chunks of C = 32 tokens with the state S in front of them:
//   O = (scale Q K^T . D) V + diag(scale g^(t+1)) Q S,   D_ts = g^(t-s) for s <= t
//   S <- g^C S + K^T diag(g^(C-1-s)) V
// The gradients are the same sums with other operands (launchers' caller), two
// of them from the last token back; LinArgs has the exponents and scales that
// differ.
//
// One workgroup walks one segment of one head with the state in registers:
// wave w holds the 32 value columns [32 w, + 32) of S as 32x32 MFMA
// accumulators over all key rows, so K, V and Q are read once and S never
// leaves the registers.  Every product is arranged so that an accumulator is
// the next product's operand without passing LDS:
//   P^T = K Q^T    lanes = query rows, registers = keys    -> B operand of V^T P^T
//   S              lanes = value columns, registers = keys -> A operand of S^T Q^T
//   O^T = S^T Q^T, scaled per query row = per lane, + V^T P^T
//   S  += K^T (w V) with V's fragments, already read for V^T P^T, weighted and
//                  split in registers
// A 32x32 result holds rows 8 (r / 4) + 4 (lane / 32) + r % 4 in registers r,
// an operand wants 8 consecutive k values 8 (lane / 32) + 0..7: the rows of
// the A operands are fed in an order with bits 2 and 3 of the index swapped
// (perm below), which makes registers 0..7 and 8..15 of a result exactly these
// runs.
//
// Few heads leave most CUs without work, so a sequence is split into segments
// (linattn_segments): one pass computes every segment's end state from K and V
// alone, one adds them up along the sequence, and the main pass starts each
// segment from its state.
//
// Rounding (bf16 operands): the decayed scores and the state's copy that
// meets Q are rounded to bf16 once, like any bf16 operand of a product whose
// result is bf16; S itself is fp32 and what is added to it is exact to about
// 2^-17, since the weighted V goes in as two bf16 terms.  fp32 operands use
// fp32 MFMAs and no rounding.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "block.h"
#include "gemm_core.h"

namespace ttt {
namespace {

constexpr int kC = kLinChunk;
constexpr float kLog2e = 1.44269504088896340736f;

// g^n for n >= 0 from log2 g (g = 0 at -inf).
__device__ __forceinline__ float decay_pow(float lg2, int n) {
  return n == 0 ? 1.0f : exp2f(lg2 * (float)n);
}

__device__ __forceinline__ int perm16(int i) {  // bits 2 and 3 swapped
  return (i & ~12) | ((i & 4) << 1) | ((i & 8) >> 1);
}

// ------------------------------------------------------- tiles and fragments
// A tile is kC token rows in LDS, cut into panels of 128 bytes per row; 16-byte
// piece c of row r of a panel is stored at c ^ lds_swz_tr(r), which is free of
// bank conflicts for row-wise 16-byte reads and for the transposing reads.
template <typename T>
struct Tile {
  static constexpr int kPerPiece = 16 / sizeof(T);
  static constexpr int kPerPanel = kRowBytes / sizeof(T);
  __device__ __forceinline__ static uint32_t offset(int row, int col) {
    return (uint32_t)((col / kPerPanel) * kC + row) * kRowBytes +
           (uint32_t)((((col % kPerPanel) / kPerPiece) ^ lds_swz_tr(row)) << 4) +
           (uint32_t)((col % kPerPiece) * sizeof(T));
  }
};

// A fragment is 8 values of k, 16 step + 8 (lane / 32) + 0..7, of one row (A) or
// column (B) per lane.
template <typename T>
struct Frag;

template <>
struct Frag<uint16_t> {
  bf16x8_t v;
  // k along the tile's columns: row `row`, columns 16 step + 8 (lane / 32) ..
  __device__ __forceinline__ static Frag rows(const lds_char* t, int row, int step, int lane) {
    return {lds_load<bf16x8_t>(t + Tile<uint16_t>::offset(row, 16 * step + 8 * (lane >> 5)))};
  }
  // k along the tile's rows (tokens): lane l takes column col0 + perm16(l % 32).
  // The transposing read gives lane j of 16 the columns of the word that
  // lanes j / 4 (mod 4) address, four rows of them; see read_a_tr.
  __device__ __forceinline__ static Frag cols(const lds_char* t, int col0, int step, int lane) {
    const int g = lane >> 4, j = lane & 15, w = j & 3;
    const int col = col0 + 16 * (g & 1) + 4 * (((w & 1) << 1) | (w >> 1));
    const int row = 16 * step + 8 * (g >> 1) + (j >> 2);
    bf16x4_t x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      x[h] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
          (__attribute__((address_space(3))) bf16x4_t*)(t + Tile<uint16_t>::offset(row + 4 * h, col)));
    return {bf16x8_t{x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]}};
  }
  // registers 8 half .. of a result
  __device__ __forceinline__ static Frag result(const floatx16_t& c, int half) {
    Frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = static_cast<__bf16>(c[8 * half + e]);
    return f;
  }
};

template <>
struct Frag<float> {
  float v[8];
  __device__ __forceinline__ static Frag rows(const lds_char* t, int row, int step, int lane) {
    Frag f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const floatx4_t x =
          lds_load<floatx4_t>(t + Tile<float>::offset(row, 16 * step + 8 * (lane >> 5) + 4 * q));
#pragma unroll
      for (int e = 0; e < 4; ++e) f.v[4 * q + e] = x[e];
    }
    return f;
  }
  __device__ __forceinline__ static Frag cols(const lds_char* t, int col0, int step, int lane) {
    Frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.v[e] = lds_load<float>(
          t + Tile<float>::offset(16 * step + 8 * (lane >> 5) + e, col0 + perm16(lane & 31)));
    return f;
  }
  __device__ __forceinline__ static Frag result(const floatx16_t& c, int half) {
    Frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = c[8 * half + e];
    return f;
  }
};

__device__ __forceinline__ void mma(floatx16_t& c, const Frag<uint16_t>& a, const Frag<uint16_t>& b) {
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ void mma(floatx16_t& c, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[e], b.v[e], c, 0, 0, 0);
}

// c += a (w v), w[e] weighting the fragment's k values.
__device__ __forceinline__ void weighted(Frag<uint16_t>* hi, Frag<uint16_t>* lo,
                                         const Frag<uint16_t>& v, const float w[8], float base) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = static_cast<float>(v.v[e]) * (w[e] * base);
    hi->v[e] = static_cast<__bf16>(x);
    lo->v[e] = static_cast<__bf16>(x - static_cast<float>(hi->v[e]));
  }
}
__device__ __forceinline__ void weighted(Frag<float>* hi, Frag<float>*, const Frag<float>& v,
                                         const float w[8], float base) {
#pragma unroll
  for (int e = 0; e < 8; ++e) hi->v[e] = v.v[e] * (w[e] * base);
}

// 8 results in a row, to the operands' type or fp32.
__device__ __forceinline__ void store8(uint16_t* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// The pieces of one operand's tile that a thread carries from memory to LDS.
template <typename T, int kCols, int kThreads>
struct Stage {
  static constexpr int kPerRow = kCols / Tile<T>::kPerPiece;
  static constexpr int kCount = kC * kPerRow / kThreads;
  static_assert(kC * kPerRow % kThreads == 0, "whole pieces per thread");
  uint4 v[kCount];
  // Rows [skip, kC) of the tile are tokens first, first + 1, ... (first - 1, ...
  // when step is negative) of `base`; other rows and columns from d on are 0.
  __device__ __forceinline__ void load(const T* base, int64_t step, int skip, int d) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int p = (int)threadIdx.x + i * kThreads;
      const int row = p / kPerRow, col = (p % kPerRow) * Tile<T>::kPerPiece;
      v[i] = make_uint4(0, 0, 0, 0);
      if (row >= skip && col < d)
        v[i] = *reinterpret_cast<const uint4*>(base + (int64_t)(row - skip) * step + col);
    }
  }
  __device__ __forceinline__ void store(lds_char* t) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int p = (int)threadIdx.x + i * kThreads;
      lds_store<u32x4_t>(
          t + Tile<T>::offset(p / kPerRow, (p % kPerRow) * Tile<T>::kPerPiece), as_u32x4(v[i]));
    }
  }
};

template <typename T>
__device__ __forceinline__ const T* head_base(const LinOperand& o, int64_t b, int64_t h) {
  return static_cast<const T*>(o.p) + b * o.sb + (h / o.rep) * o.sh;
}

__device__ __forceinline__ int64_t live_tokens(const int32_t* lengths, int64_t b, int64_t T) {
  if (!lengths) return T;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > T ? T : n;
}

// DK: key columns of the tiles (64 or 128, at least dk); NW waves of 32 value
// columns.  kOut: the main pass; otherwise the pass that leaves each segment's
// end state in `seg`, which holds a start state per segment: slot g + 1 gets
// segment g's end, slot 0 the state the sequence starts from (the main pass
// reads it from there, since s_out may be s_in).
template <typename T, int DK, int NW, bool kOut>
__global__ __launch_bounds__(64 * NW, 2) void linattn_chunked_kernel(LinArgs a, float* seg,
                                                                     int64_t seg_len, int nseg) {
  constexpr int kThreads = 64 * NW, DV = 32 * NW, KT = DK / 32;
  constexpr bool kSplit = sizeof(T) == 2;
  __shared__ __attribute__((aligned(16))) char smem[kC * (2 * DK + DV) * sizeof(T)];
  lds_char* sK = (lds_char*)smem;
  lds_char* sV = sK + kC * DK * sizeof(T);
  lds_char* sQ = sV + kC * DV * sizeof(T);

  const int per = kOut ? nseg : nseg - 1;  // nobody starts from the last segment's end
  const int g = (int)(blockIdx.x % per);
  const int64_t bh = blockIdx.x / per, b = bh / a.H, h = bh % a.H;
  const int64_t n = live_tokens(a.lengths, b, a.T);
  const int64_t t_lo = g * seg_len, t_hi = min(t_lo + seg_len, n);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int dk = (int)a.dk, dv = (int)a.dv;
  const int64_t slot_size = (int64_t)DK * DV;
  float* slot = seg ? seg + (bh * nseg + g) * slot_size + (int64_t)wave * KT * 16 * 64 + lane
                    : nullptr;

  // ---- the state: registers r of tile i hold key row 32 i + 16 (r / 8) + 8 half
  // + r % 8 of value column 32 wave + perm16(lane % 32)
  const int col = 32 * wave + perm16(lane & 31);
  floatx16_t S[KT];
  const auto state_at = [&](int i, int r) -> int64_t {
    const int row = 32 * i + 16 * (r >> 3) + 8 * half + (r & 7);
    if (row >= dk || col >= dv) return -1;
    return bh * dk * dv + (a.s_trans ? (int64_t)col * dk + row : (int64_t)row * dv + col);
  };
  if (g > 0 && t_lo < n && kOut) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[i][r] = slot[(i * 16 + r) * 64];
  } else if (g == 0 && kOut && slot) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[i][r] = slot[(i * 16 + r) * 64];
  } else {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        S[i][r] = 0.0f;
        if (g == 0 && a.s_in) {
          const int64_t at = state_at(i, r);
          if (at >= 0) S[i][r] = a.s_in[at];
        }
      }
    if (!kOut && g == 0) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) slot[(i * 16 + r) * 64] = S[i][r];
    }
  }

  // ---- decay factors
  const float lg2 = a.log_decay[h] * kLog2e;
  const int qrow = lane & 31;
  float w8[8];       // g^(7-e)
  float w_base[2];   // update: scale_u g^(kC - late - 16 step - 8 half - 7), times w8 = the token's
  float d_in[16];    // scores: scale_p g^(query - key), register = key
#pragma unroll
  for (int e = 0; e < 8; ++e) w8[e] = decay_pow(lg2, 7 - e);
#pragma unroll
  for (int s = 0; s < 2; ++s)
    w_base[s] = a.scale_u * decay_pow(lg2, kC - a.late - 16 * s - 8 * half - 7);
  if constexpr (kOut) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int dist = qrow - (16 * (r >> 3) + 8 * half + (r & 7));
      d_in[r] = dist >= 0 ? a.scale_p * decay_pow(lg2, dist) : 0.0f;
    }
  }
  float f_out = a.scale_o * decay_pow(lg2, qrow + a.late);  // query row's factor on Q S
  // g^kC as 1 + (g^kC - 1) where it is near 1: the rounded factor is applied
  // once per chunk, and its error would grow with the number of chunks that
  // the state remembers
  float step_m1 = expm1f(a.log_decay[h] * (float)kC), step = decay_pow(lg2, kC);
  const auto decay_state = [&] {
    if (step > 0.5f) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[i][r] = fmaf(S[i][r], step_m1, S[i][r]);
    } else {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[i][r] *= step;
    }
  };

  // ---- token rows: token t of the walk is row t, or row n - 1 - t of the tensors
  const T* kp = head_base<T>(a.k, b, h);
  const T* vp = head_base<T>(a.v, b, h);
  const T* qp = head_base<T>(a.q, b, h);
  const int64_t dir = a.reverse ? -1 : 1;
  Stage<T, DK, kThreads> stK, stQ;
  Stage<T, DV, kThreads> stV;
  const auto load = [&](int64_t t) {
    // a last chunk of m < kC tokens fills the tile's last m rows, so that every
    // weight above is the same as in a whole chunk
    const int skip = (int)max((int64_t)0, kC - (t_hi - t));
    const int64_t row = a.reverse ? n - 1 - t : t;
    stK.load(kp + row * a.k.st, dir * a.k.st, skip, dk);
    stV.load(vp + row * a.v.st, dir * a.v.st, skip, dv);
    if constexpr (kOut) stQ.load(qp + row * a.q.st, dir * a.q.st, skip, dk);
  };
  if (t_lo < t_hi) load(t_lo);

  for (int64_t t = t_lo; t < t_hi; t += kC) {
    __syncthreads();  // every wave is done with the last chunk's tiles
    stK.store(sK);
    stV.store(sV);
    if constexpr (kOut) stQ.store(sQ);
    __syncthreads();
    const int m = (int)min((int64_t)kC, t_hi - t), skip = kC - m;
    if (t + kC < t_hi) load(t + kC);
    if (skip) {  // the last chunk
      f_out = a.scale_o * decay_pow(lg2, max(0, qrow - skip) + a.late);
      step_m1 = expm1f(a.log_decay[h] * (float)m);
      step = decay_pow(lg2, m);
    }
    Frag<T> vf[2];  // V^T: value column col, tokens
#pragma unroll
    for (int s = 0; s < 2; ++s) vf[s] = Frag<T>::cols(sV, 32 * wave, s, lane);

    if constexpr (kOut) {
      floatx16_t P, O;
#pragma unroll
      for (int r = 0; r < 16; ++r) P[r] = O[r] = 0.0f;
#pragma unroll
      for (int s = 0; s < DK / 16; ++s) {
        const Frag<T> qf = Frag<T>::rows(sQ, qrow, s, lane);
        const Frag<T> kf = Frag<T>::rows(sK, perm16(qrow), s, lane);
        mma(P, kf, qf);
        mma(O, Frag<T>::result(S[s >> 1], s & 1), qf);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        O[r] *= f_out;
        P[r] = qrow >= 16 * (r >> 3) + 8 * half + (r & 7) ? P[r] * d_in[r] : 0.0f;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) mma(O, vf[s], Frag<T>::result(P, s));
      // registers 8 i .. of O: columns 32 wave + 16 i + 8 half .. of the lane's token
      const int64_t tok = t + qrow - skip;
      if (qrow >= skip) {
        const int64_t row = a.reverse ? n - 1 - tok : tok;
        const int64_t at = b * a.osb + row * a.ost + h * a.osh;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = 32 * wave + 16 * i + 8 * half;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = O[8 * i + e];
          if (c < dv) {
            if (a.out_f32)
              store8(static_cast<float*>(a.out) + at + c, f);
            else
              store8(static_cast<T*>(a.out) + at + c, f);
          }
        }
      }
    }

    // ---- S <- g^m S + K^T (w V)
    decay_state();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Frag<T> hi, lo;
      weighted(&hi, &lo, vf[s], w8, w_base[s]);
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const Frag<T> kf = Frag<T>::cols(sK, 32 * i, s, lane);
        mma(S[i], kf, hi);
        if constexpr (kSplit) mma(S[i], kf, lo);
      }
    }
  }

  if constexpr (!kOut) {
    float* next = slot + slot_size;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) next[(i * 16 + r) * 64] = S[i][r];
  } else {
    const bool last = t_hi == n && (t_lo < n || g == 0);  // this segment holds the last token
    if (last && a.s_out) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t at = state_at(i, r);
          if (at >= 0) a.s_out[at] = S[i][r];
        }
    }
    // rows behind the sequence's end
    const int64_t z_lo = max(t_lo, n), z_hi = min(t_lo + seg_len, a.T);
    const int pieces = dv >> 3;
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t p = threadIdx.x; p < (z_hi - z_lo) * pieces; p += kThreads) {
      const int64_t at = b * a.osb + (z_lo + p / pieces) * a.ost + h * a.osh + (p % pieces) * 8;
      if (a.out_f32)
        store8(static_cast<float*>(a.out) + at, zero);
      else
        store8(static_cast<T*>(a.out) + at, zero);
    }
  }
}

// seg[bh][g] <- seg[bh][g] + g^seg_len seg[bh][g - 1] along the segments, so
// that every slot is the state its segment starts from.  Slots of segments
// behind a sequence's end are not used.
__global__ __launch_bounds__(256) void linattn_scan_kernel(float4* seg,
                                                           const float* __restrict__ log_decay,
                                                           int64_t H, int64_t slot4, int64_t total,
                                                           int64_t seg_len, int nseg) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t bh = i / slot4, e = i % slot4;
  const float f = exp2f(log_decay[bh % H] * kLog2e * (float)seg_len);
  float4* p = seg + bh * nseg * slot4 + e;
  float4 acc = p[slot4];
#pragma unroll 4
  for (int g = 2; g < nseg; ++g) {
    float4 x = p[g * slot4];
    x.x = fmaf(f, acc.x, x.x), x.y = fmaf(f, acc.y, x.y);
    x.z = fmaf(f, acc.z, x.z), x.w = fmaf(f, acc.w, x.w);
    p[g * slot4] = acc = x;
  }
}

// ------------------------------------------------------------ recurrent form
// Bound by reading and writing the state once.  A workgroup takes 32 value
// columns of one head: 8 threads of 4 columns by 32 row groups of 4 key rows
// (rows group, group + 32, ...), all four 16-byte loads of a thread issued
// together; its tokens then run in registers, and the sums over the key rows
// end in LDS after the last token.
constexpr int kStepCols = 32;

__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinArgs a) {
  __shared__ float part[kLinStepTokens][4][kStepCols];
  const int slices = (int)((a.dv + kStepCols - 1) / kStepCols);
  const int64_t bh = blockIdx.x / slices, b = bh / a.H, h = bh % a.H;
  const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
  const int col = (int)(blockIdx.x % slices) * kStepCols + 4 * cg;
  const bool live_col = col < a.dv;
  const int dk = (int)a.dk, dv = (int)a.dv;
  const int n = (int)live_tokens(a.lengths, b, a.T);
  const int64_t base = bh * dk * dv + col;
  float S[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = rg + 32 * i;
    float4 x = make_float4(0, 0, 0, 0);
    if (a.s_in && live_col && row < dk)
      x = *reinterpret_cast<const float4*>(a.s_in + base + (int64_t)row * dv);
    S[i][0] = x.x, S[i][1] = x.y, S[i][2] = x.z, S[i][3] = x.w;
  }
  const float lg = a.log_decay[h];
  const float g = expf(lg);
  const T* qp = head_base<T>(a.q, b, h);
  const T* kp = head_base<T>(a.k, b, h);
  const T* vp = head_base<T>(a.v, b, h);
  for (int t = 0; t < n; ++t) {
    float q[4], k[4], v[4], o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = rg + 32 * i;
      q[i] = row < dk ? to_f32(qp[t * a.q.st + row]) : 0.0f;
      k[i] = row < dk ? to_f32(kp[t * a.k.st + row]) : 0.0f;
      v[i] = live_col ? to_f32(vp[t * a.v.st + col + i]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] = fmaf(g, S[i][j], k[i] * v[j]);
        o[j] = fmaf(q[i], S[i][j], o[j]);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int m = 8; m <= 32; m <<= 1) o[j] += __shfl_xor(o[j], m, 64);
      if ((threadIdx.x & 63) < 8) part[t][threadIdx.x >> 6][4 * cg + j] = o[j];
    }
  }
  if (a.s_out && live_col) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = rg + 32 * i;
      if (row < dk)
        *reinterpret_cast<float4*>(a.s_out + base + (int64_t)row * dv) =
            make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
    }
  }
  __syncthreads();
  const int64_t c0 = (blockIdx.x % slices) * kStepCols;
  for (int p = threadIdx.x; p < a.T * kStepCols; p += 256) {
    const int t = p / kStepCols, c = p % kStepCols;
    if (c0 + c >= dv) continue;
    float o = 0.0f;
    if (t < n) o = a.scale_o * (((part[t][0][c] + part[t][1][c]) + part[t][2][c]) + part[t][3][c]);
    Elem<T>::store(static_cast<T*>(a.out) + b * a.osb + t * a.ost + h * a.osh + c0 + c, o);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void linattn_sum_heads_kernel(
    const float* __restrict__ part, T* __restrict__ out, int64_t osb, int64_t ost, int64_t osh,
    int64_t B, int64_t T_, int64_t G, int64_t rep, int64_t d) {
  const int64_t pieces = d >> 3;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= B * G * T_ * pieces) return;
  const int64_t c = (i % pieces) * 8, t = i / pieces % T_, g = i / (pieces * T_) % G,
                b = i / (pieces * T_ * G);
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t r = 0; r < rep; ++r) {
    const float* p = part + (((b * G + g) * rep + r) * T_ + t) * d + c;
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
    f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w;
    f[4] += y.x, f[5] += y.y, f[6] += y.z, f[7] += y.w;
  }
  store8(out + b * osb + t * ost + g * osh + c, f);
}

template <typename T, int DK, int NW>
hipError_t chunked(const LinArgs& a, float* seg, int64_t seg_len, int nseg, hipStream_t s) {
  const int64_t heads = a.B * a.H;
  if (nseg > 1) {
    linattn_chunked_kernel<T, DK, NW, false>
        <<<dim3((unsigned)(heads * (nseg - 1))), 64 * NW, 0, s>>>(a, seg, seg_len, nseg);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (nseg > 2) {
      const int64_t slot4 = DK * 32 * NW / 4, total = heads * slot4;
      linattn_scan_kernel<<<dim3((unsigned)((total + 255) / 256)), 256, 0, s>>>(
          reinterpret_cast<float4*>(seg), a.log_decay, a.H, slot4, total, seg_len, nseg);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  linattn_chunked_kernel<T, DK, NW, true><<<dim3((unsigned)(heads * nseg)), 64 * NW, 0, s>>>(
      a, nseg > 1 ? seg : nullptr, seg_len, nseg);
  return hipGetLastError();
}

template <typename T>
hipError_t chunked_shape(const LinArgs& a, float* seg, int64_t seg_len, int nseg, hipStream_t s) {
  if (a.dk <= 64)
    return a.dv <= 64 ? chunked<T, 64, 2>(a, seg, seg_len, nseg, s)
                      : chunked<T, 64, 4>(a, seg, seg_len, nseg, s);
  return a.dv <= 64 ? chunked<T, 128, 2>(a, seg, seg_len, nseg, s)
                    : chunked<T, 128, 4>(a, seg, seg_len, nseg, s);
}

int64_t segment_tokens(int64_t T, int64_t nseg) {
  return (((T + nseg - 1) / nseg) + kC - 1) / kC * kC;
}

}  // namespace

int64_t linattn_segments(int64_t B, int64_t H, int64_t T) {
  const int64_t heads = B * H;
  int64_t nseg = std::min<int64_t>((512 + heads - 1) / heads, T / 256);
  if (heads >= 256 || nseg <= 1) return 1;
  // whole chunks per segment may need fewer segments
  const int64_t len = segment_tokens(T, nseg);
  return (T + len - 1) / len;
}

size_t linattn_segment_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv) {
  const int64_t nseg = linattn_segments(B, H, T);
  if (nseg == 1) return 0;
  return (size_t)(B * H * nseg) * (dk <= 64 ? 64 : 128) * (dv <= 64 ? 64 : 128) * sizeof(float);
}

hipError_t launch_linattn_chunked(const LinArgs& a, float* seg, hipStream_t s) {
  const int64_t nseg = linattn_segments(a.B, a.H, a.T);
  const int64_t seg_len = segment_tokens(a.T, nseg);
  return a.dt == Dtype::BF16 ? chunked_shape<uint16_t>(a, seg, seg_len, (int)nseg, s)
                             : chunked_shape<float>(a, seg, seg_len, (int)nseg, s);
}

hipError_t launch_linattn_step(const LinArgs& a, hipStream_t s) {
  const int64_t slices = (a.dv + kStepCols - 1) / kStepCols;
  const dim3 grid((unsigned)(a.B * a.H * slices));
  if (a.dt == Dtype::BF16)
    linattn_step_kernel<uint16_t><<<grid, 256, 0, s>>>(a);
  else
    linattn_step_kernel<float><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_linattn_sum_heads(const float* part, void* out, int64_t osb, int64_t ost,
                                    int64_t osh, int64_t B, int64_t T, int64_t G, int64_t rep,
                                    int64_t d, Dtype dt, hipStream_t s) {
  const int64_t n = B * G * T * (d / 8);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (dt == Dtype::BF16)
    linattn_sum_heads_kernel<uint16_t><<<grid, 256, 0, s>>>(part, static_cast<uint16_t*>(out), osb,
                                                            ost, osh, B, T, G, rep, d);
  else
    linattn_sum_heads_kernel<float><<<grid, 256, 0, s>>>(part, static_cast<float*>(out), osb, ost,
                                                         osh, B, T, G, rep, d);
  return hipGetLastError();
}

}  // namespace ttt
