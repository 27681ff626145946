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
//                  split into bf16 terms in registers
// A 32x32 result holds rows 8 (r / 4) + 4 (lane / 32) + r % 4 in registers r,
// an operand wants 8 consecutive k values 8 (lane / 32) + 0..7: the rows of
// the A operands are fed in an order with bits 2 and 3 of the index swapped
// (perm16 below), which makes registers 0..7 and 8..15 of a result exactly these
// runs.
//
// Few heads leave most CUs without work, so a sequence is split into segments
// (split() below): one pass computes every segment's end state from K and V
// alone, one adds them up along the sequence, and the main pass starts each
// segment from its state.  A chunk of 32 tokens needs no larger intermediate
// than one 32x32 tile of scores a wave, and leaves two workgroups a CU; 64
// tokens would halve the state's conversions but need 96 KB of LDS a workgroup.
//
// What bounds it: 131072 tokens x 20 heads of 128 in bf16 take 830 us (870 on
// another host); reading q, k and v and writing o is 2.7 GB (540 us at a copy's
// rate).  Traced (at a lower clock, 970 us in all) the ends' pass takes 325 us (it
// reads 0.85 of K's and V's 1.34 GB, the rest has decayed to 0), the sums over
// segments 12 and the main pass 635.
// Back to back the clock falls to 1.7 from 2.2 GHz, which then costs more than
// any one of the remaining waits: without loads the same passes take 600 us.
//
// Rounding (bf16 operands): the decayed scores and the state's copy that
// meets Q are rounded to bf16 once, like any bf16 operand of a product whose
// result is bf16 (results are off by 2.0e-3 to 2.4e-3; with a second bf16 term for
// both by the 1.66e-3 of their own rounding, 15% to 18% slower: 828 and 958 us for
// 131072 tokens, 579 and 680 for the gradients of 32768).  S itself is fp32, and the weighted V goes into it as three
// bf16 terms (24 bits), so that a state that is given out is as exact as fp32
// sums make it; two terms (2^-17) where the pass's state only ever meets bf16
// operands (the gradients of q and k).  The third term costs 3% to 4% (16
// prompts of 8192 tokens: 636 us with two terms, 656 us with three).  fp32
// operands use fp32 MFMAs and no rounding; 32768 tokens x 20 heads of 128 take 944
// us, of which the matrix instructions as issued (88 GFLOP, the scores four times)
// are 575 at the fp32 matrix rate: tiles of 4 bytes leave one wave a SIMD, so that
// what is not covered within the wave is waited for.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "gemm_core.h"

namespace ttt {
namespace {

constexpr int kC = kLinChunk;
constexpr float kLog2e = 1.44269504088896340736f;

// log2 of a decay of exp(lg), finite: below any decay that is not 0 in fp32, so
// that a power of 0 is 1 and every other one 0.
__device__ __forceinline__ float log2_decay(float lg) {
  const float x = lg * kLog2e;
  return x < -1e30f ? -1e30f : x;
}
// g^n for n >= 0.  The hardware's exp2: results below 2^-126 are 0.
__device__ __forceinline__ float decay_pow(float lg2, int n) {
  return __builtin_amdgcn_exp2f(lg2 * (float)n);
}

// A value that all lanes have, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// exp(x) as the float next to it and what that leaves.  A factor that is applied
// n times with its own rounding, up to 2^-25 near 1, is off by n of them; with the
// rest each product is rounded for itself.  From |x| = 0.5 on little is left after
// a few products, and the rest is left out.
struct Decay {
  float f = 0.0f, rest = 0.0f;
  Decay() = default;
  __device__ __forceinline__ explicit Decay(float x)
      : f(expf(x)), rest(fabsf(x) < 0.5f ? expm1f(x) - (f - 1.0f) : 0.0f) {}
  // s exp(x) + y
  __device__ __forceinline__ float operator()(float s, float y) const {
    return fmaf(f, s, fmaf(rest, s, y));
  }
};

__device__ __forceinline__ int perm16(int i) {  // bits 2 and 3 swapped
  return (i & ~12) | ((i & 4) << 1) | ((i & 8) >> 1);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two values rounded to bf16 in one instruction.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2_t{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
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
  // A transposing read gives lane j of 16 the columns of the word that lanes
  // j / 4 (mod 4) address, four rows of them (see read_a_tr); rows +4 and
  // columns +32 change the swizzle, rows +16 and panels only the address.
  // LDS address of the read of rows 4 h.., columns col0 .., k step 0.
  __device__ __forceinline__ static uint32_t tr_addr(const lds_char* t, int col0, int h, int lane) {
    const int g = lane >> 4, j = lane & 15, w = j & 3;
    const int col = col0 + 16 * (g & 1) + 4 * (((w & 1) << 1) | (w >> 1));
    return (uint32_t)(uintptr_t)(t + Tile<uint16_t>::offset(8 * (g >> 1) + (j >> 2) + 4 * h, col));
  }
  // Fragments of both k steps of columns col0 ...
  __device__ __forceinline__ static void cols2(Frag (&f)[2], const lds_char* t, int col0, int lane) {
    tr4<0, 16 * kRowBytes>(f, tr_addr(t, col0, 0, lane), tr_addr(t, col0, 1, lane));
  }
  // Fragments of k step `step` of the N tiles of 32 columns from column 0.
  template <int step, int N>
  __device__ __forceinline__ static void cols_all(Frag (&f)[N], const lds_char* t, int lane) {
    constexpr int kStep = step * 16 * kRowBytes, kPanel = kC * kRowBytes;
    const uint32_t a0 = tr_addr(t, 0, 0, lane), a1 = tr_addr(t, 0, 1, lane);
    const uint32_t b0 = tr_addr(t, 32, 0, lane), b1 = tr_addr(t, 32, 1, lane);
    if constexpr (N == 2) {
      tr4(f, a0, a1, b0, b1, kStep);
    } else {
      static_assert(N == 4, "two or four tiles");
      u32x2_t x[8];
      asm volatile(
          "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
          "ds_read_b64_tr_b16 %1, %9 offset:%12\n\t"
          "ds_read_b64_tr_b16 %2, %10 offset:%12\n\t"
          "ds_read_b64_tr_b16 %3, %11 offset:%12\n\t"
          "ds_read_b64_tr_b16 %4, %8 offset:%13\n\t"
          "ds_read_b64_tr_b16 %5, %9 offset:%13\n\t"
          "ds_read_b64_tr_b16 %6, %10 offset:%13\n\t"
          "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]),
            "=&v"(x[6]), "=&v"(x[7])
          : "v"(a0), "v"(a1), "v"(b0), "v"(b1), "n"(kStep), "n"(kStep + kPanel));
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = join(x[2 * i], x[2 * i + 1]);
    }
  }
  __device__ __forceinline__ static Frag join(u32x2_t lo, u32x2_t hi) {
    return {__builtin_bit_cast(bf16x8_t, u32x4_t{lo[0], lo[1], hi[0], hi[1]})};
  }
  // The transposing reads are inline assembly, each block with its wait: the
  // compiler lets the builtin wait for every direct-to-LDS load in flight,
  // also those into the other buffer, which would end the prefetch.
  template <int kOff0, int kOff1>
  __device__ __forceinline__ static void tr4(Frag (&f)[2], uint32_t a0, uint32_t a1) {
    u32x2_t x[4];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
        "ds_read_b64_tr_b16 %1, %5 offset:%6\n\t"
        "ds_read_b64_tr_b16 %2, %4 offset:%7\n\t"
        "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
        : "v"(a0), "v"(a1), "n"(kOff0), "n"(kOff1));
    f[0] = join(x[0], x[1]);
    f[1] = join(x[2], x[3]);
  }
  __device__ __forceinline__ static void tr4(Frag (&f)[2], uint32_t a0, uint32_t a1, uint32_t b0,
                                             uint32_t b1, int off) {
    u32x2_t x[4];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n\t"
        "ds_read_b64_tr_b16 %1, %5\n\t"
        "ds_read_b64_tr_b16 %2, %6\n\t"
        "ds_read_b64_tr_b16 %3, %7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
        : "v"(a0 + off), "v"(a1 + off), "v"(b0 + off), "v"(b1 + off));
    f[0] = join(x[0], x[1]);
    f[1] = join(x[2], x[3]);
  }
  // 0, or NaN where a value is not finite
  __device__ __forceinline__ static float not_finite(const Frag (&f)[2]) {
    const bf16x2_t zero = {static_cast<__bf16>(0.0f), static_cast<__bf16>(0.0f)};
    float acc[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t x = __builtin_bit_cast(u32x4_t, f[s].v)[e];
        acc[s] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, x), zero, acc[s], false);
      }
    return acc[0] + acc[1];
  }
  __device__ __forceinline__ bool is_finite(int e) const {
    const uint32_t x = __builtin_bit_cast(u32x4_t, v)[e / 2];
    return (~(x >> 16 * (e & 1)) & 0x7f80u) != 0;
  }
  __device__ __forceinline__ void finite() {  // 0 for the values that are not
    u32x4_t x = __builtin_bit_cast(u32x4_t, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!is_finite(e)) x[e / 2] &= e & 1 ? 0xffffu : 0xffff0000u;
    v = __builtin_bit_cast(bf16x8_t, x);
  }
  // registers 8 half .. of a result
  __device__ __forceinline__ static Frag result(const floatx16_t& c, int half) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = cvt_bf16x2(c[8 * half + 2 * e], c[8 * half + 2 * e + 1]);
    return {__builtin_bit_cast(bf16x8_t, u32x4_t{w[0], w[1], w[2], w[3]})};
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
  __device__ __forceinline__ static void cols2(Frag (&f)[2], const lds_char* t, int col0, int lane) {
#pragma unroll
    for (int s = 0; s < 2; ++s) f[s] = cols(t, col0, s, lane);
  }
  template <int step, int N>
  __device__ __forceinline__ static void cols_all(Frag (&f)[N], const lds_char* t, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = cols(t, 32 * i, step, lane);
  }
  __device__ __forceinline__ static float not_finite(const Frag (&f)[2]) {
    float acc[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int s = 0; s < 2; ++s) acc[s] = fmaf(f[s].v[e], 0.0f, acc[s]);
    return acc[0] + acc[1];
  }
  __device__ __forceinline__ bool is_finite(int e) const {
    return (~__float_as_uint(v[e]) & 0x7f800000u) != 0;
  }
  __device__ __forceinline__ void finite() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = is_finite(e) ? v[e] : 0.0f;
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

// Values 2 e and 2 e + 1 of a fragment, weighted, as a sum of kTerms bf16 terms
// (or in fp32).
template <int kTerms>
__device__ __forceinline__ void weighted(Frag<uint16_t> (&out)[kTerms], const Frag<uint16_t>& v,
                                         const float* w, int e) {
  const uint32_t in = __builtin_bit_cast(u32x4_t, v.v)[e];
  float x = __uint_as_float(in << 16) * w[2 * e];
  float y = __uint_as_float(in & 0xffff0000u) * w[2 * e + 1];
#pragma unroll
  for (int i = 0; i < kTerms; ++i) {
    uint32_t top = cvt_bf16x2(x, y);
    asm("" : "+v"(top));  // one paired conversion: seen through, the halves are converted again
    u32x4_t all = __builtin_bit_cast(u32x4_t, out[i].v);
    all[e] = top;
    out[i].v = __builtin_bit_cast(bf16x8_t, all);
    x -= __uint_as_float(top << 16);
    y -= __uint_as_float(top & 0xffff0000u);
  }
}
__device__ __forceinline__ void weighted(Frag<float> (&out)[1], const Frag<float>& v,
                                         const float* w, int e) {
  out[0].v[2 * e] = v.v[2 * e] * w[2 * e];
  out[0].v[2 * e + 1] = v.v[2 * e + 1] * w[2 * e + 1];
}

template <typename T>
__device__ __forceinline__ T nan_of() {
  if constexpr (sizeof(T) == 2)
    return 0x7fc0;  // bf16
  else
    return __builtin_nanf("");
}

// 8 results in a row, to the operands' type or fp32.
__device__ __forceinline__ void store8(uint16_t* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]),
                                            cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// Direct-to-LDS loads of one operand's tile: an instruction moves 8 rows of a
// panel (1 KB, lane l to byte 16 l), NW waves share a tile's instructions.  The
// lane's source piece is chosen so that the tile comes out swizzled.  Offsets
// are from the lowest row of the chunk; columns that the head does not have, and
// rows in front of a last chunk's tokens, lie outside the descriptor's range,
// which makes their values zero.
constexpr uint32_t kRange = 0xffffff00u, kOutside = 0xffffff80u;

template <typename T, int kCols, int NW>
struct Loader {
  static constexpr int kPer = kC / 8 * (kCols / Tile<T>::kPerPanel) / NW;
  static_assert(kC / 8 * (kCols / Tile<T>::kPerPanel) % NW == 0, "whole instructions per wave");
  const char* base;     // the lowest row of the next chunk
  int64_t chunk_bytes;  // to the chunk after it
  uint32_t off[kPer];
  int row0;

  // `first`: the head's row of the walk's first token; rows of the walk are
  // `st` values apart, downwards if `reverse`.
  __device__ __forceinline__ void init(const T* first, int64_t st, bool reverse, int d, int wave,
                                       int lane) {
    const int64_t bytes = st * (int64_t)sizeof(T);
    base = reinterpret_cast<const char*>(first) - (reverse ? (kC - 1) * bytes : 0);
    chunk_bytes = reverse ? -kC * bytes : kC * bytes;
    row0 = lane >> 3;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int row = row_of(q, wave);
      const int col = panel_of(q, wave) * Tile<T>::kPerPanel +
                      ((lane & 7) ^ lds_swz_tr(row)) * Tile<T>::kPerPiece;
      off[q] = col < d ? (uint32_t)((reverse ? kC - 1 - row : row) * bytes + col * (int)sizeof(T))
                       : kOutside;
    }
  }
  __device__ __forceinline__ int row_of(int q, int wave) const {
    return (wave * kPer + q) % (kC / 8) * 8 + row0;
  }
  __device__ __forceinline__ static int panel_of(int q, int wave) {
    return (wave * kPer + q) / (kC / 8);
  }
  __device__ __forceinline__ void move(lds_char* tile, const char* from, int q, uint32_t o,
                                       int wave) const {
    const rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), (short)0,
                                                       (int)kRange, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(tile + (wave * kPer + q) * 8 * kRowBytes), 16,
        o, 0, 0, 0);
  }
  __device__ __forceinline__ void issue(lds_char* tile, int wave) {  // a whole chunk
#pragma unroll
    for (int q = 0; q < kPer; ++q) move(tile, base, q, off[q], wave);
    base += chunk_bytes;
  }
  // A last chunk, whose tokens are the tile's last kC - skip rows.
  __device__ __forceinline__ void issue_last(lds_char* tile, int skip, int wave) {
    const char* from = base - chunk_bytes / kC * skip;
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      move(tile, from, q, row_of(q, wave) >= skip ? off[q] : kOutside, wave);
  }
};

template <typename T>
__device__ __forceinline__ const T* head_base(const LinOperand& o, int64_t b, int64_t h) {
  return static_cast<const T*>(o.p) + b * o.sb + (h / o.rep) * o.sh;
}

__device__ __forceinline__ int live_tokens(const int32_t* lengths, int64_t b, int64_t T) {
  return lengths ? max(0, min(lengths[b], (int)T)) : (int)T;
}

// Which of a pass's workgroups, `per` for each head, this one is, where the
// sequences have lengths.  The first kCUs workgroups get a CU each, the next ones
// (kTwo: two fit a CU) join the first; then each takes the place of one that has
// ended.  So the shortest sequences go to the CUs that hold two, a longer one of
// them beside a shorter, and where not all are resident the longest go first.
// Lengths of T / 4 to T, 20 heads of 128, bf16, without and with it: 16 x 8192
// tokens 581 and 488 us, their gradients 1440 and 1261, 64 x 2048 437 and 427,
// 40 x 1024 163 and 161; from 1024 tokens on, as 64 x 512 with 16 heads took 95
// without and 101 with it.
constexpr uint32_t kCUs = 256;
constexpr int kOrderTokens = 1024, kOrderBatch = 64;
template <bool kTwo>
__device__ __forceinline__ uint32_t by_length(const LinArgs& a, int per) {
  const uint32_t p = blockIdx.x, all = gridDim.x;
  if (!a.lengths || all <= kCUs || a.B == 1 || a.B > kOrderBatch || a.T < kOrderTokens) return p;
  const uint32_t more = all - kCUs;
  uint32_t rank = all - 1 - p;  // among all workgroups, from the shortest sequence's
  if (kTwo && more <= kCUs) rank = p >= kCUs ? p - kCUs : p < more ? 2 * more - 1 - p : p + more;
  const uint32_t each = (uint32_t)(a.H * per);  // workgroups of a sequence
  const int lane = threadIdx.x & 63, count = (int)a.B;
  const int n = live_tokens(a.lengths, min(lane, count - 1), a.T);
  int shorter = 0;
  for (int j = 0; j < count; ++j) {
    const int other = __builtin_amdgcn_readlane(n, j);
    shorter += other < n || (other == n && j < lane);
  }
  const uint64_t mine = __builtin_amdgcn_ballot_w64(lane < count && shorter == (int)(rank / each));
  return (uint32_t)__builtin_ctzll(mine) * each + rank % each;
}

// Up to so many segments the main pass adds their ends up itself.
constexpr int kScanInPlace = 8;

// DK: key columns of the tiles (64 or 128, at least dk); NW waves of 32 value
// columns.  kOut: the main pass; otherwise the pass that leaves each segment's
// end state in `seg`, which holds a start state per segment: slot g + 1 gets
// segment g's end, slot 0 the state the sequence starts from (the main pass
// reads it from there, since s_out may be s_in).
// kPair: two passes side by side that share their operands, each with NW waves of
// its own: the one that `a` describes, and the one with q = w, k = v, v = k and
// its outputs in out2, whose state is the first one's transposed (the gradients
// of v and k: k, q, dO and v, dO, q).
template <typename T, int DK, int NW, bool kOut, int kTerms, bool kF32Out, bool kPair>
__device__ __forceinline__ void chunked_pass(const LinArgs& a, float4* seg, int seg_len, int nseg) {
  constexpr int kThreads = 64 * NW, DV = 32 * NW, KT = DK / 32, kAllWaves = NW * (kPair ? 2 : 1);
  constexpr int kOffV = kC * DK * sizeof(T), kOffQ = kOffV + kC * DV * sizeof(T);
  constexpr int kOffW = kOffQ + (kOut ? kC * DK * (int)sizeof(T) : 0);
  constexpr int kBuf = kOffW + (kPair ? kC * DV * (int)sizeof(T) : 0);
  static_assert(!kPair || (kOut && DK == DV), "the two passes have tiles of one shape");
  __shared__ __attribute__((aligned(16))) char smem[2 * kBuf];

  const int per = kOut ? nseg : nseg - 1;  // nobody starts from the last segment's end
  const uint32_t at = kOut ? __builtin_amdgcn_readfirstlane(
                                 by_length<sizeof(T) == 2 && !kPair>(a, per))
                           : blockIdx.x;
  const int g = (int)(at % per);
  const int64_t bh = at / per, b = bh / a.H, h = bh % a.H;
  const int n = live_tokens(a.lengths, b, a.T);
  const float lg = a.log_decay[h];
  int t_lo = g * seg_len;
  const int t_hi = min(t_lo + seg_len, n);
  if constexpr (!kOut) {
    // tokens whose decay to the segment's end is 0 in fp32 (below 2^-150) do
    // not reach the state there
    const float reach = -104.0f / lg;
    if (lg < 0.0f && reach < (float)(t_hi - t_lo))
      t_lo = max(t_lo, t_hi - ((int)reach / kC + 1) * kC);
  }
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int uwave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pass = kPair ? uwave / NW : 0, wave = uwave % NW, tid = wave * 64 + lane;
  const int dk = (int)(pass ? a.dv : a.dk), dv = (int)(pass ? a.dk : a.dv);
  // ---- token rows: token t of the walk is row t, or row n - 1 - t of the tensors
  const int64_t row0 = a.reverse ? n - 1 - t_lo : t_lo;
  Loader<T, DK, kAllWaves> ldK, ldQ;
  Loader<T, DV, kAllWaves> ldV, ldW;
  const auto first = [&](const LinOperand& o) { return head_base<T>(o, b, h) + row0 * o.st; };
  ldK.init(first(a.k), a.k.st, a.reverse, (int)a.dk, uwave, lane);
  ldV.init(first(a.v), a.v.st, a.reverse, (int)a.dv, uwave, lane);
  if constexpr (kOut) ldQ.init(first(a.q), a.q.st, a.reverse, (int)a.dk, uwave, lane);
  if constexpr (kPair) ldW.init(first(a.w), a.w.st, a.reverse, (int)a.dv, uwave, lane);
  const auto issue = [&](int t, lds_char* tiles_of) {
    // a last chunk of m < kC tokens fills the tiles' last m rows, so that every
    // weight below is the same as in a whole chunk
    const int skip = kC - (t_hi - t);
    if (skip <= 0) {
      ldK.issue(tiles_of, uwave);
      ldV.issue(tiles_of + kOffV, uwave);
      if constexpr (kOut) ldQ.issue(tiles_of + kOffQ, uwave);
      if constexpr (kPair) ldW.issue(tiles_of + kOffW, uwave);
    } else {
      ldK.issue_last(tiles_of, skip, uwave);
      ldV.issue_last(tiles_of + kOffV, skip, uwave);
      if constexpr (kOut) ldQ.issue_last(tiles_of + kOffQ, skip, uwave);
      if constexpr (kPair) ldW.issue_last(tiles_of + kOffW, skip, uwave);
    }
  };
  if (t_lo < t_hi) issue(t_lo, (lds_char*)smem);  // on its way while the rest is set up

  // a slot of the workspace: register 4 r.. of tile i of wave w at float4
  // ((w KT + i) 4 + r) 64 + lane
  const int64_t slot4 = (int64_t)DK * DV / 4;
  float4* slot = seg ? seg + bh * nseg * slot4 : nullptr;

  // ---- the state: registers r of tile i hold key row 32 i + 16 (r / 8) + 8 half
  // + r % 8 of value column 32 wave + perm16(lane % 32)
  const int col = 32 * wave + perm16(lane & 31);
  floatx16_t S[KT];
  const bool s_trans = a.s_trans != (pass == 1);
  const int rs = s_trans ? 1 : dv, cs = s_trans ? dk : 1;  // steps of a key row, a value column
  const int64_t head_state = bh * dk * dv;
  const auto state_row = [&](int i, int r) { return 32 * i + 16 * (r >> 3) + 8 * half + (r & 7); };
  const int at0 = 8 * half * rs + col * cs;
  const auto state_off = [&](int i, int r) { return at0 + (32 * i + 16 * (r >> 3) + (r & 7)) * rs; };
  const auto from_slot = [&](int64_t j, const Decay& f) {  // S = f S + slot j
    const float4* p = slot + j * slot4;
    if (kPair ? pass == 1 : a.seg_trans) {
      // written by the pass with keys and values exchanged: this lane's key row
      // is its value column, in tile `wave` of the wave that has it
      const int w = col & 31, lane_bits = ((w >> 3) & 1) * 32;
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int other = perm16(16 * (r >> 3) + 8 * half + (r & 7)) + lane_bits;
          const float x = reinterpret_cast<const float*>(
              p + ((i * NW + wave) * 4 + 2 * (w >> 4) + ((w & 7) >> 2)) * 64 + other)[w & 3];
          S[i][r] = f(S[i][r], x);
        }
      return;
    }
    p += wave * KT * 4 * 64 + lane;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 x = p[(i * 4 + r) * 64];
        S[i][4 * r] = f(S[i][4 * r], x.x), S[i][4 * r + 1] = f(S[i][4 * r + 1], x.y);
        S[i][4 * r + 2] = f(S[i][4 * r + 2], x.z), S[i][4 * r + 3] = f(S[i][4 * r + 3], x.w);
      }
  };
  const auto to_slot = [&](int64_t j) {
    float4* p = slot + j * slot4 + wave * KT * 4 * 64 + lane;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        p[(i * 4 + r) * 64] =
            make_float4(S[i][4 * r], S[i][4 * r + 1], S[i][4 * r + 2], S[i][4 * r + 3]);
  };
#pragma unroll
  for (int i = 0; i < KT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) S[i][r] = 0.0f;
  if (kOut && slot) {
    if (t_lo < n || g == 0) {
      // few segments: their ends are added up here, otherwise by linattn_scan_kernel
      const int first = nseg <= kScanInPlace ? min(g, 1) : g;
      from_slot(first, Decay());
      if (first < g) {
        const Decay f(lg * (float)seg_len);
        for (int j = first + 1; j <= g; ++j) from_slot(j, f);
      }
    }
  } else if (g == 0 && a.s_in) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (state_row(i, r) < dk && col < dv) S[i][r] = a.s_in[head_state + state_off(i, r)];
      }
  }
  const float lg2 = log2_decay(lg);
  if (!kOut && g == 0) {
    to_slot(0);
    // the state given decays over the tokens that are left out as well
    if (t_lo > 0) {
      const float f = decay_pow(lg2, t_lo);
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[i][r] *= f;
    }
  }

  // ---- decay factors
  const int qrow = lane & 31;
  float w_up[16];  // update: scale_u g^(kC - late - token), token 16 (r / 8) + 8 half + r % 8
  float d_in[16];  // scores: scale_p g^(query - key), the same keys
#pragma unroll
  for (int r = 0; r < 16; ++r)
    w_up[r] = a.scale_u * decay_pow(lg2, kC - a.late - (16 * (r >> 3) + 8 * half + (r & 7)));
  if constexpr (kOut) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int dist = qrow - (16 * (r >> 3) + 8 * half + (r & 7));
      d_in[r] = dist >= 0 ? a.scale_p * decay_pow(lg2, dist) : 0.0f;
    }
  }
  float f_out = a.scale_o * decay_pow(lg2, qrow + a.late);  // query row's factor on Q S
  // g^kC is applied once per chunk, so the error of a rounded factor would grow
  // with the chunks that the state remembers: the two floats around g^kC take
  // turns so that their product stays within one rounding of the power.  In front of
  // the last chunk of a sequence, or of a segment whose end is wanted, what is left of
  // that rounding and of the last factor's goes into the product with that factor (a
  // correction for itself would be rounded off): over a session's calls it would add
  // up in the same way.  8192 tokens, 5 or 8 a call, memories of 10^4 to 5 10^5: the
  // state 2.2e-6 off at most, 4.8e-5 without; calls of 5 tokens 38.8 -> 39.6 us (64
  // sessions), long ones within 1%.
  const double step64 = exp((double)lg * kC);
  const float step_lo = uniform(__double2float_rd(step64)), step_hi = uniform(__double2float_ru(step64));
  const float err_lo = uniform(step_lo > 0.0f ? (float)(step_lo / step64 - 1.0) : 0.0f);
  const float err_hi = uniform(step_lo > 0.0f ? (float)(step_hi / step64 - 1.0) : 0.0f);
  float err = 0.0f;

  // A chunk's outputs pass through LDS, where the waves' columns become whole
  // rows: stored from the registers, 16 neighbouring lanes would write 16 bytes
  // of 16 rows.  They are stored at the next chunk's start, together with the
  // loads of the chunk after it, so that both have a chunk's time before the
  // wait that ends it.
  using TO = std::conditional_t<kF32Out, float, T>;
  constexpr int kRowPieces = DV * (int)sizeof(TO) / 16, kSwz = kRowPieces < 16 ? 7 : 15;
  constexpr int kOutB = kOut ? kC * DV * sizeof(TO) : 16;
  __shared__ __attribute__((aligned(16))) char out_smem[(kPair ? 4 : 2) * kOutB];
  lds_char* const out_tiles = (lds_char*)out_smem + pass * 2 * kOutB;
  const auto out_at = [&](int row, int piece) {
    return (uint32_t)(row * kRowPieces + (piece ^ (row & kSwz))) * 16;
  };
  constexpr int kPutRows = kThreads / kRowPieces;  // rows of a store instruction
  const int put_row = tid / kRowPieces, put_piece = tid % kRowPieces;
  const bool put_col = put_piece * (16 / (int)sizeof(TO)) < dv;
  const int64_t ost = pass ? a.ost2 : a.ost;
  const int64_t out_head = pass ? b * a.osb2 + h * a.osh2 : b * a.osb + h * a.osh;
  TO* const out_base = static_cast<TO*>(pass ? a.out2 : a.out) + out_head;
  const int64_t put_step = a.reverse ? -ost : ost;  // values to the next token of the walk
  TO* op = out_base + row0 * ost + put_row * put_step + put_piece * (16 / (int)sizeof(TO));
  const auto put = [&](int skip, const lds_char* tile) {  // and on to the next chunk
#pragma unroll
    for (int i = 0; i < kC / kPutRows; ++i) {
      const int row = put_row + i * kPutRows;
      const u32x4_t x = lds_load<u32x4_t>(tile + out_at(row, put_piece));
      if (put_col && row >= skip)
        *reinterpret_cast<u32x4_t*>(op + (i * kPutRows - skip) * put_step) = x;
    }
    op += kC * put_step;
  };
  wait_vmcnt<0>();
  lds_barrier();
  const auto chunk = [&](int t, float step, const lds_char* tiles, lds_char* other, lds_char* out,
                         const lds_char* out_before) {
    const lds_char* sK = tiles + (pass ? kOffV : 0);
    const lds_char* sV = tiles + (pass ? 0 : kOffV);
    const lds_char* sQ = tiles + (pass ? kOffW : kOffQ);
    const int m = min(kC, t_hi - t), skip = kC - m;
    if constexpr (kOut) {
      if (t > t_lo) put(0, out_before);
    }
    if (t + kC < t_hi) issue(t + kC, other);
    const auto decay = [&](int i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) S[i][r] *= step;
    };
    Frag<T> vf[2];  // V^T: value column col, tokens
    Frag<T>::cols2(vf, sV, 32 * wave, lane);
    Frag<T> wv[2][kTerms];  // the same weighted
    const auto weigh = [&](int pair) { weighted(wv[pair >> 2], vf[pair >> 2], w_up + 8 * (pair >> 2), pair & 3); };
    floatx16_t P, O;
    // A masked score is 0, but 0 times an infinity or NaN is NaN: such a value of
    // V would reach the tokens in front of its own.  The products leave it out;
    // what it does reach is made NaN behind them.
    bool odd = false;
    if constexpr (kOut) {
      odd = __builtin_amdgcn_ballot_w64(Frag<T>::not_finite(vf) != 0.0f) != 0;
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int s = 0; s < 2; ++s) vf[s].finite();
      }
    }
    if constexpr (kOut) {
      // O = S^T Q^T and P^T = K Q^T.  A matrix instruction takes as long as eight
      // vector instructions: the weighting of V, the state's conversion and its
      // decay run beside the products.  Fragments are read from LDS ahead of
      // their use, and products that follow each other go to different
      // accumulators; the scheduling barriers keep this order.
      constexpr int kSteps = DK / 16, kAhead = 1;
      Frag<T> qf[2], kf[2], sf[2];
      const auto read = [&](int s) {
        qf[s & 1] = Frag<T>::rows(sQ, qrow, s, lane);
        kf[s & 1] = Frag<T>::rows(sK, perm16(qrow), s, lane);
      };
#pragma unroll
      for (int s = 0; s < kAhead; ++s) read(s);
#pragma unroll
      for (int r = 0; r < 16; ++r) P[r] = O[r] = 0.0f;
      sf[0] = Frag<T>::result(S[0], 0);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        __builtin_amdgcn_sched_barrier(0);
        if (s + kAhead < kSteps) read(s + kAhead);
        mma(P, kf[s & 1], qf[s & 1]);
        mma(O, sf[s & 1], qf[s & 1]);
        if (s + 1 < kSteps) sf[(s + 1) & 1] = Frag<T>::result(S[(s + 1) >> 1], (s + 1) & 1);
#pragma unroll
        for (int p = 8 * s / kSteps; p < 8 * (s + 1) / kSteps; ++p) weigh(p);
        if (s & 1) decay(s >> 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int p = 0; p < 8; ++p) weigh(p);
#pragma unroll
      for (int i = 0; i < KT; ++i) decay(i);
    }

    // ---- S <- g^m S + K^T (w V), and O <- f O + V^T P^T
    Frag<T> kc[KT];  // K^T: key rows of tile i, 16 tokens
    const auto update = [&](int s) {
#pragma unroll
      for (int j = 0; j < kTerms; ++j)
#pragma unroll
        for (int i = 0; i < KT; ++i) mma(S[i], kc[i], wv[s][j]);
    };
    Frag<T>::template cols_all<0>(kc, sK, lane);
    update(0);
    Frag<T>::template cols_all<1>(kc, sK, lane);
    if constexpr (kOut) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        O[r] *= f_out;
        float p = qrow >= 16 * (r >> 3) + 8 * half + (r & 7) ? P[r] * d_in[r] : 0.0f;
        asm("" : "+v"(p));  // selected, then converted in pairs
        P[r] = p;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) mma(O, vf[s], Frag<T>::result(P, s));
    }
    update(1);

    if constexpr (kOut) {
      // registers 8 i .. of the result: the lane's token, columns 32 wave + 16 i + 8 half ..
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int piece = (32 * wave + 16 * i + 8 * half) * (int)sizeof(TO) / 16;
        if constexpr (sizeof(TO) == 2) {
          lds_store<u32x4_t>(out + out_at(qrow, piece),
                             u32x4_t{cvt_bf16x2(O[8 * i], O[8 * i + 1]),
                                     cvt_bf16x2(O[8 * i + 2], O[8 * i + 3]),
                                     cvt_bf16x2(O[8 * i + 4], O[8 * i + 5]),
                                     cvt_bf16x2(O[8 * i + 6], O[8 * i + 7])});
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            lds_store<floatx4_t>(out + out_at(qrow, piece + q),
                                 floatx4_t{O[8 * i + 4 * q], O[8 * i + 4 * q + 1],
                                           O[8 * i + 4 * q + 2], O[8 * i + 4 * q + 3]});
        }
      }
    }
    if (__builtin_expect(odd, 0)) {
      // recomputed here, not kept in registers through every chunk
      uint32_t none = 0;
      asm volatile("" : "+s"(none) : : "memory");  // and behind the stores above
      const int l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, none));
      const int hi = l >> 5, row = l & 31;
      Frag<T> raw[2];
      Frag<T>::cols2(raw, sV, 32 * wave, l);
      int from = kC;  // the first token of the lane's value column that is not finite
#pragma unroll
      for (int r = 15; r >= 0; --r)
        if (!raw[r >> 3].is_finite(r & 7)) from = 16 * (r >> 3) + 8 * hi + (r & 7);
      from = min(from, __builtin_amdgcn_ds_bpermute((l ^ 32) * 4, from));
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[i][r] = from < kC ? __builtin_nanf("") : S[i][r];
#pragma unroll 1
      for (int c = 0; c < 32; ++c) {  // value column c, the lane's token
        const int at = (32 * wave + c) * (int)sizeof(TO);
        const int first_of_c = __builtin_amdgcn_readlane(from, perm16(c));
        if (row >= first_of_c && hi == 0)
          lds_store<TO>(out + out_at(row, at >> 4) + (at & 15), nan_of<TO>());
      }
    }
    wait_vmcnt<0>();  // the next chunk's tiles are here, the last one's outputs gone
    lds_barrier();
  };
  // (from a segment's end a state goes on to the next call only if one came in)
  const int last_of = kOut ? n : g == 0 && a.s_in ? t_hi : INT32_MAX;
  int buf = 0;
  for (int t = t_lo; t < t_hi; t += kC, buf ^= 1) {
    float step = err < 0.0f ? step_hi : step_lo;
    err += err < 0.0f ? err_hi : err_lo;
    if (t + kC >= last_of) {  // the last chunk
      const int m = t_hi - t;
      if (m < kC) {
        const Decay d(lg * (float)m);
        err += d.f > 0.0f ? -d.rest / d.f : 0.0f;
        err -= step == step_lo ? err_lo : err_hi;
        step = d.f;
        f_out = a.scale_o * decay_pow(lg2, max(0, qrow - (kC - m)) + a.late);
      }
      if (step > 0.5f && err != 0.0f) {
        const float rest = -step * err;
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) S[i][r] = fmaf(step, S[i][r], rest * S[i][r]);
        f_out /= step;
        step = 1.0f;
      }
    }
    chunk(t, step, (const lds_char*)smem + buf * kBuf, (lds_char*)smem + (buf ^ 1) * kBuf,
          out_tiles + buf * kOutB, out_tiles + (buf ^ 1) * kOutB);
  }
  if constexpr (kOut) {
    if (t_lo < t_hi)
      put((kC - (t_hi - t_lo) % kC) % kC, out_tiles + (buf ^ 1) * kOutB);
  }

  if constexpr (!kOut) {
    to_slot(g + 1);
  } else {
    const bool last = t_hi == n && (t_lo < n || g == 0);  // this segment holds the last token
    if (last && a.s_out && pass == 0) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (state_row(i, r) < dk && col < dv)
            a.s_out[head_state + state_off(i, r)] = S[i][r];
        }
    }
    // rows behind the sequence's end
    const int z_lo = max(t_lo, n), z_hi = min(t_lo + seg_len, (int)a.T);
    const int pieces = dv >> 3;
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t p = tid; p < (int64_t)(z_hi - z_lo) * pieces; p += kThreads)
      store8(out_base + (z_lo + p / pieces) * ost + (p % pieces) * 8, zero);
  }
}

// Two waves a SIMD need half the register file each; fp32 tiles leave LDS for one,
// and so do the bf16 tiles of 128 keys and 64 values with fp32 outputs (56 KB, two
// workgroups of two waves a CU), whose registers the compiler then does not limit.
template <typename T>
constexpr int kMinWaves = sizeof(T) == 2 ? 2 : 1;

template <typename T, int DK, int NW, int kTerms, bool kF32Out = false, bool kPair = false>
__global__ __launch_bounds__(64 * NW * (kPair ? 2 : 1), kMinWaves<T>) void linattn_main_kernel(
    LinArgs a, float4* seg, int seg_len, int nseg) {
  chunked_pass<T, DK, NW, true, kTerms, kF32Out, kPair>(a, seg, seg_len, nseg);
}

// The ends of one or two passes' segments (gridDim.y), one region of slots each.
struct LinTwo {
  LinArgs a[2];
};
template <typename T, int DK, int NW, int kTerms>
__global__ __launch_bounds__(64 * NW, kMinWaves<T>) void linattn_ends_kernel(LinTwo two,
                                                                             float4* seg,
                                                                             int seg_len,
                                                                             int nseg) {
  const LinArgs& a = two.a[blockIdx.y];
  const int64_t region = a.B * a.H * nseg * (DK * NW * 32 / 4);
  chunked_pass<T, DK, NW, false, kTerms, false, false>(a, seg + blockIdx.y * region, seg_len,
                                                       nseg);
}

// seg[head][g] <- seg[head][g] + g^seg_len seg[head][g - 1] along the segments, so
// that every slot is the state its segment starts from.  Slots of segments
// behind a sequence's end are not used.  The factor as one float leaves 1.0e-5 in
// the state of 131072 tokens in 512 segments that remembers a million; as Decay
// 4.9e-7, in the same time (12 us of the 128K prompt).
__global__ __launch_bounds__(64) void linattn_scan_kernel(float4* seg,
                                                           const float* __restrict__ log_decay,
                                                           int64_t H, int64_t slot4, int64_t total,
                                                           int seg_len, int nseg) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= total) return;
  const int64_t head = i / slot4, e = i % slot4;
  float4* p = seg + head * nseg * slot4 + e;
  float4 acc = p[slot4];
  const Decay step(log_decay[head % H] * (float)seg_len);
  constexpr int kBatch = 8;  // loads in flight
  for (int g = 2; g < nseg; g += kBatch) {
    float4 x[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (g + j < nseg) x[j] = p[(g + j) * slot4];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (g + j < nseg) {
        acc.x = step(acc.x, x[j].x), acc.y = step(acc.y, x[j].y);
        acc.z = step(acc.z, x[j].z), acc.w = step(acc.w, x[j].w);
        p[(g + j) * slot4] = acc;
      }
  }
}

// ------------------------------------------------------------ recurrent form
// Bound by reading and writing the state once.  A workgroup takes 32 value
// columns of one head: 8 threads of 4 columns by 32 groups of 4 key rows, all
// four 16-byte loads of a thread issued together.  The tokens' q, k and v go to
// LDS as fp32 while the state is on its way (read from memory token by token
// they cost 1.4 us a token); the tokens then run in registers, and the sums over
// the key rows end in LDS after the last token.  The decay is applied with what its
// rounding leaves (4000 tokens, memory of 500000: the state 2.5e-6 off, 9.5e-5
// without; 64 sessions of 4 tokens 38.9 us, 38.1 without).  From 5 tokens on the chunked
// form is faster (us for 1, 8 and 64 sessions of 20, 16 and 20 heads: 4 tokens
// 6.4, 6.2, 39 here and 10.1, 7.4, 39 chunked; 8 tokens 9.3, 9.2, 50 and 10.1,
// 7.4, 39).
constexpr int kStepCols = 32;

__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinArgs a) {
  __shared__ __attribute__((aligned(16))) float q_s[kLinStepTokens][kLinMaxHead];
  __shared__ __attribute__((aligned(16))) float k_s[kLinStepTokens][kLinMaxHead];
  __shared__ __attribute__((aligned(16))) float v_s[kLinStepTokens][kStepCols];
  __shared__ float part[kLinStepTokens][4][kStepCols];
  const int slices = (int)((a.dv + kStepCols - 1) / kStepCols);
  const int64_t bh = blockIdx.x / slices, b = bh / a.H, h = bh % a.H;
  const int cg = threadIdx.x & 7, row0 = (threadIdx.x >> 3) * 4;
  const int c0 = (int)(blockIdx.x % slices) * kStepCols, col = c0 + 4 * cg;
  const int dk = (int)a.dk, dv = (int)a.dv;
  const bool live = col < dv && row0 < dk;  // whole groups: d_key and d_value are multiples of 8
  const int n = live_tokens(a.lengths, b, a.T);
  const int64_t base = bh * dk * dv + (int64_t)row0 * dv + col;
  float4 S[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    S[i] = make_float4(0, 0, 0, 0);
    if (a.s_in && live) S[i] = *reinterpret_cast<const float4*>(a.s_in + base + i * dv);
  }
  const T* qp = head_base<T>(a.q, b, h);
  const T* kp = head_base<T>(a.k, b, h);
  const T* vp = head_base<T>(a.v, b, h);
  const Decay decay(a.log_decay[h]);
  for (int p = threadIdx.x; p < n * kLinMaxHead; p += 256) {
    const int t = p / kLinMaxHead, r = p % kLinMaxHead;
    q_s[t][r] = r < dk ? to_f32(qp[t * a.q.st + r]) : 0.0f;
    k_s[t][r] = r < dk ? to_f32(kp[t * a.k.st + r]) : 0.0f;
    if (r < kStepCols) v_s[t][r] = c0 + r < dv ? to_f32(vp[t * a.v.st + c0 + r]) : 0.0f;
  }
  __syncthreads();
  for (int t = 0; t < n; ++t) {
    const float4 q = *reinterpret_cast<const float4*>(&q_s[t][row0]);
    const float4 k = *reinterpret_cast<const float4*>(&k_s[t][row0]);
    const float4 v = *reinterpret_cast<const float4*>(&v_s[t][4 * cg]);
    float o[4] = {0, 0, 0, 0};
    const auto row = [&](float4& x, float ki, float qi) {
      x.x = decay(x.x, ki * v.x), x.y = decay(x.y, ki * v.y);
      x.z = decay(x.z, ki * v.z), x.w = decay(x.w, ki * v.w);
      o[0] = fmaf(qi, x.x, o[0]), o[1] = fmaf(qi, x.y, o[1]);
      o[2] = fmaf(qi, x.z, o[2]), o[3] = fmaf(qi, x.w, o[3]);
    };
    row(S[0], k.x, q.x), row(S[1], k.y, q.y), row(S[2], k.z, q.z), row(S[3], k.w, q.w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int m = 8; m <= 32; m <<= 1) o[j] += __shfl_xor(o[j], m, 64);
      if ((threadIdx.x & 63) < 8) part[t][threadIdx.x >> 6][4 * cg + j] = o[j];
    }
  }
  if (a.s_out && live) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(a.s_out + base + i * dv) = S[i];
  }
  __syncthreads();
  for (int p = threadIdx.x; p < a.T * kStepCols; p += 256) {
    const int t = p / kStepCols, c = p % kStepCols;
    if (c0 + c >= dv) continue;
    float o = 0.0f;
    if (t < n) o = a.scale_o * (((part[t][0][c] + part[t][1][c]) + part[t][2][c]) + part[t][3][c]);
    Elem<T>::store(static_cast<T*>(a.out) + b * a.osb + t * a.ost + h * a.osh + c0 + c, o);
  }
}

// out[b][t][g][:] = sum over r < rep of part[b][g rep + r][t][:], a tensor for
// each blockIdx.y.
struct HeadSums {
  const float* part[2];
  void* out[2];
  int64_t d[2];
};
template <typename T>
__global__ __launch_bounds__(256) void linattn_sum_heads_kernel(HeadSums h, int64_t B, int64_t T_,
                                                                int64_t G, int64_t rep) {
  const int y = blockIdx.y;
  const int64_t d = h.d[y], pieces = d >> 3;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= B * G * T_ * pieces) return;
  const int64_t c = (i % pieces) * 8, t = i / pieces % T_, g = i / (pieces * T_) % G,
                b = i / (pieces * T_ * G);
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t r = 0; r < rep; ++r) {
    const float* p = h.part[y] + (((b * G + g) * rep + r) * T_ + t) * d + c;
    const float4 x = *reinterpret_cast<const float4*>(p), z = *reinterpret_cast<const float4*>(p + 4);
    f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w;
    f[4] += z.x, f[5] += z.y, f[6] += z.z, f[7] += z.w;
  }
  store8(static_cast<T*>(h.out[y]) + ((b * T_ + t) * G + g) * d + c, f);
}

int64_t padded(int64_t d) { return d <= 64 ? 64 : 128; }

// How a pass splits sequences into segments of whole chunks: into as many as
// have their workgroups resident together (256 CUs, two waves a SIMD in bf16 and
// one in fp32, whose tiles leave LDS for no more), of two chunks at least.  More
// of them cost more in states than they gain: gradients of 32768 tokens, 20
// heads of 128, bf16: 629 us with 2048 waves, 716 us with 4096; 4096 tokens, 16
// heads of 64, fp32: 110 us with 1024, 154 us with 2048, and 50 and 60 us without
// gradients (32768 tokens, 20 heads of 128 the other way round: 2.50 and 2.41 ms,
// 944 and 874 us).  At least 128 tokens a segment
// are slower for small calls (1024 tokens, 4 heads, fp32: 37 us, 29 us).
constexpr int64_t kResidentWavesBf16 = 2048, kResidentWavesF32 = 1024, kMinSegment = 64;
struct Split {
  int seg_len, nseg;
};

Split split(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv, Dtype dt) {
  const int64_t heads = B * H, waves = std::max(padded(dk), padded(dv)) / 32;
  const int64_t resident = dt == Dtype::BF16 ? kResidentWavesBf16 : kResidentWavesF32;
  const int64_t nseg = std::max<int64_t>(1, std::min(resident / waves / heads, T / kMinSegment));
  // whole chunks per segment may need fewer segments
  Split p;
  p.seg_len = (int)(((T + nseg - 1) / nseg + kC - 1) / kC * kC);
  p.nseg = (int)((T + p.seg_len - 1) / p.seg_len);
  return p;
}

// The states that the segments of `count` passes start from.
template <typename T, int DK, int NW, int kTerms>
hipError_t starts(const LinArgs* a, int count, float4* seg, const Split& p, hipStream_t s) {
  if (p.nseg == 1) return hipSuccess;
  const int64_t heads = a->B * a->H;
  LinTwo two{{a[0], a[count - 1]}};
  linattn_ends_kernel<T, DK, NW, kTerms>
      <<<dim3((unsigned)(heads * (p.nseg - 1)), count), 64 * NW, 0, s>>>(two, seg, p.seg_len,
                                                                        p.nseg);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nseg <= kScanInPlace) return e;
  const int64_t slot4 = DK * 32 * NW / 4, total = count * heads * slot4;
  linattn_scan_kernel<<<dim3((unsigned)((total + 63) / 64)), 64, 0, s>>>(
      seg, a->log_decay, a->H, slot4, total, p.seg_len, p.nseg);
  return hipGetLastError();
}

template <typename T, int DK, int NW, int kTerms>
hipError_t main_pass(const LinArgs& a, float4* seg, const Split& p, hipStream_t s) {
  if (!a.seg_ready && !a.seg_trans) {
    const hipError_t e = starts<T, DK, NW, kTerms>(&a, 1, seg, p, s);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)(a.B * a.H * p.nseg));
  float4* start = p.nseg > 1 ? seg : nullptr;
  // fp32 outputs of bf16 passes are gradients on their way to a sum over heads,
  // which come from a pair where the tiles are of one size
  constexpr bool kBf16 = sizeof(T) == 2, kSquare = DK == 32 * NW;
  if (a.pair) {
    if constexpr (kBf16 && kSquare && kTerms == 3) {
      if (a.out_f32)
        linattn_main_kernel<T, DK, NW, kTerms, true, true>
            <<<grid, 128 * NW, 0, s>>>(a, start, p.seg_len, p.nseg);
      else
        linattn_main_kernel<T, DK, NW, kTerms, false, true>
            <<<grid, 128 * NW, 0, s>>>(a, start, p.seg_len, p.nseg);
      return hipGetLastError();
    }
    return hipErrorInvalidValue;
  }
  if (kBf16 && a.out_f32) {
    if constexpr (kBf16 && !kSquare) {
      linattn_main_kernel<T, DK, NW, kTerms, true>
          <<<grid, 64 * NW, 0, s>>>(a, start, p.seg_len, p.nseg);
      return hipGetLastError();
    }
    return hipErrorInvalidValue;
  }
  linattn_main_kernel<T, DK, NW, kTerms><<<grid, 64 * NW, 0, s>>>(a, start, p.seg_len, p.nseg);
  return hipGetLastError();
}

// Calls f with the pass's type, tile sizes and terms as constants.
template <typename F>
hipError_t with_tiles(const LinArgs& a, F&& f) {
  const auto tiles = [&](auto t, auto terms) {
    using std::integral_constant;
    if (a.dk <= 64)
      return a.dv <= 64 ? f(t, integral_constant<int, 64>{}, integral_constant<int, 2>{}, terms)
                        : f(t, integral_constant<int, 64>{}, integral_constant<int, 4>{}, terms);
    return a.dv <= 64 ? f(t, integral_constant<int, 128>{}, integral_constant<int, 2>{}, terms)
                      : f(t, integral_constant<int, 128>{}, integral_constant<int, 4>{}, terms);
  };
  if (a.dt == Dtype::F32) return tiles(float{}, std::integral_constant<int, 1>{});
  return a.exact_state ? tiles(uint16_t{}, std::integral_constant<int, 3>{})
                       : tiles(uint16_t{}, std::integral_constant<int, 2>{});
}

}  // namespace

bool linattn_square(int64_t dk, int64_t dv) { return padded(dk) == padded(dv); }

size_t linattn_segment_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv, Dtype dt) {
  const Split p = split(B, H, T, dk, dv, dt);
  if (p.nseg == 1) return 0;
  return (size_t)(B * H * p.nseg) * padded(dk) * padded(dv) * sizeof(float);
}

hipError_t launch_linattn_starts(const LinArgs* a, int count, float* seg, hipStream_t s) {
  return with_tiles(*a, [&](auto t, auto dk, auto nw, auto terms) {
    return starts<decltype(t), decltype(dk)::value, decltype(nw)::value, decltype(terms)::value>(
        a, count, reinterpret_cast<float4*>(seg), split(a->B, a->H, a->T, a->dk, a->dv, a->dt), s);
  });
}

hipError_t launch_linattn_chunked(const LinArgs& a, float* seg, hipStream_t s) {
  return with_tiles(a, [&](auto t, auto dk, auto nw, auto terms) {
    return main_pass<decltype(t), decltype(dk)::value, decltype(nw)::value,
                     decltype(terms)::value>(a, reinterpret_cast<float4*>(seg),
                                             split(a.B, a.H, a.T, a.dk, a.dv, a.dt), s);
  });
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

hipError_t launch_linattn_sum_heads(const float* part_k, void* dk, int64_t d_key,
                                    const float* part_v, void* dv, int64_t d_value, int64_t B,
                                    int64_t T, int64_t G, int64_t rep, Dtype dt, hipStream_t s) {
  const HeadSums h{{part_k, part_v}, {dk, dv}, {d_key, d_value}};
  const int64_t n = B * G * T * (std::max(d_key, d_value) / 8);
  const dim3 grid((unsigned)((n + 255) / 256), 2);
  if (dt == Dtype::BF16)
    linattn_sum_heads_kernel<uint16_t><<<grid, 256, 0, s>>>(h, B, T, G, rep);
  else
    linattn_sum_heads_kernel<float><<<grid, 256, 0, s>>>(h, B, T, G, rep);
  return hipGetLastError();
}

}  // namespace ttt
