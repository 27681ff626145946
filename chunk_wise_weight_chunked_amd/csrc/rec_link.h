// rec_link.h -- the arithmetic of the gated recurrence's decays, and the words that link its
// tiles (gatedrec.hip).  Everything here runs on the host too, where the tests call it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttt {

#define TTT_BOTH __host__ __device__ __forceinline__

// Exponents are base 2 throughout: z is log2 a = -rate log2(e) r.
constexpr float kLog2e = 0x1.715476p+0f;

TTT_BOTH float power_of_2(float z) {
#ifdef __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_exp2f(z);
#else
  return exp2f(z);
#endif
}
TTT_BOTH uint32_t bits_of(float x) { return __builtin_bit_cast(uint32_t, x); }
TTT_BOTH float float_of(uint32_t bits) { return __builtin_bit_cast(float, bits); }

// A decay over a run of tokens as one float: 2^z itself (sign bit clear) or, where
// z > -1/2, 2^z - 1 (sign bit set, -0 for z = 0).  The second keeps what a decay near 1
// loses by its rounding, which would be repeated for as long as the channel remembers.
// The polynomial is 2^z - 1 to 3.3e-8 of it (Chebyshev nodes in [-1/2, 0]).
TTT_BOTH float decay_of(float z) {
  float p = __builtin_fmaf(z, 0x1.2ee444p-10f, 0x1.38ae68p-7f);
  p = __builtin_fmaf(z, p, 0x1.c6947ap-5f);
  p = __builtin_fmaf(z, p, 0x1.ebfb70p-3f);
  p = __builtin_fmaf(z, p, 0x1.62e430p-1f);
  const float near = z * p, far = power_of_2(z);
  return z > -0.5f ? near : far;  // a z of -0 gives -0
}
TTT_BOTH bool near_one(float dec) { return bits_of(dec) >> 31; }
// The decay over two runs.
TTT_BOTH float decay_both(float d1, float d2) {
  const bool n1 = near_one(d1), n2 = near_one(d2);
  // a1 a2 - 1, never positive, and a1 a2 where that is far from 0
  const float near = -fabsf(__builtin_fmaf(d1, d2, d1 + d2));
  const float both = near < -0.5f ? 1.0f + near : near;
  const float far = __builtin_fmaf(d1, d2, n1 ? d2 : n2 ? d1 : 0.0f);
  return n1 && n2 ? both : far;
}
// a h + u
TTT_BOTH float decayed(float dec, float h, float u) {
  return __builtin_fmaf(dec, h, u) + (near_one(dec) ? h : 0.0f);
}

// -log2(e) rate; z is never positive: a rate below 0 counts as NaN, and one of 0 of either sign
// gives -0, a z that decay_of keeps the sign of.  2^100 is as good as any above it, and 0 times
// it is 0.
TTT_BOTH float log_rate(float r) {
  return r >= 0.0f ? -kLog2e * fminf(fabsf(r), 0x1p100f) : __builtin_nanf("");
}

// ------------------------------------------------- what links tiles
// A tile leaves a word for the tiles behind it (backward: in front of it), one for each
// channel: its map, the decay over the tile and the state behind it from 0.  kGroup tiles
// make a group, whose word is the group's map or, once it is known, the state behind it,
// marked by +inf, which no decay is.  So the state in front of a tile comes through the
// groups in front of its own, from the nearest that has its state, and through its own group's
// maps: always by the same products, whatever was there first, and over 48 tiles in the
// time that a word takes from one workgroup to another (about 1 us: 131072 tokens of 64
// channels take 45 us, 133 where tiles take their states from the 8 in front of them;
// 32768 of 200 with gradients 89 and 118, of 2560 440 and 434).
// Both halves of a word come and go in one 64-bit access, so it needs no other ordering; it
// starts as kUnset, a NaN that no decay is stored as.
constexpr int kGroup = 8;
constexpr uint64_t kUnset = ~0ull;
constexpr uint32_t kState = 0x7f800000u;
TTT_BOTH uint64_t word_of(float dec, float h) {
  const uint32_t hi = dec != dec ? 0x7fc00000u : bits_of(dec);
  return (uint64_t)hi << 32 | bits_of(h);
}
TTT_BOTH uint64_t state_word(float h) { return (uint64_t)kState << 32 | bits_of(h); }

struct Links {
  uint64_t* maps;    // [B][tiles][d], null where there is one tile
  uint64_t* states;  // [B][groups][d]: group g's has the word of g - 1, the first one a state
  uint32_t* begun;
  int64_t tiles, groups;
};

// The workgroup's tile.
struct TileAt {
  int64_t b, j, strip, k;  // k: tiles that come before it in its sequence
};

// Waits end by themselves (tile_at in gatedrec.hip); only where another call clears the same
// words meanwhile, which no workspace allows, they end here, after some seconds and with NaN.
constexpr int kTries = 1 << 22;

// The words are read and written by Mem's get and put, with its pause between two looks.

// The map over a group's first n tiles (1 <= n < kGroup), from their words, `step` words apart.
template <class Mem>
TTT_BOTH void map_before(const uint64_t* word, int64_t step, int n, float* dec, float* h) {
  for (int tries = 0; tries < kTries; ++tries) {
    uint64_t w[kGroup - 1];
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
      if (i < n) w[i] = Mem::get(word + i * step);
    bool all = true;
    *dec = -0.0f, *h = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i) {
      if (i >= n) break;
      const float d = float_of((uint32_t)(w[i] >> 32));
      all = all && w[i] != kUnset;
      *dec = decay_both(*dec, d);
      *h = decayed(d, *h, float_of((uint32_t)w[i]));
    }
    if (all) return;
    Mem::pause();
  }
  *dec = *h = __builtin_nanf("");
}

// The state in front of a group, from its word and those of the k groups in front of it at
// `word`, `word` - step, ...: from the nearest of kAhead that is a state, the maps behind
// that one applied in order.
template <class Mem>
TTT_BOTH float state_before(const uint64_t* word, int64_t step, int64_t k) {
  constexpr int kAhead = 6;
  for (int tries = 0; tries < kTries; ++tries) {
    uint64_t w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) w[i] = Mem::get(word - (i < k ? i : k) * step);
    bool found = false;
    float s = 0.0f;
#pragma unroll
    for (int i = kAhead - 1; i >= 0; --i) {
      const uint32_t hi = (uint32_t)(w[i] >> 32);
      const float f = float_of((uint32_t)w[i]);
      found = hi == kState || (found && w[i] != kUnset);
      s = hi == kState ? f : decayed(float_of(hi), s, f);
    }
    if (found) return s;
    Mem::pause();
  }
  return __builtin_nanf("");
}

// The state in front of a tile of a channel, from the tile's map: what the tiles behind it
// need is left to them, as soon as it is known.
template <class Mem, class First>
TTT_BOTH float link(const Links& links, const TileAt& at, int64_t d, int64_t c, float dec, float h,
                    First&& first) {
  const int64_t g = at.k / kGroup;
  const int in = (int)(at.k % kGroup);
  uint64_t* const map = links.maps + (at.b * links.tiles + at.k) * d + c;
  uint64_t* const state = links.states + (at.b * links.groups + g) * d + c;
  const bool last = in == kGroup - 1 && g + 1 < links.groups;
  if (in < kGroup - 1 && at.k + 1 < links.tiles) Mem::put(map, word_of(dec, h));
  float before = -0.0f, from0 = 0.0f;  // the map over the group's tiles in front
  if (in > 0) map_before<Mem>(map - in * d, d, in, &before, &from0);
  const float all = decay_both(before, dec), all0 = decayed(dec, from0, h);
  if (last) Mem::put(state + d, word_of(all, all0));
  float s;
  if (at.k == 0) {
    s = first(c);
    Mem::put(state, state_word(s));
  } else {
    s = state_before<Mem>(state, d, g);
  }
  if (last) Mem::put(state + d, state_word(decayed(all, s, all0)));
  return in > 0 ? decayed(before, s, from0) : s;
}

}  // namespace ttt
