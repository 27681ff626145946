// The gated recurrence's decays and the links of its tiles (rec_link.h), compiled for the host
// for test_rec_link.py: the functions that the kernels call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <chrono>
#include <thread>
#include <vector>

#include "../chunk_wise_weight_chunked_amd/csrc/rec_link.h"

namespace {

struct HostWords {
  static void put(uint64_t* p, uint64_t w) { __atomic_store_n(p, w, __ATOMIC_RELAXED); }
  static uint64_t get(const uint64_t* p) { return __atomic_load_n(p, __ATOMIC_RELAXED); }
  static void pause() { std::this_thread::yield(); }
};

}  // namespace

extern "C" {

float rec_log_rate(float r) { return ttt::log_rate(r); }
float rec_decay_of(float z) { return ttt::decay_of(z); }
float rec_decay_both(float d1, float d2) { return ttt::decay_both(d1, d2); }
float rec_decayed(float dec, float h, float u) { return ttt::decayed(dec, h, u); }
uint64_t rec_word_of(float dec, float h) { return ttt::word_of(dec, h); }
uint64_t rec_state_word(float h) { return ttt::state_word(h); }
uint64_t rec_unset() { return ttt::kUnset; }
int rec_group() { return ttt::kGroup; }

// The state in front of a group from words[k], its own, and those of the k groups in front of it
// behind each other.  What is there has to be enough.
float rec_state_before(const uint64_t* words, int64_t k) {
  return ttt::state_before<HostWords>(words + k, 1, k);
}

// before[b][k][c]: the state in front of tile k, from the tiles' maps dec, h [b][tiles][c] and the
// states first [b][c].  Tiles are taken in the order of a counter by `threads` workers; a
// worker naps after taking a tile where nap[tile] is set, so that others find words unset.  Returns
// whether the memory behind the words was left alone.
int rec_link_all(int64_t B, int64_t tiles, int64_t d, const float* dec, const float* h,
                  const float* first, const uint8_t* nap, int threads, float* before) {
  const int64_t groups = (tiles + ttt::kGroup - 1) / ttt::kGroup;
  const int64_t n = B * (tiles + groups) * d;
  std::vector<uint64_t> words(n + d, ttt::kUnset);
  const ttt::Links links{words.data(), words.data() + B * tiles * d, nullptr, tiles, groups};
  std::atomic<int64_t> ticket{0};
  const auto work = [&] {
    for (;;) {
      const int64_t t = ticket.fetch_add(1);
      if (t >= B * tiles) return;
      const ttt::TileAt at{t % B, t / B, 0, t / B};
      if (nap[t]) std::this_thread::sleep_for(std::chrono::microseconds(50 * nap[t]));
      for (int64_t c = 0; c < d; ++c) {
        const int64_t i = (at.b * tiles + at.k) * d + c;
        before[i] = ttt::link<HostWords>(links, at, d, c, dec[i], h[i],
                                         [&](int64_t c) { return first[at.b * d + c]; });
      }
    }
  };
  std::vector<std::thread> pool;
  for (int i = 1; i < threads; ++i) pool.emplace_back(work);
  work();
  for (auto& t : pool) t.join();
  for (int64_t i = n; i < n + d; ++i)
    if (words[i] != ttt::kUnset) return 0;
  return 1;
}

}  // extern "C"
