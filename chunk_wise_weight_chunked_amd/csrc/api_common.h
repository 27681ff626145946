// api_common.h -- helpers shared by the C ABI's source files: the calling
// thread's error message, descriptor validation and buffer range checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ttt_mlp.h"
#include "layer.h"

namespace ttt {
namespace api {

// Records the message for ttt_last_error() and returns `code`.
ttt_status_t fail(ttt_status_t code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message and returns TTT_OK.
ttt_status_t ok();
// TTT_ERR_HIP with the HIP error's text.
ttt_status_t hip_fail(hipError_t e, const char* what);

// Validates a descriptor and derives the call's shapes.
ttt_status_t make_dims(const ttt_mlp_desc_t* desc, Dims* dm);

// A named byte range [lo, hi) of a buffer, for overlap checks.
struct Range {
  const char* name;
  uintptr_t lo, hi;
};
Range range(const char* name, const void* p, size_t bytes);
bool overlaps(const Range& x, const Range& y);
bool aligned(const void* p, size_t a);

inline bool valid_dtype(ttt_dtype_t t) { return t == TTT_F32 || t == TTT_BF16; }
inline Dtype to_dtype(ttt_dtype_t t) { return t == TTT_BF16 ? Dtype::BF16 : Dtype::F32; }
inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Buffers of one call: every one that is given must be 16-byte aligned, and no
// output may overlap another buffer, except one it may be the same as.
struct BufferList {
  struct Item {
    Range r;
    const void* p;
    bool out;
    const void* may_be;  // an input this output may share its address with
  };
  Item items[16];  // more than any call has
  int count = 0;
  void in(const char* name, const void* p, size_t bytes) {
    if (p) items[count++] = {range(name, p, bytes), p, false, nullptr};
  }
  void out(const char* name, const void* p, size_t bytes, const void* may_be = nullptr) {
    if (p) items[count++] = {range(name, p, bytes), p, true, may_be};
  }
  ttt_status_t check() const {
    for (int i = 0; i < count; ++i)
      if (!aligned(items[i].p, 16))
        return fail(TTT_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", items[i].r.name);
    for (int i = 0; i < count; ++i)
      for (int j = 0; j < count; ++j) {
        const Item &a = items[i], &b = items[j];
        if (i == j || !a.out || (b.out && j < i) || !overlaps(a.r, b.r)) continue;
        if (a.may_be && a.may_be == b.p && a.p == b.p && !b.out) continue;
        return fail(TTT_ERR_INVALID_ARGUMENT, "%s overlaps %s", a.r.name, b.r.name);
      }
    return TTT_OK;
  }
  // A small input that needs no 16-byte alignment.
  ttt_status_t check_against(const Range& in) const {
    for (int i = 0; i < count; ++i)
      if (items[i].out && in.hi > in.lo && overlaps(in, items[i].r))
        return fail(TTT_ERR_INVALID_ARGUMENT, "%s overlaps %s", items[i].r.name, in.name);
    return TTT_OK;
  }
};

inline ttt_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return TTT_OK;
  if (!ws) return fail(TTT_ERR_INVALID_ARGUMENT, "ws is NULL (%zu bytes are needed)", need);
  if (!aligned(ws, 256)) return fail(TTT_ERR_INVALID_ARGUMENT, "ws must be 256-byte aligned");
  if (have < need)
    return fail(TTT_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes is too small, %zu are needed",
                have, need);
  return TTT_OK;
}

}  // namespace api
}  // namespace ttt
