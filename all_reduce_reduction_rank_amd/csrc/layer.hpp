// layer.hpp -- argument checks shared by the layer operators' C entry points.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "schedule.hpp"

namespace ar {

// Limits.  Widths (hidden, inner, piece): 256 rows of a tile stay within the
// 2^30 bytes a buffer descriptor covers.  Rows: 32-bit counts with room for
// a tile.
constexpr uint64_t LAYER_MAX_WIDTH = 1ull << 20;
constexpr uint64_t LAYER_MAX_ROWS = 1ull << 30;

inline uint64_t layer_align(uint64_t x) { return (x + 255) & ~255ull; }

// The device buffers of one call: every one of nonzero size must be non-null
// and aligned (matrices to 16 bytes, vectors to an element), and no output may overlap any other buffer.
class LayerBuffers {
 public:
  void in(const void* p, uint64_t bytes, uint32_t align = 16) { add(p, bytes, align, false); }
  void out(const void* p, uint64_t bytes, uint32_t align = 16) { add(p, bytes, align, true); }
  bool ok() {
    if (bad_) return false;
    std::sort(s_, s_ + n_, [](const Span& a, const Span& b) { return a.at < b.at; });
    // Sorted by address, a span overlaps an earlier one exactly if it starts
    // before the furthest end so far; an output overlaps anything, an input
    // only an output.
    uintptr_t end = 0, out_end = 0;
    for (int i = 0; i < n_; ++i) {
      if (s_[i].at < (s_[i].out ? end : out_end)) return false;
      end = std::max(end, s_[i].at + s_[i].bytes);
      if (s_[i].out) out_end = std::max(out_end, s_[i].at + s_[i].bytes);
    }
    return true;
  }

 private:
  struct Span {
    uintptr_t at;
    uint64_t bytes;
    bool out;
  };
  void add(const void* p, uint64_t bytes, uint32_t align, bool out) {
    if (!bytes) return;
    if (!p || (uintptr_t)p % align || n_ == MAX_SPANS) bad_ = true;
    else s_[n_++] = {(uintptr_t)p, bytes, out};
  }
  static constexpr int MAX_SPANS = 12 * MAX_RANKS + 8;
  Span s_[MAX_SPANS];
  int n_ = 0;
  bool bad_ = false;
};

}  // namespace ar
