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
  // An output of `rows` rows of `width` bytes, `pitch` bytes apart: what lies
  // between its rows may be another such output's.
  void out_rows(const void* p, uint64_t rows, uint64_t pitch, uint64_t width) {
    if (!rows) return;
    add(p, (rows - 1) * pitch + width, 16, true);
    if (!bad_) s_[n_ - 1].pitch = pitch, s_[n_ - 1].width = width;
  }
  bool ok() {
    if (bad_) return false;
    std::sort(s_, s_ + n_, [](const Span& a, const Span& b) { return a.at < b.at; });
    // Sorted by address, a span overlaps an earlier one exactly if it starts
    // before the furthest end so far; an output overlaps anything, an input
    // only an output.
    uintptr_t end = 0, out_end = 0;
    for (int i = 0; i < n_; ++i) {
      if (s_[i].at < (s_[i].out ? end : out_end)) return apart();
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
    uint64_t pitch, width;  // rows (pitch 0: one piece)
  };
  // Pair by pair: two outputs in rows of one pitch whose columns are apart do
  // not overlap.
  bool apart() const {
    for (int i = 0; i < n_; ++i)
      for (int j = i + 1; j < n_ && s_[j].at < s_[i].at + s_[i].bytes; ++j) {
        if (!s_[i].out && !s_[j].out) continue;
        if (!s_[i].pitch || s_[i].pitch != s_[j].pitch) return false;
        const uint64_t d = (s_[j].at - s_[i].at) % s_[i].pitch;
        if (d < s_[i].width || d + s_[j].width > s_[i].pitch) return false;
      }
    return true;
  }
  void add(const void* p, uint64_t bytes, uint32_t align, bool out) {
    if (!bytes) return;
    if (!p || (uintptr_t)p % align || n_ == MAX_SPANS) bad_ = true;
    else s_[n_++] = {(uintptr_t)p, bytes, out, 0, 0};
  }
  static constexpr int MAX_SPANS = 12 * MAX_RANKS + 8;
  Span s_[MAX_SPANS];
  int n_ = 0;
  bool bad_ = false;
};

}  // namespace ar
