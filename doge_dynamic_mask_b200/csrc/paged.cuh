// The paged cache as the decode kernels see it.
#pragma once

#include "common.cuh"

namespace dma {

// One sequence's visible keys.  With a window the visible positions are
// [0, sinks) and [len - window, len) (their union once they meet), else
// [0, len): n of them, the i-th at position i, or i + shift from the sinks on.
struct SeqView {
  int len, n, shift;
};

__device__ __forceinline__ SeqView seq_view(const PagedCache& c, int b) {
  int len = c.lengths[b];
  const int cap = c.max_pages * c.page_size;
  if (len < 0 || len > cap) {
    raise_error(c.err, kDevErrBadLength);
    len = len < 0 ? 0 : cap;
  }
  const int shift = c.window > 0 ? max(0, len - c.window - c.sinks) : 0;
  return SeqView{len, len - shift, shift};
}

__device__ __forceinline__ int key_position(const PagedCache& c, const SeqView& v, int i) {
  return v.shift > 0 && i >= c.sinks ? i + v.shift : i;
}

// position -> (page slot of the table, row of the page).  Positions lie below 2^20, so
// the product with the reciprocal is off by less than a quarter of 1 / page_size:
// its whole part is the slot, or one below it where the position begins a page.
__device__ __forceinline__ int page_slot(const PagedCache& c, int j, int& off) {
  int slot;
  if (c.page_shift >= 0) {
    slot = j >> c.page_shift;
    off = j - slot * c.page_size;
  } else {
    slot = static_cast<int>(static_cast<float>(j) * c.page_inv);
    off = j - slot * c.page_size;
    if (off >= c.page_size) {
      off -= c.page_size;
      ++slot;
    }
  }
  return slot;
}

// the pool page behind a table entry, or -1 (reported) when it is outside the pool
__device__ __forceinline__ int checked_page(const PagedCache& c, int page) {
  if (page >= 0 && page < c.num_pages) return page;
  raise_error(c.err, kDevErrBadPage);
  return -1;
}

// Offset of a head's row in k_pages / v_pages in 16-byte units (the entry
// points refuse pools where it does not fit 32 bits).
__device__ __forceinline__ uint32_t row_offset16(const PagedCache& c, int page, int off, int g) {
  return static_cast<uint32_t>(page) * static_cast<uint32_t>(c.page_stride16) +
         static_cast<uint32_t>((off * c.Hkv + g) * (c.d / 8));
}

// Offset of a key's dt (32 bits hold it: a pool of K rows has at most 2^32
// 16-byte units, so fewer than 2^30 rows of a head).
__device__ __forceinline__ uint32_t dt_offset(const PagedCache& c, int page, int off, int g) {
  return static_cast<uint32_t>(page) * static_cast<uint32_t>(c.Hkv * c.page_size) +
         static_cast<uint32_t>(g * c.page_size + off);
}

// a row offset that stands for no key
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

}  // namespace dma
