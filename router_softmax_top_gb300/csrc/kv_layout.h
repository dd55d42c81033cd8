// Index arithmetic of the paged 4-bit key/value cache: plain C++ that the
// kernels and the host share, with every check of device-side numbers (page
// table entries, lengths, positions) that stands between them and an access.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KV_HD __host__ __device__ inline
#else
#define KV_HD inline
#endif

namespace moe {

constexpr int kKvTile = 32;  // tokens of one tile

// a / b for 0 <= a, 0 < b: 64-bit division is a long sequence of instructions, and rarely needed.
KV_HD int64_t kv_div(int64_t a, int64_t b) {
  if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Bytes of one tile (32 tokens of one head of width D): codes and scales of keys, then of values.
KV_HD int kv_tile_bytes(int D) { return 36 * D; }
// Offsets inside a tile.
KV_HD int kv_code_off(int D, int value, int block, int tok) { return value * 18 * D + (block * 32 + tok) * 16; }
KV_HD int kv_scale_off(int D, int value, int block, int tok) {
  return value * 18 * D + 16 * D + (tok * (D / 32) + block) * 2;
}
// Byte offset of a tile from the start of its page.
KV_HD int64_t kv_tile_off(int D, int page_size, int head, int tile_in_page) {
  return ((int64_t)head * (page_size / kKvTile) + tile_in_page) * kv_tile_bytes(D);
}

// Page of the 32-token tile `tile` of a sequence, or -1 when the table has no
// such entry or its entry is out of range.  row: the sequence's table row.
KV_HD int kv_page(const int32_t *row, int table_width, int n_pages, int page_size, int64_t tile, int *in_page) {
  const int per = page_size / kKvTile;
  *in_page = 0;
  if (tile < 0) return -1;
  const int64_t i = kv_div(tile, per);
  *in_page = (int)(tile - i * per);
  if (i >= table_width) return -1;
  const int32_t p = row[i];
  return (p >= 0 && p < n_pages) ? p : -1;
}

// Position of token i of a call in its sequence, or -1 when the offsets or the
// start make no sense: lo = cu[s], hi = cu[s + 1].
KV_HD int64_t kv_position(int64_t i, int64_t lo, int64_t hi, int64_t start) {
  if (i < lo || i >= hi || start < 0) return -1;
  return start + (i - lo);
}

// Range of keys [lo, hi) that row j of a sequence's q_tokens sees.
KV_HD void kv_visible(int64_t len, int q_tokens, int j, int window, int64_t *lo, int64_t *hi) {
  const int64_t h = len - q_tokens + j + 1;
  *hi = h < 0 ? 0 : h;
  *lo = (window > 0 && h > window) ? h - window : 0;
}

// Tiles [first, first + count) that hold what any row of a sequence sees; -1 when the
// length is not one that the page table can hold.
KV_HD int64_t kv_tiles(int64_t len, int q_tokens, int window, int table_width, int page_size, int64_t *first) {
  *first = 0;
  if (len < 0 || len > (int64_t)table_width * page_size) return -1;
  int64_t lo, hi;
  kv_visible(len, q_tokens, 0, window, &lo, &hi);
  *first = lo / kKvTile;
  return (len + kKvTile - 1) / kKvTile - *first;
}

// A warp's tiles on their way through its ring of S stages: tile x is in stage x % S and completes phase x / S of that
// stage's barrier, which takes one arrival per phase.  Tiles 0..S - 1 are asked for at first, and tile x + S once tile x
// has been taken, but only while every wait has been kept: a stage whose copy never came has a phase that is not over,
// and must be neither armed nor written again.
template <int S>
struct TileRing {
  uint32_t used = 0;  // tiles taken
  bool dead = false;  // a wait gave up: nothing taken from then on counts, and nothing more may be asked for

  static KV_HD uint32_t stage(uint32_t x) { return x % S; }
  static KV_HD uint32_t parity(uint32_t x) { return (x / S) & 1u; }
  // Takes the next tile.  there(x) looks, wait(x) waits, for a limited time, and says whether it came.  When it did not,
  // whatever is on its way is waited for, with the same limit each, so that no copy goes into the ring any more; of a
  // stage that nothing was asked into, the limit runs out.
  template <typename There, typename Wait>
  KV_HD void take(There there, Wait wait) {
    const uint32_t x = used++;
    if (there(x) || dead || wait(x)) return;
    dead = true;
    for (uint32_t y = x; y != x + S; ++y) (void)wait(y);
  }
};

}  // namespace moe
