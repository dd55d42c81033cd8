// Attention of a few query tokens per sequence over the paged 4-bit cache.
//
// For a row (one query token of one head) with scores s_j = scale q . k_j over the
// keys it sees, o = sum_j 2^(t_j - r) v_j / sum_j 2^(t_j - r), t = s log2(e), for any
// reference r; a warp keeps one reference per row and moves it only when a score
// exceeds it by more than 2^8 (the sums then scale by a power of two, rarely).
//
// Bound: the cache's bytes (1.125 bytes per cached value of a head pair, each read
// once, for all query heads that share the head).  What makes that hard is the
// unpacking: at 6.8 TB/s an SM receives ~40 codes per cycle, so a code may cost it
// two or three instruction lanes.  Hence:
//  * Codes go to the matrix unit as they are.  A nibble masked out in place is, read
//    as fp16, the subnormal q 2^-24 (bits 0-3) or q 2^-20 (bits 4-7), which the
//    matrix instructions multiply exactly; so 8 codes take 4 masks and 1 shift, no
//    conversion.  The -8 of (q - 8) is a constant of the query for the scores (it
//    starts the accumulator) and a product with a constant matrix for the values.
//    The two nibbles' factors meet in the query (q 2^-4 for high nibbles) and in the
//    output's last scaling.
//  * Scores: S^T = K Q^T (m16n8k16): 16 keys x 8 rows, one accumulator per 32-value
//    block, which the key's scale multiplies in fp32.  The query is rounded to fp16
//    after a power-of-two scaling per row (exact for bf16 and fp16 inputs down to
//    2^-24 of the row's largest value).
//  * Values: O^T = V^T P^T, P^T from the scores by an 8x8 transpose, multiplied by the
//    value's scale per block (fp16: p and p d are each off by at most 2^-11 of
//    themselves; sums are fp32).  The reference r includes the largest scale seen, so
//    p d stays inside fp16 whatever the scales are.
//  * Rows in the matrix's N: 8 of them (heads sharing a key head x query tokens).
//
// Work: the 32-token tiles of all (sequence, key head) pairs in a row are split evenly
// over the CTAs (a sequence's length does not matter), and the tiles of a CTA's piece
// of one pair go round its warps.  Each warp copies its own tiles (one bulk copy per
// tile, as the layout keeps a tile contiguous) into a ring of its own, running ahead
// across pieces, so no CTA barrier stands in the loop.  Pieces are merged over the
// warps in shared memory; a pair that several CTAs share is merged by the last of
// them from partial results in the workspace, in the order of the CTAs, so results do
// not depend on timing.
#include <algorithm>

#include "attn_common.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;  // log2 by which a score may exceed its row's reference
constexpr int kRows = 8;      // rows (heads x query tokens) of one work unit

struct DecodeJob {
  moe_kv_cache c;
  const int32_t *lens;
  moe_tensor q;
  int hq, group, q_tokens, window, row_tiles;
  float scale;
  void *out;
  float *lse;
  float *part;        // [grid][2][kRows][D + 2]: partial sums, reference and weight sum per row
  uint32_t *count;    // [grid]: pieces done of the pair whose first piece that CTA has
  int min_share;      // fewest tiles of one CTA
};

template <int D>
struct DecodeCfg {
  static constexpr int kWarps = 8;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kTile = 36 * D;
  static constexpr int kOut = kRows * D;  // values of one merged result
  static constexpr size_t kRing = (size_t)kWarps * kStages * kTile;
  static constexpr size_t kSmem = kRing + (size_t)(kWarps / 2) * (kOut + 2 * kRows) * sizeof(float);
  static constexpr int kCtas = D == 256 ? 1 : 2;  // resident per SM
};

__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  return h2_bits(__hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b)));
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store_pair(__half *p, float a, float b) {
  *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b);
}

// A walk over the pieces of a CTA's range of units.  Units are ordered by
// sequence, then key head and row tile, then tile.
struct Walk {
  int64_t left;   // units not yet walked
  int seq, hr;    // current pair: sequence, key head * row_tiles + row tile
  int first;      // first tile of what the sequence's rows see
  int n;          // tiles of the pair
  int at, end;    // this piece: tiles [at, end) of the pair (counted from `first`)
};

__device__ __forceinline__ int seq_tiles(const DecodeJob &j, int s, int *first) {
  int64_t f;
  const int64_t n = kv_tiles(__ldg(j.lens + s), j.q_tokens, j.window, j.c.table_width, j.c.page_size, &f);
  *first = (int)f;
  return n < 0 ? 0 : (int)n;
}

__device__ __forceinline__ void walk_clip(Walk &w) {
  w.end = (int)(w.left < (int64_t)(w.n - w.at) ? w.at + w.left : w.n);
  w.left -= w.end - w.at;
}
// Next piece; false when the range is done.
__device__ __forceinline__ bool walk_next(const DecodeJob &j, Walk &w) {
  if (w.left <= 0) return false;
  if (++w.hr == j.c.n_kv_heads * j.row_tiles) {
    w.hr = 0;
    do {
      if (++w.seq >= j.c.n_seqs) return false;
      w.n = seq_tiles(j, w.seq, &w.first);
    } while (w.n == 0);
  }
  w.at = 0;
  walk_clip(w);
  return true;
}

template <int D, typename T>
__global__ void __launch_bounds__(32 * DecodeCfg<D>::kWarps, DecodeCfg<D>::kCtas) kv_attention_kernel(const DecodeJob j) {
  using C = DecodeCfg<D>;
  constexpr int W = C::kWarps, S = C::kStages, NB = D / 32, kThreads = 32 * W;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t bars[W][S];
  __shared__ int64_t scan[W], sh_off;
  __shared__ int sh_seq, sh_last;
  float *merge = reinterpret_cast<float *>(sm + C::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int heads = j.c.n_kv_heads * j.row_tiles;
  uint64_t *bar = bars[warp];
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) a_mbar_init(&bar[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();

  // ---- this CTA's share of the units
  int64_t mine = 0;
  for (int s = tid; s < j.c.n_seqs; s += kThreads) {
    int first;
    mine += seq_tiles(j, s, &first);
  }
  int64_t sum = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) scan[warp] = sum;
  if (tid == 0) sh_seq = -1;
  __syncthreads();
  int64_t units = 0;
  for (int w = 0; w < W; ++w) units += scan[w];
  units *= heads;
  int64_t share = (units + gridDim.x - 1) / gridDim.x;
  if (share < j.min_share) share = j.min_share;
  const int64_t u0 = share * blockIdx.x;

  // ---- sequences without tiles (empty, or a length the table cannot hold): their rows
  for (int s = blockIdx.x; s < j.c.n_seqs; s += gridDim.x) {
    const int len = __ldg(j.lens + s);
    int first;
    if (seq_tiles(j, s, &first) > 0) continue;
    const bool bad = len != 0;
    if (bad && tid == 0 && j.c.status) atomicOr(j.c.status, MOE_KV_BAD_LENGTH);
    const float fill = bad ? a_nan() : 0.f;
    const int64_t n = (int64_t)j.q_tokens * j.hq;
    T *o = static_cast<T *>(j.out) + (int64_t)s * n * D;
    for (int64_t i = tid; i < n * D / 2; i += kThreads) store_pair(o + 2 * i, fill, fill);
    if (j.lse)
      for (int64_t i = tid; i < n; i += kThreads) j.lse[(int64_t)s * n + i] = bad ? a_nan() : -a_inf();
  }
  if (u0 >= units) return;

  // ---- where the share begins
  Walk walk;
  {
    int64_t run = 0;
    __syncthreads();
    for (int base = 0; base < j.c.n_seqs; base += kThreads) {
      const int s = base + tid;
      int first = 0;
      const int64_t n = s < j.c.n_seqs ? (int64_t)seq_tiles(j, s, &first) * heads : 0;
      int64_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      int64_t before = run, all = run;
      for (int w = 0; w < W; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
      }
      if (u0 >= before + inc - n && u0 < before + inc) {
        sh_seq = s;
        sh_off = u0 - (before + inc - n);
      }
      __syncthreads();
      run = all;
      if (sh_seq >= 0) break;
    }
    walk.seq = sh_seq;
    walk.n = seq_tiles(j, walk.seq, &walk.first);
    walk.hr = (int)(sh_off / walk.n);
    walk.at = (int)(sh_off % walk.n);
    walk.left = min(share, units - u0);
    walk_clip(walk);
  }
  // unit index of the current pair's first tile
  int64_t pair0 = u0 - walk.at;

  // ---- this warp's copies: a second walk that runs up to S tiles ahead
  unsigned char *ring = sm + (size_t)warp * S * C::kTile;
  Walk load = walk;
  int load_tile = load.at + warp;  // next tile to copy
  bool load_more = true;
  uint32_t issued = 0, used = 0;
  int pages = 0, pages_at = -1, pages_seq = -1;  // page numbers of the next tiles, one per lane
  uint32_t bad_mask = 0;  // of the last 32 copies, by (issued & 31): a tile without a page

  auto issue = [&]() {
    // the next tile of this warp, or nothing
    while (load_more && load_tile >= load.end) {
      load_more = walk_next(j, load);
      load_tile = load.at + warp;
    }
    if (!load_more) return;
    if (pages_seq != load.seq || load_tile < pages_at || load_tile >= pages_at + 32 * W ||
        (load_tile - pages_at) % W != 0) {
      pages_seq = load.seq;
      pages_at = load_tile;
      const int tile = load_tile + lane * W;
      int in_page = 0, p = -1;
      if (tile < load.n)
        p = kv_page(j.c.page_table + (int64_t)load.seq * j.c.table_stride, j.c.table_width, j.c.n_pages,
                    j.c.page_size, load.first + tile, &in_page);
      pages = p;
    }
    const int page = __shfl_sync(0xffffffffu, pages, (load_tile - pages_at) / W);
    const int st = issued % S;
    const int per = j.c.page_size / kKvTile;
    const int in_page = (load.first + load_tile) % per;
    bad_mask &= ~(1u << (issued & 31));
    if (page < 0) {
      bad_mask |= 1u << (issued & 31);
      if (lane == 0) a_mbar_arrive(&bar[st]);
    } else if (lane == 0) {
      a_expect_tx(&bar[st], C::kTile);
      a_bulk_load(ring + (size_t)st * C::kTile,
                  static_cast<const uint8_t *>(j.c.pages) + (int64_t)page * j.c.page_stride +
                      kv_tile_off(D, j.c.page_size, load.hr / j.row_tiles, in_page),
                  C::kTile, &bar[st]);
    }
    ++issued;
    load_tile += W;
  };
#pragma unroll
  for (int s = 0; s < S; ++s) issue();

  bool dead = false;  // a wait gave up: nothing more is copied or read
  do {
    const int kvh = walk.hr / j.row_tiles, rt = walk.hr % j.row_tiles;
    const int64_t len = __ldg(j.lens + walk.seq);
    const int n_rows = j.group * j.q_tokens;
    // ---- the rows' queries: lane (g, t) holds row g's values 4t.. of each half block
    uint32_t qf[NB][4];
    float qinit[NB][2], f[2];
    int lo[2], hi[2], all_lo = 0, all_hi = 0x7fffffff;
    {
      const int r = rt * kRows + g;
      float x[NB][8];
      float top = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int z = 0; z < 8; ++z) x[b][z] = 0.f;
      if (r < n_rows) {
        const T *src = static_cast<const T *>(j.q.data) +
                       ((int64_t)walk.seq * j.q_tokens + r / j.group) * j.q.token_stride +
                       (int64_t)(kvh * j.group + r % j.group) * j.q.head_stride;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint2 raw = *reinterpret_cast<const uint2 *>(src + 32 * b + 16 * half + 4 * t);
            const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              x[b][4 * half + z] = to_float(e[z]);
              top = fmaxf(top, fabsf(x[b][4 * half + z]));
            }
          }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e with the row's largest value below 2^13 after it (an infinity or NaN stays what it is)
      int e = 12;
      if (top > 0.f && top < a_inf()) e = 12 - ((int)((__float_as_uint(top) >> 23) & 255) - 127);
      e = min(max(e, -120), 120);
      const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float total = 0.f;
        __half h[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          // high nibbles are 2^4 too large as fp16: their query values are 2^-4
          h[z] = __float2half_rn(x[b][z] * up * (z < 4 ? 1.f : 0.0625f));
          total += __half2float(h[z]) * (z < 4 ? 1.f : 16.f);
        }
        qf[b][0] = h2_bits(__halves2half2(h[0], h[2]));
        qf[b][1] = h2_bits(__halves2half2(h[1], h[3]));
        qf[b][2] = h2_bits(__halves2half2(h[4], h[6]));
        qf[b][3] = h2_bits(__halves2half2(h[5], h[7]));
        total += __shfl_xor_sync(0xffffffffu, total, 1);
        total += __shfl_xor_sync(0xffffffffu, total, 2);
        total *= -8.f * 5.9604644775390625e-08f;  // -8 x 2^-24
        qinit[b][0] = __shfl_sync(0xffffffffu, total, 8 * t);
        qinit[b][1] = __shfl_sync(0xffffffffu, total, 8 * t + 4);
      }
      const float mine_f = j.scale * kLog2e * down * 16777216.f;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        f[z] = __shfl_sync(0xffffffffu, mine_f, 8 * t + 4 * z);
        const int rr = rt * kRows + 2 * t + z;
        int64_t l = 0, h = 0;
        if (rr < n_rows) kv_visible(len, j.q_tokens, rr / j.group, j.window, &l, &h);
        lo[z] = (int)l;
        hi[z] = (int)h;
      }
      // a tile inside [all_lo, all_hi) is seen whole by every row
      const int last = min(n_rows, (rt + 1) * kRows) - 1;
      int64_t l, h;
      kv_visible(len, j.q_tokens, last / j.group, j.window, &l, &h);
      all_lo = (int)l;
      kv_visible(len, j.q_tokens, rt * kRows / j.group, j.window, &l, &h);
      all_hi = (int)h;
    }
    // ---- this warp's tiles of the piece
    float acc[NB][2][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[b][h][z] = 0.f;
    float m[2] = {-a_inf(), -a_inf()}, l[2] = {0.f, 0.f};
    float dtop = 0.f;   // largest value scale seen
    float shift = -7.f; // reference = m + shift
    bool poison = false;

    for (int tile = walk.at + warp; tile < walk.end; tile += W) {
      const int st = used % S;
      const bool bad = (bad_mask >> (used & 31)) & 1u;
      if (!dead) dead = !__all_sync(0xffffffffu, a_mbar_wait(&bar[st], (used / S) & 1u));
      ++used;
      if (dead || bad) {
        poison = true;
        if (lane == 0 && j.c.status) atomicOr(j.c.status, dead ? MOE_KV_TIMED_OUT : MOE_KV_BAD_PAGE);
        __syncwarp();
        if (!dead) issue();
        continue;
      }
      const unsigned char *tp = ring + (size_t)st * C::kTile;
      const int tok0 = (walk.first + tile) * kKvTile;
      const bool whole = tok0 >= all_lo && tok0 + kKvTile <= all_hi;
      // key k of the matrix (of 8) is token perm(k) = k / 2 + 4 (k odd), so that the value operand's
      // pairs (2t, 2t + 1) are tokens t and t + 4 and a load covers neighbouring tokens
      const int pg = (g >> 1) + ((g & 1) << 2);
      float s[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int ra = mt * 16 + pg;
        __half2 ka[NB / 2], kb[NB / 2];
        {
          const unsigned char *sa = tp + 16 * D + ra * (D / 16), *sb = sa + 8 * (D / 16);
          if constexpr (NB == 2) {
            ka[0] = *reinterpret_cast<const __half2 *>(sa);
            kb[0] = *reinterpret_cast<const __half2 *>(sb);
          } else {
#pragma unroll
            for (int z = 0; z < NB / 4; ++z) {
              *reinterpret_cast<uint2 *>(&ka[2 * z]) = *reinterpret_cast<const uint2 *>(sa + 8 * z);
              *reinterpret_cast<uint2 *>(&kb[2 * z]) = *reinterpret_cast<const uint2 *>(sb + 8 * z);
            }
          }
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) s[mt][z] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t wa = *reinterpret_cast<const uint32_t *>(tp + (b * 32 + ra) * 16 + 4 * t);
          const uint32_t wb = *reinterpret_cast<const uint32_t *>(tp + (b * 32 + ra + 8) * 16 + 4 * t);
          const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
          float c[4] = {qinit[b][0], qinit[b][1], qinit[b][0], qinit[b][1]};
          mma16816(c, wa & 0x000F000Fu, wb & 0x000F000Fu, wa8 & 0x000F000Fu, wb8 & 0x000F000Fu, qf[b][0], qf[b][1]);
          mma16816(c, wa & 0x00F000F0u, wb & 0x00F000F0u, wa8 & 0x00F000F0u, wb8 & 0x00F000F0u, qf[b][2], qf[b][3]);
          const float2 da = __half22float2(ka[b / 2]), db = __half22float2(kb[b / 2]);
          const float fa = (b & 1) ? da.y : da.x, fb = (b & 1) ? db.y : db.x;
          s[mt][0] = fmaf(c[0], fa, s[mt][0]);
          s[mt][1] = fmaf(c[1], fa, s[mt][1]);
          s[mt][2] = fmaf(c[2], fb, s[mt][2]);
          s[mt][3] = fmaf(c[3], fb, s[mt][3]);
        }
      }
      // ---- scores in log2 units; what a row does not see is -inf
      bool over = false;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          s[mt][z] *= f[z & 1];
          if (!whole) {
            const int key = tok0 + mt * 16 + (z >= 2 ? 8 : 0) + pg;
            if (key < lo[z & 1] || key >= hi[z & 1]) s[mt][z] = -a_inf();
          }
          over |= s[mt][z] > m[z & 1] + kLazy;
        }
      // ---- the largest value scale of the tile (those of tokens past the sequence count as 0)
      const unsigned char *vs = tp + 34 * D;
      uint32_t dmax = 0;
#pragma unroll
      for (int z = 0; z < D / 64; ++z) {
        const int off = (z * 32 + lane) * 4;  // two scales of one token
        uint32_t w = *reinterpret_cast<const uint32_t *>(vs + off) & 0x7FFF7FFFu;
        if (!whole && tok0 + off / (D / 16) >= (int)len) w = 0;
        dmax = __vmaxu2(dmax, w & ~__vcmpgtu2(w, 0x7BFF7BFFu));  // a NaN is no scale to make room for
      }
      const float dlane = fmaxf(__low2float(*reinterpret_cast<__half2 *>(&dmax)),
                                __high2float(*reinterpret_cast<__half2 *>(&dmax)));
      over |= dlane > dtop;
      if (__any_sync(0xffffffffu, over)) {
        float dn = dlane, mn[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) mn[z] = fmaxf(fmaxf(s[0][z], s[0][z + 2]), fmaxf(s[1][z], s[1][z + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mn[0] = fmaxf(mn[0], __shfl_xor_sync(0xffffffffu, mn[0], o));
          mn[1] = fmaxf(mn[1], __shfl_xor_sync(0xffffffffu, mn[1], o));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) dn = fmaxf(dn, __shfl_xor_sync(0xffffffffu, dn, o));
        float shift_n = shift;
        if (dn > dtop) {
          // the new bound leaves room for scales up to twice the largest one; 2^(8 - shift) dtop < 2^16
          dtop = fminf(dn, 65504.f) * 2.f;
          const int ex = (int)((__float_as_uint(dtop) >> 23) & 255) - 126;  // dtop < 2^ex
          shift_n = fmaxf((float)ex - 6.f, -7.f);
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float m_new = fmaxf(m[z], mn[z]);
          const float a = m[z] == -a_inf() ? 0.f : a_exp2((m[z] - m_new) + (shift - shift_n));
          m[z] = m_new;
          l[z] *= a;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              acc[b][h][z] *= a;
              acc[b][h][z + 2] *= a;
            }
        }
        shift = shift_n;
      }
      const float r0 = m[0] == -a_inf() ? 0.f : m[0] + shift, r1 = m[1] == -a_inf() ? 0.f : m[1] + shift;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float p0 = a_exp2(s[mt][0] - r0), p1 = a_exp2(s[mt][1] - r1);
        const float p2 = a_exp2(s[mt][2] - r0), p3 = a_exp2(s[mt][3] - r1);
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        const uint32_t b0 = transpose8x8(h2_bits(__floats2half2_rn(p0, p1)));  // row g, tokens t and t + 4
        const uint32_t b1 = transpose8x8(h2_bits(__floats2half2_rn(p2, p3)));  // row g, tokens t + 8 and t + 12
        const int k0 = mt * 16 + t;
        uint32_t d[4][NB / 2];  // scales of tokens t, t + 4, t + 8, t + 12
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const unsigned char *sp = vs + (k0 + 4 * z) * (D / 16);
          if constexpr (NB == 2) {
            d[z][0] = *reinterpret_cast<const uint32_t *>(sp);
          } else {
#pragma unroll
            for (int y = 0; y < NB / 4; ++y) {
              const uint2 v = *reinterpret_cast<const uint2 *>(sp + 8 * y);
              d[z][2 * y] = v.x;
              d[z][2 * y + 1] = v.y;
            }
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t sel = (b & 1) ? 0x7632u : 0x5410u;
          uint32_t e0 = mul_h2(b0, __byte_perm(d[0][b / 2], d[1][b / 2], sel));
          uint32_t e1 = mul_h2(b1, __byte_perm(d[2][b / 2], d[3][b / 2], sel));
          if (!whole) {
            // a weight of 0 contributes 0 even where the scale is not finite: such a token may be unseen
            const uint32_t z0 = __vcmpeq2(b0, 0u), z1 = __vcmpeq2(b1, 0u);
            e0 &= ~z0;
            e1 &= ~z1;
          }
          const unsigned char *cp = tp + 18 * D + (b * 32 + k0) * 16 + 2 * g;
          const uint32_t v0 = *reinterpret_cast<const uint16_t *>(cp), v1 = *reinterpret_cast<const uint16_t *>(cp + 64);
          const uint32_t v2 = *reinterpret_cast<const uint16_t *>(cp + 128),
                         v3 = *reinterpret_cast<const uint16_t *>(cp + 192);
          const uint32_t x = __byte_perm(v0, v1, 0x5410u), y = __byte_perm(v2, v3, 0x5410u);
          const uint32_t x8 = x >> 8, y8 = y >> 8;
          mma16816(acc[b][0], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, e0, e1);
          mma16816(acc[b][1], x8 & 0x000F000Fu, x8 & 0x00F000F0u, y8 & 0x000F000Fu, y8 & 0x00F000F0u, e0, e1);
          // -8: as fp16, -8 2^-24 for the low nibbles' rows and -8 2^-20 for the high ones'
          mma16816(acc[b][0], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, e0, e1);
          mma16816(acc[b][1], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, e0, e1);
        }
      }
      __syncwarp();
      issue();
    }
    // ---- merge the warps: l over the lanes that share a row, then pairwise over the warps
    if (__any_sync(0xffffffffu, poison)) l[0] = l[1] = a_nan();
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    float r[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) r[z] = m[z] == -a_inf() ? -a_inf() : m[z] + shift;
    constexpr int kSlot = C::kOut + 2 * kRows;
#pragma unroll 1
    for (int half = W / 2; half > 0; half >>= 1) {
      __syncthreads();
      if (warp >= half && warp < 2 * half) {
        float *o = merge + (size_t)(warp - half) * kSlot;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float4 *>(o + ((b * 2 + h) * 32 + lane) * 4) =
                make_float4(acc[b][h][0], acc[b][h][1], acc[b][h][2], acc[b][h][3]);
        if (g == 0)
          *reinterpret_cast<float4 *>(o + C::kOut + 4 * t) = make_float4(r[0], r[1], l[0], l[1]);
      }
      __syncthreads();
      if (warp < half) {
        const float *o = merge + (size_t)warp * kSlot;
        const float4 w = *reinterpret_cast<const float4 *>(o + C::kOut + 4 * t);
        const float ro[2] = {w.x, w.y}, lo2[2] = {w.z, w.w};
        float wa[2], wb[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float top = fmaxf(r[z], ro[z]);
          wa[z] = r[z] == -a_inf() ? 0.f : a_exp2(r[z] - top);
          wb[z] = ro[z] == -a_inf() ? 0.f : a_exp2(ro[z] - top);
          // a poisoned warp may hold no weight: its NaN must not be multiplied away
          l[z] = (l[z] != l[z] || lo2[z] != lo2[z]) ? a_nan() : l[z] * wa[z] + lo2[z] * wb[z];
          r[z] = top;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 v = *reinterpret_cast<const float4 *>(o + ((b * 2 + h) * 32 + lane) * 4);
            acc[b][h][0] = acc[b][h][0] * wa[0] + v.x * wb[0];
            acc[b][h][1] = acc[b][h][1] * wa[1] + v.y * wb[1];
            acc[b][h][2] = acc[b][h][2] * wa[0] + v.z * wb[0];
            acc[b][h][3] = acc[b][h][3] * wa[1] + v.w * wb[1];
          }
      }
    }
    // ---- the piece's result, or its part of the pair's
    const int64_t first_cta = pair0 / share, last_cta = (pair0 + walk.n - 1) / share;
    const bool alone = first_cta == last_cta;
    const int64_t tok = (int64_t)walk.seq * j.q_tokens;
    if (warp == 0) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int row = 2 * t + z, rr = rt * kRows + row;
        float *po = j.part + ((size_t)(blockIdx.x * 2 + (blockIdx.x == first_cta ? 1 : 0)) * kRows + row) * (D + 2);
        const float inv = l[z] > 0.f || l[z] != l[z] ? 1.f / l[z] : 0.f;
        const bool live = rr < n_rows;
        const int64_t at = (tok + rr / j.group) * j.hq + kvh * j.group + rr % j.group;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float k = half ? 1048576.f : 16777216.f;
            const float a = acc[b][0][z + 2 * half] * k, c = acc[b][1][z + 2 * half] * k;
            const int dim = 32 * b + 16 * half + 2 * g;
            if (alone) {
              if (live) store_pair(static_cast<T *>(j.out) + at * D + dim, a * inv, c * inv);
            } else {
              *reinterpret_cast<float2 *>(po + dim) = make_float2(a, c);
            }
          }
        if (g == 0) {
          if (!alone) *reinterpret_cast<float2 *>(po + D) = make_float2(r[z], l[z]);
          else if (live && j.lse) j.lse[at] = l[z] == 0.f ? -a_inf() : (r[z] + log2f(l[z])) * kLn2;
        }
      }
    }
    if (!alone) {
      __threadfence();
      __syncthreads();
      const int parts = (int)(last_cta - first_cta) + 1;
      if (tid == 0) {
        __threadfence();
        sh_last = atomicAdd(j.count + first_cta, 1u) == (uint32_t)(parts - 1);
      }
      __syncthreads();
      if (sh_last) {
        __threadfence();
        if (tid == 0) j.count[first_cta] = 0;
        auto piece = [&](int i) {
          return j.part + (size_t)((first_cta + i) * 2 + (i == 0 ? 1 : 0)) * kRows * (D + 2);
        };
        for (int x = tid; x < kRows * D / 2; x += kThreads) {
          const int row = x / (D / 2), dim = (x % (D / 2)) * 2, rr = rt * kRows + row;
          if (rr >= n_rows) continue;
          float top = -a_inf();
          for (int i = 0; i < parts; ++i) top = fmaxf(top, __ldcg(piece(i) + row * (D + 2) + D));
          float a = 0.f, c = 0.f, sum_l = 0.f;
          for (int i = 0; i < parts; ++i) {
            const float *p = piece(i) + row * (D + 2);
            const float2 rl = __ldcg(reinterpret_cast<const float2 *>(p + D));
            const float2 v = __ldcg(reinterpret_cast<const float2 *>(p + dim));
            if (rl.y != rl.y) sum_l = a_nan();
            if (rl.x == -a_inf()) continue;
            const float w = a_exp2(rl.x - top);
            a += v.x * w;
            c += v.y * w;
            sum_l += rl.y * w;
          }
          const float inv = sum_l > 0.f || sum_l != sum_l ? 1.f / sum_l : 0.f;
          const int64_t at = (tok + rr / j.group) * j.hq + kvh * j.group + rr % j.group;
          store_pair(static_cast<T *>(j.out) + at * D + dim, a * inv, c * inv);
          if (dim == 0 && j.lse) j.lse[at] = sum_l == 0.f ? -a_inf() : (top + log2f(sum_l)) * kLn2;
        }
      }
    }
    // ---- next piece
    pair0 += walk.n;
  } while (walk_next(j, walk));
  // copies that a wait gave up on, or that came after it, must have landed before the CTA's memory is gone
  if (dead)
    for (uint32_t i = issued > S ? issued - S : 0; i < issued; ++i) (void)a_mbar_wait(&bar[i % S], (i / S) & 1u);
}

constexpr int kDecodeSms = 152;

int decode_grid_cap(int D) { return kDecodeSms * (D == 256 ? 1 : 2); }

template <int D, typename T>
int launch_decode(const DecodeJob &j, int grid, cudaStream_t st) {
  static DynSmemLimit limit;
  if (ensure_dyn_smem(kv_attention_kernel<D, T>, DecodeCfg<D>::kSmem, limit) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  kv_attention_kernel<D, T><<<grid, 32 * DecodeCfg<D>::kWarps, DecodeCfg<D>::kSmem, st>>>(j);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

constexpr int64_t kCountBytes = 4096;  // counters at the head of the workspace

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int64_t moe_kv_attention_workspace(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t q_tokens) {
  if (n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || q_tokens <= 0 || !kv_sizes_ok(n_kv_heads, head_dim, 32))
    return 0;
  return kCountBytes + (int64_t)decode_grid_cap(head_dim) * 2 * kRows * (head_dim + 2) * 4;
}

MOE_API int moe_kv_attention(const moe_kv_cache *c, const int32_t *seq_lens, const moe_tensor *q, int32_t n_q_heads,
                             int32_t q_tokens, float scale, int32_t window, void *out, float *lse, int32_t dtype,
                             void *workspace, int64_t workspace_bytes, void *cuda_stream) {
  if (c && c->n_seqs == 0) return MOE_OK;
  if (const int rc = check_cache(c)) return rc;
  if (!seq_lens || !out || n_q_heads <= 0 || n_q_heads % c->n_kv_heads || q_tokens <= 0 || window < 0 ||
      !(scale > 0.f && scale <= 3.4e38f))
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (n_q_heads > kMaxAttnHeads || q_tokens > 1024) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)c->table_width * c->page_size > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  if (const int rc = check_tensor(q, 2)) return rc;
  if ((uintptr_t)out % 16 || (uintptr_t)lse % 4 || !workspace || (uintptr_t)workspace % 256 ||
      workspace_bytes < moe_kv_attention_workspace(n_q_heads, c->n_kv_heads, c->head_dim, q_tokens))
    return MOE_ERR_INVALID_ARG;
  DecodeJob j = {};
  j.c = *c;
  j.lens = seq_lens;
  j.q = *q;
  j.hq = n_q_heads;
  j.group = n_q_heads / c->n_kv_heads;
  j.q_tokens = q_tokens;
  j.window = window;
  j.row_tiles = (j.group * q_tokens + kRows - 1) / kRows;
  j.scale = scale;
  j.out = out;
  j.lse = lse;
  j.count = static_cast<uint32_t *>(workspace);
  j.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCountBytes);
  j.min_share = 16;
  // no more CTAs than there can be shares
  const int64_t tiles = (int64_t)c->n_seqs * c->n_kv_heads * j.row_tiles *
                        std::max<int64_t>(1, (int64_t)c->table_width * (c->page_size / kKvTile));
  const int64_t most = std::max<int64_t>(1, (tiles + j.min_share - 1) / j.min_share);
  const int grid = (int)std::min<int64_t>(most, decode_grid_cap(c->head_dim));
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const int D = c->head_dim;
  if (dtype == MOE_BF16)
    return D == 64 ? launch_decode<64, __nv_bfloat16>(j, grid, st)
                   : D == 128 ? launch_decode<128, __nv_bfloat16>(j, grid, st) : launch_decode<256, __nv_bfloat16>(j, grid, st);
  return D == 64 ? launch_decode<64, __half>(j, grid, st)
                 : D == 128 ? launch_decode<128, __half>(j, grid, st) : launch_decode<256, __half>(j, grid, st);
}
