// Attention of a few query tokens per sequence over the paged 4-bit cache.
//
// For a row (one query token of one head) with scores s_j = scale q . k_j over the
// keys it sees, o = sum_j 2^(t_j - r) v_j / sum_j 2^(t_j - r), t = s log2(e), for any
// reference r; a warp keeps one reference per row and moves it rarely (the sums then
// scale by a power of two).
//
// Bound: the cache's bytes (1.125 bytes per cached value of a head pair, each read once
// for up to 8 rows, query heads that share the head times query tokens; every further 8
// rows read and unpack them again: 64 sequences of 64 to 8192 tokens on 4 key heads of 128
// take 49 us with 8 rows, 79 with 16 and 135 with 32).  What makes that hard is the
// unpacking: at 6.8 TB/s an SM receives ~40 codes per cycle, so a code may cost it
// two or three instruction lanes.  Hence:
//  * Codes go to the matrix unit as they are.  A nibble masked out in place is, read
//    as fp16, the subnormal q 2^-24 (bits 0-3) or q 2^-20 (bits 4-7), which the
//    matrix instructions multiply exactly; so 8 key codes take 4 masks and 1 shift, 8
//    value codes 4 masks and 3 shifts, no conversion.  The -8 of (q - 8) is a constant
//    of the query for the scores (it starts the accumulator) and a product with a
//    constant matrix for the values.  The keys' nibbles' factors meet in the query
//    (q 2^-4 for high nibbles).
//  * Scores: S^T = K Q^T (m16n8k16): 16 keys x 8 rows, one accumulator per 32-value
//    block, which the key's scale multiplies in fp32.  The query is rounded to fp16
//    after a power-of-two scaling per row (exact for bf16 and fp16 inputs down to
//    2^-24 of the row's largest value).  Sums are fp32, cut off 2^-18 below the low
//    nibbles' largest product of a block: 2^-17 scale sum |q k| covers a score.
//  * Values: O^T = V^T E^T, E = p d, a weight times its value's scale per block, formed
//    in fp32, rounded to fp16 once and transposed 8x8 on the way.  A row's reference
//    goes by its largest product p d, not by p and d apart: that product lies between
//    2^10 (when the reference is set) and 2^14, so any other is off by at most 2^-11 of
//    itself or by 2^-35 of the largest, however far apart scales and weights are, and
//    what a row does not see has no part in it.  (With a reference from the largest score
//    and the largest scale, a large scale on a key of no weight took the small weights'
//    products to 0.)  Weights and their sums are fp32.
//  * Rows in the matrix's N: 8 of them (heads sharing a key head x query tokens).
// Measured: 128 sequences of 64 to 8192 tokens (8 key heads of 128, 611 MB of cache) in
// 133 us, 4.6 TB/s or 0.68 of the measured copy rate; 6 us of it go to finding shares and
// the first bytes, 15 to 20 us to slower SMs and the last merges (stamps).  One sequence of
// 131071 tokens takes 47 us, its bytes alone 22.  About 700 instructions per tile, all told,
// keep the integer pipe half busy and the matrix pipe a third.  Scores and values
// interleaved over two tiles, more or fewer warps, deeper rings and whole bytes instead of
// masked high nibbles were all slower or less exact.
//
// Work: the 32-token tiles of all (sequence, key head) pairs in a row, plus a few
// tiles' worth per pair for its set-up and result, are split evenly over all warps of
// the grid, so neither a sequence's length nor its place matters.  A warp walks its
// share alone: it copies its own tiles (one bulk copy per tile, as the layout keeps a
// tile contiguous) into a ring of its own, running ahead across pairs, and writes the
// result of every pair that it has whole; no barrier stands in the loop.  A pair that
// warps of one CTA share is merged by the last of them to be done; one that several CTAs
// share by the last of those, from partial results in the workspace; always in the order
// of the keys, so results do not depend on timing.  Few short pairs instead take a CTA
// each, whose warps share its tiles: nothing is merged across CTAs.
#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"

namespace moe {
namespace {

// A row's reference is set so that its largest product of a weight with a scale is 2^kCentre, and moves when one exceeds
// kMost; or, where values are small against their weights, so that no weight exceeds 2^kDeep, and moves at kDeepMost.
constexpr float kCentre = 10.f, kMost = 16384.f, kDeep = 70.f, kDeepMost = 7.5557864e22f /* 2^76 */;
constexpr float kEarly = 1.3877787807814457e-17f;  // 2^-56: 2^24 less 2^80 (see the score's factor)
constexpr float kNone = -3.3e38f;  // the reference of a row that has seen nothing: below any score
constexpr int kDecodeWarps = 8;
constexpr int kDecodeSms = 152, kDecodeCtasMost = 2 * kDecodeSms;  // CTAs of a launch at most
constexpr int kRows = 8;      // rows (heads x query tokens) of one work unit

struct DecodeJob {
  moe_kv_cache c;
  const int32_t *lens;
  moe_tensor q;
  int hq, group, q_tokens, window, row_tiles;
  float scale;
  void *out;
  float *lse;
  float *part;        // [grid][2 + kWarps][kPart]: partial results of the pairs that a CTA shares with the one before
                      // or after, then those of the first pieces of its warps
  uint32_t *count;    // [grid]: CTAs done with the pair whose first tiles that CTA has
};

template <int D>
struct DecodeCfg {
  static constexpr int kWarps = kDecodeWarps;
  static constexpr int kStages = 2;  // (four, for heads of 64, are no faster)
  static constexpr int kTile = 36 * D;
  // a partial result: accumulators as the matrix unit leaves them, [D/16][32 lanes][4], then per t of a lane the
  // references and weight sums of rows 2t and 2t + 1
  static constexpr int kOut = kRows * D, kPart = kOut + 16;
  static constexpr size_t kRing = (size_t)kWarps * kStages * kTile;
  // per warp and block: the query operand (16 bytes per lane), and the accumulators' start (16 bytes per t)
  static constexpr int kQuery = (D / 32) * (32 + 4) * 16;
  static constexpr size_t kSmem = kRing + (size_t)kWarps * kQuery;
  static constexpr int kCtas = D == 256 ? 1 : 2;  // resident per SM
  static_assert((size_t)kStages * kTile >= kPart * sizeof(float), "a warp's ring holds its last partial result");
};

// d = a b + c
__device__ __forceinline__ void mma16816_from(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// c += a b
__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store_pair(__half *p, float a, float b) {
  *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b);
}

// (out of line: a copy is nearly always there)
__device__ __noinline__ bool wait_for_tile(uint64_t *bar, uint32_t parity) { return a_mbar_wait(bar, parity); }

// What a pair costs beside its tiles, in tiles (its queries' set-up and its result).  Measured with 1, 2, 4, 8 and 16:
// 128 sequences of 64 to 8192 tokens 139, 133, 133, 136 and 144 us; one of 131071 tokens 53, 49, 47.5, 47 and 47 us.
constexpr int kPairCost = 4;
// Where there are CTAs for all pairs, a pair takes a CTA of its own and no more if its longest warp then has at most
// this many tiles more than with even shares, which the merges across CTAs cost.  A CTA per pair against shares: 333
// tokens 10.3 and 14.6 us, 1000 tokens 13.2 and 15.0 us, 32 sequences of 1024 tokens of 64 (256 pairs) 13.2 and 17.9 us,
// 8 of 1000 (64 pairs) 13.7 and 15.8 us, 8 of 2000 18.5 and 18.9 us; but one of 2000 17.9 and 14.8 us, of 4000 27.1 and
// 14.6 us.
constexpr int kAloneMore = 4;

// A walk over the pieces (tiles of one pair) of a warp's share.  Pairs are ordered by sequence, then key head
// and row tile; a pair of n tiles takes kPairCost + n places, its tiles the last n of them.
struct Walk {
  int64_t left;   // places of the share not yet walked
  int64_t pair0;  // the current pair's first place
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

// The piece of the current pair from its place `off` on; false when the share holds none of its tiles.
__device__ __forceinline__ bool walk_clip(Walk &w, int64_t off) {
  const int64_t take = min(w.left, (int64_t)(w.n + kPairCost) - off);
  w.at = (int)max((int64_t)0, off - kPairCost);
  w.end = (int)max((int64_t)w.at, off + take - kPairCost);
  w.left -= take;
  return w.end > w.at;
}
// Next piece; false when the share is done.
__device__ __forceinline__ bool walk_next(const DecodeJob &j, Walk &w) {
  const int heads = j.c.n_kv_heads * j.row_tiles;
  do {
    if (w.left <= 0) return false;
    w.pair0 += w.n + kPairCost;
    if (++w.hr == heads) {
      w.hr = 0;
      do {
        if (++w.seq >= j.c.n_seqs) return false;
        w.n = seq_tiles(j, w.seq, &w.first);
      } while (w.n == 0);
    }
  } while (!walk_clip(w, 0));
  return true;
}

// A pair that several warps share.
struct SharedPair {
  int seq, hr;
  int wa, wb;      // the warps of this CTA that hold parts of it
  int cta0, cta1;  // the CTAs that hold tiles of it
};

// The part that warp w of this CTA holds of a pair: its last piece, in its ring, or, where the pair did not begin in w
// and w goes on with other pairs, its first piece, in the workspace.
template <int D>
__device__ __forceinline__ const float *warp_part(const DecodeJob &j, const SharedPair &sp, unsigned char *sm,
                                                  const int *in_heads, int w) {
  using C = DecodeCfg<D>;
  const bool began_here = w == sp.wa && sp.cta0 == (int)blockIdx.x;
  return !began_here && in_heads[w] ? j.part + ((size_t)blockIdx.x * (2 + C::kWarps) + 2 + w) * C::kPart
                                   : reinterpret_cast<const float *>(sm + (size_t)w * C::kStages * C::kTile);
}

// Weight of a part with reference r under the reference `top`, and its weight sum l under it.
__device__ __forceinline__ float part_weight(float r, float top) { return r == -a_inf() ? 0.f : a_exp2(r - top); }
// a poisoned part may hold no weight: its NaN must not be multiplied away
__device__ __forceinline__ float part_sum(float l, float w) { return l != l ? l : l * w; }
__device__ __forceinline__ float part_inverse(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }
__device__ __forceinline__ float part_lse(float r, float l) { return l == 0.f ? -a_inf() : (r + log2f(l)) * kLn2; }

// Element of the output's rows: query token and head of row rr of a pair.
__device__ __forceinline__ int64_t row_at(const DecodeJob &j, int seq, int hr, int rr) {
  if (j.q_tokens == 1 && j.row_tiles == 1) return (int64_t)seq * j.hq + hr * j.group + rr;  // the usual one, without divisions
  return ((int64_t)seq * j.q_tokens + rr / j.group) * j.hq + hr / j.row_tiles * j.group + rr % j.group;
}

// A pair whose tiles are all in this CTA, in some of its warps: merged by the one warp that is done last.
template <int D, typename T>
__device__ __noinline__ void merge_by_warp(const DecodeJob &j, const SharedPair &sp, unsigned char *sm,
                                           const int *in_heads) {
  using C = DecodeCfg<D>;
  constexpr int N = C::kOut / 128;  // accumulator words (of 4) per lane
  const int lane = threadIdx.x & 31, t = lane & 3;
  float top[2] = {-a_inf(), -a_inf()}, l[2] = {0.f, 0.f};
  for (int w = sp.wa; w <= sp.wb; ++w) {
    const float4 x = *reinterpret_cast<const float4 *>(warp_part<D>(j, sp, sm, in_heads, w) + C::kOut + 4 * t);
    top[0] = fmaxf(top[0], x.x);
    top[1] = fmaxf(top[1], x.y);
  }
  float4 a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int w = sp.wa; w <= sp.wb; ++w) {
    const float *p = warp_part<D>(j, sp, sm, in_heads, w);
    const float4 x = *reinterpret_cast<const float4 *>(p + C::kOut + 4 * t);
    const float w0 = part_weight(x.x, top[0]), w1 = part_weight(x.y, top[1]);
    l[0] += part_sum(x.z, w0);
    l[1] += part_sum(x.w, w1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(p + 4 * (32 * i + lane));
      a[i].x += v.x * w0;
      a[i].y += v.y * w1;
      a[i].z += v.z * w0;
      a[i].w += v.w * w1;
    }
  }
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const int rr = sp.hr % j.row_tiles * kRows + 2 * t + z;
    if (rr >= j.group * j.q_tokens) continue;
    const float inv = part_inverse(l[z]);
    const int64_t at = row_at(j, sp.seq, sp.hr, rr);
    T *o = static_cast<T *>(j.out) + at * D + 2 * (lane >> 2);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      store_pair(o + 16 * i, (z ? a[i].y : a[i].x) * inv, (z ? a[i + 1].y : a[i + 1].x) * inv);
      store_pair(o + 16 * i + 16, (z ? a[i].w : a[i].z) * inv, (z ? a[i + 1].w : a[i + 1].z) * inv);
    }
    if (lane < 4 && j.lse) j.lse[at] = part_lse(top[z], l[z]);
  }
}

// Pairs that the whole CTA merges once its warps are done, up to three: [0] one that warps of earlier CTAs hold tiles
// of too, [1] one that goes on in later CTAs (and began here), [2] one of this CTA alone that all its warps hold parts
// of.  The last CTA to be done with a pair merges the CTAs' results.
template <int D, typename T>
__device__ __noinline__ void merge_by_cta(const DecodeJob &j, const SharedPair *sps, const int *has, unsigned char *sm,
                                          const int *in_heads, int *is_last) {
  using C = DecodeCfg<D>;
  constexpr int W = C::kWarps, kThreads = 32 * W;
  const int tid = threadIdx.x, lane = tid & 31, t = lane & 3;
  auto result = [&](const SharedPair &sp, int f, const float4 v, const float r[2], const float l[2]) {
    const int dim = 32 * (f / 64) + 2 * (lane >> 2) + ((f >> 5) & 1);
#pragma unroll
    for (int z = 0; z < 2; ++z) {  // rows 2t and 2t + 1
      const int rr = sp.hr % j.row_tiles * kRows + 2 * t + z;
      if (rr >= j.group * j.q_tokens) continue;
      const int64_t at = row_at(j, sp.seq, sp.hr, rr);
      const float inv = part_inverse(l[z]);
      T *o = static_cast<T *>(j.out) + at * D + dim;
      o[0] = T((z ? v.y : v.x) * inv);
      o[16] = T((z ? v.w : v.z) * inv);
      if (f < 4 && j.lse) j.lse[at] = part_lse(r[z], l[z]);
    }
  };
#pragma unroll 1
  for (int x = 0; x < 3; ++x) {
    if (!has[x]) continue;
    const SharedPair &sp = sps[x];
    float *mine = j.part + ((size_t)blockIdx.x * (2 + W) + ((int)blockIdx.x == sp.cta0 ? 1 : 0)) * C::kPart;
    for (int f = tid; f < C::kOut / 4; f += kThreads) {
      // all parts asked for before the first is used
      float4 v[W], y[W];
      float r[2] = {-a_inf(), -a_inf()}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        y[w] = make_float4(-a_inf(), -a_inf(), 0.f, 0.f);
        v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w >= sp.wa && w <= sp.wb) {
          const float *p = warp_part<D>(j, sp, sm, in_heads, w);
          y[w] = *reinterpret_cast<const float4 *>(p + C::kOut + 4 * t);
          v[w] = *reinterpret_cast<const float4 *>(p + 4 * f);
        }
        r[0] = fmaxf(r[0], y[w].x);
        r[1] = fmaxf(r[1], y[w].y);
      }
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float w0 = part_weight(y[w].x, r[0]), w1 = part_weight(y[w].y, r[1]);
        l[0] += part_sum(y[w].z, w0);
        l[1] += part_sum(y[w].w, w1);
        a.x += v[w].x * w0;
        a.y += v[w].y * w1;
        a.z += v[w].z * w0;
        a.w += v[w].w * w1;
      }
      if (sp.cta0 == sp.cta1) {
        result(sp, f, a, r, l);
      } else {
        *reinterpret_cast<float4 *>(mine + 4 * f) = a;
        if (f < 4) *reinterpret_cast<float4 *>(mine + C::kOut + 4 * f) = make_float4(r[0], r[1], l[0], l[1]);
      }
    }
  }
  const bool shared0 = has[0] && sps[0].cta0 != sps[0].cta1, shared1 = has[1] && sps[1].cta0 != sps[1].cta1;
  if (!shared0 && !shared1) return;
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    const bool mine = tid ? shared1 : shared0;
    const SharedPair &sp = sps[tid];
    is_last[tid] = mine && atomicAdd(j.count + sp.cta0, 1u) == (uint32_t)(sp.cta1 - sp.cta0);
    if (is_last[tid]) j.count[sp.cta0] = 0;
  }
  __syncthreads();
  __threadfence();
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    if (!is_last[x]) continue;
    const SharedPair &sp = sps[x];
    const int ctas = sp.cta1 - sp.cta0 + 1;
    auto part = [&](int k) { return j.part + ((size_t)(sp.cta0 + k) * (2 + W) + (k == 0 ? 1 : 0)) * C::kPart; };
    for (int f = tid; f < C::kOut / 4; f += kThreads) {
      // eight parts at a time, all asked for before the first is used: each takes a trip to the L2
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float top[2] = {-a_inf(), -a_inf()}, l[2] = {0.f, 0.f};
#pragma unroll 1
      for (int k0 = 0; k0 < ctas; k0 += 8) {
        float4 v[8], y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float *p = part(min(k0 + k, ctas - 1));
          y[k] = __ldcg(reinterpret_cast<const float4 *>(p + C::kOut + 4 * t));
          v[k] = __ldcg(reinterpret_cast<const float4 *>(p + 4 * f));
          if (k0 + k >= ctas) y[k] = make_float4(-a_inf(), -a_inf(), 0.f, 0.f);
        }
        float n0 = top[0], n1 = top[1];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          n0 = fmaxf(n0, y[k].x);
          n1 = fmaxf(n1, y[k].y);
        }
        const float s0 = part_weight(top[0], n0), s1 = part_weight(top[1], n1);
        top[0] = n0;
        top[1] = n1;
        a.x *= s0;
        a.y *= s1;
        a.z *= s0;
        a.w *= s1;
        l[0] *= s0;
        l[1] *= s1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float w0 = part_weight(y[k].x, n0), w1 = part_weight(y[k].y, n1);
          l[0] += part_sum(y[k].z, w0);
          l[1] += part_sum(y[k].w, w1);
          a.x += v[k].x * w0;
          a.y += v[k].y * w1;
          a.z += v[k].z * w0;
          a.w += v[k].w * w1;
        }
      }
      result(sp, f, a, top, l);
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(32 * DecodeCfg<D>::kWarps, DecodeCfg<D>::kCtas) kv_attention_kernel(const DecodeJob j) {
  using C = DecodeCfg<D>;
  constexpr int W = C::kWarps, S = C::kStages, NB = D / 32;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t bars[W][S];
  __shared__ SharedPair cta_pairs[3];  // pairs that the whole CTA merges
  __shared__ int has_pair[3], sh_last[2];
  __shared__ int parts_done[W];     // per pair that only warps of this CTA share, by its first warp
  __shared__ int in_heads[W];       // per warp: its first piece is a part in the workspace
  __shared__ Walk walks[W][2];      // per warp: the piece that it computes, and the one that its copies are at
  __shared__ int load_tile[W];      // per warp: the first tile of that piece whose page is not looked up yet
  __shared__ int no_page[W][8];     // per warp and piece (its number & 7; copies run at most 4 pieces ahead): a tile has no page
  float *heads_mem = j.part + ((size_t)blockIdx.x * (2 + W) + 2) * C::kPart;
  uint4 *q_mem = reinterpret_cast<uint4 *>(sm + C::kRing + (size_t)(threadIdx.x >> 5) * C::kQuery);  // [NB][32]
  float4 *q_start = reinterpret_cast<float4 *>(q_mem + D);                                          // [NB][4]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int heads = j.c.n_kv_heads * j.row_tiles;
  const int64_t n_rows_all = (int64_t)j.q_tokens * j.hq;
  const int n_rows = j.group * j.q_tokens;
  uint64_t *bar = bars[warp];
  unsigned char *ring = sm + (size_t)warp * S * C::kTile;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) a_mbar_init(&bar[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    parts_done[warp] = in_heads[warp] = 0;
    if (warp == 0) has_pair[0] = has_pair[1] = has_pair[2] = 0;
  }
  __syncthreads();

  // ---- this warp's share of the places: a lane counts `per` consecutive sequences
  const int per = (j.c.n_seqs + 31) / 32;
  int64_t total = 0;
  int most = 0;
  bool some_empty = false;
#pragma unroll 4
  for (int k = 0; k < per; ++k) {
    const int s = lane * per + k;
    int first, n = 0;
    if (s < j.c.n_seqs) n = seq_tiles(j, s, &first);
    some_empty |= s < j.c.n_seqs && n == 0;
    total += n ? n + kPairCost : 0;
    most = max(most, n);
  }
  // sequences without tiles (empty, or of a length that the table cannot hold): their rows
  if (__any_sync(0xffffffffu, some_empty))
    for (int s = warp * gridDim.x + blockIdx.x; s < j.c.n_seqs; s += gridDim.x * W) {
      int first;
      if (seq_tiles(j, s, &first) > 0) continue;
      const bool bad = __ldg(j.lens + s) != 0;
      if (bad && lane == 0 && j.c.status) atomicOr(j.c.status, MOE_KV_BAD_LENGTH);
      const float fill = bad ? a_nan() : 0.f;
      T *o = static_cast<T *>(j.out) + (int64_t)s * n_rows_all * D;
      for (int64_t i = lane; i < n_rows_all * D / 2; i += 32) store_pair(o + 2 * i, fill, fill);
      if (j.lse)
        for (int64_t i = lane; i < n_rows_all; i += 32) j.lse[(int64_t)s * n_rows_all + i] = bad ? a_nan() : -a_inf();
    }
  const int64_t mine = total * heads;
  int64_t before = mine;  // sums over the lanes before, in places
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  const int64_t pairs = (int64_t)j.c.n_seqs * heads;
  const int64_t share = kv_div(total + (int64_t)gridDim.x * W - 1, (int64_t)gridDim.x * W);
  const bool alone = pairs <= (int64_t)gridDim.x && most <= W * (share + kAloneMore);  // a CTA per pair
  Walk walk = {0, 0, 0, 0, 0, 0, 0, 0};
  bool work;
  if (alone) {
    work = blockIdx.x < pairs;
    if (work) {
      walk.seq = blockIdx.x / heads;
      walk.hr = blockIdx.x % heads;
      walk.n = seq_tiles(j, walk.seq, &walk.first);
      const int n = max(walk.n, W);  // fewer tiles than warps: one each
      walk.at = min(n * warp / W, walk.n);
      walk.end = min(n * (warp + 1) / W, walk.n);
      work = walk.end > walk.at;
    }
  } else {
    const int64_t u0 = share * ((int64_t)blockIdx.x * W + warp);
    work = u0 < total;
    if (work) {
      const int src = __ffs(__ballot_sync(0xffffffffu, u0 >= before && u0 < before + mine)) - 1;
      int64_t run = __shfl_sync(0xffffffffu, before, src);
      for (int base = 0; base < per; base += 32) {
        const int k = base + lane, s = src * per + k;
        int first = 0, n = 0;
        if (k < per && s < j.c.n_seqs) n = seq_tiles(j, s, &first);
        const int64_t cost = n ? (int64_t)(n + kPairCost) * heads : 0;
        int64_t inc = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const int64_t begin = run + inc - cost;
        const uint32_t who = __ballot_sync(0xffffffffu, u0 >= begin && u0 < begin + cost);
        run += __shfl_sync(0xffffffffu, inc, 31);
        if (who) {
          const int at = __ffs(who) - 1;
          walk.seq = src * per + base + at;
          walk.n = __shfl_sync(0xffffffffu, n, at);
          walk.first = __shfl_sync(0xffffffffu, first, at);
          walk.pair0 = __shfl_sync(0xffffffffu, begin, at);
          break;
        }
      }
      walk.hr = (int)kv_div(u0 - walk.pair0, walk.n + kPairCost);
      walk.pair0 += (int64_t)walk.hr * (walk.n + kPairCost);
      walk.left = min(share, total - u0);
      work = walk_clip(walk, u0 - walk.pair0) || walk_next(j, walk);
    }
  }
  // ---- the rows' queries, as they are: lane (g, t) holds row g's values 4t.. of each half block.  Asked for before
  // the copies, behind which they would queue.
  uint2 raw[NB][2];
  auto load_q = [&](const Walk &w) {
    const int kvh = w.hr / j.row_tiles, r = w.hr % j.row_tiles * kRows + g;
#pragma unroll
    for (int b = 0; b < NB; ++b) raw[b][0] = raw[b][1] = make_uint2(0u, 0u);
    if (r < n_rows) {
      const T *src = static_cast<const T *>(j.q.data) + ((int64_t)w.seq * j.q_tokens + r / j.group) * j.q.token_stride +
                     (int64_t)(kvh * j.group + r % j.group) * j.q.head_stride;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          raw[b][half] = *reinterpret_cast<const uint2 *>(src + 32 * b + 16 * half + 4 * t);
    }
  };
  if (work) load_q(walk);

  // ---- this warp's copies: a second walk that runs up to S tiles ahead.  The walks live in shared memory: they
  // change once per piece, and registers are what bounds the tile's code.
  if (lane == 0) {
    walks[warp][0] = walks[warp][1] = walk;
    load_tile[warp] = walk.at;
    no_page[warp][0] = 0;
  }
  __syncwarp();
  TileRing<S> tiles_on_way;
  int64_t src_off = -1;         // per lane: where one of the next tiles is in the cache, -1: the tile has no page
  int src_next = 0, src_n = 0;  // next lane's turn, and lanes in use
  uint32_t load_piece = 0;      // number of the copies' piece; ~0: no more

  auto refill = [&]() {
    if (load_piece == ~0u) return;
    Walk w = walks[warp][1];
    int tile = load_tile[warp];
    __syncwarp();
    if (tile >= w.end) {
      if (!walk_next(j, w)) {
        load_piece = ~0u;
        return;
      }
      ++load_piece;
      tile = w.at;
      if (lane == 0) {
        walks[warp][1] = w;
        no_page[warp][load_piece & 7] = 0;
      }
    }
    src_next = 0;
    src_n = min(32, w.end - tile);
    src_off = -1;
    if (lane < src_n) {
      int in_page = 0;
      const int p = kv_page(j.c.page_table + (int64_t)w.seq * j.c.table_stride, j.c.table_width, j.c.n_pages,
                            j.c.page_size, w.first + tile + lane, &in_page);
      if (p >= 0)
        src_off = (int64_t)p * j.c.page_stride + kv_tile_off(D, j.c.page_size, w.hr / j.row_tiles, in_page);
    }
    const bool missing = __any_sync(0xffffffffu, lane < src_n && src_off < 0);
    if (lane == 0) {
      load_tile[warp] = tile + src_n;
      if (missing) no_page[warp][load_piece & 7] = 1;
    }
    __syncwarp();
  };
  // Copies the share's tile x, if there is one, into its stage.
  auto issue = [&](uint32_t x) {
    if (tiles_on_way.dead) return;
    if (src_next == src_n) {
      src_next = src_n = 0;
      refill();
      if (src_n == 0) return;
    }
    const int64_t off = __shfl_sync(0xffffffffu, src_off, src_next++);
    if (lane == 0) {
      uint64_t *b = bar + x % S;
      if (off < 0) {
        a_mbar_arrive(b);
      } else {
        a_expect_tx(b, C::kTile);
        a_bulk_load(ring + (x % S) * C::kTile, static_cast<const uint8_t *>(j.c.pages) + off, C::kTile, b);
      }
    }
  };
  if (work)
#pragma unroll 1
    for (int x = 0; x < S; ++x) issue(x);

  // -8 2^-20 as fp16 pairs.  Four registers that the compiler cannot see through: it would build the operand anew, move
  // by move, for every instruction.
  uint32_t eight[4];
  asm volatile("mov.b32 %0, 0x80808080;\n mov.b32 %1, 0x80808080;\n mov.b32 %2, 0x80808080;\n mov.b32 %3, 0x80808080;"
               : "=r"(eight[0]), "=r"(eight[1]), "=r"(eight[2]), "=r"(eight[3]));

  for (uint32_t piece = 0; work; ++piece) {
    __syncwarp();
    const Walk &walk = walks[warp][0];
    const int kvh = walk.hr / j.row_tiles, rt = walk.hr % j.row_tiles;
    const int len = __ldg(j.lens + walk.seq);
    // ---- the rows' queries as matrix operands
    float f[2];
    bool big;
    int w0, w1;  // tiles [w0, w1) of the piece are seen whole by every row
    {
      float top = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int z = 0; z < 8; ++z)
          top = fmaxf(top, fabsf(to_float(reinterpret_cast<const T *>(&raw[b][z / 4])[z % 4])));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e with the row's largest value below 2^13 after it (an infinity or NaN stays what it is)
      int e = 12;
      if (top > 0.f && top < a_inf()) e = 12 - ((int)((__float_as_uint(top) >> 23) & 255) - 127);
      e = min(max(e, -120), 120);
      const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float sum = 0.f;
        __half h[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          // high nibbles are 2^4 too large as fp16: their query values are 2^-4
          h[z] = __float2half_rn(to_float(reinterpret_cast<const T *>(&raw[b][z / 4])[z % 4]) * up *
                                 (z < 4 ? 1.f : 0.0625f));
          sum += __half2float(h[z]) * (z < 4 ? 1.f : 16.f);
        }
        q_mem[b * 32 + lane] = make_uint4(h2_bits(__halves2half2(h[0], h[2])), h2_bits(__halves2half2(h[1], h[3])),
                                          h2_bits(__halves2half2(h[4], h[6])), h2_bits(__halves2half2(h[5], h[7])));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.f * 5.9604644775390625e-08f;  // -8 x 2^-24
        const float s0 = __shfl_sync(0xffffffffu, sum, 8 * t), s1 = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
        if (g == 0) q_start[b * 4 + t] = make_float4(s0, s1, s0, s1);
      }
      __syncwarp();
      // The score's factor, scale log2(e) 2^(24 - e).  Where it is past what fp32 holds (queries of 2^100 and more), 2^80
      // of it go ahead into the scores, which are below 2^20.  (0 times the -inf of what is not seen would be NaN.)
      const float to_log2 = j.scale * kLog2e;
      big = __any_sync(0xffffffffu, to_log2 * down * 16777216.f > 1e30f);
      const float mine_f = fminf(fmaxf(big ? to_log2 * (down * kEarly) : to_log2 * down * 16777216.f, 1.17549435e-38f), 3.4e38f);
#pragma unroll
      for (int z = 0; z < 2; ++z) f[z] = __shfl_sync(0xffffffffu, mine_f, 8 * t + 4 * z);
      int64_t a, b, lo, hi;
      kv_visible(len, j.q_tokens, (min(n_rows, (rt + 1) * kRows) - 1) / j.group, j.window, &lo, &b);
      kv_visible(len, j.q_tokens, rt * kRows / j.group, j.window, &a, &hi);
      w0 = min(max((int)((lo + kKvTile - 1) / kKvTile) - walk.first, walk.at), walk.end);
      w1 = min(max((int)(hi / kKvTile) - walk.first, w0), walk.end);
    }
    // ---- this warp's tiles of the piece
    float acc[NB][2][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[b][h][z] = 0.f;
    float ref[2] = {kNone, kNone}, l[2] = {0.f, 0.f};  // references (log2 units) and sums of the weights

    // One tile.  Whole: every row sees all of it.
    auto compute = [&](const unsigned char *tp, const int tok0, auto is_whole) {
      constexpr bool whole = decltype(is_whole)::value;
      // key k of the matrix (of 8) is token perm(k) = k / 2 + 4 (k odd), so that the value operand's
      // pairs (2t, 2t + 1) are tokens t and t + 4 and a load covers neighbouring tokens
      const int pg = (g >> 1) + ((g & 1) << 2);
      float s[2][4];
      __half2 kd[2][2][NB / 2];  // key scales of tokens 16 mt + pg and 8 more
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned char *sa = tp + 16 * D + (8 * x + pg) * (D / 16);
        if constexpr (NB == 2) {
          kd[x / 2][x % 2][0] = *reinterpret_cast<const __half2 *>(sa);
        } else {
#pragma unroll
          for (int z = 0; z < NB / 4; ++z)
            *reinterpret_cast<uint2 *>(&kd[x / 2][x % 2][2 * z]) = *reinterpret_cast<const uint2 *>(sa + 8 * z);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float c[2][4];
        const uint4 qf = q_mem[b * 32 + lane];
        const float4 start = q_start[b * 4 + t];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const unsigned char *kp = tp + (b * 32 + mt * 16 + pg) * 16 + 4 * t;
          const uint32_t wa = *reinterpret_cast<const uint32_t *>(kp), wb = *reinterpret_cast<const uint32_t *>(kp + 128);
          const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
          mma16816_from(c[mt], wa & 0x000F000Fu, wb & 0x000F000Fu, wa8 & 0x000F000Fu, wb8 & 0x000F000Fu, qf.x, qf.y,
                        start.x, start.y, start.z, start.w);
          mma16816(c[mt], wa & 0x00F000F0u, wb & 0x00F000F0u, wa8 & 0x00F000F0u, wb8 & 0x00F000F0u, qf.z, qf.w);
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float fa = (b & 1) ? __high2float(kd[mt][0][b / 2]) : __low2float(kd[mt][0][b / 2]);
          const float fb = (b & 1) ? __high2float(kd[mt][1][b / 2]) : __low2float(kd[mt][1][b / 2]);
          s[mt][0] = b ? fmaf(c[mt][0], fa, s[mt][0]) : c[mt][0] * fa;
          s[mt][1] = b ? fmaf(c[mt][1], fa, s[mt][1]) : c[mt][1] * fa;
          s[mt][2] = b ? fmaf(c[mt][2], fb, s[mt][2]) : c[mt][2] * fb;
          s[mt][3] = b ? fmaf(c[mt][3], fb, s[mt][3]) : c[mt][3] * fb;
        }
      }
      if (big)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[0][x] *= 16777216.f / kEarly;
          s[1][x] *= 16777216.f / kEarly;
        }
      // ---- what a row does not see scores -inf
      uint32_t seen[4];  // of tokens 8 x + pg: all bits of the halves of the rows that see it
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 4; ++x) seen[x] = 0;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int rr = rt * kRows + 2 * t + z;
          int64_t lo = 0, hi = 0;
          if (rr < n_rows) kv_visible(len, j.q_tokens, rr / j.group, j.window, &lo, &hi);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = tok0 + 8 * x + pg;
            if (key < lo || key >= hi) s[x / 2][2 * (x % 2) + z] = -a_inf();
            else seen[x] |= z ? 0xffff0000u : 0xffffu;
          }
        }
      }
      // ---- the value scales of the lane's tokens, and the largest of them (NaN as none)
      const unsigned char *vs = tp + 34 * D + pg * (D / 16);
      __half2 vd[4][NB / 2];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if constexpr (NB == 2) {
          vd[x][0] = *reinterpret_cast<const __half2 *>(vs + 8 * x * (D / 16));
        } else {
#pragma unroll
          for (int z = 0; z < NB / 4; ++z)
            *reinterpret_cast<uint2 *>(&vd[x][2 * z]) = *reinterpret_cast<const uint2 *>(vs + 8 * x * (D / 16) + 8 * z);
        }
      }
      auto largest = [&](int x) {
        __half2 m = __habs2(vd[x][0]);
#pragma unroll
        for (int z = 1; z < NB / 2; ++z) m = __hmax2(m, __habs2(vd[x][z]));
        return m;
      };
      // ---- weights.  (The score is rounded before the reference is taken away, as it was when the reference was set: of
      // scores so large that their rounding is more than a weight can bear, the largest has a weight of its own size.)
      float p[4][2];
      uint64_t sum;
      auto weigh = [&]() {
        const uint64_t f2 = f2_pack(f[0], f[1]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // (the sums one by one: of packed pairs a product and the sum after it come out fused)
          float a, b;
          f2_unpack(f2_mul(f2_pack(s[x / 2][2 * (x % 2)], s[x / 2][2 * (x % 2) + 1]), f2), a, b);
          p[x][0] = a_exp2(__fadd_rn(a, -ref[0]));
          p[x][1] = a_exp2(__fadd_rn(b, -ref[1]));
          sum = x ? f2_add(sum, f2_pack(p[x][0], p[x][1])) : f2_pack(p[x][0], p[x][1]);
        }
      };
      weigh();
      // The lane's weights times its largest scale bound its products.  Where that is too much, each row's own products
      // say whether its reference moves, so that nothing that a row does not see takes part in that.
      {
        const __half2 d2 = __hmax2(__hmax2(largest(0), largest(1)), __hmax2(largest(2), largest(3)));
        float sum0, sum1;
        f2_unpack(sum, sum0, sum1);
        const float most = fmaxf(sum0, sum1);
        if (__any_sync(0xffffffffu, most * fmaxf(__low2float(d2), __high2float(d2)) > kMost || most > kDeepMost)) {
          float pd[2] = {0.f, 0.f}, pm[2] = {0.f, 0.f}, td[2] = {-a_inf(), -a_inf()}, tm[2] = {-a_inf(), -a_inf()};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const __half2 m = largest(x);
            const float d = fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);
            const float lg = __log2f(d);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float sc = __fmul_rn(s[x / 2][2 * (x % 2) + z], f[z]);
              pd[z] = fmaxf(pd[z], p[x][z] * d);
              pm[z] = fmaxf(pm[z], p[x][z]);
              td[z] = fmaxf(td[z], __fadd_ru(sc, lg));
              tm[z] = fmaxf(tm[z], sc);
            }
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              pd[z] = fmaxf(pd[z], __shfl_xor_sync(0xffffffffu, pd[z], o));
              pm[z] = fmaxf(pm[z], __shfl_xor_sync(0xffffffffu, pm[z], o));
              td[z] = fmaxf(td[z], __shfl_xor_sync(0xffffffffu, td[z], o));
              tm[z] = fmaxf(tm[z], __shfl_xor_sync(0xffffffffu, tm[z], o));
            }
            if (pd[z] > kMost || pm[z] > kDeepMost) {
              const float to = fmaxf(ref[z], fmaxf(__fadd_ru(td[z], -kCentre), __fadd_ru(tm[z], -kDeep)));
              const float a = a_exp2(ref[z] - to);
              ref[z] = to;
              l[z] *= a;
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  acc[b][h][z] *= a;
                  acc[b][h][z + 2] *= a;
                }
            }
          }
          weigh();
        }
      }
      {
        float sum0, sum1;
        f2_unpack(sum, sum0, sum1);
        l[0] += sum0;
        l[1] += sum1;
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int k0 = mt * 16 + t;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          // weights times scales, rounded once; row g's of tokens t, t + 4 and t + 8, t + 12 (an 8x8 transpose each)
          uint32_t e[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int x = 2 * mt + y;
            const float d = (b & 1) ? __high2float(vd[x][b / 2]) : __low2float(vd[x][b / 2]);
            uint32_t h = h2_bits(__floats2half2_rn(p[x][0] * d, p[x][1] * d));
            if (!whole) h &= seen[x];  // (a weight of 0 times a scale that is not finite is none)
            e[y] = transpose8x8(h);
          }
          const unsigned char *cp = tp + 18 * D + (b * 32 + k0) * 16 + 2 * g;
          const uint32_t v0 = *reinterpret_cast<const uint16_t *>(cp), v1 = *reinterpret_cast<const uint16_t *>(cp + 64);
          const uint32_t v2 = *reinterpret_cast<const uint16_t *>(cp + 128),
                         v3 = *reinterpret_cast<const uint16_t *>(cp + 192);
          const uint32_t x = __byte_perm(v0, v1, 0x5410u), y = __byte_perm(v2, v3, 0x5410u);
          // All codes go to bits 4 to 7: of an operand below the normal numbers the product is added by the exponent of
          // the least normal one.  With the low nibbles left in bits 0 to 3 whatever is below 2^-18 of 8 w d was cut off
          // the sums (so 2^-22; 128 sequences 131 and 134 us).
          mma16816(acc[b][0], (x << 4) & 0x00F000F0u, x & 0x00F000F0u, (y << 4) & 0x00F000F0u, y & 0x00F000F0u, e[0], e[1]);
          mma16816(acc[b][1], (x >> 4) & 0x00F000F0u, (x >> 8) & 0x00F000F0u, (y >> 4) & 0x00F000F0u,
                   (y >> 8) & 0x00F000F0u, e[0], e[1]);
          mma16816(acc[b][0], eight[0], eight[1], eight[2], eight[3], e[0], e[1]);
          mma16816(acc[b][1], eight[0], eight[1], eight[2], eight[3], e[0], e[1]);
        }
      }
    };
    auto tiles = [&](int from, int to, auto is_whole) {
#pragma unroll 1
      for (int tile = from; tile < to; ++tile) {
        const uint32_t x = tiles_on_way.used;
        tiles_on_way.take(
            [&](uint32_t y) { return __all_sync(0xffffffffu, a_mbar_try(&bar[y % S], TileRing<S>::parity(y))) != 0; },
            [&](uint32_t y) { return __all_sync(0xffffffffu, wait_for_tile(&bar[y % S], TileRing<S>::parity(y))) != 0; });
        // (a tile that never came is computed on as it lies there: the result is NaN)
        compute(ring + (x % S) * C::kTile, (walk.first + tile) * kKvTile, is_whole);
        __syncwarp();
        issue(x + S);
      }
    };
    // tiles that some row sees in part, tiles that all rows see whole, and again those in part
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      tiles(pass ? w1 : walk.at, pass ? walk.end : w0, std::false_type());
      if (pass == 0) tiles(w0, w1, std::true_type());
    }
    // ---- the piece: l over the lanes that share a row; accumulators without the codes' factor
    int poison = 0;  // status bits: what the piece's result is worth
    if (no_page[warp][piece & 7]) poison |= MOE_KV_BAD_PAGE;
    if (tiles_on_way.dead) poison |= MOE_KV_TIMED_OUT;
    if (poison) {
      l[0] = l[1] = a_nan();
      if (lane == 0 && j.c.status) atomicOr(j.c.status, poison);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    float r[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) r[z] = ref[z] == kNone ? -a_inf() : ref[z];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[b][h][z] *= 1048576.f;
    Walk next = walk;
    const bool more = walk_next(j, next);
    if (more) load_q(next);
    if (walk.at == 0 && walk.end == walk.n) {
      // all of the pair: its result
      const int64_t tok = (int64_t)walk.seq * j.q_tokens;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int rr = rt * kRows + 2 * t + z;
        if (rr >= n_rows) continue;
        const float inv = l[z] > 0.f || l[z] != l[z] ? 1.f / l[z] : 0.f;
        const int64_t at = (tok + rr / j.group) * j.hq + kvh * j.group + rr % j.group;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            store_pair(static_cast<T *>(j.out) + at * D + 32 * b + 16 * half + 2 * g, acc[b][0][z + 2 * half] * inv,
                       acc[b][1][z + 2 * half] * inv);
        if (g == 0 && j.lse) j.lse[at] = l[z] == 0.f ? -a_inf() : (r[z] + log2f(l[z])) * kLn2;
      }
    } else {
      // a part: a last piece waits in the ring (no copy is on its way by then), a first one that others follow
      // in the workspace
      float *o = more ? heads_mem + (size_t)warp * C::kPart : reinterpret_cast<float *>(ring);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4 *>(o + ((b * 2 + h) * 32 + lane) * 4) =
              make_float4(acc[b][h][0], acc[b][h][1], acc[b][h][2], acc[b][h][3]);
      if (g == 0) *reinterpret_cast<float4 *>(o + C::kOut + 4 * t) = make_float4(r[0], r[1], l[0], l[1]);
      if (more && lane == 0) in_heads[warp] = 1;
      SharedPair sp = {walk.seq, walk.hr, 0, min(W, walk.n) - 1, (int)blockIdx.x, (int)blockIdx.x};
      bool begun = false, goes_on = false;  // tiles of the pair in an earlier CTA, in a later one
      if (!alone) {
        // warps of the grid that hold the pair's first and last tiles
        const int64_t g0 = kv_div(walk.pair0 + kPairCost, share), g1 = kv_div(walk.pair0 + kPairCost + walk.n - 1, share);
        sp.cta0 = (int)(g0 / W);
        sp.cta1 = (int)(g1 / W);
        begun = sp.cta0 < (int)blockIdx.x;
        goes_on = sp.cta1 > (int)blockIdx.x;
        sp.wa = begun ? 0 : (int)(g0 % W);
        sp.wb = goes_on ? W - 1 : (int)(g1 % W);
      }
      if (begun || goes_on || sp.wb - sp.wa == W - 1) {
        const int x = begun ? 0 : goes_on ? 1 : 2;
        if (lane == 0) {
          cta_pairs[x] = sp;
          has_pair[x] = 1;
        }
      } else {
        __threadfence_block();
        __syncwarp();
        int last = 0;
        if (lane == 0) last = atomicAdd(&parts_done[sp.wa], 1) == sp.wb - sp.wa;
        last = __shfl_sync(0xffffffffu, last, 0);
        __threadfence_block();
        if (last) merge_by_warp<D, T>(j, sp, sm, in_heads);
      }
    }
    work = more;
    __syncwarp();
    if (lane == 0) walks[warp][0] = next;
  }
  __syncthreads();
  if (has_pair[0] || has_pair[1] || has_pair[2])
    merge_by_cta<D, T>(j, cta_pairs, has_pair, sm, in_heads, sh_last);
}

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

constexpr int64_t kCountBytes = MOE_KV_COUNTER_BYTES;  // counters at the head of the workspace
static_assert(kDecodeCtasMost * 4 <= kCountBytes, "a counter per CTA");

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int64_t moe_kv_attention_workspace(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t q_tokens) {
  if (n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || q_tokens <= 0 || !kv_sizes_ok(n_kv_heads, head_dim, 32))
    return 0;
  return kCountBytes + (int64_t)decode_grid_cap(head_dim) * (2 + kDecodeWarps) * (kRows * head_dim + 16) * 4;
}

MOE_API int moe_kv_attention(const moe_kv_cache *c, const int32_t *seq_lens, const moe_tensor *q, int32_t n_q_heads,
                             int32_t q_tokens, float scale, int32_t window, void *out, float *lse, int32_t dtype,
                             void *workspace, int64_t workspace_bytes, void *cuda_stream) {
  if (c && c->n_seqs == 0) return MOE_OK;
  if (const int rc = check_cache(c)) return rc;
  if (!seq_lens || !out || n_q_heads <= 0 || n_q_heads % c->n_kv_heads || q_tokens <= 0 || window < 0 ||
      !(scale > 0.f && scale <= kMostScale))
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
  // no more CTAs than there are tiles for their warps, unless pairs can have one each
  const int64_t pairs = (int64_t)c->n_seqs * c->n_kv_heads * j.row_tiles;
  const int64_t tiles = pairs * std::max<int64_t>(1, (int64_t)c->table_width * (c->page_size / kKvTile));
  const int64_t most = std::max<int64_t>(pairs, (tiles + 7) / 8);
  const int grid = (int)std::min<int64_t>(most, decode_grid_cap(c->head_dim));
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const int D = c->head_dim;
  if (dtype == MOE_BF16)
    return D == 64 ? launch_decode<64, __nv_bfloat16>(j, grid, st)
                   : D == 128 ? launch_decode<128, __nv_bfloat16>(j, grid, st) : launch_decode<256, __nv_bfloat16>(j, grid, st);
  return D == 64 ? launch_decode<64, __half>(j, grid, st)
                 : D == 128 ? launch_decode<128, __half>(j, grid, st) : launch_decode<256, __half>(j, grid, st);
}
