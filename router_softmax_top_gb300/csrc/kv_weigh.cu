// The attention weight that cached tokens receive from a few query tokens per sequence.
//
// total[key] (+)= sum over the rows that see it of exp(scale q . k - lse), the rows being the
// query tokens of the heads that share the key head, lse what attention gave beside its
// result: no maximum, no sum over keys, so tiles of keys have nothing to do with each other.
//
// Bound: the key half of the cache (18 D bytes per tile of 32 tokens and head), and the
// totals, read and written; in fact instructions: about 470 per tile of 128 wide heads, an SM
// issuing 70% of the time.  By the source 144 of them unpack codes (9 per 8), some 120 are
// products, scales and weights, of which four rows per key head leave half the columns
// empty, and the rest the ring, waits, addresses and branches.  The 32-token tiles of all
// (sequence, key head) pairs in a row, plus a few tiles' worth per pair for its set-up, are
// split evenly over all warps; a warp copies its own tiles (the key half of a tile is
// contiguous: one bulk copy) into a ring of its own, two to four ahead, and no barrier stands
// in the loop.
//  * Scores: K Q^T (m16n8k16), codes as the whole numbers q - 8 in fp16 (high nibbles times 16,
//    which the query's share takes back): a nibble under the exponent of 1024 is one operation
//    and one packed addition away from it.  The query is rounded to fp16 after a power-of-two
//    scaling per row (exact for bf16 and fp16 inputs down to 2^-23 of the row's largest value,
//    what is smaller to 2^-34 of that); products are exact, sums fp32.
//  * The score less lse is formed before the factor log2(e): of large weights, whose
//    difference is small, only the score's own rounding is left.
//  * Sums over rows stay in registers, then among the four lanes that share a token; the
//    lane that writes a token's total is the one that reads it, whatever the pass.
// Measured, 32 heads of 128 on 8: 128 sequences of 64 to 8192 tokens 78 us (4.4 TB/s of what
// it has to read and write; loads into registers instead of the rings 91), one of 131071
// 25 us (31), one of 333 5.6 us.  32 sequences of 64 to 8192 tokens, 4 query tokens, 32 heads on
// 4 of 128 (32 rows a key head: four row tiles, 238 registers, one CTA per SM): 31 us.
#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"

namespace moe {
namespace {

constexpr int kWeighWarps = 8;
constexpr int kWeighSms = 152;
constexpr int64_t kMostTokens = 1 << 30;  // that a row of the page table may hold
// What a pair costs beside its tiles, in tiles (its queries, lse and page numbers are about as many instructions).  With 0, 2
// and 4: 128 sequences of up to 8192 tokens 84, 77 and 79 us, of up to 200 12.3, 11.0 and 12.3; 32 of up to 8192 on 4 heads of
// 256 26, 22 and 23, on 4 of 128 with 32 rows a head 53, 31 and 29.
constexpr int kWeighPairCost = 2;

struct WeighJob {
  moe_kv_cache c;
  const int32_t *lens;
  moe_tensor q;
  const float *lse;
  float *totals;
  int hq, group, q_tokens, window, restart;
  float scale;
};

template <int D, int RT>
struct WeighCfg {
  static constexpr int NB = D / 32;
  // Of a warp's ring: what is on its way per SM is then 48 to 110 KB, 44 KB at the full rate and a microsecond's latency.
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kTile = 18 * D;                                   // bytes of a tile's keys and their scales
  static constexpr int kQuery = RT * NB * 32 * 16;                       // bytes of a warp's query operand
  static constexpr int kWarp = kStages * kTile + kQuery;
  static constexpr size_t kSmem = (size_t)kWeighWarps * kWarp;
  // per SM, by registers (24, 16 or 8 warps) and shared memory
  static constexpr int kCtas = RT == 1 ? (D == 256 ? 2 : 3) : RT == 2 ? (D == 256 ? 1 : 2) : 1;
  static_assert(kCtas * (kSmem + 2048) <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float w_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float w_float(__half x) { return __half2float(x); }
__device__ __forceinline__ uint32_t w_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
// (not volatile: the compiler may hoist it over the arithmetic before it)
__device__ __forceinline__ void w_mma(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void w_mma_first(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Codes of bytes 0 and 2 under the exponent of 1024 (magic: 0x64006400, in a register that the compiler cannot see
// through: it would split the operation for two constants), less 1032: q - 8 of low nibbles, exactly; 16 (q - 8) of high
// ones, less 1152.
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(x) : "r"(w), "r"(magic));
  return w_bits(__hadd2(*reinterpret_cast<const __half2 *>(&x), __floats2half2_rn(-1032.f, -1032.f)));
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(x) : "r"(w), "r"(magic));
  return w_bits(__hadd2(*reinterpret_cast<const __half2 *>(&x), __floats2half2_rn(-1152.f, -1152.f)));
}

// Tiles of sequence s that the call has to do with; the first of them.  0 for a length that makes no sense.
__device__ __forceinline__ int weigh_tiles(const WeighJob &j, int s, int *first, bool *bad) {
  int64_t f;
  const int len = __ldg(j.lens + s);
  int64_t n = kv_tiles(len, j.q_tokens, j.window, j.c.table_width, j.c.page_size, &f);
  *bad = n < 0;
  if (n >= 0 && j.restart) {
    n += f;
    f = 0;
  }
  *first = (int)f;
  return n < 0 ? 0 : (int)n;
}

// (out of line: a copy is nearly always there)
__device__ __noinline__ bool w_wait(uint64_t *bar, uint32_t parity) { return a_mbar_wait(bar, parity); }

template <int D, int RT, typename T>
__global__ void __launch_bounds__(32 * kWeighWarps, WeighCfg<D, RT>::kCtas) kv_weigh_kernel(const WeighJob j) {
  using C = WeighCfg<D, RT>;
  constexpr int NB = C::NB, W = kWeighWarps, S = C::kStages;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t bars[W][S];
  __shared__ int64_t totals_at[W][S];  // index of a stage's tile's totals, -1: it has no page
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  unsigned char *ring = sm + (size_t)warp * C::kWarp;
  uint4 *q_mem = reinterpret_cast<uint4 *>(ring + S * C::kTile);  // [RT][NB][32]
  uint64_t *bar = bars[warp];
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) a_mbar_init(&bar[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  const int heads = j.c.n_kv_heads, n_rows = j.group * j.q_tokens;

  // ---- this warp's share of the places
  const int per = (j.c.n_seqs + 31) / 32;
  int64_t total = 0;
  bool some_bad = false;
#pragma unroll 4
  for (int k = 0; k < per; ++k) {
    const int s = lane * per + k;
    int first, n = 0;
    bool bad = false;
    if (s < j.c.n_seqs) n = weigh_tiles(j, s, &first, &bad);
    some_bad |= bad;
    total += n ? n + kWeighPairCost : 0;
  }
  if (some_bad && blockIdx.x == 0 && warp == 0 && j.c.status) atomicOr(j.c.status, MOE_KV_BAD_LENGTH);
  const int64_t mine = total * heads;
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  const int64_t share = kv_div(total + (int64_t)gridDim.x * W - 1, (int64_t)gridDim.x * W);
  const int64_t u0 = share * ((int64_t)blockIdx.x * W + warp);
  if (u0 >= total) return;
  int seq = 0, first = 0, n = 0;
  int64_t pair0 = 0;  // the current sequence's first place, then the current pair's
  {
    const int src = __ffs(__ballot_sync(0xffffffffu, u0 >= before && u0 < before + mine)) - 1;
    int64_t run = __shfl_sync(0xffffffffu, before, src);
    for (int base = 0; base < per; base += 32) {
      const int k = base + lane, s = src * per + k;
      int f = 0, m = 0;
      bool bad;
      if (k < per && s < j.c.n_seqs) m = weigh_tiles(j, s, &f, &bad);
      const int64_t cost = m ? (int64_t)(m + kWeighPairCost) * heads : 0;
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
        seq = src * per + base + at;
        n = __shfl_sync(0xffffffffu, m, at);
        first = __shfl_sync(0xffffffffu, f, at);
        pair0 = __shfl_sync(0xffffffffu, begin, at);
        break;
      }
    }
  }
  int head = (int)kv_div(u0 - pair0, n + kWeighPairCost);
  pair0 += (int64_t)head * (n + kWeighPairCost);
  int64_t left = min(share, total - u0), off = u0 - pair0;

  uint32_t magic;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
  // ---- pieces: tiles [at, end) of a pair
  TileRing<S> on_way;
  while (left > 0) {
    const int64_t take = min(left, (int64_t)(n + kWeighPairCost) - off);
    const int at = (int)max((int64_t)0, off - kWeighPairCost), end = (int)max((int64_t)at, off + take - kWeighPairCost);
    left -= take;
    if (end > at) {
      const int len = __ldg(j.lens + seq);
      int64_t first_seen, unused;
      kv_visible(len, j.q_tokens, 0, j.window, &first_seen, &unused);
      // tokens whose totals begin at 0, and those that are written at all
      const int new_from = j.restart ? 0 : max(0, len - j.q_tokens);
      const int write_from = j.restart ? 0 : (int)first_seen;
      const int32_t *row = j.c.page_table + (int64_t)seq * j.c.table_stride;
#pragma unroll 1
      for (int r0 = 0; r0 < n_rows; r0 += 8 * RT) {
        // ---- the rows' queries as matrix operands: lane (g, t) holds row g's values 4t.. of each half block
        float f[RT][2], ahead[RT][2], lse[RT][2];
        bool big = false;
        __syncwarp();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const int r = r0 + 8 * rt + g;
          uint2 raw[NB][2];
#pragma unroll
          for (int b = 0; b < NB; ++b) raw[b][0] = raw[b][1] = make_uint2(0u, 0u);
          if (r < n_rows) {
            const T *src = static_cast<const T *>(j.q.data) + ((int64_t)seq * j.q_tokens + r / j.group) * j.q.token_stride +
                           (int64_t)(head * j.group + r % j.group) * j.q.head_stride;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int half = 0; half < 2; ++half)
                raw[b][half] = *reinterpret_cast<const uint2 *>(src + 32 * b + 16 * half + 4 * t);
          }
          float top = 0.f;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int z = 0; z < 8; ++z)
              top = fmaxf(top, fabsf(w_float(reinterpret_cast<const T *>(&raw[b][z / 4])[z % 4])));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^e with the row's largest value below 2^13 after it (an infinity or NaN stays what it is)
          int e = 12;
          if (top > 0.f && top < a_inf()) e = 12 - ((int)((__float_as_uint(top) >> 23) & 255) - 127);
          e = min(max(e, -120), 120);
          const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            __half h[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) h[z] = __float2half_rn(w_float(reinterpret_cast<const T *>(&raw[b][z / 4])[z % 4]) * up * (z < 4 ? 1.f : 0.0625f));
            q_mem[(rt * NB + b) * 32 + lane] =
                make_uint4(w_bits(__halves2half2(h[0], h[2])), w_bits(__halves2half2(h[1], h[3])),
                           w_bits(__halves2half2(h[4], h[6])), w_bits(__halves2half2(h[5], h[7])));
          }
          // The score's factor scale 2^-e, in one where fp32 holds it well; else the small one of the two goes ahead.
          const float both = j.scale * down;
          const bool far = !(both > 1e-30f && both < 1e30f);
          big |= far;
          const float mine_f = far ? fmaxf(j.scale, down) : both, mine_a = far ? fminf(j.scale, down) : 1.f;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            f[rt][z] = __shfl_sync(0xffffffffu, mine_f, 8 * t + 4 * z);
            ahead[rt][z] = __shfl_sync(0xffffffffu, mine_a, 8 * t + 4 * z);
            const int rr = r0 + 8 * rt + 2 * t + z;
            lse[rt][z] = rr < n_rows ? __ldg(j.lse + ((int64_t)seq * j.q_tokens + rr / j.group) * j.hq + head * j.group + rr % j.group)
                                     : a_inf();
          }
        }
        big = __any_sync(0xffffffffu, big);
        __syncwarp();
        // tiles that all rows of this pass see whole
        int whole_lo, whole_hi;
        {
          int64_t lo, hi, a, b;
          kv_visible(len, j.q_tokens, (min(n_rows, r0 + 8 * RT) - 1) / j.group, j.window, &a, &hi);
          kv_visible(len, j.q_tokens, r0 / j.group, j.window, &lo, &b);
          whole_lo = (int)a;
          whole_hi = (int)b;
        }

        // ---- copies, S tiles ahead; a lane looks up the page of one of the next 32 tiles
        int64_t my_src = -1, my_total = -1;
        int looked = at;  // tiles before it are looked up
        auto issue = [&](int tile, uint32_t x) {
          if (tile >= end || on_way.dead) return;
          if (tile == looked) {
            my_src = my_total = -1;
            if (tile + lane < end) {
              int in_page = 0;
              const int p = kv_page(row, j.c.table_width, j.c.n_pages, j.c.page_size, first + tile + lane, &in_page);
              if (p >= 0) {
                my_src = (int64_t)p * j.c.page_stride + kv_tile_off(D, j.c.page_size, head, in_page);
                my_total = ((int64_t)p * heads + head) * j.c.page_size + in_page * kKvTile;
              } else if (j.c.status) {
                atomicOr(j.c.status, MOE_KV_BAD_PAGE);
              }
            }
            looked += 32;
          }
          if (lane == tile - (looked - 32)) {
            const uint32_t st = TileRing<S>::stage(x);
            totals_at[warp][st] = my_total;
            if (my_src < 0) {
              a_mbar_arrive(&bar[st]);
            } else {
              a_expect_tx(&bar[st], C::kTile);
              a_bulk_load(ring + st * C::kTile, static_cast<const unsigned char *>(j.c.pages) + my_src, C::kTile, &bar[st]);
            }
          }
        };
        auto compute = [&](const unsigned char *tp, int64_t at_total, int tile) {
          const float before = j.totals[at_total + 8 * t + g];
          const int tok0 = (first + tile) * kKvTile;
          uint32_t kd[4][D / 64];  // key scales of tokens 8 x + g
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const unsigned char *sa = tp + 16 * D + (8 * x + g) * (D / 16);
            if constexpr (D == 64) {
              kd[x][0] = *reinterpret_cast<const uint32_t *>(sa);
            } else {
#pragma unroll
              for (int z = 0; z < D / 128; ++z)
                *reinterpret_cast<uint2 *>(&kd[x][2 * z]) = *reinterpret_cast<const uint2 *>(sa + 8 * z);
            }
          }
          float s[RT][2][4];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float c[RT][2][4];
            uint4 qf[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) qf[rt] = q_mem[(rt * NB + b) * 32 + lane];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const unsigned char *kp = tp + (b * 32 + mt * 16 + g) * 16 + 4 * t;
              const uint32_t wa = *reinterpret_cast<const uint32_t *>(kp), wb = *reinterpret_cast<const uint32_t *>(kp + 128);
              const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
              const uint32_t a0 = low_codes(wa, magic), a1 = low_codes(wb, magic), a2 = low_codes(wa8, magic), a3 = low_codes(wb8, magic);
              const uint32_t h0 = high_codes(wa, magic), h1 = high_codes(wb, magic), h2 = high_codes(wa8, magic), h3 = high_codes(wb8, magic);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                w_mma_first(c[rt][mt], a0, a1, a2, a3, qf[rt].x, qf[rt].y);
                w_mma(c[rt][mt], h0, h1, h2, h3, qf[rt].z, qf[rt].w);
              }
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const __half2 da = *reinterpret_cast<const __half2 *>(&kd[2 * mt][b / 2]);
              const __half2 db = *reinterpret_cast<const __half2 *>(&kd[2 * mt + 1][b / 2]);
              const float fa = (b & 1) ? __high2float(da) : __low2float(da), fb = (b & 1) ? __high2float(db) : __low2float(db);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                s[rt][mt][0] = b ? fmaf(c[rt][mt][0], fa, s[rt][mt][0]) : c[rt][mt][0] * fa;
                s[rt][mt][1] = b ? fmaf(c[rt][mt][1], fa, s[rt][mt][1]) : c[rt][mt][1] * fa;
                s[rt][mt][2] = b ? fmaf(c[rt][mt][2], fb, s[rt][mt][2]) : c[rt][mt][2] * fb;
                s[rt][mt][3] = b ? fmaf(c[rt][mt][3], fb, s[rt][mt][3]) : c[rt][mt][3] * fb;
              }
            }
          }
          if (big)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int x = 0; x < 8; ++x) s[rt][x / 4][x % 4] *= ahead[rt][x & 1];
          float sum[4] = {0.f, 0.f, 0.f, 0.f};  // of tokens 8 x + g
          auto weights = [&](auto is_whole) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                int rlo = 0, rhi = 0;
                if (!decltype(is_whole)::value) {
                  const int rr = r0 + 8 * rt + 2 * t + z;
                  int64_t lo64 = 0, hi64 = 0;
                  if (rr < n_rows) kv_visible(len, j.q_tokens, rr / j.group, j.window, &lo64, &hi64);
                  rlo = (int)lo64;
                  rhi = (int)hi64;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float p = a_exp2(fmaf(s[rt][x / 2][2 * (x % 2) + z], f[rt][z], -lse[rt][z]) * kLog2e);
                  const int tok = tok0 + 8 * x + g;
                  sum[x] += decltype(is_whole)::value || (tok >= rlo && tok < rhi) ? p : 0.f;
                }
              }
          };
          if (tok0 >= whole_lo && tok0 + kKvTile <= whole_hi) weights(std::true_type());
          else weights(std::false_type());
          // over the four lanes of a token; lane t is left with tokens 8 t + g
          const float a0 = t & 2 ? sum[2] : sum[0], a1 = t & 2 ? sum[3] : sum[1];
          const float b0 = t & 2 ? sum[0] : sum[2], b1 = t & 2 ? sum[1] : sum[3];
          const float c0 = a0 + __shfl_xor_sync(0xffffffffu, b0, 2), c1 = a1 + __shfl_xor_sync(0xffffffffu, b1, 2);
          const float own = (t & 1 ? c1 : c0) + __shfl_xor_sync(0xffffffffu, t & 1 ? c0 : c1, 1);
          const int tok = tok0 + 8 * t + g;
          if (tok >= write_from && tok < len)
            j.totals[at_total + 8 * t + g] = (r0 == 0 && tok >= new_from ? 0.f : before) + own;
        };
        const uint32_t x0 = on_way.used;
#pragma unroll 1
        for (int s = 0; s < S; ++s) issue(at + s, x0 + s);
        __syncwarp();
#pragma unroll 1
        for (int tile = at; tile < end; ++tile) {
          const uint32_t x = on_way.used;
          on_way.take(
              [&](uint32_t y) { return __all_sync(0xffffffffu, a_mbar_try(&bar[y % S], TileRing<S>::parity(y))) != 0; },
              [&](uint32_t y) { return __all_sync(0xffffffffu, w_wait(&bar[y % S], TileRing<S>::parity(y))) != 0; });
          if (on_way.dead) {
            // a copy that never came, and what nothing is asked for any more after it: NaN
            int in_page = 0;
            const int p = kv_page(row, j.c.table_width, j.c.n_pages, j.c.page_size, first + tile, &in_page);
            const int tok = (first + tile) * kKvTile + lane;
            if (p >= 0 && tok >= write_from && tok < len)
              j.totals[((int64_t)p * heads + head) * j.c.page_size + in_page * kKvTile + lane] = a_nan();
            if (lane == 0 && j.c.status) atomicOr(j.c.status, MOE_KV_TIMED_OUT);
            continue;
          }
          const int64_t at_total = totals_at[warp][x % S];
          if (at_total >= 0) compute(ring + (x % S) * C::kTile, at_total, tile);
          __syncwarp();
          issue(tile + S, x + S);
        }
      }
    }
    // the next pair
    off = 0;
    if (++head == heads) {
      head = 0;
      do {
        if (++seq >= j.c.n_seqs) return;
        bool bad;
        n = weigh_tiles(j, seq, &first, &bad);
      } while (n == 0);
    }
  }
}

template <int D, int RT, typename T>
int launch_weigh_rows(const WeighJob &j, int64_t places, cudaStream_t st) {
  using C = WeighCfg<D, RT>;
  static DynSmemLimit limit;
  if (ensure_dyn_smem(kv_weigh_kernel<D, RT, T>, C::kSmem, limit) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const int grid = (int)std::min<int64_t>((places + kWeighWarps - 1) / kWeighWarps, kWeighSms * C::kCtas);
  kv_weigh_kernel<D, RT, T><<<grid, 32 * kWeighWarps, C::kSmem, st>>>(j);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Row tiles of 8 that a pass over a tile's keys takes.
template <int D, typename T>
int launch_weigh(const WeighJob &j, int64_t places, cudaStream_t st) {
  const int rows = j.group * j.q_tokens;
  if (rows <= 8) return launch_weigh_rows<D, 1, T>(j, places, st);
  if (D == 256 || rows <= 16) return launch_weigh_rows<D, 2, T>(j, places, st);
  return launch_weigh_rows<D, D == 256 ? 2 : 4, T>(j, places, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int moe_kv_weigh(const moe_kv_cache *c, const int32_t *seq_lens, const moe_tensor *q, int32_t n_q_heads,
                         int32_t q_tokens, float scale, int32_t window, const float *lse, float *totals, int32_t restart,
                         int32_t dtype, void *cuda_stream) {
  if (c && c->n_seqs == 0) return MOE_OK;
  if (const int rc = check_cache(c)) return rc;
  if (!seq_lens || !lse || (!totals && c->n_pages > 0) || n_q_heads <= 0 || n_q_heads % c->n_kv_heads || q_tokens <= 0 || window < 0 ||
      !(scale > 0.f && scale <= kMostScale) || (uintptr_t)lse % 4 || (uintptr_t)totals % 4)
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (n_q_heads > kMaxAttnHeads || q_tokens > 1024) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)c->table_width * c->page_size > kMostTokens) return MOE_ERR_UNSUPPORTED;
  if (const int rc = check_tensor(q, 2)) return rc;
  WeighJob j = {};
  j.c = *c;
  j.lens = seq_lens;
  j.q = *q;
  j.lse = lse;
  j.totals = totals;
  j.hq = n_q_heads;
  j.group = n_q_heads / c->n_kv_heads;
  j.q_tokens = q_tokens;
  j.window = window;
  j.restart = restart != 0;
  j.scale = scale;
  const int64_t places =
      (int64_t)c->n_seqs * c->n_kv_heads * ((int64_t)c->table_width * (c->page_size / kKvTile) + kWeighPairCost);
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const int D = c->head_dim;
  if (dtype == MOE_BF16)
    return D == 64    ? launch_weigh<64, __nv_bfloat16>(j, places, st)
           : D == 128 ? launch_weigh<128, __nv_bfloat16>(j, places, st)
                      : launch_weigh<256, __nv_bfloat16>(j, places, st);
  return D == 64    ? launch_weigh<64, __half>(j, places, st)
         : D == 128 ? launch_weigh<128, __half>(j, places, st)
                    : launch_weigh<256, __half>(j, places, st);
}
