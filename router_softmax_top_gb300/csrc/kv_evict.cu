// Keeping the cached tokens that have received most attention weight, and moving them together.
//
// Per sequence of n > budget tokens and key head: the first `first` and the last `recent`
// tokens stay, and of those between the budget - first - recent with the largest totals
// (ties: the earlier token), all in their order, in the slots [0, budget).
//
// Choosing: a radix search for the smallest total that stays, 11, 11 and 10 bits of a key
// that orders like the value, until few keys are left, which are compared each with each; by
// a CTA, or a cluster of them, per (sequence, head): each holds its part of the keys in shared
// memory, counts are added over the cluster's shared memory.  Then the kept tokens' numbers
// are written in order, from counts per warp.
//
// Moving, in place: the token of rank r goes to slot r, which is never after its own.  A CTA
// takes the 256 tokens of a group: it loads those that stay into shared memory, says so, waits
// for the groups whose tokens are in the slots that these go to to have said so (at most two,
// and none later than itself), and writes.  Groups are handed out in order, so whatever one
// waits for has been begun by a CTA that is running, and loading waits for nothing.
//
// Bound: memory (the kept tokens' bytes read and written; DRAM gives 64 bytes at least, which
// four neighbouring tokens' pieces of 16 bytes share, so that where half the tokens stay
// nearly all of the cache is read), the totals, and for one sequence the search's passes over a
// few CTAs and the barriers between them.
// Measured: one sequence of 131071 tokens on 8 heads of 128, half of them kept, 67 us: search
// 23 (at the copy rate all bytes that DRAM has to move would take 35).  32 sequences of 3000 to
// 12000 tokens on 4 heads of 256, 4096 kept, 89 us (search 14; DRAM 52).  One of 1100 tokens,
// 1024 kept, 13 us.
#include <algorithm>
#include <cooperative_groups.h>

#include "attn_common.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kBins = 2048;
constexpr int kFew = 128;         // keys that are compared each with each
constexpr int kMostHeld = 49152;  // keys that a CTA's shared memory holds (more are read again for every pass)
constexpr int kMostHeldByTwo = 16384;  // of two CTAs on an SM
// Caches of so many tokens a sequence at most take a CTA of 256 threads, of which several share an SM, rather than 1024 (1, 32
// and 512 pairs of 1500 tokens: 13.6, 14.9 and 35.5 us by 256 threads, 12.9, 14.2 and 36.1 by more; of 2400 tokens 15.1, 17.7
// and 52.5, and 13.1, 15.9 and 53.1).
constexpr int kSmallTokens = 2048;
// Tokens per CTA from which on a pair takes a cluster of twice as many (a sequence on 4 heads by one, two and four CTAs a
// head: of 6000 tokens 15.0 and 16.5 us, of 12000 18.9, 20.0 and 18.8, of 16384 20.5, 20.2 and 19.0).
constexpr int kClusterTokens = 8192;
constexpr int kSlots = 128;       // tokens of a step, four a lane
// Tokens that a CTA moves, a thread each, two steps' worth: what it has loaded is announced once, and the announcement waits
// for the SM's writes (32 sequences of 12000 tokens on 4 heads of 256, 3600 kept: 128 us by 128 tokens, 120 so; one of 1100
// tokens 0.6 us more).
constexpr int kGroup = 256, kSteps = kGroup / kSlots;
// Kept tokens of a group from which on its tiles are loaded whole, by a bulk copy each, rather than the tokens' pieces: 32
// sequences of 12000 tokens on 4 heads of 64, 128 and 256 take 53, 73 and 111 us whole and 55, 76 and 115 in pieces with 51 of
// 256 kept, 55, 79 and 121 and 60, 85 and 131 with 77, 50, 68 and 102 and 50, 65 and 95 with 26.
constexpr int kWhole = 40;
constexpr int kEvictSms = 152;
constexpr int64_t kMostTokens = 1 << 30;  // that a row of the page table may hold (counts and steps stay within 32 bits)

struct EvictJob {
  moe_kv_cache c;
  const int32_t *lens;
  float *totals;
  int budget, first, recent, heads;
  int32_t *new_lens, *kept;
  // workspace: next group; per pair whether it stays as it is; per pair and step: the kept tokens before it; per pair and
  // group: whether its tokens have been loaded
  uint32_t *ticket;
  int32_t *skip, *before;
  uint32_t *loaded;
  int groups;  // entries per pair: all the page table can hold, and one more
  int held;    // keys that a CTA holds
};

// Orders like the value; NaN above all, -0 as +0.
__device__ __forceinline__ uint32_t total_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ bool length_ok(const EvictJob &j, int n) {
  return n >= 0 && n <= (int64_t)j.c.table_width * j.c.page_size;
}

struct __align__(8) BinPair {
  int low, high;
};

// CL: a cluster per pair, else one CTA.  NT: its threads.
template <int NT, bool CL>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictJob j) {
  constexpr int NW = NT / 32, PER = kBins / NT;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t s_keys[kFew];
  __shared__ int s_bad, s_found[3][3], s_warp[2][32], s_count[2], s_scan[32], s_few;
  __shared__ uint32_t s_least;
  __shared__ int s_need;
  asm volatile("griddepcontrol.launch_dependents;");
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = CL ? (int)cluster.num_blocks() : 1, rank = CL ? (int)cluster.block_rank() : 0;
  auto sync = [&]() {
    if constexpr (CL) cluster.sync();
    else __syncthreads();
  };
  auto of_rank = [&](auto *p, int r) {
    if constexpr (CL) return cluster.map_shared_rank(p, r);
    else return p;
  };
  const int pair = blockIdx.x / ranks, seq = pair / j.heads, head = pair % j.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = __ldg(j.lens + seq);
  int32_t *kept = j.kept + (int64_t)pair * j.budget;
  if (blockIdx.x == 0 && tid == 0) *j.ticket = 0;
  const bool ok = length_ok(j, n);
  if (!ok || n <= j.budget) {  // (all CTAs of the cluster alike)
    for (int i = rank * NT + tid; i < j.budget; i += ranks * NT) kept[i] = ok && i < n ? i : -1;
    if (rank == 0 && tid == 0) {
      j.skip[pair] = 1;
      if (head == 0) j.new_lens[seq] = n;
      if (!ok && j.c.status) atomicOr(j.c.status, MOE_KV_BAD_LENGTH);
    }
    return;
  }
  const int32_t *row = j.c.page_table + (int64_t)seq * j.c.table_stride;
  const int per = ((n + ranks - 1) / ranks + kSlots - 1) / kSlots * kSlots, a = min(n, rank * per), b = min(n, a + per);
  const bool hold = per <= j.held;
  const float inverse = 1.f / (float)j.c.page_size;
  // the keys of tokens i to i + 3, i a multiple of 4 below n; tokens without a page have none
  auto load = [&](int i) {
    int slot;
    if (n <= 1 << 22) {
      slot = (int)((float)i * inverse);  // its page, or one beside: the product is off by 2^-22 of itself, below 2^17
      slot -= slot * j.c.page_size > i;
      slot += (slot + 1) * j.c.page_size <= i;
    } else {
      slot = i / j.c.page_size;
    }
    const int p = __ldg(row + slot);
    if (p < 0 || p >= j.c.n_pages) {
      s_bad = 1;
      return make_uint4(0u, 0u, 0u, 0u);
    }
    const float4 v = *reinterpret_cast<const float4 *>(j.totals + ((int64_t)p * j.heads + head) * j.c.page_size + (i - slot * j.c.page_size));
    const uint4 u = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
    if (max(max(u.x, u.y), max(u.z, u.w)) <= 0x7f800000u)  // the usual: none negative, none NaN
      return make_uint4(u.x | 0x80000000u, u.y | 0x80000000u, u.z | 0x80000000u, u.w | 0x80000000u);
    return make_uint4(total_key(v.x), total_key(v.y), total_key(v.z), total_key(v.w));
  };
  auto four = [&](int i) { return hold ? *reinterpret_cast<const uint4 *>(keys + (i - a)) : load(i); };
  // f(token, key) for those of tokens i to i + 3 that may go
  const int c0 = j.first, c1 = n - j.recent;
  auto each = [&](int i, const uint4 &k, auto f) {
    if (i >= c0 && i + 4 <= min(b, c1)) {
      f(i, k.x);
      f(i + 1, k.y);
      f(i + 2, k.z);
      f(i + 3, k.w);
    } else {
      const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (i + z >= c0 && i + z < min(b, c1)) f(i + z, w[z]);
    }
  };
  if (tid == 0) s_bad = s_few = 0;
  for (int i = tid; i < 3 * kBins; i += NT) hist[0][i] = 0;
  __syncthreads();
  // ---- the smallest key that stays, and how many of that key
  int need = j.budget - j.first - j.recent;
  const bool some = need > 0;
#pragma unroll 4
  for (int i = a + 4 * tid; i < b; i += 4 * NT) {
    const uint4 k = load(i);
    if (hold) *reinterpret_cast<uint4 *>(keys + (i - a)) = k;
    each(i, k, [&](int, uint32_t x) { atomicAdd(&hist[0][x >> 21], 1u); });
  }
  for (int g = rank * NT + tid; g < (n + kSlots - 1) / kSlots; g += ranks * NT) j.loaded[(int64_t)pair * j.groups + g] = 0;
  sync();
  // (a lane looks at a CTA of the cluster, here and below: one after another they would be a chain of waits)
  const bool bad = __any_sync(0xffffffffu, lane < ranks && *of_rank(&s_bad, lane) != 0);
  if (bad) {
    for (int i = rank * NT + tid; i < j.budget; i += ranks * NT) kept[i] = -1;
    if (rank == 0 && tid == 0) {
      j.skip[pair] = 1;
      if (head == 0) j.new_lens[seq] = n;
      if (j.c.status) atomicOr(j.c.status, MOE_KV_BAD_PAGE);
    }
    sync();  // (the others look at this one's word)
    return;
  }
  uint32_t least = 0;
  if (some) {
    int shift = 21;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      // Counts over the cluster, largest key first, PER bins a thread.  Every CTA adds up all bins: a share of them each
      // would cost two more barriers over the cluster.
      const int hi = kBins - 1 - PER * tid;
      int n_bin[PER], inc = 0;
#pragma unroll
      for (int z = 0; z < PER; ++z) n_bin[z] = 0;
      constexpr int AT_ONCE = CL ? 8 : 1;  // loads on their way together
      for (int r0 = 0; r0 < ranks; r0 += AT_ONCE) {
        BinPair v[AT_ONCE][PER / 2];
#pragma unroll
        for (int r = 0; r < AT_ONCE; ++r)
#pragma unroll
          for (int z = 0; z < PER / 2; ++z) {
            v[r][z] = {0, 0};
            if (r0 + r < ranks) v[r][z] = *reinterpret_cast<const BinPair *>(of_rank(&hist[pass][0], r0 + r) + hi - 2 * z - 1);
          }
#pragma unroll
        for (int r = 0; r < AT_ONCE; ++r)
#pragma unroll
          for (int z = 0; z < PER / 2; ++z) {
            n_bin[2 * z] += v[r][z].high;
            n_bin[2 * z + 1] += v[r][z].low;
          }
      }
#pragma unroll
      for (int z = 0; z < PER; ++z) inc += n_bin[z];
      const int mine = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s_scan[warp] = inc;
      __syncthreads();
      int before = inc - mine + (int)__reduce_add_sync(0xffffffffu, (uint32_t)(lane < warp ? s_scan[lane] : 0));
#pragma unroll
      for (int z = 0; z < PER; ++z) {
        if (before < need && before + n_bin[z] >= need) {
          s_found[pass][0] = hi - z;
          s_found[pass][1] = before;
          s_found[pass][2] = n_bin[z];
        }
        before += n_bin[z];
      }
      __syncthreads();
      const int *found = s_found[pass];
      least = pass == 0 ? (uint32_t)found[0] : (least << (pass == 1 ? 11 : 10)) | (uint32_t)found[0];
      need -= found[1];
      const int in = found[2];
      if (pass == 2) break;
      if (in <= kFew) {
        // few enough to be compared each with each: the first CTA's list has them all
        int *count = of_rank(&s_few, 0);
        uint32_t *list = of_rank(s_keys, 0);
        for (int i = a + 4 * tid; i < b; i += 4 * NT)
          each(i, four(i), [&](int, uint32_t x) {
            if ((x >> shift) == least) list[atomicAdd(count, 1)] = x;
          });
        sync();
        uint32_t own = 0;
        if (tid < in) own = list[tid];
        if constexpr (CL) {
          if (rank > 0 && tid < in) s_keys[tid] = own;  // (the first CTA's stays as it is)
          __syncthreads();
        }
        if (tid < in) {
          int more = 0, equal = 0;
          for (int s = 0; s < in; ++s) {
            more += s_keys[s] > own;
            equal += s_keys[s] == own;
          }
          if (more < need && more + equal >= need) {  // (threads of the same key write the same)
            s_least = own;
            s_need = need - more;
          }
        }
        __syncthreads();
        least = s_least;
        need = s_need;
        break;
      }
      // the next digit of those keys
      const int bits = pass == 0 ? 11 : 10, down = shift - bits;
      for (int i = a + 4 * tid; i < b; i += 4 * NT)
        each(i, four(i), [&](int, uint32_t x) {
          if ((x >> shift) == least) atomicAdd(&hist[pass + 1][(x >> down) & ((1u << bits) - 1u)], 1u);
        });
      shift = down;
      sync();
    }
  }
  // ---- the kept tokens in order.  Before a token come S that stay in any case and E whose key is the least that stays:
  // its rank is S + min(E, need).  A warp takes neighbouring steps of 128 tokens; first their counts.
  const int steps = (b - a + kSlots - 1) / kSlots, w0 = (int)((int64_t)steps * warp / NW), w1 = (int)((int64_t)steps * (warp + 1) / NW);
  // of tokens i to i + 3: bit z for one that stays, bit 4 + z for one of the least key
  auto kinds = [&](int i) {
    uint32_t bits = 0;
    if (i >= b) return bits;
    if (some) {
      const uint4 k = four(i);
      bits = (k.x > least ? 1u : 0u) | (k.y > least ? 2u : 0u) | (k.z > least ? 4u : 0u) | (k.w > least ? 8u : 0u);
      bits |= (k.x == least ? 16u : 0u) | (k.y == least ? 32u : 0u) | (k.z == least ? 64u : 0u) | (k.w == least ? 128u : 0u);
    }
    if (i < c0 || i + 4 > c1) {
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (i + z < c0 || i + z >= c1) bits = (bits & ~(17u << z)) | (i + z < b ? 1u << z : 0u);
    }
    return bits;
  };
  uint32_t saved = 0;  // of the warp's first four steps
  int sure = 0, eq = 0;
  for (int s = w0; s < w1; ++s) {
    const uint32_t bits = kinds(a + kSlots * s + 4 * lane);
    if (s < w0 + 4) saved |= bits << (8 * (s - w0));
    sure += __popc(bits & 15u);
    eq += __popc(bits >> 4);
  }
  sure = (int)__reduce_add_sync(0xffffffffu, (uint32_t)sure);
  eq = (int)__reduce_add_sync(0xffffffffu, (uint32_t)eq);
  if (lane == 0) {
    s_warp[0][warp] = sure;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (warp < 2) {
    int v = lane < NW ? s_warp[warp][lane] : 0;
    const int own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    s_warp[warp][lane] = v - own;
    if (lane == 31) s_count[warp] = v;
  }
  sync();
  sure = s_warp[0][warp];
  eq = s_warp[1][warp];
  if constexpr (CL) {
    sure += __reduce_add_sync(0xffffffffu, lane < rank ? of_rank(&s_count[0], lane)[0] : 0);
    eq += __reduce_add_sync(0xffffffffu, lane < rank ? of_rank(&s_count[0], lane)[1] : 0);
  }
  int32_t *group_before = j.before + (int64_t)pair * j.groups;
  for (int s = w0; s < w1; ++s) {
    const int i = a + kSlots * s + 4 * lane;
    const uint32_t bits = s < w0 + 4 ? (saved >> (8 * (s - w0))) & 255u : kinds(i);
    // counts of the lanes before, of a step at most 128 each
    uint32_t own = (uint32_t)__popc(bits & 15u) | (uint32_t)__popc(bits >> 4) << 16, inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    int S = sure + (int)((inc - own) & 0xffffu), E = eq + (int)((inc - own) >> 16);
    if (lane == 0) group_before[(a + kSlots * s) / kSlots] = S + min(E, need);
    int32_t *to = kept + S + min(E, need);
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const bool stays = ((bits >> z) & 1u) || (((bits >> (4 + z)) & 1u) && E++ < need);
      if (stays) *to++ = i + z;
    }
    inc = __shfl_sync(0xffffffffu, inc, 31);
    sure += (int)(inc & 0xffffu);
    eq += (int)(inc >> 16);
  }
  if (rank == 0 && tid == 0) {
    group_before[(n + kSlots - 1) / kSlots] = j.budget;
    j.skip[pair] = 0;
    if (head == 0) j.new_lens[seq] = j.budget;
  }
  if constexpr (CL) cluster.sync();  // (a CTA's counts are read by those after it)
}

// N bytes (4, 8 or 16) into shared memory, asynchronously.
template <int N>
__device__ __forceinline__ void e_copy(void *dst, const void *src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a_smem(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(a_smem(dst)), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ bool is_loaded(const uint32_t *flag) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
  return v != 0;
}
__device__ __forceinline__ bool wait_loaded(const uint32_t *flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < kAttnSpin; ++i) {
    if (is_loaded(flag)) return true;
    if ((i & 255u) == 255u) {
      const uint64_t now = a_now_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kAttnWaitNs) return false;
    }
  }
  return false;
}

template <int D>
struct MoveCfg {
  static constexpr int kPieces = 2 * (D / 32);  // 16-byte pieces of codes of a token
  static constexpr int kScale = D / 16;         // bytes of a token's scales of keys, and of values
  static constexpr int kTile = 36 * D;
  // a group's tiles, or its kept tokens: of each a row of pieces over the threads, then of scales
  static constexpr size_t kSmem = (size_t)kGroup / kKvTile * kTile;
  static_assert(kSmem == (size_t)kGroup * (16 * kPieces + 2 * kScale), "the two ways of holding a group");
  static constexpr int kCtas = D == 256 ? 3 : D == 128 ? 5 : 8;  // per SM, by shared memory and threads
};

template <int D>
__global__ void __launch_bounds__(kGroup, MoveCfg<D>::kCtas) evict_move_kernel(const EvictJob j) {
  using C = MoveCfg<D>;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t bar;
  __shared__ int s_seq, s_head, s_group, s_ok, s_wait;
  __shared__ float s_total[kGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (j.c.n_seqs + 31) / 32;
  uint32_t phase = 0;
  if (tid == 0) {
    a_mbar_init(&bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (;;) {
    if (warp == 0) {
      // the next group: sequences in order, in one the heads' groups side by side
      uint32_t u = 0;
      if (lane == 0) u = atomicAdd(j.ticket, 1u);
      int64_t mine = 0, before;
      for (int k = 0; k < per; ++k) {
        const int s = lane * per + k;
        if (s >= j.c.n_seqs) break;
        const int n = __ldg(j.lens + s);
        if (length_ok(j, n) && n > j.budget) mine += (int64_t)((n + kGroup - 1) / kGroup) * j.heads;
      }
      before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= mine;
      u = __shfl_sync(0xffffffffu, u, 0);
      if (lane == 0) {
        s_seq = -1;
        s_ok = 1;
      }
      __syncwarp();
      if ((int64_t)u >= before && (int64_t)u < before + mine) {
        int64_t left = (int64_t)u - before;
        for (int k = 0; k < per; ++k) {
          const int s = lane * per + k, n = __ldg(j.lens + s);
          const int64_t of = length_ok(j, n) && n > j.budget ? (int64_t)((n + kGroup - 1) / kGroup) * j.heads : 0;
          if (left < of) {
            s_seq = s;
            s_head = (int)(left % j.heads);
            s_group = (int)(left / j.heads);
            break;
          }
          left -= of;
        }
      }
    }
    __syncthreads();
    const int seq = s_seq, head = s_head, g = s_group;
    if (seq < 0) return;
    const int pair = seq * j.heads + head;
    const int n = __ldg(j.lens + seq), t0 = g * kGroup, n_own = min(kGroup, n - t0);  // the group's tokens
    const int32_t *row = j.c.page_table + (int64_t)seq * j.c.table_stride;
    const bool skip = j.skip[pair] != 0;
    // the ranks of those that stay: [r0, r1).  (Where the sequence is left as it is, neither is of use.)
    const int32_t *before = j.before + (int64_t)pair * j.groups;
    const int r0 = before[g * kSteps], r1 = before[min((g + 1) * kSteps, (n + kSlots - 1) / kSlots)], count = r1 - r0;
    uint32_t *loaded = j.loaded + (int64_t)pair * j.groups;
    if (skip) {
      __syncthreads();  // (what to work on is read until here)
      continue;
    }
    // (with all tokens before kept, and all of its own, they are in their places)
    const bool moves = count > 0 && !(r0 == t0 && count == n_own), whole = count >= kWhole;
    unsigned char *const pages = static_cast<unsigned char *>(j.c.pages);
    // where a token's tile is, and the token in it; the page was seen to be there
    auto place = [&](int i, int64_t *tile, int64_t *total) {
      const int at = i / j.c.page_size, in = i - at * j.c.page_size;
      const int64_t p = __ldg(row + at);
      *tile = p * j.c.page_stride + kv_tile_off(D, j.c.page_size, head, in / kKvTile);
      *total = (p * j.heads + head) * j.c.page_size + in;
      return in % kKvTile;
    };
    auto codes = [&](int piece) { return sm + ((size_t)piece * kGroup + tid) * 16; };
    auto scales = [&](int v) { return sm + (size_t)kGroup * 16 * C::kPieces + ((size_t)v * kGroup + tid) * C::kScale; };
    int64_t own_total = 0, tile = 0, total = 0;
    int tok = 0, src = -1;
    bool came = true;
    const int to = r0 + tid;  // this thread's rank
    if (tid < n_own) {
      int64_t own_tile;
      const int own_tok = place(t0 + tid, &own_tile, &own_total);
      if (moves && whole && own_tok == 0) a_bulk_load(sm + tid / kKvTile * C::kTile, pages + own_tile, C::kTile, &bar);
      s_total[tid] = j.totals[own_total];  // (in shared memory, so that it has arrived)
    }
    if (moves) {
      if (whole && tid == 0) a_expect_tx(&bar, (uint32_t)((n_own + kKvTile - 1) / kKvTile * C::kTile));
      if (tid < count) {
        src = j.kept[(int64_t)pair * j.budget + to];
        tok = place(to, &tile, &total);
      }
      // whose tokens are in the slots that are written: of two groups at most, which often have said so by now
      if (warp == 1) {
        const int h = r0 / kGroup + lane;
        const bool wait = h <= (r1 - 1) / kGroup && h < g && !is_loaded(loaded + h);
        if (const bool any = __any_sync(0xffffffffu, wait); lane == 0) s_wait = any;
      }
      if (whole) {
        came = a_mbar_wait(&bar, phase);
        phase ^= 1;
      } else {
        if (src > to) {
          int64_t src_tile, unused;
          const int src_tok = place(src, &src_tile, &unused);
          const unsigned char *tp = pages + src_tile;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
#pragma unroll
            for (int b = 0; b < D / 32; ++b) e_copy<16>(codes(v * (D / 32) + b), tp + kv_code_off(D, v, b, src_tok));
            e_copy<C::kScale>(scales(v), tp + kv_scale_off(D, v, 0, src_tok));
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
    }
    if (!__syncthreads_and(came)) {
      // a copy that never came: nothing is said to be loaded, nor written, any more
      if (tid == 0) {
        if (j.c.status) atomicOr(j.c.status, MOE_KV_TIMED_OUT);
        (void)a_mbar_drain(&bar, phase ^ 1);
      }
      return;
    }
    // (A release: what the CTA's threads have read before the barrier, they have read before this.  It waits for the SM's
    // writes on their way, so it is left out where nobody comes to write.)
    if (tid == 0 && t0 < j.budget) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(loaded + g), "r"(1u) : "memory");
    if (tid < n_own && t0 + tid >= j.budget) j.totals[own_total] = 0.f;
    if (moves) {
      if (s_wait) {
        if (warp == 0) {
          const int h = r0 / kGroup + lane;
          if (h <= (r1 - 1) / kGroup && h < g && !wait_loaded(loaded + h)) s_ok = 0;
        }
        __syncthreads();
      }
      if (!s_ok) {
        if (tid == 0 && j.c.status) atomicOr(j.c.status, MOE_KV_TIMED_OUT);
      } else if (src > to) {
        unsigned char *tp = pages + tile;
        const int in = src - t0;
        const unsigned char *from = sm + in / kKvTile * C::kTile;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
          for (int b = 0; b < D / 32; ++b)
            *reinterpret_cast<uint4 *>(tp + kv_code_off(D, v, b, tok)) = *reinterpret_cast<const uint4 *>(
                whole ? from + kv_code_off(D, v, b, in % kKvTile) : codes(v * (D / 32) + b));
          unsigned char *sp = tp + kv_scale_off(D, v, 0, tok);
          const unsigned char *fp = whole ? from + kv_scale_off(D, v, 0, in % kKvTile) : scales(v);
          if constexpr (C::kScale == 4) *reinterpret_cast<uint32_t *>(sp) = *reinterpret_cast<const uint32_t *>(fp);
          else if constexpr (C::kScale == 8) *reinterpret_cast<uint2 *>(sp) = *reinterpret_cast<const uint2 *>(fp);
          else *reinterpret_cast<uint4 *>(sp) = *reinterpret_cast<const uint4 *>(fp);
        }
        j.totals[total] = s_total[in];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (before the next tiles come where these were read)
    }
    __syncthreads();
  }
}

template <typename... A>
cudaError_t launch_with(void (*kernel)(A...), int64_t grid, int threads, size_t smem, cudaLaunchAttribute attr, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int NT, bool CL>
DynSmemLimit &select_limit() {
  static DynSmemLimit limit;
  return limit;
}

template <int NT, bool CL>
cudaError_t launch_select(const EvictJob &j, int64_t pairs, int ranks, cudaStream_t st) {
  const size_t smem = (size_t)j.held * 4;
  // (raised from 16 KB on: the kernel's own arrays, 25 KB, count towards what needs no raising)
  const cudaError_t e = ensure_dyn_smem(evict_select_kernel<NT, CL>, smem > 16 * 1024 ? std::max<size_t>(smem, 64 * 1024) : smem,
                                        select_limit<NT, CL>());
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  if (ranks > 8) {
    const cudaError_t f = cudaFuncSetAttribute(evict_select_kernel<NT, CL>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (f != cudaSuccess) return f;
  }
  return launch_with(evict_select_kernel<NT, CL>, pairs * ranks, NT, smem, attr, st, j);
}

// Clusters of 16 CTAs that run at once on the current device.
int wide_clusters() {
  static std::atomic<int> known[DynSmemLimit::kDevices] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= DynSmemLimit::kDevices) return 0;
  if (const int k = known[dev].load(std::memory_order_relaxed)) return k - 1;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = kMostHeld * 4;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  const auto kernel = evict_select_kernel<1024, true>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      ensure_dyn_smem(kernel, cfg.dynamicSmemBytes, select_limit<1024, true>()) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int D>
cudaError_t launch_move(const EvictJob &j, int64_t groups, cudaStream_t st) {
  using C = MoveCfg<D>;
  static DynSmemLimit limit;
  const cudaError_t e = ensure_dyn_smem(evict_move_kernel<D>, C::kSmem, limit);
  if (e != cudaSuccess) return e;
  // a programmatic dependent of the kernel before it: its CTAs are there when that ends
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return launch_with(evict_move_kernel<D>, std::min<int64_t>(groups, (int64_t)kEvictSms * C::kCtas), kGroup, C::kSmem, attr, st, j);
}

int64_t evict_groups(const moe_kv_cache *c) { return ((int64_t)c->table_width * c->page_size + kSlots - 1) / kSlots + 1; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int64_t moe_kv_evict_workspace(const moe_kv_cache *c) {
  if (check_cache(c) != MOE_OK || (int64_t)c->table_width * c->page_size > kMostTokens) return 0;
  return 256 + (int64_t)c->n_seqs * c->n_kv_heads * (4 + 8 * evict_groups(c));
}

MOE_API int moe_kv_evict(const moe_kv_cache *c, const int32_t *seq_lens, float *totals, int32_t budget, int32_t first,
                         int32_t recent, int32_t *new_lens, int32_t *kept, void *workspace, int64_t workspace_bytes,
                         void *cuda_stream) {
  if (c && c->n_seqs == 0) return MOE_OK;
  if (const int rc = check_cache(c)) return rc;
  if (!seq_lens || (!totals && c->n_pages > 0) || !new_lens || budget < 0 || first < 0 || recent < 0 || (int64_t)first + recent > budget ||
      (!kept && budget > 0) || (uintptr_t)totals % 16 || (uintptr_t)kept % 4 || (uintptr_t)new_lens % 4)
    return MOE_ERR_INVALID_ARG;
  if (budget > kMostTokens || (int64_t)c->table_width * c->page_size > kMostTokens ||
      (int64_t)c->n_seqs * c->n_kv_heads > 0x7fffffff / 8)
    return MOE_ERR_UNSUPPORTED;
  if (new_lens == seq_lens || !workspace || (uintptr_t)workspace % 256 || workspace_bytes < moe_kv_evict_workspace(c))
    return MOE_ERR_INVALID_ARG;
  const int64_t pairs = (int64_t)c->n_seqs * c->n_kv_heads, tokens = (int64_t)c->table_width * c->page_size;
  EvictJob j = {};
  j.c = *c;
  j.lens = seq_lens;
  j.totals = totals;
  j.budget = budget;
  j.first = first;
  j.recent = recent;
  j.heads = c->n_kv_heads;
  j.new_lens = new_lens;
  j.kept = kept;
  j.groups = (int)evict_groups(c);
  j.ticket = static_cast<uint32_t *>(workspace);
  j.skip = static_cast<int32_t *>(workspace) + 64;
  j.before = j.skip + pairs;
  j.loaded = reinterpret_cast<uint32_t *>(j.before + pairs * j.groups);
  // A cluster per pair where pairs alone leave SMs idle and have many keys (32 sequences of 12000 tokens on 4 heads: 21 us
  // as clusters of two, 15 us so; one of 131071 on 8 heads 8 CTAs each).  A CTA of 1024 threads is alone on its SM, of 512
  // two are.  Sixteen CTAs, if the GPU has room for such clusters, of more keys than fill three quarters of what eight hold
  // (one head by eight and by sixteen, both kernels, half of the tokens kept: 230000 tokens 41 and 45 us, 290000 45 and 47,
  // 350000 54 and 53, 390000 60 and 56, 400000 82 and 58; four heads of 230000 71 and 73, of 350000 95 and 92).
  int ranks = 1;
  while (ranks < 8 && pairs * ranks * 2 <= kEvictSms && tokens > kClusterTokens * (int64_t)ranks) ranks *= 2;
  if (ranks == 8 && pairs * 16 <= kEvictSms && tokens > (int64_t)kMostHeld * 6 && wide_clusters() >= pairs) ranks = 16;
  j.held = (int)std::min<int64_t>(kMostHeld, ((tokens + ranks - 1) / ranks + kSlots - 1) / kSlots * kSlots);
  cudaStream_t st = (cudaStream_t)cuda_stream;
  cudaError_t e = ranks > 1                                            ? launch_select<1024, true>(j, pairs, ranks, st)
                  : tokens <= kSmallTokens                             ? launch_select<256, false>(j, pairs, 1, st)
                  : pairs <= kEvictSms || j.held > kMostHeldByTwo ? launch_select<1024, false>(j, pairs, 1, st)
                                                                       : launch_select<512, false>(j, pairs, 1, st);
  if (e == cudaSuccess && tokens > budget) {  // (else no sequence is over it)
    const int64_t groups = pairs * ((j.groups - 1 + kSteps - 1) / kSteps);
    e = c->head_dim == 64    ? launch_move<64>(j, groups, st)
        : c->head_dim == 128 ? launch_move<128>(j, groups, st)
                             : launch_move<256>(j, groups, st);
  }
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}
