// The attention weight that the keys of whole prompts receive from the prompts' queries, on
// the 5th-gen tensor cores.
//
// total[key] (+)= sum over the rows (token, head of the key's group) that see it of
// exp(scale q . k - lse), lse what attention gave beside its result.
//
// Bound: 2 D flops and an exponential (32 per cycle and SM) per pair of a row and a key that
// sees it: for heads of 128 the one takes about as long as the other, for 64 the exponential
// twice as long.  What the kernel comes to first is the path to shared memory: the matrix
// unit reads both operands of every product there, and threads the lse of every column.
// The product is formed as K Q^T, 128 keys by 128 rows, so that a thread owns a key: it reads
// its scores from tensor memory, forms the weights and sums them in registers; nothing is
// exchanged between threads.
//  * A CTA keeps a tile of 128 keys of one key head in shared memory and walks over the rows
//    that see any of them (causality: those from the keys on; a window: not far past them).
//    Rows come by TMA, 128 / group tokens of all heads of the group at a time, two tiles
//    ahead; two score buffers in tensor memory with a warpgroup each; two CTAs per SM (one for
//    heads of 256), so that one's start and end hide behind the other.  8192 tokens, when
//    they took 232 us so: one stage and buffer and three CTAs per SM 269, one CTA of four
//    buffers that stays and takes tile after tile 278; one warpgroup for both buffers took
//    100 us more.
//  * Tiles of keys are handed out in their order: earlier ones are seen by more rows, so the
//    longest come first.  Where there are fewer tiles than room for CTAs, a cluster shares a
//    tile's rows, and sums are joined in a fixed order: results do not depend on timing.
//  * The score less lse is formed before the factor log2(e): of large weights, whose difference
//    is small, only the score's own rounding is left.  (With that factor in the scale and in lse
//    it took 2% less, with twice the error, from lse's rounding.)  Sums are fp32, of a tile's rows
//    first.
//  * Only tiles of rows that do not all see all keys are masked: the rows that see a thread's
//    key are a run of columns, a bit each (by positions per column the packed prompts took 46
//    us instead of 37).  A row that a key does not see cannot reach it, whatever it holds.
// Measured: 8192 tokens, 32 heads of 128 on 8: 223 us (0.63 of the measured bf16 rate), of the
// pipes tensor 53%, exponentials 53%, shared memory busy for threads 64% and for the matrix
// unit 51% of the time.  Twelve packed prompts of up to 1500 tokens, 24 heads of 64 on 8, fp16:
// 37 us.  4 x 2048 tokens, 16 heads of 256 on 8: 67 us.
// Every wait is bounded; when one gives up all roles stop, the tile's totals become NaN and the
// status word says so.
#include <algorithm>
#include <cooperative_groups.h>
#include <type_traits>

#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

struct SumMaps {
  CUtensorMap q, k;
};

struct SumJob {
  const float *lse;
  float *totals;
  const int32_t *cu_q, *cu_k, *page_table;
  int64_t table_stride;
  int table_width, n_pages, page_size;
  int n_q, n_k, n_seqs, hq, hkv, group, tile_tokens, window, restart;
  float scale;
  int32_t *status;
};

constexpr int kSumSms = 152;
// CTAs that a call is to have at least, in those that run at once: with 1, 2 and 4 of them 8192 tokens of 32 heads of 128 on
// 8 take 244, 223 and 239 us, twelve packed prompts with 24 heads of 64 on 8 37, 37 and 50, 4 x 2048 tokens of 16 heads of 256 on
// 8 67, 67 and 89, 512 tokens after 8192 of 32 heads of 128 on 8 (where the first CTAs are not the longest) 38, 46 and 63.
constexpr int kSumShare = 2;

// SHORT: of a call whose rows fit one tile, so that a CTA is a chain of waits: more of them, with one stage and buffer.  16
// tokens of 32 heads on 60016 keys of 8 heads of 128 take 65 us with two of each and two CTAs per SM, and 47 us so.
template <int D, bool SHORT>
struct SumCfg {
  static constexpr int kStages = SHORT ? 1 : 2;
  static constexpr int kBufs = SHORT ? 1 : 2;
  static constexpr int kCtas = D == 256 ? 1 : SHORT ? (D == 64 ? 4 : 3) : 2;
  // a warpgroup for the weights of each score buffer
  static constexpr int kSoftWarps = 4 * kBufs, kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
  static constexpr int kThreads = 32 * (kSoftWarps + 2);
  static constexpr uint32_t kTile = kTileRows * D * 2;  // bytes of 128 rows or keys
  static constexpr uint32_t kQOff = kTile;
  static constexpr size_t kSmem = (1 + kStages) * (size_t)kTile + 1024;
  static constexpr uint32_t kTmemCols = kBufs * kTileRows;
  static_assert(kCtas * kTmemCols <= 512, "tensor memory");
};

// The wait for a load from tensor memory, tied to what it loads.
__device__ __forceinline__ void ld_wait32(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// Bits n and up, of 32.
__device__ __forceinline__ uint32_t bits_from(int n) { return n >= 32 ? 0u : 0xffffffffu << max(n, 0); }

// What one CTA works on: a tile of 128 keys of a sequence and key head.
struct SumWork {
  int seq;               // -1: nothing
  int q0, n_q, k0, n_k;  // tokens of the sequence
  int key0;              // first key of the tile
  int head;
  int row0, row1;        // query tokens that see any of its keys
};

template <int D, typename T, bool SHORT>
__global__ void __launch_bounds__(SumCfg<D, SHORT>::kThreads, SumCfg<D, SHORT>::kCtas)
    prompt_weigh_kernel(const __grid_constant__ SumMaps maps, const SumJob j) {
  using C = SumCfg<D, SHORT>;
  constexpr int ST = C::kStages, NB = C::kBufs, DC = D / 64;
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  __shared__ uint64_t k_full, q_full[ST], q_empty[ST], s_full[NB], s_empty[NB], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  __shared__ SumWork s_work;
  __shared__ __align__(16) float s_lse[NB][2][kTileRows];
  __shared__ float s_sum[NB][kTileRows];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  unsigned char *const sm_al = sm_raw + ((1024u - (a_smem(sm_raw) & 1023u)) & 1023u);
  const uint32_t sm = a_smem(sm_al);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == C::kLoadWarp && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &maps.q : &maps.k)));
  if (tid == 0) {
    s_fail = 0;
    a_mbar_init(&k_full, 1);
    for (int i = 0; i < ST; ++i) {
      a_mbar_init(&q_full[i], 1);
      a_mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      a_mbar_init(&s_full[i], 1);
      a_mbar_init(&s_empty[i], 4);
    }
    a_mbar_init(&done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    // The sequence and tile of this CTA, the key heads of a tile side by side.  Tiles far from their sequence's end are seen
    // by most rows: of up to 32 sequences they are taken by that, of more sequence by sequence.
    const int unit = blockIdx.x / ranks, mine = unit / j.hkv;
    const bool look_at_all = blockIdx.x == 0 && j.status;  // (the first CTA tells what is wrong with any offset)
    int before = 0, end = 0;  // tiles of the sequences before; where the latest of their keys end
    bool found = false;
    for (int base = 0; base < j.n_seqs && (!found || look_at_all); base += 32) {
      const int s = base + lane;
      int a = 0, b = 0, c = 0, d = 0, n = 0;
      if (s < j.n_seqs) {
        a = __ldg(j.cu_q + s);
        b = __ldg(j.cu_q + s + 1);
        c = __ldg(j.cu_k + s);
        d = __ldg(j.cu_k + s + 1);
      }
      int last = d;  // the largest end up to this sequence
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, last, o);
        if (lane >= o) last = max(last, v);
      }
      int prev = __shfl_up_sync(0xffffffffu, last, 1);
      prev = lane ? max(prev, end) : end;
      end = max(end, __shfl_sync(0xffffffffu, last, 31));
      if (s < j.n_seqs) {
        // (keys that begin before an earlier sequence's have ended: their tiles would be more than there are CTAs)
        const bool bad = a < 0 || b < a || b > j.n_q || c < 0 || d < c || d > j.n_k || c < prev ||
                         d - c > (int64_t)j.table_width * j.page_size;
        if (bad && look_at_all) atomicOr(j.status, MOE_KV_BAD_LENGTH);
        n = bad ? 0 : (d - c + kTileRows - 1) / kTileRows;
      }
      bool hit = false;
      int tile = 0;
      if (j.n_seqs <= 32) {
        // all sequences' tiles, furthest from their sequence's end first: tiles that are `level` before the last
        auto beyond = [&](int level) { return (int)__reduce_add_sync(0xffffffffu, max(0, n - level)); };
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, n);
        if (mine < beyond(0)) {
          while (hi - lo > 1) {  // beyond(lo) > mine >= beyond(hi)
            const int mid = (lo + hi) / 2;
            if (beyond(mid) > mine) lo = mid;
            else hi = mid;
          }
          const int rank_in = mine - beyond(lo + 1);  // among the sequences that reach this level
          const uint32_t reach = __ballot_sync(0xffffffffu, n > lo);
          hit = n > lo && __popc(reach & ((1u << lane) - 1u)) == rank_in;
        }
        tile = n - 1 - lo;
      } else {
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        hit = mine >= before + inc - n && mine < before + inc;
        tile = mine - (before + inc - n);
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (hit) {
        const int off = (d - c) - (b - a), key0 = tile * kTileRows;
        const int last_key = min(d - c, key0 + kTileRows) - 1;
        // rows stand at off + i; those from key0 on see some of the keys, unless they are a window past the last
        const int row0 = min(b - a, max(0, key0 - off));
        int row1 = b - a;
        if (j.window > 0) row1 = (int)min((int64_t)row1, max((int64_t)row0, (int64_t)last_key + j.window - off));
        s_work = {s, a, b - a, c, d - c, key0, unit % j.hkv, row0, row1};
      }
      found |= __any_sync(0xffffffffu, hit) != 0;
    }
    if (!found && lane == 0) s_work = {-1, 0, 0, 0, 0, 0, 0, 0, 0};
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(a_smem(&s_tmem)), "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // rows of a tile that no token fills are never loaded: they are 0
  const int live_rows = j.group * j.tile_tokens;
  if (live_rows < kTileRows) {
    const int n16 = (kTileRows - live_rows) * 8;  // 16-byte pieces of a chunk of 64 columns
    for (int i = tid; i < ST * DC * n16; i += C::kThreads)
      *reinterpret_cast<uint4 *>(sm_al + C::kQOff + (i / n16) * (kTileRows * 128) + live_rows * 128 + (i % n16) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  p_fence_before();
  __syncthreads();
  p_fence_after();
  const uint32_t tmem = s_tmem;
  const SumWork w = s_work;
  // this CTA's tiles of rows: every ranks-th
  const int all_tiles = w.seq < 0 ? 0 : (w.row1 - w.row0 + j.tile_tokens - 1) / j.tile_tokens;
  const int n_tiles = all_tiles > rank ? (all_tiles - rank + ranks - 1) / ranks : 0;
  auto first_token = [&](int i) { return w.row0 + (rank + i * ranks) * j.tile_tokens; };
  // A thread's key's total and what it was: looked up ahead, as it is a chain of loads.
  float *to = nullptr;
  float before = 0.f;
  if (rank == 0 && w.seq >= 0 && tid < kTileRows && w.key0 + tid < w.n_k && (all_tiles > 0 || j.restart)) {
    const int key = w.key0 + tid;
    int in_page = 0;
    const int p = kv_page(j.page_table + (int64_t)w.seq * j.table_stride, j.table_width, j.n_pages, j.page_size, key / kKvTile,
                          &in_page);
    if (p >= 0) {
      to = j.totals + ((int64_t)p * j.hkv + w.head) * j.page_size + in_page * kKvTile + key % kKvTile;
      if (!j.restart && key < w.n_k - w.n_q) before = *to;
    } else if (j.status) {
      atomicOr(j.status, MOE_KV_BAD_PAGE);
    }
  }

  if (warp == C::kLoadWarp) {
    if (lane == 0 && n_tiles > 0) {
      bool ok = true;
      a_expect_tx(&k_full, C::kTile);
      for (int c = 0; c < DC; ++c) p_tma_3d(sm + c * kTileRows * 128, &maps.k, 64 * c, w.head, w.k0 + w.key0, &k_full);
      int n_loaded = 0;
      for (int i = 0; i < n_tiles; ++i) {
        const int st = i % ST;
        if (i >= ST && !(ok = a_mbar_wait(&q_empty[st], (uint32_t)(i / ST - 1) & 1u, &s_fail))) break;
        a_expect_tx(&q_full[st], (uint32_t)(DC * live_rows) * 128u);
        for (int c = 0; c < DC; ++c)
          p_tma_3d(sm + C::kQOff + st * C::kTile + c * kTileRows * 128, &maps.q, 64 * c, w.head * j.group, w.q0 + first_token(i),
                   &q_full[st]);
        n_loaded = i + 1;
      }
      if (!ok) s_fail = 1;
      // no copy may be in flight when the CTA leaves
      (void)a_mbar_drain(&k_full, 0);
      for (int i = max(0, n_loaded - ST); i < n_loaded; ++i) (void)a_mbar_drain(&q_full[i % ST], (uint32_t)(i / ST) & 1u);
    }
  } else if (warp == C::kMmaWarp) {
    if (n_tiles > 0) {
      const bool one = elect_one();
      constexpr uint32_t id = p_idesc<T>(kTileRows, false);
      auto wait = [&](uint64_t *bar, uint32_t ph) { return __all_sync(0xffffffffu, a_mbar_wait(bar, ph, &s_fail)) != 0; };
      bool ok = wait(&k_full, 0);
      const uint64_t a0 = p_desc_k(sm);
      for (int i = 0; i < n_tiles && ok; ++i) {
        const int st = i % ST, buf = i % NB;
        if (i >= NB && !(ok = wait(&s_empty[buf], (uint32_t)(i / NB - 1) & 1u))) break;
        if (!(ok = wait(&q_full[st], (uint32_t)(i / ST) & 1u))) break;
        p_fence_after();
        const uint64_t b0 = p_desc_k(sm + C::kQOff + st * C::kTile);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t at = (kk / 4) * (kTileRows * 128 / 16) + (kk % 4) * 2;
            p_mma_ss(tmem + buf * kTileRows, a0 + at, b0 + at, id, kk > 0);
          }
          p_commit(&s_full[buf]);
          p_commit(&q_empty[st]);
        }
        __syncwarp();
      }
      if (!ok) s_fail = 1;
      // no product may be running when the CTA gives its memory back
      if (one) p_commit(&done);
      __syncwarp();
      (void)a_mbar_drain(&done, 0);
      __syncwarp();
    }
  } else {
    // ---- weights: thread = key; warpgroup `buf` has the tiles of that buffer
    const int buf = warp / 4, r = tid & 127;
    const int key = w.key0 + r, off = w.n_k - w.n_q, last_key = min(w.n_k, w.key0 + kTileRows) - 1;
    const int back = j.window > 0 ? j.window : 0x7fffffff;
    const uint32_t s_col = tmem + ((uint32_t)(warp & 3) << 21) + buf * kTileRows;  // 32 (warp % 4) in the lane field
    const int r_tok = r / j.group, r_head = w.head * j.group + r % j.group;
    bool ok = true;
    float total = 0.f;
    // the lse of row r of a tile (infinity for a row that is none)
    auto lse_of = [&](int i) {
      const int tok = first_token(i) + r_tok;
      return r < live_rows && tok < w.row1 ? __ldg(j.lse + (int64_t)(w.q0 + tok) * j.hq + r_head) : a_inf();
    };
    // for the warpgroup: less the lse (of a row that is none: less infinity)
    auto put_lse = [&](int at, float l) {
      s_lse[buf][at][r] = -l;
      asm volatile("bar.sync %0, 128;" ::"r"(1 + buf) : "memory");
    };
    if (buf < n_tiles) put_lse(0, lse_of(buf));
    const uint64_t scale2 = f2_pack(j.scale, j.scale), log2e2 = f2_pack(kLog2e, kLog2e);
    // 32 columns' weights, of those whose bit is set in `seen`, added to sum.  (No other branch within a tile: it would leave
    // less to overlap.)
    auto weigh = [&](const float *v, const float *ls, uint32_t seen, uint64_t (&sum)[2], auto is_masked) {
#pragma unroll
      for (int z = 0; z < 32; z += 4) {
        const float4 l4 = *reinterpret_cast<const float4 *>(ls + z);
        float a, b, c, d;
        f2_unpack(f2_mul(f2_fma(f2_pack(v[z], v[z + 1]), scale2, f2_pack(l4.x, l4.y)), log2e2), a, b);
        f2_unpack(f2_mul(f2_fma(f2_pack(v[z + 2], v[z + 3]), scale2, f2_pack(l4.z, l4.w)), log2e2), c, d);
        if constexpr (decltype(is_masked)::value) {
          a = (seen >> z) & 1u ? a : -a_inf();
          b = (seen >> (z + 1)) & 1u ? b : -a_inf();
          c = (seen >> (z + 2)) & 1u ? c : -a_inf();
          d = (seen >> (z + 3)) & 1u ? d : -a_inf();
        }
        sum[0] = f2_add(sum[0], f2_pack(a_exp2(a), a_exp2(b)));
        sum[1] = f2_add(sum[1], f2_pack(a_exp2(c), a_exp2(d)));
      }
    };
    // A tile's 128 columns, the first `plain` 32s of them not masked, of the others those of [c0, c1) seen.
    auto tile = [&](const float *ls, int c0, int c1, uint64_t (&sum)[2], auto plain) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v[32];
        p_ld32(s_col + 32 * x, v);
        ld_wait32(v);
        if (x == 3) {
          // (all scores are in registers)
          p_fence_before();
          __syncwarp();
          if (lane == 0) a_mbar_arrive(&s_empty[buf]);
        }
        if (x < decltype(plain)::value) {
          weigh(v, ls + 32 * x, 0u, sum, std::false_type());
        } else {
          const uint32_t seen = bits_from(c0 - 32 * x) & ~bits_from(c1 - 32 * x);
          // (in tiles on the border there are 32s that none of the warp's keys is seen by)
          if (decltype(plain)::value || __any_sync(0xffffffffu, seen != 0)) weigh(v, ls + 32 * x, seen, sum, std::true_type());
        }
      }
    };
    for (int i = buf, n = 0; i < n_tiles; i += NB, ++n) {
      float l = 0.f;
      if (i + NB < n_tiles) l = lse_of(i + NB);
      // (after a failure the warp goes on to the barrier, which counts all four)
      ok = ok && __all_sync(0xffffffffu, a_mbar_wait(&s_full[buf], (uint32_t)n & 1u, &s_fail)) != 0;
      if (!ok) s_fail = 1;
      if (ok) {
        p_fence_after();
        const int t0 = first_token(i), t1 = min(w.row1, t0 + j.tile_tokens) - 1;  // the tile's tokens
        const bool whole = off + t0 >= last_key && (int64_t)off + t1 - back < w.key0 && t1 - t0 + 1 == j.tile_tokens;
        const float *ls = s_lse[buf][n & 1];
        // the columns whose tokens see this thread's key: tokens stand in their order, `group` columns each
        const int c0 = min(max(key - off - t0, 0), kTileRows) * j.group;
        const int c1 = (int)min((int64_t)(t1 - t0 + 1), max((int64_t)0, (int64_t)key + back - off - t0)) * j.group;
        uint64_t sum[2] = {0, 0};
        if (whole && live_rows == kTileRows) tile(ls, c0, c1, sum, std::integral_constant<int, 4>());
        else if (whole && live_rows >= 96) tile(ls, c0, c1, sum, std::integral_constant<int, 3>());
        else tile(ls, c0, c1, sum, std::integral_constant<int, 0>());
        float a, b;
        f2_unpack(f2_add(sum[0], sum[1]), a, b);
        total += a + b;
      }
      put_lse((n + 1) & 1, l);
    }
    s_sum[buf][r] = ok ? total : a_nan();
  }
  p_fence_before();
  __syncthreads();
  if (s_fail && tid == 0 && j.status) atomicOr(j.status, MOE_KV_TIMED_OUT);
  if (warp == C::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
  if (ranks > 1) cluster.sync();
  if (to) {
    float total = 0.f;
    for (int r = 0; r < ranks; ++r) {
      const float *sum = ranks > 1 ? cluster.map_shared_rank(&s_sum[0][tid], r) : &s_sum[0][tid];
#pragma unroll
      for (int b = 0; b < NB; ++b) total += sum[b * kTileRows];
    }
    *to = before + total;
  }
  if (ranks > 1) cluster.sync();  // (the sums are read until here)
}

template <int D, typename T, bool SHORT>
int run_sum(const SumJob &j, const moe_tensor &q, const moe_tensor &k, int dtype, cudaStream_t st) {
  using C = SumCfg<D, SHORT>;
  static DynSmemLimit limit;
  if (ensure_dyn_smem(prompt_weigh_kernel<D, T, SHORT>, C::kSmem, limit) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  SumMaps maps;
  if (!encode_map(&maps.q, q, std::max(1, j.n_q), j.hq, D, j.group, j.tile_tokens, dtype) ||
      !encode_map(&maps.k, k, j.n_k, j.hkv, D, 1, kTileRows, dtype))
    return MOE_ERR_INVALID_ARG;
  // at most this many tiles of keys: a sequence's last one may be partly filled
  const int64_t units = ((int64_t)j.n_k / kTileRows + std::min<int64_t>(j.n_seqs, j.n_k)) * j.hkv;
  if (units * 8 > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  // A tile's rows are shared by a cluster, so that the longest tile is no more than a part of what an SM gets of all:
  // a causal sequence's first tile has twice the mean.  Never more CTAs than tiles of rows for their warpgroups.
  int ranks = 1;
  while (ranks < 8 && units * ranks < (int64_t)kSumShare * kSumSms * C::kCtas && (int64_t)ranks * 2 * C::kBufs * j.tile_tokens <= j.n_q)
    ranks *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ranks));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prompt_weigh_kernel<D, T, SHORT>, maps, j) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

template <int D, typename T>
int launch_sum(const SumJob &j, const moe_tensor &q, const moe_tensor &k, int dtype, cudaStream_t st) {
  return j.n_q <= j.tile_tokens ? run_sum<D, T, true>(j, q, k, dtype, st) : run_sum<D, T, false>(j, q, k, dtype, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int moe_prompt_weigh(const moe_tensor *q, int32_t n_q_tokens, int32_t n_q_heads, const moe_tensor *k,
                             int32_t n_k_tokens, int32_t n_kv_heads, int32_t head_dim, const int32_t *cu_q,
                             const int32_t *cu_k, int32_t n_seqs, float scale, int32_t window, const float *lse,
                             const int32_t *page_table, int64_t table_stride, int32_t table_width, int32_t n_pages,
                             int32_t page_size, float *totals, int32_t restart, int32_t dtype, int32_t *status,
                             void *cuda_stream) {
  if (n_q_tokens < 0 || n_k_tokens < 0 || n_seqs < 0 || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads ||
      window < 0 || !(scale > 0.f && scale <= kMostScale) || table_width < 0 || n_pages < 0)
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  const int group = n_q_heads / n_kv_heads;
  if (!kv_sizes_ok(n_kv_heads, head_dim, page_size) || n_q_heads > kMaxAttnHeads || group > 64 ||
      n_q_tokens > (1 << 29) || n_k_tokens > (1 << 29) || (int64_t)table_width * page_size > (1 << 30))
    return MOE_ERR_UNSUPPORTED;
  if (n_seqs == 0 || n_k_tokens == 0) return MOE_OK;
  if (!cu_q || !cu_k || (!totals && n_pages > 0) || (uintptr_t)totals % 4 || (uintptr_t)lse % 4 || (uintptr_t)status % 4 ||
      (n_q_tokens > 0 && !lse) || (table_width > 0 && (!page_table || table_stride < table_width)))
    return MOE_ERR_INVALID_ARG;
  if (n_q_tokens > 0)
    if (const int rc = check_tensor(q, 2)) return rc;
  if (const int rc = check_tensor(k, 2)) return rc;
  SumJob j = {};
  j.lse = lse;
  j.totals = totals;
  j.cu_q = cu_q;
  j.cu_k = cu_k;
  j.page_table = page_table;
  j.table_stride = table_stride;
  j.table_width = table_width;
  j.n_pages = n_pages;
  j.page_size = page_size;
  j.n_q = n_q_tokens;
  j.n_k = n_k_tokens;
  j.n_seqs = n_seqs;
  j.hq = n_q_heads;
  j.hkv = n_kv_heads;
  j.group = group;
  j.tile_tokens = kTileRows / group;
  j.window = window;
  j.restart = restart != 0;
  j.scale = scale;
  j.status = status;
  // without queries none are loaded, but the map wants an address and a size
  if (n_q_tokens == 0 && !j.restart) return MOE_OK;
  const moe_tensor qt = n_q_tokens > 0 ? *q : moe_tensor{k->data, head_dim, head_dim};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  if (dtype == MOE_BF16)
    return head_dim == 64    ? launch_sum<64, __nv_bfloat16>(j, qt, *k, dtype, st)
           : head_dim == 128 ? launch_sum<128, __nv_bfloat16>(j, qt, *k, dtype, st)
                             : launch_sum<256, __nv_bfloat16>(j, qt, *k, dtype, st);
  return head_dim == 64    ? launch_sum<64, __half>(j, qt, *k, dtype, st)
         : head_dim == 128 ? launch_sum<128, __half>(j, qt, *k, dtype, st)
                           : launch_sum<256, __half>(j, qt, *k, dtype, st);
}
