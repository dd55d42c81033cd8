// Keeping the cached tokens that have received most attention weight, and moving them together.
//
// Per sequence of n > budget tokens and key head: the first `first` and the last `recent`
// tokens stay, and of those between the budget - first - recent with the largest totals
// (ties: the earlier token), all in their order, in the slots [0, budget).
//
// Choosing: a radix search for the smallest total that stays, 11, 11 and 10 bits of a key
// that orders like the value, by a cluster of CTAs per (sequence, head): each holds its part
// of the keys in shared memory, counts are added over the cluster's shared memory.  Then the
// kept tokens' numbers are written in order, from counts per warp.
//
// Moving, in place: the token of rank r goes to slot r, which is never after its own.  A CTA
// takes the 256 slots of a group: it loads what is to go there into registers, says so, waits
// for the groups that load from its own 256 slots to have said so (at most two, and none
// later than itself), and writes.  Groups are handed out in order, so whatever one waits for
// has been begun by a CTA that is running, and loading waits for nothing.
//
// Bound: memory (the kept tokens' bytes read and written; 16-byte pieces of neighbouring
// tokens, so that most of every sector read is of use), the totals, and for a short cache
// the chain of two launches.
#include <algorithm>
#include <cooperative_groups.h>

#include "attn_common.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostHeld = 49152;  // keys that a CTA's shared memory holds (more are read again for every pass)
constexpr int kMoveThreads = 256;
constexpr int kSlots = 256;       // slots of a group
constexpr int kEvictSms = 152;

struct EvictJob {
  moe_kv_cache c;
  const int32_t *lens;
  float *totals;
  int budget, first, recent, heads;
  int32_t *new_lens, *kept;
  // workspace: next group; per pair whether it stays as it is; per pair and group: the kept tokens before its slots, and
  // whether what goes there has been loaded
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

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictJob j) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kBins];
  __shared__ int s_bad, s_bin, s_above, s_warp[2][kSelectWarps], s_count[2], s_scan[kSelectWarps];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int pair = blockIdx.x / ranks, seq = pair / j.heads, head = pair % j.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = __ldg(j.lens + seq);
  int32_t *kept = j.kept + (int64_t)pair * j.budget;
  if (blockIdx.x == 0 && tid == 0) *j.ticket = 0;
  const bool ok = length_ok(j, n);
  if (!ok || n <= j.budget) {  // (all CTAs of the cluster alike)
    for (int i = rank * kSelectThreads + tid; i < j.budget; i += ranks * kSelectThreads) kept[i] = ok && i < n ? i : -1;
    if (rank == 0 && tid == 0) {
      j.skip[pair] = 1;
      if (head == 0) j.new_lens[seq] = n;
      if (!ok && j.c.status) atomicOr(j.c.status, MOE_KV_BAD_LENGTH);
    }
    return;
  }
  const int32_t *row = j.c.page_table + (int64_t)seq * j.c.table_stride;
  const int per = ((n + ranks - 1) / ranks + 31) / 32 * 32, a = min(n, rank * per), b = min(n, a + per);
  const bool hold = per <= j.held;
  auto load = [&](int i) {  // the key of token i; a token without a page has none
    const int slot = i / j.c.page_size;
    const int p = __ldg(row + slot);
    if (p < 0 || p >= j.c.n_pages) {
      s_bad = 1;
      return 0u;
    }
    return total_key(j.totals[((int64_t)p * j.heads + head) * j.c.page_size + (i - slot * j.c.page_size)]);
  };
  auto key = [&](int i) { return hold ? keys[i - a] : load(i); };
  if (tid == 0) s_bad = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = a + tid; i < b; i += kSelectThreads) {
    const uint32_t k = load(i);
    if (hold) keys[i - a] = k;
  }
  for (int g = rank * kSelectThreads + tid; g < (n + kSlots - 1) / kSlots; g += ranks * kSelectThreads)
    j.loaded[(int64_t)pair * j.groups + g] = 0;
  cluster.sync();
  bool bad = false;
  for (int r = 0; r < ranks; ++r) bad |= *cluster.map_shared_rank(&s_bad, r) != 0;
  if (bad) {
    for (int i = rank * kSelectThreads + tid; i < j.budget; i += ranks * kSelectThreads) kept[i] = -1;
    if (rank == 0 && tid == 0) {
      j.skip[pair] = 1;
      if (head == 0) j.new_lens[seq] = n;
      if (j.c.status) atomicOr(j.c.status, MOE_KV_BAD_PAGE);
    }
    cluster.sync();  // (the others look at this one's word)
    return;
  }
  // ---- the smallest key that stays, and how many of that key
  const int c0 = j.first, c1 = n - j.recent;  // tokens that may go
  int need = j.budget - j.first - j.recent;
  uint32_t least = 0;
  const bool some = need > 0;
  if (some) {
    int done = 0;  // bits found
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = 32 - done - bits;
      for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int i = max(a, c0) + tid; i < min(b, c1); i += kSelectThreads) {
        const uint32_t k = key(i);
        if (done == 0 || (k >> (shift + bits)) == least) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      cluster.sync();
      // counts over the cluster, largest key first: this thread's two bins
      const int hi = kBins - 1 - 2 * tid;
      int n0 = 0, n1 = 0;
      for (int r = 0; r < ranks; ++r) {
        const uint32_t *h = cluster.map_shared_rank(hist, r);
        n0 += (int)h[hi];
        n1 += (int)h[hi - 1];
      }
      int inc = n0 + n1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s_scan[warp] = inc;
      __syncthreads();
      if (warp == 0) {
        int v = s_scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += u;
        }
        s_scan[lane] = v;
      }
      __syncthreads();
      const int before = inc - n0 - n1 + (warp ? s_scan[warp - 1] : 0);
      if (before < need && before + n0 >= need) {
        s_bin = hi;
        s_above = before;
      } else if (before + n0 < need && before + n0 + n1 >= need) {
        s_bin = hi - 1;
        s_above = before + n0;
      }
      cluster.sync();  // (no CTA's counts are needed any more)
      least = (least << bits) | (uint32_t)s_bin;
      need -= s_above;
      done += bits;
      __syncthreads();
    }
  }
  // ---- the kept tokens in order: a warp takes neighbouring steps of 32; first their counts
  const int steps = (b - a + 31) / 32, w0 = (int)((int64_t)steps * warp / kSelectWarps), w1 = (int)((int64_t)steps * (warp + 1) / kSelectWarps);
  auto more = [&](int i) { return some && i >= c0 && i < c1 && i < b && key(i) > least; };
  auto equal = [&](int i) { return some && i >= c0 && i < c1 && i < b && key(i) == least; };
  int gt = 0, eq = 0;
  for (int s = w0; s < w1; ++s) {
    const int i = a + 32 * s + lane;
    gt += more(i);
    eq += equal(i);
  }
  gt = (int)__reduce_add_sync(0xffffffffu, gt);
  eq = (int)__reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (warp < 2) {
    int v = s_warp[warp][lane];
    const int own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    s_warp[warp][lane] = v - own;
    if (lane == 31) s_count[warp] = v;
  }
  cluster.sync();
  gt = s_warp[0][warp];
  eq = s_warp[1][warp];
  for (int r = 0; r < rank; ++r) {
    const int *c = cluster.map_shared_rank(s_count, r);
    gt += c[0];
    eq += c[1];
  }
  int32_t *group_before = j.before + (int64_t)pair * j.groups;
  {
    const int start = a + 32 * w0;
    int at = min(start, c0) + max(0, start - c1) + gt + min(eq, need);  // kept tokens before the step
    for (int s = w0; s < w1; ++s) {
      const int i = a + 32 * s + lane;
      const uint32_t eqs = __ballot_sync(0xffffffffu, equal(i));
      const bool stay = i < b && (i < c0 || i >= c1 || more(i) ||
                                  (equal(i) && eq + __popc(eqs & ((1u << lane) - 1u)) < need));
      const uint32_t stays = __ballot_sync(0xffffffffu, stay);
      if (lane == 0 && (a + 32 * s) % kSlots == 0) group_before[(a + 32 * s) / kSlots] = at;
      if (stay) kept[at + __popc(stays & ((1u << lane) - 1u))] = i;
      at += __popc(stays);
      eq += __popc(eqs);
    }
  }
  if (rank == 0 && tid == 0) {
    group_before[(n + kSlots - 1) / kSlots] = j.budget;
    j.skip[pair] = 0;
    if (head == 0) j.new_lens[seq] = j.budget;
  }
  cluster.sync();  // (a CTA's counts are read by those after it)
}

__device__ __forceinline__ uint4 e_load16(const unsigned char *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool wait_loaded(const uint32_t *flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < kAttnSpin; ++i) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v) return true;
    if ((i & 255u) == 255u) {
      const uint64_t now = a_now_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kAttnWaitNs) return false;
    }
  }
  return false;
}

// A token's bytes: codes of keys and values, block by block, their scales, and its total.
template <int D>
struct TokenBytes {
  uint4 codes[2][D / 32];
  uint32_t scales[2][D / 64];
  float total;
};

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictJob j) {
  __shared__ int s_seq, s_head, s_group, s_ok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (j.c.n_seqs + 31) / 32;
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
        if (length_ok(j, n) && n > j.budget) mine += (int64_t)((n + kSlots - 1) / kSlots) * j.heads;
      }
      before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= mine;
      u = __shfl_sync(0xffffffffu, u, 0);
      if (lane == 0) s_seq = -1;
      __syncwarp();
      if ((int64_t)u >= before && (int64_t)u < before + mine) {
        int64_t left = (int64_t)u - before;
        for (int k = 0; k < per; ++k) {
          const int s = lane * per + k, n = __ldg(j.lens + s);
          const int64_t of = length_ok(j, n) && n > j.budget ? (int64_t)((n + kSlots - 1) / kSlots) * j.heads : 0;
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
    if (j.skip[pair]) {
      __syncthreads();
      continue;
    }
    const int n = __ldg(j.lens + seq), slot = g * kSlots + tid;
    const int32_t *row = j.c.page_table + (int64_t)seq * j.c.table_stride;
    const int src = slot < j.budget ? j.kept[(int64_t)pair * j.budget + slot] : -1;
    const bool moves = src > slot, clears = slot >= j.budget && slot < n;
    uint32_t *loaded = j.loaded + (int64_t)pair * j.groups;
    unsigned char *const pages = static_cast<unsigned char *>(j.c.pages);
    // where a token's tile is, and the token in it; the page was seen to be there
    auto place = [&](int i, int64_t *tile, int64_t *total) {
      const int at = i / j.c.page_size, in = i - at * j.c.page_size;
      const int64_t p = __ldg(row + at);
      *tile = p * j.c.page_stride + kv_tile_off(D, j.c.page_size, head, in / kKvTile);
      *total = (p * j.heads + head) * j.c.page_size + in;
      return in % kKvTile;
    };
    TokenBytes<D> x;
    if (moves) {
      int64_t tile, total;
      const int tok = place(src, &tile, &total);
      const unsigned char *tp = pages + tile;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b) x.codes[v][b] = e_load16(tp + kv_code_off(D, v, b, tok));
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          x.scales[v][b] = *reinterpret_cast<const volatile uint32_t *>(tp + kv_scale_off(D, v, 2 * b, tok));
      }
      x.total = *const_cast<const volatile float *>(j.totals + total);
    }
    __threadfence();
    const bool work = __syncthreads_or(moves || clears);
    if (tid == 0) {
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(loaded + g), "r"(1u) : "memory");
      s_ok = 1;
    }
    if (!work) continue;
    __syncthreads();
    if (warp == 0) {
      // who loads from these slots: the groups of the ranks that their tokens have (256 at most)
      const int r0 = j.before[(int64_t)pair * j.groups + g], r1 = j.before[(int64_t)pair * j.groups + g + 1];
      const int h = r0 / kSlots + lane;
      if (r1 > r0 && h <= (r1 - 1) / kSlots && h < g && !wait_loaded(loaded + h)) s_ok = 0;
    }
    __syncthreads();
    if (!s_ok) {
      if (tid == 0 && j.c.status) atomicOr(j.c.status, MOE_KV_TIMED_OUT);
      __syncthreads();
      continue;
    }
    __threadfence();
    if (moves || clears) {
      int64_t tile, total;
      const int tok = place(slot, &tile, &total);
      if (moves) {
        unsigned char *tp = pages + tile;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
          for (int b = 0; b < D / 32; ++b) *reinterpret_cast<uint4 *>(tp + kv_code_off(D, v, b, tok)) = x.codes[v][b];
#pragma unroll
          for (int b = 0; b < D / 64; ++b) *reinterpret_cast<uint32_t *>(tp + kv_scale_off(D, v, 2 * b, tok)) = x.scales[v][b];
        }
      }
      j.totals[total] = moves ? x.total : 0.f;
    }
    __syncthreads();
  }
}

template <int D>
int launch_move(const EvictJob &j, int64_t groups, cudaStream_t st) {
  const int grid = (int)std::min<int64_t>(groups, kEvictSms * (D == 256 ? 2 : 4));
  evict_move_kernel<D><<<grid, kMoveThreads, 0, st>>>(j);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int64_t evict_groups(const moe_kv_cache *c) { return ((int64_t)c->table_width * c->page_size + kSlots - 1) / kSlots + 1; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int64_t moe_kv_evict_workspace(const moe_kv_cache *c) {
  if (check_cache(c) != MOE_OK || (int64_t)c->table_width * c->page_size > 0x7fffffff) return 0;
  return 256 + (int64_t)c->n_seqs * c->n_kv_heads * (4 + 8 * evict_groups(c));
}

MOE_API int moe_kv_evict(const moe_kv_cache *c, const int32_t *seq_lens, float *totals, int32_t budget, int32_t first,
                         int32_t recent, int32_t *new_lens, int32_t *kept, void *workspace, int64_t workspace_bytes,
                         void *cuda_stream) {
  if (c && c->n_seqs == 0) return MOE_OK;
  if (const int rc = check_cache(c)) return rc;
  if (!seq_lens || !totals || !new_lens || budget < 0 || first < 0 || recent < 0 || (int64_t)first + recent > budget ||
      (!kept && budget > 0) || (uintptr_t)totals % 4 || (uintptr_t)kept % 4 || (uintptr_t)new_lens % 4)
    return MOE_ERR_INVALID_ARG;
  if ((int64_t)c->table_width * c->page_size > 0x7fffffff || (int64_t)c->n_seqs * c->n_kv_heads > 0x7fffffff / 8)
    return MOE_ERR_UNSUPPORTED;
  if (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < moe_kv_evict_workspace(c)) return MOE_ERR_INVALID_ARG;
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
  // a cluster per pair, of as many CTAs as there is room for and keys to count
  int ranks = 1;
  while (ranks < 8 && pairs * ranks < 2 * kEvictSms && tokens > 2048 * (int64_t)ranks) ranks *= 2;
  j.held = (int)std::min<int64_t>(kMostHeld, ((tokens + ranks - 1) / ranks + 31) / 32 * 32);
  cudaStream_t st = (cudaStream_t)cuda_stream;
  static DynSmemLimit limit;
  const size_t smem = (size_t)j.held * 4;
  // (raised from 32 KB on: the kernel's own arrays count towards what needs no raising)
  if (ensure_dyn_smem(evict_select_kernel, smem > 32 * 1024 ? std::max<size_t>(smem, 64 * 1024) : smem, limit) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * ranks));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, j) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  if (tokens <= budget) return MOE_OK;  // no sequence is over it
  const int64_t groups = pairs * (j.groups - 1);
  return c->head_dim == 64 ? launch_move<64>(j, groups, st) : c->head_dim == 128 ? launch_move<128>(j, groups, st) : launch_move<256>(j, groups, st);
}
