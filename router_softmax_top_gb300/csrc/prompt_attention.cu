// Causal attention over whole prompts, packed one after another, on the 5th-gen
// tensor cores.
//
// o_i = sum_j 2^(t_ij - r_i) v_j / sum_j 2^(t_ij - r_i), t = scale log2(e) q_i . k_j,
// over the keys that row i sees, in one pass over the keys.  A block's weights are formed
// with the reference as it stands; only if their sum exceeds 2^8 (fp16: 2^14; no weight of
// a smaller sum is larger) is the block's largest score looked for and the reference moved to it,
// and the sums so far scale.
//
// Bound: the tensor cores, 4 D flops per (query, key) pair and head; beside them an
// exponential per pair and head, which the same SM does at about the rate that the
// matrices allow.  So both have to run at once:
//  * A CTA works on NQ tiles of 128 rows (two where tensor memory holds two score
//    tiles and two outputs, D <= 128).  While one tile's scores are turned into
//    weights by its own four warps, the other tile's products run.  At D = 256 one
//    tile with two score buffers takes turns.
//  * A row is (token, head): the heads that share a key head are rows of the same
//    tile, 128 / group tokens of each, so keys and values are loaded once for all of
//    them and the diagonal cuts off at most that many tokens' worth of work.
//  * Q K^T: both operands K-major in shared memory (TMA, 128-byte swizzle), scores in
//    tensor memory.  A thread owns a row: it loads its scores, forms weights and their
//    sum in registers without any shuffle, and writes the weights (16 bits) over them.
//  * P V: weights from tensor memory, values from shared memory as the TMA left them
//    (the contraction runs across their rows: an MN-major operand), output
//    accumulated in tensor memory across all key blocks.
//  * One warp issues all matrix instructions in an order in which every product of
//    one tile has the other tile's exponentials behind it; one thread loads.  What the
//    issuing warp waits for is time that the tensor cores lose, as their queue is short:
//    it waits once per product, on the weights' barrier, which a helper holds back
//    until the keys and values are there too.
// Measured: 8192 tokens, 32 heads of 128 on 8: 357 us in short runs and 382 in long ones,
// 1.54 and 1.44 PFLOP/s or 0.80 and 0.75 of the measured bf16 rate (454 us with
// descriptors outside uniform registers, 393 us with four waits and six commits per
// block).  The tensor pipe is active 65% of all cycles; in the loop a block takes ~2700
// cycles, 2048 of them matrix instructions at their full rate, and a CTA's ends about a
// tenth of its time.  Heads of 64 (twelve packed prompts 61 us, their products alone 15)
// fill no pipe: tensor cores and exponentials a quarter each, issue slots 42%.  Their warps
// wait, for scores to arrive from tensor memory and for each other; a block has 64 keys,
// so half the work between two waits, and CTAs are short.  Two CTAs per SM fill some of
// that (75 -> 68 us, in the order of the sequences).  Heads of 256 have one row tile: their
// queries are moved to tensor memory, where they do not take a third of the shared
// memory's bandwidth, and their place holds a third stage of keys and values (a block of
// 64 keys takes 0.78 us so,
// 0.92 before; its products alone take 0.55: 32 cycles each of 64 keys with queries from
// tensor memory, 48 from shared memory).  Neither the exponentials nor their chain bound
// it: two threads per row took 0.79 us, weights through shared memory, so that scores run
// two blocks ahead, 0.87.  What is left are the copies, 64 KB per block, 44 bytes per cycle.
// Few rows with many keys do not fill the GPU: their keys are shared out over several CTAs (below).
// Two issuing warps (one per tile) were slower (422 us), as were handing the weights on
// in two parts and testing barriers before suspending on them.
// Blocks of keys that no row of a tile sees are skipped; only blocks that a row sees in
// part are masked.  A masked weight is an exact 0; since 0 x infinity and 0 x NaN are not,
// a row whose result is not finite although its sum is gets its result again from the
// keys it sees, one by one (never in ordinary data).
// Every wait is bounded; when one gives up all roles stop, rows become NaN and the
// status word says so.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_common.cuh"

namespace moe {
namespace {

constexpr int kTileRows = 128;
constexpr float kFar = 1024.f;  // log2 units

struct PromptMaps {
  CUtensorMap q, k, v;
};

struct PromptJob {
  moe_tensor q, k, v;
  const int32_t *cu_q, *cu_k;
  int n_q, n_k, n_seqs, hq, hkv, group, tile_tokens, window;
  float scale;
  void *out;
  float *lse;
  int32_t *status;
  // for sharing out keys (see kMinPart): CTAs that run at once, or 0 for no sharing; most parts of a group
  int slots, most_parts;
  float *part;      // [slots]: sums of a part
  uint32_t *count;  // [slots]: parts of a group that are done
};

// Where a call's tile groups leave half the GPU idle or more, each group's keys are shared out over as many CTAs as there
// is room for, and the last one done joins the parts.  It reads a part in about the time of a block, so there are no more
// parts than a part has blocks.  Whole and shared, 32 heads of 128 on 8: 16 tokens after 1000 15.9 and 15.4 us, 37 after
// 2000 29 and 22, 512 after 4096 57 and 45, 256 after 60,000 645 and 185, 5 after 100,000 968 and 77 us.
// A part has at least kMinPart blocks (parts of 4 blocks of 64, 512 tokens: heads of 64 17.4 us, whole 13.8; heads of 256
// 22.3, whole 14.2), and, where two parts are on the same SM (heads of 64), at least kMinPair (2 of 8, 1024 tokens: 24.0,
// whole 20.6; 2 of 16, 1024 after 1024: 32.8, whole 33.1; 2 of 24, 16 sequences of 7 after 3000: 33.1, whole 41.6).
// Groups of a last, partly filled wave are not shared: 300 tokens after 3000 of 4 sequences, window 1024, took 43.8 us so
// and 41.2 whole, 777 and 1024 after 4096 of heads of 256 74.3 and 76.2 (with queries in shared memory).
template <int D>
constexpr int kMinPart = D == 128 ? 4 : 6;
constexpr int kMinPair = 12;
constexpr int kMostParts = 32;
constexpr int kMaxSplitSeqs = 32;  // (those whose groups are counted by one warp at once)

template <int D>
struct PromptCfg {
  static constexpr int kNQ = D == 256 ? 1 : 2;         // row tiles
  static constexpr int kBuf = 2;                       // score buffers (one per tile, or two of the one tile)
  static constexpr int kBK = D == 128 ? 128 : 64;      // keys of a block
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 2 : 3;  // of keys, and of values
  static constexpr bool kQTmem = D == 256;             // queries in tensor memory (of two tiles it has no room for them)
  static constexpr uint32_t kQBytes = kTileRows * D * 2, kKBytes = kBK * D * 2;
  static constexpr uint32_t kKOff = kQTmem ? 0 : kNQ * kQBytes, kVOff = kKOff + kStages * kKBytes,
                            kQOff = kQTmem ? kVOff : 0;  // (on their way to tensor memory: where values come later)
  // a part of a shared group: its sums as [tile][D / 4][128 rows] of 4, then per row its reference and weight sum
  static constexpr size_t kSums = (size_t)kNQ * kTileRows * D, kPart = kSums + 2 * kNQ * kTileRows;
  static constexpr size_t kSmem = kVOff + kStages * kKBytes + 1024;
  // tensor memory: score buffers, then outputs, then queries
  static constexpr uint32_t kOCol = kBuf * kBK, kQCol = kOCol + kNQ * D;
  static constexpr int kSoftWarps = 4 * kNQ, kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1,
                       kReadyWarp = kSoftWarps + 2,  // (two tiles only)
                       kCheckWarp = kSoftWarps + 3;  // (at the start of the first CTA only)
  // a warpgroup for these (a register split goes by warpgroups)
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  // registers per thread: what 384 threads can have at launch, then split; 256 threads need no split
  static constexpr int kCtas = D == 64 ? 2 : 1;  // on an SM: what one CTA waits for at its ends, the other hides
  static constexpr int kRegLaunch = D == 64 ? 80 : 168, kRegSoft = D == 64 ? 104 : 224, kRegRest = D == 64 ? 32 : 56;
  static constexpr uint32_t kTmemCols = D == 64 ? 256 : 512;
  static constexpr bool kSplit = kNQ == 2;
  static_assert(!kSplit || 2 * kRegSoft + kRegRest <= 3 * kRegLaunch, "a split draws on what the launch has");
  static_assert(kQCol + (kQTmem ? D / 2 : 0) <= kTmemCols, "tensor memory");
  static_assert(kCtas * (kSmem + 2048) <= 227 * 1024, "shared memory");
};

template <typename T>
constexpr uint32_t kFmt = 0;  // fp16
template <>
constexpr uint32_t kFmt<__nv_bfloat16> = 1;

// Instruction descriptor, kind::f16, fp32 accumulate, both operands of type T; b_mn: B is MN-major.
template <typename T>
__host__ __device__ constexpr uint32_t p_idesc(int N, bool b_mn) {
  return (1u << 4) | (kFmt<T> << 7) | (kFmt<T> << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kTileRows >> 4) << 24);
}
// Shared-memory descriptors, 128-byte swizzle.  K-major: groups of 8 rows 1024 bytes
// apart.  MN-major: groups of 8 contraction rows 1024 bytes apart, next 64 columns `lbo` bytes on.
__device__ __forceinline__ uint64_t p_desc_k(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t p_desc_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)(lbo >> 4) << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}
__device__ __forceinline__ void p_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void p_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void p_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(a_smem(bar))
               : "memory");
}
__device__ __forceinline__ void p_ld32(uint32_t addr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void p_st32(uint32_t addr, const float *v) {
  const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void p_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void p_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void p_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void p_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void p_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void p_tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(a_smem(bar))
      : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float p_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float p_float(__half x) { return __half2float(x); }

// What one CTA works on: tiles of one sequence's rows.
struct PromptWork {
  int seq;                 // -1: nothing
  int q0, n_q, k0, n_k;    // tokens of the sequence
  int bad_k;               // the key offsets make no sense
  int first_token;         // of tile 0, within the sequence
  int kvh;
  int unit, units;         // number of this group and key head, of how many (if keys are shared out)
  int part, parts;         // this CTA's part of the keys, of how many
  int begin, end;          // its blocks, if there are several
};

// Key blocks [jb, je) that a tile's rows see, and the range [whole_lo, whole_hi) that all its rows see.
struct TileRange {
  int jb, je, whole_lo, whole_hi;
};
template <int BK>
__device__ __forceinline__ TileRange tile_range(const PromptJob &j, const PromptWork &w, int tile) {
  TileRange r = {0, 0, 0, 0};
  const int a = w.first_token + tile * j.tile_tokens, b = min(w.n_q, a + j.tile_tokens) - 1;
  if (a > b || w.bad_k) return r;
  const int off = w.n_k - w.n_q, hi = off + b + 1;  // n_k, n_q < 2^30
  if (hi <= 0) return r;
  r.whole_hi = max(0, off + a + 1);
  int lo = 0;
  if (j.window > 0) {
    // (a row before the first key: less the widest windows, its position would pass 32 bits)
    lo = max(0, max(0, off + a + 1) - j.window);
    r.whole_lo = max(0, hi - j.window);
  }
  r.jb = lo / BK;
  r.je = (hi + BK - 1) / BK;
  return r;
}

// The blocks of a shared group's part, of at most `parts`.
template <int D>
__device__ __noinline__ void share_keys(const PromptJob &j, PromptWork &w, int parts) {
  using C = PromptCfg<D>;
  int lo = 0x7fffffff, hi = 0;
  for (int t = 0; t < C::kNQ; ++t) {
    const TileRange r = tile_range<C::kBK>(j, w, t);
    if (r.je <= r.jb) continue;
    lo = min(lo, r.jb);
    hi = max(hi, r.je);
  }
  const int n = max(0, hi - lo);
  parts = max(1, min(min(parts, n / kMinPart<D>), (int)sqrtf((float)n)));
  const int sms = j.slots / C::kCtas;
  if (C::kCtas > 1 && n < kMinPair * parts) parts = min(parts, max(1, sms / w.units));
  w.parts = parts;
  if (w.part >= parts) {
    w.seq = -1;
  } else {
    w.begin = lo + (int)((int64_t)n * w.part / parts);
    w.end = lo + (int)((int64_t)n * (w.part + 1) / parts);
  }
}

// For offsets that do not all make sense: which of the sequences from `base` on (a lane's has the queries [a, b)) are worked
// on; b = -1 for the others.  One that begins before another that counts has ended is none of them:
// it would be worked on twice, and the tile groups of all would be more than the launch has CTAs for.  end: where the
// sequences before these end (-1: they made sense, so that they end where these begin); returns where these end.
__device__ __noinline__ int queries_that_count(const PromptJob &j, int base, int a, int &b, int end) {
  const int s = base + (threadIdx.x & 31);
  if (end < 0) end = base > 0 ? __ldg(j.cu_q + base) : 0;
  const bool bad = s >= j.n_seqs || a < 0 || b < a || b > j.n_q;
  bool counts = false;
  for (int k = 0; k < 32; ++k) {
    const int ka = __shfl_sync(0xffffffffu, a, k), kb = __shfl_sync(0xffffffffu, b, k);
    if (__shfl_sync(0xffffffffu, (int)bad, k) || ka < end) continue;
    end = kb;
    counts |= s == base + k;
  }
  if (!counts) b = -1;
  return end;
}

// Whether the queries' offsets leave tokens that no sequence holds, or make no sense; by a warp of the first CTA.
__device__ __noinline__ bool rows_left_over(const PromptJob &j) {
  const int lane = threadIdx.x & 31;
  bool odd = __ldg(j.cu_q) != 0 || __ldg(j.cu_q + j.n_seqs) != j.n_q;
  for (int s = lane; s < j.n_seqs; s += 32) {
    const int a = __ldg(j.cu_q + s), b = __ldg(j.cu_q + s + 1);
    odd |= a < 0 || b < a || b > j.n_q;
  }
  odd = __any_sync(0xffffffffu, odd);
  if (odd && lane == 0 && j.status) atomicOr(j.status, MOE_KV_BAD_LENGTH);
  return odd;
}

// NaN for the tokens [from, to), by all threads of the CTA.
template <int D>
__device__ __forceinline__ void fill_rows(const PromptJob &j, int from, int to) {
  const uint4 none = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // NaN as bf16 and as fp16
  uint4 *out = static_cast<uint4 *>(j.out);
  for (int64_t i = (int64_t)from * j.hq * (D / 8) + threadIdx.x; i < (int64_t)to * j.hq * (D / 8); i += blockDim.x) out[i] = none;
  if (j.lse)
    for (int64_t i = (int64_t)from * j.hq + threadIdx.x; i < (int64_t)to * j.hq; i += blockDim.x) j.lse[i] = a_nan();
}
// The tokens that none of the sequences that are worked on (see queries_that_count) holds.
template <int D>
__device__ __noinline__ void fill_rows_left_over(const PromptJob &j) {
  int end = 0;
  for (int s = 0; s < j.n_seqs; ++s) {
    const int a = __ldg(j.cu_q + s), b = __ldg(j.cu_q + s + 1);
    if (a < end || b < a || b > j.n_q) continue;
    fill_rows<D>(j, end, a);
    end = b;
  }
  fill_rows<D>(j, end, j.n_q);
}

// A part's sums to the workspace; whether it was the last of the group.
template <int D>
__device__ __noinline__ bool write_part(const PromptJob &j, const PromptWork &w, uint32_t o_col, bool some, bool live,
                                        float m, float l, int *last, uint32_t *redo) {
  using C = PromptCfg<D>;
  float *mine = j.part + (size_t)blockIdx.x * C::kPart;
  const int tid = threadIdx.x, t = tid / kTileRows, r = tid % kTileRows;
  if (live) reinterpret_cast<float2 *>(mine + C::kSums)[t * kTileRows + r] = make_float2(m, l);
#pragma unroll 1
  for (int x = 0; x < D; x += 32) {
    float o[32];
    if (some) {
      p_ld32(o_col + x, o);
      p_ld_wait();
    } else {
#pragma unroll
      for (int z = 0; z < 32; ++z) o[z] = 0.f;
    }
    if (live)
#pragma unroll
      for (int z = 0; z < 32; z += 4)
        reinterpret_cast<float4 *>(mine)[(size_t)(t * (D / 4) + (x + z) / 4) * kTileRows + r] =
            make_float4(o[z], o[z + 1], o[z + 2], o[z + 3]);
  }
  __threadfence();
  asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kSoftWarps) : "memory");
  if (tid == 0) {
    *last = atomicAdd(j.count + w.unit, 1u) == (uint32_t)w.parts - 1;
    if (*last) j.count[w.unit] = 0;  // for the next call
  }
  if (tid < C::kSoftWarps) redo[tid] = 0;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kSoftWarps) : "memory");
  __threadfence();
  return *last != 0;
}

// One row's output from the keys it sees, one by one: the warp's lanes hold D / 32 values each.
template <int D, typename T>
__device__ __noinline__ void row_by_keys(const PromptJob &j, int q_tok, int head, int64_t k0, int lo, int hi, float ref,
                                         T *out) {
  const int lane = threadIdx.x & 31, kvh = head / j.group;
  constexpr int N = D / 32;
  float q[N], acc[N], sum = 0.f;
  const T *qp = static_cast<const T *>(j.q.data) + q_tok * j.q.token_stride + head * j.q.head_stride + lane * N;
  for (int i = 0; i < N; ++i) {
    q[i] = p_float(qp[i]);
    acc[i] = 0.f;
  }
  for (int key = lo; key < hi; ++key) {
    const T *kp = static_cast<const T *>(j.k.data) + (k0 + key) * j.k.token_stride + kvh * j.k.head_stride + lane * N;
    const T *vp = static_cast<const T *>(j.v.data) + (k0 + key) * j.v.token_stride + kvh * j.v.head_stride + lane * N;
    float s = 0.f;
    for (int i = 0; i < N; ++i) s = fmaf(q[i], p_float(kp[i]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float p = a_exp2(__fmul_rn(s, j.scale * kLog2e) - ref);
    sum += p;
    for (int i = 0; i < N; ++i) acc[i] = fmaf(p, p_float(vp[i]), acc[i]);
  }
  for (int i = 0; i < N; ++i) out[lane * N + i] = T(acc[i] / sum);
}

// The results of a shared group from its parts, in the order of the keys.  A warp takes 32 rows, a lane each, and Q quads
// of their columns, two parts at a time: enough loads in flight for what a trip to the L2 takes, however few rows there
// are.  `redo` (0 before): per 32 rows, those whose result takes a second look.
template <int D, typename T>
__device__ __noinline__ void join_parts(const PromptJob &j, const PromptWork &w, uint32_t *redo) {
  using C = PromptCfg<D>;
  const float *first = j.part + (size_t)w.unit * C::kPart;
  const size_t step = (size_t)w.units * C::kPart;  // from part to part
  const int parts = w.parts;
  constexpr int Q = D / 16, kItems = D / 4 / Q;  // (four items per 32 rows, as many as there are registers for)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows0 = min(j.tile_tokens, w.n_q - w.first_token) * j.group;
  const int rows1 = C::kNQ == 1 ? 0 : max(0, min(j.tile_tokens, w.n_q - w.first_token - j.tile_tokens)) * j.group;
  const int many0 = (rows0 + 31) / 32, many = many0 + (rows1 + 31) / 32;
  for (int item = warp; item < many * kItems; item += C::kSoftWarps) {
    const int rows32 = item / kItems, q0 = item % kItems * Q;
    const int t = rows32 >= many0, r = 32 * (rows32 - (t ? many0 : 0)) + lane;
    const bool live = r < (t ? rows1 : rows0);
    const size_t at_ml = C::kSums + 2 * (t * kTileRows + r), at_q = 4 * ((size_t)(t * (D / 4) + q0) * kTileRows + r);
    float m = -a_inf(), l = 0.f, acc[4 * Q];
#pragma unroll
    for (int x = 0; x < 4 * Q; ++x) acc[x] = 0.f;
#pragma unroll 1
    for (int y = 0; y < parts; y += 2) {
      float2 ml[2];
      float4 v[2][Q];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        ml[z] = make_float2(-a_inf(), 0.f);
        if (live && y + z < parts) {
          const float *p = first + (y + z) * step;
          ml[z] = __ldcg(reinterpret_cast<const float2 *>(p + at_ml));
#pragma unroll
          for (int x = 0; x < Q; ++x) v[z][x] = __ldcg(reinterpret_cast<const float4 *>(p + at_q) + x * kTileRows);
        }
      }
      const float top = fmaxf(m, fmaxf(ml[0].x, ml[1].x)), a = m == -a_inf() ? 0.f : a_exp2(m - top);
      m = top;
      l *= a;
#pragma unroll
      for (int x = 0; x < 4 * Q; ++x) acc[x] *= a;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (ml[z].y == 0.f) continue;  // the row sees none of the part's keys: its sums may be 0 x infinity
        const float b = ml[z].x == -a_inf() ? 0.f : a_exp2(ml[z].x - top);
        l += ml[z].y != ml[z].y ? ml[z].y : ml[z].y * b;
#pragma unroll
        for (int x = 0; x < Q; ++x) {
          acc[4 * x] = fmaf(v[z][x].x, b, acc[4 * x]);
          acc[4 * x + 1] = fmaf(v[z][x].y, b, acc[4 * x + 1]);
          acc[4 * x + 2] = fmaf(v[z][x].z, b, acc[4 * x + 2]);
          acc[4 * x + 3] = fmaf(v[z][x].w, b, acc[4 * x + 3]);
        }
      }
    }
    const int64_t at = (int64_t)(w.q0 + w.first_token + t * j.tile_tokens + r / j.group) * j.hq + w.kvh * j.group + r % j.group;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    bool finite = true;
    uint32_t p[2 * Q];
#pragma unroll
    for (int x = 0; x < 2 * Q; ++x) {
      finite = finite && fabsf(acc[2 * x]) < a_inf() && fabsf(acc[2 * x + 1]) < a_inf();
      p[x] = l == 0.f ? 0u : pack16<T>(acc[2 * x] * inv, acc[2 * x + 1] * inv);
    }
    if (live) {
      uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(j.out) + at * D + 4 * q0);
#pragma unroll
      for (int x = 0; x < Q / 2; ++x) o[x] = make_uint4(p[4 * x], p[4 * x + 1], p[4 * x + 2], p[4 * x + 3]);
      if (q0 == 0 && j.lse) j.lse[at] = l == 0.f ? -a_inf() : (m + log2f(l)) * kLn2;
    }
    const uint32_t again = __ballot_sync(0xffffffffu, live && !finite && l > 0.f && l < a_inf());
    if (again && lane == 0) atomicOr(&redo[rows32], again);
  }
  asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kSoftWarps) : "memory");
  for (int rows32 = warp; rows32 < many; rows32 += C::kSoftWarps)
    for (uint32_t again = redo[rows32]; again; again &= again - 1) {
      const int t = rows32 >= many0, r = 32 * (rows32 - (t ? many0 : 0)) + __ffs(again) - 1;
      const int tok = w.first_token + t * j.tile_tokens + r / j.group, head = w.kvh * j.group + r % j.group;
      float m = -a_inf();
      for (int y = 0; y < parts; ++y) m = fmaxf(m, __ldcg(first + y * step + C::kSums + 2 * (t * kTileRows + r)));
      const int hi = max(0, w.n_k - w.n_q + tok + 1);
      row_by_keys<D, T>(j, w.q0 + tok, head, w.k0, j.window > 0 ? max(0, hi - j.window) : 0, hi, m,
                        static_cast<T *>(j.out) + ((int64_t)(w.q0 + tok) * j.hq + head) * D);
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(PromptCfg<D>::kThreads, PromptCfg<D>::kCtas)
    prompt_attention_kernel(const __grid_constant__ PromptMaps maps, const PromptJob j) {
  using C = PromptCfg<D>;
  constexpr int NQ = C::kNQ, BK = C::kBK, ST = C::kStages, DC = D / 64;
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  __shared__ uint64_t q_smem, q_full, k_full[ST], k_empty[ST], v_full[ST], v_empty[ST], s_full[2], p_full[2], pv_done[NQ], k_first, done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail, s_last, s_left_over;
  __shared__ uint32_t s_redo[C::kSoftWarps];  // (a warp has 32 rows)
  __shared__ PromptWork s_work;
  const uint32_t sm = (a_smem(sm_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == C::kLoadWarp && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v)));
  if (tid == 0) {
    s_fail = 0;
    a_mbar_init(&q_smem, 1);
    a_mbar_init(&q_full, C::kQTmem ? kTileRows : 1);
    for (int i = 0; i < ST; ++i) {
      a_mbar_init(&k_full[i], 1);
      a_mbar_init(&k_empty[i], 1);
      a_mbar_init(&v_full[i], 1);
      a_mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      a_mbar_init(&s_full[i], 1);
      a_mbar_init(&p_full[i], NQ == 2 ? 129 : 128);
    }
    for (int i = 0; i < NQ; ++i) a_mbar_init(&pv_done[i], 1);
    a_mbar_init(&k_first, 1);
    a_mbar_init(&done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    // The sequence and tiles of this CTA.  Groups of tiles far along a sequence look back furthest: of up to 32
    // sequences all groups are taken by how far along they are, furthest first, so that what runs last is short (twelve
    // packed prompts of 3 to 1500 tokens: 68 us in the order of the sequences, 60 us so); of more, sequence by
    // sequence, as finding a group's place would take a CTA longer than it saves.
    const int per = NQ * j.tile_tokens;
    int unit = blockIdx.x, of = 0, part = 0, parts = 1;  // unit: group and key head
    const bool by_level = j.n_seqs <= kMaxSplitSeqs;
    int before = 0, seq = -1, group = 0, a = 0, b = 0, c = 0, d = 0, at = 0;
    int end = -1;  // where some offsets make no sense: where the sequences before these end
    for (int base = 0; base < j.n_seqs; base += 32) {
      const int s = base + lane;
      int n = 0;
      bool bad = false;
      if (s < j.n_seqs) {
        a = __ldg(j.cu_q + s);
        b = __ldg(j.cu_q + s + 1);
        c = __ldg(j.cu_k + s);  // with the others: a trip to memory less
        d = __ldg(j.cu_k + s + 1);
        bad = a < 0 || b < a || b > j.n_q;
        n = (b - a + per - 1) / per;
      }
      if (__any_sync(0xffffffffu, bad) || end >= 0) {
        end = queries_that_count(j, base, a, b, end);
        if (b < 0) a = b = n = 0;
      }
      bool hit = false;
      auto beyond = [&](int level) { return (int)__reduce_add_sync(0xffffffffu, max(0, n - level)); };
      if (j.slots > 0) {  // (then there are at most kMaxSplitSeqs sequences)
        // every part has to have its CTA: the last one done is told by their number
        const int units = beyond(0) * j.hkv, room = min(j.slots, (int)gridDim.x);
        if (units > 0 && 2 * units <= room) {
          parts = min(room / units, j.most_parts);
          part = unit / units;  // (first parts first: not all groups may have more)
          unit %= units;
          of = units;
        }
      }
      const int mine = unit / j.hkv;
      if (by_level) {
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, n);
        if (j.n_seqs == 1) {
          lo = n - 1 - mine;
          lo = __shfl_sync(0xffffffffu, lo, 0);
          hit = lane == 0 && lo >= 0;
        } else if (mine < beyond(0)) {
          while (hi - lo > 1) {  // beyond(lo) > mine >= beyond(hi)
            const int mid = (lo + hi) / 2;
            if (beyond(mid) > mine) lo = mid;
            else hi = mid;
          }
          const int rank = mine - beyond(lo + 1);  // among the sequences that reach this level
          const uint32_t reach = __ballot_sync(0xffffffffu, n > lo);  // (by all lanes, whether they reach it or not)
          hit = n > lo && __popc(reach & ((1u << lane) - 1u)) == rank;
        }
        group = lo;
      } else {
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        hit = mine >= before + inc - n && mine < before + inc;
        group = before + inc - 1 - mine;
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      const uint32_t who = __ballot_sync(0xffffffffu, hit);
      if (who) {
        at = __ffs(who) - 1;
        seq = base + at;
        if (lane == at) {
          const bool bad_k = c < 0 || d < c || d > j.n_k;
          if (bad_k && j.status) atomicOr(j.status, MOE_KV_BAD_LENGTH);
          PromptWork w = {seq, a, b - a, bad_k ? 0 : c, bad_k ? 0 : d - c, bad_k, group * per, unit % j.hkv, unit, of, part, 1, 0, 0};
          if (parts > 1) share_keys<D>(j, w, parts);
          s_work = w;
        }
        break;
      }
    }
    if (seq < 0 && lane == 0) s_work = {-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0, 0};
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(a_smem(&s_tmem)), "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (blockIdx.x == 0 && warp == C::kCheckWarp) {
    const bool some = rows_left_over(j);
    if (lane == 0) s_left_over = some;
  }
  p_fence_before();
  __syncthreads();
  p_fence_after();
  if (blockIdx.x == 0 && s_left_over) fill_rows_left_over<D>(j);
  const uint32_t tmem = s_tmem;
  const PromptWork w = s_work;
  const int kvh = w.kvh;

  TileRange tr[NQ];
  int J0 = 0x7fffffff, J1 = 0;
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    tr[t] = w.seq < 0 ? TileRange{0, 0, 0, 0} : tile_range<BK>(j, w, t);
    if (w.parts > 1) {
      tr[t].jb = max(tr[t].jb, w.begin);
      tr[t].je = min(tr[t].je, w.end);
    }
    if (tr[t].je > tr[t].jb) {
      J0 = min(J0, tr[t].jb);
      J1 = max(J1, tr[t].je);
    }
  }
  const int n_blocks = max(0, J1 - J0);

  // (each role takes its registers in its own branch: the compiler allocates by them from there on)
  if (warp >= C::kSoftWarps) {
  if (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegRest));
  if (warp == C::kLoadWarp) {
    if (lane == 0 && n_blocks > 0) {
      bool ok = true;
      const uint32_t q_rows_bytes = (uint32_t)(j.group * j.tile_tokens) * 128u;
      uint32_t q_bytes = 0;
#pragma unroll
      for (int t = 0; t < NQ; ++t)
        if (tr[t].je > tr[t].jb) q_bytes += DC * q_rows_bytes;
      uint64_t *q_bar = C::kQTmem ? &q_smem : &q_full;
      a_expect_tx(q_bar, q_bytes);
#pragma unroll
      for (int t = 0; t < NQ; ++t)
        if (tr[t].je > tr[t].jb)
          for (int c = 0; c < DC; ++c)
            p_tma_3d(sm + C::kQOff + t * C::kQBytes + c * kTileRows * 128, &maps.q, 64 * c, kvh * j.group,
                     w.q0 + w.first_token + t * j.tile_tokens, q_bar);
      // block i's keys or values into their stage; keys go a block ahead of values, as they are used
      auto load = [&](const CUtensorMap *map, uint32_t off, uint64_t *full, int i, int &count) {
        const int st = i % ST;
        a_expect_tx(&full[st], C::kKBytes);
        for (int c = 0; c < DC; ++c)
          p_tma_3d(sm + off + st * C::kKBytes + c * BK * 128, map, 64 * c, kvh, w.k0 + (J0 + i) * BK, &full[st]);
        count = i + 1;
      };
      auto free_from = [&](uint64_t *empty, int i) {  // the stage's use `i` (0, 1, ... over all stages) is over
        return a_mbar_wait(&empty[i % ST], (uint32_t)(i / ST) & 1u, &s_fail);
      };
      int k_loaded = 0, v_loaded = 0;
      load(&maps.k, C::kKOff, k_full, 0, k_loaded);
      for (int i = 0; i < n_blocks; ++i) {
        const int x = i + 1;
        if (x >= ST && x <= n_blocks) {
          if (NQ == 2) {
            // one signal for the values of block i - ST and the keys of the block after it
            ok = x == ST ? x == n_blocks || a_mbar_wait(&k_first, 0, &s_fail) : free_from(v_empty, x - ST - 1);
          } else if (x < n_blocks) {
            ok = free_from(k_empty, x - ST);
          }
          if (!ok) break;
        }
        if (x < n_blocks) load(&maps.k, C::kKOff, k_full, x, k_loaded);
        if (NQ == 1 && i >= ST && !(ok = free_from(v_empty, i - ST))) break;
        if (C::kQTmem && i == 0 && !(ok = a_mbar_wait(&q_full, 0, &s_fail))) break;  // the queries are out of the way
        load(&maps.v, C::kVOff, v_full, i, v_loaded);
      }
      if (!ok) s_fail = 1;
      // no copy may be in flight when the CTA leaves
      if (*(volatile int *)&s_fail) (void)a_mbar_drain(q_bar, 0);
      for (int i = max(0, k_loaded - ST); i < k_loaded; ++i) (void)a_mbar_drain(&k_full[i % ST], (uint32_t)(i / ST) & 1u);
      for (int i = max(0, v_loaded - ST); i < v_loaded; ++i) (void)a_mbar_drain(&v_full[i % ST], (uint32_t)(i / ST) & 1u);
    }
  } else if (warp == C::kMmaWarp) {
    // The whole warp walks through the blocks and one elected lane issues: descriptors then stay in uniform registers,
    // where the instructions want them.
    if (n_blocks > 0) {
      const bool one = elect_one();
      constexpr uint32_t id_qk = p_idesc<T>(BK, false), id_pv = p_idesc<T>(D, true);
      auto qk = [&](int t, int buf, int i) {
        const uint64_t a0 = p_desc_k(sm + C::kQOff + t * C::kQBytes);
        const uint64_t b0 = p_desc_k(sm + C::kKOff + (i % ST) * C::kKBytes);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t b = b0 + (kk / 4) * (BK * 128 / 16) + (kk % 4) * 2;
            if constexpr (C::kQTmem)
              p_mma_ts(tmem + buf * BK, tmem + C::kQCol + kk * 8, b, id_qk, kk > 0);
            else
              p_mma_ss(tmem + buf * BK, a0 + (kk / 4) * (kTileRows * 128 / 16) + (kk % 4) * 2, b, id_qk, kk > 0);
          }
          p_commit(&s_full[buf]);
        }
        __syncwarp();
      };
      auto pv = [&](int t, int buf, int i, bool first, bool last) {
        const uint64_t b0 = p_desc_mn(sm + C::kVOff + (i % ST) * C::kKBytes, BK * 128);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            p_mma_ts(tmem + C::kOCol + t * D, tmem + buf * BK + kk * 8, b0 + kk * (2048 / 16), id_pv, !first || kk > 0);
          // (of two tiles, the scores of the next block, asked for later, tell that this is done)
          if (NQ == 1 || last) p_commit(&pv_done[t]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t *bar) {
        if (one) p_commit(bar);
        __syncwarp();
      };
      auto wait = [&](uint64_t *bar, uint32_t ph) { return __all_sync(0xffffffffu, a_mbar_wait(bar, ph, &s_fail)) != 0; };
      bool ok = wait(&q_full, 0) && wait(&k_full[0], 0);
      if (ok) {
        p_fence_after();
#pragma unroll
        for (int t = 0; t < NQ; ++t)
          if (J0 >= tr[t].jb && J0 < tr[t].je) qk(t, t, 0);
        commit(NQ == 2 ? &k_first : &k_empty[0]);
      }
      for (int i = 0; i < n_blocks && ok; ++i) {
        const int jj = J0 + i;
        const bool more = i + 1 < n_blocks;
        if constexpr (NQ == 2) {
          // A wait costs this warp a few hundred cycles even where there is nothing to wait for, and the tensor cores
          // run dry meanwhile: so the weights' barrier also stands for block i's values and block i + 1's keys (another
          // warp waits for them), and one commit frees both stages.
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool now = jj >= tr[t].jb && jj < tr[t].je, next = more && jj + 1 >= tr[t].jb && jj + 1 < tr[t].je;
            if (now) {
              if (!(ok = wait(&p_full[t], (uint32_t)(jj - tr[t].jb) & 1u))) break;
              p_fence_after();
              pv(t, t, i, jj == tr[t].jb, jj + 1 == tr[t].je);
            } else if (next) {
              if (!(ok = wait(&k_full[(i + 1) % ST], (uint32_t)((i + 1) / ST) & 1u))) break;
              p_fence_after();
            }
            // (the weights that these scores overwrite have been read by then: one thread's instructions run in order)
            if (next) qk(t, t, i + 1);
          }
          if (!ok) break;
          commit(&v_empty[i % ST]);
        } else {
          if (more && !(ok = wait(&k_full[(i + 1) % ST], (uint32_t)((i + 1) / ST) & 1u))) break;
          if (more) {
            p_fence_after();
            qk(0, (i + 1) & 1, i + 1);
            commit(&k_empty[(i + 1) % ST]);
          }
          if (!(ok = wait(&v_full[i % ST], (uint32_t)(i / ST) & 1u))) break;
          if (!(ok = wait(&p_full[i & 1], (uint32_t)(i >> 1) & 1u))) break;
          p_fence_after();
          pv(0, i & 1, i, i == 0, false);
          commit(&v_empty[i % ST]);
        }
      }
      if (!ok) s_fail = 1;
      // no product may be running when the CTA gives its memory back, least of all after a wait that gave up
      commit(&done);
      (void)a_mbar_drain(&done, 0);
      __syncwarp();
    }
  } else if (NQ == 2 && warp == C::kReadyWarp) {
    // block i's values and block i + 1's keys are there: one more arrival for the weights of block i
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < n_blocks && ok; ++i) {
        // Not before the weights of the block before are complete: an arrival that comes early would count for them, and
        // a stage's barrier might not have seen its block before, whose parity is that of the next.
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          const int n = J0 + i - 1 - tr[t].jb;
          if (ok && i > 0 && n >= 0 && J0 + i - 1 < tr[t].je) ok = a_mbar_wait(&p_full[t], (uint32_t)n & 1u, &s_fail);
        }
        ok = ok && (i + 1 == n_blocks || a_mbar_wait(&k_full[(i + 1) % ST], (uint32_t)((i + 1) / ST) & 1u, &s_fail)) &&
             a_mbar_wait(&v_full[i % ST], (uint32_t)(i / ST) & 1u, &s_fail);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < NQ; ++t)
          if (J0 + i >= tr[t].jb && J0 + i < tr[t].je) a_mbar_arrive(&p_full[t]);
      }
      if (!ok) s_fail = 1;
    }
  }
  } else {
    if (C::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegSoft));
    // ---- softmax: thread = row of tile t
    const int t = warp / 4, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 (warp % 4) in the lane field
    const TileRange range = NQ == 1 ? tr[0] : (t == 0 ? tr[0] : tr[NQ - 1]);
    const int tok = w.first_token + t * j.tile_tokens + r / j.group, head = kvh * j.group + r % j.group;
    const bool live = w.seq >= 0 && r < j.group * j.tile_tokens && tok < w.n_q;
    const int hi = live ? max(0, w.n_k - w.n_q + tok + 1) : 0;
    const int lo = j.window > 0 ? max(0, hi - j.window) : 0;
    // fp16 has few numbers far below 1, so its weights go up to 2^6 before the reference has to move, and to 2^14 then
    constexpr float kBelow = std::is_same<T, __half>::value ? 6.f : 0.f;
    constexpr float kMostSum = std::is_same<T, __half>::value ? 16384.f : 256.f;
    float m = live ? -a_inf() : 0.f, l = 0.f;  // reference (log2 units) and sum
    const float c = j.scale * kLog2e;
    bool ok = true;
    const uint32_t o_col = tmem + lanes + C::kOCol + t * D;
    if constexpr (C::kQTmem) {
      if (n_blocks > 0) {
        ok = __all_sync(0xffffffffu, a_mbar_wait(&q_smem, 0, &s_fail));
        const unsigned char *row = sm_raw + (sm - a_smem(sm_raw)) + C::kQOff + r * 128;
#pragma unroll
        for (int x = 0; x < DC; ++x) {
          float q[32];
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const float4 v = live && ok ? *reinterpret_cast<const float4 *>(row + x * kTileRows * 128 + ((z ^ (r & 7)) << 4))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
            q[4 * z] = v.x;
            q[4 * z + 1] = v.y;
            q[4 * z + 2] = v.z;
            q[4 * z + 3] = v.w;
          }
          p_st32(tmem + lanes + C::kQCol + 32 * x, q);
        }
        p_st_wait();
        p_fence_before();
        a_mbar_arrive(&q_full);
      }
    }
    for (int jj = range.jb; jj < range.je && ok; ++jj) {
      const int n = jj - range.jb, buf = NQ == 1 ? (n & 1) : t;
      const uint32_t ph = (uint32_t)(NQ == 1 ? n >> 1 : n) & 1u;
      // (no reference yet, or one so far from 0 that the fast way would show it)
      bool again = n == 0 || __any_sync(0xffffffffu, live && !(fabsf(m) < kFar));
      ok = __all_sync(0xffffffffu, a_mbar_wait(&s_full[buf], ph, &s_fail));
      if (!ok) break;
      p_fence_after();
      const uint32_t s_col = tmem + lanes + buf * BK;
      float s[BK];
#pragma unroll
      for (int x = 0; x < BK; x += 32) p_ld32(s_col + x, s + x);
      p_ld_wait();
      const int key0 = jj * BK;
      if (key0 < range.whole_lo || key0 + BK > range.whole_hi) {
#pragma unroll
        for (int x = 0; x < BK; ++x)
          if (key0 + x < lo || key0 + x >= hi) s[x] = -a_inf();
      }
      // Weights of 32 columns from x on, over the scores' first half; their sum.  Scores so large that their rounding (2^-14
      // at kFar) shows in a weight are rounded before the reference is taken away, as the largest was for the reference:
      // its weight then is of its own size.
      auto weights = [&](int x, float ref, auto rounded) {
        const uint64_t c2 = f2_pack(c, c), r2 = f2_pack(-ref, -ref);
        uint64_t sum[2] = {0, 0};
        uint32_t p[16];
#pragma unroll
        for (int z = 0; z < 16; ++z) {
          float a, b;
          if (decltype(rounded)::value) {  // (one by one: of packed pairs a product and the sum after it come out fused)
            a = __fadd_rn(__fmul_rn(s[x + 2 * z], c), -ref);
            b = __fadd_rn(__fmul_rn(s[x + 2 * z + 1], c), -ref);
          } else {
            f2_unpack(f2_fma(f2_pack(s[x + 2 * z], s[x + 2 * z + 1]), c2, r2), a, b);
          }
          a = a_exp2(a);
          b = a_exp2(b);
          sum[z & 1] = f2_add(sum[z & 1], f2_pack(a, b));
          p[z] = pack16<T>(a, b);
        }
        p_st16(s_col + x / 2, p);
        float a, b;
        f2_unpack(f2_add(sum[0], sum[1]), a, b);
        return a + b;
      };
      // The old reference first, without looking for the largest score: a sum of at most kMostSum says that no weight of
      // it was larger.
      float sum = 0.f;
      if (!again) {
#pragma unroll
        for (int x = 0; x < BK; x += 32) sum += weights(x, m, std::false_type());
        again = __any_sync(0xffffffffu, live && !(sum <= kMostSum));
      }
      if (again) {
        float top[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) top[z] = -a_inf();
#pragma unroll
        for (int x = 0; x < BK; x += 8)
#pragma unroll
          for (int z = 0; z < 4; ++z) top[z] = fmaxf(top[z], fmaxf(s[x + z], s[x + 4 + z]));
        const float m_new =
            fmaxf(m, __fadd_rn(__fmul_rn(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), c), -kBelow));  // c > 0
        p_st_wait();  // of the weights that are written again
        const float a = m == -a_inf() ? 0.f : a_exp2(m - m_new);
        m = m_new;
        l *= a;
        if (n > 0) {
          // the products so far: of two tiles, these scores were asked for after them
          if (NQ == 1) ok = __all_sync(0xffffffffu, a_mbar_wait(&pv_done[t], (uint32_t)(n - 1) & 1u, &s_fail));
          if (!ok) break;
          p_fence_after();
#pragma unroll 1
          for (int x = 0; x < D; x += 32) {
            float o[32];
            p_ld32(o_col + x, o);
            p_ld_wait();
#pragma unroll
            for (int z = 0; z < 32; ++z) o[z] *= a;
            p_st32(o_col + x, o);
          }
          p_st_wait();
        }
        const float ref = m == -a_inf() ? 0.f : m;
        sum = 0.f;
        // (with the slower form alone: twelve packed prompts 65 us, 63 so)
        if (__any_sync(0xffffffffu, live && fabsf(m) >= kFar && m > -a_inf())) {
#pragma unroll
          for (int x = 0; x < BK; x += 32) sum += weights(x, ref, std::true_type());
        } else {
#pragma unroll
          for (int x = 0; x < BK; x += 32) sum += weights(x, ref, std::false_type());
        }
      }
      l += sum;
      p_st_wait();
      // The final wait below tells the last product's phase by its parity, so the one before has to be over by then.
      // With a tile per score buffer it is (its scores were asked for after it); with two buffers of one tile it is
      // waited for here, before the last product can run.
      if (NQ == 1 && n > 0 && jj + 1 == range.je) {
        ok = __all_sync(0xffffffffu, a_mbar_wait(&pv_done[t], (uint32_t)(n - 1) & 1u, &s_fail));
        if (!ok) break;
      }
      p_fence_before();
      a_mbar_arrive(&p_full[buf]);
    }
    // ---- the rows' results
    const int n_mine = range.je - range.jb;
    if (ok && n_mine > 0)
      ok = __all_sync(0xffffffffu, a_mbar_wait(&pv_done[t], NQ == 1 ? (uint32_t)(n_mine - 1) & 1u : 0u, &s_fail));
    if (!ok) s_fail = 1;
    p_fence_after();
    const bool some = n_mine > 0 && ok;
    if (w.seq >= 0 && w.parts > 1) {
      // a part of a shared group; the last one done joins all of them
      if (write_part<D>(j, s_work, o_col, some, live, m, ok ? l : a_nan(), &s_last, s_redo))
        join_parts<D, T>(j, s_work, s_redo);
    } else if (w.seq >= 0) {
      const int64_t at = (int64_t)(w.q0 + tok) * j.hq + head;
      T *out = static_cast<T *>(j.out) + at * D;
      if (!ok || w.bad_k) l = a_nan();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      bool finite = true;
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        float o[32];
        if (some) {
          p_ld32(o_col + x, o);
          p_ld_wait();
        } else {
#pragma unroll
          for (int z = 0; z < 32; ++z) o[z] = 0.f;
        }
        uint32_t p[16];
#pragma unroll
        for (int z = 0; z < 16; ++z) {
          finite = finite && fabsf(o[2 * z]) < a_inf() && fabsf(o[2 * z + 1]) < a_inf();
          // a row that sees nothing is 0 even where its accumulator took a 0 x infinity
          p[z] = l == 0.f ? 0u : pack16<T>(o[2 * z] * inv, o[2 * z + 1] * inv);
        }
        if (live)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            *reinterpret_cast<uint4 *>(out + x + 8 * z) = make_uint4(p[4 * z], p[4 * z + 1], p[4 * z + 2], p[4 * z + 3]);
      }
      if (live && j.lse) j.lse[at] = l == 0.f ? -a_inf() : (m + log2f(l)) * kLn2;
      // a product of a zero weight with a value that is not finite: once more, without the unseen keys
      uint32_t again = __ballot_sync(0xffffffffu, live && some && !finite && l > 0.f && l < a_inf());
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        const int rtok = __shfl_sync(0xffffffffu, tok, src), rhead = __shfl_sync(0xffffffffu, head, src);
        const int rlo = __shfl_sync(0xffffffffu, lo, src), rhi = __shfl_sync(0xffffffffu, hi, src);
        const float rm = __shfl_sync(0xffffffffu, m, src);
        __syncwarp();
        row_by_keys<D, T>(j, w.q0 + rtok, rhead, w.k0, rlo, rhi, rm,
                          static_cast<T *>(j.out) + ((int64_t)(w.q0 + rtok) * j.hq + rhead) * D);
      }
    }
  }
  p_fence_before();
  __syncthreads();
  if (s_fail && tid == 0 && j.status) atomicOr(j.status, MOE_KV_TIMED_OUT);
  if (warp == C::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  return fn;
}

// Tensor [tokens][heads][D] as boxes of 64 values x box_heads heads x box_tokens tokens, 128-byte swizzle.
bool encode_map(CUtensorMap *m, const moe_tensor &t, int tokens, int heads, int D, int box_heads, int box_tokens,
                int dtype) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  // with one head its stride is never used, but has to be one that the encoder takes
  const uint64_t hs = heads > 1 ? (uint64_t)t.head_stride * 2 : (uint64_t)D * 2;
  const uint64_t ts = tokens > 1 ? (uint64_t)t.token_stride * 2 : (uint64_t)heads * D * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens}, strides[2] = {hs, ts};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, elem[3] = {1, 1, 1};
  return fn(m, dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void *>(t.data), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxSlots = 1024;  // parts' counters are MOE_KV_COUNTER_BYTES
static_assert(kMaxSlots * 4 <= MOE_KV_COUNTER_BYTES, "a counter per group");

// CTAs that run at once, for heads of D.
int prompt_slots(int D) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return std::min(kMaxSlots, sms * (D == 64 ? PromptCfg<64>::kCtas : 1));
}
size_t prompt_part_bytes(int D) {
  return 4 * (D == 64 ? PromptCfg<64>::kPart : D == 128 ? PromptCfg<128>::kPart : PromptCfg<256>::kPart);
}
// Most parts that a tile group of a call can have: at most this many blocks of keys are seen by its rows.
int prompt_most_parts(int n_k, int n_seqs, int group, int D, int window) {
  if (n_seqs > kMaxSplitSeqs) return 1;
  const int bk = D == 128 ? PromptCfg<128>::kBK : 64, per = (D == 256 ? 1 : 2) * (kTileRows / group);
  const int64_t keys = window > 0 ? std::min<int64_t>(n_k, (int64_t)window + per) : n_k, blocks = keys / bk + 2;
  return (int)std::max(1.0, std::min({(double)kMostParts, (double)(blocks / (D == 64 ? kMinPart<64> : D == 128 ? kMinPart<128> : kMinPart<256>)), std::sqrt((double)blocks)}));
}

template <int D, typename T>
int launch_prompt(PromptJob j, int dtype, cudaStream_t st) {
  using C = PromptCfg<D>;
  static DynSmemLimit limit;
  if (ensure_dyn_smem(prompt_attention_kernel<D, T>, C::kSmem, limit) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  PromptMaps maps;
  if (!encode_map(&maps.q, j.q, j.n_q, j.hq, D, j.group, j.tile_tokens, dtype) ||
      !encode_map(&maps.k, j.k, std::max(1, j.n_k), j.hkv, D, 1, C::kBK, dtype) ||
      !encode_map(&maps.v, j.v, std::max(1, j.n_k), j.hkv, D, 1, C::kBK, dtype))
    return MOE_ERR_INVALID_ARG;
  const int64_t per = (int64_t)C::kNQ * j.tile_tokens;
  // at most this many tile groups: a sequence's last one may be partly filled
  const int64_t groups = j.n_q / per + std::min<int64_t>(j.n_seqs, j.n_q);
  if (groups * j.hkv > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  int64_t grid = groups * j.hkv;
  if (grid < j.slots) grid = std::min<int64_t>(j.slots, grid * j.most_parts);
  prompt_attention_kernel<D, T><<<(unsigned)grid, C::kThreads, C::kSmem, st>>>(maps, j);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int64_t moe_prompt_attention_workspace(int32_t n_q_tokens, int32_t n_q_heads, int32_t n_k_tokens,
                                               int32_t n_kv_heads, int32_t head_dim, int32_t n_seqs, int32_t window) {
  if (n_q_tokens <= 0 || n_k_tokens <= 0 || n_seqs <= 0 || n_kv_heads <= 0 || n_q_heads <= 0 ||
      n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64 || window < 0 || !kv_sizes_ok(n_kv_heads, head_dim, kKvTile))
    return 0;
  if (prompt_most_parts(n_k_tokens, n_seqs, n_q_heads / n_kv_heads, head_dim, window) < 2) return 0;
  const int slots = prompt_slots(head_dim), per = (head_dim == 256 ? 1 : 2) * (kTileRows * n_kv_heads / n_q_heads);
  const int64_t units = (int64_t)((n_q_tokens + per - 1) / per) * n_kv_heads;  // at least
  return 2 * units <= slots ? MOE_KV_COUNTER_BYTES + (int64_t)slots * (int64_t)prompt_part_bytes(head_dim) : 0;
}

MOE_API int moe_prompt_attention(const moe_tensor *q, int32_t n_q_tokens, int32_t n_q_heads, const moe_tensor *k,
                                 const moe_tensor *v, int32_t n_k_tokens, int32_t n_kv_heads, int32_t head_dim,
                                 const int32_t *cu_q, const int32_t *cu_k, int32_t n_seqs, float scale, int32_t window,
                                 void *out, float *lse, int32_t dtype, int32_t *status, void *cuda_stream) {
  return moe_prompt_attention_shared(q, n_q_tokens, n_q_heads, k, v, n_k_tokens, n_kv_heads, head_dim, cu_q, cu_k, n_seqs,
                                     scale, window, out, lse, dtype, status, nullptr, 0, cuda_stream);
}

MOE_API int moe_prompt_attention_shared(const moe_tensor *q, int32_t n_q_tokens, int32_t n_q_heads, const moe_tensor *k,
                                        const moe_tensor *v, int32_t n_k_tokens, int32_t n_kv_heads, int32_t head_dim,
                                        const int32_t *cu_q, const int32_t *cu_k, int32_t n_seqs, float scale,
                                        int32_t window, void *out, float *lse, int32_t dtype, int32_t *status,
                                        void *workspace, int64_t workspace_bytes, void *cuda_stream) {
  if (n_q_tokens < 0 || n_k_tokens < 0 || n_seqs < 0 || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads ||
      window < 0 || !(scale > 0.f && scale <= kMostScale))
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  const int group = n_q_heads / n_kv_heads;
  if (!kv_sizes_ok(n_kv_heads, head_dim, kKvTile) || n_q_heads > kMaxAttnHeads || group > 64 ||
      n_q_tokens > (1 << 29) || n_k_tokens > (1 << 29))
    return MOE_ERR_UNSUPPORTED;
  if (n_q_tokens == 0 || n_seqs == 0) return MOE_OK;
  if (!cu_q || !cu_k || !out || (uintptr_t)out % 16 || (uintptr_t)lse % 4) return MOE_ERR_INVALID_ARG;
  if (const int rc = check_tensor(q, 2)) return rc;
  if (n_k_tokens > 0) {
    if (const int rc = check_tensor(k, 2)) return rc;
    if (const int rc = check_tensor(v, 2)) return rc;
  }
  PromptJob j = {};
  j.q = *q;
  // without keys nothing is loaded, but the maps want an address
  j.k = n_k_tokens > 0 ? *k : moe_tensor{q->data, head_dim, head_dim};
  j.v = n_k_tokens > 0 ? *v : j.k;
  j.cu_q = cu_q;
  j.cu_k = cu_k;
  j.n_q = n_q_tokens;
  j.n_k = n_k_tokens;
  j.n_seqs = n_seqs;
  j.hq = n_q_heads;
  j.hkv = n_kv_heads;
  j.group = group;
  j.tile_tokens = kTileRows / group;
  j.window = window;
  j.scale = scale;
  j.out = out;
  j.lse = lse;
  j.status = status;
  if (workspace) {
    const int64_t need = moe_prompt_attention_workspace(n_q_tokens, n_q_heads, n_k_tokens, n_kv_heads, head_dim, n_seqs, window);
    if ((uintptr_t)workspace % 256 || workspace_bytes < need) return MOE_ERR_INVALID_ARG;
    if (need > 0) {
      j.slots = prompt_slots(head_dim);
      j.most_parts = prompt_most_parts(n_k_tokens, n_seqs, group, head_dim, window);
      j.count = static_cast<uint32_t *>(workspace);
      j.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + MOE_KV_COUNTER_BYTES);
    }
  }
  cudaStream_t st = (cudaStream_t)cuda_stream;
  if (dtype == MOE_BF16)
    return head_dim == 64    ? launch_prompt<64, __nv_bfloat16>(j, dtype, st)
           : head_dim == 128 ? launch_prompt<128, __nv_bfloat16>(j, dtype, st)
                             : launch_prompt<256, __nv_bfloat16>(j, dtype, st);
  return head_dim == 64    ? launch_prompt<64, __half>(j, dtype, st)
         : head_dim == 128 ? launch_prompt<128, __half>(j, dtype, st)
                           : launch_prompt<256, __half>(j, dtype, st);
}
