// Appending to the paged 4-bit cache, and reading it back.
//
// Append: rotation y_a = a c - b s, y_b = b c + a s of queries and keys, then per
// 32 values of a key or value head m = the value of largest magnitude, d = m / -8,
// q = min(15, trunc(x / d + 8.5)).  Rotation and quantisation keep every fp32
// operation separately rounded (no contraction): a code is decided by a comparison
// with a border, and the same border has to be met by any other implementation.
//
// Bound: memory (every value is read once and written once); for a token or two, the
// latency of the chain cu -> start -> table -> store.  18439 prompt tokens of 48 heads of
// 128 are appended in 85 us as bf16, 0.77 of the measured copy rate, with the SMs issuing
// in three cycles of four: the division of every key and value by its block's scale and
// the packing of codes cost as much as the bytes do; as fp32, twice the bytes, in 137 us,
// 0.93 of that rate.  A single token takes 3 us, its launch among them.  Reading 65536
// cached tokens of 8 heads of 128 back takes 70 us, 0.73 of the copy rate, and the 18439
// that were just appended 23.5 us (14.3 would be the copy rate): a warp reads a token, so
// it uses half of every 32-byte sector of codes and 8 bytes of one of scales, and the
// warps of the neighbouring tokens ask for the same sectors again.
// Layout of the work: a thread takes 8 consecutive
// values (one 16-byte load of a 16-bit type), so a head is D/8 lanes of one warp,
// the rotation's other half sits in another lane of the same head (a shuffle), and
// a quantisation block is 4 neighbouring lanes.  A warp stays on one token and
// walks over its heads, so the token's cosines and sines, its sequence and its
// page are found once and kept in registers.
#include <algorithm>

#include "attn_common.cuh"

namespace moe {
namespace {

struct AppendJob {
  moe_kv_cache c;
  const int32_t *starts, *cu;
  int n_tokens;
  moe_tensor q, k, v;
  int hq, hkv;
  const float *cos, *sin;
  int rot, n_pos, interleaved;
  void *q_out, *k_out, *v_out;
  int per_warp;  // heads (of q, k and v together) that one warp takes
};

constexpr int kAppendWarps = 4, kAppendCtas = 8;  // warps of a CTA, and CTAs that registers leave room for on an SM

// The sequence of token i: the last s with cu[s] <= i, by all lanes of a warp.
__device__ __forceinline__ int find_seq(const int32_t *cu, int n_seqs, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seqs;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool le = at < n && __ldg(cu + lo + at) <= i;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    const int skip = cnt > 0 ? (cnt - 1) * step : 0;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

struct TokenPlace {
  int seq;
  int64_t pos;    // -1: the offsets make no sense
  int page;       // -1: none
  int in_page;
  int row;        // token within its tile
};

__device__ __forceinline__ TokenPlace place_token(const moe_kv_cache &c, const int32_t *starts, const int32_t *cu,
                                                  int i) {
  TokenPlace p;
  p.seq = find_seq(cu, c.n_seqs, i);
  p.pos = kv_position(i, __ldg(cu + p.seq), __ldg(cu + p.seq + 1), __ldg(starts + p.seq));
  p.page = -1;
  p.in_page = 0;
  p.row = (int)(p.pos & 31);
  if (p.pos >= 0)
    p.page = kv_page(c.page_table + (int64_t)p.seq * c.table_stride, c.table_width, c.n_pages, c.page_size,
                     p.pos / kKvTile, &p.in_page);
  return p;
}

// 8 consecutive values as loaded, and to and from fp32.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void copy_raw(Raw8<T> *to, const T *from) {  // asynchronous, into shared memory
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a_smem(&to->w[i])),
                 "l"(reinterpret_cast<const uint4 *>(from) + i)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
  return r;
}
__device__ __forceinline__ void expand8(const Raw8<float> &r, float x[8]) {
  const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void expand8(const Raw8<__nv_bfloat16> &r, float x[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void expand8(const Raw8<__half> &r, float x[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float *p, const float x[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
template <typename T2, typename T>
__device__ __forceinline__ void store8_16(T *p, const float x[8], T2 (*pack)(float, float)) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T2 h = pack(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ __nv_bfloat162 pack_bf16(float a, float b) { return __floats2bfloat162_rn(a, b); }
__device__ __forceinline__ __half2 pack_f16(float a, float b) { return __floats2half2_rn(a, b); }
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float x[8]) { store8_16<__nv_bfloat162>(p, x, pack_bf16); }
__device__ __forceinline__ void store8(__half *p, const float x[8]) { store8_16<__half2>(p, x, pack_f16); }

// Quantise the 32 values held by 4 neighbouring lanes (8 each) and store codes
// and scale of one block.  Every lane of the warp calls it; `live` lanes store.
__device__ __forceinline__ void quantise_store(const float x[8], uint8_t *tile, int D, int value, int block, int tok,
                                               bool live) {
  const int part = threadIdx.x & 3;
  float hi = x[0], lo = x[0];
  uint64_t x2[4], none = 0;  // `none` stays 0 unless a value is not finite: 0 x infinity and 0 x NaN are NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = fmaxf(hi, x[i]);
    lo = fminf(lo, x[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x2[i] = f2_pack(x[2 * i], x[2 * i + 1]);
    none = f2_fma(x2[i], 0, none);
  }
  float n0, n1;
  f2_unpack(none, n0, n1);
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  const uint32_t bad = __ballot_sync(0xffffffffu, !(n0 + n1 == 0.f));
  const bool fine = ((bad >> (threadIdx.x & 28)) & 15u) == 0;
  const float d = (hi >= -lo ? hi : lo) * -0.125f;
  uint32_t q[8];  // the codes, in the low bytes
  if (fabsf(d) > 1e-30f) {
    // x / d, correctly rounded, by Markstein's method: with r the rounded reciprocal, a quotient corrected once by
    // its remainder is the rounded one.  (A quotient so small that the remainder underflows changes nothing: 8.5 is
    // added to it.)  x / d >= -8, so the code is not negative; floor by rounding down at 2^23.
    const float r = __frcp_rn(d);
    const uint64_t r2 = f2_pack(r, r), d2 = f2_pack(-d, -d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t q0 = f2_mul(x2[i], r2), q1 = f2_fma(f2_fma(q0, d2, x2[i]), r2, q0);
      float a, b;
      f2_unpack(f2_add(q1, f2_pack(8.5f, 8.5f)), a, b);
      q[2 * i] = __float_as_uint(__fadd_rd(fminf(a, 15.5f), 8388608.f));
      q[2 * i + 1] = __float_as_uint(__fadd_rd(fminf(b, 15.5f), 8388608.f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i] = (uint32_t)(d == 0.f ? 8.f : fminf(__fadd_rn(__fdiv_rn(x[i], d), 8.5f), 15.5f));
  }
  // byte j of the block = code j | code j + 16 << 4: lanes 0 and 1 hold codes 0..15, lanes 2 and 3 codes 16..31
  uint32_t w[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const uint32_t c = __byte_perm(__byte_perm(q[4 * z], q[4 * z + 1], 0x0040), __byte_perm(q[4 * z + 2], q[4 * z + 3], 0x0040), 0x5410);
    w[z] = c | (__shfl_xor_sync(0xffffffffu, c, 2) << 4);
    if (!fine) w[z] = 0;
  }
  if (!live) return;
  if (part < 2) {
    *reinterpret_cast<uint2 *>(tile + kv_code_off(D, value, block, tok) + 8 * part) = make_uint2(w[0], w[1]);
  } else if (part == 2) {
    const __half h = fine ? __float2half_rn(fminf(fmaxf(d, -65504.f), 65504.f)) : __ushort_as_half(0x7E00);
    *reinterpret_cast<__half *>(tile + kv_scale_off(D, value, block, tok)) = h;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendCtas) kv_append_kernel(const AppendJob j) {
  constexpr int L = D / 8;         // lanes of one head
  constexpr int HPW = 32 / L;      // heads that a warp handles at once
  constexpr int kAhead = 4;        // turns on their way (six or eight are no faster)
  __shared__ Raw8<T> ring[kAppendWarps][kAhead][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int total = j.hq + 2 * j.hkv, parts = (total + j.per_warp - 1) / j.per_warp;
  const int64_t item = (int64_t)blockIdx.x * kAppendWarps + warp;
  const int i = (int)(item / parts), part = (int)(item % parts);
  if (i >= j.n_tokens) return;
  const int sub = lane / L, dim = (lane % L) * 8;
  const int h0 = part * j.per_warp, h1 = min(h0 + j.per_warp, total);
  // this lane's values of the turn that begins at head hb (past the last head: that head's again)
  const T *const q_in = static_cast<const T *>(j.q.data) + i * j.q.token_stride + dim;
  const T *const k_in = static_cast<const T *>(j.k.data) + i * j.k.token_stride + dim;
  const T *const v_in = static_cast<const T *>(j.v.data) + i * j.v.token_stride + dim;
  const int first_k = j.hq, first_v = j.hq + j.hkv;  // in the list of q, k and v heads
  Raw8<T>(*const mine)[32] = ring[warp];
  auto fetch = [&](int hb, int slot) {
    const int h = min(hb + sub, h1 - 1);
    if (hb < h1)
      copy_raw(&mine[slot][lane], h < first_k ? q_in + h * j.q.head_stride
                                              : h < first_v ? k_in + (h - first_k) * j.k.head_stride
                                                            : v_in + (h - first_v) * j.v.head_stride);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // The values come through shared memory, kAhead turns before they are used: enough bytes on their way without
  // holding registers, which are what limits the warps.  The first ones are asked for before the token's place, which is
  // a chain of loads.
#pragma unroll 1
  for (int u = 0; u < kAhead; ++u) fetch(h0 + u * HPW, u);
  const TokenPlace at = place_token(j.c, j.starts, j.cu, i);
  const bool no_rot = j.rot > 0 && (at.pos < 0 || at.pos >= j.n_pos);
  if (lane == 0 && j.c.status) {
    const int bits = (at.pos < 0 ? MOE_KV_BAD_LENGTH : (at.page < 0 ? MOE_KV_BAD_PAGE : 0)) |
                     (at.pos >= 0 && no_rot ? MOE_KV_BAD_POSITION : 0);
    if (bits) atomicOr(j.c.status, bits);
  }
  T *const q_to = static_cast<T *>(j.q_out) + (int64_t)i * j.hq * D + dim;
  T *const k_to = static_cast<T *>(j.k_out) + (int64_t)i * j.hkv * D + dim;
  if (at.pos < 0 || no_rot) {  // the token has no place: its rows are NaN
    asm volatile("cp.async.wait_all;" ::: "memory");
    const float none[8] = {a_nan(), a_nan(), a_nan(), a_nan(), a_nan(), a_nan(), a_nan(), a_nan()};
    for (int h = h0 + sub; h < min(h1, first_v); h += HPW) {
      if (h < first_k) store8(q_to + h * D, none);
      else if (j.k_out) store8(k_to + (h - first_k) * D, none);
    }
    return;
  }
  const bool turned = dim < j.rot;
  float c[8], s[8];  // of this thread's values; s carries the sign of the rotation's other term
  int partner = lane;
  if (turned) {
    const float *ct = j.cos + at.pos * (j.rot / 2), *st = j.sin + at.pos * (j.rot / 2);
    if (j.interleaved) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(ct + dim / 2));
      const float4 b = __ldg(reinterpret_cast<const float4 *>(st + dim / 2));
      const float cc[4] = {a.x, a.y, a.z, a.w}, ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        c[z] = cc[z / 2];
        s[z] = (z & 1) ? ss[z / 2] : -ss[z / 2];
      }
    } else {
      const int first = dim < j.rot / 2, o = first ? dim : dim - j.rot / 2;
      float ss[8];
      expand8(load_raw(ct + o), c);
      expand8(load_raw(st + o), ss);
#pragma unroll
      for (int z = 0; z < 8; ++z) s[z] = first ? -ss[z] : ss[z];
      partner = first ? lane + j.rot / 16 : lane - j.rot / 16;
    }
  }
  const bool writes = at.page >= 0;
  uint8_t *const tiles = static_cast<uint8_t *>(j.c.pages) + (int64_t)(at.page < 0 ? 0 : at.page) * j.c.page_stride +
                         kv_tile_off(D, j.c.page_size, 0, at.in_page);
  const int64_t tile_stride = kv_tile_off(D, j.c.page_size, 1, 0);  // from head to head
  // (one copy of the turn's code: for a token or two, fetching it is a good part of the time)
  int slot = 0;
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += HPW) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    __syncwarp();
    const Raw8<T> now = mine[slot][lane], far = mine[slot][partner];
    __syncwarp();
    fetch(hb + kAhead * HPW, slot);
    slot = (slot + 1) % kAhead;
    const int h = min(hb + sub, h1 - 1);
    const bool live = hb + sub < h1;
    const int hh = h < first_v ? h - first_k : h - first_v;  // key or value head
    float x[8];
    expand8(now, x);
    if (j.rot > 0 && hb < first_v) {  // warp-uniform: some lane holds a query or key head
      // a pair is (z, z ^ 1) of this thread, or the partner lane's value z
      float o[8];
      if (j.interleaved) {
#pragma unroll
        for (int z = 0; z < 8; ++z) o[z] = x[z ^ 1];
      } else {
        expand8(far, o);
      }
      // (one by one: of packed pairs a product and the sum after it came out fused)
      if (turned && h < first_v)
#pragma unroll
        for (int z = 0; z < 8; ++z) x[z] = __fadd_rn(__fmul_rn(x[z], c[z]), __fmul_rn(o[z], s[z]));
      if (live && h < first_k) store8(q_to + h * D, x);
      else if (live && h < first_v && j.k_out) store8(k_to + hh * D, x);
    } else if (live && h < first_v) {
      if (h < first_k) store8(q_to + h * D, x);
      else if (j.k_out) store8(k_to + hh * D, x);
    }
    if (hb + HPW > first_k)  // warp-uniform: some lane holds a key or value head
      quantise_store(x, tiles + hh * tile_stride, D, h >= first_v, dim / 32, at.row, live && writes && h >= first_k);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_read_kernel(const AppendJob j) {
  constexpr int L = D / 8, HPW = 32 / L;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int total = 2 * j.hkv, parts = (total + j.per_warp - 1) / j.per_warp;
  const int64_t item = (int64_t)blockIdx.x * kAppendWarps + warp;
  const int i = (int)(item / parts), part = (int)(item % parts);
  if (i >= j.n_tokens) return;
  const int sub = lane / L, dim = (lane % L) * 8;
  const TokenPlace at = place_token(j.c, j.starts, j.cu, i);
  if (lane == 0 && j.c.status && at.page < 0)
    atomicOr(j.c.status, at.pos < 0 ? MOE_KV_BAD_LENGTH : MOE_KV_BAD_PAGE);
  const int h0 = part * j.per_warp, h1 = min(h0 + j.per_warp, total);
  const uint8_t *page = static_cast<const uint8_t *>(j.c.pages) + (int64_t)(at.page < 0 ? 0 : at.page) * j.c.page_stride;
  const int sh = (dim & 16) ? 4 : 0;
  constexpr int kBatch = 4;  // heads asked for before the first is used
#pragma unroll 1
  for (int hb = h0 + sub; hb < h1; hb += kBatch * HPW) {
    uint2 w[kBatch];
    __half d[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      w[u] = make_uint2(0u, 0u);
      d[u] = __ushort_as_half(0x7E00);  // without a page: NaN
      const int h = hb + u * HPW, value = h >= j.hkv;
      if (h < h1 && at.page >= 0) {
        const uint8_t *tile = page + kv_tile_off(D, j.c.page_size, value ? h - j.hkv : h, at.in_page);
        w[u] = __ldcs(reinterpret_cast<const uint2 *>(tile + kv_code_off(D, value, dim / 32, at.row) + (dim & 8)));
        d[u] = *reinterpret_cast<const __half *>(tile + kv_scale_off(D, value, dim / 32, at.row));
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = hb + u * HPW, value = h >= j.hkv;
      T *out = static_cast<T *>(value ? j.v_out : j.k_out);
      if (h >= h1 || !out) continue;
      float y[8];
#pragma unroll
      for (int z = 0; z < 8; ++z)
        y[z] = (float)((int)(((z < 4 ? w[u].x : w[u].y) >> (8 * (z & 3) + sh)) & 15u) - 8) * __half2float(d[u]);
      store8(out + ((int64_t)i * j.hkv + (value ? h - j.hkv : h)) * D + dim, y);
    }
  }
}

// Heads per warp, in whole turns of the warp: all of a token's where the tokens alone make 32 warps per SM, fewer where
// they do not, one turn at least.  Measured with the read: 18439 tokens 107 us so and 308 us at one turn per warp (every
// warp finds its token's place anew); one token 5.1 us so and 11.0 us with all heads in one warp, 64 tokens 7.1 and 18.2.
int heads_per_warp(int n_tokens, int total, int per_turn) {
  const int64_t warps = 152 * 32;
  const int64_t turns = (total + per_turn - 1) / per_turn;
  const int64_t want = std::min<int64_t>(turns, std::max<int64_t>(1, (int64_t)n_tokens * turns / warps));
  return (int)want * per_turn;
}

template <template <typename, int> class Launch>
int by_type(const AppendJob &j, int dtype, cudaStream_t st) {
  const int D = j.c.head_dim;
#define MOE_BY_D(T)                                     \
  (D == 64 ? Launch<T, 64>::go(j, st) : D == 128 ? Launch<T, 128>::go(j, st) : Launch<T, 256>::go(j, st))
  switch (dtype) {
    case MOE_F32: return MOE_BY_D(float);
    case MOE_BF16: return MOE_BY_D(__nv_bfloat16);
    default: return MOE_BY_D(__half);
  }
#undef MOE_BY_D
}

template <typename T, int D>
struct LaunchAppend {
  static int go(AppendJob j, cudaStream_t st) {
    const int total = j.hq + 2 * j.hkv;
    j.per_warp = heads_per_warp(j.n_tokens, total, 256 / D);
    const int64_t items = (int64_t)j.n_tokens * ((total + j.per_warp - 1) / j.per_warp);
    kv_append_kernel<T, D><<<(unsigned)((items + kAppendWarps - 1) / kAppendWarps), 32 * kAppendWarps, 0, st>>>(j);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
};
template <typename T, int D>
struct LaunchRead {
  static int go(AppendJob j, cudaStream_t st) {
    const int total = 2 * j.hkv;
    j.per_warp = heads_per_warp(j.n_tokens, total, 256 / D);
    const int64_t items = (int64_t)j.n_tokens * ((total + j.per_warp - 1) / j.per_warp);
    kv_read_kernel<T, D><<<(unsigned)((items + kAppendWarps - 1) / kAppendWarps), 32 * kAppendWarps, 0, st>>>(j);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
};

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int64_t moe_kv_page_bytes(int32_t n_kv_heads, int32_t head_dim, int32_t page_size) {
  if (!kv_sizes_ok(n_kv_heads, head_dim, page_size)) return 0;
  return (int64_t)n_kv_heads * (page_size / kKvTile) * kv_tile_bytes(head_dim);
}

MOE_API int moe_kv_append(const moe_kv_cache *c, const int32_t *starts, const int32_t *cu_tokens, int32_t n_tokens,
                          const moe_tensor *q, int32_t n_q_heads, const moe_tensor *k, const moe_tensor *v,
                          const float *cos, const float *sin, int32_t rot_dim, int32_t n_positions,
                          int32_t interleaved, void *q_out, void *k_out, int32_t dtype, void *cuda_stream) {
  if (const int rc = check_cache(c)) return rc;
  if (n_tokens < 0 || !k || !v || dtype < MOE_F32 || dtype > MOE_F16) return MOE_ERR_INVALID_ARG;
  if (n_tokens == 0) return MOE_OK;
  if (c->n_seqs == 0) return MOE_ERR_INVALID_ARG;
  const int size = dtype == MOE_F32 ? 4 : 2;
  const bool has_q = q && q->data;
  if (!starts || !cu_tokens || rot_dim < 0 || rot_dim > c->head_dim || rot_dim % 16) return MOE_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!cos || !sin || n_positions <= 0 || (uintptr_t)cos % 16 || (uintptr_t)sin % 16))
    return MOE_ERR_INVALID_ARG;
  if (has_q && (n_q_heads <= 0 || n_q_heads > kMaxAttnHeads || !q_out)) return MOE_ERR_INVALID_ARG;
  if (const int rc = check_tensor(k, size)) return rc;
  if (const int rc = check_tensor(v, size)) return rc;
  if (has_q)
    if (const int rc = check_tensor(q, size)) return rc;
  if ((uintptr_t)q_out % 16 || (uintptr_t)k_out % 16) return MOE_ERR_INVALID_ARG;
  AppendJob j = {};
  j.c = *c;
  j.starts = starts;
  j.cu = cu_tokens;
  j.n_tokens = n_tokens;
  if (has_q) j.q = *q;
  j.k = *k;
  j.v = *v;
  j.hq = has_q ? n_q_heads : 0;
  j.hkv = c->n_kv_heads;
  j.cos = cos;
  j.sin = sin;
  j.rot = rot_dim;
  j.n_pos = n_positions;
  j.interleaved = interleaved != 0;
  j.q_out = q_out;
  j.k_out = k_out;
  return by_type<LaunchAppend>(j, dtype, (cudaStream_t)cuda_stream);
}

MOE_API int moe_kv_read(const moe_kv_cache *c, const int32_t *starts, const int32_t *cu_tokens, int32_t n_tokens,
                        void *k_out, void *v_out, int32_t dtype, void *cuda_stream) {
  if (const int rc = check_cache(c)) return rc;
  if (n_tokens < 0 || dtype < MOE_F32 || dtype > MOE_F16) return MOE_ERR_INVALID_ARG;
  if (n_tokens == 0 || (!k_out && !v_out)) return MOE_OK;
  if (c->n_seqs == 0) return MOE_ERR_INVALID_ARG;
  if (!starts || !cu_tokens || (uintptr_t)k_out % 16 || (uintptr_t)v_out % 16) return MOE_ERR_INVALID_ARG;
  AppendJob j = {};
  j.c = *c;
  j.starts = starts;
  j.cu = cu_tokens;
  j.n_tokens = n_tokens;
  j.hkv = c->n_kv_heads;
  j.k_out = k_out;
  j.v_out = v_out;
  return by_type<LaunchRead>(j, dtype, (cudaStream_t)cuda_stream);
}
