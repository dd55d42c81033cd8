// Shared by the attention operators: argument checks, and the mbarrier, bulk-copy
// and matrix-instruction helpers of their kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_layout.h"
#include "moe_attention.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {

constexpr int kMaxAttnHeads = 1024;
constexpr int kMaxPageSize = 65536;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMostScale = 2.3e38f;  // of a score: times log2(e) it is still a number
constexpr uint64_t kAttnWaitNs = 2000000000ull;  // limit of every device wait
constexpr uint32_t kAttnSpin = 1u << 26;

inline bool kv_sizes_ok(int n_kv_heads, int head_dim, int page_size) {
  return n_kv_heads > 0 && n_kv_heads <= kMaxAttnHeads && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         page_size > 0 && page_size <= kMaxPageSize && page_size % kKvTile == 0;
}

inline int check_cache(const moe_kv_cache *c) {
  if (!c || c->n_seqs < 0 || c->n_pages < 0 || c->table_width < 0 || c->n_kv_heads <= 0 || c->page_size <= 0)
    return MOE_ERR_INVALID_ARG;
  if (!kv_sizes_ok(c->n_kv_heads, c->head_dim, c->page_size)) return MOE_ERR_UNSUPPORTED;
  const int64_t need = (int64_t)c->n_kv_heads * (c->page_size / kKvTile) * kv_tile_bytes(c->head_dim);
  if (c->page_stride < need || c->page_stride % 16 || (uintptr_t)c->pages % 16 || (!c->pages && c->n_pages > 0))
    return MOE_ERR_INVALID_ARG;
  if (c->n_seqs > 0 && c->table_width > 0 && (!c->page_table || c->table_stride < c->table_width)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Token-major input: present, base and strides whole multiples of 16 bytes.
inline int check_tensor(const moe_tensor *t, int size) {
  if (!t || !t->data) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)t->data % 16 || t->token_stride * size % 16 || t->head_stride * size % 16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t a_smem(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void a_mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a_smem(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void a_mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a_smem(bar)) : "memory");
}
__device__ __forceinline__ void a_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a_smem(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint64_t a_now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool a_mbar_try(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(a_smem(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for the phase of `bar` with the given parity; false once it gave
// up (kAttnWaitNs, kAttnSpin polls) or *fail is set by another role of the CTA.
__device__ __forceinline__ bool a_mbar_wait(uint64_t *bar, uint32_t parity, const int *fail = nullptr) {
  if (a_mbar_try(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < kAttnSpin; ++i) {
    if (a_mbar_try(bar, parity)) return true;
    if ((i & 255u) == 255u) {
      if (fail && *reinterpret_cast<const volatile int *>(fail)) return false;
      const uint64_t now = a_now_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kAttnWaitNs) return false;
    }
  }
  return false;
}
// The wait for work that still reads or writes memory about to be given back: bounded by time, but not cut short by
// *fail, which is set just where such work may be in flight.
__device__ __forceinline__ bool a_mbar_drain(uint64_t *bar, uint32_t parity) { return a_mbar_wait(bar, parity, nullptr); }
// Bulk copy of contiguous bytes into shared memory (addresses and size multiples of 16).
__device__ __forceinline__ void a_bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   a_smem(dst)),
               "l"(src), "r"(bytes), "r"(a_smem(bar))
               : "memory");
}
// Two fp32 values in one instruction, each rounded by itself.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float a_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float a_inf() { return __int_as_float(0x7f800000); }
__device__ __forceinline__ float a_nan() { return __int_as_float(0x7fffffff); }
#endif

}  // namespace moe
