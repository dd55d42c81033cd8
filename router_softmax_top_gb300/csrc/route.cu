// Routing: scores, a bias for balance, groups, top-k, weights.
//
// p = softmax(x) or 1 / (1 + exp(-x)), c = p + b, the top_groups groups of largest worth
// (largest c, or sum of the two largest), the k largest c of their experts, weights
// scale p (/ sum p).
//
// Bound: launch and latency for a few tokens, issue slots for many.  A warp takes a
// token, a lane VPL neighbouring experts: the lowest lane that holds the largest key
// then holds the lowest expert among equals, so a round of the choice is one warp
// maximum, one ballot and the winner's own search.
//
// Which experts are chosen must not depend on how p was rounded, as a border may lie
// between two values.  Without a bias the order is that of the logits, exactly.  With
// one (or with sums per group) values are formed in 32 bits with a bound on their error;
// where two neighbours in the order are nearer than their bounds, and are not equal by
// having the same logit and bias, the token is done again in 64 bits.
#include <math.h>

#include "attn_common.cuh"
#include "moe_route.h"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;

struct RouteJob {
  const void *logits;
  int64_t stride;
  int n, E, k, sigmoid, groups, kept, size, top2, renorm;
  float scale;
  const float *bias;
  int32_t *ids;
  float *weights;
  int32_t *status;
};

__device__ __forceinline__ float r_float(float x) { return x; }
__device__ __forceinline__ float r_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float r_float(__half x) { return __half2float(x); }

// Keys that order like the values (-0 as +0); 0 is below all of them.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v == 0. ? 0. : v);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ double of_key(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float x_exp(float x) { return expf(x); }
__device__ __forceinline__ double x_exp(double x) { return exp(x); }
template <typename F>
__device__ __forceinline__ F inf_of() { return (F)a_inf(); }

// Bound on the error of a value c = p + b formed in 32 bits: `arg` is the exponential's argument, whose rounding (softmax
// takes the largest logit away) is relative to p.  expf is good to 2 steps, the sum over E to 2^-19 for E <= 1024 in
// strides and a tree (32 + 5 additions), quotient and sum to a step each.
__device__ __forceinline__ float error_of(float p, float arg, float c) {
  return p * fmaf(fabsf(arg), 1.2e-7f, 4e-6f) + fabsf(c) * 1.2e-7f + 1e-37f;
}

// The choice, with values of type F (float or double): ids on lanes 0..k (the k + 1st too, where there is one; -1: none).
// Float: returns whether the choice is certain.  v: the lane's logits; x of experts past E is never looked at.
template <typename F, int VPL>
__device__ __forceinline__ bool choose(const RouteJob &j, const float (&x)[VPL], float top, float *group_mem, int *id_out) {
  using K = decltype(key_of(F(0)));
  const int lane = threadIdx.x & 31, e0 = lane * VPL;
  constexpr bool rough = sizeof(F) == 4;
  K key[VPL];
  const bool by_logit = !j.bias;
  F z = 0;
  if (!j.sigmoid && (j.bias || (j.groups > 1 && j.top2))) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < j.E) z += x_exp((F)x[i] - (F)top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  auto score = [&](float v) -> F {
    return j.sigmoid ? F(1) / (F(1) + x_exp(-(F)v)) : x_exp((F)v - (F)top) / z;
  };
  auto argument = [&](float v) { return j.sigmoid ? v : v - top; };
  bool sure = true;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0;
    if (e0 + i < j.E) {
      F c = (F)x[i];
      if (!by_logit && x[i] > -a_inf()) c = score(x[i]) + (F)__ldg(j.bias + e0 + i);
      key[i] = key_of(c);
    }
  }
  if (j.groups > 1) {
    // a group's worth: its members by `lanes` lanes each, then theirs joined
    F *mem = reinterpret_cast<F *>(group_mem);
    float *err_mem = group_mem + (rough ? 1 : 2) * 32 * VPL;
    const bool sums = j.top2 && j.size > 1;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < j.E) {
        F c = of_key(key[i]);
        float err = 0.f;
        if (sums && x[i] > -a_inf()) {
          const F p = score(x[i]);
          if (by_logit) c = p;
          if (rough) err = error_of((float)p, argument(x[i]), (float)c);
        } else if (rough && !by_logit && x[i] > -a_inf()) {
          err = error_of((float)score(x[i]), argument(x[i]), (float)c);
        }
        mem[e0 + i] = c;
        if (rough) err_mem[e0 + i] = err;
      }
    __syncwarp();
    int lanes = 1;
    while (2 * lanes * j.groups <= 32) lanes *= 2;
    const int g = lane / lanes;
    F a = -inf_of<F>(), b = -inf_of<F>();
    float err = 0.f;  // the largest of the group's (of two members: twice that)
    if (g < j.groups)
      for (int m = lane % lanes; m < j.size; m += lanes) {
        const F c = mem[g * j.size + m];
        if (rough) err = fmaxf(err, err_mem[g * j.size + m]);
        b = c > a ? a : (c > b ? c : b);
        a = c > a ? c : a;
      }
    for (int o = 1; o < lanes; o <<= 1) {
      const F oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
      if (rough) err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
      b = oa > a ? (a > ob ? a : ob) : (oa > b ? oa : b);
      a = oa > a ? oa : a;
    }
    F worth = a;
    if (sums && b > -inf_of<F>()) {
      worth = a + b;
      err = 2.f * err + fabsf((float)worth) * 1.2e-7f;
    }
    // kept: fewer than `kept` groups are worth more (or as much, and come before)
    int rank = 0;
    for (int h = 0; h < j.groups; ++h) {
      const F w = __shfl_sync(0xffffffffu, worth, h * lanes);
      rank += w > worth || (w == worth && h < g);
    }
    const bool mine = g < j.groups && lane % lanes == 0;
    const uint32_t keep = __ballot_sync(0xffffffffu, mine && rank < j.kept);  // bit g * lanes
    if (rough && j.kept < j.groups && !(by_logit && !sums)) {
      const int in = __ffs(__ballot_sync(0xffffffffu, mine && rank == j.kept - 1)) - 1;
      const int out = __ffs(__ballot_sync(0xffffffffu, mine && rank == j.kept)) - 1;
      const F wi = __shfl_sync(0xffffffffu, worth, in), wo = __shfl_sync(0xffffffffu, worth, out);
      // (of the groups beyond these two some may have a larger bound)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
      sure = (float)wi - (float)wo > 2.f * err || (wo == -inf_of<F>() && wi > wo);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < j.E && !((keep >> ((e0 + i) / j.size * lanes)) & 1u)) key[i] = 0;
    __syncwarp();
  }
  // rounds: the largest key left; the lane's own largest, and where it is (its first among equals)
  K best = 0;
  int at = 0;
  auto search = [&]() {
    best = key[0];
    at = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
  };
  search();
  K my_key = 0;
  int my_id = -1;
  const int rounds = min(j.k + (rough && !by_logit ? 1 : 0), 32 + 1);
  K extra = 0;
  int extra_id = -1;
  for (int q = 0; q < rounds; ++q) {
    const K m = warp_max(best);
    if (m == 0) break;  // none left
    const int who = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
    const int id = __shfl_sync(0xffffffffu, e0 + at, who);
    if (q < 32) {
      if (lane == q) {
        my_key = m;
        my_id = id;
      }
    } else {
      extra = m;
      extra_id = id;
    }
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = 0;
      search();
    }
  }
  *id_out = my_id;
  if constexpr (rough) {
    if (by_logit) return sure;
    // neighbours in the order: lane q against lane q + 1
    K next = __shfl_down_sync(0xffffffffu, my_key, 1);
    int next_id = __shfl_down_sync(0xffffffffu, my_id, 1);
    if (lane == 31) {
      next = extra;
      next_id = extra_id;
    }
    // their logits, from the lanes that hold them
    float mine_x = 0.f, next_x = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float a = __shfl_sync(0xffffffffu, x[i], max(my_id, 0) / VPL), b = __shfl_sync(0xffffffffu, x[i], max(next_id, 0) / VPL);
      if (max(my_id, 0) % VPL == i) mine_x = a;
      if (max(next_id, 0) % VPL == i) next_x = b;
    }
    bool near = false;
    if (lane < j.k && my_id >= 0 && next_id >= 0) {
      const float c = of_key((uint32_t)my_key), d = of_key((uint32_t)next);
      const bool open = mine_x > -a_inf(), next_open = next_x > -a_inf();
      if (open && next_open) {
        const float err = error_of((float)score(mine_x), argument(mine_x), c) +
                          error_of((float)score(next_x), argument(next_x), d);
        near = !(c - d > err) && !(mine_x == next_x && __ldg(j.bias + my_id) == __ldg(j.bias + next_id));
      }
    }
    return sure && !__any_sync(0xffffffffu, near);
  }
  return true;
}

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteJob j) {
  // per warp: values and bounds of the experts, for the groups' worth
  __shared__ __align__(16) float group_mem[kRouteWarps][VPL * 32 * 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * VPL;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= j.n) return;
  const T *row = static_cast<const T *>(j.logits) + (int64_t)t * j.stride;
  float x[VPL];
  constexpr int kVec = VPL * (int)sizeof(T) >= 16 ? 16 : VPL * (int)sizeof(T);  // bytes of a load
  if (VPL > 1 && j.E % VPL == 0 && ((uintptr_t)row & (kVec - 1)) == 0) {
    if (e0 < j.E) {
      if constexpr (kVec == 16) {
        uint4 w[VPL * sizeof(T) / 16];
#pragma unroll
        for (int i = 0; i < (int)(VPL * sizeof(T) / 16); ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(row + e0) + i);
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = r_float(reinterpret_cast<const T *>(w)[i]);
      } else if constexpr (kVec == 8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(row + e0));
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = r_float(reinterpret_cast<const T *>(&w)[i]);
      } else if constexpr (kVec == 4) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(row + e0));
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = r_float(reinterpret_cast<const T *>(&w)[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < j.E) x[i] = r_float(row[e0 + i]);
  }
  float top = -a_inf();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (e0 + i >= j.E) {
      x[i] = -a_inf();
    } else {
      bad |= !(x[i] < a_inf());
      if (j.bias) bad |= !(fabsf(__ldg(j.bias + e0 + i)) < a_inf());
    }
    top = fmaxf(top, x[i]);
  }
  int32_t *ids = j.ids + (int64_t)t * j.k;
  float *weights = j.weights + (int64_t)t * j.k;
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0 && j.status) atomicOr(j.status, MOE_ROUTE_BAD_LOGIT);
    if (lane < j.k) {
      ids[lane] = lane;
      weights[lane] = a_nan();
    }
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top == -a_inf()) top = 0.f;  // all closed
  int id;
  if (!choose<float, VPL>(j, x, top, group_mem[warp], &id)) choose<double, VPL>(j, x, top, group_mem[warp], &id);
  // ---- weights: lane q has the choice q
  const bool live = lane < j.k;
  float v = -a_inf();
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float a = __shfl_sync(0xffffffffu, x[i], max(id, 0) / VPL);
    if (max(id, 0) % VPL == i) v = a;
  }
  if (!live) v = -a_inf();
  float w;
  if (j.renorm) {
    // p over the sum of p, with a common factor taken out that keeps both numbers
    float m = j.sigmoid ? fminf(v, 0.f) : v;
    float most = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    w = v > -a_inf() ? expf(m - most) : 0.f;
    if (j.sigmoid) w /= 1.f + expf(-fabsf(v));
    if (!(v > -a_inf())) w = 0.f;
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.f ? w / sum : 0.f;
  } else if (j.sigmoid) {
    w = 1.f / (1.f + expf(-v));
  } else {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) z += expf(x[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    w = z > 0.f ? expf(v - top) / z : 0.f;
  }
  if (live) {
    ids[lane] = id;
    weights[lane] = w * j.scale;
  }
}

template <typename T>
int launch_route(const RouteJob &j, cudaStream_t st) {
  const unsigned grid = (unsigned)((j.n + kRouteWarps - 1) / kRouteWarps);
  const int v = (j.E + 31) / 32;
  if (v <= 1) route_kernel<T, 1><<<grid, 32 * kRouteWarps, 0, st>>>(j);
  else if (v <= 2) route_kernel<T, 2><<<grid, 32 * kRouteWarps, 0, st>>>(j);
  else if (v <= 4) route_kernel<T, 4><<<grid, 32 * kRouteWarps, 0, st>>>(j);
  else if (v <= 8) route_kernel<T, 8><<<grid, 32 * kRouteWarps, 0, st>>>(j);
  else if (v <= 16) route_kernel<T, 16><<<grid, 32 * kRouteWarps, 0, st>>>(j);
  else route_kernel<T, 32><<<grid, 32 * kRouteWarps, 0, st>>>(j);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int moe_route(const moe_routing *r, const void *logits, int64_t token_stride, int32_t n_tokens, const float *bias,
                      int32_t *ids, float *weights, int32_t dtype, int32_t *status, void *cuda_stream) {
  if (!r || n_tokens < 0 || r->n_experts <= 0 || r->top_k <= 0 || r->n_groups <= 0 || r->top_groups <= 0 ||
      r->top_groups > r->n_groups || r->n_experts % r->n_groups ||
      r->top_k > r->n_experts / r->n_groups * r->top_groups || r->score < MOE_SCORE_SOFTMAX ||
      r->score > MOE_SCORE_SIGMOID || r->group_score < MOE_GROUP_MAX || r->group_score > MOE_GROUP_TOP2 ||
      !(fabsf(r->scale) <= 3.4e38f) || dtype < MOE_F32 || dtype > MOE_F16)
    return MOE_ERR_INVALID_ARG;
  if (r->n_experts > kMaxExperts || r->top_k > kMaxTopK || r->n_groups > 32) return MOE_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MOE_OK;
  const int size = dtype == MOE_F32 ? 4 : 2;
  if (!logits || !ids || !weights || (uintptr_t)logits % size || (uintptr_t)bias % 4 || (uintptr_t)ids % 4 ||
      (uintptr_t)weights % 4 || (uintptr_t)status % 4)
    return MOE_ERR_INVALID_ARG;
  const RouteJob j = {logits,        token_stride, n_tokens,       r->n_experts, r->top_k, r->score, r->n_groups,
                      r->top_groups, r->n_experts / r->n_groups, r->group_score, r->renormalise != 0, r->scale, bias, ids,
                      weights,       status};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  return dtype == MOE_F32    ? launch_route<float>(j, st)
         : dtype == MOE_BF16 ? launch_route<__nv_bfloat16>(j, st)
                             : launch_route<__half>(j, st);
}
