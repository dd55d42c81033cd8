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
// where two of the chosen that are neighbours in the order, or the last of them and any that
// is not chosen, are nearer than their bounds, and are not equal by having the same logit and
// bias, the few candidates, or the token, are done again in 64 bits.
//
// Measured: 16384 tokens of 256 experts in 8 groups, bf16, sigmoid, bias, 8 of 4 groups: 26.5
// us, 950 instructions a token, of an SM's issue slots 64%; in 64 bits throughout it was 72 us.
// 64 tokens 4.0 us, one of 128 experts 2.7 us.  How many tokens need 64 bits depends on the
// values: with a bias of zeros and logits of standard deviation 1.5, 6 and 15 the same call
// takes 34, 109 and 285 us (scores crowd at 1, and 32 bits cannot tell groups apart), without
// groups 16, 36 and 231 us, and by softmax 16, 17 and 19 us.
#include <math.h>

#include <algorithm>

#include "attn_common.cuh"
#include "moe_route.h"

namespace moe {
namespace {

constexpr int kRouteWarps = 4, kRouteSms = 152;

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

// A key that orders like the value (-0 as +0); 0 is below all of them.
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v == 0. ? 0. : v);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}
// The largest of a warp's values; NaN where there is one.
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// VPL neighbouring values, in as wide loads as their address allows.
template <int VPL, typename T>
__device__ __forceinline__ void load_values(const T *p, float (&x)[VPL]) {
  constexpr int kBytes = VPL * (int)sizeof(T), kVec = kBytes >= 16 ? 16 : kBytes;
  if (VPL > 1 && ((uintptr_t)p & (kVec - 1)) == 0) {
    if constexpr (kVec == 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        constexpr int n = 16 / (int)sizeof(T);
#pragma unroll
        for (int z = 0; z < n; ++z) x[i * n + z] = r_float(reinterpret_cast<const T *>(&w)[z]);
      }
    } else if constexpr (kVec == 8) {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
#pragma unroll
      for (int z = 0; z < VPL; ++z) x[z] = r_float(reinterpret_cast<const T *>(&w)[z]);
    } else if constexpr (kVec == 4) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(p));
#pragma unroll
      for (int z = 0; z < VPL; ++z) x[z] = r_float(reinterpret_cast<const T *>(&w)[z]);
    }
  } else {
#pragma unroll
    for (int z = 0; z < VPL; ++z) x[z] = r_float(p[z]);
  }
}

// A score in 32 bits, and what its error is at most relative to it: the exponential's argument counts 2^-24 of itself twice,
// ex2 and the quotient 2^-22 each, the sum over E <= 1024 of softmax (32 + 5 additions) 2^-18.
__device__ __forceinline__ float quick_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float quick_sigmoid(float x) { return quick_inverse(1.f + a_exp2(x * -kLog2e)); }
__device__ __forceinline__ float quick_exp(float x) { return a_exp2(x * kLog2e); }
__device__ __forceinline__ float score_error(bool sigmoid, float arg) { return fmaf(fabsf(arg), 2e-7f, sigmoid ? 8e-7f : 5e-6f); }
constexpr float kSumStep = 1.2e-7f;   // of a sum's two roundings
constexpr float kFloor = 1e-37f;      // below it, scores are not held with their bits

// What the groups' members are worth, by lanes that have some of them each: a the largest, b the next.
__device__ __forceinline__ float least_of(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ float most_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double least_of(double a, double b) { return fmin(a, b); }
__device__ __forceinline__ double most_of(double a, double b) { return fmax(a, b); }
template <typename F>
__device__ __forceinline__ void top_two(F c, F &a, F &b) {
  b = most_of(b, least_of(a, c));
  a = most_of(a, c);
}
template <typename F>
__device__ __forceinline__ void join_two(F &a, F &b, int o) {
  const F oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
  b = most_of(least_of(a, oa), most_of(b, ob));
  a = most_of(a, oa);
}

// The kept groups: the 2^lg lanes of group h, from h 2^lg on, have its worth.  Returns a bit per group, at h 2^lg; rank:
// the calling lane's group's.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(F worth, int groups, int kept, int lg, int *rank) {
  const int lane = threadIdx.x & 31, g = lane >> lg;
  int r = 0;
#pragma unroll 4
  for (int h = 0; h < groups; ++h) {
    const F w = __shfl_sync(0xffffffffu, worth, h << lg);
    r += w > worth || (w == worth && h < g);
  }
  *rank = r;
  return __ballot_sync(0xffffffffu, g < groups && (g << lg) == lane && r < kept);
}

struct __align__(16) Pick {
  float cand_c[32];  // values that may be among the chosen, in the order of their experts
  int cand_id[32];
  float c[33];
  int id[33];
};

// The choice in 32 bits, into `pick`; whether it is certain.  x: the lane's logits (-inf past E), b: their bias.
template <int VPL, typename T>
__device__ __forceinline__ bool choose_quick(const RouteJob &j, const T *row, const float (&x)[VPL], const float (&b)[VPL],
                                             float top, float z, float *group_mem, Pick &pick) {
  const int lane = threadIdx.x & 31, e0 = lane * VPL;
  const bool by_logit = !j.bias, sums = j.top2 && j.size > 1;
  float c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) c[i] = x[i];
  float most_p = 0.f;
  if (!by_logit) {
    const float inv = quick_inverse(z);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float p = j.sigmoid ? quick_sigmoid(x[i]) : quick_exp(x[i] - top) * inv;
      most_p = fmaxf(most_p, p);
      c[i] = x[i] > -a_inf() ? p + b[i] : -a_inf();
    }
  }
  bool sure = true;
  if (j.groups > 1) {
    float d[VPL];
    if (by_logit && sums) {
      const float inv = quick_inverse(z);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float p = j.sigmoid ? quick_sigmoid(x[i]) : quick_exp(x[i] - top) * inv;
        most_p = fmaxf(most_p, p);
        d[i] = x[i] > -a_inf() ? p : -a_inf();
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = c[i];
    }
    // (a power of two of lanes per group, each lane's experts of one group: no shared memory needed)
    const int many = j.size / VPL;
    const bool direct = j.size % VPL == 0 && (many & (many - 1)) == 0;
    int lg = 31 - __clz(many);
    float w1 = -a_inf(), w2 = -a_inf();
    if (direct) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) top_two(d[i], w1, w2);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < j.E) group_mem[e0 + i] = d[i];
      __syncwarp();
      lg = 0;
      while ((2 << lg) * j.groups <= 32) ++lg;
      if ((lane >> lg) < j.groups)
        for (int m = lane & ((1 << lg) - 1); m < j.size; m += 1 << lg) top_two(group_mem[(lane >> lg) * j.size + m], w1, w2);
    }
    const int g = lane >> lg;
    for (int o = 0; o < lg; ++o) join_two(w1, w2, 1 << o);
    const float worth = sums && w2 > -a_inf() ? w1 + w2 : w1;
    int rank;
    const uint32_t keep = keep_groups(worth, j.groups, j.kept, lg, &rank);
    if (j.kept < j.groups && !(by_logit && !sums)) {
      const uint32_t first = __ballot_sync(0xffffffffu, g < j.groups && (g << lg) == lane);
      const int in = __ffs(__ballot_sync(0xffffffffu, rank == j.kept - 1) & first) - 1;
      const int out = __ffs(__ballot_sync(0xffffffffu, rank == j.kept) & first) - 1;
      const float wi = __shfl_sync(0xffffffffu, worth, in), wo = __shfl_sync(0xffffffffu, worth, out);
      // any group's error: p |argument| is at most 0.37 for what is below 1, and (1 - p) x for sigmoid's large ones
      const float size = w1 > -a_inf() && g < j.groups ? fmaxf(fabsf(w1), w2 > -a_inf() ? fabsf(w2) : 0.f) : 0.f;
      const float err = 2.f * (warp_max(most_p) * (j.sigmoid ? 8e-7f : 5e-6f) + 1e-7f + 2.f * kSumStep * warp_max(size));
      sure = wi - wo > 2.f * err || (wo == -a_inf() && wi > wo);
    }
    if (direct) {
      if (!((keep >> (g << lg)) & 1u)) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = -a_inf();
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < j.E && !((keep >> ((e0 + i) / j.size << lg)) & 1u)) c[i] = -a_inf();
    }
  }
  float best = c[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) best = fmaxf(best, c[i]);
  const int rounds = j.k + (by_logit ? 0 : 1);
  // Values from `least` on to the candidates, and nothing to the places after them; how many there are (of more than 32
  // not all are kept).
  auto collect = [&](float from) {
    const float least = fmaxf(from, -3.4028235e38f);  // what is closed is none
    int n = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) n += c[i] >= least;
    int end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    int at = end - n;
    n = __shfl_sync(0xffffffffu, end, 31);
    pick.cand_c[lane] = -a_inf();
    __syncwarp();
    if (n <= 32) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (c[i] >= least) {
          pick.cand_c[at] = c[i];
          pick.cand_id[at++] = e0 + i;
        }
    }
    __syncwarp();
    return n;
  };
  // The lanes' largest: with `rounds` of them taken, what is below the last of these is not among the chosen.  What is
  // left is as a rule few enough for a lane each, and a candidate's place is the number of those before it.
  float least = best, mine = best;
  for (int q = 0; q < rounds; ++q) {
    least = warp_max(mine);
    if (mine == least) mine = -a_inf();
  }
  const int n = collect(least);
  if (n < j.k) return false;  // closed experts follow, of the kept groups first: not told apart here
  if (n <= 32) {
    const float own = pick.cand_c[lane];
    int place = 0;
    uint32_t equal = 0;
    for (int s = 0; s < n; s += 4) {
      const float4 o = *reinterpret_cast<const float4 *>(&pick.cand_c[s]);
      place += (o.x > own) + (o.y > own) + (o.z > own) + (o.w > own);
      equal |= (uint32_t)((o.x == own ? 1 : 0) | (o.y == own ? 2 : 0) | (o.z == own ? 4 : 0) | (o.w == own ? 8 : 0)) << s;
    }
    place += __popc(equal & ((1u << lane) - 1u));  // (the candidates are in the order of their experts)
    if (lane < n && place < rounds) {
      pick.c[place] = own;
      pick.id[place] = pick.cand_id[lane];
    }
    if (lane == 0 && n < rounds) pick.id[n] = -1;
    __syncwarp();
  } else {
    // round by round: the largest left, of equal ones the lowest; the lane that has it looks for its next
    float left[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) left[i] = c[i];
    for (int q = 0; q < rounds; ++q) {
      const float m = warp_max(best);  // (there are more than 32)
      if (lane == __ffs(__ballot_sync(0xffffffffu, best == m)) - 1) {
        bool taken = false;
        int at = 0;
        best = -a_inf();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (!taken && left[i] == m) {
            taken = true;
            at = i;
            left[i] = -a_inf();
          }
          best = fmaxf(best, left[i]);
        }
        pick.c[q] = m;
        pick.id[q] = e0 + at;
      }
      __syncwarp();
    }
  }
  if (!sure || by_logit) return sure;
  // The chosen, neighbours in their order, are further apart than their errors, or equal by having the same logit and bias;
  // and so is the last of them from all that are not chosen: from the largest of those by the largest error that any
  // expert's value has (a smaller one may come from a larger score), or else from each.
  const float inv = quick_inverse(z);
  auto error_of = [&](float v, float c) {
    const float arg = j.sigmoid ? v : v - top;
    return (j.sigmoid ? quick_sigmoid(v) : quick_exp(arg) * inv) * score_error(j.sigmoid, arg) + kSumStep * fabsf(c) + kFloor;
  };
  const int a = lane < j.k ? pick.id[lane] : 0;
  const float ca = pick.c[lane], va = r_float(row[a]), ba = __ldg(j.bias + a), ea = error_of(va, ca);
  const float ce = __shfl_down_sync(0xffffffffu, ca, 1), ve = __shfl_down_sync(0xffffffffu, va, 1);
  const float be = __shfl_down_sync(0xffffffffu, ba, 1), ee = __shfl_down_sync(0xffffffffu, ea, 1);
  const bool near = lane < j.k - 1 && !(ca - ce > ea + ee) && !(va == ve && ba == be);
  const float last = pick.c[j.k - 1];
  const float off = warp_max(most_p) * (j.sigmoid ? 8e-7f : 5e-6f) + 1e-7f + kSumStep * fabsf(last);
  const bool crowded = pick.id[j.k] >= 0 && !(last - pick.c[j.k] > 2.1f * off);
  if (!__any_sync(0xffffffffu, near)) {
    if (!crowded) return true;
    // each by its own error: of those equal to the last chosen one the lower experts were taken
    const int last_id = pick.id[j.k - 1];
    const float last_v = __shfl_sync(0xffffffffu, va, j.k - 1), last_b = __shfl_sync(0xffffffffu, ba, j.k - 1);
    const float last_e = __shfl_sync(0xffffffffu, ea, j.k - 1);
    const float from = last - 2.1f * off;
    bool other = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (c[i] >= from && !(x[i] == last_v && b[i] == last_b) && (c[i] < last || (c[i] == last && e0 + i > last_id)))
        other |= !(last - c[i] > last_e + error_of(x[i], c[i]));
    if (!__any_sync(0xffffffffu, other)) return true;
  }
  // Some are not: 64 bits for the few that may be chosen.
  const int few = collect(last - 2.1f * off);
  if (few > 32) return false;
  uint64_t own = 0;
  int id = 0;
  double z64 = 0.;
  if (!j.sigmoid) {
#pragma unroll 4
    for (int i = 0; i < VPL; ++i) z64 += x[i] > -a_inf() ? exp((double)x[i] - (double)top) : 0.;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z64 += __shfl_xor_sync(0xffffffffu, z64, o);
  }
  if (lane < few) {
    id = pick.cand_id[lane];
    const double v = (double)r_float(row[id]);
    own = key_of((j.sigmoid ? 1. / (1. + exp(-v)) : exp(v - (double)top) / z64) + (double)__ldg(j.bias + id));
  }
  int place = 0;
  for (int s = 0; s < few; ++s) {
    const uint64_t o = __shfl_sync(0xffffffffu, own, s);
    const int oid = __shfl_sync(0xffffffffu, id, s);
    place += o > own || (o == own && oid < id);
  }
  __syncwarp();
  if (lane < few && place < j.k) pick.id[place] = id;
  __syncwarp();
  return true;
}

// The choice in 64 bits: ids into `pick`.
template <int VPL>
__device__ __noinline__ void choose_exact(const RouteJob &j, const float (&x)[VPL], float top, double *group_mem, Pick &pick) {
  const int lane = threadIdx.x & 31, e0 = lane * VPL;
  const bool by_logit = !j.bias, sums = j.top2 && j.size > 1;
  double z = 0.;
  if (!j.sigmoid) {
#pragma unroll 1
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < j.E) z += exp((double)x[i] - (double)top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  uint64_t key[VPL];
  const bool grouped = j.groups > 1;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0;
    if (e0 + i < j.E) {
      double c = (double)x[i], d = c;
      if (x[i] > -a_inf() && (!by_logit || (grouped && sums))) {
        const double p = j.sigmoid ? 1. / (1. + exp(-(double)x[i])) : exp((double)x[i] - (double)top) / z;
        if (by_logit) d = p;
        else c = d = p + (double)__ldg(j.bias + e0 + i);
      }
      key[i] = key_of(c);
      if (grouped) group_mem[e0 + i] = d;
    }
  }
  __syncwarp();
  if (grouped) {
    const double none = -(double)a_inf();
    int lg = 0;
    while ((2 << lg) * j.groups <= 32) ++lg;
    double w1 = none, w2 = none;
    if ((lane >> lg) < j.groups)
      for (int m = lane & ((1 << lg) - 1); m < j.size; m += 1 << lg) top_two(group_mem[(lane >> lg) * j.size + m], w1, w2);
    for (int o = 0; o < lg; ++o) join_two(w1, w2, 1 << o);
    int rank;
    const uint32_t keep = keep_groups(sums && w2 > none ? w1 + w2 : w1, j.groups, j.kept, lg, &rank);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < j.E && !((keep >> ((e0 + i) / j.size << lg)) & 1u)) key[i] = 0;
  }
  for (int q = 0; q < j.k; ++q) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint64_t m = warp_max(best);
    if (lane == __ffs(__ballot_sync(0xffffffffu, best == m)) - 1) {
      pick.id[q] = e0 + at;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = 0;
    }
  }
  __syncwarp();
}

// CTAs of an SM that registers are left for.
template <int VPL>
constexpr int kRouteCtas = VPL <= 8 ? 6 : VPL <= 16 ? 4 : 2;

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps, kRouteCtas<VPL>) route_kernel(const RouteJob j) {
  __shared__ __align__(16) double group_mem[kRouteWarps][VPL * 32];  // values of the experts, for the groups' worth
  __shared__ Pick picks[kRouteWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * VPL;
  Pick &pick = picks[warp];
  float b[VPL];
  float finite = 0.f;  // stays 0 unless a bias is not finite
  if (j.bias) {
    if (e0 + VPL <= j.E) {
      load_values<VPL>(j.bias + e0, b);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) b[i] = e0 + i < j.E ? __ldg(j.bias + e0 + i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) finite = fmaf(b[i], 0.f, finite);
  }
  const bool bad_bias = __any_sync(0xffffffffu, !(finite == 0.f));
  const bool live = lane < j.k;
#pragma unroll 1
  for (int64_t t = blockIdx.x * kRouteWarps + warp; t < j.n; t += gridDim.x * kRouteWarps) {
    const T *row = static_cast<const T *>(j.logits) + t * j.stride;
    float x[VPL];
    if (e0 + VPL <= j.E) {
      load_values<VPL>(row + e0, x);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = e0 + i < j.E ? r_float(row[e0 + i]) : -a_inf();
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = max_nan(top, x[i]);
    top = warp_max(top);
    int32_t *ids = j.ids + t * j.k + lane;
    float *weights = j.weights + t * j.k + lane;
    if (!(top < a_inf()) || bad_bias) {
      if (lane == 0 && j.status) atomicOr(j.status, MOE_ROUTE_BAD_LOGIT);
      if (live) {
        *ids = lane;
        *weights = a_nan();
      }
      continue;
    }
    if (top == -a_inf()) top = 0.f;  // all closed
    float z = 1.f;
    if (!j.sigmoid && !(j.renorm && !j.bias && j.groups == 1)) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) z += quick_exp(x[i] - top);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    const bool sure = choose_quick<VPL>(j, row, x, b, top, z, reinterpret_cast<float *>(group_mem[warp]), pick);
    __syncwarp();
    if (!sure) choose_exact<VPL>(j, x, top, group_mem[warp], pick);
    // ---- weights: lane q has the choice q
    const int id = live ? pick.id[lane] : 0;
    const float v = live ? r_float(row[id]) : -a_inf();
    __syncwarp();
    float w;
    if (j.renorm) {
      // p over the sum of p, with a common factor taken out that keeps both numbers
      const float m = j.sigmoid ? fminf(v, 0.f) : v, most = warp_max(m);
      w = v > -a_inf() ? expf(m - most) : 0.f;
      if (j.sigmoid) w = v > -a_inf() ? __fdividef(w, 1.f + expf(-fabsf(v))) : 0.f;
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w = sum > 0.f ? __fdividef(w, sum) : 0.f;
    } else if (j.sigmoid) {
      const float e = expf(-fabsf(v));  // (exp(-v) is past fp32 where p is among its smallest numbers)
      w = (v < 0.f ? e : 1.f) / (1.f + e);
    } else {
      w = z > 0.f ? expf(v - top) / z : 0.f;
    }
    if (live) {
      *ids = id;
      *weights = w * j.scale;
    }
  }
}

template <typename T, int VPL>
void run_route(const RouteJob &j, cudaStream_t st) {
  // (CTAs that run at once: of more tokens a warp takes several, and loads the bias once)
  const int grid = std::min((j.n - 1) / kRouteWarps + 1, kRouteSms * kRouteCtas<VPL>);
  route_kernel<T, VPL><<<grid, 32 * kRouteWarps, 0, st>>>(j);
}
template <typename T>
int launch_route(const RouteJob &j, cudaStream_t st) {
  const int v = (j.E + 31) / 32;
  if (v <= 1) run_route<T, 1>(j, st);
  else if (v <= 2) run_route<T, 2>(j, st);
  else if (v <= 4) run_route<T, 4>(j, st);
  else if (v <= 8) run_route<T, 8>(j, st);
  else if (v <= 16) run_route<T, 16>(j, st);
  else run_route<T, 32>(j, st);
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
