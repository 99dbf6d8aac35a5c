// route.cu -- the router: scores, group-limited top-k, weights; and the
// gradient of the logits.
//
// One warp per token, its logits in registers: lane l holds experts
// 128 i + 4 l + {0..3}. What bounds it is the number of instructions, not the
// bytes, so the choice works on one integer per expert: the key in 22 bits of
// fixed point above the expert's index (counted down, so that of equal keys
// the lowest index is the largest integer). Each lane sorts its own into
// shared memory; then each of the k places takes one redux over the lanes'
// heads, and the lane that gave it reads its next.
//
// Fixed point covers the keys from the smallest lane maximum up (32 lanes hold
// 32 keys at least that large, and k <= 32), and below it those that lie within
// the keys' errors, which is about as fine as fp32.
// It is monotone, so keys that differ in it are in order; where two keys whose
// order matters do not differ by more than the keys' own errors, the experts
// in question get fp64 keys (settle_groups, settle_order; where they are more
// than 32, order_in_64 does the whole token), so that the choice is always
// that of 64-bit arithmetic. For 256 experts with a bias that happens to about
// one token in five hundred, and costs it two microseconds.
//
// The range is only as fine as it is short. A lane whose largest key is a mask
// of -1e9 (a range of four or eight neighbours taken out), or a bias of 1e9 or
// +inf that forces an expert, leaves the other keys a few steps, and every
// token goes to order_in_64: 16384 tokens, 128 experts, logits masked by -1e9
// 134 us, by -1e4 13 us, by -inf or the type's lowest value 11 us; a forced
// expert 228 us.
#include <limits.h>
#include <math.h>

#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kRouteWarps = 4;
constexpr int kBackwardWarps = 8;  // 16384 tokens: 4.6 us, with four 5.1 us (blocks to start)
constexpr unsigned kAll = 0xffffffffu;
constexpr float kUnit = 5.9604645e-8f;  // 2^-24, half a step of fp32
constexpr float kLargest = 3.402823466e38f;

__device__ __forceinline__ float raw_logit(const RouteParams& p, int64_t t, int e) {
  const int64_t i = t * p.stride + e;
  return p.logits_kind == MOE_LOGITS_BF16 ? __uint_as_float((uint32_t)((const uint16_t*)p.logits)[i] << 16)
                                          : ((const float*)p.logits)[i];
}
// NaN goes the way of -inf (fmaxf takes the number), +inf becomes FLT_MAX, -0 becomes +0.
__device__ __forceinline__ float cleaned(float x) { return fminf(fmaxf(x, -INFINITY), kLargest) + 0.0f; }
__device__ __forceinline__ float load_logit(const RouteParams& p, int64_t t, int e) {
  return cleaned(raw_logit(p, t, e));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The lowest index among the largest values of all lanes' (v, i).
__device__ __forceinline__ void warp_argmax(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(kAll, v, o);
    const int j = __shfl_xor_sync(kAll, i, o);
    if (w > v || (w == v && j < i)) {
      v = w;
      i = j;
    }
  }
}

// Integers that order as the floats do (no NaN, no -0).
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(v);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
constexpr int kNone = (int)0x807fffff;  // ordered(-inf): an expert that is taken out

__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kAll, ordered(v))); }

// exp(x) and 1 / x in one instruction each beside the product with log2 e:
// within 4 units of 2^-24 and the rounding of the argument, and 2 units;
// results below the normal range are 0. (The keys' error bound counts this. In
// the full gradient of a softmax it shows far below the largest logit alone:
// 5e-6 relative at 80 below, 0 from 87.4 below.)
__device__ __forceinline__ float quick_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float quick_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The weights of the chosen before the scale, from their logits y (-inf: none):
// s, or s over its sum. The renormalised ones are taken relative to the
// largest, so that no sum underflows; a lone expert's is 1 exactly. fall:
// 1 - s of a sigmoid. top, den: the row's, for the softmax alone. expf is
// within 2 ulp, __fdividef too. No shuffle stands behind a condition.
template <bool SOFTMAX>
__device__ __forceinline__ float weight_of_chosen(float y, bool on, bool renormalize, float top, float den,
                                                  float& fall) {
  float part;
  if (SOFTMAX) {
    const float most = warp_max(y);
    part = expf(y - (renormalize ? most : top));
  } else {
    const float low = fminf(y, 0.0f), most = warp_max(low), far = expf(-fabsf(y));
    const float r = __fdividef(1.0f, 1.0f + far);
    part = renormalize ? expf(low - most) * r : y >= 0.0f ? r : far * r;
    fall = y >= 0.0f ? far * r : r;
    den = 1.0f;
  }
  part = on ? part : 0.0f;
  const float sum = warp_sum(part);
  den = renormalize ? sum : den;
  const float w = __fdividef(part, den);
  return !on ? 0.0f : part == den ? 1.0f : w;
}

// Shared memory of one warp, in doubles: fp64 keys; or the fp32 keys of the
// groups with their gaps; or two lists of 32; or the lanes' sorted lists.
__host__ __device__ constexpr int room_of(int v, int experts) {
  return experts + 32 > (v + 1) * 16 ? experts + 32 : (v + 1) * 16;
}

// How groups lie over the lanes, from the host.
struct Grouping {
  int per;     // experts a group
  int mul;     // ceil(2^20 / per): e / per for 0 <= e < 1024
  int whole;   // a group is per / 4 neighbouring lanes of one 128 (per a power of two, 4 to 128)
  int shift;   // whole: log2 of the lanes a group has; else log2 of the lanes that share its scan
  __device__ __forceinline__ int of(int e) const { return (e * mul) >> 20; }
};

// The sum that softmax keys are divided by, in fp64. Without a bias nothing is
// added to the scores, and they order the same undivided.
__device__ __noinline__ double sum_in_64(const RouteParams& p, int64_t t, float top) {
  double den = 0.0;
#pragma unroll 4
  for (int e = (int)lane_id(); e < p.num_experts; e += 32) den += exp((double)load_logit(p, t, e) - (double)top);
  return warp_sum(den);
}

// The fp64 key of this lane's expert e (-inf where e < 0); scored: of its
// score, else (without a bias) the logit.
__device__ __noinline__ double key_in_64(const RouteParams& p, int64_t t, int e, float top, bool scored) {
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  const double den = softmax && p.bias ? sum_in_64(p, t, top) : 1.0;
  if (e < 0) return -INFINITY;
  const double x = (double)load_logit(p, t, e);
  if (!scored) return x;
  const double v = softmax ? exp(x - (double)top) / den : 1.0 / (1.0 + exp(-x));
  return p.bias ? v + (double)p.bias[e] : v;
}

// Lane j's id of the choice among the candidates that the lanes hold (at most
// one each, -1: none), in fp64. place: 32 ints of shared memory.
__device__ __noinline__ int settle_order(const RouteParams& p, int64_t t, int e, int total, float top, int* place) {
  const double v = key_in_64(p, t, e, top, p.bias != nullptr);
  int rank = 0;
  for (int j = 0; j < total; ++j) {
    const double w = __shfl_sync(kAll, v, j);
    const int f = __shfl_sync(kAll, e, j);
    rank += w > v || (w == v && f < e);
  }
  const int lane = (int)lane_id();
  __syncwarp();
  if (e >= 0) place[rank] = e;
  __syncwarp();
  return lane < min(p.topk, total) ? place[lane] : -1;
}

// Adds `want` of the groups in question to keep, by their counts in fp64; the
// lanes hold the experts that can be among the two best of those groups.
__device__ __noinline__ unsigned settle_groups(const RouteParams& p, int64_t t, int e, int group, unsigned question,
                                               int want, unsigned keep, float top) {
  const double v = key_in_64(p, t, e, top, true);
  const int lane = (int)lane_id();
  double count = -INFINITY;  // of group `lane`
  for (unsigned left = question; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    double a = e >= 0 && group == g ? v : -INFINITY;
    const double mine = a;
    int i = lane;
    warp_argmax(a, i);
    double b = lane == i ? -INFINITY : mine;
    i = lane;
    warp_argmax(b, i);
    if (lane == g) count = p.group_score == MOE_GROUP_TOP2_SUM && b > -INFINITY ? a + b : a;
  }
  for (int r = 0; r < want; ++r) {
    double v2 = (keep >> lane) & 1u ? -INFINITY : count;
    int i = (question >> lane) & 1u && !((keep >> lane) & 1u) ? lane : 64 + lane;
    warp_argmax(v2, i);
    if (i < 32) keep |= 1u << i;
  }
  return keep;
}

// This lane's one of the experts whose bits are set in the lanes' masks (bit
// 4 i + j: expert 128 i + 4 lane + j), -1 past their number. list: 32 ints.
__device__ __forceinline__ int share_out(unsigned mask, int* list, int& total) {
  const int lane = (int)lane_id(), n = __popc(mask);
  const int upto = warp_inclusive_scan(n);
  total = __shfl_sync(kAll, upto, 31);
  if (total > 32) return -1;
  __syncwarp();
  for (int at = upto - n; mask; mask &= mask - 1, ++at) {
    const int i = __ffs(mask) - 1;
    list[at] = (i / 4) * 128 + lane * 4 + i % 4;
  }
  __syncwarp();
  const int e = lane < total ? list[lane] : -1;
  __syncwarp();
  return e;
}

// The choice of token t in fp64, keys in shared memory; returns lane j's id.
__device__ __noinline__ int order_in_64(const RouteParams& p, int64_t t, double* key, float top) {
  const int lane = (int)lane_id();
  const int E = p.num_experts, G = p.num_groups, per = E / G;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  const bool scored = p.bias || (G > 1 && p.group_score == MOE_GROUP_TOP2_SUM);
  const double den = softmax && scored ? sum_in_64(p, t, top) : 1.0;
  for (int e = lane; e < E; e += 32) {
    const float x = load_logit(p, t, e);
    double v = -INFINITY;
    if (x > -INFINITY) {
      v = x;
      if (scored) v = softmax ? exp((double)x - (double)top) / den : 1.0 / (1.0 + exp(-(double)x));
      if (p.bias) v += (double)p.bias[e];
      if (!(v > -INFINITY)) v = -INFINITY;
    }
    key[e] = v;
  }
  __syncwarp();
  if (G > 1) {
    double count = -INFINITY;
    if (lane < G) {
      double a = -INFINITY, b = -INFINITY;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const double v = key[e];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      count = a;
      if (p.group_score == MOE_GROUP_TOP2_SUM && b > -INFINITY) count = a + b;
    }
    unsigned keep = 0;
    for (int r = 0; r < p.topk_groups; ++r) {
      double v = (keep >> lane) & 1u ? -INFINITY : count;
      int i = lane < G && !((keep >> lane) & 1u) ? lane : 64 + lane;
      warp_argmax(v, i);
      if (i < 32) keep |= 1u << i;
    }
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
      if (!((keep >> (e / per)) & 1u))
        key[e] = -INFINITY;
      else if (!p.bias && key[e] > -INFINITY)
        key[e] = load_logit(p, t, e);
    }
    __syncwarp();
  }
  int mine = -1;
  for (int j = 0; j < p.topk; ++j) {
    double v = -INFINITY;
    int i = E;
    for (int e = lane; e < E; e += 32)
      if (key[e] > v) {
        v = key[e];
        i = e;
      }
    warp_argmax(v, i);
    if (!(v > -INFINITY)) break;
    if (lane == j) mine = i;
    __syncwarp();
    if (lane == 0) key[i] = -INFINITY;
    __syncwarp();
  }
  return mine;
}

// A row's values v[4 i + j] of experts 128 i + 4 lane + j, as they stand (-inf
// behind the last). VEC: rows are aligned to four elements and E is a multiple
// of four.
template <int V, bool VEC>
__device__ __forceinline__ void load_row(const RouteParams& p, int64_t t, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int e = i * 128 + (int)lane_id() * 4;
    float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (VEC) {
      if (e < p.num_experts) {
        if (p.logits_kind == MOE_LOGITS_BF16) {
          const uint2 w = *reinterpret_cast<const uint2*>((const uint16_t*)p.logits + t * p.stride + e);
          q[0] = bf16_lo(w.x);
          q[1] = bf16_hi(w.x);
          q[2] = bf16_lo(w.y);
          q[3] = bf16_hi(w.y);
        } else {
          const float4 w = *reinterpret_cast<const float4*>((const float*)p.logits + t * p.stride + e);
          q[0] = w.x;
          q[1] = w.y;
          q[2] = w.z;
          q[3] = w.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < p.num_experts) q[j] = raw_logit(p, t, e + j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = q[j];
  }
}

// v in descending order.
template <int V>
__device__ __forceinline__ void sort_down(unsigned (&v)[V]) {
#pragma unroll
  for (int size = 2; size <= V; size *= 2)
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = i ^ stride;
        if (j > i) {
          const unsigned hi = max(v[i], v[j]), lo = min(v[i], v[j]);
          v[i] = i & size ? lo : hi;
          v[j] = i & size ? hi : lo;
        }
      }
}

// Keys in [lo, lo + range] as 1 .. 2^22 - 1, monotone; smaller keys, and those
// of experts that are taken out (-inf, NaN), are 0.
struct FixedPoint {
  float lo, hi, per_range, margin;
  __device__ __forceinline__ unsigned bits(float key) const {
    // the saturating sum ends at 0 and 1 and takes NaN to 0; 2^23 puts the
    // steps into the low bits
    const float u = __saturatef(fmaf(key - lo, per_range, 2.384185791015625e-7f));
    return __float_as_uint(fmaf(u, 4194303.0f, 8388608.0f));
  }
  __device__ __forceinline__ unsigned of(float key) const { return bits(key) & 0x3fffffu; }
  // Above the index, counted down.
  __device__ __forceinline__ unsigned packed(float key, int e) const { return (bits(key) << 10) + (unsigned)(1023 - e); }
};

constexpr float kOrdinary = 1e30f;  // larger magnitudes (masks of the type's lowest value) share the ends of the range

// exact: keys are what they stand for; else err is how far one may be off beside
// its own rounding.
template <int V>
__device__ __forceinline__ FixedPoint range_of(const float (&key)[V], bool exact, float err) {
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) most = fmaxf(most, key[i]);
  FixedPoint f;
  f.hi = fminf(warp_max(most), kOrdinary);
  float least = most;
  if (__any_sync(kAll, most < -kOrdinary)) {
    // not every lane has a key: the smallest of all
    least = f.hi;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] >= -kOrdinary) least = fminf(least, key[i]);
  }
  f.lo = fminf(unordered(__reduce_min_sync(kAll, ordered(least))), f.hi);
  // Two keys whose order is open are at most margin apart. One that could
  // belong before the smallest lane maximum has to be in the range too: where
  // the k = 32 places are the lanes' maxima, only then does it show behind the
  // last. (Twice, for the difference's own rounding.)
  f.margin = exact ? 0.0f : 2.0f * (err + kUnit * fmaxf(fabsf(f.lo), fabsf(f.hi)));
  f.lo -= 2.0f * f.margin;
  // (Without a range keys from lo up are one step; not times 0, which would
  // lose those that are infinite.)
  f.per_range = f.hi > f.lo ? __fdividef(0.999999f, f.hi - f.lo) : 1e-37f;
  return f;
}

// V: registers a lane spends on its experts (E <= 32 V). SCORED: keys are
// computed (bias, or sums of scores by group), else they are the logits.
template <int V, bool VEC, bool SCORED, bool SOFTMAX>
__global__ void __launch_bounds__(kRouteWarps * 32, V <= 8 ? 8 : V <= 16 ? 6 : 4)
    k_route(RouteParams p, Grouping groups) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ double s_keys[];
  const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
  const int E = p.num_experts, G = p.num_groups;
  // no warp leaves early: the shuffles below want all lanes, and a warp behind
  // the last token does that token again and stores nothing
  const int64_t at = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const int64_t t = min(at, (int64_t)p.num_tokens - 1);
  double* room = s_keys + (size_t)warp * room_of(V, E);

  float x[V];
  load_row<V, VEC>(p, t, x);
  float top = 0.0f, den = 0.0f;
  if (SOFTMAX) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = cleaned(x[i]);
      top = fmaxf(top, x[i]);
    }
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < V; ++i) den += x[i] > -INFINITY ? quick_exp(x[i] - top) : 0.0f;
    den = warp_sum(den);
  }

  float key[V];
  float err = 0.0f;   // how far an fp32 score may be off; a key adds its own rounding
  bool open = false;  // more experts in question than lanes: the whole token in fp64
  if (SCORED) {
    const float inv = SOFTMAX ? __fdividef(1.0f, den) : 0.0f;
    // In units of 2^-24. sigmoid: s (1 - s) <= 1/4 of the exponential's 4 and
    // of its argument's |x| (x s (1 - s) < 1/4), the sum 1, the inverse 2, and
    // room for 3 more. softmax: the exponential 4 here and 4 in the sum, the
    // sum's V + 5 roundings, quotient and product 6, the arguments' two
    // roundings 16 (|x - top| exp(x - top) < 0.4 here, and its mean under the
    // distribution <= ln E < 7 in the sum), and room for 1 more.
    err = SOFTMAX ? (V + 36) * kUnit * inv : 8 * kUnit;
    float add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) add[i] = 0.0f;
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int e = i * 32 + lane * 4;
        if (VEC) {
          if (e < E) *reinterpret_cast<float4*>(add + i) = *reinterpret_cast<const float4*>(p.bias + e);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (e + j < E) add[i + j] = p.bias[e + j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = SOFTMAX ? quick_exp(x[i] - top) * inv : quick_inverse(1.0f + quick_exp(-x[i]));
      // a bias of NaN or -inf takes the expert out, as the logit does
      key[i] = x[i] > -INFINITY ? fmaxf(v + add[i], -INFINITY) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = x[i];
  }

  if (G > 1) {
    // Every group's two largest keys, and from them its count: in lane g, or
    // in the first of the lanes that scanned it.
    const bool two = p.group_score == MOE_GROUP_TOP2_SUM;
    float a = -INFINITY, b = -INFINITY;
    const int lanes_log = groups.whole ? 0 : groups.shift;
    if (VEC && groups.whole) {
      const int span = 1 << groups.shift, blocks = 32 >> groups.shift;  // lanes a group, groups in 128 experts
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        float c = fmaxf(key[4 * i], key[4 * i + 1]), d = fminf(key[4 * i], key[4 * i + 1]);
        const float f = fmaxf(key[4 * i + 2], key[4 * i + 3]), h = fminf(key[4 * i + 2], key[4 * i + 3]);
        d = fmaxf(fmaxf(d, h), fminf(c, f));
        c = fmaxf(c, f);
        for (int o = 1; o < span; o <<= 1) {
          const float u = __shfl_xor_sync(kAll, c, o), w = __shfl_xor_sync(kAll, d, o);
          d = fmaxf(fmaxf(d, w), fminf(c, u));
          c = fmaxf(c, u);
        }
        const int from = lane - i * blocks;  // lane g takes group g
        const float u = __shfl_sync(kAll, c, (from << groups.shift) & 31);
        const float w = __shfl_sync(kAll, d, (from << groups.shift) & 31);
        const bool here = (unsigned)from < (unsigned)blocks;
        a = here ? u : a;
        b = here ? w : b;
      }
    } else {
      // keys cross over in shared memory, four words apart every 32 so that
      // groups of 32 start in different banks
      float* buf = reinterpret_cast<float*>(room);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = (i / 4) * 128 + lane * 4 + i % 4;
        if (e < E) buf[e + (e >> 5) * 4] = key[i];
      }
      __syncwarp();
      const int g = lane >> lanes_log, lanes = 1 << lanes_log;
      if (g < G)
        for (int q = lane & (lanes - 1); q < groups.per; q += lanes) {
          const int e = g * groups.per + q;
          const float v = buf[e + (e >> 5) * 4];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
      __syncwarp();
      for (int o = lanes / 2; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(kAll, a, o), d = __shfl_xor_sync(kAll, b, o);
        b = fmaxf(fmaxf(b, d), fminf(a, c));
        a = fmaxf(a, c);
      }
    }
    const int g = lane >> lanes_log;
    const bool head = g << lanes_log == lane && g < G;
    // Counts and their size stay finite where a key is infinite (a bias that
    // forces an expert) or two of them overflow, so that the differences below
    // have a value: such counts are equal here, and fp64 tells them apart.
    float count = a, size = head && a > -INFINITY ? fabsf(a) : 0.0f;
    if (two && b > -INFINITY) {
      count += b;
      size += fabsf(b);
    }
    if (a > -INFINITY) count = fminf(fmaxf(count, -kLargest), kLargest);
    size = fminf(size, kLargest);
    const int mark = head ? ordered(count + 0.0f) : INT_MIN;
    int left = mark, m = kNone;
    unsigned keep = 0;
    for (int r = 0; r < p.topk_groups; ++r) {
      m = __reduce_max_sync(kAll, left);
      const int from = __ffs(__ballot_sync(kAll, left == m)) - 1;
      keep |= 1u << (from >> lanes_log);
      left = lane == from ? INT_MIN : left;
    }
    if (SCORED && p.topk_groups < G) {
      const int next = __reduce_max_sync(kAll, left);
      size = warp_max(size);
      // the keys' errors and roundings on both sides, and the sums' own
      const float last = unordered(m), lim = (two ? 4.0f : 2.0f) * err + 4.0f * kUnit * size;
      if (next > kNone && last - unordered(next) <= lim) {
        // the counts are off by at most lim / 2 each: what lies within lim of
        // the last one in is in question, what lies above stays
        const bool some = head && mark > kNone;
        const unsigned asked = __ballot_sync(kAll, some && count - last <= lim && last - count <= lim);
        const unsigned sure = __ballot_sync(kAll, some && count - last > lim);
        unsigned question = 0, stay = 0;
        for (int q = 0; q < G; ++q) {
          question |= ((asked >> (q << lanes_log)) & 1u) << q;
          stay |= ((sure >> (q << lanes_log)) & 1u) << q;
        }
        // each group's smallest key that may be among its two best
        float* least = reinterpret_cast<float*>(room);
        if (some) least[g] = (two && b > -INFINITY ? b : a) - (2.0f * err + 4.0f * kUnit * size);
        __syncwarp();
        unsigned mask = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int gi = groups.of((i / 4) * 128 + lane * 4 + i % 4) & 31;
          if (key[i] > -INFINITY && ((question >> gi) & 1u) && key[i] >= least[gi]) mask |= 1u << i;
        }
        int total;
        const int e = share_out(mask, reinterpret_cast<int*>(room) + 32, total);
        if (total <= 32)
          keep = settle_groups(p, t, e, e >= 0 ? groups.of(e) : -1, question, p.topk_groups - __popc(stay), stay, top);
        else
          open = true;
      }
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int e = (i / 4) * 128 + lane * 4;
      bool in = (keep >> (groups.of(e) & 31)) & 1u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j && !(VEC && groups.whole)) in = (keep >> (groups.of(e + j) & 31)) & 1u;
        // without a bias the logits order the experts inside the groups
        key[i + j] = in ? (SCORED && !p.bias ? x[i + j] : key[i + j]) : -INFINITY;
      }
    }
  }

  const bool exact = !(SCORED && p.bias);  // without a bias the keys are logits by now
  const FixedPoint fixed = range_of<V>(key, exact, err);
  unsigned head;       // the largest of this lane's list
  unsigned own = 0;    // what place `lane` got
  {
    unsigned list[V];
#pragma unroll
    for (int i = 0; i < V; ++i) list[i] = fixed.packed(key[i], (i / 4) * 128 + lane * 4 + i % 4);
    sort_down<V>(list);
    unsigned* mem = reinterpret_cast<unsigned*>(room) + lane;
#pragma unroll
    for (int i = 1; i < V; ++i) mem[i * 32] = list[i];
    mem[V * 32] = 0;
    head = list[0];
    __syncwarp();
    for (int j = 0; j < p.topk; ++j) {
      const unsigned m = __reduce_max_sync(kAll, head);
      if (m < 1024) break;
      own = lane == j ? m : own;
      if (head == m) {
        mem += 32;
        head = *mem;
      }
    }
    __syncwarp();
  }
  if (__popc(__ballot_sync(kAll, own != 0)) < p.topk) {
    // places left: does anything below the range remain?
    int have = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) have += key[i] > -INFINITY;
    have = __reduce_add_sync(kAll, have);
    if (have > __popc(__ballot_sync(kAll, own != 0))) open = true;
  }
  int mine = own ? 1023 - (int)(own & 1023u) : -1;
  {
    // An order is open where a place and the next (behind the last place: the
    // largest that is left) lie within the keys' error of one another: none
    // for logits, which only have to differ. Equal logits with equal biases
    // are equal in any arithmetic; but behind the last place such a one may
    // stand before others that are larger in 64 bits.
    unsigned slack = 0;
    if (!exact) slack = (unsigned)fminf(fixed.margin * fixed.per_range * 4194304.0f, 4e6f) + 3u;
    const unsigned after = __shfl_down_sync(kAll, own, 1), next = __reduce_max_sync(kAll, head);
    const unsigned below = lane == p.topk - 1 ? next : after;
    bool near = own && below >= 1024 && (own >> 10) - (below >> 10) <= slack;
    if (__any_sync(kAll, near)) {
      const int other = 1023 - (int)(below & 1023u);
      const bool same = near && load_logit(p, t, mine) == load_logit(p, t, other) &&
                        (!p.bias || p.bias[mine] == p.bias[other]);
      near = near && !same;
      const bool tied = __any_sync(kAll, same && lane == p.topk - 1);
      if ((tied || __any_sync(kAll, near)) && !open) {
        // the experts in question, and of those that are not chosen the ones
        // that may differ from the last (exact keys are the logits)
        const unsigned end = __reduce_min_sync(kAll, own ? own : 0xffffffffu);
        const int e_end = 1023 - (int)(end & 1023u);
        const float x_end = load_logit(p, t, e_end);
        unsigned mask = 0, left = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const unsigned v = fixed.packed(key[i], (i / 4) * 128 + lane * 4 + i % 4);
          if (key[i] > -INFINITY && (v >> 10) + slack >= end >> 10) {
            mask |= 1u << i;
            if (v < end && !(exact && key[i] == x_end)) left |= 1u << i;
          }
        }
        if (tied)
          for (; left && !near; left &= left - 1) {
            const int i = __ffs(left) - 1, e = (i / 4) * 128 + lane * 4 + i % 4;
            near = load_logit(p, t, e) != x_end || (p.bias && p.bias[e] != p.bias[e_end]);
          }
        if (__any_sync(kAll, near)) {
          int total;
          int* seats = reinterpret_cast<int*>(room);
          const int e = share_out(mask, seats, total);
          if (total <= 32)
            mine = settle_order(p, t, e, total, top, seats);
          else
            open = true;
        }
      }
    }
    if (open) mine = order_in_64(p, t, room, top);
  }

  const bool on = mine >= 0;
  const float y = on ? load_logit(p, t, mine) : -INFINITY;
  float fall;
  const float w = p.scale * weight_of_chosen<SOFTMAX>(y, on, p.renormalize, top, den, fall);
  if (lane < p.topk && at == t) {
    p.topk_idx[t * p.topk + lane] = mine;
    p.topk_weights[t * p.topk + lane] = w;
  }
}

// The gradient of one row: d of each chosen logit, in shared memory by
// expert, then the whole row in one pass of vector stores. FULL (softmax
// without renormalisation): every logit has a gradient.
template <int V, bool VEC, bool SOFTMAX, bool FULL>
__global__ void __launch_bounds__(kBackwardWarps * 32) k_route_backward(RouteParams p, float inv_scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_row[kBackwardWarps][V * 32];
  const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
  const int E = p.num_experts;
  // as above, no warp leaves early
  const int64_t place = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const int64_t t = min(place, (int64_t)p.num_tokens - 1);
  float* row = s_row[warp];
  int mine = lane < p.topk ? p.topk_idx[t * p.topk + lane] : -1;
  const float gw = lane < p.topk ? p.grad_weights[t * p.topk + lane] : 0.0f;
  float x[V];
  if (FULL) load_row<V, VEC>(p, t, x);
#pragma unroll
  for (int i = 0; i < V / 4; ++i) *reinterpret_cast<float4*>(row + i * 128 + lane * 4) = make_float4(0, 0, 0, 0);
  if (mine >= E) mine = -1;
  const bool on = mine >= 0;
  const float y = on ? load_logit(p, t, mine) : -INFINITY;
  const float g = on ? gw : 0.0f;
  float d = 0.0f, top = -INFINITY, den = 0.0f, mean = 0.0f;
  if (FULL) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = cleaned(x[i]);
      top = fmaxf(top, x[i]);
    }
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = x[i] > -INFINITY ? quick_exp(x[i] - top) : 0.0f;
      den += x[i];
    }
    den = warp_sum(den);
  }
  float fall = 1.0f;
  const float w = p.scale * weight_of_chosen<SOFTMAX>(y, on, !FULL && p.renormalize, top, den, fall);
  if (FULL) {
    d = p.scale * g;
    mean = warp_sum(g * w);
  } else {
    mean = __fmul_rn(warp_sum(__fmul_rn(g, w)), inv_scale);
    d = w * fall * (p.renormalize ? g - mean : g);
  }
  __syncwarp();
  if (on) row[mine] = d;
  __syncwarp();
  if (place != t) return;
  const bool bf16 = p.logits_kind == MOE_LOGITS_BF16;
  const float inv = FULL && den > 0.0f ? __fdividef(1.0f, den) : 0.0f;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int e = i * 128 + lane * 4;
    float4 r = *reinterpret_cast<const float4*>(row + e);
    if (FULL) {
      r.x = x[4 * i] * inv * (r.x - mean);
      r.y = x[4 * i + 1] * inv * (r.y - mean);
      r.z = x[4 * i + 2] * inv * (r.z - mean);
      r.w = x[4 * i + 3] * inv * (r.w - mean);
    }
    const int64_t at = t * E + e;
    if (VEC) {
      if (e >= E) continue;
      if (bf16)
        *reinterpret_cast<uint2*>((uint16_t*)p.grad_logits + at) =
            make_uint2(pack_bf16x2_rn(r.x, r.y), pack_bf16x2_rn(r.z, r.w));
      else
        *reinterpret_cast<float4*>((float*)p.grad_logits + at) = r;
    } else {
      const float v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e + j >= E) continue;
        if (bf16)
          ((uint16_t*)p.grad_logits)[at + j] = (uint16_t)(pack_bf16x2_rn(v[j], 0.0f) & 0xffffu);
        else
          ((float*)p.grad_logits)[at + j] = v[j];
      }
    }
  }
}

}  // namespace

namespace {

template <int V, bool VEC>
const void* route_kernel(bool scored, bool softmax) {
  return scored ? (softmax ? (const void*)k_route<V, VEC, true, true> : (const void*)k_route<V, VEC, true, false>)
                : (softmax ? (const void*)k_route<V, VEC, false, true> : (const void*)k_route<V, VEC, false, false>);
}
template <int V>
const void* route_kernel(bool vec, bool scored, bool softmax) {
  return vec ? route_kernel<V, true>(scored, softmax) : route_kernel<V, false>(scored, softmax);
}

// Rows that four elements at a time can be read from (or written to).
bool rows_in_fours(const RouteParams& p, const void* base, int64_t stride) {
  const uintptr_t four = p.logits_kind == MOE_LOGITS_BF16 ? 8 : 16;
  return p.num_experts % 4 == 0 && stride % 4 == 0 && (uintptr_t)base % four == 0;
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t s) {
  const bool vec = rows_in_fours(p, p.logits, p.stride) && (uintptr_t)p.bias % 16 == 0;
  const bool scored = p.bias || (p.num_groups > 1 && p.group_score == MOE_GROUP_TOP2_SUM);
  const int E = p.num_experts;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  const void* fn = E <= 128   ? route_kernel<4>(vec, scored, softmax)
                   : E <= 256 ? route_kernel<8>(vec, scored, softmax)
                   : E <= 512 ? route_kernel<16>(vec, scored, softmax)
                              : route_kernel<32>(vec, scored, softmax);
  const int warps = p.num_tokens > 1024 ? kRouteWarps : 1;
  const unsigned blocks = (unsigned)((p.num_tokens + warps - 1) / warps);
  const size_t room = (size_t)room_of(E <= 128 ? 4 : E <= 256 ? 8 : E <= 512 ? 16 : 32, E) * sizeof(double);
  RouteParams q = p;
  const int G = p.num_groups, per = E / G;
  Grouping groups = {per, ((1 << 20) + per - 1) / per, vec && per >= 4 && per <= 128 && (per & (per - 1)) == 0, 0};
  if (groups.whole)
    while (4 << groups.shift < per) ++groups.shift;
  else  // 32 / G' lanes, G' the next power of two
    while (G << (groups.shift + 1) <= 32) ++groups.shift;
  void* args[] = {&q, &groups};
  return launch_pdl(fn, dim3(blocks), dim3(warps * 32), warps * room, s, args);
}

namespace {

template <int V, bool VEC>
const void* backward_kernel(bool softmax, bool full) {
  return full      ? (const void*)k_route_backward<V, VEC, true, true>
         : softmax ? (const void*)k_route_backward<V, VEC, true, false>
                   : (const void*)k_route_backward<V, VEC, false, false>;
}
template <int V>
const void* backward_kernel(bool vec, bool softmax, bool full) {
  return vec ? backward_kernel<V, true>(softmax, full) : backward_kernel<V, false>(softmax, full);
}

}  // namespace

cudaError_t launch_route_backward(const RouteParams& p, cudaStream_t s) {
  const bool vec = rows_in_fours(p, p.logits, p.stride) && rows_in_fours(p, p.grad_logits, p.num_experts);
  const bool softmax = p.score == MOE_SCORE_SOFTMAX, full = softmax && !p.renormalize;
  const int E = p.num_experts;
  const void* fn = E <= 128   ? backward_kernel<4>(vec, softmax, full)
                   : E <= 256 ? backward_kernel<8>(vec, softmax, full)
                   : E <= 512 ? backward_kernel<16>(vec, softmax, full)
                              : backward_kernel<32>(vec, softmax, full);
  const int warps = p.num_tokens > 1024 ? kBackwardWarps : 1;
  const unsigned blocks = (unsigned)((p.num_tokens + warps - 1) / warps);
  RouteParams q = p;
  float inv_scale = p.scale != 0.0f ? 1.0f / p.scale : 0.0f;
  void* args[] = {&q, &inv_scale};
  return launch_pdl(fn, dim3(blocks), dim3(warps * 32), 0, s, args);
}

}  // namespace moe
