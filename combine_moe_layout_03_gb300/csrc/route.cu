// route.cu -- the router: scores, group-limited top-k, weights; and the
// gradient of the logits.
#include <math.h>

#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const RouteParams& p, int64_t t, int e) {
  const int64_t i = t * p.stride + e;
  const float x = p.logits_kind == MOE_LOGITS_BF16
                      ? __uint_as_float((uint32_t)((const uint16_t*)p.logits)[i] << 16)
                      : ((const float*)p.logits)[i];
  // NaN compares false, so it is taken out as -inf is; +inf becomes FLT_MAX
  return x > -INFINITY ? fminf(x, 3.402823466e38f) : -INFINITY;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
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

// The weight of a chosen logit before the scale, and 1 - s where it is a
// sigmoid. top: the row's largest logit; den: the softmax's sum.
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// One warp per token; keys in shared memory, in fp64.
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(RouteParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ double s_keys[];
  const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
  const int E = p.num_experts, G = p.num_groups, per = E / G;
  double* key = s_keys + (size_t)warp * E;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= p.num_tokens) return;
  float top = -INFINITY;
  for (int e = lane; e < E; e += 32) top = fmaxf(top, load_logit(p, t, e));
  top = warp_max(top);
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  double den = 0.0;
  float den32 = 0.0f;
  if (softmax && top > -INFINITY) {
    for (int e = lane; e < E; e += 32) {
      const float x = load_logit(p, t, e);
      den += exp((double)x - (double)top);
      den32 += expf(x - top);
    }
    den = warp_sum(den);
    den32 = warp_sum(den32);
  }
  const bool scored = p.bias || (G > 1 && p.group_score == MOE_GROUP_TOP2_SUM);
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
      else if (!p.bias && scored && key[e] > -INFINITY)
        key[e] = load_logit(p, t, e);
    }
    __syncwarp();
  }
  int mine = -1;  // the id that lane j holds for place j
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
  float w = 0.0f;
  const float x = mine >= 0 ? load_logit(p, t, mine) : -INFINITY;
  if (p.renormalize) {
    // relative to the largest chosen, so that no sum underflows
    float part;
    if (softmax) {
      const float m = warp_max(x);
      part = mine >= 0 ? expf(x - m) : 0.0f;
    } else {
      const float low = fminf(x, 0.0f), m = warp_max(low);
      part = mine >= 0 ? expf(low - m) / (1.0f + expf(-fabsf(x))) : 0.0f;
    }
    const float sum = warp_sum(part);
    if (mine >= 0) w = p.scale * (part / sum);
  } else if (mine >= 0) {
    w = p.scale * (softmax ? expf(x - top) / den32 : sigmoid(x));
  }
  if (lane < p.topk) {
    p.topk_idx[t * p.topk + lane] = mine;
    p.topk_weights[t * p.topk + lane] = w;
  }
}

__device__ __forceinline__ void store_grad(const RouteParams& p, int64_t t, int e, float g) {
  const int64_t i = t * p.num_experts + e;
  if (p.logits_kind == MOE_LOGITS_BF16)
    ((uint16_t*)p.grad_logits)[i] = (uint16_t)(pack_bf16x2_rn(g, 0.0f) & 0xffffu);
  else
    ((float*)p.grad_logits)[i] = g;
}

__global__ void __launch_bounds__(kRouteWarps * 32) k_route_backward(RouteParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
  const int E = p.num_experts;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= p.num_tokens) return;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  int mine = lane < p.topk ? p.topk_idx[t * p.topk + lane] : -1;
  if (mine >= E) mine = -1;
  const float g = mine >= 0 ? p.grad_weights[t * p.topk + lane] : 0.0f;
  const float x = mine >= 0 ? load_logit(p, t, mine) : -INFINITY;
  float d = 0.0f;  // the chosen logit's own gradient
  if (p.renormalize) {
    float part, fall = 1.0f;
    if (softmax) {
      const float m = warp_max(x);
      part = mine >= 0 ? expf(x - m) : 0.0f;
    } else {
      const float low = fminf(x, 0.0f), m = warp_max(low);
      part = mine >= 0 ? expf(low - m) / (1.0f + expf(-fabsf(x))) : 0.0f;
      fall = sigmoid(-x);
    }
    const float sum = warp_sum(part);
    const float v = mine >= 0 ? part / sum : 0.0f;
    const float mean = warp_sum(g * v);
    if (mine >= 0) d = p.scale * v * fall * (g - mean);
  } else if (!softmax) {
    if (mine >= 0) d = p.scale * g * sigmoid(x) * sigmoid(-x);
  }
  if (softmax && !p.renormalize) {
    float top = -INFINITY, den = 0.0f;
    for (int e = lane; e < E; e += 32) top = fmaxf(top, load_logit(p, t, e));
    top = warp_max(top);
    for (int e = lane; e < E; e += 32) {
      const float y = load_logit(p, t, e);
      if (y > -INFINITY) den += expf(y - top);
    }
    den = warp_sum(den);
    const float pm = mine >= 0 ? expf(x - top) / den : 0.0f;
    const float mean = warp_sum(p.scale * g * pm);
    for (int e = lane; e < E; e += 32) {
      const float y = load_logit(p, t, e);
      const float s = y > -INFINITY ? expf(y - top) / den : 0.0f;
      store_grad(p, t, e, -s * mean);
    }
    __syncwarp();
    if (mine >= 0) store_grad(p, t, mine, pm * (p.scale * g - mean));
    return;
  }
  for (int e = lane; e < E; e += 32) store_grad(p, t, e, 0.0f);
  __syncwarp();
  if (mine >= 0) store_grad(p, t, mine, d);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t s) {
  const unsigned blocks = (unsigned)((p.num_tokens + kRouteWarps - 1) / kRouteWarps);
  RouteParams q = p;
  void* args[] = {&q};
  return launch_pdl((const void*)k_route, dim3(blocks), dim3(kRouteWarps * 32),
                    (size_t)kRouteWarps * p.num_experts * sizeof(double), s, args);
}

cudaError_t launch_route_backward(const RouteParams& p, cudaStream_t s) {
  const unsigned blocks = (unsigned)((p.num_tokens + kRouteWarps - 1) / kRouteWarps);
  RouteParams q = p;
  void* args[] = {&q};
  return launch_pdl((const void*)k_route_backward, dim3(blocks), dim3(kRouteWarps * 32), 0, s, args);
}

}  // namespace moe
