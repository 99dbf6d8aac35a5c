// swiglu.cu -- silu(gate) * up with an e4m3 checkpoint of gate and up, and
// the backward pass from that checkpoint.
#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kGluThreads = 256;

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
  x[0] = bf16_lo(v.x);
  x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y);
  x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z);
  x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w);
  x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]), pack_bf16x2_rn(x[4], x[5]),
                    pack_bf16x2_rn(x[6], x[7]));
}

// Half a warp owns one group of 128 channels of one row: gate and up, 8
// channels a lane.
__global__ void __launch_bounds__(kGluThreads) k_swiglu(GluParams p) {
  pdl_wait();
  pdl_trigger();
  const int64_t rows = p.num_rows ? min((int64_t)max(*p.num_rows, 0), p.rows) : p.rows;
  const int F = p.width, groups = (F + 127) / 128;
  const int64_t units = rows * groups;
  const int li = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * (kGluThreads / 16);
  const int64_t first = (int64_t)blockIdx.x * (kGluThreads / 16) + (threadIdx.x >> 4);
  const int64_t padded = (units + 1) / 2 * 2;  // both halves of a warp run the shuffles
  for (int64_t u = first; u < padded; u += step) {
    const int64_t r = u / groups;
    const int gp = (int)(u % groups), c = gp * 128 + li * 8;
    const bool on = u < units && c < F;
    float g[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (on) {
      unpack8(ld_stream_v4(p.gate_up + (r * 2 * F + c) * 2), g);
      unpack8(ld_stream_v4(p.gate_up + (r * 2 * F + F + c) * 2), v);
    }
    if (on && p.act) {
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = swiglu_of(g[i], v[i]);
      st_v4(p.act + (r * F + c) * 2, pack8(a));
    }
    if (p.ckpt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* x = h ? v : g;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float a = fmaxf(amax, 1e-4f), inv = __fdiv_rn(448.0f, a);
        uint2 q;
        q.x = cvt_e4m3x2(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv)) |
              cvt_e4m3x2(__fmul_rn(x[2], inv), __fmul_rn(x[3], inv)) << 16;
        q.y = cvt_e4m3x2(__fmul_rn(x[4], inv), __fmul_rn(x[5], inv)) |
              cvt_e4m3x2(__fmul_rn(x[6], inv), __fmul_rn(x[7], inv)) << 16;
        if (on) *reinterpret_cast<uint2*>(p.ckpt + r * 2 * F + h * F + c) = q;
        if (u < units && li == 0) p.scales[r * 2 * groups + h * groups + gp] = __fdiv_rn(a, 448.0f);
      }
    }
  }
}

__global__ void __launch_bounds__(kGluThreads) k_swiglu_backward(GluParams p) {
  pdl_wait();
  pdl_trigger();
  const int64_t rows = p.num_rows ? min((int64_t)max(*p.num_rows, 0), p.rows) : p.rows;
  const int F = p.width, groups = (F + 127) / 128, chunks = F / 8;
  for (int64_t u = (int64_t)blockIdx.x * kGluThreads + threadIdx.x; u < rows * chunks;
       u += (int64_t)gridDim.x * kGluThreads) {
    const int64_t r = u / chunks;
    const int c = (int)(u % chunks) * 8;
    const uint2 qg = *reinterpret_cast<const uint2*>(p.ckpt + r * 2 * F + c);
    const uint2 qu = *reinterpret_cast<const uint2*>(p.ckpt + r * 2 * F + F + c);
    const float sg = p.scales[r * 2 * groups + c / 128], su = p.scales[r * 2 * groups + groups + c / 128];
    float d[8], dg[8], du[8], a[8];
    unpack8(ld_stream_v4(p.grad_act + (r * F + c) * 2), d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = e4m3_to_f32((i < 4 ? qg.x : qg.y) >> (8 * (i & 3))) * sg;
      const float v = e4m3_to_f32((i < 4 ? qu.x : qu.y) >> (8 * (i & 3))) * su;
      float sig, rest;
      sigmoid_pair(g, sig, rest);
      dg[i] = d[i] * v * sig * (1.0f + g * rest);
      du[i] = d[i] * g * sig;
      a[i] = g * sig * v;
    }
    st_v4(p.grad_gate_up + (r * 2 * F + c) * 2, pack8(dg));
    st_v4(p.grad_gate_up + (r * 2 * F + F + c) * 2, pack8(du));
    if (p.act) st_v4(p.act + (r * F + c) * 2, pack8(a));
  }
}

unsigned blocks_for(int64_t units, int64_t per_block) {
  int dev = 0, sms = 152;
  current_device(&dev, &sms);
  const int64_t need = (units + per_block - 1) / per_block, most = (int64_t)sms * 8;
  return (unsigned)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_swiglu(const GluParams& p, cudaStream_t s) {
  GluParams q = p;
  void* args[] = {&q};
  return launch_pdl((const void*)k_swiglu, dim3(blocks_for(p.rows * ((p.width + 127) / 128), kGluThreads / 16)),
                    dim3(kGluThreads), 0, s, args);
}

cudaError_t launch_swiglu_backward(const GluParams& p, cudaStream_t s) {
  GluParams q = p;
  void* args[] = {&q};
  return launch_pdl((const void*)k_swiglu_backward, dim3(blocks_for(p.rows * (p.width / 8), kGluThreads)),
                    dim3(kGluThreads), 0, s, args);
}

}  // namespace moe
