// swiglu.cu -- silu(gate) * up with an e4m3 checkpoint of gate and up, and
// the backward pass from that checkpoint.
//
// Both passes read and write every value once and are bound by memory, so a
// thread has the loads of two places under way at a time and the arithmetic is
// kept short: the magnitudes of a group of 128 are compared in pairs of bf16
// (exact), gate's and up's together in one word over the 16 lanes that hold
// the group, and of the four quotients that a group needs (448 / a and a / 448
// of gate and of up, IEEE) four lanes compute one each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kGluThreads = 256;
// Blocks per SM: as many as leave a thread the registers for two places.
// 32768 rows of 2048 with 3, 4, 5 and 6: forward with checkpoint 94, 88, 93 and
// 98 us (541 MB), backward with act 106, 119, 118 and 153 us (675 MB).
constexpr int kForwardBlocks = 4, kBackwardBlocks = 3;
constexpr unsigned kAll = 0xffffffffu;

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

// The larger of two words' bf16 halves, of numbers without their signs; NaN
// gives way to a number.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
// The largest magnitude of eight bf16, in both halves' maximum (low | high).
__device__ __forceinline__ uint32_t largest2(uint4 v) {
  constexpr uint32_t kMagnitude = 0x7fff7fffu;
  return max2(max2(v.x & kMagnitude, v.y & kMagnitude), max2(v.z & kMagnitude, v.w & kMagnitude));
}

__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  return make_uint2(cvt_e4m3x2(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv)) |
                        cvt_e4m3x2(__fmul_rn(x[2], inv), __fmul_rn(x[3], inv)) << 16,
                    cvt_e4m3x2(__fmul_rn(x[4], inv), __fmul_rn(x[5], inv)) |
                        cvt_e4m3x2(__fmul_rn(x[6], inv), __fmul_rn(x[7], inv)) << 16);
}
// Four codes -> their values (exact in f16 and f32) times the scale.
__device__ __forceinline__ void values4(uint32_t codes, float scale, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"((uint16_t)(codes >> (16 * h))));
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&two));
    x[2 * h] = f.x * scale;
    x[2 * h + 1] = f.y * scale;
  }
}

// Where a thread is: row, and eight channels of it (`at` counts them in
// eights, `across` to a row), moving on by a fixed distance without divisions.
struct Place {
  int64_t row;
  int at;
};
struct Stride {
  int64_t rows;
  int ats;
};
__device__ __forceinline__ Place place_of(int64_t u, int across) {
  Place p;
  p.row = u / across;
  p.at = (int)(u - p.row * across);
  return p;
}
__device__ __forceinline__ void move_on(Place& p, Stride s, int across) {
  p.row += s.rows;
  p.at += s.ats;
  if (p.at >= across) {
    p.at -= across;
    ++p.row;
  }
}

// A row is taken as whole groups (16 lanes each), so that a group lies in half
// a warp whatever the width; lanes behind the last channel only help compare.
template <bool ACT, bool CKPT>
__global__ void __launch_bounds__(kGluThreads, kForwardBlocks) k_swiglu(GluParams p, Stride stride) {
  pdl_wait();
  pdl_trigger();
  const int64_t rows = p.num_rows ? min((int64_t)max(*p.num_rows, 0), p.rows) : p.rows;
  const int F = p.width, groups = (F + 127) / 128, across = groups * 16;
  const int li = threadIdx.x & 15;
  Place here = place_of((int64_t)blockIdx.x * kGluThreads + threadIdx.x, across);
  // (the warp goes on while one of its halves has a row)
  while (__any_sync(kAll, here.row < rows)) {
    Place next[2];
    uint4 g[2], u[2];
    bool on[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      next[j] = here;
      on[j] = here.row < rows && here.at * 8 < F;
      g[j] = u[j] = make_uint4(0, 0, 0, 0);
      if (on[j]) {
        const uint8_t* from = p.gate_up + (here.row * 2 * F + here.at * 8) * 2;
        g[j] = ld_stream_v4(from);
        u[j] = ld_stream_v4(from + (int64_t)F * 2);
      }
      move_on(here, stride, across);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t r = next[j].row;
      const int c = next[j].at * 8;
      float gf[8], uf[8];
      unpack8(g[j], gf);
      unpack8(u[j], uf);
      if (ACT && on[j]) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = swiglu_of(gf[i], uf[i]);
        st_v4(p.act + (r * F + c) * 2, pack8(a));
      }
      if (CKPT) {
        const uint32_t lg = largest2(g[j]), lu = largest2(u[j]);
        // gate's largest below, up's above
        uint32_t most = max2(__byte_perm(lg, lu, 0x5410), __byte_perm(lg, lu, 0x7632));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) most = max2(most, __shfl_xor_sync(kAll, most, o));
        const float ag = fmaxf(bf16_lo(most), 1e-4f), au = fmaxf(bf16_hi(most), 1e-4f);
        const float a = li & 1 ? au : ag;
        const float q = __fdiv_rn(li & 2 ? a : 448.0f, li & 2 ? 448.0f : a);
        const float inv_g = __shfl_sync(kAll, q, 0, 16), inv_u = __shfl_sync(kAll, q, 1, 16);
        if (on[j]) {
          uint8_t* to = p.ckpt + r * 2 * F + c;
          *reinterpret_cast<uint2*>(to) = codes8(gf, inv_g);
          *reinterpret_cast<uint2*>(to + F) = codes8(uf, inv_u);
        }
        if (r < rows && (li == 2 || li == 3)) p.scales[r * 2 * groups + (li & 1) * groups + c / 128] = q;
      }
    }
  }
}

template <bool ACT>
__global__ void __launch_bounds__(kGluThreads, kBackwardBlocks) k_swiglu_backward(GluParams p, Stride stride) {
  pdl_wait();
  pdl_trigger();
  const int64_t rows = p.num_rows ? min((int64_t)max(*p.num_rows, 0), p.rows) : p.rows;
  const int F = p.width, groups = (F + 127) / 128, across = F / 8;
  Place here = place_of((int64_t)blockIdx.x * kGluThreads + threadIdx.x, across);
  while (here.row < rows) {
    Place next[2];
    uint2 qg[2], qu[2];
    uint4 da[2];
    float sg[2], su[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      next[j] = here;
      if (here.row < rows) {
        const int c = here.at * 8;
        const uint8_t* from = p.ckpt + here.row * 2 * F + c;
        qg[j] = *reinterpret_cast<const uint2*>(from);
        qu[j] = *reinterpret_cast<const uint2*>(from + F);
        da[j] = ld_stream_v4(p.grad_act + (here.row * F + c) * 2);
        sg[j] = p.scales[here.row * 2 * groups + c / 128];
        su[j] = p.scales[here.row * 2 * groups + groups + c / 128];
      }
      move_on(here, stride, across);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t r = next[j].row;
      if (r >= rows) break;
      const int c = next[j].at * 8;
      float g[8], u[8], d[8], a[8];
      values4(qg[j].x, sg[j], g);
      values4(qg[j].y, sg[j], g + 4);
      values4(qu[j].x, su[j], u);
      values4(qu[j].y, su[j], u + 4);
      unpack8(da[j], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float sig, rest;
        sigmoid_pair(g[i], sig, rest);
        const float silu = g[i] * sig, v = u[i];
        u[i] = d[i] * silu;                                     // gradient of up
        g[i] = d[i] * v * sig * fmaf(g[i], rest, 1.0f);         // gradient of gate
        a[i] = silu * v;
      }
      uint8_t* to = p.grad_gate_up + (r * 2 * F + c) * 2;
      st_v4(to, pack8(g));
      st_v4(to + (int64_t)F * 2, pack8(u));
      if (ACT) st_v4(p.act + (r * F + c) * 2, pack8(a));
    }
  }
}

// Launches fn over `units` eights of channels, `across` to a row.
cudaError_t launch_over(const void* fn, const GluParams& p, int64_t units, int across, int per_sm, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
  const int64_t need = (units + kGluThreads - 1) / kGluThreads, most = (int64_t)sms * per_sm;
  const int64_t blocks = need < most ? need : most, step = blocks * kGluThreads;
  GluParams q = p;
  Stride stride = {step / across, (int)(step % across)};
  void* args[] = {&q, &stride};
  return launch_pdl(fn, dim3((unsigned)blocks), dim3(kGluThreads), 0, s, args);
}

}  // namespace

cudaError_t launch_swiglu(const GluParams& p, cudaStream_t s) {
  const int across = (p.width + 127) / 128 * 16;
  const void* fn = !p.ckpt  ? (const void*)k_swiglu<true, false>
                   : p.act ? (const void*)k_swiglu<true, true>
                           : (const void*)k_swiglu<false, true>;
  return launch_over(fn, p, p.rows * across, across, kForwardBlocks, s);
}

cudaError_t launch_swiglu_backward(const GluParams& p, cudaStream_t s) {
  const int across = p.width / 8;
  return launch_over(p.act ? (const void*)k_swiglu_backward<true> : (const void*)k_swiglu_backward<false>, p,
                     p.rows * across, across, kBackwardBlocks, s);
}

}  // namespace moe
