// experts_i8.cu -- the experts' products of 8-bit integers.
//
//   product  y[s, n] = (sum_k x[s, k] w[e, n, k]) * (sx[s] * sw[e, n])
//   swiglu   the same for gate and up rows of w, and silu(gate) * up
//
// A block walks over one expert's rows, 32 at a time, for 64 features; sums are
// 32-bit integers.
#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kFeatures = 64, kRows = 32, kWords = 16, kThreads = 256;

template <bool GLU>
__global__ void __launch_bounds__(kThreads) k_expert_i8(ExpertI8Params p) {
  constexpr int kHalves = GLU ? 2 : 1;
  __shared__ int32_t ws[kHalves][kFeatures][kWords + 1], xs[kRows][kWords + 1];
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.y, f0 = blockIdx.x * kFeatures, K = p.in_features, N = p.out_features;
  const int64_t lo = max(p.row_begin[e], 0), hi = min((int64_t)max(p.row_end[e], 0), p.rows);
  const int f = threadIdx.x & 63, part = threadIdx.x >> 6;  // eight rows to a thread
  for (int64_t r0 = lo; r0 < hi; r0 += kRows) {
    int32_t acc[kHalves][8] = {};
    for (int k0 = 0; k0 < K; k0 += kWords * 4) {
      __syncthreads();
      for (int i = threadIdx.x; i < kHalves * kFeatures * kWords; i += kThreads) {
        const int c = i % kWords, row = i / kWords % kFeatures, h = i / kWords / kFeatures;
        int32_t v = 0;
        if (f0 + row < N && k0 + c * 4 < K)
          v = *reinterpret_cast<const int32_t*>(p.w + (((int64_t)e * kHalves + h) * N + f0 + row) * K + k0 + c * 4);
        ws[h][row][c] = v;
      }
      for (int i = threadIdx.x; i < kRows * kWords; i += kThreads) {
        const int c = i % kWords, row = i / kWords;
        int32_t v = 0;
        if (r0 + row < hi && k0 + c * 4 < K)
          v = *reinterpret_cast<const int32_t*>(p.x + (r0 + row) * p.x_stride + k0 + c * 4);
        xs[row][c] = v;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kWords; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int h = 0; h < kHalves; ++h) acc[h][i] = __dp4a(ws[h][f][c], xs[part * 8 + i][c], acc[h][i]);
    }
    if (f0 + f >= N) continue;
    const float* sw = p.w_scales + (int64_t)e * kHalves * N + f0 + f;
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + part * 8 + i;
      if (r >= hi) break;
      const float sx = p.x_scales[r * p.x_scale_stride];
      float v = __int2float_rn(acc[0][i]) * (sx * sw[0]);
      if (GLU) v = swiglu_of(v, __int2float_rn(acc[kHalves - 1][i]) * (sx * sw[N]));
      reinterpret_cast<uint16_t*>(p.out)[r * N + f0 + f] = (uint16_t)pack_bf16x2_rn(v, 0.0f);
    }
  }
}

template <bool GLU>
cudaError_t launch(const ExpertI8Params& p, cudaStream_t s) {
  ExpertI8Params q = p;
  void* args[] = {&q};
  return launch_pdl((const void*)k_expert_i8<GLU>, dim3((unsigned)((p.out_features + kFeatures - 1) / kFeatures), (unsigned)p.num_experts),
                    dim3(kThreads), 0, s, args);
}

}  // namespace

cudaError_t launch_expert_product_i8(const ExpertI8Params& p, cudaStream_t s) { return launch<false>(p, s); }
cudaError_t launch_expert_swiglu_i8(const ExpertI8Params& p, cudaStream_t s) { return launch<true>(p, s); }

}  // namespace moe
