// quantize.cu -- rows to 8-bit integers with one scale each.
//
//   a = max(max_k |x[r, k]|, 1e-30), q[r, k] = rint(x[r, k] * (127 / a)), scale[r] = a / 127
//
// Every value is read once: a row stays with the threads that share it while its
// largest magnitude is found, and its codes leave from there. It stays in their
// registers, but for fp32 rows of more than 16384 elements: 1024 threads have 64
// registers each, which eight pieces fill, and 116 bytes of a thread's 256 pass
// through local memory.
// What bounds it: memory (32768 x 2048 bf16 30.4 us, 201 MB at 6.6 TB/s; 32768 x
// 7168 fp32 164 us, 1.17 GB at 7.2 TB/s, more reads than a copy has; 8192 x 16384
// fp32 7.0 TB/s, the wider ones 4.5 to 5.0 for 4096 x 32768 and 2048 x 65536), and
// the launch for a few rows (2.4 us).
#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kQuantThreads = 128;  // of a block, where a row takes no more (32768 x 2048 bf16: 30.4 us, with 256 34.0, with 512 31.1)
constexpr unsigned kAll = 0xffffffffu;

// Eight elements as fp32.
template <bool F32>
struct Eight {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p) {
    a = ld_stream_v4(p);
    if (F32) b = ld_stream_v4(p + 16);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float* x) const {
    if (F32) {
      x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
      x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y), x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
    } else {
      x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
      x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
    }
  }
  // The largest magnitude's bits. As whole numbers infinities are above every
  // number and NaN above them, so neither is lost.
  __device__ __forceinline__ uint32_t largest() const {
    float x[8];
    values(x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
  }
};

// rint(x * inv) as a byte: the sum with 1.5 * 2^23 has it, halves to the even
// one, in its low bits. (x * inv is rounded first, as the rule says.)
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
}
__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  const uint32_t lo = __byte_perm(code_bits(x[0], inv), code_bits(x[1], inv), 0x0040);
  const uint32_t hi = __byte_perm(code_bits(x[2], inv), code_bits(x[3], inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// T threads to a row, each with up to V times eight elements of it.
template <int T, int V, bool F32>
__global__ void __launch_bounds__(T > kQuantThreads ? T : kQuantThreads) k_quantize(QuantParams p) {
  constexpr int kThreads = T > kQuantThreads ? T : kQuantThreads;
  constexpr int kRows = kThreads / T;  // of a block
  __shared__ uint32_t part[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int64_t rows = p.num_rows ? min((int64_t)max(*p.num_rows, 0), p.rows) : p.rows;
  const int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
  const int i = threadIdx.x % T, vecs = p.width / 8;
  const bool on = r < rows;
  constexpr int kBytes = F32 ? 32 : 16;
  const uint8_t* from = p.x + r * p.x_stride * (F32 ? 4 : 2);
  Eight<F32> v[V];
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = j * T + i;
    if (on && at < vecs)
      v[j].load(from + (int64_t)at * kBytes);
    else
      v[j].zero();
  }
#pragma unroll
  for (int j = 0; j < V; ++j) most = max(most, v[j].largest());
  most = __reduce_max_sync(kAll, most);
  if (T > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) most = max(most, part[threadIdx.x / T * (T / 32) + w]);
  }
  if (!on) return;
  const bool fine = most < 0x7f800000u;
  const float a = fmaxf(__uint_as_float(fine ? most : 0), 1e-30f);
  const float inv = fine ? __fdiv_rn(127.0f, a) : 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = j * T + i;
    if (at >= vecs) break;
    float x[8];
    v[j].values(x);
    const uint2 q = fine ? make_uint2(codes4(x, inv), codes4(x + 4, inv)) : make_uint2(0, 0);
    *reinterpret_cast<uint2*>(p.q + r * p.width + (int64_t)at * 8) = q;
  }
  if (i == 0) {
    const float scale = fine ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fffffffu);
    if (p.scale_stride == 4)
      *reinterpret_cast<float4*>(p.scales + r * 4) = make_float4(scale, 0.0f, 0.0f, 0.0f);
    else
      p.scales[r] = scale;
  }
}

template <int T, int V>
cudaError_t launch(const QuantParams& p, cudaStream_t s) {
  constexpr int kThreads = T > kQuantThreads ? T : kQuantThreads;
  constexpr int kRows = kThreads / T;
  QuantParams q = p;
  void* args[] = {&q};
  return launch_pdl(p.x_kind == MOE_ROWS_F32 ? (const void*)k_quantize<T, V, true> : (const void*)k_quantize<T, V, false>,
                    dim3((unsigned)((p.rows + kRows - 1) / kRows)), dim3(kThreads), 0, s, args);
}

}  // namespace

// As few threads to a row as hold it in four or eight pieces of eight elements
// each (2048 wide, in blocks of 256: a warp to a row 34.0 us, two 33.6, four 36.7).
cudaError_t launch_quantize(const QuantParams& p, cudaStream_t s) {
  const int vecs = p.width / 8;
  if (vecs <= 32 * 4) return launch<32, 4>(p, s);
  if (vecs <= 32 * 8) return launch<32, 8>(p, s);
  if (vecs <= 128 * 4) return launch<128, 4>(p, s);
  if (vecs <= 256 * 4) return launch<256, 4>(p, s);
  if (vecs <= 512 * 4) return launch<512, 4>(p, s);
  return launch<1024, 8>(p, s);
}

}  // namespace moe
