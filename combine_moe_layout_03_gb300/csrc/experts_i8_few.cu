// experts_i8_few.cu -- the experts' products of 8-bit integers for a few rows.
//
// With at most kFewRows rows in the buffers (a token's or a few tokens') the
// weights' bytes are all the work, and tiles of 256 features of a pair of blocks
// are too coarse to keep every SM busy to the end. Here a unit of work is four
// rows of w (of gate and up two each), and a warp's: it reads 512 bytes of each
// at a time, straight into registers, multiplies them four at a time (dp4a,
// 32-bit sums) with the expert's rows, which stay in L1, and adds up over its
// lanes at the end. The next piece of w is under way before the last one is
// multiplied, across units. Where there are fewer units than warps, 2 or 4 warps
// share one and add up in shared memory (one row of one expert, 7168 -> 2 x 2048:
// 12.4 us by one warp each, 7.4 by four).
//
// What bounds it: memory. One token's first product (8 experts, 7168 -> 2 x 2048,
// 235 MB) takes 36.5 to 37.5 us (6.3 to 6.4 TB/s), its second (2048 -> 7168, 117 MB)
// 18.6 to 19.4. Four blocks an SM, a piece of four rows each way: three or two
// blocks 42 and 46 us, with a second piece under way 44 to 52 (registers: four
// blocks leave a thread 64, and 40 bytes of it are in local memory as it is). Whole 512 bytes of a row
// count: 64 bytes of eight rows at a time, as a matrix product's fragment wants
// them, came to 47 us, and the integer matrix instruction on them to 45 (it is
// slow on this chip, 60% busy with one row of eight in use).
#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kBlocks = 4;  // blocks of an SM
constexpr int kPiece = 512;                                         // bytes of a row that a warp reads at a time
constexpr int kUnit = 4;                                            // rows of w
constexpr int kRows = 2;                                            // rows multiplied at a time; w is read again for more

struct Piece {
  uint4 w[kUnit];
};

__device__ __forceinline__ int32_t dot16(uint4 a, uint4 b, int32_t c) {
  c = __dp4a((int)a.x, (int)b.x, c);
  c = __dp4a((int)a.y, (int)b.y, c);
  c = __dp4a((int)a.z, (int)b.z, c);
  return __dp4a((int)a.w, (int)b.w, c);
}

constexpr int features_of(bool glu) { return glu ? kUnit / 2 : kUnit; }  // of a unit

struct Shared {
  int32_t busy[kFewRows][3];  // experts with rows: index, first row, rows
  int32_t num_busy;
  int32_t part[kWarps][kRows][kUnit];
};

// S: warps to a unit.
template <bool GLU, int S>
__device__ __forceinline__ void work_on(const ExpertI8Params& p, Shared& sm, int warp, int lane) {
  const int32_t(&busy)[kFewRows][3] = sm.busy;
  int32_t(&part)[kWarps][kRows][kUnit] = sm.part;
  const int K = p.in_features, N = p.out_features;
  constexpr int kFeatures = features_of(GLU);
  const int groups = N / kFeatures;                   // units of an expert
  const int units = sm.num_busy * groups, step = gridDim.x * (kWarps / S);
  const int first = warp / S * gridDim.x + blockIdx.x;  // this warp's first unit: the last ones are spread over the SMs
  const int own = warp % S;                             // its pieces: own, own + S, ...
  const int end = (K + kPiece - 1) / kPiece * kPiece, begin = own * kPiece + lane * 16;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  // The stream of pieces that this warp reads: a unit's, once for each kRows
  // rows, then those of its next unit.
  int ahead_u = begin < end ? first : units, ahead_k = begin, ahead_r = 0;
  const int8_t* w = nullptr;
  auto fetch = [&](Piece& v) {
    if (ahead_u >= units) return;
    if (ahead_k == begin) {
      const int b = ahead_u / groups;
      w = p.w + ((int64_t)busy[b][0] * (GLU ? 2 : 1) * N + (int64_t)(ahead_u - b * groups) * kFeatures) * K;
    }
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const int64_t row = GLU ? (int64_t)(i / 2) * N + i % 2 : i;  // gate, gate, up, up
      v.w[i] = ahead_k < K ? ld_stream_v4(w + row * K + ahead_k) : zero;
    }
    ahead_k += S * kPiece;
    if (ahead_k < end) return;
    ahead_k = begin;
    ahead_r += kRows;
    if (ahead_r < busy[ahead_u / groups][2]) return;
    ahead_r = 0;
    ahead_u += step;
  };
  Piece next;
  fetch(next);
  for (int u = first; u < units; u += step) {
    const int b = u / groups, f = (u - b * groups) * kFeatures;
    for (int r0 = 0; r0 < busy[b][2]; r0 += kRows) {
      const int rows = min(busy[b][2] - r0, kRows);
      const int64_t row0 = (int64_t)busy[b][1] + r0;
      const int8_t* x = p.x + row0 * p.x_stride;
      int32_t acc[kRows][kUnit] = {};
      for (int k = begin; k < end; k += S * kPiece) {
        const Piece v = next;
        fetch(next);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (r >= rows) break;
          // (w reads as zero behind the last element)
          const uint4 c = k < K ? __ldg(reinterpret_cast<const uint4*>(x + r * p.x_stride + k)) : zero;
#pragma unroll
          for (int i = 0; i < kUnit; ++i) acc[r][i] = dot16(v.w[i], c, acc[r][i]);
        }
      }
      if (S > 1) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r < rows)
#pragma unroll
            for (int i = 0; i < kUnit; ++i) acc[r][i] = __reduce_add_sync(0xffffffffu, acc[r][i]);
        const int barrier = 1 + warp / S;  // of the unit's warps
        if (own > 0 && lane == 0) {
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int i = 0; i < kUnit; ++i) part[warp][r][i] = acc[r][i];
        }
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(barrier), "n"(S * 32) : "memory");
        if (own == 0) {
#pragma unroll
          for (int q = 1; q < S; ++q)
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
              for (int i = 0; i < kUnit; ++i) acc[r][i] += part[warp + q][r][i];
        }
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(barrier), "n"(S * 32) : "memory");
        if (own > 0) continue;
      }
      const float* sw = p.w_scales + (int64_t)busy[b][0] * (GLU ? 2 : 1) * N + f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;
        float y[kUnit];
        const float sx = p.x_scales[(row0 + r) * p.x_scale_stride];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          const int sum = S > 1 ? acc[r][i] : __reduce_add_sync(0xffffffffu, acc[r][i]);
          y[i] = __int2float_rn(sum) * (sx * sw[GLU ? i / 2 * N + i % 2 : i]);
        }
        uint8_t* to = p.out + ((row0 + r) * N + f) * 2;
        if (lane == 0) {
          if (GLU)
            *reinterpret_cast<uint32_t*>(to) = pack_bf16x2_rn(swiglu_of(y[0], y[2]), swiglu_of(y[1], y[3]));
          else
            *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2_rn(y[0], y[1]), pack_bf16x2_rn(y[2], y[3]));
        }
      }
    }
  }
}

template <bool GLU>
__global__ void __launch_bounds__(kThreads, kBlocks) k_expert_i8_few(ExpertI8Params p) {
  __shared__ Shared sm;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = (int)lane_id();
  const int E = p.num_experts;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int many = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, rows = 0;
      if (e < E) {
        lo = max(p.row_begin[e], 0);
        rows = (int)min((int64_t)max(p.row_end[e], 0), p.rows) - lo;
      }
      const unsigned some = __ballot_sync(0xffffffffu, rows > 0);
      const int at = many + __popc(some & ((1u << lane) - 1));
      if (rows > 0 && at < kFewRows) {
        sm.busy[at][0] = e;
        sm.busy[at][1] = lo;
        sm.busy[at][2] = rows;
      }
      many += __popc(some);
    }
    if (lane == 0) sm.num_busy = min(many, kFewRows);
  }
  __syncthreads();
  // As many warps to a unit as there are for all units, which only the counts of
  // rows tell: at most four.
  const int units = sm.num_busy * (p.out_features / features_of(GLU)), warps = gridDim.x * kWarps;
  if (units * 4 <= warps)
    work_on<GLU, 4>(p, sm, warp, lane);
  else if (units * 2 <= warps)
    work_on<GLU, 2>(p, sm, warp, lane);
  else
    work_on<GLU, 1>(p, sm, warp, lane);
}

template <bool GLU>
cudaError_t launch(const ExpertI8Params& p, int sms, cudaStream_t s) {
  const int64_t units = (p.rows < p.num_experts ? p.rows : p.num_experts) * (p.out_features / features_of(GLU));  // at most
  const int64_t need = (units * 4 + kWarps - 1) / kWarps, most = (int64_t)sms * kBlocks;
  ExpertI8Params q = p;
  void* args[] = {&q};
  return launch_pdl((const void*)k_expert_i8_few<GLU>, dim3((unsigned)(need < most ? need : most)), dim3(kThreads), 0, s, args);
}

}  // namespace

cudaError_t launch_expert_i8_few(const ExpertI8Params& p, bool glu, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
  return glu ? launch<true>(p, sms, s) : launch<false>(p, sms, s);
}

}  // namespace moe
