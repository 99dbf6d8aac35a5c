// experts.cu -- the experts' products on the tensor cores.
//
//   forward       y[s, n]  = sum_k x[s, k] w[e, n, k]
//   swiglu        the same for gate and up rows of w, silu(gate) * up and the
//                 8-bit checkpoint of gate and up in the epilogue
//   grad input    dx[s, k] = sum_n dy[s, n] w[e, n, k]
//   grad weight   dw[e, n, k] = sum_s dy[s, n] x[s, k]
//
// One persistent block per SM walks over the 128 x 256 output tiles of all
// experts, which it finds from the row ranges on the device. Warp 0 brings
// operand tiles of 64 reduction steps into shared memory with TMA (128-byte
// swizzle), warp 1 issues tcgen05.mma (bf16 in, fp32 accumulators in tensor
// memory), warps 2-5 read finished accumulators and store them. Tensor memory
// holds two accumulators of 256 columns, so a tile's epilogue runs while the
// next one is multiplied. The reduction runs along the stored rows of both
// operands in the forward product (K-major operands); the gradients read the
// same buffers with the reduction across rows (MN-major operands), so nothing
// is transposed in memory.
#include <cuda.h>

#include "moe_internal.cuh"

namespace moe {

namespace {

enum { kForward = 0, kGlu = 1, kGradInput = 2, kGradWeight = 3 };

constexpr int kTileM = 128, kTileN = 256, kTileK = 64;
constexpr int kBytesA = kTileM * kTileK * 2, kBytesB = kTileN * kTileK * 2;
constexpr int kStages = 4;
constexpr int kExpertThreads = 192;
constexpr int kTmemColumns = 512;

__device__ int32_t g_expert_status;  // MOE_OK, or MOE_ERR_TIMEOUT once a wait gave up

// ---- tcgen05 and TMA --------------------------------------------------------

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// Arrives on bar when every MMA issued so far by this thread has completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 lanes x 32 columns of fp32: lane l of the warp gets tensor-memory lane
// (warp % 4) * 32 + l, columns [addr, addr + 32).
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Shared-memory operand descriptor, 128-byte swizzle (16-byte units: start in
// bits 0-13, leading stride in 16-29, stride in 32-45; bit 46 set; swizzle in
// 61-63). An atom is 8 rows of 128 bytes = 1024 bytes.
//  K-major: rows are the M or N index; the next 8 rows follow at 1024 bytes.
//  MN-major: rows are reduction steps, 64 M or N indices each; the next 8
//  steps follow at 1024 bytes, the next 64 indices at 64 rows = 8192 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn_major) {
  const uint64_t lead = mn_major ? 8192 / 16 : 1, stride = 1024 / 16;
  return (uint64_t)((addr >> 4) & 0x3fff) | lead << 16 | stride << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor: fp32 accumulators (bit 4), bf16 A and B (bits 7 and
// 10), MN-major A and B (bits 15 and 16), N / 8 in bits 17-22, M / 16 in 24-28.
__host__ __device__ constexpr uint32_t instr_desc(bool a_mn, bool b_mn, int n) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn ? 1u << 15 : 0) | (b_mn ? 1u << 16 : 0) | (uint32_t)(n / 8) << 17 |
         (uint32_t)(kTileM / 16) << 24;
}

struct ExpertMaps {
  CUtensorMap a, b;
};

// One output tile.
struct Tile {
  int e, m0, c0;  // expert, first row (a row of w for the weight gradient), first column
  int lo, rows;   // the expert's rows
};

struct ExpertSmem {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int32_t lo[MOE_MAX_EXPERTS], rows[MOE_MAX_EXPERTS];
  int32_t first[MOE_MAX_EXPERTS + 1];  // row tiles before expert e
};
constexpr size_t kExpertSmemBytes = 1024 + (size_t)kStages * (kBytesA + kBytesB) + sizeof(ExpertSmem);

__device__ __forceinline__ void pack_store(uint8_t* dst, const float* v) {
  st_v4(dst, make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                        pack_bf16x2_rn(v[6], v[7])));
}
__device__ __forceinline__ uint2 codes8(const float* v, float inv) {
  return make_uint2(cvt_e4m3x2(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)) |
                        cvt_e4m3x2(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv)) << 16,
                    cvt_e4m3x2(__fmul_rn(v[4], inv), __fmul_rn(v[5], inv)) |
                        cvt_e4m3x2(__fmul_rn(v[6], inv), __fmul_rn(v[7], inv)) << 16);
}

template <int MODE>
__global__ void __launch_bounds__(kExpertThreads, 1)
    k_expert(ExpertParams p, const __grid_constant__ ExpertMaps maps, uint64_t wait_ns) {
  extern __shared__ uint8_t expert_smem[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>(((uintptr_t)expert_smem + 1023) & ~(uintptr_t)1023);
  ExpertSmem& sm = *reinterpret_cast<ExpertSmem*>(tiles + (size_t)kStages * (kBytesA + kBytesB));
  const int warp = threadIdx.x >> 5, lane = (int)lane_id();
  const int E = p.num_experts, K = p.in_features, N = p.out_features;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], 4);
    }
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(&sm.tmem, kTmemColumns);
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e < E; e += kExpertThreads) {
    const int lo = max(p.row_begin[e], 0);
    const int hi = (int)min((int64_t)p.row_end[e], p.rows);
    sm.lo[e] = lo;
    sm.rows[e] = max(hi - lo, 0);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 0) {  // row tiles before each expert
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < E ? (sm.rows[e] + kTileM - 1) / kTileM : 0;
      const int inc = warp_inclusive_scan(n);
      if (e < E) sm.first[e] = carry + inc - n;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) sm.first[E] = carry;
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;

  // Tiles in order: expert, then column tile, then row tile; blocks take
  // every gridDim.x-th.
  const int cols = MODE == kGradInput || MODE == kGradWeight ? K : N;
  const int tile_cols = MODE == kGlu ? kTileN / 2 : kTileN;
  const int across = (cols + tile_cols - 1) / tile_cols;
  const int down = (N + kTileM - 1) / kTileM;  // weight gradient: row tiles of dw
  const int64_t num_tiles = MODE == kGradWeight ? (int64_t)E * across * down : (int64_t)sm.first[E] * across;
  auto find = [&](int64_t t, int& e) {  // e: the expert of this warp's last tile
    Tile o;
    int m, c;
    if (MODE == kGradWeight) {
      e = (int)(t / (across * down));
      const int i = (int)(t % (across * down));
      m = i / across;
      c = i % across;
    } else {
      while (t >= (int64_t)sm.first[e + 1] * across) ++e;
      const int n = sm.first[e + 1] - sm.first[e];
      const int i = (int)(t - (int64_t)sm.first[e] * across);
      m = i % n;
      c = i / n;
    }
    o.e = e;
    o.m0 = m * kTileM;
    o.c0 = c * tile_cols;
    o.lo = sm.lo[e];
    o.rows = sm.rows[e];
    return o;
  };
  auto steps_of = [&](const Tile& t) {
    const int red = MODE == kGradWeight ? t.rows : MODE == kGradInput ? N : K;
    return (red + kTileK - 1) / kTileK;
  };
  bool ok = true;

  if (warp == 0) {  // operand tiles into shared memory
    if (lane == 0) {
      int e = 0;
      int64_t issued = 0;
      for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const Tile o = find(t, e);
        const int steps = steps_of(o);
        for (int k = 0; k < steps; ++k, ++issued) {
          const int st = (int)(issued % kStages);
          if (issued >= kStages && !mbar_wait(&sm.empty[st], (uint32_t)((issued / kStages + 1) & 1), wait_ns)) {
            ok = false;
            break;
          }
          uint8_t* a = tiles + (size_t)st * (kBytesA + kBytesB);
          uint8_t* b = a + kBytesA;
          uint64_t* bar = &sm.full[st];
          mbar_arrive_expect_tx(bar, kBytesA + kBytesB);
          const int k0 = k * kTileK;
          if (MODE == kGradWeight) {
            for (int i = 0; i < kTileM / 64; ++i) tma_load_2d(a + i * 8192, &maps.a, o.m0 + i * 64, o.lo + k0, bar);
            for (int i = 0; i < kTileN / 64; ++i) tma_load_2d(b + i * 8192, &maps.b, o.c0 + i * 64, o.lo + k0, bar);
          } else {
            tma_load_2d(a, &maps.a, k0, o.lo + o.m0, bar);
            if (MODE == kForward) {
              tma_load_3d(b, &maps.b, k0, o.c0, o.e, bar);
            } else if (MODE == kGlu) {
              tma_load_3d(b, &maps.b, k0, o.c0, o.e, bar);
              tma_load_3d(b + kBytesB / 2, &maps.b, k0, N + o.c0, o.e, bar);
            } else {
              for (int i = 0; i < kTileN / 64; ++i) tma_load_3d(b + i * 8192, &maps.b, o.c0 + i * 64, k0, o.e, bar);
            }
          }
        }
      }
      if (!ok) g_expert_status = MOE_ERR_TIMEOUT;
      // no copy may land after the block has exited: the last phase of every
      // stage in use, with the full budget
      for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        mbar_wait(&sm.full[i % kStages], (uint32_t)((i / kStages) & 1));
    }
  } else if (warp == 1) {  // tensor cores
    constexpr bool a_mn = MODE == kGradWeight, b_mn = MODE == kGradInput || MODE == kGradWeight;
    constexpr uint32_t idesc = instr_desc(a_mn, b_mn, kTileN);
    int e = 0;
    int64_t taken = 0;
    int acc = 0;  // accumulators begun
    for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
      const Tile o = find(t, e);
      const int steps = steps_of(o);
      if (steps == 0) continue;
      const int as = acc & 1;
      if (acc >= 2 && !__all_sync(0xffffffffu, mbar_wait(&sm.acc_empty[as], (uint32_t)((acc / 2 + 1) & 1), wait_ns))) {
        ok = false;
        break;
      }
      tmem_fence_after();
      for (int k = 0; k < steps; ++k, ++taken) {
        const int st = (int)(taken % kStages);
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[st], (uint32_t)((taken / kStages) & 1), wait_ns))) {
          ok = false;
          break;
        }
        tmem_fence_after();
        uint8_t* a = tiles + (size_t)st * (kBytesA + kBytesB);
        int parts = kTileK / 16;
        if (MODE == kGradWeight && k == steps - 1) {
          // the rows after the expert's last belong to others: zeros instead,
          // up to the next whole step of 16
          const int left = o.rows - k * kTileK;
          parts = (left + 15) / 16;
          const int zero = (parts * 16 - left) * 8;  // 16-byte pieces per 64 columns
          for (int i = lane; i < zero; i += 32)
            for (int c = 0; c < (kTileM + kTileN) / 64; ++c)
              *reinterpret_cast<uint4*>(a + c * 8192 + left * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          const uint64_t da = operand_desc(smem_u32(a), a_mn), db = operand_desc(smem_u32(a + kBytesA), b_mn);
          for (int i = 0; i < parts; ++i)
            mma_bf16(tmem + as * kTileN, da + i * (a_mn ? 2048 : 32) / 16, db + i * (b_mn ? 2048 : 32) / 16, idesc,
                     k > 0 || i > 0);
          mma_commit(&sm.empty[st]);
          if (k == steps - 1) mma_commit(&sm.acc_full[as]);
        }
        __syncwarp();
      }
      ++acc;
    }
    if (!ok && lane == 0) g_expert_status = MOE_ERR_TIMEOUT;
    // tensor memory is freed below: wait for the last MMAs, with the full budget
    if (taken > 0) mbar_wait(&sm.empty[(taken - 1) % kStages], (uint32_t)(((taken - 1) / kStages) & 1));
  } else {  // accumulators to memory: warp w reads tensor-memory lanes (w % 4) * 32 ..
    const int quarter = warp & 3;
    int e = 0;
    int acc = 0;
    for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
      const Tile o = find(t, e);
      const int m = o.m0 + quarter * 32 + lane;
      const bool some = steps_of(o) > 0;  // without rows a weight gradient is zero
      const int as = acc & 1;
      if (some) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.acc_full[as], (uint32_t)((acc / 2) & 1), wait_ns))) {
          ok = false;
          break;
        }
        tmem_fence_after();
      }
      const uint32_t src = tmem + (uint32_t)(quarter * 32) * 65536u + (uint32_t)(as * kTileN);
      const int width = min(cols - o.c0, tile_cols);  // columns of this tile, a multiple of 8
      if (MODE == kGlu) {
        const bool on = m < o.rows;
        const int64_t row = (int64_t)o.lo + m;
        const int groups = (N + 127) / 128;
        float inv_g = 0.0f, inv_u = 0.0f;
        if (p.ckpt) {  // first pass: the largest magnitudes of the group
          float ag = 0.0f, au = 0.0f;
          for (int c = 0; c < width; c += 32) {
            float g[32], u[32];
            tmem_load32(src + c, g);
            tmem_load32(src + kTileN / 2 + c, u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i < width) {
                ag = fmaxf(ag, fabsf(g[i]));
                au = fmaxf(au, fabsf(u[i]));
              }
          }
          ag = fmaxf(ag, 1e-4f);
          au = fmaxf(au, 1e-4f);
          inv_g = __fdiv_rn(448.0f, ag);
          inv_u = __fdiv_rn(448.0f, au);
          if (on) {
            float* s = p.scales + row * 2 * groups + o.c0 / 128;
            s[0] = __fdiv_rn(ag, 448.0f);
            s[groups] = __fdiv_rn(au, 448.0f);
          }
        }
        for (int c = 0; c < width; c += 32) {
          float g[32], u[32];
          tmem_load32(src + c, g);
          tmem_load32(src + kTileN / 2 + c, u);
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (!on || c + i >= width) continue;
            const int64_t at = o.c0 + c + i;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = swiglu_of(g[i + j], u[i + j]);
            pack_store(p.out + (row * N + at) * 2, v);
            if (p.ckpt) {
              *reinterpret_cast<uint2*>(p.ckpt + row * 2 * N + at) = codes8(g + i, inv_g);
              *reinterpret_cast<uint2*>(p.ckpt + row * 2 * N + N + at) = codes8(u + i, inv_u);
            }
          }
        }
      } else {
        const bool on = MODE == kGradWeight ? m < N : m < o.rows;
        const int64_t row = MODE == kGradWeight ? (int64_t)o.e * N + m : (int64_t)o.lo + m;
        for (int c = 0; c < width; c += 32) {
          float v[32];
          if (some) {
            tmem_load32(src + c, v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (!on || c + i >= width) continue;
            const int64_t at = row * cols + o.c0 + c + i;
            if (MODE != kGradWeight || p.grad_kind == MOE_GRAD_BF16) {
              pack_store(p.out + at * 2, v + i);
            } else if (p.grad_kind == MOE_GRAD_F32 || some) {
              float4* d = reinterpret_cast<float4*>(p.out + at * 4);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float4 r = make_float4(v[i + 4 * h], v[i + 4 * h + 1], v[i + 4 * h + 2], v[i + 4 * h + 3]);
                if (p.grad_kind == MOE_GRAD_F32_ADD) {
                  const float4 was = d[h];
                  r = make_float4(was.x + r.x, was.y + r.y, was.z + r.z, was.w + r.w);
                }
                d[h] = r;
              }
            }
          }
        }
      }
      if (some) {
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.acc_empty[as]);
        ++acc;
      }
    }
    if (!ok && lane == 0) g_expert_status = MOE_ERR_TIMEOUT;
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 1) tmem_free(tmem, kTmemColumns);
}

// cuTensorMapEncodeTiled, looked up once (the library links no driver stub).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return (EncodeTiled)f;
  }();
  return fn;
}

// bf16 tensor [depth][rows][width] with `stride` elements between rows, read
// in boxes of 64 x box_rows; what lies outside reads as zero.
bool make_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t depth, int64_t stride,
              int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)stride * 2 * (cuuint64_t)rows};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, depth > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch(const ExpertParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
  const int64_t K = p.in_features, N = p.out_features, E = p.num_experts;
  ExpertMaps maps;
  bool ok;
  if (MODE == kForward || MODE == kGlu)
    ok = make_map(&maps.a, p.x, K, p.rows, 0, p.x_stride, kTileM) &&
         make_map(&maps.b, p.w, K, MODE == kGlu ? 2 * N : N, E, K, MODE == kGlu ? kTileN / 2 : kTileN);
  else if (MODE == kGradInput)
    ok = make_map(&maps.a, p.x, N, p.rows, 0, N, kTileM) && make_map(&maps.b, p.w, K, N, E, K, kTileK);
  else
    ok = make_map(&maps.a, p.x, N, p.rows, 0, N, kTileK) && make_map(&maps.b, p.x2, K, p.rows, 0, p.x_stride, kTileK);
  if (!ok) return cudaErrorUnknown;
  const void* fn = (const void*)k_expert<MODE>;
  cudaError_t err = ensure_dynamic_smem(fn, kExpertSmemBytes);
  if (err != cudaSuccess) return err;
  // the row counts are on the device: as many blocks as there can be tiles
  const int64_t cols = MODE == kForward || MODE == kGlu ? N : K, width = MODE == kGlu ? kTileN / 2 : kTileN;
  const int64_t row_tiles = MODE == kGradWeight ? E * ((N + kTileM - 1) / kTileM) : E + p.rows / kTileM;
  const int64_t most = row_tiles * ((cols + width - 1) / width);
  ExpertParams q = p;
  uint64_t wait_ns = wait_limit_ns();
  void* args[] = {&q, &maps, &wait_ns};
  return launch_pdl(fn, dim3((unsigned)(most < sms ? most : sms)), dim3(kExpertThreads), kExpertSmemBytes, s, args);
}

}  // namespace

int read_expert_status(int32_t* out, bool clear) {
  int32_t v = 0;
  const int32_t zero = MOE_OK;
  if (cudaMemcpyFromSymbol(&v, g_expert_status, 4) != cudaSuccess ||
      (clear && cudaMemcpyToSymbol(g_expert_status, &zero, 4) != cudaSuccess)) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  *out = v;
  return MOE_OK;
}

cudaError_t launch_expert_product(const ExpertParams& p, cudaStream_t s) { return launch<kForward>(p, s); }
cudaError_t launch_expert_swiglu(const ExpertParams& p, cudaStream_t s) { return launch<kGlu>(p, s); }
cudaError_t launch_expert_grad_input(const ExpertParams& p, cudaStream_t s) { return launch<kGradInput>(p, s); }
cudaError_t launch_expert_grad_weight(const ExpertParams& p, cudaStream_t s) { return launch<kGradWeight>(p, s); }

}  // namespace moe
