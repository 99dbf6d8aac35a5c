// experts.cu -- the experts' products on the tensor cores.
//
//   forward       y[s, n]  = sum_k x[s, k] w[e, n, k]
//   swiglu        the same for gate and up rows of w, silu(gate) * up and the
//                 8-bit checkpoint of gate and up in the epilogue
//   grad input    dx[s, k] = sum_n dy[s, n] w[e, n, k]
//   grad weight   dw[e, n, k] = sum_s dy[s, n] x[s, k]
//
// A pair of blocks (a cluster of two, tcgen05 cta_group::2) walks over output
// tiles of all experts, which it finds from the row ranges on the device. The
// tile's 256 M indices are features, 128 to a block, and its N indices up to
// 256 rows of one expert (256 columns of dw): an expert's rows are covered in
// steps of 32, so ragged experts cost little, and a few rows cost little more
// than reading the weights once. Each block brings its own 128 features and
// half of the N operand, 64 reduction steps at a time, so a block moves 32 KB
// per 128 x 256 x 64 products through L2 and shared memory, which is what a
// single block with a tile of that size (48 KB) is bound by.
//
// Warps 0 and 2 load features and rows with TMA (128-byte swizzle) into five
// or six stages; warp 1 of the even block issues tcgen05.mma (bf16 in, fp32
// accumulators in tensor memory) for both; warp 3 clears what a ragged
// reduction must not see; warps 4-11 store what is finished. Tensor memory
// holds two accumulators of 256 columns, so a tile's epilogue runs while the
// next one is multiplied. The forward product's operands are stored along the
// reduction (K-major); the gradients read the same buffers across it
// (MN-major), so nothing is transposed in memory.
//
// The accumulators of the row products lie feature by feature; 32 rows at a
// time they cross shared memory and leave as whole rows of 128 features. dw
// leaves as TMA boxes, added in L2 where it accumulates.
//
// What bounds it (peaks as measured: 6.79 TB/s, 1957 TFLOP/s burst and 1758
// sustained under the power cap). Many rows: the tensor cores, a step of a
// 256 x 256 tile takes 515 cycles of which 512 are theirs, and then the power
// cap: 16384 rows x 7168 -> 4096 over 32 experts of 512 take 522 us (1840
// TFLOP/s) in short runs and 573 to 643 us (a library's batched product 614 us)
// in long ones. A tile of n rows takes 2 n cycles a step in the tensor cores,
// and 256 + n for its operands (16 KB of features and 64 n bytes of rows for
// each SM, at 64 bytes a cycle from L2; measured 452 cycles at 192 rows, 504 at
// 224): 480 rows an expert 501 to 538 us, 416 rows 492; experts of 412 to 616
// rows take 670 to 725 us in long runs. Few rows: the weights, 8 rows an expert
// 274 to 283 us for 1.88 GB (6.9 TB/s). Weight gradients: their result, 3.76 GB
// of fp32 780 to 880 us (bf16 695 to 705, added to fp32 1483).
#include <mutex>

#include "row_tiles.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

enum { kForward = 0, kGlu = 1, kGradInput = 2, kGradWeight = 3 };

constexpr int kTileM = 256, kTileN = 256, kTileK = 64;  // of a pair
constexpr int kHalfM = 128;                             // of a block
constexpr int kBytesA = kHalfM * kTileK * 2, kBytesB = kTileN / 2 * kTileK * 2;
constexpr int kMaxStages = 6;
constexpr int kExpertThreads = 384;
constexpr int kEpilogueWarps = 8;  // two sets of four, a set covers the 128 features
constexpr int kTmemColumns = 512;
constexpr int kChunk = 32;                   // rows that cross shared memory together
constexpr int kChunkBytes = kChunk * 256;    // a row's part: 128 features in bf16, or 64 and their codes
constexpr int kBoxBytes = 4096;              // 32 rows of 128 bytes of dw
constexpr int kBoxes = 2;                    // of each warp
// A weight gradient's tile is short (a step per 64 rows of an expert) and its
// result large, so it has more room for what leaves and a stage less.
constexpr int stages_of(int mode) { return mode == kGradWeight ? 5 : 6; }

__device__ int32_t g_expert_status;  // MOE_OK, or MOE_ERR_TIMEOUT once a wait gave up

// The same where what is waited for may be as far away as an expert's last row
// (a weight gradient reduces over all of them): the budget is for one step. It
// starts again as long as this block's producer has begun steps since.
__device__ __forceinline__ bool warp_wait_steps(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                                const volatile uint32_t* begun) {
  uint32_t seen = *begun;
  while (!warp_wait(bar, parity, limit_ns)) {
    const uint32_t now = *begun;
    if (__all_sync(0xffffffffu, now == seen)) return false;
    seen = now;
  }
  return true;
}

// Named barriers of the epilogue warps. They wait without a limit, so whoever
// comes to one must know that the others do: a wait with a limit is followed
// by a vote, and one that ran out anywhere ends the loop everywhere. (With
// mbarriers instead, a tile's epilogue took half as long again.)
__device__ __forceinline__ void set_sync(int set) {
  if (set == 0)
    asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
  else
    asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
}
__device__ __forceinline__ void epilogue_sync() { asm volatile("barrier.cta.sync 3, 256;" ::: "memory"); }
__device__ __forceinline__ bool epilogue_agrees(bool yes) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 3, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)yes)
      : "memory");
  return all != 0;
}

// (evict-first: written once and read by another kernel later; it takes 3 to 8%
// off weight gradients of few rows)
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %6;\n\t}" ::"l"(
          map),
      "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)), "r"(on), "l"(l2_evict_first_policy())
      : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, const void* src, int x, int y, int z, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\t}" ::"l"(map),
      "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)), "r"(on)
      : "memory");
}

struct ExpertMaps {
  CUtensorMap a;     // features: w, or dy of the weight gradient
  CUtensorMap b[4];  // rows, in boxes of 16, 32, 64 and 128; the weight gradient's x in b[0]
  CUtensorMap out;   // dw
};

// One output tile of a pair.
struct Tile {
  int e, f0;      // expert, first feature
  int n0, n;      // first row of the expert (column of dw), and how many; n a multiple of 32
  int lo, rows;   // the expert's rows
};

struct ExpertControl {
  uint64_t full[kMaxStages], empty[kMaxStages], tail[kMaxStages], acc_full[2], acc_empty[2], most_full;
  uint32_t tmem;
  uint32_t begun;  // weight gradient: steps whose copies this block has asked for
};
// Shared memory behind the stages: what leaves, the control block, and
//   swiglu: the largest magnitudes of gate and up by row, of both blocks and
//           for two tiles, and their 448 / a (the partial ones of the four
//           warps pass through the room of what leaves);
//   all row products: the tiles before each expert.
constexpr size_t kStageBytes = kBytesA + kBytesB;
constexpr size_t leaving_bytes(int mode) { return mode == kGradWeight ? kEpilogueWarps * kBoxes * kBoxBytes : 2 * kChunkBytes; }
constexpr size_t glu_bytes(int mode) { return mode == kGlu ? (size_t)5 * 2 * kTileN * 4 : 0; }
constexpr size_t expert_smem(int mode, int experts) {
  return 1024 + stages_of(mode) * kStageBytes + leaving_bytes(mode) + glu_bytes(mode) +
         (mode == kGradWeight ? 0 : ((size_t)experts + 1) * 4) + sizeof(ExpertControl) + 16;
}

// A feature's gate is in the lane whose bit 3 is clear, its up eight lanes on.
// Of the 32 rows that both hold, the lower lane gets gate and up of the even
// ones, the upper lane those of the odd ones.
__device__ __forceinline__ void pair_up(const float (&v)[32], bool upper, float (&g)[16], float (&u)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float give = upper ? v[2 * i] : v[2 * i + 1], keep = upper ? v[2 * i + 1] : v[2 * i];
    const float got = __shfl_xor_sync(0xffffffffu, give, 8);
    g[i] = upper ? got : keep;
    u[i] = upper ? keep : got;
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
  return make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                    pack_bf16x2_rn(v[6], v[7]));
}

template <int MODE>
__global__ void __launch_bounds__(kExpertThreads, 1)
    k_expert(ExpertParams p, const __grid_constant__ ExpertMaps maps, uint64_t wait_ns) {
  constexpr int kStages = stages_of(MODE);
  extern __shared__ uint8_t expert_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>(((uintptr_t)expert_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* leaving = stages + kStages * kStageBytes;
  float* glu_mem = reinterpret_cast<float*>(leaving + leaving_bytes(MODE));
  ExpertControl& sm = *reinterpret_cast<ExpertControl*>(leaving + leaving_bytes(MODE) + glu_bytes(MODE));
  int32_t* first = reinterpret_cast<int32_t*>(&sm + 1);  // row tiles before expert e
  const int warp = threadIdx.x >> 5, lane = (int)lane_id();
  const int E = p.num_experts, K = p.in_features, N = p.out_features;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 4);   // at the even block: both blocks' producers (and their bytes)
      mbar_init(&sm.empty[i], 1);
      mbar_init(&sm.tail[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], 2 * kEpilogueWarps);  // at the even block, from both
    }
    mbar_init(&sm.most_full, 2 * kEpilogueWarps);
    sm.begun = 0;
    mbar_init_fence();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + (MODE == kGradWeight ? 2 : 5))  // a and b[0 .. 3], for the first copies
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<const CUtensorMap*>(&maps) + (threadIdx.x - 32))
                 : "memory");
  __syncthreads();
  // Tensor memory of a pair is allocated in both blocks, by both. Until they
  // have met, the other block may not run yet (its SM may still be busy with
  // the kernel before this one), and an allocation that reaches it then is
  // lost: both hang.
  cluster_sync();
  if (warp == 1) tmem_alloc(&sm.tmem, kTmemColumns);
  pdl_wait();
  pdl_trigger();
  auto rows_of = [&](int e, int& lo) {
    lo = max(p.row_begin[e], 0);
    return max((int)min((int64_t)max(p.row_end[e], 0), p.rows) - lo, 0);
  };
  if (MODE != kGradWeight && warp == 0) {
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int lo;
      const int n = e < E ? row_tiles(rows_of(e, lo), kTileN) : 0;
      const int inc = warp_inclusive_scan(n);
      if (e < E) first[e] = carry + inc - n;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) first[E] = carry;
  }
  tmem_fence_before();
  // (The other block's tensor memory is there once its warps 0 and 2, which
  // pass this barrier too, have arrived at a stage's barrier.)
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sm.tmem;

  // Tiles in order: expert, then features, then rows (columns of dw); pairs
  // take one each in turn, so that those running at one time share operands,
  // and each second round in the other direction: where wide and narrow tiles
  // alternate, an even number of pairs would give the wide ones to the same
  // pairs every time, and pairs that share weights would drift apart (480 rows
  // an expert: 583 to 607 us for 501 to 538).
  // (Tiles of a weight gradient's expert are alike, and neighbours in a round
  // share columns: there it costs 1%.)
  const int turn = MODE == kGradWeight ? pairs : 2 * (pairs - pair) - 1;
  const int features = MODE == kGradInput ? K : N;
  const int tile_features = MODE == kGlu ? kTileM / 2 : kTileM;
  const int across = (features + tile_features - 1) / tile_features;
  const int down = (K + kTileN - 1) / kTileN;  // weight gradient: column tiles
  const int num_tiles = MODE == kGradWeight ? E * across * down : first[E] * across;
  // The t-th tile; o is this warp's tile before, or has e = -1.
  auto find = [&](int t, Tile& o) {
    const int before = o.e;
    if (MODE == kGradWeight) {
      o.e = t / (across * down);
      const int i = t - o.e * (across * down);
      o.f0 = i / down * tile_features;
      o.n0 = i % down * kTileN;
      o.n = kTileN;
      if (o.e != before) o.rows = rows_of(o.e, o.lo);
    } else {
      o.e = max(o.e, 0);
      while (t >= first[o.e + 1] * across) ++o.e;
      if (o.e != before) o.rows = rows_of(o.e, o.lo);
      const int many = first[o.e + 1] - first[o.e];
      const int i = t - first[o.e] * across;
      o.f0 = i / many * tile_features;
      const int width = row_tile_width(o.rows, many);
      o.n0 = i % many * width;
      o.n = min(width, (max(o.rows - o.n0, 0) + 31) / 32 * 32);
    }
  };
  auto steps_of = [&](const Tile& t) {
    const int red = MODE == kGradWeight ? t.rows : MODE == kGradInput ? N : K;
    return t.n > 0 ? (red + kTileK - 1) / kTileK : 0;
  };
  bool ok = true;

  if (warp == 0 || warp == 2) {  // this block's features, and its rows, into shared memory
    const bool second = warp == 2;
    const uint32_t on = elect_one();
    const uint32_t full0 = in_block(&sm.full[0], 0), tail0 = in_block(&sm.tail[0], rank);
    Tile o;
    o.e = -1;
    int st = 0;
    uint32_t phase = 1;  // a fresh barrier's phase before the first counts as complete
    uint32_t begun = 0;
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      const int steps = steps_of(o);
      const int half = o.n / 2;
      // the boxes of this block's half: 16 << i rows each, the largest first,
      // two at most; rather than three, one that brings rows of no use
      int sizes = half / 16;
      if (__popc(sizes) > 2) sizes = 8;
      const uint32_t bytes = !second || MODE == kGradWeight ? kBytesA : (uint32_t)sizes * 16 * kTileK * 2;
      const int big = 31 - __clz(max(sizes, 1)), small = sizes & ~(1 << big);
      const CUtensorMap* map = &maps.a;
      if (second) map = &maps.b[MODE == kGradWeight ? 0 : big];
      const CUtensorMap* map2 = &maps.b[small ? 31 - __clz(small) : 0];
      const int feature = o.f0 + (int)rank * kHalfM;
      const int row = MODE == kGradWeight ? o.n0 + (int)rank * kHalfM : o.lo + o.n0 + (int)rank * half;
      for (int k = 0; k < steps; ++k) {
        if (!warp_wait(&sm.empty[st], phase, wait_ns)) {
          ok = false;
          break;
        }
        uint8_t* to = stages + st * kStageBytes + (second ? kBytesA : 0);
        const int k0 = k * kTileK;
        uint32_t bar = full0 + 8u * st;
        // a last step that ends inside 16 rows goes through the zeroing below
        if (MODE == kGradWeight && o.rows - k0 < kTileK && o.rows % 16) bar = tail0 + 8u * st;
        arrive_expect_at(bar, bytes, on);
        if (MODE == kGradWeight) {
          ++begun;
          if (on && !second) *const_cast<volatile uint32_t*>(&sm.begun) = begun;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tma_load_2d(to + i * 8192, map, (second ? row : feature) + i * 64, o.lo + k0, bar, on);
        } else if (second) {
          tma_load_2d(to, map, k0, row, bar, on);
          if (small) tma_load_2d(to + (16 << big) * 128, map2, k0, row + (16 << big), bar, on);
        } else if (MODE == kForward) {
          tma_load_3d(to, &maps.a, k0, feature, o.e, bar, on);
        } else if (MODE == kGlu) {
          // 8 features of gate, the same 8 of up, and so on
          tma_load_5d(to, &maps.a, k0, 0, 0, o.f0 / 8 + (int)rank * 8, o.e, bar, on);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) tma_load_3d(to + i * 8192, &maps.a, feature + i * 64, k0, o.e, bar, on);
        }
        next_stage<kStages>(st, phase);
      }
    }
    if (!ok) {
      // no copy may land after the block has exited; those in flight are
      // counted at the other block's barriers, so give them time instead
      if (on) g_expert_status = MOE_ERR_TIMEOUT;
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 3) {
    // The last 16 rows that a weight gradient multiplies may be in part those
    // of others: zeros instead, by each block in its own stage and ahead of
    // the products. (Both operands: what the others hold may not be finite.)
    if (MODE == kGradWeight) {
      Tile o;
      o.e = -1;
      int64_t begun = 0;
      uint32_t tail_bits = 0;  // parity of each stage's tail barrier
      for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
        find(t, o);
        begun += steps_of(o);
        const int left = o.rows % kTileK;
        if (o.rows % 16 == 0) continue;
        const int st = (int)((begun - 1) % kStages);
        if (!warp_wait_steps(&sm.tail[st], (tail_bits >> st) & 1u, wait_ns, &sm.begun)) {
          ok = false;
          break;
        }
        tail_bits ^= 1u << st;
        uint8_t* a = stages + st * kStageBytes;
        const int zero = ((left + 15) / 16 * 16 - left) * 8;  // 16-byte pieces per 64 columns
        for (int i = lane; i < zero; i += 32)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(a + c * 8192 + left * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        // for this block's two producers; the even block issues the products
        arrive_with_shared_at(in_block(&sm.full[st], 0), lane < 2);
      }
      if (!ok && lane == 0) g_expert_status = MOE_ERR_TIMEOUT;
    }
  } else if (warp == 1 && rank == 0) {  // tensor cores, for both blocks
    constexpr bool a_mn = MODE == kGradInput || MODE == kGradWeight, b_mn = MODE == kGradWeight;
    Tile o;
    o.e = -1;
    int st = 0, last = -1;  // last: the stage of the last MMAs, and its phase
    uint32_t phase = 0, last_phase = 0;
    const uint32_t on = elect_one();
    int acc = 0;             // accumulators begun
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      const int steps = steps_of(o);
      if (steps == 0) continue;
      const int as = acc & 1;
      if (acc >= 2 && !warp_wait(&sm.acc_empty[as], (uint32_t)((acc / 2 + 1) & 1), wait_ns)) {
        ok = false;
        break;
      }
      tmem_fence_after();
      const uint32_t idesc = instr_desc(true, a_mn, b_mn, kTileM, o.n);
      for (int k = 0; k < steps; ++k, next_stage<kStages>(st, phase)) {
        uint8_t* a = stages + st * kStageBytes;
        int parts = kTileK / 16;
        if (MODE == kGradWeight) parts = min(parts, (o.rows - k * kTileK + 15) / 16);
        const bool zeroed = MODE == kGradWeight && o.rows - k * kTileK < kTileK && o.rows % 16;
        // a zeroed stage was written by both blocks' warps
        if (!(MODE == kGradWeight && zeroed ? warp_wait_cluster(&sm.full[st], phase, wait_ns)
                                            : warp_wait(&sm.full[st], phase, wait_ns))) {
          ok = false;
          break;
        }
        tmem_fence_after();
        const uint64_t da = operand_desc(smem_u32(a), a_mn), db = operand_desc(smem_u32(a + kBytesA), b_mn);
        if (MODE != kGradWeight || parts == kTileK / 16) {
#pragma unroll
          for (int i = 0; i < kTileK / 16; ++i)
            mma_bf16(tmem + as * kTileN, da + i * (a_mn ? 2048 : 32) / 16, db + i * (b_mn ? 2048 : 32) / 16, idesc,
                     k > 0 || i > 0, on);
        } else {
          for (int i = 0; i < parts; ++i)
            mma_bf16(tmem + as * kTileN, da + i * 2048 / 16, db + i * 2048 / 16, idesc, k > 0 || i > 0, on);
        }
        mma_commit(&sm.empty[st], on);
        if (k == steps - 1) mma_commit(&sm.acc_full[as], on);
        last = st;
        last_phase = phase;
      }
      ++acc;
    }
    if (!ok && lane == 0) g_expert_status = MOE_ERR_TIMEOUT;
    // tensor memory is freed below: wait for the last MMAs, with the full budget
    if (last >= 0) mbar_wait(&sm.empty[last], last_phase);
  } else if (warp >= 4) {  // accumulators to memory: warp w reads tensor-memory lanes (w % 4) * 32 ..
    const int quarter = warp & 3, set = (warp - 4) >> 2;
    const uint32_t on = elect_one();
    const uint32_t acc_empty0 = in_block(&sm.acc_empty[0], 0);
    Tile o;
    o.e = -1;
    int acc = 0;
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      const bool some = steps_of(o) > 0;  // without rows a weight gradient is zero
      if (!some && MODE != kGradWeight) continue;
      const int as = acc & 1;
      if (some) {
        const uint32_t parity = (uint32_t)((acc / 2) & 1);
        ok = MODE == kGradWeight ? warp_wait_steps(&sm.acc_full[as], parity, wait_ns, &sm.begun)
                                 : epilogue_agrees(warp_wait(&sm.acc_full[as], parity, wait_ns));
        if (!ok) break;
        tmem_fence_after();
      }
      const uint32_t src = tmem + (uint32_t)(quarter * 32) * 65536u + (uint32_t)(as * kTileN);
      // the last columns have been read: the accumulator is free
      auto release = [&] {
        tmem_fence_before();
        __syncwarp();
        arrive_local_at(acc_empty0 + 8u * as, on);
      };
      if (MODE == kGradWeight) {
        // A set stores half of the columns, each warp in boxes of 32 rows x 128
        // bytes, two neighbours at a time, so that DRAM sees 256 bytes of a
        // row at a time. (16384 rows, 7168 x 4096, 32 experts, fp32: boxes one
        // by one 1033 us, in pairs 785 us. The products without any epilogue
        // take 462 us, the stores by themselves 620 us; stores of whole
        // sectors from registers, without shared memory, come to 812 us.)
        uint8_t* mine = leaving + (warp - 4) * kBoxes * kBoxBytes;
        const bool wide = p.grad_kind != MOE_GRAD_BF16;
        const int step = wide ? 32 : 64;
        const int n = o.f0 + (int)rank * kHalfM + quarter * 32;                        // first row of dw
        const int begin = set * kTileN / 2, last = n < N ? min(begin + kTileN / 2, K - o.n0) : 0;  // columns to store
        const bool store = some || p.grad_kind != MOE_GRAD_F32_ADD;
        for (int c0 = begin; store && c0 < last; c0 += kBoxes * step) {
          if (on) bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < kBoxes; ++j) {
            const int c = c0 + j * step;
            if (c >= last) break;
            uint8_t* box = mine + j * kBoxBytes;
            uint4 q[8];
            auto load = [&](int at, float (&v)[32]) {
              if (some) {
                tmem_load32(src + at, v);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.0f;
              }
            };
            float v[32];
            load(c, v);
            if (wide) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                q[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                  __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) q[i] = pack_bf16x8(v + 8 * i);
              load(c + 32, v);
#pragma unroll
              for (int i = 0; i < 4; ++i) q[4 + i] = pack_bf16x8(v + 8 * i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)  // the swizzle that the box is stored with
              *reinterpret_cast<uint4*>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) = q[i];
          }
          if (some && c0 + kBoxes * step >= last) release();
          fence_proxy_async_smem();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < kBoxes; ++j) {
            const int c = c0 + j * step;
            if (c >= last) break;
            if (p.grad_kind == MOE_GRAD_F32_ADD)
              tma_add_3d(&maps.out, mine + j * kBoxBytes, o.n0 + c, n, o.e, on);
            else
              tma_store_3d(&maps.out, mine + j * kBoxBytes, o.n0 + c, n, o.e, on);
          }
          if (on) bulk_commit();
        }
        if (some && last <= begin) release();
      } else {
        const int own = MODE == kGlu ? 64 : kHalfM;                // features of this block
        const int f = o.f0 + (int)rank * own;
        const int nf = min(max(features - f, 0), own);             // that exist, a multiple of 8
        const int valid = min(o.n, o.rows - o.n0);                 // rows of the tile that the expert has
        const bool upper = lane & 8;  // holds up
        const int here = MODE == kGlu ? quarter * 16 + (lane >> 4) * 8 + (lane & 7) : quarter * 32 + lane;  // this lane's feature
        float* scale_up = glu_mem + 4 * 2 * kTileN;                // [gate, up][row], 448 / a
        if (MODE == kGlu && p.ckpt) {
          // the largest magnitude of each row's 128 features of gate and up:
          // over the 16 lanes that hold one of the two (each step halves the
          // rows that a lane carries), over the four warps, and over the two
          // blocks, each of which gives its own to the other
          float* part = reinterpret_cast<float*>(leaving);         // [4 warps][gate, up][row]
          float* most = glu_mem + (acc & 1) * 2 * 2 * kTileN;      // [block][gate, up][row]
          for (int c = set * kChunk; c < o.n; c += 2 * kChunk) {
            float v[32];
            tmem_load32(src + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = here < nf ? fabsf(v[i]) : 0.0f;
#pragma unroll
            for (int many = 16; many > 1; many >>= 1) {
              const int o2 = many == 16 ? 16 : many / 2;  // lane bits 4, 2, 1 and 0
              const bool high = lane & o2;
#pragma unroll
              for (int i = 0; i < many; ++i) {
                const float give = high ? v[i] : v[i + many], keep = high ? v[i + many] : v[i];
                v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o2));
              }
            }
            const int row = c + (lane >> 4) * 16 + (lane & 7) * 2;  // its two rows
            *reinterpret_cast<float2*>(part + (quarter * 2 + (upper ? 1 : 0)) * kTileN + row) = make_float2(v[0], v[1]);
          }
          epilogue_sync();
          const uint32_t theirs = in_block(most, rank ^ 1);
          for (int i = set * 128 + quarter * 32 + lane; i < 2 * kTileN; i += 256) {
            const float a = fmaxf(fmaxf(part[i], part[i + 2 * kTileN]), fmaxf(part[i + 4 * kTileN], part[i + 6 * kTileN]));
            most[rank * 2 * kTileN + i] = a;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(theirs + (rank * 2 * kTileN + (uint32_t)i) * 4u), "f"(a)
                         : "memory");
          }
          __syncwarp();
          if (lane < 2) arrive_at(in_block(&sm.most_full, (uint32_t)lane));
          ok = epilogue_agrees(warp_wait_cluster(&sm.most_full, (uint32_t)(acc & 1), wait_ns));
          if (!ok) break;
          const int groups = (N + 127) / 128;
          for (int i = set * 128 + quarter * 32 + lane; i < 2 * kTileN; i += 256) {
            const int r = i % kTileN, h = i / kTileN;
            const float a = fmaxf(fmaxf(most[i], most[i + 2 * kTileN]), 1e-4f);
            scale_up[i] = __fdiv_rn(448.0f, a);
            if ((int)rank == h && r < valid)
              p.scales[((int64_t)o.lo + o.n0 + r) * 2 * groups + h * groups + o.f0 / 128] = __fdiv_rn(a, 448.0f);
          }
          epilogue_sync();
        }
        uint8_t* buf = leaving + set * kChunkBytes;
        if (set * kChunk >= o.n) release();
        for (int c = set * kChunk; c < o.n; c += 2 * kChunk) {
          // features to rows through the set's shared memory
          float v[32];
          tmem_load32(src + c, v);
          if (c + 2 * kChunk >= o.n) release();
          if (c != set * kChunk) set_sync(set);  // the rows before have been read
          if (MODE == kGlu) {
            float g[16], u[16];
            pair_up(v, upper, g, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = 2 * i + (upper ? 1 : 0);
              uint8_t* to = buf + r * 256;
              reinterpret_cast<uint16_t*>(to)[here] = (uint16_t)pack_bf16x2_rn(swiglu_of(g[i], u[i]), 0.0f);
              if (p.ckpt) {
                const uint32_t q =
                    cvt_e4m3x2(__fmul_rn(g[i], scale_up[c + r]), __fmul_rn(u[i], scale_up[kTileN + c + r]));
                to[128 + here] = (uint8_t)q;
                to[192 + here] = (uint8_t)(q >> 8);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              reinterpret_cast<uint16_t*>(buf + i * 256)[here] = (uint16_t)pack_bf16x2_rn(v[i], 0.0f);
          }
          set_sync(set);
          const int64_t row0 = (int64_t)o.lo + o.n0 + c;
          const int many = min(valid - c, kChunk);
          if (MODE == kGlu) {
            for (int i = quarter * 32 + lane; i < kChunk * 8; i += 128) {
              const int r = i / 8, at = i % 8 * 8;  // 8 features
              if (r >= many || at >= nf) continue;
              const uint8_t* from = buf + r * 256;
              st_v4(p.out + ((row0 + r) * N + f + at) * 2, *reinterpret_cast<const uint4*>(from + at * 2));
              if (p.ckpt) {
                uint8_t* to = p.ckpt + (row0 + r) * 2 * N + f + at;
                *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from + 128 + at);
                *reinterpret_cast<uint2*>(to + N) = *reinterpret_cast<const uint2*>(from + 192 + at);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < kChunk * 16 / 128; ++j) {
              const int i = j * 128 + quarter * 32 + lane, r = i / 16, at = i % 16 * 8;
              if (r < many && at < nf)
                st_v4(p.out + ((row0 + r) * features + f + at) * 2, *reinterpret_cast<const uint4*>(buf + r * 256 + at * 2));
            }
          }
        }
      }
      if (some) ++acc;
    }
    if (!ok && lane == 0) g_expert_status = MOE_ERR_TIMEOUT;
    bulk_wait_read_all();
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  if (warp == 1) tmem_free(tmem, kTmemColumns);
  __syncwarp();
  cluster_sync();  // and neither leaves before both have freed theirs
}

// Tensor [depth][rows][width] (two dimensions where depth is 0) of bf16 or
// fp32 with `stride` elements between rows, in boxes of 128 bytes x box_rows;
// what lies outside reads as zero and is not written.
bool make_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t depth, int64_t stride,
              int box_rows, bool f32 = false) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)stride * size, (cuuint64_t)stride * size * (cuuint64_t)rows};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, depth > 0 ? 3 : 2,
            const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// w [E][2F][K] as [E][F / 8][gate, up][8][K], in boxes of 64 gate features, 8
// by 8 in turn with their up features.
bool make_glu_map(CUtensorMap* map, const void* base, int64_t K, int64_t F, int64_t E) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t k = (cuuint64_t)K * 2, f = (cuuint64_t)F;
  const cuuint64_t dims[5] = {(cuuint64_t)K, 8, 2, f / 8, (cuuint64_t)E};
  const cuuint64_t strides[4] = {k, f * k, 8 * k, 2 * f * k};
  const cuuint32_t box[5] = {64, 8, 2, 8, 1}, one[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pairs that can be resident at once on the current device, looked up once
// per device and kernel.
template <int MODE>
int resident_pairs(int dev, int sms) {
  static std::once_flag once[64];
  static int found[64];
  if (dev >= 64) return 0;
  std::call_once(once[dev], [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
    cfg.blockDim = dim3(kExpertThreads);
    cfg.dynamicSmemBytes = expert_smem(MODE, MOE_MAX_EXPERTS);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (const void*)k_expert<MODE>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    found[dev] = n;
  });
  return found[dev];
}

template <int MODE>
cudaError_t launch(const ExpertParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
  const int64_t K = p.in_features, N = p.out_features, E = p.num_experts;
  ExpertMaps maps;
  bool ok = true;
  if (MODE == kGradWeight) {
    const bool f32 = p.grad_kind != MOE_GRAD_BF16;
    ok = make_map(&maps.a, p.x, N, p.rows, 0, N, kTileK) &&
         make_map(&maps.b[0], p.x2, K, p.rows, 0, p.x_stride, kTileK) &&
         make_map(&maps.out, p.out, K, N, E, K, 32, f32);
  } else {
    if (MODE == kForward) ok = make_map(&maps.a, p.w, K, N, E, K, kHalfM);
    if (MODE == kGlu) ok = make_glu_map(&maps.a, p.w, K, N, E);
    if (MODE == kGradInput) ok = make_map(&maps.a, p.w, K, N, E, K, kTileK);
    const int64_t width = MODE == kGradInput ? N : K, stride = MODE == kGradInput ? N : p.x_stride;
    for (int i = 0; i < 4; ++i) ok = ok && make_map(&maps.b[i], p.x, width, p.rows, 0, stride, 16 << i);
  }
  if (!ok) return cudaErrorUnknown;
  const void* fn = (const void*)k_expert<MODE>;
  cudaError_t err = ensure_dynamic_smem(fn, expert_smem(MODE, MOE_MAX_EXPERTS));
  if (err != cudaSuccess) return err;
  const int64_t pairs = resident_pairs<MODE>(dev, sms);
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  // the row counts are on the device: as many pairs as there can be tiles
  const int64_t features = MODE == kGradInput ? K : N, width = MODE == kGlu ? kTileM / 2 : kTileM;
  const int64_t across = (features + width - 1) / width;
  const int64_t most = across * (MODE == kGradWeight ? E * ((K + kTileN - 1) / kTileN) : E + p.rows / kTileN);
  ExpertParams q = p;
  uint64_t wait_ns = wait_limit_ns();
  void* args[] = {&q, &maps, &wait_ns};
  return launch_pdl(fn, dim3((unsigned)(2 * (most < pairs ? most : pairs))), dim3(kExpertThreads),
                    expert_smem(MODE, p.num_experts), s, args, 2);
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
