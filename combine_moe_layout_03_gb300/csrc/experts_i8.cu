// experts_i8.cu -- the experts' products of 8-bit integers on the tensor cores.
//
//   product  y[s, n] = (sum_k x[s, k] w[e, n, k]) * (sx[s] * sw[e, n])
//   swiglu   the same for gate and up rows of w, and silu(gate) * up
//
// This chip's integer tensor rate is a fraction of its 16-bit float rate, so
// whole numbers are multiplied as f16: every int8 is one exactly, products of
// two are below 2^15 and their sums exact in the fp32 accumulators up to 2^24.
// Operands travel and wait in 8 bits and become f16 on their way into the
// tensor cores.
//
// A pair of blocks (a cluster of two, tcgen05 cta_group::2) walks over output
// tiles as the bf16 products do: 256 features (M), 128 to a block, by up to 192
// rows of one expert (N), in steps of 32. Warps 0 and 2 load features and rows
// with TMA, 128 reduction steps at a time. Warps 4-11 turn features into f16 and
// put them into tensor memory, from where the products take their M operand, so
// that shared memory holds them in 8 bits only. Warps 12-19 turn rows into f16 in
// shared memory. Both are two sets of four warps, which take one load each in
// turn: a load's way through a set is longer than its products (16384 rows below:
// one set 1361 us for 939, when that was tried; three sets 668 for 646 now). Warp
// 1 of the even block issues tcgen05.mma for both blocks; warps 20-23 scale what
// is finished and store it.
//
// Tensor memory holds two accumulators as wide as the call's widest tile, so that
// a tile's epilogue runs beside the next one's products, and in the rest of its
// 512 columns features: two loads of them beside tiles of 192 rows (tiles of 160
// and 128 leave room for three and four, and are slower: 680 and 727 us for 655
// with the 16384 rows below), seven beside 32. Shared memory is shared out in the
// same way, so that few rows leave room for ten loads of weights under way.
//
// What bounds it. Many rows: three things that are close together. A load of a
// tile of n rows takes 4 n cycles in the tensor cores. It moves 32 KB of features
// (in by TMA, out to the converters) and 384 n bytes of rows (64 n in, 64 n out,
// 128 n in as f16, 128 n out to the tensor cores) through a block's shared memory,
// at 128 bytes a cycle 256 + 3 n cycles (768 + 3 n, were the features as f16
// there too). And it is 600 instructions for each of an SM's schedulers at 192
// rows, 300 of them the conversions. Full tiles take 970 cycles a load, 768 of
// them the products'. Long runs meet the power cap besides: 16384 rows in 32
// experts of 410 to 614, 7168 -> 2 x 2048, hold 1.4 kW and 1657 of 2070 MHz, 600 to
// 665 us by GPU (1450 to 1600 TFLOP/s; in bf16 691 to 726 us). 4608 rows in 8
// experts run at 1720 TFLOP/s in short runs and 1600 in long ones, 12345 uneven
// rows 2048 -> 7168 at 1370 to 1440 (248 to 265 us).
// Few rows: the weights, 256 rows in 32 experts 142 to 149 us (941 MB, 6.3 to 6.6 TB/s).
#include <mutex>

#include "row_tiles.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kTileM = 256, kTileN = 192;     // of a pair
constexpr int kHalfM = 128;                   // of a block
constexpr int kLoadK = 128, kStepK = 64;      // reduction steps loaded together, and multiplied together
// Stages: of what is loaded (5 to 10, by the widest tile; with more than some 900
// experts 4), of features as f16 (2 to 7), of rows as f16, and of barriers between
// converters and products, which are more than stages of either. (Four of rows
// and of loads: full tiles 161.7 us for 158.4, tiles of 160 rows 105 for 97.)
constexpr int kMostLoads = 10, kRowStages = 3, kRing = 8;
constexpr int kBytesA = kHalfM * kLoadK;
constexpr int kTmemColumns = 512;
constexpr int kStageColumns = kLoadK / 2;     // a load's features as f16
constexpr int kThreads = 768;
constexpr int kChunk = 32;                    // rows that leave together
constexpr int kPitch = 272;                   // bytes of a row's 128 features in bf16, and 16 so that eight rows lie in all banks
constexpr int kChunkBytes = kChunk * kPitch;

__device__ int32_t g_expert_i8_status;  // MOE_OK, or MOE_ERR_TIMEOUT once a wait gave up

struct Maps {
  CUtensorMap a;     // features
  CUtensorMap b[3];  // rows, in boxes of 16, 32 and 64
};

struct Tile {
  int e, f0;     // expert, first feature
  int n0, n;     // first row of the expert, and how many; n a multiple of 32
  int lo, rows;  // the expert's rows
};

struct Control {
  uint64_t loaded[kMostLoads], used[kMostLoads], acc_full[2], acc_empty[2];
  uint64_t full[kRing], done[kRing];
  uint32_t tmem;
  int32_t width;  // of the widest tile
  alignas(8) float row_scales[2][kTileN];  // read two at a time
};
// Shared memory: the stages have what the others leave, from a multiple of 1024 on.
constexpr uint32_t kSharedBytes = 227 * 1024;
constexpr uint32_t stage_bytes(int experts) {
  return (kSharedBytes - 1024 - kChunkBytes - (uint32_t)sizeof(Control) - ((uint32_t)experts + 1) * 4) / 1024 * 1024;
}
static_assert(stage_bytes(MOE_MAX_EXPERTS) >= 4 * (kBytesA + kTileN / 2 * kLoadK) + kRowStages * kTileN * kLoadK, "four loads beside the widest tiles");

// Named barrier of the epilogue warps, and a vote at it. It waits without a
// limit, so whoever comes must know that the others do: a wait with a limit is
// followed by the vote, and one that ran out anywhere ends the loop everywhere.
__device__ __forceinline__ void epilogue_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool epilogue_agrees(bool yes) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)yes)
      : "memory");
  return all != 0;
}

// A wait of a whole warp: all lanes ask at once and go on together, without a
// branch that the compiler would have to expect them to take apart.
template <bool CLUSTER>
__device__ __forceinline__ bool asks(uint64_t* bar, uint32_t parity) {
  if (!CLUSTER) return __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok);
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool waits(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (limit_ns < kWaitLimitNs)  // a lowered budget (test hook): polls without suspending
    return CLUSTER ? warp_wait_cluster(bar, parity, limit_ns) : warp_wait(bar, parity, limit_ns);
  if (asks<CLUSTER>(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!asks<CLUSTER>(bar, parity)) {
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > limit_ns)) return false;
  }
  return true;
}

// One step's products, the M operand from tensor memory: four of 16 reduction
// steps each, which are 8 columns of it and 32 bytes of the rows.
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(on)
      : "memory");
}

// 32 lanes x 32 columns: lane l of the warp writes tensor-memory lane
// (warp % 4) * 32 + l.
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t* r) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// Four int8 -> two f16 pairs: the byte plus 128 becomes the low bits of a f16
// of 1024 and more, from which 1024 + 128 is taken, exactly.
__device__ __forceinline__ void f16_of(uint32_t v, uint32_t* r) {
  const uint32_t t = v ^ 0x80808080u;
  r[0] = __byte_perm(t, 0x64646464u, 0x4140);
  r[1] = __byte_perm(t, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(r[0]) : "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(r[1]) : "r"(0x64806480u));
}
__device__ __forceinline__ void f16_of(uint4 v, uint32_t* r) {
  f16_of(v.x, r);
  f16_of(v.y, r + 2);
  f16_of(v.z, r + 4);
  f16_of(v.w, r + 6);
}

// 16 lanes x 32 columns of accumulators as a matrix product's fragment: v[4j]
// and v[4j + 1] are lane l / 4's columns 8j + 2 (l % 4) and the next, v[4j + 2]
// and v[4j + 3] lane l / 4 + 8's.
__device__ __forceinline__ void tmem_load16x32(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 matrices of 16-bit values, each lane with two of a column, to the
// rows whose addresses lanes 8m .. 8m + 7 give for matrix m.
__device__ __forceinline__ void store_transposed(uint32_t row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// What all lanes of a warp hold alike, in a form that tells the compiler so:
// it then keeps it, and what follows from it, in uniform registers, where the
// operands of copies and products have to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

template <bool GLU>
__global__ void __launch_bounds__(kThreads, 1) k_expert_i8(ExpertI8Params p, const __grid_constant__ Maps maps, uint64_t wait_ns) {
  extern __shared__ uint8_t expert_raw[];
  // (an offset, so that the compiler knows these for addresses of shared memory)
  uint8_t* loads = expert_raw + (-smem_u32(expert_raw) & 1023u);
  uint8_t* leaving = loads + stage_bytes(p.num_experts);
  Control& sm = *reinterpret_cast<Control*>(leaving + kChunkBytes);
  int32_t* first = reinterpret_cast<int32_t*>(&sm + 1);  // row tiles before expert e
  const int warp = uniform(threadIdx.x >> 5), lane = (int)lane_id();
  const int E = p.num_experts, K = p.in_features, N = p.out_features;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostLoads; ++i) {
      mbar_init(&sm.loaded[i], 2);  // this block's two producers (and their bytes)
      mbar_init(&sm.used[i], 8);    // the warps of a set
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 16);  // at the even block: a set's warps of both blocks
      mbar_init(&sm.done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], 8);  // at the even block, from both
    }
    mbar_init_fence();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 36)  // for the first copies
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<const CUtensorMap*>(&maps) + (threadIdx.x - 32)) : "memory");
  __syncthreads();
  // (both blocks run before either allocates: the allocation works in both; the
  // fence behind the barriers' initialisation is what orders them for the other)
  cluster_meet();
  if (warp == 1) tmem_alloc(&sm.tmem, kTmemColumns);
  pdl_wait();
  pdl_trigger();
  auto rows_of = [&](int e, int& lo) {
    lo = max(p.row_begin[e], 0);
    return max((int)min((int64_t)max(p.row_end[e], 0), p.rows) - lo, 0);
  };
  if (warp == 0) {
    int carry = 0, width = 32;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int lo;
      const int rows = e < E ? rows_of(e, lo) : 0, n = row_tiles(rows, kTileN);
      if (n > 0) width = max(width, row_tile_width(rows, n));
      const int inc = warp_inclusive_scan(n);
      if (e < E) first[e] = carry + inc - n;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    width = __reduce_max_sync(0xffffffffu, width);
    if (lane == 0) {
      first[E] = carry;
      sm.width = width;
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)sm.tmem);
  // Tensor memory: two accumulators as wide as the widest tile, and in the rest
  // as many stages of features as there is room for, 2 (192 rows) to 7 (32).
  const uint32_t acc_columns = (uint32_t)uniform(sm.width), stages = (kTmemColumns - 2 * acc_columns) / kStageColumns;
  // Shared memory: stages of rows for that width, and in the rest as many loads
  // as there is room for: the fewer rows, the more weights are under way.
  const uint32_t row_bytes = acc_columns * kLoadK;  // a load's rows as f16: two steps, one behind the other
  const uint32_t load_bytes = kBytesA + acc_columns / 2 * kLoadK;
  const uint32_t num_stages = min((stage_bytes(E) - kRowStages * row_bytes) / load_bytes, (uint32_t)kMostLoads);
  const uint32_t loads_mem = smem_u32(loads), rows_mem = loads_mem + num_stages * load_bytes;
  const uint32_t tmem_features = tmem + 2 * acc_columns;

  // Tiles in order: expert, then features, then rows; pairs take one each in
  // turn, each second round in the other direction (as the bf16 products do).
  const int turn = 2 * (pairs - pair) - 1;
  const int tile_features = GLU ? kTileM / 2 : kTileM;
  const int across = (N + tile_features - 1) / tile_features;
  const int num_tiles = uniform(first[E]) * across;
  const int num_loads = (K + kLoadK - 1) / kLoadK;                                // of every tile
  const bool short_end = K - (num_loads - 1) * kLoadK <= kStepK;                  // the last load is one step
  // The t-th tile; o is this warp's tile before, or has e = -1. (A lane looks at
  // one of the next 32 experts: one by one, 248 without rows before eight with 8
  // rows each took 8 of 36 us.)
  auto find = [&](int t, Tile& o) {
    const int before = o.e;
    o.e = max(o.e, 0);
    for (;; o.e += 32) {
      const unsigned has = __ballot_sync(0xffffffffu, o.e + lane < E && t < first[min(o.e + lane, E - 1) + 1] * across);
      if (has) {
        o.e += __ffs((int)has) - 1;
        break;
      }
    }
    if (o.e != before) {
      int lo;
      o.rows = uniform(rows_of(o.e, lo));
      o.lo = uniform(lo);
    }
    const int begin = uniform(first[o.e]), many = uniform(first[o.e + 1]) - begin;
    const int i = t - begin * across;
    o.f0 = i / many * tile_features;
    const int width = row_tile_width(o.rows, many);
    o.n0 = i % many * width;
    o.n = min(width, (max(o.rows - o.n0, 0) + 31) / 32 * 32);
  };
  Tile o;
  o.e = -1;
  bool ok = true;

  if (warp == 0 || warp == 2) {  // this block's features, and its rows, into shared memory
    const bool second = warp == 2;
    const uint32_t on = elect_one();
    uint32_t st = 0, phase = 1;  // a fresh barrier's phase before the first counts as complete
    uint32_t filled = 0;         // stages filled so far, up to all
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      if (o.n <= 0) continue;
      const int half = o.n / 2;
      // the boxes of this block's half: 16 << i rows each, the larger first
      const int sizes = half / 16;  // 1 to 6
      const uint32_t bytes = second ? (uint32_t)half * kLoadK : kBytesA;
      const int big = 31 - __clz(sizes), small = sizes & ~(1 << big);
      const CUtensorMap *map = &maps.b[big], *map2 = &maps.b[small ? 31 - __clz(small) : 0];
      const int feature = o.f0 + (int)rank * kHalfM;
      const int row = o.lo + o.n0 + (int)rank * half;
      for (int k0 = 0; k0 < K; k0 += kLoadK) {
        if (!waits(&sm.used[st], phase, wait_ns)) {
          ok = false;
          break;
        }
        uint8_t* to = loads + st * load_bytes + (second ? kBytesA : 0);
        const uint32_t bar = smem_u32(&sm.loaded[st]);
        arrive_expect_at(bar, bytes, on);
        if (second) {
          tma_load_2d(to, map, k0, row, bar, on);
          if (small) tma_load_2d(to + (16 << big) * kLoadK, map2, k0, row + (16 << big), bar, on);
        } else if (GLU) {
          // 8 features of gate, the same 8 of up, and so on
          tma_load_5d(to, &maps.a, k0, 0, 0, o.f0 / 8 + (int)rank * 8, o.e, bar, on);
        } else {
          tma_load_3d(to, &maps.a, k0, feature, o.e, bar, on);
        }
        if (++st == num_stages) {
          st = 0;
          phase ^= 1u;
        }
        filled = min(filled + 1, num_stages);
      }
    }
    if (!ok && on) g_expert_i8_status = MOE_ERR_TIMEOUT;
    // No copy may land after the block has exited, whoever gave up: wait for
    // those of the stages filled last (two milliseconds at most each, where the
    // other producer has not filled its part).
    for (; filled > 0; --filled) {
      if (st == 0) phase ^= 1u;
      st = st == 0 ? num_stages - 1 : st - 1;
      mbar_wait(&sm.loaded[st], phase ^ 1u, 2000000ull);
    }
  } else if (warp >= 4 && warp < 12) {  // features, 8 bits to f16
    const int quarter = warp & 3, set = (warp - 4) >> 2;
    const uint32_t on = elect_one();
    const uint32_t full0 = in_block(&sm.full[0], 0);
    const uint32_t to = tmem_features + (uint32_t)(quarter * 32) * 65536u;
    // lane = feature; its 16-byte pieces lie where the swizzle put them
    const uint32_t from0 = loads_mem + (uint32_t)((quarter * 32 + lane) * kLoadK + ((lane & 7) << 4));
    uint32_t j = set, tiles_end = 0;  // this set's next load, the loads of all tiles so far
    uint32_t fs = set;                // its stage of features
    uint32_t st = set, phase = 0;     // and of what is loaded
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      if (o.n <= 0) continue;
      for (tiles_end += num_loads; j < tiles_end; j += 2) {
        const uint32_t before = j - stages;  // the load that had the stage of features
        if (!(ok = waits(&sm.loaded[st], phase, wait_ns))) break;
        const uint32_t from = from0 + st * load_bytes;
        // (behind a last load of one step are zeros, which nothing multiplies)
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) f16_of(ld_shared_v4(from ^ (uint32_t)(h * 64 + c * 16)), r + c * 8);
          if (h == 0) {
            if (j >= stages && !(ok = waits(&sm.done[before % kRing], (before / kRing) & 1, wait_ns))) break;
            tmem_fence_after();  // the products that read the stage are done
          }
          tmem_store32(to + fs * kStageColumns + h * (kStageColumns / 2), r);
        }
        if (!ok) break;
        __syncwarp();
        if (on) mbar_arrive(&sm.used[st]);
        if ((st += 2) >= num_stages) {
          st -= num_stages;
          phase ^= 1u;
        }
        tmem_store_wait();
        tmem_fence_before();
        __syncwarp();
        arrive_local_at(full0 + 8u * (j % kRing), on);
        if ((fs += 2) >= stages) fs -= stages;
      }
    }
    if (!ok && lane == 0) g_expert_i8_status = MOE_ERR_TIMEOUT;
  } else if (warp >= 12 && warp < 20) {  // rows, 8 bits to f16
    const int quarter = warp & 3, set = (warp - 12) >> 2;
    const uint32_t on = elect_one();
    const uint32_t full0 = in_block(&sm.full[0], 0);
    // eight rows x four pieces of a step at a time, each piece to two of f16:
    // this warp has each second eight rows, of one of the two steps
    const uint32_t r8 = lane & 7, piece = lane >> 3, row = (quarter >> 1) * 8 + r8, h = quarter & 1;
    const uint32_t from0 = loads_mem + kBytesA + row * kLoadK + (((4 * h + piece) ^ r8) << 4);
    const uint32_t to0 = rows_mem + h * (row_bytes / 2) + row * 128 + (((2 * piece) ^ r8) << 4);
    uint32_t j = set, tiles_end = 0;
    uint32_t st = set, phase = 0;
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      if (o.n <= 0) continue;
      for (tiles_end += num_loads; j < tiles_end; j += 2) {
        const uint32_t before = j - kRowStages;  // the load that had the stage of rows
        if (!(ok = waits(&sm.loaded[st], phase, wait_ns))) break;
        const uint32_t from = from0 + st * load_bytes, to = to0 + j % kRowStages * row_bytes;
        if (j >= kRowStages && !(ok = waits(&sm.done[before % kRing], (before / kRing) & 1, wait_ns))) break;
#pragma unroll 1
        for (int i = 0; i < o.n / 32; ++i) {
          uint32_t r[8];
          f16_of(ld_shared_v4(from + i * 16 * kLoadK), r);
          const uint32_t at = to + i * 16 * 128;
          st_shared_v4(at, r);
          st_shared_v4(at ^ 16, r + 4);
        }
        __syncwarp();
        if (on) mbar_arrive(&sm.used[st]);
        if ((st += 2) >= num_stages) {
          st -= num_stages;
          phase ^= 1u;
        }
        fence_proxy_async_smem();
        arrive_with_shared_at(full0 + 8u * (j % kRing), on);
      }
    }
    if (!ok && lane == 0) g_expert_i8_status = MOE_ERR_TIMEOUT;
  } else if (warp == 1 && rank == 0) {  // tensor cores, for both blocks
    uint32_t j = 0;               // loads multiplied
    uint32_t fs = 0;              // stage of features
    const uint32_t on = elect_one();
    int acc = 0;  // accumulators begun
    for (int t = pair, jump = turn; ok && t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      if (o.n <= 0) continue;
      const int as = acc & 1;
      if (acc >= 2 && !waits(&sm.acc_empty[as], (uint32_t)((acc / 2 + 1) & 1), wait_ns)) {
        ok = false;
        break;
      }
      const uint32_t idesc = instr_desc(false, false, false, kTileM, o.n);
      for (int l = 0; l < num_loads; ++l, ++j) {
        if (!(ok = waits<true>(&sm.full[j % kRing], (j / kRing) & 1, wait_ns))) break;
        tmem_fence_after();
        const bool end = l == num_loads - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && end && short_end) break;
          const uint64_t db = operand_desc(rows_mem + j % kRowStages * row_bytes + h * (row_bytes / 2), false);
          const uint32_t a = tmem_features + fs * kStageColumns + h * (kStageColumns / 2);
          mma_step(tmem + as * acc_columns, a, db, idesc, l > 0 || h > 0, on);
        }
        mma_commit(&sm.done[j % kRing], on);
        if (end) mma_commit(&sm.acc_full[as], on);
        if (++fs == stages) fs = 0;
      }
      ++acc;
    }
    if (!ok && lane == 0) g_expert_i8_status = MOE_ERR_TIMEOUT;
    // tensor memory is freed below: wait for the last MMAs, with the full budget
    if (j > 0) mbar_wait(&sm.done[(j - 1) % kRing], ((j - 1) / kRing) & 1);
  } else if (warp >= 20) {  // accumulators to memory: a warp reads tensor-memory lanes (warp % 4) * 32 ..
    const int quarter = warp & 3, tid = (int)threadIdx.x - 20 * 32;
    const uint32_t on = elect_one();
    const uint32_t acc_empty0 = in_block(&sm.acc_empty[0], 0);
    // Of 16 tensor-memory lanes, two halves of a warp's, this lane has features
    // g and g + 8 (of gate and up feature g each), and of each eight rows two.
    const int g = lane >> 2, pair_of = (lane & 3) * 2;
    constexpr int kPieces = GLU ? 8 : 16, kAtOnce = 128 / kPieces;  // of eight features in a row; rows stored at once
    const int piece = tid % kPieces * 8, first_row = tid / kPieces;
    const uint32_t buf = smem_u32(leaving);
    // where this lane's row of what it stores transposed begins
    const uint32_t row_of = GLU ? buf + lane * kPitch + quarter * 32
                                : buf + ((lane >> 4) * 8 + (lane & 7)) * kPitch + (quarter * 32 + (lane & 8)) * 2;
    int acc = 0;
    for (int t = pair, jump = turn; t < num_tiles; t += jump, jump = 2 * pairs - jump) {
      find(t, o);
      if (o.n <= 0) continue;
      const int as = acc & 1;
      const int own = GLU ? 64 : kHalfM;               // features of this block
      const int f = o.f0 + (int)rank * own;
      const int nf = min(max(N - f, 0), own);          // that exist, a multiple of 8
      const int valid = min(o.n, o.rows - o.n0);       // rows of the tile that the expert has
      const int64_t row0 = (int64_t)o.lo + o.n0;
      // scales, while the products run: the lane's features', and the rows'
      // (read behind the vote below)
      float sw[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = GLU ? quarter * 16 + h * 8 + g : quarter * 32 + h * 16 + i * 8 + g;  // feature of the block
          sw[h][i] = at < nf ? p.w_scales[(int64_t)o.e * (GLU ? 2 * N : N) + (GLU ? i * N : 0) + f + at] : 0.0f;
        }
      for (int i = tid; i < o.n; i += 128) sm.row_scales[as][i] = i < valid ? p.x_scales[(row0 + i) * p.x_scale_stride] : 0.0f;
      ok = epilogue_agrees(waits(&sm.acc_full[as], (uint32_t)((acc / 2) & 1), wait_ns));
      if (!ok) break;
      tmem_fence_after();
      const uint32_t src = tmem + (uint32_t)(quarter * 32) * 65536u + as * acc_columns;
      uint8_t* to = p.out + ((row0 + first_row) * N + f + piece) * 2;
#pragma unroll 1
      for (int c = 0; c < o.n; c += kChunk) {
        // features to rows through shared memory
        if (c != 0) epilogue_sync();  // the rows before have been read (the tile's before: at the vote)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[16];
          tmem_load16x32(src + (uint32_t)(h * 16) * 65536u + c, v);
          if (h == 1 && c + kChunk >= o.n) {  // the last columns have been read: the accumulator is free
            tmem_fence_before();
            __syncwarp();
            arrive_local_at(acc_empty0 + 8u * as, on);
          }
          uint32_t low[4], high[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 sx = *reinterpret_cast<const float2*>(&sm.row_scales[as][c + 8 * j + pair_of]);
            const float a0 = v[4 * j] * (sx.x * sw[h][0]), a1 = v[4 * j + 1] * (sx.y * sw[h][0]);
            const float b0 = v[4 * j + 2] * (sx.x * sw[h][1]), b1 = v[4 * j + 3] * (sx.y * sw[h][1]);
            if (GLU) {
              low[j] = pack_bf16x2_rn(swiglu_of(a0, b0), swiglu_of(a1, b1));
            } else {
              low[j] = pack_bf16x2_rn(a0, a1);
              high[j] = pack_bf16x2_rn(b0, b1);
            }
          }
          if (GLU) {
            store_transposed(row_of + h * 16, low[0], low[1], low[2], low[3]);
          } else {
            store_transposed(row_of + h * 32, low[0], high[0], low[1], high[1]);
            store_transposed(row_of + h * 32 + 16 * kPitch, low[2], high[2], low[3], high[3]);
          }
        }
        epilogue_sync();
#pragma unroll
        for (int j = 0; j < kChunk / kAtOnce; ++j) {
          const int r = c + j * kAtOnce + first_row;
          if (r < valid && piece < nf)
            st_v4(to + (int64_t)(c + j * kAtOnce) * N * 2, ld_shared_v4(buf + (j * kAtOnce + first_row) * kPitch + piece * 2));
        }
      }
      ++acc;
    }
    if (!ok && lane == 0) g_expert_i8_status = MOE_ERR_TIMEOUT;
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  if (warp == 1) tmem_free(tmem, kTmemColumns);
  __syncwarp();
  cluster_meet();  // and neither leaves before both have freed theirs
}

// int8 in boxes of 128 bytes x `rows`; what lies outside reads as zero.
bool make_map(CUtensorMap* map, const void* base, int dims, const cuuint64_t* size, const cuuint64_t* strides,
              const cuuint32_t* box) {
  const EncodeTiled fn = encode_tiled();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<void*>(base), size, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pairs that can be resident at once on the current device, looked up once
// per device and kernel.
template <bool GLU>
int resident_pairs(int dev, int sms) {
  static std::once_flag once[64];
  static int found[64];
  if (dev >= 64) return 0;
  std::call_once(once[dev], [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSharedBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (const void*)k_expert_i8<GLU>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    found[dev] = n;
  });
  return found[dev];
}

template <bool GLU>
cudaError_t launch(const ExpertI8Params& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
  const cuuint64_t K = (cuuint64_t)p.in_features, N = (cuuint64_t)p.out_features, E = (cuuint64_t)p.num_experts;
  Maps maps;
  bool ok;
  if (GLU) {
    // w [E][2F][K] as [E][F / 8][gate, up][8][K], in boxes of 64 gate features,
    // 8 by 8 in turn with their up features
    const cuuint64_t size[5] = {K, 8, 2, N / 8, E}, strides[4] = {K, N * K, 8 * K, 2 * N * K};
    const cuuint32_t box[5] = {kLoadK, 8, 2, 8, 1};
    ok = make_map(&maps.a, p.w, 5, size, strides, box);
  } else {
    const cuuint64_t size[3] = {K, N, E}, strides[2] = {K, N * K};
    const cuuint32_t box[3] = {kLoadK, kHalfM, 1};
    ok = make_map(&maps.a, p.w, 3, size, strides, box);
  }
  for (int i = 0; i < 3; ++i) {
    const cuuint64_t size[2] = {K, (cuuint64_t)p.rows}, strides[1] = {(cuuint64_t)p.x_stride};
    const cuuint32_t box[2] = {kLoadK, 16u << i};
    ok = ok && make_map(&maps.b[i], p.x, 2, size, strides, box);
  }
  if (!ok) return cudaErrorUnknown;
  const void* fn = (const void*)k_expert_i8<GLU>;
  cudaError_t err = ensure_dynamic_smem(fn, kSharedBytes);
  if (err != cudaSuccess) return err;
  const int64_t pairs = resident_pairs<GLU>(dev, sms);
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  // the row counts are on the device: as many pairs as there can be tiles
  const int64_t width = GLU ? kTileM / 2 : kTileM, across = (p.out_features + width - 1) / width;
  const int64_t most = across * (p.num_experts + p.rows / kTileN);
  ExpertI8Params q = p;
  uint64_t wait_ns = wait_limit_ns();
  void* args[] = {&q, &maps, &wait_ns};
  return launch_pdl(fn, dim3((unsigned)(2 * (most < pairs ? most : pairs))), dim3(kThreads), kSharedBytes, s,
                    args, 2);
}

// A few rows go to a kernel that streams the weights, if there are no more than
// some two for each expert on average: it takes two at a time and reads the
// weights again (from L2) for more, and tiles take the same time for 1 to 32. What
// counts is how many rows the buffers have: the counts of each expert are on the
// device, so 16 rows of one expert among many are streamed, and a few rows in
// large buffers are not. (First product 7168 -> 2 x 2048, tiles /
// streamed: 1 row 25 / 7 us, 4 rows of one expert 24 / 12, 8 24 / 19, 16 24 / 35; 8
// rows in 8 experts 48 / 37, 16 in 16 86 / 74, in 8 48 / 38; 32 in 32 145 / 134, in
// 8 48 / 70. Second product: 8 rows of one expert 10 / 11 us.)
bool few(const ExpertI8Params& p) { return p.rows <= kFewRows && p.rows <= 2 * (int64_t)p.num_experts + 4; }

}  // namespace

int read_expert_i8_status(int32_t* out, bool clear) {
  int32_t v = 0;
  const int32_t zero = MOE_OK;
  if (cudaMemcpyFromSymbol(&v, g_expert_i8_status, 4) != cudaSuccess ||
      (clear && cudaMemcpyToSymbol(g_expert_i8_status, &zero, 4) != cudaSuccess)) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  *out = v;
  return MOE_OK;
}

cudaError_t launch_expert_product_i8(const ExpertI8Params& p, cudaStream_t s) {
  return few(p) ? launch_expert_i8_few(p, false, s) : launch<false>(p, s);
}
cudaError_t launch_expert_swiglu_i8(const ExpertI8Params& p, cudaStream_t s) {
  return few(p) ? launch_expert_i8_few(p, true, s) : launch<true>(p, s);
}

}  // namespace moe
