// row_tiles.h -- how the experts' products cut an expert's rows into tiles.
// Plain C++ besides CUDA, so that host code can check it.
#pragma once

#ifdef __CUDACC__
#define MOE_ROW_TILES __host__ __device__ __forceinline__
#else
#define MOE_ROW_TILES inline
#endif

namespace moe {

// Row tiles of an expert: as few of at most `most` rows (a multiple of 32) as
// hold its rows, of equal width in steps of 32; the last is as wide as what is
// left. Up to 2^31 - 129 rows come, so no sum may add to them: the quotients are
// rounded up behind the division. The last tile begins below `rows`, or there
// are so few tiles that its first row is far from 2^31 all the same.
MOE_ROW_TILES int row_tiles(int rows, int most) { return rows / most + (rows % most > 0 ? 1 : 0); }
// (of at least one tile, so of at least one row)
MOE_ROW_TILES int row_tile_width(int rows, int tiles) { return ((rows - 1) / tiles / 32 + 1) * 32; }

}  // namespace moe
