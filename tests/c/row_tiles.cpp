// row_tiles MOST ROWS...: for each count of rows the tiles of at most MOST that
// it is cut into and their width, one line each.
#include <cstdio>
#include <cstdlib>

#include "row_tiles.h"

int main(int argc, char** argv) {
  if (argc < 2) return 1;
  const int most = std::atoi(argv[1]);
  for (int i = 2; i < argc; ++i) {
    const int rows = std::atoi(argv[i]), tiles = moe::row_tiles(rows, most);
    std::printf("%d %d\n", tiles, tiles ? moe::row_tile_width(rows, tiles) : 0);
  }
  return 0;
}
