// How the tiles of dW are dealt out where single CTAs take runs of them
// (host only, no CUDA).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bb {

// Cuts dW's wm * dn tiles (dn columns of tiles, cols blocks of 64 columns;
// ordered by columns first) into one run per worker: worker w takes the tiles
// start[w] .. start[w + 1] - 1.  A tile costs its 64-column blocks and one
// for itself.  dh_tiles tiles of dh at ch K steps each (a full tile of dW: cw)
// were dealt out before, one by one; the workers that got one fewer take as
// much more of dW.  In integers: every worker's end is the next one's start.
inline void dw_runs(int wm, int dn, int cols, long long dh_tiles, int ch, int cw, int workers,
                    int* start) {
  const long long more = dh_tiles % workers, fewer = workers - more;
  const int64_t all = (int64_t)wm * (cols + dn) * cw;  // in units of 1 / cw
  const int64_t d = more ? 5ll * ch : 0;
  // Shares x for the first `more` workers, x + d for the others, in units of
  // 1 / unit; none below 0.
  int64_t unit = (int64_t)workers * cw, x = all - d * fewer, y = x + d * workers;
  if (x < 0) {
    unit = fewer * cw;
    x = 0;
    y = all;
  }
  for (int w = 0; w < workers; ++w) {
    const int64_t b = std::min<int64_t>(w, more) * x + std::max<int64_t>(w - more, 0) * y;
    const int64_t column = 5ll * wm * unit;
    const int n = (int)std::min<int64_t>(b / column, dn - 1);
    const int64_t tile = (std::min(4, cols - 4 * n) + 1) * unit;
    const int64_t m = (b - n * column + tile / 2) / tile;
    start[w] = n * wm + (int)std::min<int64_t>(m, wm);
  }
  start[workers] = wm * dn;
}

}  // namespace bb
