// How the absorbed form's units are dealt to the workgroups (see
// latent_attend.hip): a workgroup's share, from where the sequences start in the
// numbering of units or pieces. Nothing of HIP is used here, so that a host
// compiler takes it too.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define LATENT_HD __host__ __device__ inline
#else
#define LATENT_HD inline
#endif

struct alignas(32) WgDesc {
  int b, mt, at, n;       // first unit: sequence, row tile, place in the row tile's units; number of units
  int t0, nq, len, over;  // the sequence's bounds; units a row tile has ahead of its cache tiles
};
struct TileDesc {
  int b, mt, w0, n;  // a row tile whose cache tiles n workgroups share: w0, w0 + step, ..
  int step;
  int64_t u0;        // its first unit
};

// x >= 0 by y > 0, rounded up; 64-bit division is slow, and rarely needed
LATENT_HD int64_t latent_div_up(int64_t x, int64_t y) {
  return x + y < (1ll << 31) ? (int64_t)(((uint32_t)x + (uint32_t)y - 1) / (uint32_t)y) : (x + y - 1) / y;
}

LATENT_HD int latent_last_at_or_below(const int64_t *cum, int n, int64_t v) {  // cum ascending, cum[0] <= v: the last such i
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// Workgroup w's share, of units or pieces [v, ..) of all, v = w per < all, in
// sequence b, which starts at start and has `rows` row tiles of k cache tiles:
// d.mt, at, n, and *t (else left as it is) where w is the one that names a row
// tile that several share. piece: cache tiles of a piece at most, or 0 for even
// runs of `per` units, each row tile with `over` units ahead of its cache tiles.
// A sequence may have more than 2^31 units (2^18 tokens of 128 heads over 2^19
// rows); per is below 2^31.
LATENT_HD void latent_share(int w, int64_t v, int64_t all, int64_t per, int piece, int over, int b, int64_t start,
                            int rows, int k, WgDesc *d, TileDesc *t) {
  const int64_t r = v - start;
  if (piece) {  // at most a piece a workgroup
    // piece i of c of row tile mt; a piece's row tiles are neighbours, which read the same cache rows
    const int c = (k + piece - 1) / piece, i = (int)((uint32_t)r / (uint32_t)rows);
    d->mt = (int)((uint32_t)r % (uint32_t)rows);
    d->at = i * (k / c) + (i < k % c ? i : k % c);
    d->n = k / c + (i < k % c ? 1 : 0);
    if (i == 0 && c > 1) *t = TileDesc{b, d->mt, w, c, rows, 0};
    return;
  }
  const int units = k + over;  // of a row tile
  if (r >> 31) {
    d->mt = (int)(r / units);
    d->at = (int)(r % units);
  } else {
    d->mt = (int)((uint32_t)r / (uint32_t)units);
    d->at = (int)((uint32_t)r % (uint32_t)units);
  }
  d->n = (int)(per < all - v ? per : all - v);
  // shared with the workgroups before, and the first boundary in this row tile
  const int64_t u0 = v - d->at;
  const int first = (int)((u0 + over) / per);
  if (d->at > over && first == w - 1)
    *t = TileDesc{b, d->mt, first, (int)((u0 + over + k - 1) / per) - first + 1, 1, u0};
}
