// ortho_choice.hpp -- which form of the tile kernel a product of orthogonalize takes,
// whether it is cut along k, and where its tiles lie.  Integer and float arithmetic with no HIP dependency, for the
// launches, the workspace and a CPU test.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __HIPCC__
#define LOWBIT_HD __host__ __device__
#else
#define LOWBIT_HD
#endif

namespace lowbit {

// The forms: rows and columns of a tile; microseconds of a step of 64 of k where a CU has one
// tile (all CUs busy), of a step of one tile where it has several, and of a launch with its
// ends.  Measured in every form at 10 sizes from 256 x 1024 to 2048 x 8192; the choice is the
// fastest or within 15 % of it at each (A of 1024 x 4096: 64 17 us, 128 30, 192 55, 256 76; of
// 4096 x 4096: 130, 108, 80, 105).
struct OrthoForm {
  int tile;
  float lone, shared, base;
};
constexpr int kOrthoForms = 5;
constexpr OrthoForm kOrthoForm[kOrthoForms] = {
    {256, 1.60f, 1.60f, 9.0f},   // eight waves, two stages
    {192, 1.15f, 1.20f, 7.0f},   // four waves of 96 x 96; only of mirrored products
    {128, 0.85f, 0.60f, 6.0f},   // four waves, two stages, two workgroups a CU
    {128, 0.67f, 0.75f, 6.0f},   // eight waves, four stages
    {64, 0.27f, 0.25f, 4.5f},    // four waves, four stages, two workgroups a CU
};

struct OrthoChoice {
  int form, parts;
  int64_t tiles;
};

inline float ortho_cost(int form, int parts, int64_t tiles, int64_t steps) {
  const OrthoForm& f = kOrthoForm[form];
  const int64_t each = (tiles * parts + 255) / 256, run = (steps + parts - 1) / parts;
  const float step = each > 1 ? each * f.shared > f.lone ? each * f.shared : f.lone : f.lone;
  const float add = parts > 1 ? 6.0f + (float)tiles * parts * f.tile * f.tile * 8.0f / 4.0e6f : 0.0f;
  return f.base + run * step + add;
}

// The cheapest form for a product with m rows: of A A^T kinds (mirrored, of their tiles only
// those on and below the diagonal) with k = n (gram) or m, else m x n with k = m.
inline OrthoChoice ortho_choice(bool mirrored, bool gram, int64_t batch, int64_t m, int64_t n) {
  const int64_t steps = ((gram ? n : m) + 63) / 64;
  OrthoChoice best{-1, 1, 0};
  float least = 0.0f;
  for (int f = 0; f < kOrthoForms; ++f) {
    if (f == 1 && !mirrored) continue;
    const int64_t t = kOrthoForm[f].tile, down = (m + t - 1) / t;
    const int64_t tiles = batch * (mirrored ? down * (down + 1) / 2 : down * ((n + t - 1) / t));
    for (int parts = 1; parts <= 16; parts *= 2) {
      // (a part has 8 steps at least, and never more parts than there are CUs)
      if (parts > 1 && (steps / parts < 8 || tiles * parts > 256)) break;
      const float cost = ortho_cost(f, parts, tiles, steps);
      if (best.form < 0 || cost < least) {
        best = {f, parts, tiles};
        least = cost;
      }
    }
  }
  return best;
}

// Where a tile lies.  Tiles are counted in bands of 8 rows of tiles (4 of a mirrored product, of
// which only those on and below the diagonal count), down a band's columns: the 32 that an XCD's
// CUs hold at one time then share the panels that they read through its L2.
struct OrthoPlace {
  int tm, tn;
};
inline LOWBIT_HD OrthoPlace ortho_place(bool mirrored, int tile, int across, int down) {
  if (!mirrored) {
    const int band = tile / (8 * across), in = tile % (8 * across);
    const int high = down - band * 8 < 8 ? down - band * 8 : 8;
    return {band * 8 + in % high, in / high};
  }
  // band b begins at tile b (8 b + 2): rows 0 .. 4 b - 1 have 1, 2, ... tiles
  int b = (int)sqrtf((float)tile * 0.125f);
  while ((b + 1) * (8 * (b + 1) + 2) <= tile) ++b;
  while (b * (8 * b + 2) > tile) --b;
  const int high = down - 4 * b < 4 ? down - 4 * b : 4, whole = 4 * b + 1;
  int in = tile - b * (8 * b + 2);
  if (in < high * whole) return {4 * b + in % high, in / high};
  in -= high * whole;                              // beyond the band's first diagonal tile
  int j = 1;
  while (in >= high - j) in -= high - j++;
  return {4 * b + j + in, 4 * b + j};
}
// Unit u is a workgroup's of XCD u mod 8, of which each takes a contiguous run.
inline LOWBIT_HD int64_t ortho_run(int64_t u, int64_t count) {
  const int64_t x = u % 8, each = count / 8, more = count % 8;
  return x * each + (x < more ? x : more) + u / 8;
}

// Bytes for the parts' sums of a product.
inline int64_t ortho_part_bytes(const OrthoChoice& c) {
  const int64_t t = kOrthoForm[c.form].tile;
  return c.parts > 1 ? c.tiles * c.parts * t * t * 4 : 0;
}

}  // namespace lowbit
