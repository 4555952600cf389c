// Checks of ortho_choice.hpp: every tile of a product is placed once, every unit is run once,
// and a choice's parts fit what they are cut from.
#include <cstdio>
#include <set>
#include <utility>

#include "../weight_communication_compression_amd/csrc_train/ortho_choice.hpp"

using namespace lowbit;

static int bad(const char* what, long a, long b, long c) {
  std::printf("%s: %ld %ld %ld\n", what, a, b, c);
  return 1;
}

int main() {
  for (int down = 1; down <= 70; ++down) {
    std::set<std::pair<int, int>> seen;
    const int tiles = down * (down + 1) / 2;
    for (int t = 0; t < tiles; ++t) {
      const OrthoPlace p = ortho_place(true, t, down, down);
      if (p.tm < 0 || p.tm >= down || p.tn < 0 || p.tn > p.tm) return bad("mirrored", down, t, 0);
      seen.insert({p.tm, p.tn});
    }
    if ((int)seen.size() != tiles) return bad("mirrored twice", down, tiles, 0);
  }
  // the largest: 65536 rows in tiles of 64
  for (int t = 1024 * 1025 / 2 - 1, n = 0; n < 5000; ++n, --t) {
    const OrthoPlace p = ortho_place(true, t, 1024, 1024);
    if (p.tm < 0 || p.tm >= 1024 || p.tn < 0 || p.tn > p.tm) return bad("large", t, p.tm, p.tn);
  }
  for (int down = 1; down <= 20; ++down)
    for (int across = 1; across <= 20; ++across) {
      std::set<std::pair<int, int>> seen;
      for (int t = 0; t < down * across; ++t) {
        const OrthoPlace p = ortho_place(false, t, across, down);
        if (p.tm < 0 || p.tm >= down || p.tn < 0 || p.tn >= across) return bad("place", down, across, t);
        seen.insert({p.tm, p.tn});
      }
      if ((int)seen.size() != down * across) return bad("place twice", down, across, 0);
    }
  for (int64_t count = 1; count <= 300; ++count) {
    std::set<int64_t> seen;
    for (int64_t u = 0; u < count; ++u) {
      const int64_t r = ortho_run(u, count);
      if (r < 0 || r >= count) return bad("run", count, u, r);
      seen.insert(r);
    }
    if ((int64_t)seen.size() != count) return bad("run twice", count, 0, 0);
  }
  const int64_t sizes[] = {1, 2, 63, 64, 65, 128, 129, 200, 500, 1031, 2048, 4096, 9000, 65536};
  for (int64_t batch : {1, 3, 100})
    for (int64_t m : sizes)
      for (int64_t n : sizes) {
        if (n < m) continue;
        for (int kind = 0; kind < 3; ++kind) {
          const OrthoChoice c = ortho_choice(kind < 2, kind == 0, batch, m, n);
          const int64_t steps = ((kind == 0 ? n : m) + 63) / 64, t = kOrthoForm[c.form].tile;
          const int64_t down = (m + t - 1) / t, across = (n + t - 1) / t;
          const int64_t tiles = batch * (kind < 2 ? down * (down + 1) / 2 : down * across);
          if (c.form < 0 || c.form >= kOrthoForms || (c.form == 1 && kind == 2)) return bad("form", m, n, kind);
          if (c.tiles != tiles) return bad("tiles", m, n, kind);
          if (c.parts < 1 || c.parts > 16 || (c.parts > 1 && (steps / c.parts < 8 || tiles * c.parts > 256)))
            return bad("parts", m, n, kind);
          if (ortho_part_bytes(c) != (c.parts > 1 ? tiles * c.parts * t * t * 4 : 0)) return bad("bytes", m, n, kind);
        }
      }
  std::puts("ok");
  return 0;
}
