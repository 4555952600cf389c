// xent_cut.hpp -- which tiles of a product are cut along k, and who takes what.
// Integer code with no HIP dependency, for the kernels, the C ABI and a CPU test.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define LOWBIT_HD __host__ __device__
#else
#define LOWBIT_HD
#endif

namespace lowbit {

// A product of the loss: C[m, n] = sum_k A[m, k] B[n, k].
enum XentKind : int {
  kXentStats = 0,            // logits -> parts of the softmax
  kXentProb = 1,             // logits -> d, a piece of the vocabulary
  kXentDx = 2,               // dx += d w
  kXentDw = 3,               // dw = d^T x
};

// The tile kernels' forms: rows and columns of a tile, and how many of its
// workgroups the chip holds at one time.
struct XentForm {
  int tm, tn, slots;
};
constexpr XentForm kXentForms[4] = {{256, 256, 256}, {128, 128, 512}, {64, 128, 768}, {32, 128, 1024}};
constexpr int kXentRowBytes = 128;         // of k, in a step

inline LOWBIT_HD uint32_t xent_steps(int64_t k, int elem_size) {
  return (uint32_t)((k * elem_size + kXentRowBytes - 1) / kXentRowBytes);
}

// Whether a product of up to m rows (dw: k_steps) may cut tiles along k: not where
// the second kernel would take longer than the steps it saves, and the loss only
// where there are fewer tiles than slots: with more its workspace would grow by
// 64 MiB for what saves least, half a round of many.
inline bool xent_may_cut(const XentForm& f, int kind, int64_t m, int64_t n, uint32_t k_steps) {
  const int64_t tiles = (m + f.tm - 1) / f.tm * ((n + f.tn - 1) / f.tn);
  return kind == kXentStats  ? k_steps >= 24 && tiles < f.slots
         : kind == kXentProb ? k_steps >= 32
                             : k_steps >= 8;
}

// What one workgroup takes at a time: a tile, or a part of one (slot >= 0), and
// its steps of k.
struct XentUnit {
  uint32_t tile, tm, tn;
  int slot, s0, s1;
};

// The workgroups that the chip holds at one time (slots) take whole tiles as
// long as all of them have one; the remaining tiles are cut into as many parts
// as there are slots for them, of four steps of k at least, and the parts' sums
// are added by a second kernel.  Two rounds instead of one and a half would
// leave half of the chip idle in the second.
struct XentCut {
  uint32_t across, down, tiles, whole;           // whole: tiles that are not cut
  uint32_t rest, parts;                          // tiles that are, each into `parts`
  LOWBIT_HD XentCut(int64_t m, int64_t n, uint32_t k_steps, uint32_t tm, uint32_t tn,
                    uint32_t slots, bool may_cut) {
    across = ((uint32_t)n + tn - 1) / tn;
    down = ((uint32_t)m + tm - 1) / tm;
    tiles = across * down;
    rest = tiles % slots;
    parts = rest && may_cut ? slots / rest : 1;
    if (parts > k_steps / 4) parts = k_steps / 4;
    if (parts <= 1) {
      parts = 1;
      rest = 0;
    }
    whole = tiles - rest;
  }
  LOWBIT_HD uint32_t units() const { return whole + rest * parts; }
  // Tiles lie in bands of 8 rows of tiles: the 32 that an XCD's CUs hold at one
  // time read 8 panels of a and 4 of b through its L2.
  LOWBIT_HD void place(uint32_t tile, uint32_t& tm, uint32_t& tn) const {
    const uint32_t band = tile / (8 * across), in = tile % (8 * across);
    const uint32_t high = down - band * 8 < 8 ? down - band * 8 : 8;
    tm = band * 8 + in % high;
    tn = in / high;
  }
  // Unit u is a workgroup's of XCD u mod 8, of which each takes a contiguous run.
  static LOWBIT_HD uint32_t run(uint32_t u, uint32_t count) {
    const uint32_t x = u % 8, each = count / 8, more = count % 8;
    return x * each + (x < more ? x : more) + u / 8;
  }
  LOWBIT_HD XentUnit unit(uint32_t u, uint32_t k_steps) const {
    XentUnit v;
    v.slot = -1;
    v.s0 = 0;
    v.s1 = (int)k_steps;
    if (u < whole) {
      v.tile = run(u, whole);
    } else {
      const uint32_t slot = run(u - whole, rest * parts), part = slot / rest;
      const uint32_t each = k_steps / parts, more = k_steps % parts;
      v.slot = (int)slot;
      v.tile = whole + slot % rest;
      v.s0 = (int)(each * part + (part < more ? part : more));
      v.s1 = v.s0 + (int)(each + (part < more ? 1 : 0));
    }
    place(v.tile, v.tm, v.tn);
    return v;
  }
};

// How many parts' sums a product needs room for, of tm x tn values each, where
// up to m rows count and k is at most k_steps.
inline int64_t xent_slots(const XentForm& f, int kind, int64_t m, int64_t n, uint32_t k_steps) {
  if (!xent_may_cut(f, kind, m, n, k_steps)) return 0;
  const int64_t quarter = k_steps / 4;
  const int64_t tiles = (m + f.tm - 1) / f.tm * ((n + f.tn - 1) / f.tn);
  return tiles < f.slots && tiles * quarter < f.slots ? tiles * quarter : f.slots;
}

}  // namespace lowbit
