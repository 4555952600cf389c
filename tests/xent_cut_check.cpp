// The units of a product, as the tile kernels take them: for test_xent_cut_host.py.
#include "../weight_communication_compression_amd/csrc_train/xent_cut.hpp"

using namespace lowbit;

// 0 where the units of a product of m x n (at most most_m rows) over k_steps take
// every step of every tile once and the parts fit the room for them.
extern "C" int check(int form, int kind, int64_t m, int64_t most_m, int64_t n, uint32_t k_steps,
                     uint32_t most_steps, unsigned char* seen, int64_t seen_size) {
  const XentForm& f = kXentForms[form];
  const XentCut cut(m, n, k_steps, f.tm, f.tn, f.slots,
                    xent_may_cut(f, kind, most_m, n, most_steps));
  if ((int64_t)cut.rest * cut.parts * (cut.parts > 1) > xent_slots(f, kind, most_m, n, most_steps)) return 1;
  if (cut.whole + cut.rest != cut.tiles || cut.tiles != cut.across * cut.down) return 2;
  if ((int64_t)cut.tiles * k_steps > seen_size) return 3;
  for (uint32_t u = 0; u < cut.units(); ++u) {
    const XentUnit v = cut.unit(u, k_steps);
    if (v.tile >= cut.tiles || v.tm >= cut.down || v.tn >= cut.across) return 4;
    if (v.slot >= (int)(cut.rest * cut.parts) || (v.slot < 0) != (u < cut.whole)) return 5;
    if (v.slot >= 0 && v.tile != cut.whole + v.slot % cut.rest) return 6;
    const int64_t at = ((int64_t)v.tm * cut.across + v.tn) * k_steps;
    for (int s = v.s0; s < v.s1; ++s) {
      if (s < 0 || s >= (int)k_steps || seen[at + s]++) return 7;
    }
  }
  for (int64_t i = 0; i < (int64_t)cut.tiles * k_steps; ++i)
    if (seen[i] != 1) return 8;
  return 0;
}
