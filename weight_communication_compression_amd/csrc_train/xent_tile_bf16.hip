// linear xent: the products of bfloat16
#include "xent_tile.hpp"

namespace lowbit {

lowbit_status launch_xent_tile_bf16(int form, int kind, const XentTileArgs& g, hipStream_t s) {
  switch (form) {
    case 0: return launch_form<Form<kBF16, 256, 256, 2, 4, kXentForms[0].slots>>(kind, g, s);
    case 1: return launch_form<Form<kBF16, 128, 128, 2, 2, kXentForms[1].slots>>(kind, g, s);
    case 2: return launch_form<Form<kBF16, 64, 128, 1, 4, kXentForms[2].slots>>(kind, g, s);
    default: return launch_form<Form<kBF16, 32, 128, 1, 4, kXentForms[3].slots>>(kind, g, s);
  }
}

}  // namespace lowbit
