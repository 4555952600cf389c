// attention's gradient: binary32
#include "attn_back.hpp"

namespace lowbit {

lowbit_status launch_attn_back_f32(const AttnArgs& a, hipStream_t s) {
  return launch_attn_back<kF32>(a, s);
}

}  // namespace lowbit
