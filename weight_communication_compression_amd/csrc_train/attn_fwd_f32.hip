// attention, forward: binary32
#include "attn_fwd.hpp"

namespace lowbit {

lowbit_status launch_attn_f32(const AttnArgs& a, hipStream_t s) { return launch_attn<kF32>(a, s); }

}  // namespace lowbit
