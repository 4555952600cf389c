// attention, forward: bfloat16
#include "attn_fwd.hpp"

namespace lowbit {

lowbit_status launch_attn_bf16(const AttnArgs& a, hipStream_t s) { return launch_attn<kBF16>(a, s); }

}  // namespace lowbit
