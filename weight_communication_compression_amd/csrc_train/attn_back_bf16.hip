// attention's gradient: bfloat16
#include "attn_back.hpp"

namespace lowbit {

lowbit_status launch_attn_back_bf16(const AttnArgs& a, hipStream_t s) {
  return launch_attn_back<kBF16>(a, s);
}

}  // namespace lowbit
