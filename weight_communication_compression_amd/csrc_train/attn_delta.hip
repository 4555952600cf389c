// attn_delta.hip -- what attention's gradient needs of each query row.
#include "attn.hpp"

namespace lowbit {

namespace {

// lse in the kernels' units (0 where a row sees nothing: every weight is exp(-infinity)
// then) and -D, D being the sum of dout out: 16 lanes a row of a head, all heads of a row in turn.
// Bound by memory: 8 Ki x 32 heads of 128 bfloat16 28 us, 4.8 TB/s.
template <int DT>
__global__ void __launch_bounds__(256) attn_delta_kernel(AttnArgs g) {
  const int lane = threadIdx.x % 16;
  const int64_t pairs = (int64_t)g.q_rows * g.q_heads;
  for (int64_t u = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; u < pairs; u += (int64_t)gridDim.x * 16) {
    const int64_t row = u / g.q_heads;
    const int head = (int)(u - row * g.q_heads);
    float sum = 0.0f;
    if (lane * 8 < g.head_dim) {
      const Raw8<DT> a = load8<DT>(static_cast<const char*>(g.dout.p) + row * g.dout.row +
                                       head * g.dout.head, lane * 8, g.head_dim);
      const Raw8<DT> b = load8<DT>(static_cast<const char*>(g.o.p) + row * g.o.row +
                                       head * g.o.head, lane * 8, g.head_dim);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(a.get(j), b.get(j), sum);
    }
    sum = group_reduce<16, true>(sum);
    if (lane == 0) {
      const int64_t at = (int64_t)head * g.q_rows + row;
      const float lse = g.lse[at];
      // as the gradient's kernels take it (lse_in_sum)
      float own = lse == -INFINITY ? 0.0f : lse * unit_of<DT>();
      if (DT == kBF16 && !(g.softcap > 0.0f)) own = -own / Score<DT, kPlainScore>(g).factor;
      g.rows_info[at] = own;
      g.rows_info[pairs + at] = -sum;
    }
  }
}

}  // namespace

lowbit_status launch_attn_delta(int dt, const AttnArgs& a, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>(((int64_t)a.q_rows * a.q_heads + 15) / 16, 1 << 20);
  return dt == LOWBIT_F32 ? launch(&attn_delta_kernel<kF32>, blocks, 256, s, a)
                          : launch(&attn_delta_kernel<kBF16>, blocks, 256, s, a);
}

}  // namespace lowbit
