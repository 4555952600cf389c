// train_api.cpp -- the extern "C" entry points of the training-step operators
// (declared in include/lowbit_train.h): argument validation, the layout of the
// workspaces and dispatch.  Invalid arguments are rejected before any HIP call;
// nothing here allocates device memory or keeps any state.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "train.hpp"

namespace lowbit {

namespace {

constexpr int64_t kMaxN = (int64_t)1 << 48;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool good(const void* p) { return p && aligned(p, 16); }
bool good_or_null(const void* p) { return aligned(p, 16); }
bool valid_dtype(int dt) { return dt == LOWBIT_F32 || dt == LOWBIT_BF16; }
bool valid_p(double p) { return p >= 0.0 && p <= 1.0; }      // false for NaN

uint32_t fmix32_host(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  h ^= h >> 16;
  return h;
}

// K(seed): the key of the counter hash, as of stochastic rounding.
uint32_t seed_key(uint64_t seed) {
  return fmix32_host((uint32_t)seed ^ fmix32_host((uint32_t)(seed >> 32) ^ 0x9E3779B9u));
}

// the draws below it are dropped: p * 65536 to nearest, ties to even
uint32_t drop_cut(double p) { return (uint32_t)std::nearbyint(p * 65536.0); }
float keep_factor(uint32_t cut) { return cut < 65536 ? (float)(65536.0 / (65536 - (int)cut)) : 0.0f; }

lowbit_status dropout(const void* x, const void* r, bool with_r, lowbit_dtype t, int64_t n,
                      double p, uint64_t seed, uint64_t index_offset, void* y, hipStream_t s) {
  if (n < 0 || n > kMaxN || !valid_p(p) || !valid_dtype(t) || index_offset % 8 != 0)
    return LOWBIT_EINVAL;
  if (n == 0) return LOWBIT_OK;
  if (!good(x) || !good(y) || (with_r && !good(r))) return LOWBIT_EINVAL;
  DropoutArgs a{};
  a.x = x;
  a.r = with_r ? r : nullptr;
  a.y = y;
  a.n = n;
  a.pair0 = index_offset / 2;
  a.key = seed_key(seed);
  a.cut = drop_cut(p);
  a.factor = keep_factor(a.cut);
  return launch_dropout((int)t, a, s);
}

// OK, EINVAL or EUNSUPPORTED
lowbit_status check_join(const lowbit_join_params* p, bool gate) {
  if (!p || p->rows < 0 || p->cols < 1 || p->cols > kMaxN || p->rows > kMaxN / p->cols)
    return LOWBIT_EINVAL;
  if (gate && p->rows_per_gate < 1) return LOWBIT_EINVAL;
  if (p->norm != LOWBIT_NORM_RMS && p->norm != LOWBIT_NORM_LAYER) return LOWBIT_EINVAL;
  if (!valid_dtype(p->block_type) || !valid_dtype(p->stream_type) || !valid_dtype(p->param_type))
    return LOWBIT_EINVAL;
  if ((p->stream_type != p->block_type && p->stream_type != LOWBIT_F32) ||
      (p->param_type != p->block_type && p->param_type != LOWBIT_F32))
    return LOWBIT_EINVAL;
  if (!(p->eps >= 0.0f) || !valid_p(p->p)) return LOWBIT_EINVAL;
  return p->cols > kJoinMaxCols ? LOWBIT_EUNSUPPORTED : LOWBIT_OK;
}

JoinArgs join_args(const lowbit_join_params* p, const JoinShape& g) {
  JoinArgs a{};
  a.rows = p->rows;
  a.rows_per_block = g.rows_per_block;
  a.rows_per_gate = p->rows_per_gate;
  a.cols = (int32_t)p->cols;
  a.eps = p->eps;
  a.scale = p->residual_scale;
  a.key = seed_key(p->seed);
  a.cut = drop_cut(p->p);
  a.factor = keep_factor(a.cut);
  return a;
}

// partial sums: one row for each workgroup and parameter, two for the gate
int64_t join_part_bytes(const JoinShape& g, int64_t cols, int rows_each) {
  return (g.blocks * rows_each * cols * 4 + 255) / 256 * 256;
}

}  // namespace

}  // namespace lowbit

using namespace lowbit;

extern "C" {

lowbit_status lowbit_dropout(const void* x, const void* residual, lowbit_dtype t, int64_t n,
                             double p, uint64_t seed, uint64_t index_offset, void* y,
                             hipStream_t stream) {
  return dropout(x, residual, residual != nullptr, t, n, p, seed, index_offset, y, stream);
}

lowbit_status lowbit_dropout_backward(const void* dy, lowbit_dtype t, int64_t n, double p,
                                      uint64_t seed, uint64_t index_offset, void* dx,
                                      hipStream_t stream) {
  return dropout(dy, nullptr, false, t, n, p, seed, index_offset, dx, stream);
}

lowbit_status lowbit_block_join(const void* f, const void* x, const void* post_weight,
                                const void* post_bias, const void* gate, const void* pre_weight,
                                const void* pre_bias, const lowbit_join_params* p, void* x_out,
                                void* z, float* stats, hipStream_t stream) {
  const lowbit_status ok = check_join(p, gate != nullptr);
  if (ok != LOWBIT_OK) return ok;
  if (!good_or_null(post_weight) || !good_or_null(post_bias) || !good_or_null(gate) ||
      !good_or_null(pre_weight) || !good_or_null(pre_bias))
    return LOWBIT_EINVAL;
  if (p->rows == 0) return LOWBIT_OK;
  if (!good(f) || !good(x) || !good(x_out) || !good(z) || !good(stats)) return LOWBIT_EINVAL;
  const JoinShape g = join_shape(p->rows, (int)p->cols, false);
  JoinArgs a = join_args(p, g);
  a.f = f;
  a.x = x;
  a.post_w = post_weight;
  a.post_b = post_bias;
  a.gate = gate;
  a.pre_w = pre_weight;
  a.pre_b = pre_bias;
  a.x_out = x_out;
  a.z = z;
  a.stats = stats;
  return launch_join(p->block_type, p->stream_type, p->param_type, p->norm == LOWBIT_NORM_LAYER,
                     g, a, stream);
}

int64_t lowbit_block_join_backward_workspace(const lowbit_join_params* p) {
  if (check_join(p, false) != LOWBIT_OK) return -1;
  if (p->rows == 0) return 0;
  const JoinShape g = join_shape(p->rows, (int)p->cols, true);
  return 4 * join_part_bytes(g, p->cols, 1) + join_part_bytes(g, p->cols, 2);
}

lowbit_status lowbit_block_join_backward(const void* dx_out, const void* dz, const void* f,
                                         const void* x_out, const float* stats,
                                         const void* post_weight, const void* post_bias,
                                         const void* gate, const void* pre_weight,
                                         const lowbit_join_params* p, void* df, void* dx,
                                         float* dpost_weight, float* dpost_bias, float* dgate,
                                         float* dpre_weight, float* dpre_bias, void* workspace,
                                         int64_t workspace_bytes, hipStream_t stream) {
  const lowbit_status ok = check_join(p, gate != nullptr);
  if (ok != LOWBIT_OK) return ok;
  if (!good_or_null(post_weight) || !good_or_null(post_bias) || !good_or_null(gate) ||
      !good_or_null(pre_weight) || (dgate && !gate))
    return LOWBIT_EINVAL;
  float* const out[4] = {dpost_weight, dpost_bias, dpre_weight, dpre_bias};
  for (float* o : out)
    if (!good_or_null(o)) return LOWBIT_EINVAL;
  if (!good_or_null(dgate)) return LOWBIT_EINVAL;
  JoinSumArgs sums{};
  sums.rows = p->rows;
  sums.rows_per_gate = p->rows_per_gate;
  sums.cols = (int32_t)p->cols;
  if (p->rows == 0) {                     // sums of nothing
    for (float* o : out)
      if (o) sums.out[sums.params++] = o;
    return launch_join_sums(sums, stream);
  }
  if (!good(dx_out) || !good(dz) || !good(f) || !good(x_out) || !good(stats) || !good(df) ||
      !good(dx))
    return LOWBIT_EINVAL;
  const int64_t need = lowbit_block_join_backward_workspace(p);
  if (!good(workspace) || workspace_bytes < need) return LOWBIT_EINVAL;
  const JoinShape g = join_shape(p->rows, (int)p->cols, true);
  JoinBackArgs b{};
  b.j = join_args(p, g);
  b.j.f = f;
  b.j.x = x_out;
  b.j.post_w = post_weight;
  b.j.post_b = post_bias;
  b.j.gate = gate;
  b.j.pre_w = pre_weight;
  b.j.stats = const_cast<float*>(stats);
  b.dx_out = dx_out;
  b.dz = dz;
  b.df = df;
  b.dx = dx;
  b.dgate = dgate;
  char* at = static_cast<char*>(workspace);
  float** const part[4] = {&b.part_post_w, &b.part_post_b, &b.part_pre_w, &b.part_pre_b};
  for (int k = 0; k < 4; ++k) {
    if (out[k]) {
      *part[k] = reinterpret_cast<float*>(at);
      sums.part[sums.params] = *part[k];
      sums.out[sums.params++] = out[k];
    }
    at += join_part_bytes(g, p->cols, 1);
  }
  b.part_gate = reinterpret_cast<float*>(at);
  sums.part_gate = b.part_gate;
  sums.dgate = dgate;
  sums.rows_per_block = g.rows_per_block;
  sums.blocks = g.blocks;
  const lowbit_status st = launch_join_back(p->block_type, p->stream_type, p->param_type,
                                            p->norm == LOWBIT_NORM_LAYER, g, b, stream);
  return st == LOWBIT_OK ? launch_join_sums(sums, stream) : st;
}

}  // extern "C"
