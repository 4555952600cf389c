// block_api.cpp -- the extern "C" entry points of rotary, attention and orthogonalize
// (declared in include/lowbit_train.h): argument validation, the layout of the
// workspaces and dispatch.  Invalid arguments are rejected before any HIP call;
// nothing here allocates device memory or keeps any state.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "block.hpp"
#include "ortho_choice.hpp"

namespace lowbit {

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool good(const void* p, uintptr_t a = 16) { return p && aligned(p, a); }
bool valid_dtype(int dt) { return dt == LOWBIT_F32 || dt == LOWBIT_BF16; }
int elem(int dt) { return dt == LOWBIT_F32 ? 4 : 2; }
bool within(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

constexpr int64_t kMaxStride = (int64_t)1 << 40;

// Whether no two elements of rows x heads x dim share a place.
bool apart(const lowbit_strides& s, int64_t rows, int64_t heads, int64_t dim) {
  if (heads <= 1) return rows <= 1 || s.row >= dim;
  if (rows <= 1) return s.head >= dim;
  // one of the two steps over all that the other reaches (strides up to 2^40, counts
  // up to 2^31: a double holds the products near enough to tell)
  const double reach_head = (double)(heads - 1) * (double)s.head + (double)dim;
  const double reach_row = (double)(rows - 1) * (double)s.row + (double)dim;
  return (s.head >= dim && (double)s.row >= reach_head) || (s.row >= dim && (double)s.head >= reach_row);
}

lowbit_status rotary(const void* x, const double* freqs, const int64_t* positions,
                     const lowbit_rotary_params* p, void* y, float sign, hipStream_t stream) {
  if (!p || !within(p->rows, 0, ((int64_t)1 << 31) - 1) || !within(p->heads, 1, 65536) ||
      !within(p->head_dim, 2, 65536) || !within(p->rot_dim, 2, p->head_dim) || p->rot_dim % 2 ||
      !valid_dtype(p->type) || !std::isfinite(p->scale))
    return LOWBIT_EINVAL;
  if (p->layout != LOWBIT_ROTARY_HALF && p->layout != LOWBIT_ROTARY_INTERLEAVED) return LOWBIT_EINVAL;
  if (!positions && p->rows_per_sequence < 1) return LOWBIT_EINVAL;
  for (const lowbit_strides* s : {&p->x, &p->y})
    if (!within(s->row, 0, kMaxStride) || !within(s->head, 0, kMaxStride)) return LOWBIT_EINVAL;
  if (!apart(p->y, p->rows, p->heads, p->head_dim)) return LOWBIT_EINVAL;
  if (x == y && (p->x.row != p->y.row || p->x.head != p->y.head)) return LOWBIT_EINVAL;
  if (p->rows == 0) return LOWBIT_OK;
  if (!good(x, elem(p->type)) || !good(y, elem(p->type)) || !good(freqs, 8) || !aligned(positions, 8))
    return LOWBIT_EINVAL;
  RotaryArgs a{};
  a.x = x;
  a.y = y;
  a.freqs = freqs;
  a.positions = positions;
  a.rows = p->rows;
  a.rows_per_sequence = positions ? 1 : p->rows_per_sequence;
  a.x_row = p->x.row;
  a.x_head = p->x.head;
  a.y_row = p->y.row;
  a.y_head = p->y.head;
  a.heads = p->heads;
  a.head_dim = p->head_dim;
  a.rot_dim = p->rot_dim;
  a.scale = p->scale;
  a.sign = sign;
  return launch_rotary(p->type, p->layout, a, stream);
}

constexpr int64_t kMaxAttnRows = (int64_t)1 << 29;

// OK, EINVAL or EUNSUPPORTED; strides apart
lowbit_status check_attention(const lowbit_attention_params* p) {
  if (!p || !within(p->q_rows, 0, kMaxAttnRows) || !within(p->k_rows, 0, kMaxAttnRows) ||
      !within(p->sequences, 0, 1 << 24) || p->window < 0 || !within(p->q_heads, 1, 4096) ||
      !within(p->kv_heads, 1, p->q_heads) || p->q_heads % p->kv_heads ||
      !within(p->head_dim, 8, 65536) || p->head_dim % 8 || !valid_dtype(p->type) ||
      !within(p->causal, 0, 1) || !std::isfinite(p->scale) || !std::isfinite(p->softcap) ||
      p->softcap < 0.0f)
    return LOWBIT_EINVAL;
  return p->head_dim > 128 ? LOWBIT_EUNSUPPORTED : LOWBIT_OK;
}

bool good_rows(const lowbit_strides& s, int dim) {
  return within(s.row, dim, (int64_t)1 << 22) && s.row % 8 == 0 && within(s.head, 0, kMaxStride) &&
         s.head % 8 == 0;
}

// Offsets against rows, which the C ABI knows only where there are none.
bool good_offsets(const lowbit_attention_params* p, const int32_t* q_begin, const int32_t* k_begin,
                  const int32_t* prefix, const float* slopes) {
  if (!aligned(q_begin, 4) || !aligned(k_begin, 4) || !aligned(prefix, 4) || !aligned(slopes, 4))
    return false;
  if (p->sequences == 0) return true;
  if (!q_begin && p->q_rows % p->sequences) return false;
  if (!k_begin && (q_begin ? p->q_rows != p->k_rows : p->k_rows % p->sequences != 0)) return false;
  return true;
}

AttnMatrix matrix(const void* p, const lowbit_strides& s, int es) { return {p, s.row * es, s.head * es}; }

AttnArgs attention_args(const void* q, const void* k, const void* v, const void* out, float* lse,
                        const int32_t* q_begin, const int32_t* k_begin, const int32_t* prefix,
                        const float* slopes, const lowbit_attention_params* p) {
  const int es = elem(p->type);
  AttnArgs a{};
  a.q = matrix(q, p->q, es);
  a.k = matrix(k, p->k, es);
  a.v = matrix(v, p->v, es);
  a.o = matrix(out, p->out, es);
  a.lse = lse;
  a.q_begin = q_begin;
  a.k_begin = k_begin ? k_begin : q_begin;
  a.prefix = prefix;
  a.slopes = slopes;
  a.q_rows = (int32_t)p->q_rows;
  a.k_rows = (int32_t)p->k_rows;
  a.sequences = p->sequences;
  a.q_heads = p->q_heads;
  a.kv_heads = p->kv_heads;
  a.group = p->q_heads / p->kv_heads;
  a.head_dim = p->head_dim;
  a.causal = p->causal;
  // a window as long as all rows hides nothing
  a.window = p->window > p->q_rows + p->k_rows ? 0 : (int32_t)p->window;
  a.scale = p->scale;
  a.softcap = p->softcap;
  return a;
}

// Parts and the workspace: the gradient's lse and D of each query row, the parts' sums.
struct AttnPlan {
  int q_parts, k_parts;
  int64_t q_sums, k_sums, bytes;
};

// The chip holds 512 workgroups at one time.  Where there are fewer tiles of
// queries, their keys are cut, down to 256 on average.  By k and v the gradient's workgroups
// take from nothing to twice the mean of a causal sequence, so that more than one round of them
// is wanted, the long ones first; their queries are cut, down to as many of all heads.  Of binary32
// products take eight times as long, so that parts go down to 64, and of wide heads a CU holds one
// workgroup: as many parts as fill one round.  Whole gradients, parts by q and by k and v, the rule's
// first: five ragged documents (432 and 144 tiles) 2 and 5 106 us, 2 and 4 103, 1 and 3 105, 1 and 4
// 106, 1 and 6 117, 3 and 5 116, 1 and 2 140, uncut 234; 8 Ki tokens of 32 / 8 heads (2080 and 520) 1 and 2
// 1645, 1 and 3 1662, uncut 1690; three binary32 sequences, wide heads (54 and 78) 4 and 3 102, 3 and 2 108, 3
// and 3 112, uncut 182; 2048 binary32 tokens of 8 heads of 64 (136 and 136) 6 and 5 169, 4 and 4 170, 2 and 4 242,
// uncut 304.
AttnPlan attn_plan(const lowbit_attention_params* p, bool backward) {
  AttnPlan w{};
  const int64_t each = std::max(p->sequences, 1), group = p->q_heads / p->kv_heads;
  const bool alone = p->type == LOWBIT_F32 && p->head_dim > 64;
  auto parts = [&](int64_t wanted, int64_t tiles, int64_t most) {
    const int64_t n = !tiles ? 1 : alone ? 256 / tiles : (wanted + tiles - 1) / tiles;
    return (int)std::max<int64_t>(1, std::min<int64_t>({n, most, 16}));
  };
  const int64_t least = p->type == LOWBIT_F32 ? 64 : 256;
  const int64_t width = p->head_dim <= 64 ? 64 : p->head_dim <= 96 ? 96 : 128;
  const int64_t tile = kAttnRows * width * 4;      // a tile's sums
  const int64_t q_tiles = attn_tiles(p->q_rows, p->sequences) * (int64_t)p->q_heads;
  const int64_t k_tiles = attn_tiles(p->k_rows, p->sequences) * (int64_t)p->kv_heads;
  w.q_parts = q_tiles >= 512 ? 1 : parts(768, q_tiles, p->k_rows / each / least);
  w.k_parts = backward ? parts(640, k_tiles, p->q_rows * group / each / least) : 1;
  w.q_sums = backward ? up(p->q_rows * p->q_heads * 8, 256) : 0;
  // (the forward call keeps the maximum and the sum of a row beside the two halves of it)
  w.k_sums = w.q_sums + (w.q_parts > 1 ? q_tiles * w.q_parts * (tile + (backward ? 0 : kAttnRows * 32)) : 0);
  w.bytes = w.k_sums + (w.k_parts > 1 ? k_tiles * w.k_parts * 2 * tile : 0);
  return w;
}

bool check_ortho(const lowbit_orthogonalize_params* p) {
  if (!p || !within(p->batch, 0, 1 << 20) || !within(p->rows, 1, 65536) ||
      !within(p->cols, 1, 65536) || !valid_dtype(p->type) || !within(p->steps, 0, 64) ||
      !std::isfinite(p->a) || !std::isfinite(p->b) || !std::isfinite(p->c) || !(p->eps >= 0.0f) ||
      !std::isfinite(p->eps) || !std::isfinite(p->scale))
    return false;
  return p->batch * p->rows * p->cols <= (int64_t)1 << 40;
}

struct OrthoPlan {
  int64_t parts, x, xh, xh_next, ah, bh, partial, bytes;
  int m, n, ldm, ldn;
};

OrthoPlan ortho_plan(const lowbit_orthogonalize_params* p) {
  OrthoPlan w{};
  w.m = (int)std::min(p->rows, p->cols);
  w.n = (int)std::max(p->rows, p->cols);
  w.ldm = (int)up(w.m, kOrthoPad);
  w.ldn = (int)up(w.n, kOrthoPad);
  auto take = [&](int64_t bytes) {
    const int64_t at = w.bytes;
    w.bytes += up(bytes, 256);
    return at;
  };
  const int64_t rows = p->batch * w.m;
  w.parts = take(p->batch * kOrthoParts * 8);
  w.x = take(rows * w.ldn * 4);
  w.xh = take(rows * w.ldn * 2);
  w.xh_next = take(rows * w.ldn * 2);
  w.ah = take(rows * w.ldm * 2);
  w.bh = take(rows * w.ldm * 2);
  w.partial = take(std::max({ortho_part_bytes(ortho_choice(true, true, p->batch, w.m, w.n)),
                             ortho_part_bytes(ortho_choice(true, false, p->batch, w.m, w.n)),
                             ortho_part_bytes(ortho_choice(false, false, p->batch, w.m, w.n))}));
  return w;
}

}  // namespace

}  // namespace lowbit

using namespace lowbit;

extern "C" {

lowbit_status lowbit_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling,
                                        double factor, int64_t original_length, double slow_turns,
                                        double fast_turns, double* freqs, float* scale) {
  if (!freqs || !scale || !within(rot_dim, 2, 65536) || rot_dim % 2 || !within(scaling, 0, 3) ||
      !(base > 0.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor))
    return LOWBIT_EINVAL;
  if (scaling == LOWBIT_ROTARY_PARTS &&
      (factor < 1.0 || original_length < 1 || !(slow_turns >= 0.0) || !(fast_turns > slow_turns) ||
       !std::isfinite(fast_turns)))
    return LOWBIT_EINVAL;
  if (scaling == LOWBIT_ROTARY_BASE && rot_dim > 2)
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  *scale = scaling == LOWBIT_ROTARY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == LOWBIT_ROTARY_LINEAR) f /= factor;
    if (scaling == LOWBIT_ROTARY_PARTS) {
      const double turns = (double)original_length * f / 6.283185307179586;
      const double keep =
          std::min(1.0, std::max(0.0, (turns - slow_turns) / (fast_turns - slow_turns)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    freqs[i] = f;
  }
  return LOWBIT_OK;
}

lowbit_status lowbit_rotary(const void* x, const double* freqs, const int64_t* positions,
                            const lowbit_rotary_params* p, void* y, hipStream_t stream) {
  return rotary(x, freqs, positions, p, y, 1.0f, stream);
}

lowbit_status lowbit_rotary_backward(const void* dy, const double* freqs,
                                     const int64_t* positions, const lowbit_rotary_params* p,
                                     void* dx, hipStream_t stream) {
  return rotary(dy, freqs, positions, p, dx, -1.0f, stream);
}

lowbit_status lowbit_attention(const void* q, const void* k, const void* v,
                               const int32_t* q_begin, const int32_t* k_begin,
                               const int32_t* prefix, const float* slopes,
                               const lowbit_attention_params* p, void* out, float* lse,
                               void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const lowbit_status st = check_attention(p);
  if (st != LOWBIT_OK) return st;
  for (const lowbit_strides* s : {&p->q, &p->k, &p->v, &p->out})
    if (!good_rows(*s, p->head_dim)) return LOWBIT_EINVAL;
  if (!apart(p->out, p->q_rows, p->q_heads, p->head_dim) ||
      !good_offsets(p, q_begin, k_begin, prefix, slopes))
    return LOWBIT_EINVAL;
  if (p->q_rows == 0 || p->sequences == 0) return LOWBIT_OK;
  if (!good(q) || (p->k_rows > 0 && (!good(k) || !good(v))) || !good(out) || !good(lse))
    return LOWBIT_EINVAL;
  const AttnPlan plan = attn_plan(p, false);
  if (plan.bytes > 0 && (!good(workspace) || workspace_bytes < plan.bytes)) return LOWBIT_EINVAL;
  AttnArgs a = attention_args(q, k, v, out, lse, q_begin, k_begin, prefix, slopes, p);
  a.q_parts = plan.q_parts;
  a.q_sums = static_cast<float*>(workspace);
  return p->type == LOWBIT_F32 ? launch_attn_f32(a, stream) : launch_attn_bf16(a, stream);
}

int64_t lowbit_attention_workspace(const lowbit_attention_params* p, int32_t backward) {
  return check_attention(p) == LOWBIT_OK ? attn_plan(p, backward != 0).bytes : -1;
}

lowbit_status lowbit_attention_backward(const void* dout, const void* q, const void* k,
                                        const void* v, const void* out, const float* lse,
                                        const int32_t* q_begin, const int32_t* k_begin,
                                        const int32_t* prefix, const float* slopes,
                                        const lowbit_attention_params* p, void* dq, void* dk,
                                        void* dv, void* workspace, int64_t workspace_bytes,
                                        hipStream_t stream) {
  const lowbit_status st = check_attention(p);
  if (st != LOWBIT_OK) return st;
  for (const lowbit_strides* s : {&p->q, &p->k, &p->v, &p->out, &p->dout, &p->dq, &p->dk, &p->dv})
    if (!good_rows(*s, p->head_dim)) return LOWBIT_EINVAL;
  if (!apart(p->dq, p->q_rows, p->q_heads, p->head_dim) ||
      !apart(p->dk, p->k_rows, p->kv_heads, p->head_dim) ||
      !apart(p->dv, p->k_rows, p->kv_heads, p->head_dim) ||
      !good_offsets(p, q_begin, k_begin, prefix, slopes))
    return LOWBIT_EINVAL;
  if (p->sequences == 0 || (p->q_rows == 0 && p->k_rows == 0)) return LOWBIT_OK;
  if (p->q_rows > 0 && (!good(q) || !good(dout) || !good(out) || !good(lse) || !good(dq)))
    return LOWBIT_EINVAL;
  if (p->k_rows > 0 && (!good(k) || !good(v) || !good(dk) || !good(dv))) return LOWBIT_EINVAL;
  const AttnPlan plan = attn_plan(p, true);
  if (plan.bytes > 0 && (!good(workspace) || workspace_bytes < plan.bytes)) return LOWBIT_EINVAL;
  AttnArgs a = attention_args(q, k, v, out, const_cast<float*>(lse), q_begin, k_begin, prefix,
                              slopes, p);
  const int es = elem(p->type);
  a.dout = matrix(dout, p->dout, es);
  a.dq = matrix(dq, p->dq, es);
  a.dk = matrix(dk, p->dk, es);
  a.dv = matrix(dv, p->dv, es);
  a.rows_info = static_cast<float*>(workspace);
  a.q_parts = plan.q_parts;
  a.k_parts = plan.k_parts;
  a.q_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.q_sums);
  a.k_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.k_sums);
  if (p->q_rows > 0) {
    const lowbit_status sd = launch_attn_delta(p->type, a, stream);
    if (sd != LOWBIT_OK) return sd;
  }
  return p->type == LOWBIT_F32 ? launch_attn_back_f32(a, stream) : launch_attn_back_bf16(a, stream);
}

int64_t lowbit_orthogonalize_workspace(const lowbit_orthogonalize_params* p) {
  return check_ortho(p) ? ortho_plan(p).bytes : -1;
}

lowbit_status lowbit_orthogonalize(const void* g, const lowbit_orthogonalize_params* p, void* out,
                                   void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!check_ortho(p)) return LOWBIT_EINVAL;
  if (p->batch == 0) return LOWBIT_OK;
  const OrthoPlan w = ortho_plan(p);
  if (!good(g) || !good(out) || !good(workspace) || workspace_bytes < w.bytes) return LOWBIT_EINVAL;
  if (g == out && p->type != LOWBIT_BF16) return LOWBIT_EINVAL;
  char* const at = static_cast<char*>(workspace);
  OrthoArgs a{};
  a.g = g;
  a.out = out;
  a.parts = reinterpret_cast<double*>(at + w.parts);
  a.x = reinterpret_cast<float*>(at + w.x);
  a.xh = at + w.xh;
  a.xh_next = at + w.xh_next;
  a.ah = at + w.ah;
  a.bh = at + w.bh;
  a.partial = reinterpret_cast<float*>(at + w.partial);
  a.batch = p->batch;
  a.m = w.m;
  a.n = w.n;
  a.ldm = w.ldm;
  a.ldn = w.ldn;
  a.turned = p->rows > p->cols;
  a.nparts = (int32_t)std::min<int64_t>(kOrthoParts, ((int64_t)w.m * w.n + 16383) / 16384);
  a.a = p->a;
  a.b = p->b;
  a.c = p->c;
  a.eps = p->eps;
  a.scale = p->scale;
  return launch_ortho(p->type, a, p->steps, stream);
}

}  // extern "C"
