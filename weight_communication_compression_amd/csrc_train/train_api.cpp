// train_api.cpp -- the extern "C" entry points of the training-step operators
// (declared in include/lowbit_train.h): argument validation, the layout of the
// workspaces and dispatch.  Invalid arguments are rejected before any HIP call;
// nothing here allocates device memory or keeps any state.
#include <hip/hip_runtime.h>

#include <algorithm>
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
  a.rows_per_run = g.rows_per_run;
  a.lanes = g.lanes;
  a.rows_per_gate = std::min(p->rows_per_gate, p->rows);   // (so that sums with it fit)
  a.cols = (int32_t)p->cols;
  a.eps = p->eps;
  a.scale = p->residual_scale;
  a.key = seed_key(p->seed);
  a.cut = drop_cut(p->p);
  a.factor = keep_factor(a.cut);
  return a;
}

// partial sums: `rows` rows of a parameter or the gate
int64_t join_part_bytes(int64_t rows, int64_t cols) { return (rows * cols * 4 + 255) / 256 * 256; }

constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxVocab = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxHidden = (int64_t)1 << 20;
// d of a piece of the vocabulary takes at most this much, so that the loss
// needs far less than its logits; all of the vocabulary in one piece where it fits
constexpr int64_t kXentPieceBytes = (int64_t)512 << 20;
// copies of w's rows, where they are no multiples of 16 bytes: what the last
// level of cache still holds when the products read it
constexpr int64_t kXentPackBytes = (int64_t)128 << 20;
constexpr int64_t kXentTiles = (int64_t)1 << 22;       // of a launch, at most

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

bool check_xent(const lowbit_xent_params* p) {
  return p && p->rows >= 0 && p->rows <= kMaxRows && p->vocab >= 1 && p->vocab <= kMaxVocab &&
         p->hidden >= 1 && p->hidden <= kMaxHidden && valid_dtype(p->type);
}

// The pieces of the vocabulary, and offsets into the workspace.
struct XentPlan {
  int64_t padded, ld, parts, piece, pieces;
  bool packs;                              // w's rows are copied to rows of ld
  int form[4];                             // of each kind of product, in every piece
  bool cuts[4];                            // whether it may cut tiles along k
  int64_t pos, map, info, count, xc, wc, part, hit, d, acc, partial, bytes;
};

XentPlan xent_plan(const lowbit_xent_params* p, bool backward) {
  XentPlan w{};
  const int es = p->type == LOWBIT_F32 ? 4 : 2;
  auto take = [&](int64_t bytes) {
    const int64_t at = w.bytes;
    w.bytes += up(bytes, 256);
    return at;
  };
  // whether a product in its form cuts tiles, and the room for their parts' sums
  auto room = [&](int kind, int64_t m, int64_t n, int64_t k) {
    const XentForm& f = kXentForms[w.form[kind]];
    w.cuts[kind] = xent_may_cut(f, kind, m, n, xent_steps(k, es));
    return xent_slots(f, kind, m, n, xent_steps(k, es)) * f.tm * f.tn * 4;
  };
  w.padded = up(p->rows > 0 ? p->rows : 1, kXentPad);
  w.ld = up(p->hidden, 16 / es);
  w.packs = w.ld != p->hidden;
  w.pos = take(p->rows * 4);
  w.map = take(w.padded * 4);
  w.info = take(w.padded * 16);
  w.count = take(8);                       // and the scale
  w.xc = take(w.padded * w.ld * es);
  int64_t most = up(p->vocab, kXentPad);
  auto cut = [&](int64_t cols) {
    if (cols < most) most = cols > kXentPad ? cols / kXentPad * kXentPad : kXentPad;
  };
  w.form[kXentStats] = xent_form(p->type, kXentStats, p->rows, p->vocab, p->hidden);
  const XentForm& f = kXentForms[w.form[kXentStats]];
  if (backward) cut(std::max(kXentPieceBytes / (w.padded * es), (int64_t)1024));
  if (w.packs) cut(std::max(kXentPackBytes / (w.ld * es), (int64_t)1024));
  cut(kXentTiles / (w.padded / f.tm) * f.tn);
  w.pieces = (p->vocab + most - 1) / most;
  w.piece = up((p->vocab + w.pieces - 1) / w.pieces, kXentPad);
  w.pieces = (p->vocab + w.piece - 1) / w.piece;
  const int64_t cols = w.piece < p->vocab ? w.piece : p->vocab;
  if (w.packs) w.wc = take(w.piece * w.ld * es);
  if (backward) {
    w.d = take(w.padded * w.piece * es);
    w.form[kXentProb] = xent_form(p->type, kXentProb, p->rows, cols, p->hidden);
    w.form[kXentDx] = xent_form(p->type, kXentDx, p->rows, p->hidden, cols);
    w.form[kXentDw] = xent_form(p->type, kXentDw, cols, p->hidden, p->rows);
    const XentForm& fx = kXentForms[w.form[kXentDx]];
    if (w.pieces > 1) w.acc = take(up(p->rows, fx.tm) * up(p->hidden, fx.tn) * 4);
    w.partial = take(std::max({room(kXentProb, p->rows, cols, p->hidden),
                               room(kXentDx, p->rows, p->hidden, cols),
                               room(kXentDw, cols, p->hidden, p->rows)}));
  } else {
    w.parts = (p->vocab + f.tn - 1) / f.tn;
    w.part = take(p->rows * w.parts * 8);
    w.hit = take(w.padded * 4);
    w.partial = take(room(kXentStats, p->rows, cols, p->hidden));
  }
  return w;
}

template <typename T>
T* at(void* base, int64_t offset) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + offset);
}

// Numbers the rows that count and copies them together.
lowbit_status xent_rows(const XentPlan& w, const lowbit_xent_params* p, void* ws, const void* x,
                        const int64_t* targets, const float* lse, const float* dloss,
                        const float* dlse, void* dx, hipStream_t s) {
  XentRows r{};
  r.targets = targets;
  r.lse = lse;
  r.dloss = dloss;
  r.dlse = dlse;
  r.n = p->rows;
  r.vocab = p->vocab;
  r.ignore = p->ignore_index;
  r.pos = at<int32_t>(ws, w.pos);
  r.map = at<int32_t>(ws, w.map);
  r.info = at<float4>(ws, w.info);
  r.count = at<int32_t>(ws, w.count);
  r.scale = at<float>(ws, w.count + 4);
  r.padded = w.padded;
  XentGather g{};
  g.x = x;
  g.xc = at<char>(ws, w.xc);
  g.dx = dx;
  g.pos = r.pos;
  g.map = r.map;
  g.n = p->rows;
  g.padded = w.padded;
  g.hidden = (int32_t)p->hidden;
  g.ld = (int32_t)w.ld;
  return launch_xent_rows(p->type, r, g, s);
}

lowbit_status xent_product(const lowbit_xent_params* p, const XentPlan& w, int kind,
                           XentTileArgs& t, hipStream_t s) {
  t.may_cut = w.cuts[kind];
  return p->type == LOWBIT_F32 ? launch_xent_tile_f32(w.form[kind], kind, t, s)
                               : launch_xent_tile_bf16(w.form[kind], kind, t, s);
}

// The logits' product over piece k of the vocabulary, w's rows copied if they
// have to be; its kind and outputs are left to the caller.
lowbit_status xent_logits(const XentPlan& w, const lowbit_xent_params* p, void* ws, const void* weights,
                          int64_t k, XentTileArgs& t, hipStream_t s) {
  const int64_t es = p->type == LOWBIT_F32 ? 4 : 2;
  t = XentTileArgs{};
  t.count = at<int32_t>(ws, w.count);
  t.scale = at<float>(ws, w.count + 4);
  t.map = at<int32_t>(ws, w.map);
  t.info = at<float4>(ws, w.info);
  t.col0 = k * w.piece;
  t.a = at<char>(ws, w.xc);
  t.b = static_cast<const char*>(weights) + t.col0 * p->hidden * es;
  t.lda = t.ldb = t.k = w.ld;
  t.m = w.padded;
  t.n = t.col0 + w.piece < p->vocab ? w.piece : p->vocab - t.col0;
  if (!w.packs) return LOWBIT_OK;
  XentPack c{};
  c.w = t.b;
  c.to = at<char>(ws, w.wc);
  c.rows = t.n;
  c.hidden = (int32_t)p->hidden;
  c.ld = (int32_t)w.ld;
  t.b = c.to;
  return launch_xent_pack(p->type, c, s);
}

}  // namespace

// The form that takes least time by what its steps and tiles were measured to take
// (us): a step of k with all slots taken, a step at the least, and what a tile takes
// besides (the parts of the softmax; d, dx and dw, which are written).  At 25 sizes
// from 1 x 1690 x 640 to 8192 x 1000 x 4096 its choice takes 2 % longer than the
// fastest form on average and 21 % (5 us) at worst; a form fixed by the rows alone
// took up to 60 % longer.
int xent_form(int dt, int kind, int64_t m, int64_t n, int64_t k) {
  static const double full[2][4] = {{0, 4.6, 3.36, 2.27}, {1.73, 1.19, 1.15, 1.25}};
  static const double least[2][4] = {{0, 3.6, 2.1, 1.2}, {1.3, 0.5, 0.4, 0.25}};
  static const double tile[2][4] = {{5.0, 3.0, 2.5, 3.0}, {8.0, 4.5, 3.8, 3.0}};
  const bool bf16 = dt != LOWBIT_F32;
  m = std::min(m, (int64_t)1 << 20);       // (beyond it the answer is the same, and the counts fit)
  n = std::min(n, (int64_t)1 << 20);
  const uint32_t steps = xent_steps(k, bf16 ? 2 : 4);
  int best = 3;
  double best_time = 0.0;
  for (int i = 3; i >= (bf16 ? 0 : 1); --i) {
    const XentForm& f = kXentForms[i];
    const double own = tile[kind != kXentStats][i];
    const XentCut cut(m > 0 ? m : 1, n, steps, f.tm, f.tn, f.slots,
                      xent_may_cut(f, kind, m, n, steps));
    auto round = [&](double count, double each) {
      const double share = count / f.slots;
      return each * std::max(least[bf16][i], full[bf16][i] * share) + own * std::max(0.5, share);
    };
    double time = cut.whole / f.slots * round(f.slots, steps);
    if (cut.whole % f.slots) time += round(cut.whole % f.slots, steps);
    if (cut.rest) {                        // and the kernel that adds the parts' sums, at 4 TB/s
      const double units = (double)cut.rest * cut.parts;
      time += round(units, (double)steps / cut.parts) + 5.0 + units * f.tm * f.tn * 8 / 4e6;
    }
    if (i == 3 || time < best_time) {
      best = i;
      best_time = time;
    }
  }
  return best;
}

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
  return 4 * join_part_bytes(g.blocks, p->cols) + join_part_bytes(2 * g.runs, p->cols);
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
    at += join_part_bytes(g.blocks, p->cols);
  }
  b.part_gate = reinterpret_cast<float*>(at);
  sums.part_gate = b.part_gate;
  sums.dgate = dgate;
  sums.rows_per_gate = b.j.rows_per_gate;
  sums.rows_per_run = g.rows_per_run;
  sums.blocks = g.blocks;
  const lowbit_status st = launch_join_back(p->block_type, p->stream_type, p->param_type,
                                            p->norm == LOWBIT_NORM_LAYER, g, b, stream);
  return st == LOWBIT_OK ? launch_join_sums(sums, stream) : st;
}

int64_t lowbit_linear_xent_workspace(const lowbit_xent_params* p, int32_t backward) {
  return check_xent(p) ? xent_plan(p, backward != 0).bytes : -1;
}

lowbit_status lowbit_linear_xent(const void* x, const void* w, const int64_t* targets,
                                 const lowbit_xent_params* p, float* loss, float* lse,
                                 void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!check_xent(p)) return LOWBIT_EINVAL;
  if (p->rows == 0) return LOWBIT_OK;
  if (!good(x) || !good(w) || !targets || !aligned(targets, 8) || !good(loss) || !good(lse))
    return LOWBIT_EINVAL;
  const XentPlan q = xent_plan(p, false);
  if (!good(workspace) || workspace_bytes < q.bytes) return LOWBIT_EINVAL;
  lowbit_status st =
      xent_rows(q, p, workspace, x, targets, nullptr, nullptr, nullptr, nullptr, stream);
  if (st != LOWBIT_OK) return st;
  XentTileArgs t{};
  for (int64_t k = 0; k < q.pieces && st == LOWBIT_OK; ++k) {
    st = xent_logits(q, p, workspace, w, k, t, stream);
    t.part = at<float2>(workspace, q.part);
    t.hit = at<float>(workspace, q.hit);
    t.parts = (int32_t)q.parts;
    t.partial = at<float>(workspace, q.partial);
    t.part0 = (int32_t)(t.col0 / kXentForms[q.form[kXentStats]].tn);
    if (st == LOWBIT_OK) st = xent_product(p, q, kXentStats, t, stream);
  }
  if (st != LOWBIT_OK) return st;
  XentJoin j{};
  j.part = t.part;
  j.hit = t.hit;
  j.targets = targets;
  j.pos = at<int32_t>(workspace, q.pos);
  j.n = p->rows;
  j.vocab = p->vocab;
  j.parts = t.parts;
  j.loss = loss;
  j.lse = lse;
  return launch_xent_join(j, stream);
}

lowbit_status lowbit_linear_xent_backward(const void* x, const void* w, const int64_t* targets,
                                          const float* lse, const float* dloss, const float* dlse,
                                          const lowbit_xent_params* p, void* dx, void* dw,
                                          void* workspace, int64_t workspace_bytes,
                                          hipStream_t stream) {
  if (!check_xent(p)) return LOWBIT_EINVAL;
  if (!good_or_null(dx) || !good_or_null(dw)) return LOWBIT_EINVAL;
  if (!dw && (!dx || p->rows == 0)) return LOWBIT_OK;
  if (p->rows > 0 && (!good(x) || !targets || !aligned(targets, 8) || !good(lse) ||
                      !good(dloss) || !good_or_null(dlse)))
    return LOWBIT_EINVAL;
  const XentPlan q = xent_plan(p, true);
  if (!good(w) || !good(workspace) || workspace_bytes < q.bytes) return LOWBIT_EINVAL;
  lowbit_status st = xent_rows(q, p, workspace, x, targets, lse, dloss, dlse, dx, stream);
  const int64_t es = p->type == LOWBIT_F32 ? 4 : 2;
  for (int64_t k = 0; k < q.pieces && st == LOWBIT_OK; ++k) {
    XentTileArgs t{};
    st = xent_logits(q, p, workspace, w, k, t, stream);
    if (st != LOWBIT_OK) return st;
    const int64_t cols = t.n;
    const void* const wk = t.b;
    t.partial = at<float>(workspace, q.partial);
    t.out = at<char>(workspace, q.d);
    t.ldo = q.piece;
    st = xent_product(p, q, kXentProb, t, stream);
    t.n = p->hidden;
    t.ldb = q.ld;
    t.lda = q.piece;
    t.a = at<char>(workspace, q.d);
    t.ldo = p->hidden;
    if (st == LOWBIT_OK && dx) {
      t.b = wk;
      t.k = cols;
      t.out = dx;
      t.acc = q.pieces > 1 ? at<float>(workspace, q.acc) : nullptr;
      t.first = k == 0;
      t.last = k == q.pieces - 1;
      st = xent_product(p, q, kXentDx, t, stream);
    }
    if (st == LOWBIT_OK && dw) {
      t.b = at<char>(workspace, q.xc);
      t.m = cols;
      t.k = q.padded;
      t.out = static_cast<char*>(dw) + t.col0 * p->hidden * es;
      st = xent_product(p, q, kXentDw, t, stream);
    }
  }
  return st;
}

}  // extern "C"
