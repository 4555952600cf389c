// attn_fwd.hpp -- attention, forward.
#pragma once

#include "attn.hpp"

namespace lowbit {

namespace {

// Four waves, each 32 queries; keys and values in tiles through LDS, two buffers.
// The scores are taken transposed, keys down the registers and a query a lane,
// so that the maximum and the sum of a row stay in the lane (and its other half) and
// the weights are, as they lie, the operand of the product with the values.
template <int DT, int D, int MODE>
struct Forward {
  static constexpr int ES = elem_size<DT>(), KT = DT == kF32 ? 32 : 64, NB = KT / 32;
  using T = Tile<DT, D, KT>;
};

constexpr float kSlack = 5.5f;                     // e^5.5 < 2^8; in units of log2 2^5.5

template <int DT, int D, int MODE>
__global__ void __launch_bounds__(kAttnThreads, DT == kF32 && D > 64 ? 1 : 2) attn_kernel(AttnArgs g, int tiles) {
  using F = Forward<DT, D, MODE>;
  using T = typename F::T;
  constexpr int KT = F::KT, NB = F::NB, ES = F::ES;
  __shared__ __attribute__((aligned(1024))) char lk0[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char lv0[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char lk1[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char lv1[T::BYTES];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane % 32, half = lane / 32;
  const int width = g.head_dim * ES;
  typename T::Loader load_k, load_v;
  typename T::Along along;
  typename T::Down down;
  load_k.init(g.k.row, width, wave, lane);
  load_v.init(g.v.row, width, wave, lane);
  along.init(lane);
  down.init(lane);
  Score<DT, MODE> score(g);

  const Items items(tiles, g.kv_heads, g.group);
  for (int64_t item = blockIdx.x; item < items.total; item += gridDim.x) {
    int t, kv, in;
    items.take(item, g.kv_heads, t, kv, in);
    if (t >= tiles) continue;
    t = tiles - 1 - t;                             // causal: the last see most
    const int head = kv * g.group + in;
    const int s = find_sequence(g.q_begin, g.sequences, g.q_rows, kRowsPerTile, t);
    const Sequence q = sequence_at(g, s);
    const int i0 = (t - first_tile(g.q_begin, s, g.sequences, g.q_rows, kRowsPerTile)) * kRowsPerTile;
    if (i0 >= q.lq) continue;
    const int i = i0 + wave * 32 + col;            // the lane's query
    const int shift = q.lk - q.lq;
    const bool mine = i < q.lq;
    const int64_t row = (int64_t)q.q0 + i;

    u32x4 fq[T::STEPS];
    {
      const char* p = static_cast<const char*>(g.q.p) + row * g.q.row + head * g.q.head;
#pragma unroll
      for (int kk = 0; kk < T::STEPS; ++kk) {
        const int at = kk * 32 + half * 16;
        fq[kk] = (u32x4){0, 0, 0, 0};
        if (mine && at < width) fq[kk] = *reinterpret_cast<const u32x4*>(p + at);
        if (g.scale < 0.0f) fq[kk] = negated<DT>(fq[kk]);
      }
    }
    const Sight see = sight(g, q, i + shift);
    // tiles of keys: [0, before) of the prefix, [from, to) around the positions
    const int last = min(i0 + kRowsPerTile, q.lq) - 1;
    const Sight lo = sight(g, q, i0 + shift), hi = sight(g, q, last + shift);
    const int before = (q.prefix + KT - 1) / KT;
    const int from = lo.low > 0 ? lo.low / KT : 0;
    const int to = hi.high < 0 ? 0 : hi.high / KT + 1;
    const int end = max(before, to);
    auto after = [&](int t) { return t >= before && t < from ? from : t; };
    // whether all 32 queries of the wave see all of a tile
    const int w0 = i0 + wave * 32 + shift, w1 = min(w0 + 31, last + shift);
    const Sight wl = sight(g, q, w0), wh = sight(g, q, w1);

    const char* kp = static_cast<const char*>(g.k.p) + q.k0 * g.k.row + kv * g.k.head;
    const char* vp = static_cast<const char*>(g.v.p) + q.k0 * g.v.row + kv * g.v.head;
    auto issue = [&](int t, char* lk, char* lv) {
      const int rows = q.lk - t * KT;
      const auto rk = load_k.rows_at(kp + (int64_t)t * KT * g.k.row, (int)g.k.row, width, rows);
      const auto rv = load_v.rows_at(vp + (int64_t)t * KT * g.v.row, (int)g.v.row, width, rows);
#pragma unroll
      for (int j = 0; j < T::LOADS; ++j) load_k.load(rk, lk, wave, j);
#pragma unroll
      for (int j = 0; j < T::LOADS; ++j) load_v.load(rv, lv, wave, j);
    };

    f32x16 acc[T::BLOCKS];
#pragma unroll
    for (int n = 0; n < T::BLOCKS; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[n][r] = 0.0f;
    float top = -INFINITY, sum = 0.0f;             // sum: of this half's keys
    score.head(g, head);

    auto compute = [&](const char* lk, const char* lv, int t) {
      f32x16 x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[b][r] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < T::STEPS; ++kk) x[b] = mma<DT>(along.load(lk, b, kk), fq[kk], x[b]);
      }
      const int j0 = t * KT;
      const bool whole = (j0 + KT <= see.prefix) || (j0 >= wh.low && j0 + KT - 1 <= wl.high);
      const float distance = (float)(i + shift - j0 - 4 * half);
      float most = -INFINITY;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float bend;
          x[b][r] = score.at(x[b][r], distance, 32 * b + r / 4 * 8 + r % 4, bend);
        }
        if (!whole) {
          const int base = j0 + 32 * b + 4 * half;
          const int low = see.low - base, high = see.high - base, pre = see.prefix - base;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = r / 4 * 8 + r % 4;
            if (!(j < pre || (j >= low && j <= high))) x[b][r] = -INFINITY;
          }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) most = fmaxf(most, x[b][r]);
      }
      most = score.scaled(other_half_max(most));
      // the sums stand relative to `top`, which follows the largest score only when it is
      // passed by more than kSlack: weights then are up to 2^8, which loses nothing, and
      // later tiles hardly ever rescale what has been summed
      if (__any(most > top + kSlack)) {
        const float next = fmaxf(top, most);
        const float shrink = next == -INFINITY ? 1.0f : exp_unit<DT>(top - next);
        top = next;
        sum *= shrink;
#pragma unroll
        for (int n = 0; n < T::BLOCKS; ++n) acc[n] *= shrink;
      }
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          x[b][r] = score.weight(x[b][r], base);
          sum += x[b][r];
        }
#pragma unroll
        for (int c = 0; c < chunks<DT>(); ++c) {
          const u32x4 p = pack_chunk<DT>(x[b], c);
#pragma unroll
          for (int n = 0; n < T::BLOCKS; ++n)
            acc[n] = mma<DT>(down.load(lv, n, b * chunks<DT>() + c), p, acc[n]);
        }
      }
    };

    // one tile, in lk and lv, while the next one's loads run
    int now = after(0), next = after(now + 1);
    auto step = [&](char* lk, char* lv, char* nk, char* nv) {
      wait_all();
      barrier();
      if (next < end) issue(next, nk, nv);
      compute(lk, lv, now);
      now = next;
      next = after(now + 1);
    };
    if (now < end) issue(now, lk0, lv0);
    while (next < end) {
      step(lk0, lv0, lk1, lv1);
      step(lk1, lv1, lk0, lv0);
    }
    if (now < end) step(lk0, lv0, lk1, lv1);
    wait_all();
    barrier();                                     // (the next item writes the buffers)

    sum = both_halves_sum(sum);
    if (mine) {
      const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
      char* o = static_cast<char*>(const_cast<void*>(g.o.p)) + row * g.o.row + head * g.o.head;
#pragma unroll
      for (int n = 0; n < T::BLOCKS; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int at = n * 32 + c * 8 + half * 4;
          f32x4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc[n][4 * c + r] * scale;
          if (at < g.head_dim) {
            if constexpr (DT == kF32) *reinterpret_cast<f32x4*>(o + at * 4) = v;
            else *reinterpret_cast<u32x2*>(o + at * 2) =
                     (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
          }
        }
      if (half == 0)
        g.lse[(int64_t)head * g.q_rows + row] =
            sum == 0.0f ? -INFINITY : DT == kF32 ? top + logf(sum) : (top + log2f(sum)) * kLn2;
    }
  }
}

template <int DT, int D>
lowbit_status launch_attn_width(const AttnArgs& a, hipStream_t s) {
  const int tiles = attn_tiles(a.q_rows, a.sequences);
  const Items items(tiles, a.kv_heads, a.group);
  const int64_t blocks = items.total < kMaxBlocks ? items.total : kMaxBlocks;
  switch (score_mode(a)) {
    case kPlainScore:
      return launch(&attn_kernel<DT, D, kPlainScore>, blocks, kAttnThreads, s, a, tiles);
    case kBiasScore:
      return launch(&attn_kernel<DT, D, kBiasScore>, blocks, kAttnThreads, s, a, tiles);
    default:
      return launch(&attn_kernel<DT, D, kCapScore>, blocks, kAttnThreads, s, a, tiles);
  }
}

template <int DT>
lowbit_status launch_attn(const AttnArgs& a, hipStream_t s) {
  return a.head_dim <= 64   ? launch_attn_width<DT, 64>(a, s)
         : a.head_dim <= 96 ? launch_attn_width<DT, 96>(a, s)
                            : launch_attn_width<DT, 128>(a, s);
}

}  // namespace

}  // namespace lowbit
