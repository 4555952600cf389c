// attn_fwd.hpp -- attention, forward.
#pragma once

#include "attn.hpp"

namespace lowbit {

namespace {

// Four waves, each 32 queries; keys and values in tiles through LDS, two buffers.
// The scores are taken transposed, keys down the registers and a query a lane,
// so that the maximum and the sum of a row stay in the lane (and its other half) and
// the weights are, as they lie, the operand of the product with the values.
//
// Bound by the matrix units and the vector ALU together, at the clock that power leaves: two
// workgroups a CU, two waves a SIMD, one of which takes exps while the other multiplies (32
// products of 32 cycles and about 260 vector instructions a tile and wave).  8 Ki tokens,
// causal, 32 / 8 heads of 128 bfloat16: 512 us, 1.07 PFLOP/s of what is visible; matrix units
// busy 54 % of the cycles, no bank conflict counted.  With the operands read right before their
// products 577 us.  Nine ragged documents of 8 Ki tokens, 16 heads of 64, window 1024, capped scores:
// 74 us, and 100 where scores are beyond half the cap (Score::cap_all).
template <int DT, int D>
struct Forward {
  static constexpr int ES = elem_size<DT>(), KT = DT == kF32 ? 32 : 64, NB = KT / 32;
  using T = Tile<DT, D, KT>;
};

constexpr float kSlack = 5.5f;                     // e^5.5 < 2^8; in units of log2 2^5.5

// out and lse of a lane's row.
template <int DT, int BLOCKS>
__device__ __forceinline__ void finish_rows(const AttnArgs& g, const f32x16 (&acc)[BLOCKS],
                                            int64_t row, int head, float top, float sum, int half,
                                            int first = 0) {
  const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
  store_columns<DT>(static_cast<char*>(const_cast<void*>(g.o.p)) + row * g.o.row + head * g.o.head,
                    acc, scale, half, g.head_dim, first);
  if (half == 0 && first == 0)
    g.lse[(int64_t)head * g.q_rows + row] =
        sum == 0.0f ? -INFINITY : DT == kF32 ? top + logf(sum) : (top + log2f(sum)) * kLn2;
}

template <int DT, int D, int MODE>
__global__ void __launch_bounds__(kAttnThreads, DT == kF32 && D > 64 ? 1 : 2) attn_kernel(AttnArgs g, int tiles) {
  using F = Forward<DT, D>;
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

  const Items items(tiles, g.kv_heads, g.group * g.q_parts);
  for (int64_t item = blockIdx.x; item < items.total; item += gridDim.x) {
    const Queries w(g, items, item, tiles, g.q_parts);
    if (!w.any) continue;
    const Sequence& q = w.q;
    const int kv = w.kv, head = w.head, last = w.last;
    const int i = w.i0 + wave * 32 + col;          // the lane's query
    const int shift = q.lk - q.lq;
    const bool mine = i < q.lq;
    const int64_t row = (int64_t)q.q0 + i;

    u32x4 fq[T::STEPS];
    load_rows(fq, g.q.p, row * g.q.row + head * g.q.head, half, width, mine);
    if (g.scale < 0.0f) negate<DT>(fq);
    const Sight see = sight(g, q, i + shift);
    const KeyTiles<KT> keys(g, w, g.q_parts);
    // whether all 32 queries of the wave see all of a tile
    const int w0 = w.i0 + wave * 32 + shift, w1 = min(w0 + 31, last + shift);
    const Sight wl = sight(g, q, w0), wh = sight(g, q, w1);

    const char* kp = static_cast<const char*>(g.k.p) + q.k0 * g.k.row + kv * g.k.head;
    const char* vp = static_cast<const char*>(g.v.p) + q.k0 * g.v.row + kv * g.v.head;
    // (no rows where there is no such tile: a branch would make the compiler wait for the loads)
    auto issue = [&](int t, char* lk, char* lv, bool any) {
      const int rows = any ? q.lk - t * KT : 0;
      const auto rk = load_k.rows_at(kp + (int64_t)t * KT * g.k.row, (int)g.k.row, width, rows);
      const auto rv = load_v.rows_at(vp + (int64_t)t * KT * g.v.row, (int)g.v.row, width, rows);
#pragma unroll
      for (int j = 0; j < T::LOADS; ++j) load_k.load(rk, lk, wave, j);
#pragma unroll
      for (int j = 0; j < T::LOADS; ++j) load_v.load(rv, lv, wave, j);
    };

    f32x16 acc[T::BLOCKS];
    clear(acc);
    float top = -INFINITY, sum = 0.0f;             // sum: of this half's keys
    score.head(g, head);

    auto compute = [&](const char* lk, const char* lv, int t, bool whole) {
      along.refresh();
      down.refresh();
      f32x16 x[NB];
      clear(x);
      auto key = [&](int i) { return along.load(lk, i % NB, i / NB); };
      auto ahead = read_first<6>(key);
      products<NB * T::STEPS, 6>(ahead, key, [&](int i, const u32x4& f) {
        x[i % NB] = mma<DT>(f, fq[i / NB], x[i % NB]);
      });
      // product i: block b of keys, chunk c, columns n
      auto val = [&](int i) { return down.load(lv, i % T::BLOCKS, i / T::BLOCKS); };
      auto values = read_first<4>(val);

      const int j0 = t * KT;
      const float distance = (float)(i + shift - j0 - 4 * half);
      float most = -INFINITY;
      if constexpr (has_cap(MODE)) score.cap_all(x);
      if constexpr (has_bias(MODE)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            x[b][r] = score.at(x[b][r], distance, 32 * b + r / 4 * 8 + r % 4);
      }
      const int base_key = j0 + 4 * half;
      const int low = see.low - base_key, high = see.high - base_key, pre = see.prefix - base_key;
      auto seen = [&](int j) { return (j < pre) | ((j >= low) & (j <= high)); };
      if (!whole) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            x[b][r] = seen(32 * b + r / 4 * 8 + r % 4) ? x[b][r] : -INFINITY;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) most = fmaxf(most, x[b][r]);
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
      u32x4 p[NB * chunks<DT>()];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[b][r] = score.weight(x[b][r], base);
#pragma unroll
        for (int r = 0; r < 16; ++r) sum += x[b][r];
#pragma unroll
        for (int c = 0; c < chunks<DT>(); ++c) p[b * chunks<DT>() + c] = pack_chunk<DT>(x[b], c);
      }
      products<NB * chunks<DT>() * T::BLOCKS, 4>(values, val, [&](int i, const u32x4& f) {
        acc[i % T::BLOCKS] = mma<DT>(f, p[i / T::BLOCKS], acc[i % T::BLOCKS]);
      });
    };

    // tile u, in lk and lv, while the next one's loads run
    auto step = [&](char* lk, char* lv, char* nk, char* nv, int u) {
      wait_all();
      barrier();
      issue(keys.tile(u + 1), nk, nv, u + 1 < keys.count);
      const int t = keys.tile(u), j0 = t * KT;
      const bool whole = (j0 + KT <= q.prefix) || (j0 >= wh.low && j0 + KT - 1 <= wl.high);
      compute(lk, lv, t, whole);
    };
    issue(keys.tile(0), lk0, lv0, keys.count > 0);
    int u = 0;
    for (; u + 1 < keys.count; u += 2) {
      step(lk0, lv0, lk1, lv1, u);
      step(lk1, lv1, lk0, lv0, u + 1);
    }
    if (u < keys.count) step(lk0, lv0, lk1, lv1, u);
    wait_all();
    barrier();                                     // (the next item writes the buffers)

    sum = both_halves_sum(sum);
    if (g.q_parts > 1) {
      f32x4* to = part_at(g.q_sums, w.unit * g.q_parts + w.part, T::BLOCKS * 4 + 1);
      store_part(to, acc);
      to[T::BLOCKS * 4 * kAttnThreads] = (f32x4){top, sum, 0.0f, 0.0f};
    } else if (mine) {
      finish_rows<DT>(g, acc, row, head, top, sum, half);
    }
  }
}

// The parts of a row's keys joined, in order; a workgroup 32 columns of a tile.
template <int DT, int D>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(AttnArgs g, int tiles) {
  constexpr int BLOCKS = D / 32, VECTORS = BLOCKS * 4 + 1;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Items items(tiles, g.kv_heads, g.group * BLOCKS);
  for (int64_t item = blockIdx.x; item < items.total; item += gridDim.x) {
    const Queries w(g, items, item, tiles, BLOCKS);
    const int i = w.i0 + wave * 32 + lane % 32;
    if (!w.any || i >= w.q.lq) continue;
    const int64_t first = w.unit * g.q_parts;
    float top = -INFINITY, sum = 0.0f;
    for (int p = 0; p < g.q_parts; ++p)
      top = fmaxf(top, part_at(g.q_sums, first + p, VECTORS)[(VECTORS - 1) * kAttnThreads][0]);
    f32x16 acc[1];
    clear(acc);
    for (int p = 0; p < g.q_parts; ++p) {
      const f32x4* from = part_at(g.q_sums, first + p, VECTORS);
      const f32x4 end = from[(VECTORS - 1) * kAttnThreads];
      // (a part in which nothing is seen has sums of 0)
      const float weight = end[0] == -INFINITY ? 1.0f : exp_unit<DT>(end[0] - top);
      sum = __builtin_fmaf(end[1], weight, sum);
      add_part(acc, from + w.part * (4 * kAttnThreads), weight);
    }
    finish_rows<DT>(g, acc, (int64_t)w.q.q0 + i, w.head, top, sum, lane / 32, w.part);
  }
}

template <int DT, int D>
lowbit_status launch_attn_width(const AttnArgs& a, hipStream_t s) {
  const int tiles = attn_tiles(a.q_rows, a.sequences);
  const int64_t blocks = capped(Items(tiles, a.kv_heads, a.group * a.q_parts).total);
  const int mode = score_mode(a);
  const lowbit_status st =
      mode == kPlainScore  ? launch(&attn_kernel<DT, D, kPlainScore>, blocks, kAttnThreads, s, a, tiles)
      : mode == kBiasScore ? launch(&attn_kernel<DT, D, kBiasScore>, blocks, kAttnThreads, s, a, tiles)
      : mode == kCapScore  ? launch(&attn_kernel<DT, D, kCapScore>, blocks, kAttnThreads, s, a, tiles)
                           : launch(&attn_kernel<DT, D, kCapBiasScore>, blocks, kAttnThreads, s, a, tiles);
  if (st != LOWBIT_OK || a.q_parts == 1) return st;
  return launch(&attn_join_kernel<DT, D>, capped(Items(tiles, a.kv_heads, a.group * (D / 32)).total),
                kAttnThreads, s, a, tiles);
}

template <int DT>
lowbit_status launch_attn(const AttnArgs& a, hipStream_t s) {
  return a.head_dim <= 64   ? launch_attn_width<DT, 64>(a, s)
         : a.head_dim <= 96 ? launch_attn_width<DT, 96>(a, s)
                            : launch_attn_width<DT, 128>(a, s);
}

}  // namespace

}  // namespace lowbit
