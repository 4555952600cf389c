// attn_back.hpp -- attention's gradient.
#pragma once

#include "attn.hpp"

namespace lowbit {

namespace {

// Sizes of the two halves of the gradient.  By k and v, the wide forms' values stay in LDS,
// since a lane's registers do not hold them too.
template <int DT, int D>
struct Back {
  static constexpr int KT = DT == kF32 ? 32 : 64;  // keys of a tile that passes by
  static constexpr bool KEEP = D <= (DT == kF32 ? 96 : 64);
  static constexpr int QT = DT == kF32 || !KEEP ? 32 : 64;
  static constexpr int BYTES = Tile<DT, D, KT>::BYTES, Q_BYTES = Tile<DT, D, QT>::BYTES;
  static constexpr int VALUES = Tile<DT, D, 32>::BYTES;      // of a wave
  // the values of bfloat16 fit where the other half has its second two tiles
  static constexpr bool APART = !KEEP && 4 * Q_BYTES + kWaves * VALUES > 4 * BYTES;
};

// dq: four waves, each 32 queries, as in the forward pass; the scores and dout.v
// are taken again, transposed, and their gradient is, as it lies, the operand
// of the product with the keys: three products.
template <int DT, int D, int MODE>
__device__ __forceinline__ void attn_dq(const AttnArgs& g, int tiles, int64_t block, int64_t blocks,
                                        char* lk0, char* lv0, char* lk1, char* lv1) {
  constexpr int KT = Back<DT, D>::KT, NB = KT / 32, ES = elem_size<DT>();
  using T = Tile<DT, D, KT>;
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
  for (int64_t item = block; item < items.total; item += blocks) {
    const Queries w(g, items, item, tiles, g.q_parts);
    if (!w.any) continue;
    const Sequence& q = w.q;
    const int kv = w.kv, head = w.head, last = w.last;
    const int i = w.i0 + wave * 32 + col;
    const int shift = q.lk - q.lq;
    const bool mine = i < q.lq;
    const int64_t row = (int64_t)q.q0 + i;
    score.head(g, head);

    u32x4 fq[T::STEPS], fdo[T::STEPS];
    load_rows(fq, g.q.p, row * g.q.row + head * g.q.head, half, width, mine);
    load_rows(fdo, g.dout.p, row * g.dout.row + head * g.dout.head, half, width, mine);
    if (g.scale < 0.0f) negate<DT>(fq);
    float lse = 0.0f, minus_d = 0.0f;
    if (mine) {
      const float* info = g.rows_info + (int64_t)head * g.q_rows + row;
      lse = info[0];
      minus_d = info[(int64_t)g.q_heads * g.q_rows];
    }
    const Sight see = sight(g, q, i + shift);
    const KeyTiles<KT> keys(g, w, g.q_parts);
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

    auto compute = [&](const char* lk, const char* lv, int t) {
      const int j0 = t * KT;
      const bool whole = (j0 + KT <= see.prefix) || (j0 >= wh.low && j0 + KT - 1 <= wl.high);
      const float distance = (float)(i + shift - j0 - 4 * half);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        along.refresh();
        down.refresh();
        f32x16 x[1], dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          x[0][r] = lse_in_sum<DT, MODE>() ? lse : 0.0f;
          dp[r] = minus_d;
        }
        auto rows = [&](int kk) { return Two{along.load(lk, b, kk), along.load(lv, b, kk)}; };
        auto ahead = read_first<3>(rows);
        products<T::STEPS, 3>(ahead, rows, [&](int kk, const Two& f) {
          x[0] = mma<DT>(f.a, fq[kk], x[0]);
          dp = mma<DT>(f.b, fdo[kk], dp);
        });
        auto key = [&](int i) { return down.load(lk, i % T::BLOCKS, b * chunks<DT>() + i / T::BLOCKS); };
        auto keys_ahead = read_first<4>(key);
        const int base = j0 + 32 * b + 4 * half;
        const int low = see.low - base, high = see.high - base, pre = see.prefix - base;
        auto seen = [&](int r) {
          const int j = r / 4 * 8 + r % 4;
          return (j < pre) | ((j >= low) & (j <= high));
        };
        if constexpr (has_cap(MODE)) score.cap_all(x);
        if (!has_cap(MODE) && !whole) {
#pragma unroll
          for (int r = 0; r < 16; ++r) x[0][r] = seen(r) ? x[0][r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float y = score.at(x[0][r], distance, 32 * b + r / 4 * 8 + r % 4);
          float p = score.weight(y, lse_in_sum<DT, MODE>() ? 0.0f : lse);
          if (has_cap(MODE)) p = whole | seen(r) ? p : 0.0f;
          x[0][r] = p * dp[r] * score.bend(x[0][r]);
        }
        u32x4 p[chunks<DT>()];
#pragma unroll
        for (int c = 0; c < chunks<DT>(); ++c) p[c] = pack_chunk<DT>(x[0], c);
        products<chunks<DT>() * T::BLOCKS, 4>(keys_ahead, key, [&](int i, const u32x4& f) {
          acc[i % T::BLOCKS] = mma<DT>(f, p[i / T::BLOCKS], acc[i % T::BLOCKS]);
        });
      }
    };

    // tile u, in lk and lv, while the next one's loads run
    auto step = [&](char* lk, char* lv, char* nk, char* nv, int u) {
      wait_all();
      barrier();
      issue(keys.tile(u + 1), nk, nv, u + 1 < keys.count);
      compute(lk, lv, keys.tile(u));
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
    if (g.q_parts > 1)
      store_part(part_at(g.q_sums, w.unit * g.q_parts + w.part, T::BLOCKS * 4), acc);
    else if (mine)
      store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dq.p)) + row * g.dq.row +
                            head * g.dq.head, acc, g.scale, half, g.head_dim);
  }
}

// Where a workgroup's keys are.
struct Keys {
  Sequence q;
  int j0, kv, part;
  bool any;
  int64_t unit;                                    // tile and head, for the parts
  __device__ __forceinline__ Keys(const AttnArgs& g, const Items& items, int64_t item, int tiles) {
    int t;
    items.take(item, g.kv_heads, t, kv, part);
    any = t < tiles;                               // causal: the first keys are seen by most
    unit = (int64_t)kv * tiles + t;
    if (!any) return;
    const int s = find_sequence(g.k_begin, g.sequences, g.k_rows, kRowsPerTile, t);
    q = sequence_at(g, s);
    j0 = (t - first_tile(g.k_begin, s, g.sequences, g.k_rows, kRowsPerTile)) * kRowsPerTile;
    any = j0 >= 0 && j0 < q.lk;                    // (below 0: rows before the first sequence)
  }
};

// dk and dv: four waves, each 32 keys; the queries of every head that reads them
// pass by in tiles.  A key a lane and queries down the registers, so that the weights
// and the scores' gradient are operands as they lie here too.  Where there are too few
// tiles of keys for the chip, the queries of all heads are shared out in g.k_parts
// even parts, whose sums a second kernel adds in order: four products.
template <int DT, int D, int MODE>
__device__ __forceinline__ void attn_dkv(const AttnArgs& g, int tiles, int64_t block, int64_t blocks,
                                         char* lq0, char* ld0, char* li0, char* lq1, char* ld1,
                                         char* li1, char* values) {
  constexpr bool KEEP = Back<DT, D>::KEEP;
  constexpr int QT = Back<DT, D>::QT, NB = QT / 32, ES = elem_size<DT>();
  using T = Tile<DT, D, QT>;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane % 32, half = lane / 32;
  const int width = g.head_dim * ES;
  typename T::Loader load_q, load_d;
  typename T::Along along;
  typename T::Down down;
  load_q.init(g.q.row, width, wave, lane);
  load_d.init(g.dout.row, width, wave, lane);
  along.init(lane);
  down.init(lane);
  Score<DT, MODE> score(g);

  const Items items(tiles, g.kv_heads, g.k_parts);
  for (int64_t item = block; item < items.total; item += blocks) {
    const Keys w(g, items, item, tiles);
    if (!w.any) continue;
    const Sequence& q = w.q;
    const int kv = w.kv, j0 = w.j0;
    const int j = j0 + wave * 32 + col;            // the lane's key
    const int shift = q.lk - q.lq;
    const bool mine = j < q.lk;
    const int64_t row = (int64_t)q.k0 + j;

    u32x4 fk[T::STEPS], fv[T::STEPS];
    load_rows(fk, g.k.p, row * g.k.row + kv * g.k.head, half, width, mine);
    if (g.scale < 0.0f) negate<DT>(fk);
    load_rows(fv, g.v.p, row * g.v.row + kv * g.v.head, half, width, mine);
    char* const lv = values;                       // the wave's own
    if constexpr (!KEEP) {
#pragma unroll
      for (int kk = 0; kk < T::STEPS; ++kk) along.store(lv, kk, fv[kk]);
    }

    // queries low .. high see key j
    auto low_of = [&](int j) {
      return j < q.prefix ? 0 : g.causal ? max(0, j - shift) : g.window ? max(0, j - g.window + 1 - shift) : 0;
    };
    auto high_of = [&](int j) {
      return j < q.prefix || !g.window ? q.lq - 1 : min(q.lq - 1, j + g.window - 1 - shift);
    };
    const int low = low_of(j), high = high_of(j);
    const int last = min(j0 + kRowsPerTile, q.lk) - 1;
    const int from = low_of(j0) / QT;
    const int top = j0 < q.prefix ? q.lq - 1 : high_of(last);
    const int across = max(0, (top < 0 ? 0 : top / QT + 1) - from);   // tiles of a head's queries
    // what all 32 keys of the wave are seen by
    const int w0 = j0 + wave * 32, w1 = min(w0 + 31, last);
    const int wlow = low_of(w1), whigh = high_of(max(w0, min(q.prefix, w1)));
    // this part's tiles of all heads' queries
    const int64_t all = (int64_t)across * g.group;
    int left = (int)(all * (w.part + 1) / g.k_parts - all * w.part / g.k_parts);
    const int first = (int)(all * w.part / g.k_parts);
    int in = across ? first / across : 0, t = from + (across ? first % across : 0);

    f32x16 dk[T::BLOCKS], dv[T::BLOCKS];
    clear(dk);
    clear(dv);

    // (no rows where there is no next tile: a branch would make the compiler wait for the loads)
    auto issue = [&](char* lq, char* ld, char* li, bool any) {
      const int head = kv * g.group + in;
      const int rows = any ? q.lq - t * QT : 0;
      const int64_t at = (int64_t)q.q0 + t * QT;
      const auto rq = load_q.rows_at(static_cast<const char*>(g.q.p) + at * g.q.row + head * g.q.head,
                                     (int)g.q.row, width, rows);
      const auto rd = load_d.rows_at(static_cast<const char*>(g.dout.p) + at * g.dout.row +
                                         head * g.dout.head, (int)g.dout.row, width, rows);
#pragma unroll
      for (int j = 0; j < T::LOADS; ++j) load_q.load(rq, lq, wave, j);
#pragma unroll
      for (int j = 0; j < T::LOADS; ++j) load_d.load(rd, ld, wave, j);
      // lse (even waves) and -D (odd ones), each twice
      const auto r = open(g.rows_info + ((int64_t)(wave % 2) * g.q_heads + head) * g.q_rows + at,
                          max(0, min(rows, 64)) * 4);
      load_floats(r, li + wave * 256, lane);
    };
    auto compute = [&](const char* lq, const char* ld, const char* li, int t) {
      const int i0 = t * QT;
      const bool whole = i0 >= wlow && i0 + QT - 1 <= whigh;
      const float distance = (float)(i0 + 4 * half + shift - j);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        along.refresh();
        down.refresh();
        // a lane's sixteen queries: 4 consecutive ones, four times
        auto info = [&](int which, int c) {
          return *reinterpret_cast<const f32x4*>(li + which * 256 + (32 * b + 8 * c + 4 * half) * 4);
        };
        f32x16 x[1], dp;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x4 minus_d = info(1, c);
          const f32x4 lse = lse_in_sum<DT, MODE>() ? info(0, c) : (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[0][4 * c + e] = lse[e];
            dp[4 * c + e] = minus_d[e];
          }
        }
        auto rows = [&](int kk) {
          return Three{along.load(lq, b, kk), along.load(ld, b, kk),
                       KEEP ? fv[kk] : along.load(lv, 0, kk)};
        };
        auto ahead = read_first<2>(rows);
        products<T::STEPS, 2>(ahead, rows, [&](int kk, const Three& f) {
          x[0] = mma<DT>(f.a, fk[kk], x[0]);
          dp = mma<DT>(f.b, f.c, dp);
        });
        auto columns = [&](int i) {
          const int n = i % T::BLOCKS, c = b * chunks<DT>() + i / T::BLOCKS;
          return Two{down.load(ld, n, c), down.load(lq, n, c)};
        };
        auto columns_ahead = read_first<2>(columns);
        const int base = i0 + 32 * b + 4 * half;
        const int from = low - base, to = high - base;
        auto seen = [&](int r) {
          const int i = r / 4 * 8 + r % 4;
          return (i >= from) & (i <= to);
        };
        if constexpr (has_cap(MODE)) score.cap_all(x);
        if (!has_cap(MODE) && !whole) {
#pragma unroll
          for (int r = 0; r < 16; ++r) x[0][r] = seen(r) ? x[0][r] : -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x4 lse = lse_in_sum<DT, MODE>() ? (f32x4){0.0f, 0.0f, 0.0f, 0.0f} : info(0, c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 4 * c + e;
            const float y = score.at(x[0][r], distance, -(32 * b + 8 * c + e));
            float p = score.weight(y, lse[e]);
            if (has_cap(MODE)) p = whole | seen(r) ? p : 0.0f;
            dp[r] = p * dp[r] * score.bend(x[0][r]);
            x[0][r] = p;
          }
        }
        u32x4 p[chunks<DT>()], d[chunks<DT>()];
#pragma unroll
        for (int c = 0; c < chunks<DT>(); ++c) {
          p[c] = pack_chunk<DT>(x[0], c);
          d[c] = pack_chunk<DT>(dp, c);
        }
        products<chunks<DT>() * T::BLOCKS, 2>(columns_ahead, columns, [&](int i, const Two& f) {
          const int n = i % T::BLOCKS, c = i / T::BLOCKS;
          dv[n] = mma<DT>(f.a, p[c], dv[n]);
          dk[n] = mma<DT>(f.b, d[c], dk[n]);
        });
      }
    };
    // one step: the tile in lq .. li, while the next one's loads run
    auto step = [&](char* lq, char* ld, char* li, char* nq, char* nd, char* ni, bool more) {
      wait_all();
      barrier();
      const int now = t;
      score.head(g, kv * g.group + in);
      if (++t == from + across) {
        t = from;
        ++in;
      }
      issue(nq, nd, ni, more);
      compute(lq, ld, li, now);
    };
    issue(lq0, ld0, li0, left > 0);
    for (; left > 1; left -= 2) {
      step(lq0, ld0, li0, lq1, ld1, li1, true);
      step(lq1, ld1, li1, lq0, ld0, li0, left > 2);
    }
    if (left > 0) step(lq0, ld0, li0, lq1, ld1, li1, false);
    wait_all();
    barrier();                                     // (the next item writes the buffers)
    if (g.k_parts > 1) {
      f32x4* to = part_at(g.k_sums, w.unit * g.k_parts + w.part, 2 * T::BLOCKS * 4);
      store_part(to, dk);
      store_part(to + T::BLOCKS * 4 * kAttnThreads, dv);
    } else if (mine) {
      store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dk.p)) + row * g.dk.row +
                            kv * g.dk.head, dk, g.scale, half, g.head_dim);
      store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dv.p)) + row * g.dv.row +
                            kv * g.dv.head, dv, 1.0f, half, g.head_dim);
    }
  }
}

// The parts' sums of dq, added in order; a workgroup 32 columns of a tile.
template <int DT, int D>
__device__ __forceinline__ void attn_dq_sum(const AttnArgs& g, int tiles, int64_t block, int64_t blocks) {
  constexpr int BLOCKS = D / 32;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Items items(tiles, g.kv_heads, g.group * BLOCKS);
  for (int64_t item = block; item < items.total; item += blocks) {
    const Queries w(g, items, item, tiles, BLOCKS);
    const int i = w.i0 + wave * 32 + lane % 32;
    if (!w.any || i >= w.q.lq) continue;
    f32x16 sum[1];
    clear(sum);
#pragma unroll 4
    for (int p = 0; p < g.q_parts; ++p)
      add_part(sum, part_at(g.q_sums, w.unit * g.q_parts + p, BLOCKS * 4) +
                        w.part * (4 * kAttnThreads), 1.0f);
    store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dq.p)) +
                          ((int64_t)w.q.q0 + i) * g.dq.row + w.head * g.dq.head, sum, g.scale,
                      lane / 32, g.head_dim, w.part);
  }
}

// The parts' sums, added in order; a workgroup 32 columns of a tile of dk or dv.
template <int DT, int D>
__device__ __forceinline__ void attn_dkv_sum(const AttnArgs& g, int tiles, int64_t block, int64_t blocks) {
  constexpr int BLOCKS = D / 32;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Items items(tiles, g.kv_heads, 2 * BLOCKS);
  for (int64_t item = block; item < items.total; item += blocks) {
    const Keys w(g, items, item, tiles);
    const int j = w.j0 + wave * 32 + lane % 32;
    if (!w.any || j >= w.q.lk) continue;
    f32x16 sum[1];
    clear(sum);
#pragma unroll 4
    for (int p = 0; p < g.k_parts; ++p)
      add_part(sum, part_at(g.k_sums, w.unit * g.k_parts + p, 2 * BLOCKS * 4) +
                        w.part * (4 * kAttnThreads), 1.0f);
    const bool is_dv = w.part >= BLOCKS;
    const AttnMatrix& to = is_dv ? g.dv : g.dk;
    store_columns<DT>(static_cast<char*>(const_cast<void*>(to.p)) +
                          ((int64_t)w.q.k0 + j) * to.row + w.kv * to.head, sum,
                      is_dv ? 1.0f : g.scale, lane / 32, g.head_dim, w.part % BLOCKS);
  }
}

// Both halves in one launch: neither waits for the other's last workgroups.  The first k_blocks
// workgroups, whose work is longer, take dk and dv.  Bound by the matrix units where they are
// full: 8 Ki tokens, causal, 32 / 8 heads of 128 bfloat16, 1590 us of the gradient's 1650 (in two launches
// 1680 to 1740), 1.21 PFLOP/s of the seven products, matrix units busy 64 % of the cycles, 0.1 % of
// LDS's in conflicts.  Five ragged documents 95 us (98), three binary32 sequences 93 (110).
template <int DT, int D, int MODE>
__global__ void __launch_bounds__(kAttnThreads, DT == kF32 && D > 64 ? 1 : 2)
    attn_back_kernel(AttnArgs g, int q_tiles, int k_tiles, int k_blocks) {
  using B = Back<DT, D>;
  __shared__ __attribute__((aligned(1024))) char l0[B::BYTES];
  __shared__ __attribute__((aligned(1024))) char l1[B::BYTES];
  __shared__ __attribute__((aligned(1024))) char l2[B::BYTES];
  __shared__ __attribute__((aligned(1024))) char l3[B::BYTES];
  __shared__ __attribute__((aligned(1024))) char li0[1024];  // lse, -D of 64 queries, twice
  __shared__ __attribute__((aligned(1024))) char li1[1024];
  __shared__ __attribute__((aligned(1024))) char values[B::APART ? kWaves * B::VALUES : 16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int)blockIdx.x >= k_blocks) {
    attn_dq<DT, D, MODE>(g, q_tiles, blockIdx.x - k_blocks, gridDim.x - k_blocks, l0, l1, l2, l3);
  } else if constexpr (B::KEEP || B::APART) {
    attn_dkv<DT, D, MODE>(g, k_tiles, blockIdx.x, k_blocks, l0, l1, li0, l2, l3, li1,
                          values + wave * (B::APART ? B::VALUES : 0));
  } else {
    static_assert(2 * B::Q_BYTES <= B::BYTES && 2 * B::VALUES <= B::BYTES, "");
    attn_dkv<DT, D, MODE>(g, k_tiles, blockIdx.x, k_blocks, l0, l0 + B::Q_BYTES, li0, l1,
                          l1 + B::Q_BYTES, li1, (wave < 2 ? l2 : l3) + wave % 2 * B::VALUES);
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kAttnThreads)
    attn_sum_kernel(AttnArgs g, int q_tiles, int k_tiles, int k_blocks) {
  if ((int)blockIdx.x >= k_blocks)
    attn_dq_sum<DT, D>(g, q_tiles, blockIdx.x - k_blocks, gridDim.x - k_blocks);
  else
    attn_dkv_sum<DT, D>(g, k_tiles, blockIdx.x, k_blocks);
}

template <int DT, int D, int MODE>
lowbit_status launch_back_width(const AttnArgs& a, hipStream_t s) {
  const int qt = attn_tiles(a.q_rows, a.sequences), kt = attn_tiles(a.k_rows, a.sequences);
  const int64_t nk = capped(Items(kt, a.kv_heads, a.k_parts).total);
  const int64_t nq = capped(Items(qt, a.kv_heads, a.group * a.q_parts).total);
  const lowbit_status st = launch(&attn_back_kernel<DT, D, MODE>, nk + nq, kAttnThreads, s, a, qt, kt,
                                  (int)nk);
  if (st != LOWBIT_OK || (a.k_parts == 1 && a.q_parts == 1)) return st;
  const int64_t sk = a.k_parts > 1 ? capped(Items(kt, a.kv_heads, 2 * (D / 32)).total) : 0;
  const int64_t sq = a.q_parts > 1 ? capped(Items(qt, a.kv_heads, a.group * (D / 32)).total) : 0;
  return launch(&attn_sum_kernel<DT, D>, sk + sq, kAttnThreads, s, a, qt, kt, (int)sk);
}

template <int DT, int MODE>
lowbit_status launch_back_mode(const AttnArgs& a, hipStream_t s) {
  return a.head_dim <= 64   ? launch_back_width<DT, 64, MODE>(a, s)
         : a.head_dim <= 96 ? launch_back_width<DT, 96, MODE>(a, s)
                            : launch_back_width<DT, 128, MODE>(a, s);
}

template <int DT>
lowbit_status launch_attn_back(const AttnArgs& a, hipStream_t s) {
  switch (score_mode(a)) {
    case kPlainScore: return launch_back_mode<DT, kPlainScore>(a, s);
    case kBiasScore: return launch_back_mode<DT, kBiasScore>(a, s);
    case kCapScore: return launch_back_mode<DT, kCapScore>(a, s);
    default: return launch_back_mode<DT, kCapBiasScore>(a, s);
  }
}

}  // namespace

}  // namespace lowbit
