// attn_back.hpp -- attention's gradient.
#pragma once

#include "attn.hpp"

namespace lowbit {

namespace {

// What a score is from the products' sum: y in units, and for capped scores what its
// slope is multiplied by (1 - tanh^2).
template <int DT, bool SHAPED>
struct Score {
  float factor, cap, slope;
  __device__ __forceinline__ Score(const AttnArgs& g, int head) {
    const float unit = unit_of<DT>();
    cap = SHAPED && g.softcap > 0.0f ? g.softcap * unit : 0.0f;
    factor = cap > 0.0f ? g.scale / g.softcap : g.scale * unit;
    slope = SHAPED && g.slopes ? g.slopes[head] * unit : 0.0f;
  }
  __device__ __forceinline__ float at(float x, int distance, float& bend) const {
    float y = x * factor;
    bend = 1.0f;
    if constexpr (SHAPED) {
      if (cap > 0.0f) {
        const float t = tanhf(y);
        bend = __builtin_fmaf(-t, t, 1.0f);
        y = cap * t;
      }
      y -= slope * fabsf((float)distance);
    }
    return y;
  }
};

// Rows of a result that lies as columns d by rows of lanes: 32 x D.
template <int DT, int BLOCKS>
__device__ __forceinline__ void store_columns(char* to, const f32x16 (&acc)[BLOCKS], float scale,
                                              int half, int head_dim) {
#pragma unroll
  for (int n = 0; n < BLOCKS; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = n * 32 + c * 8 + half * 4;
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = acc[n][4 * c + r] * scale;
      if (at < head_dim) {
        if constexpr (DT == kF32) *reinterpret_cast<f32x4*>(to + at * 4) = v;
        else *reinterpret_cast<u32x2*>(to + at * 2) =
                 (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      }
    }
}

// The operands along a row of one matrix, straight from memory.
template <int STEPS>
__device__ __forceinline__ void load_rows(u32x4 (&f)[STEPS], const void* base, int64_t at, int half,
                                          int width, bool any) {
  const char* p = static_cast<const char*>(base) + at;
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) {
    const int c = kk * 32 + half * 16;
    f[kk] = (u32x4){0, 0, 0, 0};
    if (any && c < width) f[kk] = *reinterpret_cast<const u32x4*>(p + c);
  }
}

// dq: four waves, each 32 queries, as in the forward pass; the scores and dout.v
// are taken again, transposed, and their gradient is, as it lies, the operand
// of the product with the keys.
template <int DT, int D, bool SHAPED>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_dq_kernel(AttnArgs g, int tiles) {
  constexpr int KT = DT == kF32 ? 32 : 64, NB = KT / 32, ES = elem_size<DT>();
  using T = Tile<DT, D, KT>;
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

  const Items items(tiles, g.kv_heads, g.group);
  for (int64_t item = blockIdx.x; item < items.total; item += gridDim.x) {
    int t, kv, in;
    items.take(item, g.kv_heads, t, kv, in);
    if (t >= tiles) continue;
    t = tiles - 1 - t;
    const int head = kv * g.group + in;
    const int s = find_sequence(g.q_begin, g.sequences, g.q_rows, kRowsPerTile, t);
    const Sequence q = sequence_at(g, s);
    const int i0 = (t - first_tile(g.q_begin, s, g.sequences, g.q_rows, kRowsPerTile)) * kRowsPerTile;
    if (i0 >= q.lq) continue;
    const int i = i0 + wave * 32 + col;
    const int shift = q.lk - q.lq;
    const bool mine = i < q.lq;
    const int64_t row = (int64_t)q.q0 + i;
    const Score<DT, SHAPED> score(g, head);

    u32x4 fq[T::STEPS], fdo[T::STEPS];
    load_rows(fq, g.q.p, row * g.q.row + head * g.q.head, half, width, mine);
    load_rows(fdo, g.dout.p, row * g.dout.row + head * g.dout.head, half, width, mine);
    float lse = 0.0f, delta = 0.0f;
    if (mine) {
      const float* info = g.rows_info + (int64_t)head * g.q_rows + row;
      lse = info[0];
      delta = info[(int64_t)g.q_heads * g.q_rows];
    }
    const Sight see = sight(g, q, i + shift);
    const int last = min(i0 + kRowsPerTile, q.lq) - 1;
    const Sight lo = sight(g, q, i0 + shift), hi = sight(g, q, last + shift);
    const int before = (q.prefix + KT - 1) / KT;
    const int from = lo.low > 0 ? lo.low / KT : 0;
    const int to = hi.high < 0 ? 0 : hi.high / KT + 1;
    const int end = max(before, to);
    auto after = [&](int t) { return t >= before && t < from ? from : t; };
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

    auto compute = [&](const char* lk, const char* lv, int t) {
      const int j0 = t * KT;
      const bool whole = (j0 + KT <= see.prefix) || (j0 >= wh.low && j0 + KT - 1 <= wl.high);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x16 x, dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = dp[r] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < T::STEPS; ++kk) {
          x = mma<DT>(along.load(lk, b, kk), fq[kk], x);
          dp = mma<DT>(along.load(lv, b, kk), fdo[kk], dp);
        }
        const int base = j0 + 32 * b + 4 * half;
        const int low = see.low - base, high = see.high - base, pre = see.prefix - base;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = r / 4 * 8 + r % 4;
          float bend;
          const float y = score.at(x[r], i + shift - base - j, bend);
          float p = exp_unit<DT>(y - lse) * (dp[r] - delta) * bend;
          if (!whole && !(j < pre || (j >= low && j <= high))) p = 0.0f;
          x[r] = p;
        }
#pragma unroll
        for (int c = 0; c < chunks<DT>(); ++c) {
          const u32x4 p = pack_chunk<DT>(x, c);
#pragma unroll
          for (int n = 0; n < T::BLOCKS; ++n)
            acc[n] = mma<DT>(down.load(lk, n, b * chunks<DT>() + c), p, acc[n]);
        }
      }
    };

    int now = after(0);
    if (now < end) issue(now, lk0, lv0);
    while (now < end) {
      wait_all();
      barrier();
      int next = after(now + 1);
      if (next < end) issue(next, lk1, lv1);
      compute(lk0, lv0, now);
      now = next;
      if (now >= end) break;
      wait_all();
      barrier();
      next = after(now + 1);
      if (next < end) issue(next, lk0, lv0);
      compute(lk1, lv1, now);
      now = next;
    }
    wait_all();
    barrier();
    if (mine)
      store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dq.p)) + row * g.dq.row +
                            head * g.dq.head, acc, g.scale, half, g.head_dim);
  }
}

// dk and dv: four waves, each 32 keys; the queries of every head that reads them
// pass by in tiles.  A key a lane and queries down the registers, so that the weights
// and the scores' gradient are operands as they lie here too.
template <int DT, int D, bool SHAPED>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_dkv_kernel(AttnArgs g, int tiles) {
  constexpr int QT = DT == kF32 ? 32 : 64, NB = QT / 32, ES = elem_size<DT>();
  using T = Tile<DT, D, QT>;
  __shared__ __attribute__((aligned(1024))) char lq0[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char ld0[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char lq1[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char ld1[T::BYTES];
  __shared__ __attribute__((aligned(1024))) char li0[512];   // lse, D of 64 queries
  __shared__ __attribute__((aligned(1024))) char li1[512];
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
  const int32_t* const kb = g.k_begin;

  const Items items(tiles, g.kv_heads, 1);
  for (int64_t item = blockIdx.x; item < items.total; item += gridDim.x) {
    int t, kv, in;
    items.take(item, g.kv_heads, t, kv, in);
    if (t >= tiles) continue;                      // causal: the first keys are seen by most
    const int s = find_sequence(kb, g.sequences, g.k_rows, kRowsPerTile, t);
    const Sequence q = sequence_at(g, s);
    const int j0 = (t - first_tile(kb, s, g.sequences, g.k_rows, kRowsPerTile)) * kRowsPerTile;
    if (j0 >= q.lk) continue;
    const int j = j0 + wave * 32 + col;            // the lane's key
    const int shift = q.lk - q.lq;
    const bool mine = j < q.lk;
    const int64_t row = (int64_t)q.k0 + j;

    u32x4 fk[T::STEPS], fv[T::STEPS];
    load_rows(fk, g.k.p, row * g.k.row + kv * g.k.head, half, width, mine);
    load_rows(fv, g.v.p, row * g.v.row + kv * g.v.head, half, width, mine);

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
    const int end = top < 0 ? 0 : top / QT + 1;
    // what all 32 keys of the wave are seen by
    const int w0 = j0 + wave * 32, w1 = min(w0 + 31, last);
    const int wlow = low_of(w1), whigh = high_of(max(w0, min(q.prefix, w1)));

    f32x16 dk[T::BLOCKS], dv[T::BLOCKS];
#pragma unroll
    for (int n = 0; n < T::BLOCKS; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) dk[n][r] = dv[n][r] = 0.0f;

    for (int in_group = 0; in_group < g.group; ++in_group) {
      const int head = kv * g.group + in_group;
      const Score<DT, SHAPED> score(g, head);
      const char* qp = static_cast<const char*>(g.q.p) + q.q0 * g.q.row + head * g.q.head;
      const char* dp_ = static_cast<const char*>(g.dout.p) + q.q0 * g.dout.row + head * g.dout.head;
      const float* info = g.rows_info + (int64_t)head * g.q_rows + q.q0;
      auto issue = [&](int t, char* lq, char* ld, char* li) {
        const int rows = q.lq - t * QT;
        const auto rq = load_q.rows_at(qp + (int64_t)t * QT * g.q.row, (int)g.q.row, width, rows);
        const auto rd = load_d.rows_at(dp_ + (int64_t)t * QT * g.dout.row, (int)g.dout.row, width, rows);
#pragma unroll
        for (int j = 0; j < T::LOADS; ++j) load_q.load(rq, lq, wave, j);
#pragma unroll
        for (int j = 0; j < T::LOADS; ++j) load_d.load(rd, ld, wave, j);
        if (wave < 2) {                            // lse, or D
          const float* p = info + (wave ? (int64_t)g.q_heads * g.q_rows : 0) + t * QT;
          const auto r = open(p, max(0, min(rows, 64)) * 4);
          load_floats(r, li + wave * 256, lane);
        }
      };
      auto compute = [&](const char* lq, const char* ld, const char* li, int t) {
        const int i0 = t * QT;
        const bool whole = i0 >= wlow && i0 + QT - 1 <= whigh;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          f32x16 x, dp;
#pragma unroll
          for (int r = 0; r < 16; ++r) x[r] = dp[r] = 0.0f;
#pragma unroll
          for (int kk = 0; kk < T::STEPS; ++kk) {
            x = mma<DT>(along.load(lq, b, kk), fk[kk], x);
            dp = mma<DT>(along.load(ld, b, kk), fv[kk], dp);
          }
          const int base = i0 + 32 * b + 4 * half;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const f32x4 lse = *reinterpret_cast<const f32x4*>(li + (32 * b + 8 * c + 4 * half) * 4);
            const f32x4 delta =
                *reinterpret_cast<const f32x4*>(li + 256 + (32 * b + 8 * c + 4 * half) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 4 * c + e, i = base + 8 * c + e;
              float bend;
              const float y = score.at(x[r], i + shift - j, bend);
              float p = exp_unit<DT>(y - lse[e]);
              float d = p * (dp[r] - delta[e]) * bend;
              if (!whole && !(i >= low && i <= high)) p = d = 0.0f;
              x[r] = p;
              dp[r] = d;
            }
          }
#pragma unroll
          for (int c = 0; c < chunks<DT>(); ++c) {
            const u32x4 p = pack_chunk<DT>(x, c), d = pack_chunk<DT>(dp, c);
#pragma unroll
            for (int n = 0; n < T::BLOCKS; ++n) {
              dv[n] = mma<DT>(down.load(ld, n, b * chunks<DT>() + c), p, dv[n]);
              dk[n] = mma<DT>(down.load(lq, n, b * chunks<DT>() + c), d, dk[n]);
            }
          }
        }
      };
      int now = from;
      if (now < end) issue(now, lq0, ld0, li0);
      while (now < end) {
        wait_all();
        barrier();
        if (now + 1 < end) issue(now + 1, lq1, ld1, li1);
        compute(lq0, ld0, li0, now);
        if (++now >= end) break;
        wait_all();
        barrier();
        if (now + 1 < end) issue(now + 1, lq0, ld0, li0);
        compute(lq1, ld1, li1, now);
        ++now;
      }
      wait_all();
      barrier();                                   // (the next head writes the buffers)
    }
    if (mine) {
      store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dk.p)) + row * g.dk.row +
                            kv * g.dk.head, dk, g.scale, half, g.head_dim);
      store_columns<DT>(static_cast<char*>(const_cast<void*>(g.dv.p)) + row * g.dv.row +
                            kv * g.dv.head, dv, 1.0f, half, g.head_dim);
    }
  }
}

template <int DT, int D, bool SHAPED>
lowbit_status launch_back_shaped(const AttnArgs& a, hipStream_t s) {
  const int qt = a.q_rows / kRowsPerTile + a.sequences, kt = a.k_rows / kRowsPerTile + a.sequences;
  const Items iq(qt, a.kv_heads, a.group), ik(kt, a.kv_heads, 1);
  const lowbit_status st = launch(&attn_dkv_kernel<DT, D, SHAPED>,
                                  ik.total < kMaxBlocks ? ik.total : kMaxBlocks, kAttnThreads, s, a, kt);
  if (st != LOWBIT_OK) return st;
  return launch(&attn_dq_kernel<DT, D, SHAPED>, iq.total < kMaxBlocks ? iq.total : kMaxBlocks,
                kAttnThreads, s, a, qt);
}

template <int DT>
lowbit_status launch_attn_back(const AttnArgs& a, hipStream_t s) {
  if (a.softcap > 0.0f || a.slopes)
    return a.head_dim <= 64 ? launch_back_shaped<DT, 64, true>(a, s)
                            : launch_back_shaped<DT, 128, true>(a, s);
  return a.head_dim <= 64 ? launch_back_shaped<DT, 64, false>(a, s)
                          : launch_back_shaped<DT, 128, false>(a, s);
}

}  // namespace

}  // namespace lowbit
