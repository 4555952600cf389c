// block join and its gradient
#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

// A run of consecutive rows is taken by `lanes` lanes (of a wave, or a whole
// workgroup), one row at a time, whole in registers: lane t holds NV vectors of
// eight columns, so that each row is read once for both norms and written
// once.  Its columns are the same in every row: the parameters are loaded
// once, and the backward kernel keeps their gradients' sums in registers over
// all its rows.
//
// Vector i of lane t begins at column 8 (t + i lanes), but never less than
// eight before the row's end: where the width is no multiple of 8 the last
// vector takes columns again that the one before it has, computes the same for
// them and stores the same, and only the row's sums leave them out (`own`).  So no
// load or store is ever cut, whatever the width and its alignment; only rows of
// fewer than eight columns are taken element by element.
//
// Bound by memory where a row takes whole waves: 16 Ki x 4096 bfloat16 with a gate and
// dropout 104 us, 5.2 TB/s (a copy: 5.1).  Short rows share a wave: with a
// wave each, 10287 x 48 took 86 us for its gradient, now 20.
struct Cols {
  int start;                        // column of element 0
  uint32_t own;                     // bit j: element j is this vector's
  __device__ __forceinline__ void init(int c, int cols) {
    start = cols < 8 ? 0 : c < cols - 8 ? c : cols - 8;
    const int skip = c - start;     // 0; less than 8 in the row's last vector; 8 or more behind it
    own = cols < 8 ? (c == 0 ? (1u << cols) - 1 : 0) : skip < 8 ? 0xFFu << skip & 0xFF : 0;
  }
};
// v where element j is the vector's own, else 0 (RAGGED: not all of them are).
template <bool RAGGED>
__device__ __forceinline__ float only(const Cols& c, int j, float v) {
  return !RAGGED || (c.own >> j & 1) ? v : 0.0f;
}

// TINY: the row may have fewer than eight columns.
template <int DT, int NV, bool TINY>
struct RowRaw {
  Raw8<DT> v[NV];
  __device__ __forceinline__ void load(const void* base, int64_t row, int cols, const Cols* c) {
    const char* p = static_cast<const char*>(base) + row * cols * elem_size<DT>();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!TINY || cols >= 8) {
        const char* q = p + (uint32_t)c[i].start * (uint32_t)elem_size<DT>();
        if constexpr (DT == kF32) {
          v[i].w[0] = reinterpret_cast<const u32x4_4*>(q)[0];
          v[i].w[1] = reinterpret_cast<const u32x4_4*>(q)[1];
        } else {
          v[i].w[0] = *reinterpret_cast<const u32x4_2*>(q);
        }
      } else {
        v[i] = load8<DT>(p, c[i].own ? 0 : 8, cols);
      }
    }
  }
  // an absent parameter: the same value everywhere
  __device__ __forceinline__ void load_or(const void* base, int64_t row, int cols, const Cols* c,
                                          float absent) {
    if (base) {
      load(base, row, cols, c);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i].fill(absent, absent);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t row, int cols, const Cols* c) const {
    char* p = static_cast<char*>(base) + row * cols * elem_size<DT>();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!c[i].own) continue;
      char* q = p + (uint32_t)c[i].start * (uint32_t)elem_size<DT>();
      if (TINY && cols < 8) {
        store8<DT>(p, 0, cols, v[i]);
      } else if constexpr (DT == kF32) {
        reinterpret_cast<u32x4_4*>(q)[0] = v[i].w[0];
        reinterpret_cast<u32x4_4*>(q)[1] = v[i].w[1];
      } else {
        *reinterpret_cast<u32x4_2*>(q) = v[i].w[0];
      }
    }
  }
  // The loads have arrived: where an output is the input itself, a wave's store may
  // not go before another's load of the columns that both take.  And what is computed
  // from the elements after this is computed anew, not kept in registers of its own.
  __device__ __forceinline__ void arrive() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < (DT == kF32 ? 2 : 1); ++k) asm volatile("" : "+v"(v[i].w[k]));
  }
};

// The draws of a vector's elements, two a word: element j's is the low (j even) or
// high half of w[j / 2].  With an odd width its first element can be the
// second of a pair.
struct Draws {
  uint32_t w[4];
  __device__ __forceinline__ void init(const HiMix& mix, int start, int cols) {
    const uint32_t q = (uint32_t)start / 2;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = draw_word(mix, q + k);
    if (cols & 1) {
      const uint32_t more = draw_word(mix, q + 4);
      if (start & 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = w[k] >> 16 | (k < 3 ? w[k + 1] : more) << 16;
      }
    }
  }
  __device__ __forceinline__ bool keeps(int j, uint32_t cut) const {
    return j % 2 ? keeps_hi(w[j / 2], cut) : keeps_lo(w[j / 2], cut);
  }
};

// Mean (LAYER) and 1 / sqrt(mean square + eps) of a row of values; v becomes
// the centred row.  The variance is summed over centred values, which loses
// nothing where the mean is large.  Calls in a row alternate the two slots.
template <int NV, bool LAYER, bool RAGGED, bool SUB>
__device__ __forceinline__ float2 row_stats(float (*v)[8], const Cols* c, float eps, float inv_cols,
                                            float* slot0, float* slot1, int lanes) {
  float mean = 0.0f;
  if constexpr (LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += only<RAGGED>(c[i], j, v[i][j]);
    row_sum<1, SUB>(s, slot0, lanes);
    mean = s[0] * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] -= mean;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = only<RAGGED>(c[i], j, v[i][j]);
      q[0] = __builtin_fmaf(x, x, q[0]);
    }
  row_sum<1, SUB>(q, LAYER ? slot1 : slot0, lanes);
  return {mean, 1.0f / __builtin_sqrtf(q[0] * inv_cols + eps)};
}

template <int FT, int ST, int PT, int NV, bool LAYER, int MAXT, bool RAGGED, bool SUB>
__global__ void __launch_bounds__(MAXT) join_kernel(JoinArgs a) {
  __shared__ float slots[64];
  const int cols = a.cols, lanes = a.lanes, lane = lanes > 64 ? threadIdx.x : threadIdx.x & (lanes - 1);
  // (SUB: several rows a wave; else the whole wave has the same)
  const int sub = SUB ? threadIdx.x / lanes
                  : lanes > 64 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t run = (int64_t)blockIdx.x * (lanes > 64 ? 1 : 256 / lanes) + sub;
  Cols c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i].init(8 * (lane + i * lanes), cols);
  const int64_t r0 = run * a.rows_per_run;
  const int64_t r1 = r0 + a.rows_per_run < a.rows ? r0 + a.rows_per_run : a.rows;
  if (r0 >= r1) return;
  const float inv_cols = 1.0f / (float)cols;
  const uint32_t row_pairs = (uint32_t)(cols + 1) / 2;

  RowRaw<PT, NV, SUB> post_w, post_b, pre_w, pre_b, gate;
  post_w.load_or(a.post_w, 0, cols, c, 1.0f);
  post_b.load_or(a.post_b, 0, cols, c, 0.0f);
  pre_w.load_or(a.pre_w, 0, cols, c, 1.0f);
  pre_b.load_or(a.pre_b, 0, cols, c, 0.0f);
  gate.load_or(nullptr, 0, cols, c, 1.0f);
  int64_t next_gate = a.gate ? r0 : a.rows;     // the row from which another gate holds

  RowRaw<FT, NV, SUB> f;
  RowRaw<ST, NV, SUB> x;
  f.load(a.f, r0, cols, c);
  x.load(a.x, r0, cols, c);
  for (int64_t row = r0; row < r1; ++row) {
    if (row >= next_gate) {
      const int64_t g = row / a.rows_per_gate;
      gate.load(a.gate, g, cols, c);
      next_gate = (g + 1) * a.rows_per_gate;
    }
    x.arrive();
    post_w.arrive();
    post_b.arrive();
    pre_w.arrive();
    pre_b.arrive();
    gate.arrive();
    float u[NV][8], y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] = f.v[i].get(j);
        y[i][j] = x.v[i].get(j) * a.scale;
      }
    if (row + 1 < r1) {                         // the next row is on its way meanwhile
      f.load(a.f, row + 1, cols, c);
      x.load(a.x, row + 1, cols, c);
    }
    const float2 st1 = row_stats<NV, LAYER, RAGGED, SUB>(u, c, a.eps, inv_cols, slots, slots + 32, lanes);
    const HiMix mix((uint64_t)row * row_pairs, a.key);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Draws draws;
      if (a.cut) draws.init(mix, c[i].start, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float w = __builtin_fmaf(u[i][j] * st1.y, post_w.v[i].get(j), post_b.v[i].get(j));
        if (a.cut) w = draws.keeps(j, a.cut) ? w * a.factor : 0.0f;
        y[i][j] = __builtin_fmaf(gate.v[i].get(j), w, y[i][j]);
      }
    }
    RowRaw<ST, NV, SUB> out;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) out.v[i].set2(j, y[i][j], y[i][j + 1]);
    out.store(a.x_out, row, cols, c);
    const float2 st2 = row_stats<NV, LAYER, RAGGED, SUB>(y, c, a.eps, inv_cols, LAYER ? slots : slots + 32,
                                            slots + 32, lanes);
    RowRaw<FT, NV, SUB> z;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        z.v[i].set2(j, __builtin_fmaf(y[i][j] * st2.y, pre_w.v[i].get(j), pre_b.v[i].get(j)),
                    __builtin_fmaf(y[i][j + 1] * st2.y, pre_w.v[i].get(j + 1), pre_b.v[i].get(j + 1)));
    z.store(a.z, row, cols, c);
    if (lane == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(st1.x, st1.y, st2.x, st2.y);
  }
}

template <int NV, bool SUB>
struct Acc {
  float v[NV][8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  }
  __device__ __forceinline__ void store(float* base, int64_t row, int cols, const Cols* c) const {
    RowRaw<kF32, NV, SUB> r;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) r.v[i].set2(j, v[i][j], v[i][j + 1]);
    r.store(base, row, cols, c);
  }
};

// With yh = (x_out - mean2) rstd2 and fh = (f - mean1) rstd1 (x_out as it was written: a
// bfloat16 stream's yh is off by its half step, 2^-8 relative; the row before it was
// rounded is kept nowhere):
//     dy = dx_out + rstd2 (q - yh <q yh> - [<q>]),      q = dz pre_weight
//     du = D(gate dy)                       (the mask redrawn)
//     df = rstd1 (s - fh <s fh> - [<s>]),               s = du post_weight
//     dx = a dy,  and per column  dgate += D(u) dy  (u = fh post_weight + post_bias),
//     dpost_weight += du fh, dpost_bias += du, dpre_weight += dz yh, dpre_bias += dz
// <.> the mean over the row, [.] only with LAYER.
// 16 Ki x 4096 bfloat16 takes 182 to 190 us a call, 4.2 to 4.4 TB/s, 8 of them for the
// sums of its partial rows: two waves a SIMD (the sums take 40 registers for each vector), two exchanges over the
// workgroup a row, vector ALU 46 % busy with 46 instructions an element.  At 128
// registers, for twice the waves, 27 spill: 264 us.
template <int FT, int ST, int PT, int NV, bool LAYER, int MAXT, bool RAGGED, bool SUB>
__global__ void __launch_bounds__(MAXT) join_back_kernel(JoinBackArgs b) {
  __shared__ float slots[64];
  const JoinArgs& a = b.j;
  const int cols = a.cols, lanes = a.lanes, lane = lanes > 64 ? threadIdx.x : threadIdx.x & (lanes - 1);
  // (SUB: several rows a wave; else the whole wave has the same)
  const int sub = SUB ? threadIdx.x / lanes
                  : lanes > 64 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t run = (int64_t)blockIdx.x * (lanes > 64 ? 1 : 256 / lanes) + sub;
  Cols c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i].init(8 * (lane + i * lanes), cols);
  const int64_t r0 = run * a.rows_per_run;
  const int64_t r1 = r0 + a.rows_per_run < a.rows ? r0 + a.rows_per_run : a.rows;
  const float inv_cols = 1.0f / (float)cols;
  const uint32_t row_pairs = (uint32_t)(cols + 1) / 2;

  RowRaw<PT, NV, SUB> post_w, post_b, pre_w, gate;
  post_w.load_or(a.post_w, 0, cols, c, 1.0f);
  post_b.load_or(a.post_b, 0, cols, c, 0.0f);
  pre_w.load_or(a.pre_w, 0, cols, c, 1.0f);
  gate.load_or(nullptr, 0, cols, c, 1.0f);
  int64_t next_gate = a.gate ? r0 : a.rows;
  Acc<NV, SUB> d_post_w, d_post_b, d_pre_w, d_pre_b, d_gate;
  d_post_w.zero();
  d_post_b.zero();
  d_pre_w.zero();
  d_pre_b.zero();
  d_gate.zero();

  // With one vector each of a row's four inputs is loaded as soon as the row before
  // it has been through with it, into the same registers.  (With two there are none
  // left for it: the sums alone take 80.)
  constexpr bool EARLY = NV == 1;
  RowRaw<FT, NV, SUB> f, dz;
  RowRaw<ST, NV, SUB> x, dxo;
  auto load = [&](int64_t row) {
    dz.load(b.dz, row, cols, c);
    x.load(a.x, row, cols, c);
    dxo.load(b.dx_out, row, cols, c);
  };
  if (EARLY && r0 < r1) {
    load(r0);
    f.load(a.f, r0, cols, c);
  }
  // (a row ahead, too: loads and stores are waited for in their order, so that a load
  // after a row's stores and before the next row's first use would wait for them)
  float4 st_next = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r0 < r1) st_next = *reinterpret_cast<const float4*>(a.stats + 4 * r0);
  for (int64_t row = r0; row < r1; ++row) {
    const bool more = EARLY && row + 1 < r1;
    if (!EARLY) {
      load(row);
      f.load(a.f, row, cols, c);
    }
    if (!EARLY) {                                  // (with one vector there is room for them as binary32)
      post_w.arrive();
      post_b.arrive();
      pre_w.arrive();
      gate.arrive();
    }
    const float4 st = st_next;
    if (row + 1 < r1) st_next = *reinterpret_cast<const float4*>(a.stats + 4 * (row + 1));
    if (row >= next_gate) {
      const int64_t g = row / a.rows_per_gate;
      gate.load(a.gate, g, cols, c);
      next_gate = (g + 1) * a.rows_per_gate;
    }
    // (with two vectors yh, q and fh are computed twice: one array of the row's and not four)
    auto yh = [&](int i, int j) { return (LAYER ? x.v[i].get(j) - st.z : x.v[i].get(j)) * st.w; };
    auto q2 = [&](int i, int j) { return dz.v[i].get(j) * pre_w.v[i].get(j); };
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = yh(i, j), q = only<RAGGED>(c[i], j, q2(i, j)), dzv = dz.v[i].get(j);
        s2[0] = __builtin_fmaf(q, only<RAGGED>(c[i], j, h), s2[0]);
        if constexpr (LAYER) s2[1] += q;
        d_pre_w.v[i][j] = __builtin_fmaf(dzv, h, d_pre_w.v[i][j]);
        d_pre_b.v[i][j] += dzv;
      }
    if (!EARLY) {
      dz.arrive();
      x.arrive();
    }
    dxo.arrive();
    row_sum<LAYER ? 2 : 1, SUB>(s2, slots, lanes);
    const float m2 = s2[0] * inv_cols, n2 = LAYER ? s2[1] * inv_cols : 0.0f;
    float dy[NV][8];
    RowRaw<ST, NV, SUB> dx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float q = __builtin_fmaf(-yh(i, j), m2, q2(i, j));
        if constexpr (LAYER) q -= n2;
        dy[i][j] = __builtin_fmaf(q, st.w, dxo.v[i].get(j));
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) dx.v[i].set2(j, dy[i][j] * a.scale, dy[i][j + 1] * a.scale);
    }
    if (more) load(row + 1);
    dx.store(b.dx, row, cols, c);

    const HiMix mix((uint64_t)row * row_pairs, a.key);
    float s1[2] = {0.0f, 0.0f};
    auto fh = [&](int i, int j) { return (LAYER ? f.v[i].get(j) - st.x : f.v[i].get(j)) * st.y; };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Draws draws;
      if (a.cut) draws.init(mix, c[i].start, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool keep = !a.cut || draws.keeps(j, a.cut);
        const float h = fh(i, j);
        const float w = post_w.v[i].get(j);
        const float u = __builtin_fmaf(h, w, post_b.v[i].get(j));
        // a select, not a product: what stands in a dropped place does not matter
        const float dk = keep ? dy[i][j] * (a.cut ? a.factor : 1.0f) : 0.0f;
        const float du = keep ? dk * gate.v[i].get(j) : 0.0f;
        d_gate.v[i][j] = keep ? __builtin_fmaf(dk, u, d_gate.v[i][j]) : d_gate.v[i][j];
        d_post_w.v[i][j] = __builtin_fmaf(du, h, d_post_w.v[i][j]);
        d_post_b.v[i][j] += du;
        dy[i][j] = du * w;                         // s from here on
        const float q = only<RAGGED>(c[i], j, dy[i][j]);
        s1[0] = __builtin_fmaf(q, only<RAGGED>(c[i], j, h), s1[0]);
        if constexpr (LAYER) s1[1] += q;
      }
    }
    if (!EARLY) f.arrive();
    row_sum<LAYER ? 2 : 1, SUB>(s1, slots + 32, lanes);
    const float m1 = s1[0] * inv_cols, n1 = LAYER ? s1[1] * inv_cols : 0.0f;
    auto back = [&](int i, int j) {
      const float v = __builtin_fmaf(-fh(i, j), m1, dy[i][j]);
      return (LAYER ? v - n1 : v) * st.y;
    };
    RowRaw<FT, NV, SUB> df;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        df.v[i].set2(j, back(i, j), back(i, j + 1));
    if (more) f.load(a.f, row + 1, cols, c);
    df.store(b.df, row, cols, c);

    if (a.gate && b.dgate && (row + 1 == next_gate || row + 1 == r1)) {
      const int64_t g = row / a.rows_per_gate, g0 = g * a.rows_per_gate;
      const int64_t g1 = next_gate < a.rows ? next_gate : a.rows;
      if (g0 >= r0 && g1 <= r1)                                 // all its rows were this run's
        d_gate.store(b.dgate, g, cols, c);
      else
        d_gate.store(b.part_gate, 2 * run + (g0 >= r0 ? 1 : 0), cols, c);
      d_gate.zero();
    }
  }
  // (without rows of its own, a run adds zeros)
  float* const part[4] = {b.part_post_w, b.part_post_b, b.part_pre_w, b.part_pre_b};
  const Acc<NV, SUB>* const sums[4] = {&d_post_w, &d_post_b, &d_pre_w, &d_pre_b};
  __shared__ float lds[NV == 1 ? 256 * 8 : 1];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if (!part[p]) continue;
    if (NV == 1 && lanes <= 64) {    // the workgroup's runs, added in order
#pragma unroll
      for (int j = 0; j < 8; ++j) lds[threadIdx.x * 8 + j] = sums[p]->v[0][j];
      __syncthreads();
      if ((int)threadIdx.x < lanes) {
        Acc<NV, SUB> all = *sums[p];
        for (int t = threadIdx.x + lanes; t < 256; t += lanes)
#pragma unroll
          for (int j = 0; j < 8; ++j) all.v[0][j] += lds[t * 8 + j];
        all.store(part[p], blockIdx.x, cols, c);
      }
      __syncthreads();
    } else {
      sums[p]->store(part[p], blockIdx.x, cols, c);
    }
  }
}

// The sums of partial rows.  blockIdx.y: which of the parameters, or, from
// `params` on, a group of the gate, or sixteen groups where they have few partial
// rows each.  A workgroup takes 64 columns, its waves every sixteenth partial row (or a
// group each), and the waves' sums are added in order.
__global__ void __launch_bounds__(1024) join_sum_kernel(JoinSumArgs a, int64_t groups, int by_wave) {
  __shared__ float part[16][64];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const int64_t units = a.params + (by_wave ? (groups + 15) / 16 : groups);
  for (int64_t unit = blockIdx.y; unit < units; unit += gridDim.y) {
    const bool alone = by_wave && unit >= a.params;             // each wave by itself
    const float* src;
    float* out;
    int64_t b0 = 0, b1 = a.blocks, g = -1;
    if (unit < a.params) {
      src = a.part[unit];
      out = a.out[unit];
    } else {
      g = unit - a.params;
      if (alone) g = 16 * g + wave;
      if (g >= groups) continue;                                // (only waves by themselves)
      src = a.part_gate;
      out = a.dgate + g * a.cols;
      const int64_t g0 = g * a.rows_per_gate;
      const int64_t g1 = g0 + a.rows_per_gate < a.rows ? g0 + a.rows_per_gate : a.rows;
      b0 = g0 / a.rows_per_run;
      b1 = (g1 - 1) / a.rows_per_run + 1;
      if (b1 - b0 == 1) continue;                               // written by that run
    }
    float s = 0.0f;
    if (c < a.cols) {
      // a gate's group: the run's second partial row where it begins after the run's first row
      auto at = [&](int64_t b) {
        return g < 0 ? b : 2 * b + (g * a.rows_per_gate >= b * a.rows_per_run ? 1 : 0);
      };
      const int64_t step = alone ? 1 : 16;
      int64_t b = alone ? b0 : b0 + wave;
      for (; b + 7 * step < b1; b += 8 * step) {                // eight loads under way
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = src[at(b + step * k) * a.cols + c];
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
      }
      for (; b < b1; b += step) s += src[at(b) * a.cols + c];
    }
    if (alone) {
      if (c < a.cols) out[c] = s;
      continue;
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < a.cols) {
      for (int w = 1; w < 16; ++w) s += part[w][lane];
      out[c] = s;
    }
    __syncthreads();
  }
}

template <int FT, int ST, int PT, bool LAYER>
lowbit_status join_types(const JoinShape& g, const JoinArgs& a, hipStream_t s) {
  auto go = [&](auto* k) { return launch(k, g.blocks, g.threads, s, a); };
  if (g.threads > 512) return go(&join_kernel<FT, ST, PT, 2, LAYER, 1024, true, false>);
  if (g.lanes < 64) return go(&join_kernel<FT, ST, PT, 1, LAYER, 256, true, true>);
  if (g.vecs == 2)
    return g.ragged ? go(&join_kernel<FT, ST, PT, 2, LAYER, 512, true, false>)
                    : go(&join_kernel<FT, ST, PT, 2, LAYER, 512, false, false>);
  return g.ragged ? go(&join_kernel<FT, ST, PT, 1, LAYER, 256, true, false>)
                  : go(&join_kernel<FT, ST, PT, 1, LAYER, 256, false, false>);
}

template <int FT, int ST, int PT, bool LAYER>
lowbit_status join_back_types(const JoinShape& g, const JoinBackArgs& a, hipStream_t s) {
  auto go = [&](auto* k) { return launch(k, g.blocks, g.threads, s, a); };
  if (g.threads > 512) return go(&join_back_kernel<FT, ST, PT, 2, LAYER, 1024, true, false>);
  if (g.lanes < 64) return go(&join_back_kernel<FT, ST, PT, 1, LAYER, 256, true, true>);
  if (g.vecs == 2)
    return g.ragged ? go(&join_back_kernel<FT, ST, PT, 2, LAYER, 512, true, false>)
                    : go(&join_back_kernel<FT, ST, PT, 2, LAYER, 512, false, false>);
  return g.ragged ? go(&join_back_kernel<FT, ST, PT, 1, LAYER, 512, true, false>)
                  : go(&join_back_kernel<FT, ST, PT, 1, LAYER, 512, false, false>);
}

// block, residual stream and parameters' types
template <typename F>
lowbit_status by_types(int ft, int st, int pt, F go) {
  using B = std::integral_constant<int, kBF16>;
  using S = std::integral_constant<int, kF32>;
  if (ft == kF32) return go(S(), S(), S());
  if (st == kF32) return pt == kF32 ? go(B(), S(), S()) : go(B(), S(), B());
  return pt == kF32 ? go(B(), B(), S()) : go(B(), B(), B());
}

}  // namespace

// Lanes for one vector each, up to a wave; beyond it whole waves, and two vectors
// each beyond 2048 columns (gradient: 4096).
JoinShape join_shape(int64_t rows, int cols, bool backward) {
  JoinShape g;
  const int vectors = (cols + 7) / 8;
  g.lanes = 8;
  while (g.lanes < 64 && g.lanes < vectors) g.lanes *= 2;
  g.vecs = vectors > (backward ? 512 : 256) ? 2 : 1;
  if (g.lanes < vectors) g.lanes = (vectors + 64 * g.vecs - 1) / (64 * g.vecs) * 64;
  // (one workgroup of the gradient's with two vectors fits a CU: eight waves with a
  // vector and a half each are faster than six with two, 90 against 103 us for 3018 x 6056)
  if (backward && g.vecs == 2 && g.lanes < 512) g.lanes = 512;
  g.ragged = cols != 8 * g.lanes * g.vecs;
  g.threads = g.lanes <= 64 ? 256 : g.lanes;
  // runs: forward for several rounds of what the chip holds, which then ends evenly
  // (16 Ki x 4096 bfloat16 in runs for 1024, 2048 and 4096 lanes a CU: 115.6, 110 and
  // 104 us), but not a row each, which loads the parameters for every row (weights
  // and biases in binary32: 128 against 103 us; one bfloat16 weight: 97 against 103);
  // for the gradient one round, as every run leaves partial sums behind (2048
  // lanes a CU: 191 against 186 us)
  const int64_t most = (int64_t)256 * (backward ? 1024 : 4096) / (g.lanes < 64 ? 64 : g.lanes);
  g.rows_per_run = rows > most ? (rows + most - 1) / most : 1;
  if (backward) {
    // and four rows a run where that leaves one for each CU: partial sums of every
    // second row are half as much to write as the rows' own gradients
    const int64_t four = rows >= 1024 ? 4 : (rows + 255) / 256;
    if (g.rows_per_run < four) g.rows_per_run = four;
  }
  g.runs = (rows + g.rows_per_run - 1) / g.rows_per_run;
  const int64_t each = g.threads / g.lanes;
  g.blocks = (g.runs + each - 1) / each;
  return g;
}

lowbit_status launch_join(int ft, int st, int pt, bool layer, const JoinShape& g,
                          const JoinArgs& a, hipStream_t s) {
  return by_types(ft, st, pt, [&](auto f, auto x, auto p) {
    return layer ? join_types<f.value, x.value, p.value, true>(g, a, s)
                 : join_types<f.value, x.value, p.value, false>(g, a, s);
  });
}

lowbit_status launch_join_back(int ft, int st, int pt, bool layer, const JoinShape& g,
                               const JoinBackArgs& a, hipStream_t s) {
  return by_types(ft, st, pt, [&](auto f, auto x, auto p) {
    return layer ? join_back_types<f.value, x.value, p.value, true>(g, a, s)
                 : join_back_types<f.value, x.value, p.value, false>(g, a, s);
  });
}

lowbit_status launch_join_sums(const JoinSumArgs& a, hipStream_t s) {
  // no group of a gate lies in two workgroups' rows: all were written there
  const bool whole = !a.dgate || a.rows_per_run % a.rows_per_gate == 0;
  const int64_t groups = whole ? 0 : (a.rows + a.rows_per_gate - 1) / a.rows_per_gate;
  // up to 32 partial rows a wave sums as fast as sixteen waves do with their barrier
  int by_wave = groups > 0 && a.rows_per_gate / a.rows_per_run <= 32;
  const int64_t units = a.params + (by_wave ? (groups + 15) / 16 : groups);
  if (units == 0) return LOWBIT_OK;
  const dim3 grid((a.cols + 63) / 64, (uint32_t)(units < 4096 ? units : 4096));
  JoinSumArgs copy = a;
  int64_t g = groups;
  void* argv[] = {&copy, &g, &by_wave};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&join_sum_kernel), grid,
                                       dim3(1024), argv, 0, s);
  return e == hipSuccess ? LOWBIT_OK : LOWBIT_EDEVICE;
}

}  // namespace lowbit
