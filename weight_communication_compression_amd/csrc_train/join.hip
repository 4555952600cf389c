// block join and its gradient
#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

// A workgroup takes consecutive rows, one at a time, whole in registers: thread
// t holds columns 8 (t + v T) .. + 7 for v < NV, so that each row is read once
// for both norms and written once.  Its columns are the same in every row: the
// parameters are loaded once, and the backward kernel keeps their gradients'
// sums in registers over all its rows.
template <int DT, int NV>
struct RowRaw {
  Raw8<DT> v[NV];
  __device__ __forceinline__ void load(const void* base, int64_t row, int cols, int c0, int step) {
    const char* p = static_cast<const char*>(base) + row * cols * elem_size<DT>();
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = load8<DT>(p, c0 + i * step, cols);
  }
  // an absent parameter: the same value everywhere
  __device__ __forceinline__ void load_or(const void* base, int64_t row, int cols, int c0,
                                          int step, float absent) {
    if (base) {
      load(base, row, cols, c0, step);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i].fill(absent, absent);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t row, int cols, int c0, int step) const {
    char* p = static_cast<char*>(base) + row * cols * elem_size<DT>();
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<DT>(p, c0 + i * step, cols, v[i]);
  }
};

// Mean (LAYER) and 1 / sqrt(mean square + eps) of a row of values; v becomes
// the centred row.  The variance is summed over centred values, which loses
// nothing where the mean is large.  Calls in a row alternate the two slots.
template <int NV, bool LAYER>
__device__ __forceinline__ float2 row_stats(float (*v)[8], int c0, int step, int cols, float eps,
                                            float inv_cols, float* slot0, float* slot1,
                                            int waves) {
  float mean = 0.0f;
  if constexpr (LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += v[i][j];
    block_sum<1>(s, slot0, waves);
    mean = s[0] * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = c0 + i * step + j < cols ? v[i][j] - mean : 0.0f;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(v[i][j], v[i][j], q[0]);
  block_sum<1>(q, LAYER ? slot1 : slot0, waves);
  return {mean, 1.0f / __builtin_sqrtf(q[0] * inv_cols + eps)};
}

template <int FT, int ST, int PT, int NV, bool LAYER, int MAXT>
__global__ void __launch_bounds__(MAXT) join_kernel(JoinArgs a) {
  __shared__ float slots[64];
  const int cols = a.cols, T = blockDim.x, waves = T >> 6;
  const int c0 = 8 * threadIdx.x, step = 8 * T;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_block;
  const int64_t r1 = r0 + a.rows_per_block < a.rows ? r0 + a.rows_per_block : a.rows;
  if (r0 >= r1) return;
  const float inv_cols = 1.0f / (float)cols;
  const uint32_t row_pairs = (uint32_t)(cols + 1) / 2;

  RowRaw<PT, NV> post_w, post_b, pre_w, pre_b, gate;
  post_w.load_or(a.post_w, 0, cols, c0, step, 1.0f);
  post_b.load_or(a.post_b, 0, cols, c0, step, 0.0f);
  pre_w.load_or(a.pre_w, 0, cols, c0, step, 1.0f);
  pre_b.load_or(a.pre_b, 0, cols, c0, step, 0.0f);
  gate.load_or(nullptr, 0, cols, c0, step, 1.0f);
  int64_t next_gate = a.gate ? r0 : a.rows;     // the row from which another gate holds

  RowRaw<FT, NV> f;
  RowRaw<ST, NV> x;
  f.load(a.f, r0, cols, c0, step);
  x.load(a.x, r0, cols, c0, step);
  for (int64_t row = r0; row < r1; ++row) {
    if (row >= next_gate) {
      const int64_t g = row / a.rows_per_gate;
      gate.load(a.gate, g, cols, c0, step);
      next_gate = (g + 1) * a.rows_per_gate;
    }
    float u[NV][8], y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] = f.v[i].get(j);
        y[i][j] = x.v[i].get(j) * a.scale;
      }
    if (row + 1 < r1) {                         // the next row is on its way meanwhile
      f.load(a.f, row + 1, cols, c0, step);
      x.load(a.x, row + 1, cols, c0, step);
    }
    const float2 st1 = row_stats<NV, LAYER>(u, c0, step, cols, a.eps, inv_cols, slots, slots + 32,
                                             waves);
    const HiMix mix((uint64_t)row * row_pairs, a.key);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float w0 = __builtin_fmaf(u[i][j] * st1.y, post_w.v[i].get(j), post_b.v[i].get(j));
        float w1 = __builtin_fmaf(u[i][j + 1] * st1.y, post_w.v[i].get(j + 1), post_b.v[i].get(j + 1));
        if (a.cut) {
          const uint32_t word = draw_word(mix, (uint32_t)(c0 + i * step + j) / 2);
          w0 = keeps_lo(word, a.cut) ? w0 * a.factor : 0.0f;
          w1 = keeps_hi(word, a.cut) ? w1 * a.factor : 0.0f;
        }
        y[i][j] = __builtin_fmaf(gate.v[i].get(j), w0, y[i][j]);
        y[i][j + 1] = __builtin_fmaf(gate.v[i].get(j + 1), w1, y[i][j + 1]);
      }
    RowRaw<ST, NV> out;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) out.v[i].set2(j, y[i][j], y[i][j + 1]);
    out.store(a.x_out, row, cols, c0, step);
    const float2 st2 = row_stats<NV, LAYER>(y, c0, step, cols, a.eps, inv_cols,
                                            LAYER ? slots : slots + 32, slots + 32, waves);
    RowRaw<FT, NV> z;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        z.v[i].set2(j, __builtin_fmaf(y[i][j] * st2.y, pre_w.v[i].get(j), pre_b.v[i].get(j)),
                    __builtin_fmaf(y[i][j + 1] * st2.y, pre_w.v[i].get(j + 1), pre_b.v[i].get(j + 1)));
    z.store(a.z, row, cols, c0, step);
    if (threadIdx.x == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(st1.x, st1.y, st2.x, st2.y);
  }
}

template <int NV>
struct Acc {
  float v[NV][8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  }
  __device__ __forceinline__ void store(float* base, int64_t row, int cols, int c0, int step) const {
    RowRaw<kF32, NV> r;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) r.v[i].set2(j, v[i][j], v[i][j + 1]);
    r.store(base, row, cols, c0, step);
  }
};

// With yh = (x_out - mean2) rstd2 and fh = (f - mean1) rstd1:
//     dy = dx_out + rstd2 (q - yh <q yh> - [<q>]),      q = dz pre_weight
//     du = D(gate dy)                       (the mask redrawn)
//     df = rstd1 (s - fh <s fh> - [<s>]),               s = du post_weight
//     dx = a dy,  and per column  dgate += D(u) dy  (u = fh post_weight + post_bias),
//     dpost_weight += du fh, dpost_bias += du, dpre_weight += dz yh, dpre_bias += dz
// <.> the mean over the row, [.] only with LAYER.
template <int FT, int ST, int PT, int NV, bool LAYER, int MAXT>
__global__ void __launch_bounds__(MAXT) join_back_kernel(JoinBackArgs b) {
  __shared__ float slots[64];
  const JoinArgs& a = b.j;
  const int cols = a.cols, T = blockDim.x, waves = T >> 6;
  const int c0 = 8 * threadIdx.x, step = 8 * T;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_block;
  const int64_t r1 = r0 + a.rows_per_block < a.rows ? r0 + a.rows_per_block : a.rows;
  if (r0 >= r1) return;
  const float inv_cols = 1.0f / (float)cols;
  const uint32_t row_pairs = (uint32_t)(cols + 1) / 2;

  RowRaw<PT, NV> post_w, post_b, pre_w, gate;
  post_w.load_or(a.post_w, 0, cols, c0, step, 1.0f);
  post_b.load_or(a.post_b, 0, cols, c0, step, 0.0f);
  pre_w.load_or(a.pre_w, 0, cols, c0, step, 1.0f);
  gate.load_or(nullptr, 0, cols, c0, step, 1.0f);
  int64_t next_gate = a.gate ? r0 : a.rows;
  Acc<NV> d_post_w, d_post_b, d_pre_w, d_pre_b, d_gate;
  d_post_w.zero();
  d_post_b.zero();
  d_pre_w.zero();
  d_pre_b.zero();
  d_gate.zero();

  for (int64_t row = r0; row < r1; ++row) {
    RowRaw<FT, NV> f, dz;
    RowRaw<ST, NV> x, dxo;
    f.load(a.f, row, cols, c0, step);
    dz.load(b.dz, row, cols, c0, step);
    x.load(a.x, row, cols, c0, step);
    dxo.load(b.dx_out, row, cols, c0, step);
    const float4 st = *reinterpret_cast<const float4*>(a.stats + 4 * row);
    if (row >= next_gate) {
      const int64_t g = row / a.rows_per_gate;
      gate.load(a.gate, g, cols, c0, step);
      next_gate = (g + 1) * a.rows_per_gate;
    }
    float yh[NV][8], dy[NV][8];
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dzv = dz.v[i].get(j);                       // 0 beyond the row
        yh[i][j] = (x.v[i].get(j) - st.z) * st.w;
        const float q = dzv * pre_w.v[i].get(j);
        s2[0] = __builtin_fmaf(q, yh[i][j], s2[0]);
        if constexpr (LAYER) s2[1] += q;
        d_pre_w.v[i][j] = __builtin_fmaf(dzv, yh[i][j], d_pre_w.v[i][j]);
        d_pre_b.v[i][j] += dzv;
        dy[i][j] = q;
      }
    block_sum<LAYER ? 2 : 1>(s2, slots, waves);
    const float m2 = s2[0] * inv_cols, n2 = LAYER ? s2[1] * inv_cols : 0.0f;
    RowRaw<ST, NV> dx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = __builtin_fmaf(-yh[i][j], m2, dy[i][j]) - n2;
        dy[i][j] = __builtin_fmaf(q, st.w, dxo.v[i].get(j));
        if (LAYER && c0 + i * step + j >= cols) dy[i][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) dx.v[i].set2(j, dy[i][j] * a.scale, dy[i][j + 1] * a.scale);
    }
    dx.store(b.dx, row, cols, c0, step);

    const HiMix mix((uint64_t)row * row_pairs, a.key);
    float s1[2] = {0.0f, 0.0f};
    float fh[NV][8], s[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float k0 = 1.0f, k1 = 1.0f;                             // what the mask multiplies by
        if (a.cut) {
          const uint32_t word = draw_word(mix, (uint32_t)(c0 + i * step + j) / 2);
          k0 = keeps_lo(word, a.cut) ? a.factor : 0.0f;
          k1 = keeps_hi(word, a.cut) ? a.factor : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = j + e;
          const float k = e ? k1 : k0;
          const float h = (f.v[i].get(c) - st.x) * st.y;
          const float w = post_w.v[i].get(c);
          const float u = __builtin_fmaf(h, w, post_b.v[i].get(c));
          // a select, not a product: what stands in a dropped place does not matter
          const float dk = k != 0.0f ? dy[i][c] * k : 0.0f;
          const float du = k != 0.0f ? dk * gate.v[i].get(c) : 0.0f;
          d_gate.v[i][c] = k != 0.0f ? __builtin_fmaf(dk, u, d_gate.v[i][c]) : d_gate.v[i][c];
          d_post_w.v[i][c] = __builtin_fmaf(du, h, d_post_w.v[i][c]);
          d_post_b.v[i][c] += du;
          const float q = du * w;
          s1[0] = __builtin_fmaf(q, h, s1[0]);
          if constexpr (LAYER) s1[1] += q;
          fh[i][c] = h;
          s[i][c] = q;
        }
      }
    block_sum<LAYER ? 2 : 1>(s1, slots + 32, waves);
    const float m1 = s1[0] * inv_cols, n1 = LAYER ? s1[1] * inv_cols : 0.0f;
    RowRaw<FT, NV> df;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        df.v[i].set2(j, (__builtin_fmaf(-fh[i][j], m1, s[i][j]) - n1) * st.y,
                     (__builtin_fmaf(-fh[i][j + 1], m1, s[i][j + 1]) - n1) * st.y);
    df.store(b.df, row, cols, c0, step);

    if (a.gate && b.dgate && (row + 1 == next_gate || row + 1 == r1)) {
      const int64_t g = row / a.rows_per_gate, g0 = g * a.rows_per_gate;
      const int64_t g1 = next_gate < a.rows ? next_gate : a.rows;
      if (g0 >= r0 && g1 <= r1)                                 // all its rows were this workgroup's
        d_gate.store(b.dgate, g, cols, c0, step);
      else
        d_gate.store(b.part_gate, 2 * (int64_t)blockIdx.x + (g0 >= r0 ? 1 : 0), cols, c0, step);
      d_gate.zero();
    }
  }
  if (b.part_post_w) d_post_w.store(b.part_post_w, blockIdx.x, cols, c0, step);
  if (b.part_post_b) d_post_b.store(b.part_post_b, blockIdx.x, cols, c0, step);
  if (b.part_pre_w) d_pre_w.store(b.part_pre_w, blockIdx.x, cols, c0, step);
  if (b.part_pre_b) d_pre_b.store(b.part_pre_b, blockIdx.x, cols, c0, step);
}

// The sums of the workgroups' partial rows.  blockIdx.y: which of the parameters, or, from
// `params` on, which group of the gate; a workgroup takes 64 columns, its
// waves every sixteenth partial row, and the waves' sums are added in order.
__global__ void __launch_bounds__(1024) join_sum_kernel(JoinSumArgs a, int64_t groups) {
  __shared__ float part[16][64];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  for (int64_t what = blockIdx.y; what < a.params + groups; what += gridDim.y) {
    const float* src;
    float* out;
    int64_t b0 = 0, b1 = a.blocks, g = -1;
    if (what < a.params) {
      src = a.part[what];
      out = a.out[what];
    } else {
      g = what - a.params;
      src = a.part_gate;
      out = a.dgate + g * a.cols;
      const int64_t g0 = g * a.rows_per_gate;
      const int64_t g1 = g0 + a.rows_per_gate < a.rows ? g0 + a.rows_per_gate : a.rows;
      b0 = g0 / a.rows_per_block;
      b1 = (g1 - 1) / a.rows_per_block + 1;
      if (b1 - b0 == 1) continue;                               // written by that workgroup
    }
    float s = 0.0f;
    if (c < a.cols) {
      for (int64_t b = b0 + wave; b < b1; b += 16) {
        // a gate's group: the second partial row where it begins after the workgroup's first row
        const int64_t row = g < 0 ? b : 2 * b + (g * a.rows_per_gate >= b * a.rows_per_block ? 1 : 0);
        s += src[row * a.cols + c];
      }
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

template <int FT, int ST, int PT>
lowbit_status join_types(bool layer, const JoinShape& g, const JoinArgs& a, hipStream_t s) {
  auto go = [&](auto* rms, auto* centred) {
    return launch(layer ? centred : rms, g.blocks, g.threads, s, a);
  };
  if (g.threads > 512)
    return go(&join_kernel<FT, ST, PT, 2, false, 1024>, &join_kernel<FT, ST, PT, 2, true, 1024>);
  if (g.vecs == 2)
    return go(&join_kernel<FT, ST, PT, 2, false, 512>, &join_kernel<FT, ST, PT, 2, true, 512>);
  return go(&join_kernel<FT, ST, PT, 1, false, 512>, &join_kernel<FT, ST, PT, 1, true, 512>);
}

template <int FT, int ST, int PT>
lowbit_status join_back_types(bool layer, const JoinShape& g, const JoinBackArgs& a, hipStream_t s) {
  auto go = [&](auto* rms, auto* centred) {
    return launch(layer ? centred : rms, g.blocks, g.threads, s, a);
  };
  if (g.threads > 512)
    return go(&join_back_kernel<FT, ST, PT, 2, false, 1024>, &join_back_kernel<FT, ST, PT, 2, true, 1024>);
  if (g.vecs == 2)
    return go(&join_back_kernel<FT, ST, PT, 2, false, 512>, &join_back_kernel<FT, ST, PT, 2, true, 512>);
  return go(&join_back_kernel<FT, ST, PT, 1, false, 512>, &join_back_kernel<FT, ST, PT, 1, true, 512>);
}

}  // namespace

JoinShape join_shape(int64_t rows, int cols, bool backward) {
  JoinShape g;
  const int vectors = (cols + 7) / 8;
  g.threads = 64;
  while (g.threads < 256 && g.threads < vectors) g.threads *= 2;
  while (2 * g.threads < vectors) g.threads *= 2;
  g.vecs = g.threads < vectors ? 2 : 1;
  const int64_t most = (int64_t)256 * (backward ? 1024 : 2048) / g.threads;
  g.rows_per_block = rows > most ? (rows + most - 1) / most : 1;
  g.blocks = (rows + g.rows_per_block - 1) / g.rows_per_block;
  return g;
}

lowbit_status launch_join(int ft, int st, int pt, bool layer, const JoinShape& g,
                          const JoinArgs& a, hipStream_t s) {
  if (ft == kF32) return join_types<kF32, kF32, kF32>(layer, g, a, s);
  if (st == kF32)
    return pt == kF32 ? join_types<kBF16, kF32, kF32>(layer, g, a, s)
                      : join_types<kBF16, kF32, kBF16>(layer, g, a, s);
  return pt == kF32 ? join_types<kBF16, kBF16, kF32>(layer, g, a, s)
                    : join_types<kBF16, kBF16, kBF16>(layer, g, a, s);
}

lowbit_status launch_join_back(int ft, int st, int pt, bool layer, const JoinShape& g,
                               const JoinBackArgs& a, hipStream_t s) {
  if (ft == kF32) return join_back_types<kF32, kF32, kF32>(layer, g, a, s);
  if (st == kF32)
    return pt == kF32 ? join_back_types<kBF16, kF32, kF32>(layer, g, a, s)
                      : join_back_types<kBF16, kF32, kBF16>(layer, g, a, s);
  return pt == kF32 ? join_back_types<kBF16, kBF16, kF32>(layer, g, a, s)
                    : join_back_types<kBF16, kBF16, kBF16>(layer, g, a, s);
}

lowbit_status launch_join_sums(const JoinSumArgs& a, hipStream_t s) {
  // no group of a gate lies in two workgroups' rows: all were written there
  const bool whole = !a.dgate || a.rows_per_block % a.rows_per_gate == 0;
  const int64_t groups = whole ? 0 : (a.rows + a.rows_per_gate - 1) / a.rows_per_gate;
  const int64_t whats = a.params + groups;
  if (whats == 0) return LOWBIT_OK;
  const dim3 grid((a.cols + 63) / 64, (uint32_t)(whats < 4096 ? whats : 4096));
  JoinSumArgs copy = a;
  int64_t g = groups;
  void* argv[] = {&copy, &g};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&join_sum_kernel), grid,
                                       dim3(1024), argv, 0, s);
  return e == hipSuccess ? LOWBIT_OK : LOWBIT_EDEVICE;
}

}  // namespace lowbit
