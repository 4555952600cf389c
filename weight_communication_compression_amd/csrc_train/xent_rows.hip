// linear xent: which rows count, their compact copies, and the softmax's parts
#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

constexpr int kRowsEach = 8;       // rows of a thread per step

// One workgroup numbers the rows that count, in order: a count for each
// thread's eight rows, a scan over the workgroup, 8192 rows a step.  One
// workgroup is enough: the products cost thousands of times more.
__global__ void __launch_bounds__(1024) xent_rows_kernel(XentRows a) {
  __shared__ int wave_sum[16];
  __shared__ float wave_max[16];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  int64_t base = 0;                // compact rows so far
  float top = 0.0f;
  for (int64_t r0 = 0; r0 < a.n; r0 += 1024 * kRowsEach) {
    const int64_t r = r0 + (int64_t)threadIdx.x * kRowsEach;
    int64_t t[kRowsEach];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kRowsEach; ++j) {
      t[j] = r + j < a.n ? a.targets[r + j] : a.ignore;
      mine += t[j] != a.ignore;
    }
    int incl = mine;               // inclusive scan over the wave
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? wave_sum[w] : 0;
      all += wave_sum[w];
    }
    int64_t at = base + before + incl - mine;
#pragma unroll
    for (int j = 0; j < kRowsEach; ++j) {
      if (r + j >= a.n) break;
      if (t[j] == a.ignore) {
        a.pos[r + j] = -1;
        continue;
      }
      a.pos[r + j] = (int32_t)at;
      a.map[at] = (int32_t)(r + j);
      float4 info = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const bool inside = t[j] >= 0 && t[j] < a.vocab;
      info.w = __int_as_float(inside ? (int)t[j] : -1);
      if (a.dloss) {
        const float d = a.dloss[r + j];
        info.x = a.lse[r + j];
        info.z = d;
        info.y = a.dlse ? d + a.dlse[r + j] : d;
        if (!inside) info.y = __builtin_nanf("");
        if (fabsf(info.y) < INFINITY) top = fmaxf(top, fabsf(info.y));
        if (fabsf(info.z) < INFINITY) top = fmaxf(top, fabsf(info.z));
      }
      a.info[at] = info;
      ++at;
    }
    base += all;
    __syncthreads();               // wave_sum is written again
  }
  for (int64_t i = base + threadIdx.x; i < a.padded; i += 1024) {
    a.map[i] = -1;
    a.info[i] = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
  }
  top = group_max_nonneg<64>(top);
  if (lane == 0) wave_max[wave] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) top = fmaxf(top, wave_max[w]);
    *a.scale = top > 0.0f ? top : 1.0f;
    *a.count = (int32_t)base;
  }
}

// Workgroup b: compact row b of x, zeros where there is none, and row b of dx
// where that row is left out.
template <int DT>
__global__ void __launch_bounds__(256) xent_gather_kernel(XentGather a) {
  for (int64_t b = blockIdx.x; b < a.padded; b += gridDim.x) {
    const int64_t src = a.map[b];
    char* to = static_cast<char*>(a.xc) + b * a.ld * elem_size<DT>();
    const char* from = static_cast<const char*>(a.x) + src * a.hidden * elem_size<DT>();
    for (int c = 8 * threadIdx.x; c < a.ld; c += 8 * 256) {
      Raw8<DT> v;
      v.fill(0.0f, 0.0f);
      if (src >= 0) v = load8<DT>(from, c, a.hidden);
      store8<DT>(to, c, a.ld, v);
    }
    if (a.dx && b < a.n && a.pos[b] < 0) {
      Raw8<DT> zero;
      zero.fill(0.0f, 0.0f);
      char* d = static_cast<char*>(a.dx) + b * a.hidden * elem_size<DT>();
      for (int c = 8 * threadIdx.x; c < a.hidden; c += 8 * 256) store8<DT>(d, c, a.hidden, zero);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(256) xent_pack_kernel(XentPack a) {
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const char* from = static_cast<const char*>(a.w) + r * a.hidden * elem_size<DT>();
    char* to = static_cast<char*>(a.to) + r * a.ld * elem_size<DT>();
    for (int c = 8 * threadIdx.x; c < a.ld; c += 8 * 256)
      store8<DT>(to, c, a.ld, load8<DT>(from, c, a.hidden));
  }
}

// lse and loss of a row from its parts: a wave a row.
__global__ void __launch_bounds__(kBlockThreads) xent_join_kernel(XentJoin a) {
  const int lane = lane_id();
  for (int64_t r = global_wave_id(); r < a.n; r += (int64_t)gridDim.x * (kBlockThreads / kWave)) {
    const int64_t i = a.pos[r];
    float loss = 0.0f, lse = 0.0f;
    if (i >= 0) {
      const float2* part = a.part + i * a.parts;
      float top = -INFINITY;
      for (int p = lane; p < a.parts; p += 64) top = fmaxf(top, part[p].x);
      for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
      float sum = 0.0f;
      // (a part without finite logits has maximum -inf and a sum of 0 or NaN)
      for (int p = lane; p < a.parts; p += 64) {
        const float2 v = part[p];
        sum += v.x == -INFINITY ? v.y : v.y * expf(v.x - top);
      }
      for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
      lse = top + logf(sum);
      const int64_t t = a.targets[r];
      const bool inside = t >= 0 && t < a.vocab;
      if (!inside) lse = __builtin_nanf("");
      loss = inside ? lse - a.hit[i] : lse;
    }
    if (lane == 0) {
      a.loss[r] = loss;
      a.lse[r] = lse;
    }
  }
}

}  // namespace

lowbit_status launch_xent_rows(const XentRows& a, hipStream_t s) {
  return launch(&xent_rows_kernel, 1, 1024, s, a);
}

lowbit_status launch_xent_gather(int dt, const XentGather& a, hipStream_t s) {
  const int64_t blocks = a.padded < (1 << 22) ? a.padded : (1 << 22);
  if (blocks == 0) return LOWBIT_OK;
  return launch(dt == kF32 ? &xent_gather_kernel<kF32> : &xent_gather_kernel<kBF16>, blocks, 256,
                s, a);
}

lowbit_status launch_xent_pack(int dt, const XentPack& a, hipStream_t s) {
  const int64_t blocks = a.rows < (1 << 22) ? a.rows : (1 << 22);
  return launch(dt == kF32 ? &xent_pack_kernel<kF32> : &xent_pack_kernel<kBF16>, blocks, 256, s,
                a);
}

lowbit_status launch_xent_join(const XentJoin& a, hipStream_t s) {
  return launch(&xent_join_kernel, grid_for_tiles(a.n), kBlockThreads, s, a);
}

}  // namespace lowbit
