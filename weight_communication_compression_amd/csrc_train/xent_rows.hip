// linear xent: which rows count, their compact copies, and the softmax's parts
#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

constexpr int kRowsEach = 8;       // rows of a thread per step
constexpr int64_t kXentFused = 16384;

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

// Both at once, for up to kXentFused rows: every workgroup counts the rows that
// count before its own by reading all targets (128 KiB at most, from L2), so that
// nothing has to be known beforehand.  Workgroup b takes rows, and places among the
// compact rows, b * each .. + each - 1; each is at most 64, a wave's lanes.  The
// two kernels above take 19 us for 8 Ki rows before the first copy begins, and 8 us
// for a few.
template <int DT>
__global__ void __launch_bounds__(512) xent_first_kernel(XentRows a, XentGather g, int each) {
  __shared__ int before_of[8], all_of[8];
  __shared__ float max_of[8];
  __shared__ int place[64];                    // of the workgroup's rows, -1: left out
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * each;
  int before = 0, all = 0;
  float top = 0.0f;
  for (int64_t r = threadIdx.x; r < a.n; r += 512) {
    const bool counts = a.targets[r] != a.ignore;
    all += counts;
    before += counts && r < r0;
    if (blockIdx.x == 0 && a.dloss && counts) {
      const float d = a.dloss[r], both = a.dlse ? d + a.dlse[r] : d;
      const bool inside = a.targets[r] >= 0 && a.targets[r] < a.vocab;
      if (inside && fabsf(both) < INFINITY) top = fmaxf(top, fabsf(both));
      if (fabsf(d) < INFINITY) top = fmaxf(top, fabsf(d));
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    before += __shfl_xor(before, d);
    all += __shfl_xor(all, d);
  }
  top = group_max_nonneg<64>(top);
  if (lane == 0) {
    before_of[wave] = before;
    all_of[wave] = all;
    max_of[wave] = top;
  }
  __syncthreads();
  before = all = 0;
  for (int w = 0; w < 8; ++w) {
    before += before_of[w];
    all += all_of[w];
    top = fmaxf(top, max_of[w]);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.count = all;
    *a.scale = top > 0.0f ? top : 1.0f;
  }
  if (wave == 0) {
    const int64_t r = r0 + lane;
    const bool mine = lane < each;
    const int64_t t = mine && r < a.n ? a.targets[r] : a.ignore;
    const bool counts = t != a.ignore;
    const uint64_t mask = __ballot(counts);
    const int at = before + __popcll(mask & ((1ull << lane) - 1));
    if (mine && r < a.n) a.pos[r] = counts ? at : -1;
    if (counts) {
      a.map[at] = (int32_t)r;
      const bool inside = t >= 0 && t < a.vocab;
      float4 info = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(inside ? (int)t : -1));
      if (a.dloss) {
        info.x = a.lse[r];
        info.z = a.dloss[r];
        info.y = !inside ? __builtin_nanf("") : a.dlse ? info.z + a.dlse[r] : info.z;
      }
      a.info[at] = info;
    }
    if (mine && r >= all && r < a.padded) {    // a place that no row takes
      a.map[r] = -1;
      a.info[r] = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
    }
    place[lane] = counts ? at : -1;
  }
  __syncthreads();
  // four vectors of eight at a time, their loads under way together
  const uint32_t vectors = (uint32_t)(g.ld + 7) / 8, mine = each * vectors;
  for (uint32_t v0 = threadIdx.x; v0 < mine; v0 += 4 * 512) {
    Raw8<DT> x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t v = v0 + u * 512, k = v / vectors;
      x[u].fill(0.0f, 0.0f);
      if (v < mine && place[k] >= 0)
        x[u] = load8<DT>(static_cast<const char*>(g.x) + (r0 + k) * g.hidden * elem_size<DT>(),
                         (int)(v - k * vectors) * 8, g.hidden);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t v = v0 + u * 512, k = v / vectors;
      if (v >= mine) break;
      const int c = (int)(v - k * vectors) * 8;
      const int64_t r = r0 + k;
      char* const xc = static_cast<char*>(g.xc);
      if (place[k] >= 0) {
        store8<DT>(xc + (int64_t)place[k] * g.ld * elem_size<DT>(), c, g.ld, x[u]);
      } else if (g.dx && r < a.n) {
        store8<DT>(static_cast<char*>(g.dx) + r * g.hidden * elem_size<DT>(), c, g.hidden, x[u]);
      }
      if (r >= all && r < a.padded) {
        x[u].fill(0.0f, 0.0f);
        store8<DT>(xc + r * g.ld * elem_size<DT>(), c, g.ld, x[u]);
      }
    }
  }
}

// A thread a vector, whatever the rows' length.
template <int DT>
__global__ void __launch_bounds__(256) xent_pack_kernel(XentPack a) {
  const uint32_t vectors = (uint32_t)(a.ld + 7) / 8;
  const int64_t all = a.rows * vectors;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < all; v += (int64_t)gridDim.x * 256) {
    const int64_t r = all < (1ll << 32) ? (uint32_t)v / vectors : v / vectors;
    const int c = (int)(v - r * vectors) * 8;
    const char* from = static_cast<const char*>(a.w) + r * a.hidden * elem_size<DT>();
    char* to = static_cast<char*>(a.to) + r * a.ld * elem_size<DT>();
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
      float top = -INFINITY, sum = 0.0f;
      // eight parts a lane at a time, their loads under way together; the sum so far
      // is kept relative to the maximum so far
      // (a part without finite logits has maximum -inf and a sum of 0 or NaN)
      for (int p0 = lane; p0 < a.parts; p0 += 8 * 64) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = p0 + u * 64 < a.parts ? part[p0 + u * 64] : make_float2(-INFINITY, 0.0f);
        float more = top;
#pragma unroll
        for (int u = 0; u < 8; ++u) more = fmaxf(more, v[u].x);
        if (top != -INFINITY) sum *= expf(top - more);
        top = more;
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += v[u].x == -INFINITY ? v[u].y : v[u].y * expf(v[u].x - top);
      }
      float all = top;
      for (int d = 1; d < 64; d *= 2) all = fmaxf(all, __shfl_xor(all, d));
      if (top != -INFINITY) sum *= expf(top - all);
      top = all;
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

lowbit_status launch_xent_rows(int dt, const XentRows& r, const XentGather& g, hipStream_t s) {
  if (r.n <= kXentFused) {
    const int each = (int)((r.padded + 255) / 256);
    const int64_t blocks = (r.padded + each - 1) / each;
    return launch(dt == kF32 ? &xent_first_kernel<kF32> : &xent_first_kernel<kBF16>, blocks, 512, s,
                  r, g, each);
  }
  const lowbit_status st = launch(&xent_rows_kernel, 1, 1024, s, r);
  if (st != LOWBIT_OK) return st;
  const int64_t blocks = g.padded < (1 << 22) ? g.padded : (1 << 22);
  return launch(dt == kF32 ? &xent_gather_kernel<kF32> : &xent_gather_kernel<kBF16>, blocks, 256,
                s, g);
}

lowbit_status launch_xent_pack(int dt, const XentPack& a, hipStream_t s) {
  const int64_t vectors = a.rows * ((a.ld + 7) / 8), most = 1 << 22;
  const int64_t blocks = vectors / 256 + 1 < most ? vectors / 256 + 1 : most;
  return launch(dt == kF32 ? &xent_pack_kernel<kF32> : &xent_pack_kernel<kBF16>, blocks, 256, s,
                a);
}

lowbit_status launch_xent_join(const XentJoin& a, hipStream_t s) {
  return launch(&xent_join_kernel, grid_for_tiles(a.n), kBlockThreads, s, a);
}

}  // namespace lowbit
