// rotary.hip -- rotary positions and their gradient.
#include "block.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

constexpr int kThreads = 256;

// Sixteen bytes of elements at any element's alignment, those from `count` on as +0 and not
// stored.
template <int DT>
struct Vec {
  static constexpr int E = 16 / elem_size<DT>();
  u32x4 w;
  __device__ __forceinline__ float get(int j) const {
    if constexpr (DT == kF32) return __uint_as_float(w[j]);
    else return j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
  }
  __device__ __forceinline__ void set2(int j, float a, float b) {  // elements j (even) and j + 1
    if constexpr (DT == kF32) {
      w[j] = __float_as_uint(a);
      w[j + 1] = __float_as_uint(b);
    } else {
      w[j / 2] = pack_bf16(a, b);
    }
  }
  __device__ __forceinline__ void load(const char* p, int count) {
    if (count >= E) {
      if constexpr (DT == kF32) w = *reinterpret_cast<const u32x4_4*>(p);
      else w = *reinterpret_cast<const u32x4_2*>(p);
    } else {
      w = (u32x4){0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < E - 1; ++j)
        if (j < count) {
          if constexpr (DT == kF32) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
          else w[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j % 2));
        }
    }
  }
  __device__ __forceinline__ void store(char* p, int count) const {
    if (count >= E) {
      if constexpr (DT == kF32) *reinterpret_cast<u32x4_4*>(p) = w;
      else *reinterpret_cast<u32x4_2*>(p) = w;
    } else {
#pragma unroll
      for (int j = 0; j < E - 1; ++j)
        if (j < count) {
          if constexpr (DT == kF32) reinterpret_cast<uint32_t*>(p)[j] = w[j];
          else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
        }
    }
  }
};

// P pairs' cosines and sines, times the scale.  The angle is taken in turns
// in binary64, where a position of 2^30 leaves 2^-22 of a turn and better, and
// reduced to half a turn before it is rounded to binary32.
template <int P>
struct Turns {
  float c[P], s[P];
  __device__ __forceinline__ void init(const RotaryArgs& g, int64_t row, int pair0) {
    const int pairs = g.rot_dim / 2;
    const int64_t at = g.positions ? g.positions[row] : row % g.rows_per_sequence;
    const double place = (double)at * 0.15915494309189535;   // / (2 pi)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = pair0 + j < pairs ? pair0 + j : pairs - 1;
      const double turn = place * g.freqs[i];
      const float half = (float)(turn - rint(turn)) * 2.0f;
      float sn, cs;
      sincospif(half, &sn, &cs);
      c[j] = cs * g.scale;
      s[j] = sn * g.scale * g.sign;
    }
  }
  __device__ __forceinline__ void turn(int j, float& u, float& v) const {
    const float a = __builtin_fmaf(u, c[j], -(v * s[j])), b = __builtin_fmaf(u, s[j], v * c[j]);
    u = a;
    v = b;
  }
};

// A unit's pairs of one head, as many as 16 bytes have elements, as they lie in memory.
template <int DT, int LAYOUT>
struct Pairs {
  static constexpr int E = Vec<DT>::E, ES = elem_size<DT>();
  Vec<DT> a, b;              // half: firsts and seconds; interleaved: half of the pairs each
  __device__ __forceinline__ void load(const char* from, int unit, int rot) {
    if constexpr (LAYOUT == LOWBIT_ROTARY_HALF) {
      const char* p = from + unit * E * ES;
      a.load(p, rot / 2 - unit * E);
      b.load(p + rot / 2 * ES, rot / 2 - unit * E);
    } else {
      const char* p = from + unit * 2 * E * ES;
      a.load(p, rot - unit * 2 * E);
      b.load(p + E * ES, rot - unit * 2 * E - E);
    }
  }
  __device__ __forceinline__ void turn(const Turns<E>& w) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      float a0 = a.get(j), a1 = a.get(j + 1), b0 = b.get(j), b1 = b.get(j + 1);
      if constexpr (LAYOUT == LOWBIT_ROTARY_HALF) {
        w.turn(j, a0, b0);
        w.turn(j + 1, a1, b1);
      } else {
        w.turn(j / 2, a0, a1);
        w.turn(E / 2 + j / 2, b0, b1);
      }
      a.set2(j, a0, a1);
      b.set2(j, b0, b1);
    }
  }
  __device__ __forceinline__ void store(char* to, int unit, int rot) const {
    if constexpr (LAYOUT == LOWBIT_ROTARY_HALF) {
      char* p = to + unit * E * ES;
      a.store(p, rot / 2 - unit * E);
      b.store(p + rot / 2 * ES, rot / 2 - unit * E);
    } else {
      char* p = to + unit * 2 * E * ES;
      a.store(p, rot - unit * 2 * E);
      b.store(p + E * ES, rot - unit * 2 * E - E);
    }
  }
};

// A lane takes a unit of a row (of pairs, or 16 bytes that are copied) through all heads of
// its group, so that sines are taken once for them; a group's heads lie `groups` apart.  The
// first heads are loaded before the sines are taken.  Bound by memory: 16 Ki x 40 heads of 128
// bfloat16 64 us, 5.2 TB/s; 5003 x 24 heads of 80 binary32, half of each turned, 18 us (with
// units of eight pairs, whose loads lie 64 bytes apart from lane to lane, 29).
template <int DT, int LAYOUT>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs g) {
  constexpr int ES = elem_size<DT>(), E = Vec<DT>::E, N = 4;   // N heads under way
  const int per_row = g.lanes * g.groups;
  const int64_t step = (int64_t)gridDim.x * g.rows_per_block;
  for (int64_t row0 = (int64_t)blockIdx.x * g.rows_per_block; row0 < g.rows; row0 += step)
    for (int t = threadIdx.x; t < per_row * g.rows_per_block; t += kThreads) {
      const int64_t row = row0 + t / per_row;
      if (row >= g.rows) break;
      const int unit = t % per_row % g.lanes, first = t % per_row / g.lanes;
      const char* x = static_cast<const char*>(g.x) + row * g.x_row * ES;
      char* y = static_cast<char*>(g.y) + row * g.y_row * ES;
      if (unit < g.turning) {
        Turns<E> w;
        bool taken = false;
        for (int h = first; h < g.heads; h += N * g.groups) {
          Pairs<DT, LAYOUT> p[N];
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (h + k * g.groups < g.heads)
              p[k].load(x + (h + k * g.groups) * g.x_head * ES, unit, g.rot_dim);
          if (!taken) w.init(g, row, unit * E);
          taken = true;
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (h + k * g.groups < g.heads) {
              p[k].turn(w);
              p[k].store(y + (h + k * g.groups) * g.y_head * ES, unit, g.rot_dim);
            }
        }
      } else {
        const int c = g.rot_dim + (unit - g.turning) * E;
        for (int h = first; h < g.heads; h += N * g.groups) {
          Vec<DT> p[N];
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (h + k * g.groups < g.heads)
              p[k].load(x + ((h + k * g.groups) * g.x_head + c) * ES, g.head_dim - c);
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (h + k * g.groups < g.heads)
              p[k].store(y + ((h + k * g.groups) * g.y_head + c) * ES, g.head_dim - c);
        }
      }
    }
}

template <int DT>
lowbit_status launch_type(int layout, const RotaryArgs& a, int64_t blocks, hipStream_t s) {
  return layout == LOWBIT_ROTARY_HALF
             ? launch(&rotary_kernel<DT, LOWBIT_ROTARY_HALF>, blocks, kThreads, s, a)
             : launch(&rotary_kernel<DT, LOWBIT_ROTARY_INTERLEAVED>, blocks, kThreads, s, a);
}

}  // namespace

lowbit_status launch_rotary(int dt, int layout, const RotaryArgs& args, hipStream_t s) {
  RotaryArgs a = args;
  const int e = dt == LOWBIT_F32 ? 4 : 8;
  a.turning = (a.rot_dim / 2 + e - 1) / e;
  const bool copies = a.y != a.x && a.head_dim > a.rot_dim;
  a.lanes = a.turning + (copies ? (a.head_dim - a.rot_dim + e - 1) / e : 0);
  // up to eight heads a lane, as long as there are 2^19 lanes, four times what the chip holds at
  // one time (16 Ki x 40 x 128 bf16: 64 us, 5.2 TB/s; with four heads 67)
  int each = 8;
  while (each > 1 && a.rows * a.lanes * ((a.heads + each - 1) / each) < (1 << 19)) each /= 2;
  a.groups = (a.heads + each - 1) / each;
  const int64_t per_row = (int64_t)a.lanes * a.groups;
  a.rows_per_block = per_row >= kThreads ? 1 : (int32_t)(kThreads / per_row);
  const int64_t blocks = grid_blocks((a.rows + a.rows_per_block - 1) / a.rows_per_block * 4, kThreads);
  return dt == LOWBIT_F32 ? launch_type<kF32>(layout, a, blocks, s)
                          : launch_type<kBF16>(layout, a, blocks, s);
}

}  // namespace lowbit
