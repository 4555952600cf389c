// rotary.hip -- rotary positions and their gradient.
#include "block.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

constexpr int kThreads = 256;

// Eight pairs' cosines and sines, times the scale.  The angle is taken in turns
// in binary64, where a position of 2^30 leaves 2^-22 of a turn and better, and
// reduced to half a turn before it is rounded to binary32.
struct Turns {
  float c[8], s[8];
  __device__ __forceinline__ void init(const RotaryArgs& g, int64_t row, int pair0) {
    const int pairs = g.rot_dim / 2;
    const int64_t at = g.positions ? g.positions[row] : row % g.rows_per_sequence;
    const double place = (double)at * 0.15915494309189535;   // / (2 pi)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
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

// A lane takes eight pairs of a row (or eight elements that are copied) through
// all heads of its group, so that sines are taken once for them; a group's
// heads lie `groups` apart.
template <int DT, int LAYOUT>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs g) {
  constexpr int ES = elem_size<DT>();
  const int per_row = g.lanes * g.groups;
  const int half = g.rot_dim / 2;
  const int64_t step = (int64_t)gridDim.x * g.rows_per_block;
  for (int64_t row0 = (int64_t)blockIdx.x * g.rows_per_block; row0 < g.rows; row0 += step)
  for (int t = threadIdx.x; t < per_row * g.rows_per_block; t += kThreads) {
    const int64_t row = row0 + t / per_row;
    if (row >= g.rows) break;
    const int unit = t % per_row % g.lanes, first = t % per_row / g.lanes;
    const char* x = static_cast<const char*>(g.x) + row * g.x_row * ES;
    char* y = static_cast<char*>(g.y) + row * g.y_row * ES;
    if (unit < g.turning) {
      Turns w;
      w.init(g, row, unit * 8);
#pragma unroll 4
      for (int h = first; h < g.heads; h += g.groups) {
        const char* from = x + h * g.x_head * ES;
        char* to = y + h * g.y_head * ES;
        if constexpr (LAYOUT == LOWBIT_ROTARY_HALF) {
          Raw8<DT> u = load8<DT>(from, unit * 8, half);
          Raw8<DT> v = load8<DT>(from + half * ES, unit * 8, half);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float u0 = u.get(j), u1 = u.get(j + 1), v0 = v.get(j), v1 = v.get(j + 1);
            w.turn(j, u0, v0);
            w.turn(j + 1, u1, v1);
            u.set2(j, u0, u1);
            v.set2(j, v0, v1);
          }
          store8<DT>(to, unit * 8, half, u);
          store8<DT>(to + half * ES, unit * 8, half, v);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            Raw8<DT> u = load8<DT>(from, unit * 16 + k * 8, g.rot_dim);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              float u0 = u.get(j), u1 = u.get(j + 1);
              w.turn(k * 4 + j / 2, u0, u1);
              u.set2(j, u0, u1);
            }
            store8<DT>(to, unit * 16 + k * 8, g.rot_dim, u);
          }
        }
      }
    } else {
      const int c = (unit - g.turning) * 8, rest = g.head_dim - g.rot_dim;
      for (int h = first; h < g.heads; h += g.groups)
        store8<DT>(y + (h * g.y_head + g.rot_dim) * ES, c, rest,
                   load8<DT>(x + (h * g.x_head + g.rot_dim) * ES, c, rest));
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
  a.turning = (a.rot_dim / 2 + 7) / 8;
  const bool copies = a.y != a.x && a.head_dim > a.rot_dim;
  a.lanes = a.turning + (copies ? (a.head_dim - a.rot_dim + 7) / 8 : 0);
  // up to eight heads a lane, as long as the chip's 2^17 lanes are filled
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
