// dropout and its gradient
#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

// y = r + D(x).  A lane takes 16 bytes of consecutive elements per trip and row
// of the wave; the mask's word serves a pair, so that eight bfloat16 elements
// cost four hashes.  Bound by memory: x (and r) read once, y written once (64 Mi
// bfloat16 with a residual 67.5 us, 6.0 TB/s; 16 Mi binary32 19.7 us; the launch
// alone 3.7 us).
constexpr int kDropRows = 2;      // 16-byte pieces of a lane per trip

template <int DT, bool RES>
__global__ void __launch_bounds__(kBlockThreads) dropout_kernel(DropoutArgs a, int64_t ntrips) {
  constexpr int E = DT == kF32 ? 4 : 8;
  constexpr int TRIP = kDropRows * kWave * E;
  const float factor = a.factor;
  const uint32_t cut = a.cut;
  for_each_trip(
      global_wave_id(), ntrips, (int64_t)gridDim.x * (kBlockThreads / kWave), [&](int64_t trip) {
        const int64_t t0 = trip * TRIP;
        const HiMix mix(a.pair0 + (uint64_t)t0 / 2, a.key);
        const int64_t rem = a.n - t0;
        float v[kDropRows][E], r[kDropRows][E];
#pragma unroll
        for (int k = 0; k < kDropRows; ++k) {
          const uint32_t off = (uint32_t)(k * kWave + lane_id()) * E;
          if (rem >= TRIP) {
            load_vec<DT, E>(a.x, t0, off, v[k]);
            if constexpr (RES) load_vec<DT, E>(a.r, t0, off, r[k]);
          } else {
            load_tail<DT, E>(a.x, t0, off, rem, v[k]);
            if constexpr (RES) load_tail<DT, E>(a.r, t0, off, rem, r[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < kDropRows; ++k) {
          const uint32_t off = (uint32_t)(k * kWave + lane_id()) * E;
#pragma unroll
          for (int j = 0; j < E; j += 2) {
            const uint32_t word = draw_word(mix, (off + j) / 2);
            float lo = keeps_lo(word, cut) ? v[k][j] * factor : 0.0f;
            float hi = keeps_hi(word, cut) ? v[k][j + 1] * factor : 0.0f;
            if constexpr (RES) {
              lo += r[k][j];
              hi += r[k][j + 1];
            }
            v[k][j] = lo;
            v[k][j + 1] = hi;
          }
          if constexpr (DT == kF32) {
            if (rem >= TRIP) store_vec_f32<E>(static_cast<float*>(a.y), t0, off, v[k]);
            else store_tail_f32<E>(static_cast<float*>(a.y), t0, off, rem, v[k]);
          } else {
            uint16_t* y = static_cast<uint16_t*>(a.y) + t0 + off;
            u32x4 q;
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = pack_bf16(v[k][2 * j], v[k][2 * j + 1]);
            if (rem >= TRIP) {
              __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(y));
            } else {
#pragma unroll
              for (int j = 0; j < E; ++j)
                if ((int64_t)off + j < rem) y[j] = (uint16_t)(q[j / 2] >> (16 * (j % 2)));
            }
          }
        }
      });
}

lowbit_status launch_dropout(int dt, const DropoutArgs& a, hipStream_t s) {
  const int trip = kDropRows * kWave * (dt == kF32 ? 4 : 8);
  const int64_t ntrips = (a.n + trip - 1) / trip, blocks = grid_for_tiles(ntrips);
  if (dt == kF32)
    return a.r ? launch(&dropout_kernel<kF32, true>, blocks, kBlockThreads, s, a, ntrips)
               : launch(&dropout_kernel<kF32, false>, blocks, kBlockThreads, s, a, ntrips);
  return a.r ? launch(&dropout_kernel<kBF16, true>, blocks, kBlockThreads, s, a, ntrips)
             : launch(&dropout_kernel<kBF16, false>, blocks, kBlockThreads, s, a, ntrips);
}

}  // namespace lowbit
