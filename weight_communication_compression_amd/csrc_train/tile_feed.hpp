// tile_feed.hpp -- what the products in tiles share (linear xent, orthogonalize):
// operands fed through LDS, read into registers, multiplied on the matrix units, and the
// order of these for the compiler.
#pragma once

#include "matrix_unit.hpp"
#include "train_device.hpp"
#include "xent_cut.hpp"

namespace lowbit {

namespace {

typedef uint32_t u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));

constexpr int kRowBytes = kXentRowBytes;   // of k, between two barriers

// One operand's way into LDS: T rows of the tile by 128 bytes of k, 16 bytes a
// lane straight from memory, the W waves taking turns.  OUTER: k is the
// matrix's row, and LDS holds rows of k; else rows of the tile.  The pieces of
// a row in LDS are permuted by the row's number, so that the reads of Frag
// meet no bank twice; a load writes LDS in lane order, so each lane fetches
// the piece that belongs in its place.  What lies behind the matrix's end reads
// as 0.  (Rows of 64 bytes, which would let more steps be under way, load at
// half the rate: 67 against 130 bytes/ns and CU.)
template <int DT, int T, int W, bool OUTER>
struct Feed {
  static constexpr int ES = elem_size<DT>(), K = kRowBytes / ES, LOADS = T / 8 / W;
  static constexpr int KR = 1024 / (T * ES);     // OUTER: rows of k in a wave's load
  static constexpr int PIECE = DT == kF32 ? 128 : 32;   // OUTER: bytes
  const char* base;
  int64_t left, kstep;                           // bytes
  uint32_t voff[LOADS];
  int kin;                                       // the lane's first k within the step

  // OUTER: the pieces of row k are xored with this
  static __device__ __forceinline__ constexpr int mix(int k) {
    return (DT == kF32 ? k >> 2 & 1 : (k & 3) << 1 | (k >> 3 & 1)) & (T * ES / PIECE - 1);
  }
  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
    static_assert(LOADS >= 1 && (!OUTER || K % (W * KR) == 0), "");
    kstep = OUTER ? K * ld * ES : kRowBytes;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      if constexpr (OUTER) {
        constexpr int L = T * ES / 16, P = PIECE / 16;   // lanes of a row, of a piece
        const int k = (j * W + wave) * KR + lane / L, slot = lane % L;
        kin = 0;
        voff[j] = (uint32_t)(k * ld * ES) + ((slot / P ^ mix(k)) * P + slot % P) * 16;
      } else {
        const int r = (j * W + wave) * 8 + lane / 8, c = lane % 8 ^ (r >> 1 & 7);
        kin = c * (16 / ES);                             // (r >> 1 & 7 is the same for every j)
        voff[j] = (uint32_t)(r * ld * ES) + c * 16;
      }
    }
  }
  // rows: of the matrix in memory; k0: where to begin
  __device__ __forceinline__ void seek(const void* p, int64_t ld, int64_t rows, int64_t row0,
                                       int64_t k0) {
    const int64_t at = (OUTER ? k0 * ld + row0 : row0 * ld + k0) * ES;
    base = static_cast<const char*>(p) + at;
    left = rows * ld * ES - at;
  }
  // The matrix from here on, for the loads of one step (none if !any).
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t open(bool any) const {
    const int records = (int)(left < 0 || !any ? 0 : left > kNowhere ? kNowhere : left);
    return lowbit::open(base, records);
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* lds, int wave, int kleft,
                                       int j) const {
    const uint32_t v = !OUTER && kin >= kleft ? kNowhere : voff[j];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LOWBIT_LDS void*)(lds + (j * W + wave) * 1024),
                                             16, v, 0, 0, 0);
  }
  __device__ __forceinline__ void next() {
    base += kstep;
    left -= kstep;
  }
};

// A lane's part of 32 rows by 32 bytes of k: row lane mod 32, the (lane / 32)-th 16 bytes.
template <int DT, int T, bool OUTER>
struct Frag {
  static constexpr int ES = elem_size<DT>(), PITCH = T * ES;
  uint32_t at[4];
  int piece, f;                                  // OUTER
  __device__ __forceinline__ void init(int row0, int lane) {
    const int h = lane / 32;
    if constexpr (OUTER && DT == kF32) {
      f = Feed<DT, T, 1, true>::mix(4 * h);
      piece = row0 / 32;
      at[0] = 4 * h * PITCH + lane % 32 * 4;
    } else if constexpr (OUTER) {
      const int k = 8 * h + lane % 16 / 4;
      f = Feed<DT, T, 1, true>::mix(k);
      piece = row0 / 16 + lane / 16 % 2;
      at[0] = k * PITCH + lane % 4 * 8;
    } else {
      const int r = row0 + lane % 32, s = r >> 1 & 7;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) at[kk] = r * kRowBytes + ((2 * kk + h) ^ s) * 16;
    }
  }
  // 32-row piece i of the wave, quarter kk of the step
  __device__ __forceinline__ u32x4 load(const char* lds, int i, int kk) const {
    if constexpr (!OUTER) {
      return *reinterpret_cast<const u32x4*>(lds + at[kk] + i * 32 * kRowBytes);
    } else if constexpr (DT == kF32) {
      const char* p = lds + at[0] + ((piece + i) ^ f) * 128 + kk * 8 * PITCH;
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * PITCH);
      return v;
    } else {
      // 16 lanes read 16 columns of four rows of k and get a column each
      const char* p = lds + at[0] + ((piece + 2 * i) ^ f) * 32 + kk * 16 * PITCH;
      typedef LOWBIT_LDS s16x4* lp;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(LOWBIT_LDS char*)p);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(LOWBIT_LDS char*)(p + 4 * PITCH));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

template <int DT_, int TM_, int TN_, int WM_, int WN_, int SLOTS_>
struct Form {
  static constexpr int DT = DT_, TM = TM_, TN = TN_, WM = WM_, WN = WN_, SLOTS = SLOTS_;
  static constexpr int W = WM * WN, I = TM / WM / 32, J = TN / WN / 32, THREADS = 64 * W;
};

__device__ __forceinline__ f32x4 quad(const f32x16& v, int q) {
  return (f32x4){v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Order for the compiler: R reads of LDS, spread over M products.
template <int R, int M, int N = 0>
__device__ __forceinline__ void spread_reads() {
  if constexpr (N < R) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, M * (N + 1) / R - M * N / R, 0);
    spread_reads<R, M, N + 1>();
  }
}
// R reads and L loads to LDS, spread over M products of Q instructions.
template <int R, int M, int Q, int L, int N = 0>
__device__ __forceinline__ void spread_loads() {
  if constexpr (N < M) {
    __builtin_amdgcn_sched_group_barrier(0x008, Q, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, R * (N + 1) / M - R * N / M, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, L * (N + 1) / M - L * N / M, 0);
    spread_loads<R, M, Q, L, N + 1>();
  }
}

}  // namespace

}  // namespace lowbit
