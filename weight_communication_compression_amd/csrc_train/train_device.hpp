// train_device.hpp -- gfx950 device helpers of the training-step operators:
// element vectors at any element alignment, the dropout mask, workgroup sums.
#pragma once

#include "../csrc/device.hpp"

namespace lowbit {

// Sixteen bytes at any element's alignment.  Rows of odd width begin
// anywhere; global memory takes such an access whole, so that no second kernel
// for rows that are not aligned is needed.
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int DT>
constexpr int elem_size() { return DT == kF32 ? 4 : 2; }

// two binary32 values -> bfloat16, to nearest even, in one instruction
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Eight elements as they lie in memory.
template <int DT>
struct Raw8 {
  u32x4 w[DT == kF32 ? 2 : 1];
  __device__ __forceinline__ void fill(float a, float b) {
    if constexpr (DT == kF32) {
      const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
      w[0] = w[1] = (u32x4){x, y, x, y};
    } else {
      const uint32_t x = pack_bf16(a, b);
      w[0] = (u32x4){x, x, x, x};
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (DT == kF32) return __uint_as_float(w[j / 4][j % 4]);
    else return j % 2 ? bf16_hi(w[0][j / 2]) : bf16_lo(w[0][j / 2]);
  }
  __device__ __forceinline__ void set2(int j, float a, float b) {  // elements j (even) and j + 1
    if constexpr (DT == kF32) {
      w[j / 4][j % 4] = __float_as_uint(a);
      w[j / 4][j % 4 + 1] = __float_as_uint(b);
    } else {
      w[0][j / 2] = pack_bf16(a, b);
    }
  }
};

// Elements c .. c + 7 of the row at `row`, those from `cols` on as +0.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* row, int c, int cols) {
  Raw8<DT> r;
  const char* p = static_cast<const char*>(row) + (int64_t)c * elem_size<DT>();
  if (c + 8 <= cols) {
    if constexpr (DT == kF32) {
      r.w[0] = reinterpret_cast<const u32x4_4*>(p)[0];
      r.w[1] = reinterpret_cast<const u32x4_4*>(p)[1];
    } else {
      r.w[0] = *reinterpret_cast<const u32x4_2*>(p);
    }
  } else {
    r.fill(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c + j < cols) {
        if constexpr (DT == kF32) r.w[j / 4][j % 4] = reinterpret_cast<const uint32_t*>(p)[j];
        else r.w[0][j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j % 2));
      }
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store8(void* row, int c, int cols, const Raw8<DT>& r) {
  char* p = static_cast<char*>(row) + (int64_t)c * elem_size<DT>();
  if (c + 8 <= cols) {
    if constexpr (DT == kF32) {
      reinterpret_cast<u32x4_4*>(p)[0] = r.w[0];
      reinterpret_cast<u32x4_4*>(p)[1] = r.w[1];
    } else {
      *reinterpret_cast<u32x4_2*>(p) = r.w[0];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c + j < cols) {
        if constexpr (DT == kF32) reinterpret_cast<uint32_t*>(p)[j] = r.w[j / 4][j % 4];
        else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(r.w[0][j / 2] >> (16 * (j % 2)));
      }
    }
  }
}

// the word of the mask's pair q: two draws, of which those below `cut` are dropped
__device__ __forceinline__ uint32_t draw_word(const HiMix& h, uint32_t q) {
  return fmix32(h.x0(q));
}
__device__ __forceinline__ bool keeps_lo(uint32_t word, uint32_t cut) { return (word & 0xFFFFu) >= cut; }
__device__ __forceinline__ bool keeps_hi(uint32_t word, uint32_t cut) { return (word >> 16) >= cut; }

// Sums of N values over the L lanes that share a row: 8, 16, 32 or 64 of a wave, or
// whole waves of a workgroup, whose parts are added in order; every lane gets
// the result.  `slot` is LDS for N * 16 values; a caller that alternates two
// slots needs no other barrier.  (Loads and stores to memory may stay under way.)
// SUB: L is less than 64.
template <int N, bool SUB>
__device__ __forceinline__ void row_sum(float* v, float* slot, int L) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (SUB)
      v[i] = L == 8 ? group_reduce<8, true>(v[i]) : L == 16 ? group_reduce<16, true>(v[i])
                                                            : group_reduce<32, true>(v[i]);
    else
      v[i] = group_reduce<64, true>(v[i]);
  }
  if (SUB || L == 64) return;
  const int wave = threadIdx.x >> 6;
  if (lane_id() == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[wave * N + i] = v[i];
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = slot[i];
  for (int w = 1; w < L >> 6; ++w) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += slot[w * N + i];
  }
}

}  // namespace lowbit
