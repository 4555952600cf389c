// matrix_unit.hpp -- what the kernels on the matrix units share: operands, the product of 32 x 32,
// memory with bounds for loads straight to LDS, and waits.
#pragma once

#include "train_device.hpp"

namespace lowbit {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#define LOWBIT_LDS __attribute__((address_space(3)))

constexpr int kF16 = 2;                      // beside kF32 and kBF16: operands of orthogonalize
constexpr uint32_t kNowhere = 0x7FFFFFF0u;   // beyond every buffer's records

// d[row of first][column of second] += sum over 32 bytes of k.  Lane l gives row (column)
// l mod 32 and the (l / 32)-th 16 bytes, and holds of the result column l mod 32
// and rows 8 (r / 4) + 4 (l / 32) + r mod 4.  For binary32 four instructions take
// one element of each lane: k in another order, the same for both.
template <int DT>
__device__ __forceinline__ f32x16 mma(const u32x4& first, const u32x4& second, f32x16 c) {
  if constexpr (DT == kF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, first),
                                                  __builtin_bit_cast(f16x8, second), c, 0, 0, 0);
  } else if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, first),
                                                   __builtin_bit_cast(bf16x8, second), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(first[j]),
                                               __uint_as_float(second[j]), c, 0, 0, 0);
    return c;
  }
}

// The memory from p on, `records` bytes of it; what lies behind reads as 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t open(const void* p, int records) {
  const uint64_t at = (uint64_t)p;                 // (uniform, but not for the compiler)
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane(records), 0x00020000);
}

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// All that the wave has loaded, stored or read in LDS is done.
__device__ __forceinline__ void wait_all() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace

}  // namespace lowbit
