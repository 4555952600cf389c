// xent_tile.hpp -- the products of linear xent: tiles fed through LDS, summed on
// the matrix units, and what becomes of a tile's sums.
#pragma once

#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));
#define LOWBIT_LDS __attribute__((address_space(3)))

constexpr int kRowBytes = kXentRowBytes;   // of k, between two barriers
constexpr uint32_t kNowhere = 0x7FFFFFF0u; // beyond every buffer's records
constexpr float kLog2e = 1.44269502f;      // log2(e) to binary32

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
    const uint64_t at = (uint64_t)base;            // (uniform, but not for the compiler)
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(records), 0x00020000);
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

// The product of 32 rows of n with 32 rows of m over 32 bytes of k.  For
// binary32 four products take one element of each lane: k in another order, the
// same for both.
template <int DT>
__device__ __forceinline__ f32x16 mma(const u32x4& b, const u32x4& a, f32x16 c) {
  if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b),
                                                   __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(b[j]), __uint_as_float(a[j]), c, 0,
                                               0, 0);
    return c;
  }
}

// exp of a softmax term.  For binary32 results (within about 2 units in the
// last place) 2^t with t = x log2(e) and its rounding error made good; where d is
// rounded to bfloat16, or a part's sum taken from its largest term on, 2^t alone,
// off by |x| 2^-24 relative.
template <int DT>
__device__ __forceinline__ float exp_term(float x) {
  const float t = x * kLog2e;
  const float y = __builtin_amdgcn_exp2f(t);
  if constexpr (DT == kBF16) return y;
  const float e = __builtin_fmaf(x, kLog2e, -t) + x * 1.92596303e-8f;
  return x < -200.0f ? 0.0f : __builtin_fmaf(y, e * 0.693147182f, y);
}

template <int DT_, int TM_, int TN_, int WM_, int WN_, int SLOTS_>
struct Form {
  static constexpr int DT = DT_, TM = TM_, TN = TN_, WM = WM_, WN = WN_, SLOTS = SLOTS_;
  static constexpr int W = WM * WN, I = TM / WM / 32, J = TN / WN / 32, THREADS = 64 * W;
};

template <class F, int KIND>
struct TilePlan {
  XentCut cut;
  int64_t m, k;
  // count: rows that count (device), or the most there can be (host)
  __host__ __device__ TilePlan(const XentTileArgs& g, int64_t count)
      : cut(KIND == kXentDw ? g.m : count, g.n, steps(KIND == kXentDw ? count : g.k), F::TM, F::TN,
            F::SLOTS, g.may_cut != 0),
        m(KIND == kXentDw ? g.m : count), k(KIND == kXentDw ? count : g.k) {}
  static __host__ __device__ uint32_t steps(int64_t k) {
    return xent_steps(k, elem_size<F::DT>());
  }
};

__device__ __forceinline__ f32x4 quad(const f32x16& v, int q) {
  return (f32x4){v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}

// Four consecutive columns n .. n + 3 of row `row` of d, dx or dw.
template <int DT, int KIND>
__device__ __forceinline__ void emit(const XentTileArgs& g, float scale, int64_t row, int64_t n,
                                     f32x4 v) {
  if constexpr (KIND == kXentProb) {
    const float4 info = g.info[row];
    const int64_t target = (int64_t)__float_as_int(info.w) - g.col0 - n;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = exp_term<DT>(v[r] - info.x) * (info.y / scale);
      if (target == r) v[r] -= info.z / scale;
      if (n + r >= g.n) v[r] = 0.0f;
    }
    char* to = static_cast<char*>(g.out) + (row * g.ldo + n) * elem_size<DT>();
    if constexpr (DT == kF32) *reinterpret_cast<f32x4*>(to) = v;
    else *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    return;
  }
  if (n >= g.n) return;
  const int64_t to = (KIND == kXentDx ? (int64_t)g.map[row] : row) * g.ldo;
  v *= scale;
  if constexpr (DT == kF32) {
    float* p = static_cast<float*>(g.out) + to + n;
    if (n + 4 <= g.n) {
      *reinterpret_cast<u32x4_4*>(p) = __builtin_bit_cast(u32x4, v);
    } else {
      for (int r = 0; r < 3; ++r)
        if (n + r < g.n) p[r] = v[r];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(g.out) + to + n;
    const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
    if (n + 4 <= g.n) {
      *reinterpret_cast<u32x2_2*>(p) = (u32x2_2){lo, hi};
    } else {
      p[0] = (uint16_t)lo;
      if (n + 1 < g.n) p[1] = (uint16_t)(lo >> 16);
      if (n + 2 < g.n) p[2] = (uint16_t)hi;
    }
  }
}

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// All that the wave has loaded, stored or read in LDS is done.
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
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

// A tile's sums as the lanes hold them, TM x TN values in a row.
template <class F>
__device__ __forceinline__ f32x4* tile_base(float* base, int64_t tile) {
  return reinterpret_cast<f32x4*>(base) + tile * (F::TM * F::TN / 4);
}
template <class F>
__device__ __forceinline__ f32x4* lanes(float* base, int64_t tile) {
  return tile_base<F>(base, tile) + threadIdx.x;
}
template <class F>
__device__ __forceinline__ void store_lanes(f32x4* to, const f32x16 (&acc)[F::I][F::J]) {
#pragma unroll
  for (int i = 0; i < F::I; ++i)
#pragma unroll
    for (int j = 0; j < F::J; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) to[((i * F::J + j) * 4 + q) * F::THREADS] = quad(acc[i][j], q);
}

// LDS beside the two buffers: the row parts of the waves (stats), or 32 rows of 64
// columns of each wave's outputs.
template <class F, int KIND>
struct Side {
  static constexpr bool ROWS = KIND != kXentStats && F::DT == kBF16 && F::J == 2;
  static constexpr int BYTES = KIND == kXentStats ? F::WN * F::TM * 8 : ROWS ? F::W * 4096 : 16;
};

// 32 rows by 64 columns of bfloat16 outputs, which the lanes hold as in the tile
// kernel, through LDS (pieces of 16 bytes permuted by the row), so that each store
// writes whole lines: to(row, column) is where eight columns go, or null.
// Straight from the registers a store reaches 16 bytes of 32 rows each.
template <typename To>
__device__ __forceinline__ void store_rows(char* lds, int lane, const f32x16& a, const f32x16& b,
                                           To to) {
  const int r = lane % 32, h = lane / 32;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const f32x4 v = quad(q < 4 ? a : b, q % 4);
    *reinterpret_cast<u32x2*>(lds + r * 128 + (q ^ (r & 7)) * 16 + h * 8) =
        (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = k * 8 + lane / 8, c = lane % 8;
    const u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * 128 + (c ^ (row & 7)) * 16);
    uint16_t* p = to(row, c * 8);
    if (p) *reinterpret_cast<u32x4_2*>(p) = v;
  }
}

// What becomes of a tile's sums.
//
// d of bfloat16 inputs leaves in bfloat16: dx and dw are then products of bfloat16
// matrices, at 1.25 PFLOP/s, where binary32 ones reach 0.13 (a library's), so that
// two thirds of the gradient's operations would take ten times as long, and d is written
// and read twice in half the bytes.  It costs half a step of each of its elements: the
// gradient's root mean square error against 64 bits is 0.0024 of the gradient's own
// where the outputs' rounding alone makes 0.0017 (2011 x 131072 x 2048; where many
// terms add up alike, as over 8 Ki tokens, both 0.0017).
template <class F, int KIND>
__device__ __forceinline__ void finish(const XentTileArgs& g, f32x16 (&acc)[F::I][F::J], int64_t m,
                                       int64_t m0, int64_t n0, uint32_t tn, int wm, int wn, int lane,
                                       char* side) {
  constexpr int DT = F::DT, TM = F::TM, TN = F::TN, I = F::I, J = F::J;
  const int64_t ml = m0 + wm * (TM / F::WM) + lane % 32;          // + 32 i
  const int64_t nl = n0 + wn * (TN / F::WN) + lane / 32 * 4;      // + 32 j + at(r)
  const bool inside = n0 + TN <= g.n;
  auto at = [](int r) { return r / 4 * 8 + r % 4; };
  char* const mine = side + (wm * F::WN + wn) * 4096;             // (Side::ROWS)
  if constexpr (KIND == kXentStats) {
    float2* const halves = reinterpret_cast<float2*>(side);       // [WN][TM]
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t row = ml + 32 * i;
      // (nl counts from the piece's first column; a piece that ends inside a tile is the last
      // one, so that no target lies among the columns behind it)
      const int64_t target = row < m ? (int64_t)__float_as_int(g.info[row].w) - g.col0 - nl : -1;
      if (__any(target >= 0 && target < 32 * J)) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (target == 32 * j + at(r)) g.hit[row] = acc[i][j][r];
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (!inside && nl + 32 * j + at(r) >= g.n) acc[i][j][r] = -INFINITY;
          top = fmaxf(top, acc[i][j][r]);
        }
      top = fmaxf(top, __shfl_xor(top, 32));
      // bfloat16: 2^(l log2(e) - base) in two instructions; base is off by at most
      // |top| 2^-24, as lse itself
      const float base = top == -INFINITY ? 0.0f : DT == kF32 ? top : top * kLog2e;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float l = acc[i][j][r];
          if constexpr (DT == kF32) sum += exp_term<DT>(l - base);
          else sum += __builtin_amdgcn_exp2f(__builtin_fmaf(l, kLog2e, -base));
        }
      sum += __shfl_xor(sum, 32);
      __builtin_amdgcn_sched_barrier(0);
      if (lane < 32) halves[wn * TM + wm * (TM / F::WM) + i * 32 + lane] = make_float2(top, sum);
    }
    wait_lds();
    barrier();
    const int r = threadIdx.x;
    if (r < TM && m0 + r < m) {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < F::WN; ++w) top = fmaxf(top, halves[w * TM + r].x);
#pragma unroll
      for (int w = 0; w < F::WN; ++w) {
        const float2 p = halves[w * TM + r];
        sum += p.x == -INFINITY ? p.y : p.y * exp_term<kF32>(p.x - top);
      }
      g.part[(m0 + r) * g.parts + g.part0 + tn] = make_float2(top, sum);
    }
  } else if constexpr (KIND == kXentProb) {
    const float scale = DT == kF32 ? 1.0f : *g.scale;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t row = ml + 32 * i;
      const float4 info = g.info[row];             // (rows beyond those that count have some, too)
      const float both = info.y / scale, own = info.z / scale;
      const int64_t target = (int64_t)__float_as_int(info.w) - g.col0 - nl;
      char* to = static_cast<char*>(g.out) + (row * g.ldo + nl) * elem_size<DT>();
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          acc[i][j][r] = exp_term<DT>(acc[i][j][r] - info.x) * both;
          if (!inside && nl + 32 * j + at(r) >= g.n) acc[i][j][r] = 0.0f;
        }
      if (__any(target >= 0 && target < 32 * J)) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (target == 32 * j + at(r) && nl + target < g.n) acc[i][j][r] -= own;
      }
      if constexpr (Side<F, KIND>::ROWS) {
        uint16_t* const d0 = static_cast<uint16_t*>(g.out) +
                             (m0 + wm * (TM / F::WM) + 32 * i) * g.ldo + n0 + wn * (TN / F::WN);
        store_rows(mine, lane, acc[i][0], acc[i][1],
                   [&](int r, int c) { return d0 + r * g.ldo + c; });
        continue;
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 d = quad(acc[i][j], q);
          if constexpr (DT == kF32)
            *reinterpret_cast<f32x4*>(to + 128 * j + 32 * q) = d;
          else
            *reinterpret_cast<uint2*>(to + 64 * j + 16 * q) =
                make_uint2(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]));
        }
    }
  } else {
    const float scale = DT == kF32 ? 1.0f : *g.scale;
    if constexpr (Side<F, KIND>::ROWS) {
      if (inside) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int64_t first = m0 + wm * (TM / F::WM) + 32 * i;
          uint16_t* const out = static_cast<uint16_t*>(g.out) + n0 + wn * (TN / F::WN);
          store_rows(mine, lane, acc[i][0] * scale, acc[i][1] * scale, [&](int r, int c) {
            const int64_t row = first + r;
            return row < m ? out + (KIND == kXentDx ? (int64_t)g.map[row] : row) * g.ldo + c
                           : nullptr;
          });
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t row = ml + 32 * i;
      if (row < m) {
        if (inside) {
          char* to = static_cast<char*>(g.out) +
                     ((KIND == kXentDx ? (int64_t)g.map[row] : row) * g.ldo + nl) * elem_size<DT>();
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4 v = quad(acc[i][j], q) * scale;
              if constexpr (DT == kF32)
                *reinterpret_cast<u32x4_4*>(to + 128 * j + 32 * q) = __builtin_bit_cast(u32x4, v);
              else
                *reinterpret_cast<u32x2_2*>(to + 64 * j + 16 * q) =
                    (u32x2_2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            }
        } else {
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              emit<DT, KIND>(g, scale, row, nl + 32 * j + 8 * q, quad(acc[i][j], q));
        }
      }
    }
  }
}

// Bound by the matrix units at the clock that power leaves them (about 1.9 GHz in the
// largest form; machines differ): 8192 x 50257 x 4096 bfloat16 2.55 to 2.74 ms, 1.32 to
// 1.23 PFLOP/s, dx of 6144 x 25344 x 4096 1.02 ms, 1.25, dw 1.23, d 1.18; a large
// library product 1.31.
// Without the loads the loop reaches 1.55 on random data and 2.09 on zeros; with
// four waves of 128 x 128, which read a third less from LDS, it is no faster and spills.
// Few rows are bound by reading w: 13 x 50257 x 1024 17.5 us, 5.9 TB/s.
//
// W waves, each I x J products of 32 x 32.  Lane l holds of product (i, j) row
// 32 i + l mod 32 of m and rows 32 j + 8 q + 4 (l / 32) + r of n: four times
// four consecutive columns of the output's row.  Two buffers in LDS: while the
// matrix units work on one, the other is filled.
template <class F, int KIND>
__global__ void __launch_bounds__(F::THREADS, F::SLOTS * F::W / 1024) xent_tile_kernel(XentTileArgs g) {
  constexpr int DT = F::DT, TM = F::TM, TN = F::TN, W = F::W, I = F::I, J = F::J;
  constexpr bool AO = KIND == kXentDw, BO = KIND == kXentDx || KIND == kXentDw;
  constexpr int K = kRowBytes / elem_size<DT>();
  __shared__ __attribute__((aligned(1024))) char la0[TM * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb0[TN * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char la1[TM * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb1[TN * kRowBytes];
  __shared__ __attribute__((aligned(16))) char side[Side<F, KIND>::BYTES];
  const TilePlan<F, KIND> plan(g, __builtin_amdgcn_readfirstlane(*g.count));
  const XentCut& cut = plan.cut;
  const int64_t m = plan.m, k = plan.k;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / F::WN, wn = wave % F::WN;

  const int64_t steps = plan.steps(k);
  const uint32_t units = cut.units();
  int slot, s0, s1;
  uint32_t tile, tm, tn;
  auto take = [&](uint32_t u) {
    const XentUnit v = cut.unit(u, (uint32_t)steps);
    tm = __builtin_amdgcn_readfirstlane(v.tm);     // (the compiler does not see that they are uniform)
    tn = __builtin_amdgcn_readfirstlane(v.tn);
    s0 = __builtin_amdgcn_readfirstlane(v.s0);
    s1 = __builtin_amdgcn_readfirstlane(v.s1);
    slot = __builtin_amdgcn_readfirstlane(v.slot);
    tile = __builtin_amdgcn_readfirstlane(v.tile);
  };

  constexpr int NA = Feed<DT, TM, W, AO>::LOADS, NB = Feed<DT, TN, W, BO>::LOADS, N = NA + NB;
  constexpr int Q = DT == kF32 ? 4 : 1;            // matrix instructions of a product
  constexpr int RD = I * (AO ? Q > 1 ? 4 : 2 : 1) + J * (BO ? Q > 1 ? 4 : 2 : 1);
  Feed<DT, TM, W, AO> fa;
  Feed<DT, TN, W, BO> fb;
  Frag<DT, TM, AO> ra;
  Frag<DT, TN, BO> rb;
  fa.init(g.lda, wave, lane);
  fb.init(g.ldb, wave, lane);
  ra.init(wm * (TM / F::WM), lane);
  rb.init(wn * (TN / F::WN), lane);
  u32x4 fra[2][I], frb[2][J];
  f32x16 acc[I][J];

  auto kleft = [&](int s) { return (int)min(k - (int64_t)s * K, (int64_t)K); };
  auto issue = [&](char* la, char* lb, int s) {
    const auto qa = fa.open(s < s1), qb = fb.open(s < s1);
#pragma unroll
    for (int j = 0; j < NA; ++j) fa.load(qa, la, wave, kleft(s), j);
#pragma unroll
    for (int j = 0; j < NB; ++j) fb.load(qb, lb, wave, kleft(s), j);
    fa.next();
    fb.next();
  };
  auto begin = [&] {                               // the unit's first two steps
    fa.seek(g.a, g.lda, AO ? k : g.m, (int64_t)tm * TM, (int64_t)s0 * K);
    fb.seek(g.b, g.ldb, BO ? k : g.n, (int64_t)tn * TN, (int64_t)s0 * K);
    issue(la0, lb0, s0);
    issue(la1, lb1, s0 + 1);
  };
  auto read = [&](int to, const char* la, const char* lb, int kk) {
#pragma unroll
    for (int j = 0; j < J; ++j) frb[to][j] = rb.load(lb, j, kk);
#pragma unroll
    for (int i = 0; i < I; ++i) fra[to][i] = ra.load(la, i, kk);
  };
  auto mul = [&](int f) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = mma<DT>(frb[f][j], fra[f][i], acc[i][j]);
    spread_reads<RD, I * J * Q>();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step s, in la and lb, whose first quarter is in registers.  While a quarter is
  // multiplied the next is read; before the last, everybody has read all of
  // this step, the next one has arrived, and the loads of the one after it begin.
  auto step = [&](char* la, char* lb, const char* na, const char* nb, int s) {
    const auto qa = fa.open(s + 2 < s1), qb = fb.open(s + 2 < s1);
    const int kl = kleft(s + 2);
    read(1, la, lb, 1);
    mul(0);
    read(0, la, lb, 2);
    mul(1);
    read(1, la, lb, 3);
    mul(0);
    wait_loads();
    barrier();
    read(0, na, nb, 0);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        acc[i][j] = mma<DT>(frb[1][j], fra[1][i], acc[i][j]);
        const int p = i * J + j;
#pragma unroll
        for (int u = N * p / (I * J); u < N * (p + 1) / (I * J); ++u) {
          if (u < NA) fa.load(qa, la, wave, kl, u);
          else fb.load(qb, lb, wave, kl, u - NA);
        }
      }
    fa.next();
    fb.next();
    spread_loads<RD, I * J, Q, N>();
    __builtin_amdgcn_sched_barrier(0);
  };

  uint32_t unit = blockIdx.x;
  if (unit >= units) return;
  take(unit);
  begin();
  for (;;) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    if (KIND == kXentDx && !g.first && slot < 0) { // the earlier pieces' sums
      const f32x4* from = lanes<F>(g.acc, tile);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = from[((i * J + j) * 4 + q) * F::THREADS];
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][4 * q + r] = v[r];
          }
    }
    wait_loads();
    barrier();
    read(0, la0, lb0, 0);
    __builtin_amdgcn_sched_barrier(0);
    int s = s0;
    for (; s + 1 < s1; s += 2) {
      step(la0, lb0, la1, lb1, s);
      step(la1, lb1, la0, lb0, s + 1);
    }
    if (s < s1) step(la0, lb0, la1, lb1, s);
    wait_loads();
    barrier();                                     // nobody reads la0 .. lb1 any more

    const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TN;
    const uint32_t tn_done = tn;
    const int slot_done = slot;
    const uint32_t tile_done = tile;
    unit += gridDim.x;
    const bool more = unit < units;
    if (more) {                                    // the next unit's loads, meanwhile
      take(unit);
      begin();
    }
    if (slot_done >= 0)
      store_lanes<F>(lanes<F>(g.partial, slot_done), acc);
    else if (KIND == kXentDx && !g.last)
      store_lanes<F>(lanes<F>(g.acc, tile_done), acc);
    else
      finish<F, KIND>(g, acc, m, m0, n0, tn_done, wm, wn, lane, side);
    if (!more) break;
  }
}

// The cut tiles: their parts' sums added, every fourth part by one of four waves,
// and the waves' sums in order.  A unit is 64 lanes' four values.
template <class F, int KIND>
__global__ void __launch_bounds__(256) xent_add_kernel(XentTileArgs g) {
  __shared__ f32x4 sums[4][64];
  const TilePlan<F, KIND> plan(g, __builtin_amdgcn_readfirstlane(*g.count));
  const XentCut& cut = plan.cut;
  const float scale = F::DT == kF32 ? 1.0f : *g.scale;
  const int lane = lane_id(), mine = threadIdx.x >> 6;
  constexpr uint32_t C = F::I * F::J * 4 * F::W;
  for (uint32_t u = blockIdx.x; u < cut.rest * C; u += gridDim.x) {
    const uint32_t r = u / C, in = u % C;
    const int wave = in % F::W, q = in / F::W % 4;
    const int i = in / F::W / 4 / F::J, j = in / F::W / 4 % F::J;
    const int64_t at = (int64_t)(in / F::W) * F::THREADS + wave * 64 + lane;
    f32x4* sum = nullptr;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (KIND == kXentDx) {
      if (!(g.first && g.last)) sum = tile_base<F>(g.acc, cut.whole + r) + at;
      if (!g.first && mine == 0) v = *sum;
    }
    const f32x4* from = tile_base<F>(g.partial, r) + at;
    const int64_t next = (int64_t)cut.rest * (F::TM * F::TN / 4);
#pragma unroll 8
    for (uint32_t p = mine; p < cut.parts; p += 4) v += from[p * next];
    sums[mine][lane] = v;
    __syncthreads();
    if (mine == 0) {
#pragma unroll
      for (int w = 1; w < 4; ++w) v += sums[w][lane];
      uint32_t tm, tn;
      cut.place(cut.whole + r, tm, tn);
      const int64_t row = (int64_t)tm * F::TM + wave / F::WN * (F::TM / F::WM) + lane % 32 + 32 * i;
      const int64_t n = (int64_t)tn * F::TN + wave % F::WN * (F::TN / F::WN) + lane / 32 * 4 +
                        32 * j + 8 * q;
      if (KIND == kXentDx && !g.last) *sum = v;
      else if (row < plan.m) emit<F::DT, KIND>(g, scale, row, n, v);
    }
    __syncthreads();
  }
}

// The same for tiles of logits whose rows' maxima and sums are wanted: a workgroup
// a tile, whole in registers again.
template <class F>
__global__ void __launch_bounds__(F::THREADS) xent_add_stats_kernel(XentTileArgs g) {
  __shared__ __attribute__((aligned(16))) char side[Side<F, kXentStats>::BYTES];
  const TilePlan<F, kXentStats> plan(g, __builtin_amdgcn_readfirstlane(*g.count));
  const XentCut& cut = plan.cut;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = blockIdx.x;
  if (r >= cut.rest) return;
  f32x16 acc[F::I][F::J];
#pragma unroll
  for (int i = 0; i < F::I; ++i)
#pragma unroll
    for (int j = 0; j < F::J; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
#pragma unroll 2
  for (uint32_t p = 0; p < cut.parts; ++p) {
    const f32x4* from = lanes<F>(g.partial, (int64_t)p * cut.rest + r);
#pragma unroll
    for (int i = 0; i < F::I; ++i)
#pragma unroll
      for (int j = 0; j < F::J; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = from[((i * F::J + j) * 4 + q) * F::THREADS];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
        }
  }
  uint32_t tm, tn;
  cut.place(cut.whole + r, tm, tn);
  finish<F, kXentStats>(g, acc, plan.m, (int64_t)tm * F::TM, (int64_t)tn * F::TN, tn, wave / F::WN,
                        wave % F::WN, lane, side);
}

// g.m, and g.k for dw: the most rows that may count.
template <class F, int KIND>
lowbit_status launch_form_kind(const XentTileArgs& g, hipStream_t s) {
  const TilePlan<F, KIND> plan(g, KIND == kXentDw ? g.k : g.m);
  if (g.may_cut && !g.partial) return LOWBIT_EINVAL;
  // one workgroup for each slot, each taking every SLOTS-th unit (fewer rows
  // may leave fewer tiles whole and more cut: as many workgroups as tiles do not always do)
  const uint32_t blocks = plan.cut.tiles < F::SLOTS && !g.may_cut ? plan.cut.tiles : F::SLOTS;
  const lowbit_status st = launch(&xent_tile_kernel<F, KIND>, blocks, F::THREADS, s, g);
  if (st != LOWBIT_OK || !g.may_cut) return st;
  if (KIND == kXentDw && plan.cut.rest == 0) return st;    // (the same tiles whatever counts)
  if constexpr (KIND == kXentStats)        // (fewer tiles than slots, all of them cut or none)
    return launch(&xent_add_stats_kernel<F>, plan.cut.tiles, F::THREADS, s, g);
  else
    return launch(&xent_add_kernel<F, KIND>, 2048, 256, s, g);
}

template <class F>
lowbit_status launch_form(int kind, const XentTileArgs& g, hipStream_t s) {
  return kind == kXentStats  ? launch_form_kind<F, kXentStats>(g, s)
         : kind == kXentProb ? launch_form_kind<F, kXentProb>(g, s)
         : kind == kXentDx   ? launch_form_kind<F, kXentDx>(g, s)
                             : launch_form_kind<F, kXentDw>(g, s);
}

}  // namespace

}  // namespace lowbit
