// xent_tile.hpp -- the products of linear xent: tiles fed through LDS, summed on
// the matrix units, and what becomes of a tile's sums.
#pragma once

#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));
#define LOWBIT_LDS __attribute__((address_space(3)))

constexpr int kRowBytes = 128;             // of k, between two barriers
constexpr uint32_t kNowhere = 0x7FFFFFF0u; // beyond every buffer's records
constexpr float kLog2e = 1.44269502f;      // log2(e) to binary32

// One operand's way into LDS: T rows of the tile by 128 bytes of k, 16 bytes a
// lane straight from memory, the W waves taking turns.  OUTER: k is the
// matrix's row, and LDS holds rows of k; else rows of the tile.  The pieces of
// a row in LDS are permuted by the row's number, so that the reads of Frag
// meet no bank twice; a load writes LDS in lane order, so each lane fetches
// the piece that belongs in its place.  What lies behind the matrix's end reads as 0.
template <int DT, int T, int W, bool OUTER>
struct Feed {
  static constexpr int ES = elem_size<DT>(), K = kRowBytes / ES, LOADS = T / 8 / W;
  static constexpr int KR = 1024 / (T * ES);     // OUTER: rows of k in a wave's load
  const char* base;
  int64_t left, jstep, kstep;                    // bytes
  uint32_t voff, vcol;
  int kin;                                       // the lane's first k within the step

  // the pieces (32 bytes of bfloat16, 64 of binary32: 16 columns) of row k are xored with this
  static __device__ __forceinline__ constexpr int mix(int k) {
    return (DT == kF32 ? k >> 2 & 3 : (k & 3) | (k >> 1 & 4)) & (T / 16 - 1);
  }
  // rows: of the matrix in memory; k0: where to begin
  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t rows, int64_t row0,
                                       int64_t k0, int wave, int lane) {
    const char* at = static_cast<const char*>(p);
    if constexpr (OUTER) {
      constexpr int L = T * ES / 16, P = ES;     // lanes of a row, of a piece
      const int k = wave * KR + lane / L, slot = lane % L;
      base = at + (k0 * ld + row0) * ES;
      left = ((rows - k0) * ld - row0) * ES;
      jstep = (int64_t)W * KR * ld * ES;
      kstep = K * ld * ES;
      kin = 0;
      voff = (uint32_t)(k * ld * ES);
      vcol = ((slot / P ^ mix(k)) * P + slot % P) * 16;
    } else {
      const int r = wave * 8 + lane / 8, c = lane % 8 ^ (r >> 1 & 7);
      base = at + (row0 * ld + k0) * ES;
      left = ((rows - row0) * ld - k0) * ES;
      jstep = (int64_t)W * 8 * ld * ES;
      kstep = kRowBytes;
      kin = c * (16 / ES);
      voff = (uint32_t)(r * ld * ES);
      vcol = c * 16;
    }
  }
  __device__ __forceinline__ void issue(char* lds, int wave, int64_t kleft) {
    static_assert(LOADS >= 1 && (!OUTER || K % (W * KR) == 0), "");
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      uint32_t v = voff + (OUTER ? vcol ^ mix(j * W * KR) * 16 * ES : vcol);
      if (!OUTER && kin >= kleft) v = kNowhere;
      const int64_t l = left - j * jstep;
      const int records = (int)(l < 0 ? 0 : l > kNowhere ? kNowhere : l);
      __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char*>(base + j * jstep), 0, records, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LOWBIT_LDS void*)(lds + (j * W + wave) * 1024),
                                               16, v, 0, 0, 0);
    }
    base += kstep;
    left -= kstep;
  }
};

// A lane's part of 16 rows by 64 bytes of k: row lane mod 16, the (lane / 16)-th 16 bytes.
template <int DT, int T, bool OUTER>
struct Frag {
  static constexpr int ES = elem_size<DT>(), PITCH = T * ES;
  uint32_t at[2];
  int piece, f;                                  // OUTER
  __device__ __forceinline__ void init(int row0, int lane) {
    const int g = lane / 16, i = lane % 16;
    if constexpr (OUTER) {
      f = Feed<DT, T, 1, true>::mix(DT == kF32 ? 4 * g : 8 * g + i / 4);
      piece = row0 / 16;
      at[0] = DT == kF32 ? 4 * g * PITCH + i * 4 : (8 * g + i / 4) * PITCH + i % 4 * 8;
    } else {
      const int r = row0 + i, s = r >> 1 & 7;
      at[0] = r * kRowBytes + (g ^ s) * 16;
      at[1] = r * kRowBytes + ((4 + g) ^ s) * 16;
    }
  }
  // 16-row piece i of the wave, half kk of the step
  __device__ __forceinline__ u32x4 load(const char* lds, int i, int kk) const {
    if constexpr (!OUTER) {
      return *reinterpret_cast<const u32x4*>(lds + at[kk] + i * 16 * kRowBytes);
    } else if constexpr (DT == kF32) {
      const char* p = lds + at[0] + ((piece + i) ^ f) * 64 + kk * 16 * PITCH;
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * PITCH);
      return v;
    } else {
      // 16 lanes read 16 columns of four rows of k and get a column each
      const char* p = lds + at[0] + ((piece + i) ^ f) * 32 + kk * 32 * PITCH;
      typedef LOWBIT_LDS s16x4* lp;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(LOWBIT_LDS char*)p);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(LOWBIT_LDS char*)(p + 4 * PITCH));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// The product of 16 rows of n with 16 rows of m over 64 bytes of k.  For
// binary32 four products take one element of each lane: k in another order, the
// same for both.
template <int DT>
__device__ __forceinline__ f32x4 mma(const u32x4& b, const u32x4& a, f32x4 c) {
  if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b),
                                                   __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[j]), __uint_as_float(a[j]), c, 0,
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

// Which tiles of a product are cut along k.  The workgroups that the chip holds
// at one time (SLOTS) take whole tiles as long as all of them have one; the
// remaining tiles are cut into as many parts as there are slots for them, of
// four steps of k at least, and the parts' sums are added by a second kernel.
// Two rounds instead of one and a half would leave half of the chip idle in the second.
struct XentCut {
  uint32_t across, down, tiles, whole;           // whole: tiles that are not cut
  uint32_t rest, parts;                          // tiles that are, each into `parts`
  __host__ __device__ XentCut(int64_t m, int64_t n, uint32_t k_steps, uint32_t tm, uint32_t tn,
                              uint32_t slots, bool may_cut) {
    across = ((uint32_t)n + tn - 1) / tn;
    down = ((uint32_t)m + tm - 1) / tm;
    tiles = across * down;
    rest = tiles % slots;
    parts = rest && may_cut ? slots / rest : 1;
    if (parts > k_steps / 4) parts = k_steps / 4;
    if (parts <= 1) {
      parts = 1;
      rest = 0;
    }
    whole = tiles - rest;
  }
};

// XCD x of 8 takes a contiguous run of the units; -1 for workgroups beyond them.
__device__ __forceinline__ int xcd_run(uint32_t block, uint32_t units) {
  const uint32_t x = block % kXcds, q = block / kXcds;
  const uint32_t each = units / kXcds, more = units % kXcds;
  if (q >= each + (x < more ? 1 : 0)) return -1;
  return x * each + (x < more ? x : more) + q;
}

template <int DT_, int TM_, int TN_, int WM_, int WN_, int SLOTS_>
struct Form {
  static constexpr int DT = DT_, TM = TM_, TN = TN_, WM = WM_, WN = WN_, SLOTS = SLOTS_;
  static constexpr int W = WM * WN, I = TM / WM / 16, J = TN / WN / 16, THREADS = 64 * W;
};

template <class F, int KIND>
struct TilePlan {
  XentCut cut;
  int64_t m, k;
  // count: rows that count (device), or the most there can be (host)
  __host__ __device__ TilePlan(const XentTileArgs& g, int64_t count)
      : cut(KIND == kXentDw ? g.m : count, g.n, steps(KIND == kXentDw ? count : g.k), F::TM, F::TN,
            F::SLOTS, KIND == kXentDx || KIND == kXentDw),
        m(KIND == kXentDw ? g.m : count), k(KIND == kXentDw ? count : g.k) {}
  static __host__ __device__ uint32_t steps(int64_t k) {
    constexpr int K = kRowBytes / elem_size<F::DT>();
    return (uint32_t)((k + K - 1) / K);
  }
  // tiles in bands of 8 rows of tiles: the 32 that an XCD's CUs hold at one time
  // read 8 panels of a and 4 of b through its L2
  __device__ __forceinline__ void place(uint32_t tile, uint32_t& tm, uint32_t& tn) const {
    const uint32_t band = tile / (8 * cut.across), in = tile % (8 * cut.across);
    const uint32_t high = cut.down - band * 8 < 8 ? cut.down - band * 8 : 8;
    tm = band * 8 + in % high;
    tn = in / high;
  }
};

// Four consecutive columns n .. n + 3 of row `row` of dx or dw.
template <int DT, int KIND>
__device__ __forceinline__ void emit(const XentTileArgs& g, float scale, int64_t row, int64_t n,
                                     f32x4 v) {
  if (n >= g.n) return;
  int64_t to = row * g.ldo;
  if constexpr (KIND == kXentDx) {
    if (!(g.first && g.last)) {
      f32x4* sum = reinterpret_cast<f32x4*>(g.acc + row * g.ldacc + n);
      if (!g.first) v += *sum;
      if (!g.last) {
        *sum = v;
        return;
      }
    }
    to = (int64_t)g.map[row] * g.ldo;
  }
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

// W waves, each I x J products of 16 x 16.  Lane l holds of product (i, j) row
// 16 i + l mod 16 of m and rows 16 j + 4 (l / 16) + r of n: four consecutive
// columns of the output's row.  Two buffers in LDS: while the matrix units work
// on one, the other is filled.
template <class F, int KIND>
__global__ void __launch_bounds__(F::THREADS) xent_tile_kernel(XentTileArgs g) {
  constexpr int DT = F::DT, TM = F::TM, TN = F::TN, W = F::W, I = F::I, J = F::J;
  constexpr bool AO = KIND == kXentDw, BO = KIND == kXentDx || KIND == kXentDw;
  constexpr int K = kRowBytes / elem_size<DT>();
  __shared__ __attribute__((aligned(1024))) char la0[TM * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb0[TN * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char la1[TM * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb1[TN * kRowBytes];
  const TilePlan<F, KIND> plan(g, *g.count);
  const XentCut& cut = plan.cut;
  const int64_t m = plan.m, k = plan.k;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / F::WN, wn = wave % F::WN;

  int tile, slot = -1, s0 = 0, s1 = (int)plan.steps(k);
  if (blockIdx.x < cut.whole) {
    tile = xcd_run(blockIdx.x, cut.whole);
  } else {
    slot = xcd_run(blockIdx.x - cut.whole, cut.rest * cut.parts);
    if (slot < 0) return;
    const uint32_t part = (uint32_t)slot / cut.rest, all = s1;
    tile = cut.whole + (uint32_t)slot % cut.rest;
    s0 = all / cut.parts * part + min(part, all % cut.parts);
    s1 = s0 + all / cut.parts + (part < all % cut.parts ? 1 : 0);
  }
  uint32_t tm, tn;
  plan.place(tile, tm, tn);
  const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TN;

  f32x4 acc[I][J];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  Feed<DT, TM, W, AO> fa;
  Feed<DT, TN, W, BO> fb;
  fa.init(g.a, g.lda, AO ? k : g.m, m0, (int64_t)s0 * K, wave, lane);
  fb.init(g.b, g.ldb, BO ? k : g.n, n0, (int64_t)s0 * K, wave, lane);
  Frag<DT, TM, AO> ra;
  Frag<DT, TN, BO> rb;
  ra.init(wm * (TM / F::WM), lane);
  rb.init(wn * (TN / F::WN), lane);

  if (s0 < s1) {
    fa.issue(la0, wave, k - (int64_t)s0 * K);
    fb.issue(lb0, wave, k - (int64_t)s0 * K);
  }
  auto step = [&](const char* la, const char* lb, char* na, char* nb, int s) {
    __syncthreads();               // the loads have arrived, and nobody reads na and nb any more
    if (s + 1 < s1) {
      fa.issue(na, wave, k - (int64_t)(s + 1) * K);
      fb.issue(nb, wave, k - (int64_t)(s + 1) * K);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4 a[I], b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = rb.load(lb, j, kk);
#pragma unroll
      for (int i = 0; i < I; ++i) a[i] = ra.load(la, i, kk);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = mma<DT>(b[j], a[i], acc[i][j]);
    }
  };
  for (int s = s0; s < s1; s += 2) {
    step(la0, lb0, la1, lb1, s);
    if (s + 1 < s1) step(la1, lb1, la0, lb0, s + 1);
  }

  const int64_t ml = m0 + wm * (TM / F::WM) + lane % 16;          // + 16 i
  const int64_t nl = n0 + wn * (TN / F::WN) + lane / 16 * 4;      // + 16 j + r
  const bool inside = n0 + TN <= g.n;
  if constexpr (KIND == kXentStats) {
    float2* halves = reinterpret_cast<float2*>(la0);              // [WN][TM]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t row = ml + 16 * i;
      const int64_t target = row < m ? (int64_t)__float_as_int(g.info[row].w) - nl : -1;
      if (__any(target >= 0 && target < 16 * J)) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (target == 16 * j + r) g.hit[row] = acc[i][j][r];
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (!inside && nl + 16 * j + r >= g.n) acc[i][j][r] = -INFINITY;
          top = fmaxf(top, acc[i][j][r]);
        }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      // bfloat16: 2^(l log2(e) - base) in two instructions; base is off by at most
      // |top| 2^-24, as lse itself
      const float base = top == -INFINITY ? 0.0f : DT == kF32 ? top : top * kLog2e;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float l = acc[i][j][r];
          if constexpr (DT == kF32) sum += exp_term<DT>(l - base);
          else sum += __builtin_amdgcn_exp2f(__builtin_fmaf(l, kLog2e, -base));
        }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (lane < 16) halves[wn * TM + wm * (TM / F::WM) + i * 16 + lane] = make_float2(top, sum);
    }
    __syncthreads();
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
      const int64_t row = ml + 16 * i;
      const float4 info = row < m ? g.info[row] : make_float4(0, 0, 0, __int_as_float(-1));
      const float both = info.y / scale, own = info.z / scale;
      const int64_t target = (int64_t)__float_as_int(info.w) - g.col0 - nl;
      char* to = static_cast<char*>(g.out) + (row * g.ldo + nl) * elem_size<DT>();
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[i][j][r] = exp_term<DT>(acc[i][j][r] - info.x) * both;
          if (!inside && nl + 16 * j + r >= g.n) acc[i][j][r] = 0.0f;
        }
      if (__any(target >= 0 && target < 16 * J)) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (target == 16 * j + r && nl + target < g.n) acc[i][j][r] -= own;
      }
      if (row < m) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const f32x4 d = acc[i][j];
          if constexpr (DT == kF32)
            *reinterpret_cast<f32x4*>(to + 64 * j) = d;
          else
            *reinterpret_cast<uint2*>(to + 32 * j) =
                make_uint2(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]));
        }
      }
    }
  } else {
    if (slot >= 0) {               // a part's sums, as the lanes hold them
      f32x4* to = reinterpret_cast<f32x4*>(g.partial) + (int64_t)slot * (TM * TN / 4) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) to[(i * J + j) * F::THREADS] = acc[i][j];
      return;
    }
    const float scale = DT == kF32 ? 1.0f : *g.scale;
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (ml + 16 * i < m) {
#pragma unroll
        for (int j = 0; j < J; ++j) emit<DT, KIND>(g, scale, ml + 16 * i, nl + 16 * j, acc[i][j]);
      }
  }
}

// The cut tiles: their parts' sums added in order.
template <class F, int KIND>
__global__ void __launch_bounds__(F::THREADS) xent_add_kernel(XentTileArgs g) {
  const TilePlan<F, KIND> plan(g, *g.count);
  const XentCut& cut = plan.cut;
  const float scale = F::DT == kF32 ? 1.0f : *g.scale;
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  constexpr int C = F::I * F::J;
  for (uint32_t u = blockIdx.x; u < cut.rest * C; u += gridDim.x) {
    const uint32_t r = u / C;
    const int i = (int)(u % C) / F::J, j = (int)(u % C) % F::J;
    uint32_t tm, tn;
    plan.place(cut.whole + r, tm, tn);
    const int64_t row = (int64_t)tm * F::TM + wave / F::WN * (F::TM / F::WM) + lane % 16 + 16 * i;
    const int64_t n = (int64_t)tn * F::TN + wave % F::WN * (F::TN / F::WN) + lane / 16 * 4 + 16 * j;
    if (row >= plan.m) continue;
    const f32x4* from = reinterpret_cast<const f32x4*>(g.partial) + (int64_t)r * (F::TM * F::TN / 4) +
                        (u % C) * F::THREADS + threadIdx.x;
    f32x4 v = from[0];
#pragma unroll 8
    for (uint32_t p = 1; p < cut.parts; ++p)
      v += from[(int64_t)(p * cut.rest) * (F::TM * F::TN / 4)];
    emit<F::DT, KIND>(g, scale, row, n, v);
  }
}

// g.m, and g.k for dw: the most rows that may count.
template <class F, int KIND>
lowbit_status launch_form_kind(const XentTileArgs& g, hipStream_t s) {
  const TilePlan<F, KIND> plan(g, KIND == kXentDw ? g.k : g.m);
  // Where fewer rows count, fewer tiles may be whole, and more cut, into SLOTS
  // parts at most (dx), or the tiles be cut into fewer parts (dw).
  const uint32_t blocks = KIND == kXentDx   ? plan.cut.tiles + F::SLOTS
                          : KIND == kXentDw ? plan.cut.whole + plan.cut.rest * plan.cut.parts
                                            : plan.cut.tiles;
  const lowbit_status st = launch(&xent_tile_kernel<F, KIND>, blocks, F::THREADS, s, g);
  if constexpr (KIND == kXentDx || KIND == kXentDw) {
    if (st == LOWBIT_OK && (KIND == kXentDx || plan.cut.rest))
      return launch(&xent_add_kernel<F, KIND>, 512, F::THREADS, s, g);
  }
  return st;
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
