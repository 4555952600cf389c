// attn.hpp -- what the attention kernels share: the tiles' way through LDS into
// the operands of the matrix instructions, which sequence a tile belongs to, and what
// its queries see.
#pragma once

#include "block.hpp"
#include "matrix_unit.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

constexpr float kLog2e = 1.44269502f;        // log2(e) to binary32
constexpr float kLn2 = 0.693147182f;

constexpr int kWaves = 4, kAttnThreads = 64 * kWaves;
constexpr int kRowsPerTile = kAttnRows;      // of a workgroup: 32 of each wave
static_assert(kRowsPerTile == 32 * kWaves, "");

// Scores are kept in units of which exp takes the fewest instructions: of log2 for
// bfloat16 (2^t), natural ones for binary32, where the rounding error of x log2(e)
// is made good so that results keep binary32's accuracy.
template <int DT>
__host__ __device__ constexpr float unit_of() { return DT == kF32 ? 1.0f : kLog2e; }
// Of binary32 arguments up to 80: beyond, an infinity times a correction of 0 or less would be NaN.
template <int DT>
__device__ __forceinline__ float exp_unit(float x) {
  if constexpr (DT == kBF16) return __builtin_amdgcn_exp2f(x);
  const float t = x * kLog2e;
  const float y = __builtin_amdgcn_exp2f(t);
  const float e = __builtin_fmaf(x, kLog2e, -t) + x * 1.92596303e-8f;
  return x < -200.0f ? 0.0f : __builtin_fmaf(y, e * kLn2, y);
}

// v of the lane and of the one 32 further on, or back.
__device__ __forceinline__ float other_half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_halves_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// N products whose operands come from LDS: load(i) reads the i-th's, use(i, operands)
// multiplies.  The reads run A products ahead, in this order: left alone, the compiler reads
// each operand right before its product and waits for it.
template <int A, class Load>
__device__ __forceinline__ auto read_first(Load load) {
  struct Ahead {
    decltype(load(0)) f[A];
  } r;
#pragma unroll
  for (int i = 0; i < A; ++i) r.f[i] = load(i);
  __builtin_amdgcn_sched_barrier(0);
  return r;
}
template <int N, int A, class Ahead, class Load, class Use>
__device__ __forceinline__ void products(Ahead& r, Load load, Use use) {
  static_assert(A <= N, "");
  // (before the other wave's exps: 2 to 4 % of the whole)
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    use(i, r.f[i % A]);
    if (i + A < N) r.f[i % A] = load(i + A);
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_setprio(0);
}
struct Two {
  u32x4 a, b;
};
struct Three {
  u32x4 a, b, c;
};

// Of 32 results in rows, those that make one operand along the rows: chunk c's.  The order of
// k that this gives is that of Tile::column.
template <int DT>
__device__ __forceinline__ u32x4 pack_chunk(const f32x16& v, int c) {
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (DT == kBF16) w[j] = pack_bf16(v[8 * c + 2 * j], v[8 * c + 2 * j + 1]);
    else w[j] = __float_as_uint(v[4 * c + j]);
  }
  return w;
}
template <int DT>
__host__ __device__ constexpr int chunks() { return DT == kF32 ? 4 : 2; }   // of 32 rows

// 16 bytes a lane to LDS, in lane order.  (A function of its own: called within a member of
// a nested class template, this builtin makes the compiler drop host stubs of the kernels.)
__device__ __forceinline__ void load_pieces(__amdgpu_buffer_rsrc_t q, char* lds, uint32_t at) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(q, (LOWBIT_LDS void*)lds, 16, at, 0, 0, 0);
}
// 64 consecutive words to LDS.
__device__ __forceinline__ void load_floats(__amdgpu_buffer_rsrc_t q, char* lds, int lane) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(q, (LOWBIT_LDS void*)lds, 4, lane * 4, 0, 0, 0);
}

// A tile of ROWS rows of D elements in LDS (rows of 96 take the room of 128).  The 16-byte
// pieces of a row are permuted by its number so that neither the operands that run along a row (32
// rows, one piece each) nor those that run down the columns (four rows, 32 bytes
// each) meet a bank of LDS more often than they must.
template <int DT, int D, int ROWS>
struct Tile {
  static constexpr int ES = elem_size<DT>(), PITCH = (D <= 64 ? 64 : 128) * ES, NP = PITCH / 16;
  static constexpr int BYTES = ROWS * PITCH;
  static constexpr int STEPS = D * ES / 32;        // operands along a row
  static constexpr int BLOCKS = D / 32;            // blocks of 32 columns
  static constexpr int LOADS = BYTES / 1024 / kWaves, PER_LOAD = 1024 / PITCH;

  static __device__ __forceinline__ constexpr int mix(int r) {
    if constexpr (DT == kF32) return (r & 3) | (r >> 2 & 1) << 3 | (r >> 3 & 1) << 2;
    else if constexpr (NP == 16) return (r & 3) << 2 | (r >> 2 & 3);
    else return (r >> 1 & 1) << 2 | (r >> 2 & 3);
  }

  // The way in: 16 bytes a lane straight from memory, the waves taking turns.
  struct Loader {
    uint32_t voff[LOADS];
    __device__ __forceinline__ void init(int64_t row_bytes, int width_bytes, int wave, int lane) {
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int r = (j * kWaves + wave) * PER_LOAD + lane / NP;
        const int piece = lane % NP ^ mix(r);
        voff[j] = piece * 16 < width_bytes ? (uint32_t)(r * (int)row_bytes) + piece * 16 : kNowhere;
      }
    }
    // rows: how many there are from `p` on; those behind read as 0
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const char* p, int row_bytes,
                                                                     int width_bytes, int rows) {
      const int n = rows < ROWS ? rows : ROWS;
      return open(p, n > 0 ? (n - 1) * row_bytes + width_bytes : 0);
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t q, char* lds, int wave, int j) const {
      load_pieces(q, lds + (j * kWaves + wave) * 1024, voff[j]);
    }
  };

  // Operands along a row: row b * 32 + lane mod 32, step kk.
  struct Along {
    uint32_t at;
    // makes the compiler take the addresses anew instead of keeping all of them in registers
    __device__ __forceinline__ void refresh() { asm volatile("" : "+v"(at)); }
    __device__ __forceinline__ void init(int lane) {
      const int r = lane % 32;
      at = r * PITCH + ((lane / 32) ^ mix(r)) * 16;
    }
    __device__ __forceinline__ u32x4 load(const char* lds, int b, int kk) const {
      return *reinterpret_cast<const u32x4*>(lds + (at ^ (kk * 32)) + b * 32 * PITCH);
    }
    __device__ __forceinline__ void store(char* lds, int kk, u32x4 v) const {
      *reinterpret_cast<u32x4*>(lds + (at ^ (kk * 32))) = v;
    }
  };

  // Operands down a column: column i * 32 + lane mod 32, rows of chunk c.
  struct Down {
    uint32_t at;
    __device__ __forceinline__ void refresh() { asm volatile("" : "+v"(at)); }
    __device__ __forceinline__ void init(int lane) {
      const int h = lane / 32;
      if constexpr (DT == kF32) {
        at = 4 * h * PITCH + ((lane % 32 / 4) ^ mix(4 * h)) * 16 + lane % 4 * 4;
      } else {
        const int r = 4 * h + lane % 16 / 4;
        at = r * PITCH + ((lane / 16 % 2 * 2 + lane % 4 / 2) ^ mix(r)) * 16 + lane % 2 * 8;
      }
    }
    __device__ __forceinline__ u32x4 load(const char* lds, int i, int c) const {
      if constexpr (DT == kF32) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const char* p = lds + (at ^ ((i * 8 ^ mix(8 * c + j)) * 16)) + (8 * c + j) * PITCH;
          v[j] = *reinterpret_cast<const uint32_t*>(p);
        }
        return v;
      } else {
        // 16 lanes read 16 columns of four rows and get a column each
        const uint32_t a = at ^ (i * 64);
        typedef LOWBIT_LDS s16x4* lp;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lp)(LOWBIT_LDS char*)(lds + a + 16 * c * PITCH));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lp)(LOWBIT_LDS char*)(lds + (a ^ 32) + (16 * c + 8) * PITCH));
        return __builtin_bit_cast(u32x4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  };
};

// Which scores a kernel is built for: plain ones, ones with a distance bias, capped ones, both.
enum ScoreMode : int { kPlainScore = 0, kBiasScore = 1, kCapScore = 2, kCapBiasScore = 3 };
inline int score_mode(const AttnArgs& a) {
  return a.softcap > 0.0f ? a.slopes ? kCapBiasScore : kCapScore
                          : a.slopes ? kBiasScore : kPlainScore;
}
constexpr bool has_cap(int mode) { return mode >= kCapScore; }
constexpr bool has_bias(int mode) { return mode % 2 == 1; }

// What a score is from the products' sum.  Without a bias it grows with the sum, so that a
// row's largest score is that of its largest sum, and the others are taken only within their
// exp, whose argument then is one fused product and sum.  A negative scale is turned
// into the sign of the operand that is held in registers.
template <int DT, int MODE>
struct Score {
  float factor, cap, uncap, slope, straight;
  __device__ __forceinline__ explicit Score(const AttnArgs& g) {
    const float unit = unit_of<DT>(), scale = fabsf(g.scale);
    // (a subnormal cap as 2^-126, whose reciprocal binary32 holds)
    const float softcap = fmaxf(g.softcap, 0x1p-126f);
    cap = softcap * unit;
    uncap = 1.0f / cap;
    // (a scale of 0 as 2^-100: -infinity times it has to stay what it is)
    factor = has_cap(MODE) ? scale / softcap : fmaxf(scale * unit, 0x1p-100f);
    factor = fminf(factor, 0x1.fffffep127f);       // (infinity times a sum of 0 would be NaN)
    straight = fminf(scale * unit, 0x1.fffffep127f);
    slope = 0.0f;
  }
  __device__ __forceinline__ void head(const AttnArgs& g, int h) {
    if (has_bias(MODE)) slope = g.slopes[h] * unit_of<DT>();
  }
  // Capped scores of N sums, in their place.  Where a sum is small beside the cap, tanh(x) / x by a
  // series times the score without a cap, which keeps its relative accuracy under any cap; elsewhere,
  // of bfloat16, by an exp and a reciprocal, off by less than 2^-20, relative.  A wave whose sums are
  // all below kFlat skips these two, which run at a quarter of the rate (nine ragged documents of 8 Ki
  // tokens, 16 heads of 64, window 1024: 74 us, gradient 202; 100 and 243 where no wave can).  Both ways
  // give a score the same bits.
  static constexpr float kFlat = 0.5f;
  template <int N>
  __device__ __forceinline__ void cap_all(f32x16 (&x)[N]) const {
    if constexpr (DT == kF32) {
#pragma unroll
      for (int b = 0; b < N; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[b][r] = capped(x[b][r]);
    } else {
      float largest = 0.0f;
#pragma unroll
      for (int b = 0; b < N; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) largest = fmaxf(largest, fabsf(x[b][r]));
      const bool flat = !__any(largest * factor >= kFlat);
      // (the factors are taken anew in each branch, or the compiler would take what both have in common
      // for all sums before it)
      float f = factor, s = straight;
      if (flat) {
        asm volatile("" : "+v"(f), "+v"(s));
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[b][r] = series(x[b][r] * f) * (x[b][r] * s);
      } else {
        asm volatile("" : "+v"(f), "+v"(s));
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float v = x[b][r] * f;
            const float small = series(v) * (x[b][r] * s);
            // tanh = 1 - 2 r, r = 1 / (exp(2 x) + 1)
            const float e = __builtin_amdgcn_exp2f(v * (2.0f * kLog2e));
            const float large = __builtin_fmaf(-2.0f * cap, __builtin_amdgcn_rcpf(e + 1.0f), cap);
            x[b][r] = fabsf(v) < kFlat ? small : large;
            if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // (or registers run out)
          }
      }
    }
  }
  // tanh(x) / x, off by up to 2^-26 below kFlat
  static __device__ __forceinline__ float series(float x) {
    const float z = x * x;
    float s = __builtin_fmaf(z, 1.72414891e-2f, -5.30454926e-2f);
    s = __builtin_fmaf(z, s, 1.33258790e-1f);
    s = __builtin_fmaf(z, s, -3.33331436e-1f);
    return __builtin_fmaf(z, s, 1.0f);
  }
  __device__ __forceinline__ float capped(float x) const {   // binary32
    const float plain = x * straight;
    x *= factor;
    const float z = x * x;
    float s = __builtin_fmaf(z, 3.59212803e-3f, -8.86323552e-3f);
    s = __builtin_fmaf(z, s, 2.18694885e-2f);
    s = __builtin_fmaf(z, s, -5.39682540e-2f);
    s = __builtin_fmaf(z, s, 1.33333333e-1f);
    s = __builtin_fmaf(z, s, -3.33333333e-1f);
    s = __builtin_fmaf(z, s, 1.0f);
    // 1 - 2 e / (1 + e) of e = exp(-2 |x|), which falls to 0 for the largest ones
    const float e = exp_unit<kF32>(-2.0f * fabsf(x));
    const float l = copysignf(__builtin_fmaf(-2.0f * e, __builtin_amdgcn_rcpf(1.0f + e), 1.0f), x);
    return fabsf(x) < 0.4f ? plain * s : cap * l;
  }
  // 1 - tanh^2 of a capped score, which the gradient takes
  __device__ __forceinline__ float bend(float y) const {
    if constexpr (!has_cap(MODE)) return 1.0f;
    const float t = y * uncap;
    return __builtin_fmaf(-t, t, 1.0f);
  }

  // x: a sum of products, or its capped score; distance: |distance - c| to the key
  __device__ __forceinline__ float at(float x, float distance, int c) const {
    if constexpr (!has_bias(MODE)) return x;
    return __builtin_fmaf(-slope, fabsf(distance - (float)c), has_cap(MODE) ? x : x * factor);
  }
  // the largest score, in units, from the largest of what `at` gives
  __device__ __forceinline__ float scaled(float y) const {
    return MODE == kPlainScore ? y * factor : y;
  }
  // exp(score - base); of a masked -infinity 0
  __device__ __forceinline__ float weight(float y, float base) const {
    return exp_unit<DT>(MODE == kPlainScore ? __builtin_fmaf(y, factor, -base) : y - base);
  }
};

// The gradient's sums of products may begin with -lse / factor and -D, so that both are
// subtracted for nothing.  Not of capped scores, whose lse is no sum's; nor of binary32,
// whose scores would lose digits beside a large lse.
template <int DT, int MODE>
constexpr bool lse_in_sum() { return DT == kBF16 && !has_cap(MODE); }

// The signs of an operand's elements turned.
template <int DT>
__device__ __forceinline__ u32x4 negated(u32x4 v) {
  return v ^ (DT == kF32 ? 0x80000000u : 0x80008000u);
}

// One sequence: its queries and keys in the buffers.
struct Sequence {
  int q0, lq, k0, lk, prefix;
};

__device__ __forceinline__ int offset_at(const int32_t* begin, int s, int sequences, int rows) {
  if (!begin) return (int)((int64_t)rows / sequences * s);
  const int v = begin[s];
  return v < 0 ? 0 : v > rows ? rows : v;
}

__device__ __forceinline__ Sequence sequence_at(const AttnArgs& g, int s) {
  const int32_t* kb = g.k_begin;
  Sequence q;
  q.q0 = offset_at(g.q_begin, s, g.sequences, g.q_rows);
  q.lq = offset_at(g.q_begin, s + 1, g.sequences, g.q_rows) - q.q0;
  q.k0 = offset_at(kb, s, g.sequences, g.k_rows);
  q.lk = offset_at(kb, s + 1, g.sequences, g.k_rows) - q.k0;
  q.lq = q.lq < 0 ? 0 : q.lq;
  q.lk = q.lk < 0 ? 0 : q.lk;
  q.prefix = g.prefix ? g.prefix[s] : 0;
  q.prefix = q.prefix < 0 ? 0 : q.prefix > q.lk ? q.lk : q.prefix;
  return q;
}

// Sequence s has the tiles from begin[s] / T + s on, whose count, ceil(length / T), never
// reaches the next sequence's first: a tile's sequence is found without a table of
// tiles, 64 sequences at a time.
__device__ __forceinline__ int find_sequence(const int32_t* begin, int sequences, int rows, int T,
                                             int tile) {
  int first = 0, count = sequences;                // the answer is one of these
  while (count > 1) {
    const int step = (count + 63) / 64;
    const int off = lane_id() * step;
    const bool at_or_before =
        off < count && offset_at(begin, first + off, sequences, rows) / T + first + off <= tile;
    const int n = __popcll(__ballot(at_or_before));
    const int skip = (n > 0 ? n - 1 : 0) * step;
    first += skip;
    count = count - skip < step ? count - skip : step;
  }
  return __builtin_amdgcn_readfirstlane(first);
}
__device__ __forceinline__ int first_tile(const int32_t* begin, int s, int sequences, int rows, int T) {
  return offset_at(begin, s, sequences, rows) / T + s;
}

// What query `pos` sees: keys below `prefix` and those from low to high.
struct Sight {
  int low, high, prefix;
};
__device__ __forceinline__ Sight sight(const AttnArgs& g, const Sequence& q, int pos) {
  Sight v;
  v.low = g.window ? pos - g.window + 1 : 0;
  v.high = q.lk - 1;
  if (g.causal) v.high = min(v.high, pos);
  else if (g.window) v.high = min(v.high, pos + g.window - 1);
  v.prefix = q.prefix;
  return v;
}

// Which work item a workgroup takes.  Workgroup b runs on XCD b mod 8; the
// tiles of a key-value head go to as few XCDs as keep all eight busy, whose L2 then
// holds its keys and values, and the longest tiles come first.
struct Items {
  int per_head, parts, spread, group;
  int64_t total;
  __host__ __device__ Items(int tiles, int heads, int group_) {
    group = group_;
    spread = heads % 8 == 0 ? 8 : heads % 4 == 0 ? 4 : heads % 2 == 0 ? 2 : 1;
    parts = 8 / spread;                            // XCDs of a head
    per_head = (tiles + parts - 1) / parts;
    total = (int64_t)per_head * (heads / spread) * group * 8;
  }
  // tile: may be beyond the last
  __device__ __forceinline__ void take(int64_t item, int heads, int& tile, int& head, int& in) const {
    const int xcd = (int)(item % 8);
    const int64_t u = item / 8;
    const int each = heads / spread;
    in = (int)(u % group);
    const int64_t v = u / group;
    head = xcd / parts + (int)(v % each) * spread;
    tile = (int)(v / each) * parts + xcd % parts;
  }
};

constexpr int64_t kMaxBlocks = 1 << 20;            // (a multiple of 8)
inline int64_t capped(int64_t blocks) { return blocks < kMaxBlocks ? blocks : kMaxBlocks; }

// A workgroup's tile of queries of one head, and which part of their keys it takes.
struct Queries {
  Sequence q;
  int i0, last, head, kv, part;                    // last: the last query of the tile
  bool any;
  int64_t unit;                                    // tile and head
  __device__ __forceinline__ Queries(const AttnArgs& g, const Items& items, int64_t item, int tiles,
                                     int parts) {
    int t, in;
    items.take(item, g.kv_heads, t, kv, in);
    part = in % parts;
    head = kv * g.group + in / parts;
    any = t < tiles;
    t = tiles - 1 - t;                             // causal: the last see most
    unit = (int64_t)head * tiles + t;
    if (!any) return;
    const int s = find_sequence(g.q_begin, g.sequences, g.q_rows, kRowsPerTile, t);
    q = sequence_at(g, s);
    i0 = (t - first_tile(g.q_begin, s, g.sequences, g.q_rows, kRowsPerTile)) * kRowsPerTile;
    last = min(i0 + kRowsPerTile, q.lq) - 1;
    any = i0 >= 0 && i0 < q.lq;                    // (below 0: rows before the first sequence)
  }
};

// The tiles of KT keys that a tile of queries sees: those of the prefix, then those around
// the positions; in order, and those of one of `parts` even parts.
template <int KT>
struct KeyTiles {
  int before, from, first, count;
  __device__ __forceinline__ KeyTiles(const AttnArgs& g, const Queries& w, int parts) {
    const int shift = w.q.lk - w.q.lq;
    const Sight lo = sight(g, w.q, w.i0 + shift), hi = sight(g, w.q, w.last + shift);
    before = (w.q.prefix + KT - 1) / KT;
    from = max(before, lo.low > 0 ? lo.low / KT : 0);
    const int to = hi.high < 0 ? 0 : hi.high / KT + 1;
    const int64_t all = before + max(0, to - from);
    first = (int)(all * w.part / parts);
    count = (int)(all * (w.part + 1) / parts) - first;
  }
  // the u-th of this part
  __device__ __forceinline__ int tile(int u) const {
    u += first;
    return u < before ? u : from + (u - before);
  }
};

// Room for a part's sums, as the lanes hold them: `vectors` of four for each.
__device__ __forceinline__ f32x4* part_at(float* parts, int64_t unit, int vectors) {
  return reinterpret_cast<f32x4*>(parts) + unit * (vectors * kAttnThreads) + threadIdx.x;
}
template <int BLOCKS>
__device__ __forceinline__ void store_part(f32x4* to, const f32x16 (&acc)[BLOCKS]) {
#pragma unroll
  for (int n = 0; n < BLOCKS; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      to[(n * 4 + c) * kAttnThreads] =
          (f32x4){acc[n][4 * c], acc[n][4 * c + 1], acc[n][4 * c + 2], acc[n][4 * c + 3]};
}
template <int BLOCKS>
__device__ __forceinline__ void add_part(f32x16 (&sum)[BLOCKS], const f32x4* from, float weight) {
#pragma unroll
  for (int n = 0; n < BLOCKS; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f32x4 v = from[(n * 4 + c) * kAttnThreads];
#pragma unroll
      for (int r = 0; r < 4; ++r) sum[n][4 * c + r] = __builtin_fmaf(v[r], weight, sum[n][4 * c + r]);
    }
}
template <int BLOCKS>
__device__ __forceinline__ void clear(f32x16 (&acc)[BLOCKS]) {
#pragma unroll
  for (int n = 0; n < BLOCKS; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[n][r] = 0.0f;
}

// Rows of a result that lies as columns d by rows of lanes; its blocks of 32 columns are the
// matrix's from `first` on.
template <int DT, int BLOCKS>
__device__ __forceinline__ void store_columns(char* to, const f32x16 (&acc)[BLOCKS], float scale,
                                              int half, int head_dim, int first = 0) {
#pragma unroll
  for (int n = 0; n < BLOCKS; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = (first + n) * 32 + c * 8 + half * 4;
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = acc[n][4 * c + r] * scale;
      if (at < head_dim) {
        if constexpr (DT == kF32) *reinterpret_cast<f32x4*>(to + at * 4) = v;
        else *reinterpret_cast<u32x2*>(to + at * 2) =
                 (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      }
    }
}

// The operands along a row of one matrix, straight from memory.
template <int STEPS>
__device__ __forceinline__ void load_rows(u32x4 (&f)[STEPS], const void* base, int64_t at, int half,
                                          int width, bool any) {
  const char* p = static_cast<const char*>(base) + at;
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) {
    const int c = kk * 32 + half * 16;
    f[kk] = (u32x4){0, 0, 0, 0};
    if (any && c < width) f[kk] = *reinterpret_cast<const u32x4*>(p + c);
  }
}
template <int DT, int STEPS>
__device__ __forceinline__ void negate(u32x4 (&f)[STEPS]) {
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) f[kk] = negated<DT>(f[kk]);
}

}  // namespace

}  // namespace lowbit
