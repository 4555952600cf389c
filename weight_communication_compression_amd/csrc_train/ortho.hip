// ortho.hip -- orthogonalize: Newton-Schulz products.
#include "block.hpp"
#include "ortho_choice.hpp"
#include "tile_feed.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

// The products' operands are binary16 times a power of two: entries of X begin at about
// 1 / sqrt(m n) and those of A beside its diagonal at 1 / (m sqrt(n)), near the smallest
// that binary16 holds in full, and none of X, A or B (b A + c A A) grows beyond a few units.
constexpr float kX = 64.0f, kA = 1024.0f, kB = 64.0f;

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 pack_f16(f32x4 v) {
  return __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4));
}
__device__ __forceinline__ f32x4 unpack_f16(u32x2 v) {
  return __builtin_convertvector(__builtin_bit_cast(f16x4, v), f32x4);
}

// ------------------------------------------------------------ norm, ends --
// Sums of squares in binary64, which no binary32 input leaves: nparts of each matrix.  Bound by
// memory: 4096 x 4096 binary32 15 us, 4.5 TB/s.
template <int DT>
__global__ void __launch_bounds__(256) ortho_norm_kernel(OrthoArgs g) {
  __shared__ double sums[4];
  const int64_t n = (int64_t)g.m * g.n;
  const int64_t chunks = (n + 7) / 8;
  for (int64_t u = blockIdx.x; u < g.batch * g.nparts; u += gridDim.x) {
    const int64_t matrix = u / g.nparts, part = u % g.nparts;
    const char* p = static_cast<const char*>(g.g) + matrix * n * elem_size<DT>();
    double sum = 0.0;
    for (int64_t k = part * 256 + threadIdx.x; k < chunks; k += (int64_t)g.nparts * 256) {
      const int64_t left = n - k * 8;
      const Raw8<DT> v = load8<DT>(p + k * 8 * elem_size<DT>(), 0, left < 8 ? (int)left : 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double x = v.get(j);
        sum += x * x;
      }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane_id() == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) g.parts[u] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    __syncthreads();
  }
}

// X = g / (norm + eps) in binary32 and binary16, a tile of 64 x 64 a workgroup,
// turned through LDS where the matrix is.  Bound by memory: 4096 x 4096 binary32 37 us, 4.5 TB/s.
template <int DT>
__global__ void __launch_bounds__(256) ortho_start_kernel(OrthoArgs g) {
  __shared__ float tile[64][65];
  const int across = g.ldn / 64, down = (g.m + 63) / 64;
  const int r = threadIdx.x / 64, c = threadIdx.x % 64;
  for (int64_t u = blockIdx.x; u < g.batch * across * down; u += gridDim.x) {
    const int64_t matrix = u / ((int64_t)across * down);
    const int in = (int)(u - matrix * across * down);
    const int i0 = in / across * 64, j0 = in % across * 64;
    double total = 0.0;
    for (int k = lane_id(); k < g.nparts; k += 64) total += g.parts[matrix * g.nparts + k];
#pragma unroll
    for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
    const double factor = 1.0 / (sqrt(total) + (double)g.eps);
    const char* p = static_cast<const char*>(g.g) + matrix * g.m * g.n * elem_size<DT>();
    auto at = [&](int64_t k) {
      float v;
      if constexpr (DT == kF32) v = reinterpret_cast<const float*>(p)[k];
      else v = bf16_lo(reinterpret_cast<const uint16_t*>(p)[k]);
      return (float)(v * factor);
    };
    if (g.turned) {
      for (int k = r; k < 64; k += 4) {
        const int j = j0 + k, i = i0 + c;
        tile[c][k] = j < g.n && i < g.m ? at((int64_t)j * g.m + i) : 0.0f;
      }
      __syncthreads();
    }
    for (int k = r; k < 64; k += 4) {
      const int i = i0 + k, j = j0 + c;
      if (i >= g.m) break;
      const float v = g.turned ? tile[k][c] : j < g.n ? at((int64_t)i * g.n + j) : 0.0f;
      const int64_t to = ((int64_t)matrix * g.m + i) * g.ldn + j;
      g.x[to] = v;
      static_cast<_Float16*>(g.xh)[to] = (_Float16)(v * kX);
    }
    if (g.turned) __syncthreads();
  }
}

// out = scale X, turned back.
__global__ void __launch_bounds__(256) ortho_end_kernel(OrthoArgs g) {
  __shared__ float tile[64][65];
  const int across = g.ldn / 64, down = (g.m + 63) / 64;
  const int r = threadIdx.x / 64, c = threadIdx.x % 64;
  for (int64_t u = blockIdx.x; u < g.batch * across * down; u += gridDim.x) {
    const int64_t matrix = u / ((int64_t)across * down);
    const int in = (int)(u - matrix * across * down);
    const int i0 = in / across * 64, j0 = in % across * 64;
    uint16_t* const out = static_cast<uint16_t*>(g.out) + matrix * g.m * g.n;
    const float* const x = g.x + matrix * g.m * g.ldn;
    if (g.turned) {
      for (int k = r; k < 64; k += 4)
        tile[c][k] = i0 + k < g.m ? x[(int64_t)(i0 + k) * g.ldn + j0 + c] : 0.0f;
      __syncthreads();
      for (int k = r; k < 64; k += 4) {
        const int j = j0 + k, i = i0 + c;
        if (j < g.n && i < g.m)
          out[(int64_t)j * g.m + i] = (uint16_t)pack_bf16(tile[k][c] * g.scale, 0.0f);
      }
      __syncthreads();
    } else {
      for (int k = r; k < 64; k += 4) {
        const int i = i0 + k, j = j0 + c;
        if (i < g.m && j < g.n)
          out[(int64_t)i * g.n + j] =
              (uint16_t)pack_bf16(x[(int64_t)i * g.ldn + j] * g.scale, 0.0f);
      }
    }
  }
}

// -------------------------------------------------------------- products --
enum OrthoKind : int {
  kGram = 0,                 // A = X X^T
  kPoly = 1,                 // B = b A + c A A
  kUpdate = 2,               // X = a X + B X
  kLast = 3,                 // the same, and out = scale X, turned back, in its place
};

// Tiles of A and B lie on and below the diagonal; the others are their mirror images.
template <int KIND>
constexpr bool kMirrored = KIND == kGram || KIND == kPoly;

// Four columns col .. col + 3 of a row of the result, from the products' sums.
template <int KIND>
__device__ __forceinline__ f32x4 value(const OrthoArgs& g, int64_t matrix, int row, int col, f32x4 v) {
  if constexpr (KIND == kGram) {
    return v * (kA / (kX * kX));
  } else if constexpr (KIND == kPoly) {
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    if (row >= g.m || col >= g.ldm) return y;
    const f32x4 a = unpack_f16(*reinterpret_cast<const u32x2*>(
        static_cast<_Float16*>(g.ah) + (matrix * g.m + row) * g.ldm + col));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      y[r] = __builtin_fmaf(g.b * (kB / kA), a[r], v[r] * (g.c * (kB / (kA * kA))));
    return y;
  } else {
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    if (row >= g.m || col >= g.ldn) return y;
    const f32x4 x = *reinterpret_cast<const f32x4*>(g.x + (matrix * g.m + row) * g.ldn + col);
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(g.a, x[r], v[r] * (1.0f / (kB * kX)));
    return y;
  }
}

// n (at most 4) consecutive values as bfloat16.
__device__ __forceinline__ void put_bf16(uint16_t* p, f32x4 v, int n) {
  const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
  if (n >= 4) {
    *reinterpret_cast<u32x2_2*>(p) = (u32x2_2){lo, hi};
  } else {
    if (n > 0) p[0] = (uint16_t)lo;
    if (n > 1) p[1] = (uint16_t)(lo >> 16);
    if (n > 2) p[2] = (uint16_t)hi;
  }
}

template <int KIND>
__device__ __forceinline__ void put(const OrthoArgs& g, int64_t matrix, int row, int col, f32x4 y) {
  if (row >= g.m) return;
  if constexpr (KIND == kLast) {
    if (col < g.n)
      put_bf16(static_cast<uint16_t*>(g.out) + (matrix * g.m + row) * g.n + col, y * g.scale, g.n - col);
  } else if constexpr (KIND == kUpdate) {
    if (col >= g.ldn) return;
    const int64_t at = (matrix * g.m + row) * g.ldn + col;
    *reinterpret_cast<f32x4*>(g.x + at) = y;
    *reinterpret_cast<u32x2*>(static_cast<_Float16*>(g.xh_next) + at) = pack_f16(y * kX);
  } else {
    if (col >= g.ldm) return;
    *reinterpret_cast<u32x2*>(static_cast<_Float16*>(KIND == kGram ? g.ah : g.bh) +
                              (matrix * g.m + row) * g.ldm + col) = pack_f16(y);
  }
}

// 32 x 32 sums, as the lanes hold them, become results: through LDS (4 KB of the wave's own), so
// that loads and stores take whole lines of a row, and once more, turned, for a mirror image or a
// result that is turned back.
template <int KIND>
__device__ __forceinline__ void finish_block(const OrthoArgs& g, int64_t matrix, const f32x16& acc,
                                             int row0, int col0, bool mirror, int lane, char* lds) {
  const int r = lane % 32, h = lane / 32, line = lane / 8, piece = lane % 8;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<f32x4*>(lds + r * 128 + ((2 * q + h) ^ (r & 7)) * 16) = quad(acc, q);
  f32x4 y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = k * 8 + line;
    y[k] = *reinterpret_cast<const f32x4*>(lds + row * 128 + (piece ^ (row & 7)) * 16);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    y[k] = value<KIND>(g, matrix, row0 + k * 8 + line, col0 + piece * 4, y[k]);
  if (KIND != kLast || !g.turned) {
#pragma unroll
    for (int k = 0; k < 4; ++k) put<KIND>(g, matrix, row0 + k * 8 + line, col0 + piece * 4, y[k]);
  }
  if constexpr (kMirrored<KIND> || KIND == kLast) {
    if (!mirror) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = piece * 4 + e, row = k * 8 + line;
        *reinterpret_cast<float*>(lds + c * 128 + ((row / 4) ^ (c >> 2 & 7)) * 16 + row % 4 * 4) = y[k][e];
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = k * 8 + line;
      const f32x4 v = *reinterpret_cast<const f32x4*>(lds + c * 128 + (piece ^ (c >> 2 & 7)) * 16);
      if constexpr (KIND == kLast) {
        const int row = row0 + piece * 4;          // of X; a column of the result
        if (col0 + c < g.n && row < g.m)
          put_bf16(static_cast<uint16_t*>(g.out) + (matrix * g.n + col0 + c) * g.m + row, v * g.scale,
                   g.m - row);
      } else {
        put<KIND>(g, matrix, col0 + c, row0 + piece * 4, v);
      }
    }
  }
}

// Where the sums of a part of a tile are, as the lanes hold them.
template <class F>
__device__ __forceinline__ f32x4* part_of(float* partial, int64_t part) {
  return reinterpret_cast<f32x4*>(partial) + part * (F::TM * F::TN / 4) + threadIdx.x;
}

// A form of the tile kernel: TM x TN by W = WM x WN waves, STAGES steps of k in LDS, PER_CU
// workgroups on a CU.
template <int TM_, int TN_, int WM_, int WN_, int STAGES_, int PER_CU_>
struct Shape {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, STAGES = STAGES_, PER_CU = PER_CU_;
  static constexpr int W = WM * WN, I = TM / WM / 32, J = TN / WN / 32, THREADS = 64 * W;
  static constexpr int A = TM * kRowBytes, STAGE = (TM + TN) * kRowBytes;
};

// All loads but the last N are done, and all that the wave has read in LDS.
template <int N>
__device__ __forceinline__ void wait_loads_but() {
  if constexpr (N == 0) wait_all();
  else {
    static_assert(N < 64, "");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4 | 0 << 8);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
}

// W waves, each I x J products of 32 x 32; lanes hold of one what finish_block says.  STAGES
// buffers in LDS: while the matrix units work on one, the others are filled, so that a step's
// loads have STAGES - 1 steps' time.
//
// Bound by the matrix units at the clock that power leaves, and by the tail of the update, which
// reads and writes X: 4096 x 4096 A 78 us (253 tiles of 192: 76 GFLOP, 0.98 PFLOP/s; whole
// in 256 tiles of 256 105), b A + c A A 86, the update 135 to 143 (256 tiles of 256; about 30
// are its tail's 160 MB), the last product 133.  Smaller ones are bound by the loads' latency where a
// CU has one tile: a step of 64 of k takes 0.27 us in tiles of 64 (0.45 with two stages instead
// of four), 0.46 to 0.67 in tiles of 128, while its products take 0.03 to 0.2.
template <class F, int KIND>
__global__ void __launch_bounds__(F::THREADS, F::PER_CU * F::W / 4) ortho_tile_kernel(OrthoArgs g) {
  constexpr int TM = F::TM, TN = F::TN, W = F::W, I = F::I, J = F::J, S = F::STAGES;
  constexpr bool BO = !kMirrored<KIND>;
  constexpr int K = kRowBytes / 2;
  static_assert(F::STAGE >= W * 4096, "");           // (finish_block goes through the first stage)
  __shared__ __attribute__((aligned(1024))) char l0[F::STAGE];
  __shared__ __attribute__((aligned(1024))) char l1[F::STAGE];
  __shared__ __attribute__((aligned(1024))) char l2[S > 2 ? F::STAGE : 16];
  __shared__ __attribute__((aligned(1024))) char l3[S > 3 ? F::STAGE : 16];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / F::WN, wn = wave % F::WN;
  char* const side = l0 + wave * 4096;
  const int k = KIND == kGram ? g.n : g.m, n = kMirrored<KIND> ? g.m : g.n;
  const int lda = KIND == kGram ? g.ldn : g.ldm, ldb = KIND == kPoly ? g.ldm : g.ldn;
  const int across = (n + TN - 1) / TN, down = (g.m + TM - 1) / TM;
  const int64_t tiles = kMirrored<KIND> ? (int64_t)down * (down + 1) / 2 : (int64_t)across * down;
  const int all_steps = (k + K - 1) / K;

  constexpr int NA = Feed<kF16, TM, W, false>::LOADS, NB = Feed<kF16, TN, W, BO>::LOADS, N = NA + NB;
  constexpr int RD = I + J * (BO ? 2 : 1);
  Feed<kF16, TM, W, false> fa;
  Feed<kF16, TN, W, BO> fb;
  Frag<kF16, TM, false> ra;
  Frag<kF16, TN, BO> rb;
  fa.init(lda, wave, lane);
  fb.init(ldb, wave, lane);
  ra.init(wm * (TM / F::WM), lane);
  rb.init(wn * (TN / F::WN), lane);
  u32x4 fra[2][I], frb[2][J];
  f32x16 acc[I][J];
  int s0, s1;                                      // steps of this unit

  auto kleft = [&](int s) { return min(k - s * K, K); };
  auto issue = [&](char* l, int s) {
    const auto qa = fa.open(s < s1), qb = fb.open(s < s1);
#pragma unroll
    for (int j = 0; j < NA; ++j) fa.load(qa, l, wave, kleft(s), j);
#pragma unroll
    for (int j = 0; j < NB; ++j) fb.load(qb, l + F::A, wave, kleft(s), j);
    fa.next();
    fb.next();
  };
  auto read = [&](int to, const char* l, int kk) {
#pragma unroll
    for (int j = 0; j < J; ++j) frb[to][j] = rb.load(l + F::A, j, kk);
#pragma unroll
    for (int i = 0; i < I; ++i) fra[to][i] = ra.load(l, i, kk);
  };
  auto mul = [&](int f) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = mma<kF16>(frb[f][j], fra[f][i], acc[i][j]);
    spread_reads<RD, I * J>();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step s, in l, whose first quarter is in registers.  While a quarter is multiplied the next
  // is read; before the last, everybody has read all of this step, the next one has arrived (in
  // `next`), and the loads of step s + STAGES begin.
  auto step = [&](char* l, const char* next, int s) {
    const auto qa = fa.open(s + S < s1), qb = fb.open(s + S < s1);
    const int kl = kleft(s + S);
    read(1, l, 1);
    mul(0);
    read(0, l, 2);
    mul(1);
    read(1, l, 3);
    mul(0);
    wait_loads_but<(S - 2) * N>();
    barrier();
    read(0, next, 0);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        acc[i][j] = mma<kF16>(frb[1][j], fra[1][i], acc[i][j]);
        const int p = i * J + j;
#pragma unroll
        for (int u = N * p / (I * J); u < N * (p + 1) / (I * J); ++u) {
          if (u < NA) fa.load(qa, l, wave, kl, u);
          else fb.load(qb, l + F::A, wave, kl, u - NA);
        }
      }
    fa.next();
    fb.next();
    spread_loads<RD, I * J, 1, N>();
    __builtin_amdgcn_sched_barrier(0);
  };

  const int64_t total = tiles * g.batch * g.k_parts;
  for (int64_t unit = blockIdx.x; unit < total; unit += gridDim.x) {
    const int64_t mine = ortho_run(unit, total);
    const int64_t which = mine / g.k_parts;
    const int part = (int)(mine - which * g.k_parts);
    const int64_t matrix = which / tiles;
    const OrthoPlace at = ortho_place(kMirrored<KIND>, (int)(which - matrix * tiles), across, down);
    const int tm = __builtin_amdgcn_readfirstlane(at.tm), tn = __builtin_amdgcn_readfirstlane(at.tn);
    s0 = __builtin_amdgcn_readfirstlane((int)((int64_t)all_steps * part / g.k_parts));
    s1 = __builtin_amdgcn_readfirstlane((int)((int64_t)all_steps * (part + 1) / g.k_parts));
    const int64_t mm = matrix * g.m;
    const _Float16* a = static_cast<const _Float16*>(KIND == kGram ? g.xh : KIND == kPoly ? g.ah : g.bh);
    const _Float16* b = static_cast<const _Float16*>(KIND == kPoly ? g.ah : g.xh);
    fa.seek(a + mm * lda, lda, g.m, (int64_t)tm * TM, (int64_t)s0 * K);
    fb.seek(b + mm * ldb, ldb, g.m, (int64_t)tn * TN, (int64_t)s0 * K);
    issue(l0, s0);
    issue(l1, s0 + 1);
    if constexpr (S > 2) issue(l2, s0 + 2);
    if constexpr (S > 3) issue(l3, s0 + 3);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    wait_loads_but<(S - 1) * N>();
    barrier();
    read(0, l0, 0);
    __builtin_amdgcn_sched_barrier(0);
    int s = s0;
    for (; s + S <= s1; s += S) {
      step(l0, l1, s);
      if constexpr (S == 2) {
        step(l1, l0, s + 1);
      } else if constexpr (S == 3) {
        step(l1, l2, s + 1);
        step(l2, l0, s + 2);
      } else {
        step(l1, l2, s + 1);
        step(l2, l3, s + 2);
        step(l3, l0, s + 3);
      }
    }
    if (s < s1) step(l0, l1, s);
    if constexpr (S > 2) {
      if (s + 1 < s1) step(l1, l2, s + 1);
    }
    if constexpr (S > 3) {
      if (s + 2 < s1) step(l2, l3, s + 2);
    }
    wait_all();
    barrier();                                     // (nobody reads the buffers any more)
    if (g.k_parts > 1) {
      f32x4* const to = part_of<F>(g.partial, which * g.k_parts + part);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) to[((i * J + j) * 4 + q) * F::THREADS] = quad(acc[i][j], q);
    } else {
      const bool mirror = KIND == kLast ? g.turned != 0 : tm != tn;
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
          finish_block<KIND>(g, matrix, acc[i][j], tm * TM + wm * (TM / F::WM) + 32 * i,
                             tn * TN + wn * (TN / F::WN) + 32 * j, mirror, lane, side);
    }
    __syncthreads();                               // (the next tile's loads go where the waves wrote)
  }
}

// Matrices of at most M = 64 or 128 rows: b A + c A A and the product with X in one launch.  A
// workgroup takes 64 columns of X with all rows and makes all of B for itself, 2 M^3
// operations, where a launch of their own takes 5 us.  128 x 512: 7 us (in two launches 10), most of
// it the latency of the loads and of the four ways through LDS.
template <int M, int KIND>
__global__ void __launch_bounds__(256) ortho_short_kernel(OrthoArgs g) {
  constexpr int W = 4, I = M / 64, STEPS = M / 64;       // waves 2 x 2; steps of 64 of k
  __shared__ __attribute__((aligned(1024))) char la[STEPS * M * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb[STEPS * M * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lx[STEPS * 64 * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char side[W * 4096];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / 2, wn = wave % 2, r = lane % 32, h = lane / 32;
  Feed<kF16, M, W, false> fa;
  Feed<kF16, 64, W, true> fx;
  Frag<kF16, M, false> rows, columns;
  Frag<kF16, 64, true> rx;
  fa.init(g.ldm, wave, lane);
  fx.init(g.ldn, wave, lane);
  rows.init(wm * (M / 2), lane);
  columns.init(wn * (M / 2), lane);
  rx.init(wn * 32, lane);
  const int across = (g.n + 63) / 64;
  // where four columns from col on of a row lie, as the operands are read
  auto place_of = [&](char* l, int row, int col) {
    return reinterpret_cast<u32x2*>(l + col / 64 * (M * kRowBytes) + row * kRowBytes +
                                    ((col % 64 / 8) ^ (row >> 1 & 7)) * 16 + col % 8 * 2);
  };
  for (int64_t unit = blockIdx.x; unit < g.batch * across; unit += gridDim.x) {
    const int64_t matrix = unit / across;
    const int col0 = (int)(unit - matrix * across) * 64;
    const int64_t mm = matrix * g.m;
    fa.seek(static_cast<const _Float16*>(g.ah) + mm * g.ldm, g.ldm, g.m, 0, 0);
    fx.seek(static_cast<const _Float16*>(g.xh) + mm * g.ldn, g.ldn, g.m, col0, 0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const auto qa = fa.open(true), qx = fx.open(true);
#pragma unroll
      for (int j = 0; j < Feed<kF16, M, W, false>::LOADS; ++j)
        fa.load(qa, la + s * M * kRowBytes, wave, g.m - s * 64, j);
#pragma unroll
      for (int j = 0; j < Feed<kF16, 64, W, true>::LOADS; ++j)
        fx.load(qx, lx + s * 64 * kRowBytes, wave, 64, j);
      fa.next();
      fx.next();
    }
    wait_all();
    barrier();
    f32x16 acc[I][I];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < I; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < 4 * STEPS; ++k) {
      const char* const l = la + k / 4 * (M * kRowBytes);
      u32x4 fm[I], fn[I];
#pragma unroll
      for (int i = 0; i < I; ++i) {
        fm[i] = rows.load(l, i, k % 4);
        fn[i] = columns.load(l, i, k % 4);
      }
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < I; ++j) acc[i][j] = mma<kF16>(fn[j], fm[i], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < I; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = wm * (M / 2) + 32 * i + r, col = wn * (M / 2) + 32 * j + 8 * q + 4 * h;
          const f32x4 a = unpack_f16(*place_of(la, row, col)), v = quad(acc[i][j], q);
          f32x4 y;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = __builtin_fmaf(g.b * (kB / kA), a[e], v[e] * (g.c * (kB / (kA * kA))));
          *place_of(lb, row, col) = pack_f16(y);
        }
    __syncthreads();
    f32x16 sum[I];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) sum[i][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < 4 * STEPS; ++k) {
      const u32x4 x = rx.load(lx + k / 4 * (64 * kRowBytes), 0, k % 4);
#pragma unroll
      for (int i = 0; i < I; ++i)
        sum[i] = mma<kF16>(x, rows.load(lb + k / 4 * (M * kRowBytes), i, k % 4), sum[i]);
    }
#pragma unroll
    for (int i = 0; i < I; ++i)
      finish_block<KIND>(g, matrix, sum[i], wm * (M / 2) + 32 * i, col0 + wn * 32,
                         KIND == kLast && g.turned, lane, side + wave * 4096);
    __syncthreads();                               // (the next unit's loads go where the waves read)
  }
}

// The parts' sums of a tile that is cut along k, added in order.
template <class F, int KIND>
__global__ void __launch_bounds__(F::THREADS) ortho_add_kernel(OrthoArgs g) {
  constexpr int I = F::I, J = F::J;
  __shared__ __attribute__((aligned(1024))) char side[F::W * 4096];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = kMirrored<KIND> ? g.m : g.n;
  const int across = (n + F::TN - 1) / F::TN, down = (g.m + F::TM - 1) / F::TM;
  const int64_t tiles = kMirrored<KIND> ? (int64_t)down * (down + 1) / 2 : (int64_t)across * down;
  // a workgroup takes one 32 x 32 block of each wave
  for (int64_t unit = blockIdx.x; unit < tiles * g.batch * (I * J); unit += gridDim.x) {
    const int64_t which = unit / (I * J);
    const int block = (int)(unit - which * (I * J)), i = block / J, j = block % J;
    const int64_t matrix = which / tiles;
    const OrthoPlace at = ortho_place(kMirrored<KIND>, (int)(which - matrix * tiles), across, down);
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    for (int p = 0; p < g.k_parts; ++p) {
      const f32x4* const from = part_of<F>(g.partial, which * g.k_parts + p) + block * 4 * F::THREADS;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = from[q * F::THREADS];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[4 * q + r] += v[r];
      }
    }
    finish_block<KIND>(g, matrix, acc, at.tm * F::TM + wave / F::WN * (F::TM / F::WM) + 32 * i,
                       at.tn * F::TN + wave % F::WN * (F::TN / F::WN) + 32 * j,
                       KIND == kLast ? g.turned != 0 : at.tm != at.tn, lane, side + wave * 4096);
  }
}

template <class F, int KIND>
lowbit_status launch_form(const OrthoArgs& g, hipStream_t s) {
  const int64_t down = (g.m + F::TM - 1) / F::TM, across = (g.n + F::TN - 1) / F::TN;
  const int64_t tiles = g.batch * (kMirrored<KIND> ? down * (down + 1) / 2 : down * across);
  if (g.k_parts > 1 && !g.partial) return LOWBIT_EINVAL;
  const lowbit_status st = launch(&ortho_tile_kernel<F, KIND>,
                                  std::min<int64_t>(tiles * g.k_parts, 1 << 20), F::THREADS, s, g);
  if (st != LOWBIT_OK || g.k_parts == 1) return st;
  return launch(&ortho_add_kernel<F, KIND>, std::min<int64_t>(tiles * F::I * F::J, 1 << 20),
                F::THREADS, s, g);
}

template <int KIND>
lowbit_status launch_product(const OrthoArgs& args, hipStream_t s) {
  OrthoArgs g = args;
  const OrthoChoice c = ortho_choice(kMirrored<KIND>, KIND == kGram, g.batch, g.m, g.n);
  g.k_parts = c.parts;
  switch (c.form) {
    case 0: return launch_form<Shape<256, 256, 2, 4, 2, 1>, KIND>(g, s);
    case 1:
      if constexpr (kMirrored<KIND>) return launch_form<Shape<192, 192, 2, 2, 2, 1>, KIND>(g, s);
      return LOWBIT_EINVAL;                        // (not among the other products' forms)
    case 2: return launch_form<Shape<128, 128, 2, 2, 2, 2>, KIND>(g, s);
    case 3: return launch_form<Shape<128, 128, 2, 4, 4, 1>, KIND>(g, s);
    default: return launch_form<Shape<64, 64, 2, 2, 4, 2>, KIND>(g, s);
  }
}

template <int KIND>
lowbit_status launch_short(const OrthoArgs& g, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>(g.batch * ((g.n + 63) / 64), 1 << 20);
  return g.m <= 64 ? launch(&ortho_short_kernel<64, KIND>, blocks, 256, s, g)
                   : launch(&ortho_short_kernel<128, KIND>, blocks, 256, s, g);
}

}  // namespace

lowbit_status launch_ortho(int dt, const OrthoArgs& args, int steps, hipStream_t s) {
  OrthoArgs g = args;
  const int64_t parts = g.batch * g.nparts;
  const int64_t squares = g.batch * (g.ldn / 64) * ((g.m + 63) / 64);
  const int64_t blocks = std::min<int64_t>(squares, 1 << 20);
  lowbit_status st = dt == LOWBIT_F32
      ? launch(&ortho_norm_kernel<kF32>, std::min<int64_t>(parts, 1 << 20), 256, s, g)
      : launch(&ortho_norm_kernel<kBF16>, std::min<int64_t>(parts, 1 << 20), 256, s, g);
  if (st == LOWBIT_OK)
    st = dt == LOWBIT_F32 ? launch(&ortho_start_kernel<kF32>, blocks, 256, s, g)
                          : launch(&ortho_start_kernel<kBF16>, blocks, 256, s, g);
  for (int k = 0; k < steps && st == LOWBIT_OK; ++k) {
    st = launch_product<kGram>(g, s);
    const bool last = k + 1 == steps;
    if (g.m <= 128) {
      if (st == LOWBIT_OK) st = last ? launch_short<kLast>(g, s) : launch_short<kUpdate>(g, s);
    } else {
      if (st == LOWBIT_OK) st = launch_product<kPoly>(g, s);
      if (st == LOWBIT_OK) st = last ? launch_product<kLast>(g, s) : launch_product<kUpdate>(g, s);
    }
    std::swap(g.xh, g.xh_next);
  }
  return st == LOWBIT_OK && steps == 0 ? launch(&ortho_end_kernel, blocks, 256, s, g) : st;
}

}  // namespace lowbit
