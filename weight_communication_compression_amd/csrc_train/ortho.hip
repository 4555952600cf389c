// ortho.hip -- orthogonalize: Newton-Schulz products.
#include "block.hpp"
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
// Sums of squares in binary64, which no binary32 input leaves: nparts of each matrix.
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
// turned through LDS where the matrix is.
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
};

// What becomes of four consecutive columns of a row.
template <int KIND>
__device__ __forceinline__ void emit(const OrthoArgs& g, int64_t matrix, int row, int col, f32x4 v) {
  if (row >= g.m) return;
  if constexpr (KIND == kUpdate) {
    if (col >= g.ldn) return;
    const int64_t at = (matrix * g.m + row) * g.ldn + col;
    const f32x4 x = *reinterpret_cast<const f32x4*>(g.x + at);
    f32x4 y;
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(g.a, x[r], v[r] * (1.0f / (kB * kX)));
    *reinterpret_cast<f32x4*>(g.x + at) = y;
    *reinterpret_cast<u32x2*>(static_cast<_Float16*>(g.xh_next) + at) = pack_f16(y * kX);
  } else {
    if (col >= g.ldm) return;
    const int64_t at = (matrix * g.m + row) * g.ldm + col;
    if constexpr (KIND == kGram) {
      *reinterpret_cast<u32x2*>(static_cast<_Float16*>(g.ah) + at) = pack_f16(v * (kA / (kX * kX)));
    } else {
      const f32x4 a = unpack_f16(*reinterpret_cast<const u32x2*>(static_cast<_Float16*>(g.ah) + at));
      f32x4 y;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        y[r] = __builtin_fmaf(g.b * (kB / kA), a[r], v[r] * (g.c * (kB / (kA * kA))));
      *reinterpret_cast<u32x2*>(static_cast<_Float16*>(g.bh) + at) = pack_f16(y);
    }
  }
}

template <class F, int KIND>
__global__ void __launch_bounds__(F::THREADS, F::SLOTS * F::W / 1024) ortho_tile_kernel(OrthoArgs g) {
  constexpr int DT = F::DT, TM = F::TM, TN = F::TN, W = F::W, I = F::I, J = F::J;
  constexpr bool BO = KIND == kUpdate;
  constexpr int K = kRowBytes / 2;
  __shared__ __attribute__((aligned(1024))) char la0[TM * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb0[TN * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char la1[TM * kRowBytes];
  __shared__ __attribute__((aligned(1024))) char lb1[TN * kRowBytes];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / F::WN, wn = wave % F::WN;
  const int k = KIND == kGram ? g.n : g.m, n = KIND == kUpdate ? g.n : g.m;
  const int lda = KIND == kGram ? g.ldn : g.ldm, ldb = KIND == kPoly ? g.ldm : g.ldn;
  const int across = (n + TN - 1) / TN, down = (g.m + TM - 1) / TM;
  const int64_t tiles = (int64_t)across * down;
  const int steps = (k + K - 1) / K;

  constexpr int NA = Feed<DT, TM, W, false>::LOADS, NB = Feed<DT, TN, W, BO>::LOADS, N = NA + NB;
  constexpr int RD = I + J * (BO ? 2 : 1);
  Feed<DT, TM, W, false> fa;
  Feed<DT, TN, W, BO> fb;
  Frag<DT, TM, false> ra;
  Frag<DT, TN, BO> rb;
  fa.init(lda, wave, lane);
  fb.init(ldb, wave, lane);
  ra.init(wm * (TM / F::WM), lane);
  rb.init(wn * (TN / F::WN), lane);
  u32x4 fra[2][I], frb[2][J];
  f32x16 acc[I][J];

  auto kleft = [&](int s) { return min(k - s * K, K); };
  auto issue = [&](char* la, char* lb, int s) {
    const auto qa = fa.open(s < steps), qb = fb.open(s < steps);
#pragma unroll
    for (int j = 0; j < NA; ++j) fa.load(qa, la, wave, kleft(s), j);
#pragma unroll
    for (int j = 0; j < NB; ++j) fb.load(qb, lb, wave, kleft(s), j);
    fa.next();
    fb.next();
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
    spread_reads<RD, I * J>();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step s, in la and lb, whose first quarter is in registers.  While a quarter is
  // multiplied the next is read; before the last, everybody has read all of
  // this step, the next one has arrived, and the loads of the one after it begin.
  auto step = [&](char* la, char* lb, const char* na, const char* nb, int s) {
    const auto qa = fa.open(s + 2 < steps), qb = fb.open(s + 2 < steps);
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
    spread_loads<RD, I * J, 1, N>();
    __builtin_amdgcn_sched_barrier(0);
  };

  for (int64_t unit = blockIdx.x; unit < tiles * g.batch; unit += gridDim.x) {
    const int64_t matrix = unit / tiles;
    const int in = (int)(unit - matrix * tiles);
    const int tm = in / across, tn = in % across;
    const int64_t mm = matrix * g.m;
    const _Float16* a = static_cast<const _Float16*>(KIND == kGram ? g.xh : KIND == kPoly ? g.ah : g.bh);
    const _Float16* b = static_cast<const _Float16*>(KIND == kPoly ? g.ah : g.xh);
    fa.seek(a + mm * lda, lda, g.m, (int64_t)tm * TM, 0);
    fb.seek(b + mm * ldb, ldb, g.m, (int64_t)tn * TN, 0);
    issue(la0, lb0, 0);
    issue(la1, lb1, 1);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    wait_loads();
    barrier();
    read(0, la0, lb0, 0);
    __builtin_amdgcn_sched_barrier(0);
    int s = 0;
    for (; s + 1 < steps; s += 2) {
      step(la0, lb0, la1, lb1, s);
      step(la1, lb1, la0, lb0, s + 1);
    }
    if (s < steps) step(la0, lb0, la1, lb1, s);
    wait_loads();
    barrier();
    const int row = tm * TM + wm * (TM / F::WM) + lane % 32;
    const int col = tn * TN + wn * (TN / F::WN) + lane / 32 * 4;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          emit<KIND>(g, matrix, row + 32 * i, col + 32 * j + 8 * q, quad(acc[i][j], q));
  }
}

template <int KIND>
lowbit_status launch_product(const OrthoArgs& g, hipStream_t s) {
  const int n = KIND == kUpdate ? g.n : g.m;
  auto tiles = [&](int t) { return g.batch * ((g.m + t - 1) / t) * ((n + t - 1) / t); };
  if (tiles(256) >= 256)
    return launch(&ortho_tile_kernel<Form<kF16, 256, 256, 2, 4, 256>, KIND>,
                  std::min<int64_t>(tiles(256), 1 << 20), 512, s, g);
  return launch(&ortho_tile_kernel<Form<kF16, 128, 128, 2, 2, 512>, KIND>,
                std::min<int64_t>(tiles(128), 1 << 20), 256, s, g);
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
    if (st == LOWBIT_OK) st = launch_product<kPoly>(g, s);
    if (st == LOWBIT_OK) st = launch_product<kUpdate>(g, s);
    std::swap(g.xh, g.xh_next);
  }
  return st == LOWBIT_OK ? launch(&ortho_end_kernel, blocks, 256, s, g) : st;
}

}  // namespace lowbit
