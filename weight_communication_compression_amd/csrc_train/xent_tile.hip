// linear xent: its products in 128 x 128 tiles
#include "train.hpp"
#include "train_device.hpp"
#include "../csrc/launch.hpp"

namespace lowbit {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = kXentTile;
constexpr int kRowBytes = 64;              // of a tile's row: 32 bfloat16 or 16 binary32 of k
constexpr int kRowStride = kRowBytes + 16; // in LDS: rows 20 banks apart

// 16 bytes of consecutive elements at p, `left` of them there (the rest 0).
template <int DT>
__device__ __forceinline__ u32x4 load16(const char* p, int64_t left) {
  constexpr int E = 16 / elem_size<DT>();
  if (left >= E) {
    if constexpr (DT == kF32) return *reinterpret_cast<const u32x4_4*>(p);
    else return *reinterpret_cast<const u32x4_2*>(p);
  }
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (j < left) {
      if constexpr (DT == kF32) v[j] = reinterpret_cast<const uint32_t*>(p)[j];
      else v[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j % 2));
    }
  }
  return v;
}

// A thread's two 16-byte pieces of a 128-row tile's next 64 bytes of k.
// OUTER: k is the matrix's row, and a piece holds consecutive rows of the tile.
template <int DT, bool OUTER>
struct Stage {
  static constexpr int ES = elem_size<DT>(), E = 16 / ES, K = kRowBytes / ES;
  u32x4 v[2];
  __device__ __forceinline__ void load(const void* base, int64_t ld, int64_t row0, int64_t rows,
                                       int64_t k0, int64_t k) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = threadIdx.x + i * 256;
      int64_t r, c, left;
      if constexpr (OUTER) {
        c = k0 + p / (kTile / E);
        r = row0 + p % (kTile / E) * E;
        left = c < k ? rows - r : 0;
        v[i] = load16<DT>(static_cast<const char*>(base) + (c * ld + r) * ES, left);
      } else {
        r = row0 + p / 4;
        c = k0 + p % 4 * E;
        left = r < rows ? k - c : 0;
        v[i] = load16<DT>(static_cast<const char*>(base) + (r * ld + c) * ES, left);
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = threadIdx.x + i * 256;
      if constexpr (OUTER) {
        const int c = p / (kTile / E), r = p % (kTile / E) * E;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          char* to = lds + (r + j) * kRowStride + c * ES;
          if constexpr (DT == kF32) *reinterpret_cast<uint32_t*>(to) = v[i][j];
          else *reinterpret_cast<uint16_t*>(to) = (uint16_t)(v[i][j / 2] >> (16 * (j % 2)));
        }
      } else {
        *reinterpret_cast<u32x4*>(lds + p / 4 * kRowStride + p % 4 * 16) = v[i];
      }
    }
  }
};

// The product of 16 rows of n with 16 rows of m over 64 bytes of k, of which
// lane l holds row l mod 16, the (l / 16)-th 16 bytes.  For binary32 four
// products take one element of each lane: k in another order, the same for both.
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

// exp in binary32 (within about 2 units in the last place): 2^t with
// t = x log2(e) and its rounding error made good
__device__ __forceinline__ float exp_f32(float x) {
  const float t = x * 1.44269502f;                        // log2(e) to binary32
  const float e = __builtin_fmaf(x, 1.44269502f, -t) + x * 1.92596303e-8f;
  const float y = __builtin_amdgcn_exp2f(t);
  return x < -200.0f ? 0.0f : __builtin_fmaf(y, e * 0.693147182f, y);
}

// Four waves, each 64 x 64 of the tile: 4 x 4 products of 16 x 16.  Lane l holds
// of product (i, j) column m = 16 i + l mod 16 and rows n = 16 j + 4 (l / 16) + r:
// four consecutive columns of the output's row m.
template <int DT, int KIND>
__global__ void __launch_bounds__(256) xent_tile_kernel(XentTileArgs g) {
  constexpr bool AO = KIND == kXentDw, BO = KIND == kXentDx || KIND == kXentDw;
  __shared__ __attribute__((aligned(16))) char lds[2][2][kTile * kRowStride];
  __shared__ float2 halves[2][kTile];
  const int64_t count = *g.count;
  const int64_t m = KIND == kXentDw ? g.m : count, k = KIND == kXentDw ? count : g.k;
  const int64_t across = (g.n + kTile - 1) / kTile, tiles = across * ((m + kTile - 1) / kTile);
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int wm = wave & 1, wn = wave >> 1;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile / across * kTile, n0 = tile % across * kTile;
    f32x4 acc[4][4];
  #pragma unroll
    for (int i = 0; i < 4; ++i)
  #pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

    Stage<DT, AO> sa;
    Stage<DT, BO> sb;
    constexpr int K = kRowBytes / elem_size<DT>();
    const int64_t steps = (k + K - 1) / K;
    if (steps > 0) {
      sa.load(g.a, g.lda, m0, m, 0, k);
      sb.load(g.b, g.ldb, n0, g.n, 0, k);
      sa.store(lds[0][0]);
      sb.store(lds[0][1]);
    }
    for (int64_t s = 0; s < steps; ++s) {
      __syncthreads();
      if (s + 1 < steps) {
        sa.load(g.a, g.lda, m0, m, (s + 1) * K, k);
        sb.load(g.b, g.ldb, n0, g.n, (s + 1) * K, k);
      }
      const char* la = lds[s & 1][0] + (wm * 64 + lane % 16) * kRowStride + lane / 16 * 16;
      const char* lb = lds[s & 1][1] + (wn * 64 + lane % 16) * kRowStride + lane / 16 * 16;
      u32x4 a[4], b[4];
  #pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = *reinterpret_cast<const u32x4*>(la + i * 16 * kRowStride);
        b[i] = *reinterpret_cast<const u32x4*>(lb + i * 16 * kRowStride);
      }
  #pragma unroll
      for (int i = 0; i < 4; ++i)
  #pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mma<DT>(b[j], a[i], acc[i][j]);
      if (s + 1 < steps) {
        sa.store(lds[(s + 1) & 1][0]);
        sb.store(lds[(s + 1) & 1][1]);
      }
    }

    const int64_t nl = n0 + wn * 64 + lane / 16 * 4;     // + 16 j + r
  #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = m0 + wm * 64 + i * 16 + lane % 16;
      if constexpr (KIND == kXentStats) {
        float top = -INFINITY;
        const int target = row < m ? __float_as_int(g.info[row].w) : -1;
  #pragma unroll
        for (int j = 0; j < 4; ++j)
  #pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t n = nl + 16 * j + r;
            if (n < g.n) top = fmaxf(top, acc[i][j][r]);
            if (n == target) g.hit[row] = acc[i][j][r];
          }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
  #pragma unroll
        for (int j = 0; j < 4; ++j)
  #pragma unroll
          for (int r = 0; r < 4; ++r)
            if (nl + 16 * j + r < g.n) sum += exp_f32(acc[i][j][r] - base);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (lane < 16) halves[wn][wm * 64 + i * 16 + lane] = make_float2(top, sum);
      } else if constexpr (KIND == kXentProb) {
        const float4 info = row < m ? g.info[row] : make_float4(0, 0, 0, 0);
        const float scale = DT == kF32 ? 1.0f : *g.scale;
        const float both = info.y / scale, own = info.z / scale;
        const int64_t target = __float_as_int(info.w) - g.col0;
        if (row < m) {
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            float d[4];
  #pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int64_t n = nl + 16 * j + r;
              d[r] = exp_f32(acc[i][j][r] - info.x) * both - (n == target ? own : 0.0f);
              if (n >= g.n) d[r] = 0.0f;
            }
            char* to = static_cast<char*>(g.out) + (row * g.ldo + nl + 16 * j) * elem_size<DT>();
            if constexpr (DT == kF32)
              *reinterpret_cast<float4*>(to) = make_float4(d[0], d[1], d[2], d[3]);
            else
              *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]));
          }
        }
      } else if (row < m) {
        const float scale = DT == kF32 ? 1.0f : *g.scale;
        int64_t to = row * g.ldo;
        if constexpr (KIND == kXentDx)
          if (g.last) to = (int64_t)g.map[row] * g.ldo;
  #pragma unroll
        for (int j = 0; j < 4; ++j)
  #pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t n = nl + 16 * j + r;
            if (n >= g.n) continue;
            float v = acc[i][j][r];
            if constexpr (KIND == kXentDx) {
              if (!g.first) v += g.acc[row * g.ldo + n];
              if (!g.last) {
                g.acc[row * g.ldo + n] = v;
                continue;
              }
            }
            v *= scale;
            if constexpr (DT == kF32) static_cast<float*>(g.out)[to + n] = v;
            else static_cast<uint16_t*>(g.out)[to + n] = (uint16_t)pack_bf16(v, 0.0f);
          }
      }
    }
    if constexpr (KIND == kXentStats) {
      __syncthreads();
      const int64_t row = m0 + threadIdx.x;
      if (threadIdx.x < kTile && row < m) {
        const float2 p = halves[0][threadIdx.x], q = halves[1][threadIdx.x];
        const float top = fmaxf(p.x, q.x);
        const float sum = (p.x == -INFINITY ? p.y : p.y * exp_f32(p.x - top)) +
                          (q.x == -INFINITY ? q.y : q.y * exp_f32(q.x - top));
        g.part[row * g.parts + tile % across] = make_float2(top, sum);
      }
    }
    __syncthreads();                       // the next tile's loads overwrite these
  }
}

template <int DT>
lowbit_status tile_kind(int kind, const XentTileArgs& a, hipStream_t s) {
  void (*k)(XentTileArgs) = kind == kXentStats  ? &xent_tile_kernel<DT, kXentStats>
                            : kind == kXentProb ? &xent_tile_kernel<DT, kXentProb>
                            : kind == kXentDx   ? &xent_tile_kernel<DT, kXentDx>
                                                : &xent_tile_kernel<DT, kXentDw>;
  // one tile for each workgroup; what lies beyond the grid's limit, and nothing
  // where fewer rows count than there are, in its loop
  const int64_t tiles = ((a.n + kTile - 1) / kTile) * ((a.m + kTile - 1) / kTile);
  return launch(k, grid_blocks(tiles * 4, 256), 256, s, a);
}

}  // namespace

lowbit_status launch_xent_tile(int dt, int kind, const XentTileArgs& a, hipStream_t s) {
  return dt == kF32 ? tile_kind<kF32>(kind, a, s) : tile_kind<kBF16>(kind, a, s);
}

}  // namespace lowbit
