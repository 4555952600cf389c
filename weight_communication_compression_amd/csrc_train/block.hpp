// block.hpp -- kernel argument blocks and launchers of rotary, attention and
// orthogonalize, shared by the kernels and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lowbit_train.h"

namespace lowbit {

struct RotaryArgs {
  const void* x;
  void* y;
  const double* freqs;
  const int64_t* positions;  // may be null
  int64_t rows, rows_per_sequence;
  int64_t x_row, x_head, y_row, y_head;
  int32_t heads, head_dim, rot_dim;
  int32_t lanes;             // units of a head: of pairs, then of 16 copied bytes
  int32_t turning;           // units that turn pairs
  int32_t groups;            // the heads are shared out among so many lanes
  int32_t rows_per_block;
  float scale, sign;
};

lowbit_status launch_rotary(int dt, int layout, const RotaryArgs& a, hipStream_t s);

struct AttnMatrix {
  const void* p;
  int64_t row, head;         // bytes
};

constexpr int kAttnRows = 128;   // of a workgroup's tile of queries, or of keys

// As many tiles as sequences of any lengths may have.
inline int attn_tiles(int64_t rows, int sequences) { return (int)(rows / kAttnRows) + sequences; }

struct AttnArgs {
  AttnMatrix q, k, v, o, dout, dq, dk, dv;
  const int32_t *q_begin, *k_begin, *prefix;   // may be null
  const float* slopes;       // may be null
  float* lse;                // q_heads x q_rows
  float* rows_info;          // gradient: q_heads x q_rows of lse, then of D
  // where there are too few tiles for the chip: into how many parts the keys of a tile of
  // queries are cut, and the gradient's queries of a tile of keys; and the parts' sums
  int32_t q_parts, k_parts;
  float *q_sums, *k_sums;
  int32_t q_rows, k_rows, sequences;
  int32_t q_heads, kv_heads, group;
  int32_t head_dim;
  int32_t causal, window;    // window 0: none
  float scale, softcap;
};

lowbit_status launch_attn_bf16(const AttnArgs& a, hipStream_t s);
lowbit_status launch_attn_f32(const AttnArgs& a, hipStream_t s);
lowbit_status launch_attn_back_bf16(const AttnArgs& a, hipStream_t s);
lowbit_status launch_attn_back_f32(const AttnArgs& a, hipStream_t s);
lowbit_status launch_attn_delta(int dt, const AttnArgs& a, hipStream_t s);

// ------------------------------------------------------- orthogonalize --
// X is m x n with m <= n: g or, for `turned`, its transpose.  Rows of the copies in
// the workspace are padded with zeros to multiples of kOrthoPad.
constexpr int kOrthoPad = 64;
constexpr int kOrthoParts = 256;   // of the sum of squares, at most

struct OrthoArgs {
  const void* g;
  void* out;
  double* parts;             // batch x kOrthoParts
  float* x;                  // batch x m x ldn
  void *xh, *xh_next;        // X in binary16, times a power of two (kX of ortho.hip)
  void *ah, *bh;             // A and b A + c A A in binary16, times others (kA, kB)
  float* partial;            // sums of parts of tiles that are cut along k
  int32_t k_parts;           // of the product that is launched
  int64_t batch;
  int32_t m, n, ldm, ldn;
  int32_t turned, nparts;
  float a, b, c, eps, scale;
};

lowbit_status launch_ortho(int dt, const OrthoArgs& a, int steps, hipStream_t s);

}  // namespace lowbit
