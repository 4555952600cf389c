// train.hpp -- kernel argument blocks and launchers of the training-step
// operators, shared by the kernels and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lowbit_train.h"
#include "xent_cut.hpp"

namespace lowbit {

struct DropoutArgs {
  const void* x;
  const void* r;            // residual, may be null
  void* y;
  int64_t n;
  uint64_t pair0;           // mask pair of elements 0 and 1
  uint32_t key, cut;
  float factor;
};

constexpr int kJoinMaxCols = 16384;
struct JoinShape {
  int threads;              // of a workgroup
  int lanes;                // of a row: 8 to 64 (several rows a workgroup), or all threads
  int vecs;                 // vectors of 8 elements per lane: 1 or 2
  bool ragged;              // the lanes have more elements than a row
  int64_t runs;             // runs of rows_per_run consecutive rows, each `lanes` lanes'
  int64_t rows_per_run;
  int64_t blocks;           // workgroups of threads / lanes runs
};

struct JoinArgs {
  const void *f, *x;        // backward: x is x_out
  const void *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *x_out, *z;
  float* stats;
  int64_t rows, rows_per_run, rows_per_gate;
  int32_t cols, lanes;
  float eps, scale;
  uint32_t key, cut;
  float factor;
};

struct JoinBackArgs {
  JoinArgs j;
  const void *dx_out, *dz;
  void *df, *dx;
  // rows of `cols` partial sums, one for each workgroup (for the gate two for each
  // run: the group that its first row belongs to, the one its last row belongs to)
  float *part_post_w, *part_post_b, *part_pre_w, *part_pre_b, *part_gate;
  float* dgate;             // groups that lie within one run
};

struct JoinSumArgs {
  const float* part[4];     // partial sums of the weights and biases
  float* out[4];
  const float* part_gate;
  float* dgate;
  int64_t rows, rows_per_run, rows_per_gate, blocks;
  int32_t cols;
  int32_t params;           // how many of part[] there are
};

lowbit_status launch_dropout(int dt, const DropoutArgs& a, hipStream_t s);

JoinShape join_shape(int64_t rows, int cols, bool backward);
lowbit_status launch_join(int ft, int st, int pt, bool layer, const JoinShape& g,
                          const JoinArgs& a, hipStream_t s);
lowbit_status launch_join_back(int ft, int st, int pt, bool layer, const JoinShape& g,
                               const JoinBackArgs& a, hipStream_t s);
lowbit_status launch_join_sums(const JoinSumArgs& a, hipStream_t s);

// ---------------------------------------------------------- linear xent --
// The rows that count are taken together: compact row i stands for row map[i].
struct XentRows {
  const int64_t* targets;
  const float *lse, *dloss, *dlse;   // backward; dlse may be null
  int64_t n, vocab, ignore;
  int32_t* pos;              // n: compact row of a row, or -1
  int32_t* map;              // padded rows: row of a compact row, or -1
  // padded rows: lse, dloss + dlse, dloss, target (bits; -1: none); zeros beyond
  // the rows that count
  float4* info;
  int32_t* count;            // how many count
  float* scale;              // the largest finite |dloss| or |dloss + dlse|, or 1
  int64_t padded;
};

struct XentGather {
  const void* x;
  void* xc;                  // compact rows, zeros beyond the count
  void* dx;                  // backward: rows that are left out are set to 0; may be null
  const int32_t *pos, *map;
  int64_t n, padded;
  int32_t hidden, ld;        // of x and dx; of xc
};

// Rows of w with a multiple of 16 bytes each, zeros at their ends.
struct XentPack {
  const void* w;
  void* to;
  int64_t rows;
  int32_t hidden, ld;
};

struct XentJoin {
  const float2* part;        // compact row x parts: maximum, sum of exp(l - maximum)
  const float* hit;          // the target's logit
  const int64_t* targets;
  const int32_t* pos;
  int64_t n, vocab;
  int32_t parts;
  float *loss, *lse;
};

struct XentTileArgs {
  const void *a, *b;         // a[m lda + k], or a[k lda + m] where the kind has it so
  int64_t lda, ldb;          // multiples of 16 bytes
  int64_t m, n, k;           // m, n of the output, k summed over; a dimension of
                             // rows is the padded count, cut to the real one
  const int32_t* count;
  const int32_t* map;
  const float4* info;
  const float* scale;
  int64_t col0;              // vocabulary column of n = 0 (logits)
  float2* part;
  float* hit;
  int32_t parts, part0;      // of a row; the first of n = 0
  void* out;                 // d, dx or dw
  int64_t ldo;
  float* acc;                // dx over several pieces: their sum so far, tile by tile
  int32_t first, last;       // piece of the vocabulary
  float* partial;            // sums of the parts of tiles that are cut along k
  int32_t may_cut;           // whether there are any
};

lowbit_status launch_xent_rows(int dt, const XentRows& r, const XentGather& g, hipStream_t s);
lowbit_status launch_xent_pack(int dt, const XentPack& a, hipStream_t s);
lowbit_status launch_xent_join(const XentJoin& a, hipStream_t s);
lowbit_status launch_xent_tile_bf16(int form, int kind, const XentTileArgs& a, hipStream_t s);
lowbit_status launch_xent_tile_f32(int form, int kind, const XentTileArgs& a, hipStream_t s);

constexpr int64_t kXentPad = 256;  // rows and pieces of the vocabulary: multiples of every tile's
int xent_form(int dt, int kind, int64_t m, int64_t n, int64_t k);

}  // namespace lowbit
