// train.hpp -- kernel argument blocks and launchers of the training-step
// operators, shared by the kernels and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lowbit_train.h"

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
  int threads;              // of a workgroup, which takes whole rows
  int vecs;                 // vectors of 8 elements per thread: 1 or 2
  int64_t blocks;
  int64_t rows_per_block;   // consecutive
};

struct JoinArgs {
  const void *f, *x;        // backward: x is x_out
  const void *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *x_out, *z;
  float* stats;
  int64_t rows, rows_per_block, rows_per_gate;
  int32_t cols;
  float eps, scale;
  uint32_t key, cut;
  float factor;
};

struct JoinBackArgs {
  JoinArgs j;
  const void *dx_out, *dz;
  void *df, *dx;
  // rows of `cols` partial sums, one for each workgroup (two for the gate: the
  // group that its first row belongs to, the one its last row belongs to)
  float *part_post_w, *part_post_b, *part_pre_w, *part_pre_b, *part_gate;
  float* dgate;             // groups that lie within one workgroup's rows
};

struct JoinSumArgs {
  const float* part[4];     // partial sums of the weights and biases
  float* out[4];
  const float* part_gate;
  float* dgate;
  int64_t rows, rows_per_block, rows_per_gate, blocks;
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

}  // namespace lowbit
