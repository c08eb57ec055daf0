// Declarations shared by the block norm's kernels: the scalar ones
// (block_norm.cu) and the staged ones (block_norm_tma.cu).
#pragma once

#include "launch.h"

namespace rmsn {

// Where a unit's rows meet the gate's rows.  Unit u of U owns the rows
// [u R / U, (u + 1) R / U); gate row q owns rows_per_gate rows.  The pieces
// in which both are constant are the segments: each step from one segment to
// the next raises u or q (or both), so u + q numbers the segments without a
// clash, and below U + gate_rows.  Each segment has its own partial row of A.
struct BlockBwdParams {
  const void* dy;
  const void* dr;
  const void* x;
  const void* r;
  const void* gamma_post;
  const void* gate;
  const void* gamma_next;
  const float* rstd_post;
  const float* rstd_next;
  void* dx;
  void* dres;
  float* p_next;   // [units, hidden] partial rows of dgamma_next
  float* p_post;   // [units, hidden] partial rows of dgamma_post
  float* p_a;      // [units + gate rows, hidden] partial rows of A
  int64_t rows;
  int64_t rows_per_gate;
  int hidden;
  float a, b, off;
};

// Staged kernels (block_norm_tma.cu).  Each returns false, having enqueued
// nothing, where the sizes or the alignment do not suit it; otherwise true
// with the launch status in *err.  The backward sets p's partial rows and
// *units, for the sums that follow.
bool try_launch_block_fwd_tma(int dtype, int res_dtype, const BlockFwdArgs& a, cudaStream_t s,
                              cudaError_t* err);
bool try_launch_block_bwd_tma(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p,
                              int* units, cudaStream_t s, cudaError_t* err);
// Bounded waits of theirs that ran out.
cudaError_t read_block_wait_timeouts(unsigned int* out);

// The partial rows of `units` units in the caller's workspace.
inline void place_partials(const BlockBwdArgs& a, int units, BlockBwdParams& p) {
  p.p_next = a.partial;
  p.p_post = a.partial + (int64_t)units * a.hidden;
  p.p_a = a.partial + 2 * (int64_t)units * a.hidden;
}

}  // namespace rmsn
