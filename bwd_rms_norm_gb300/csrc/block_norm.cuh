// Declarations shared by the block norm's kernels: the scalar ones
// (block_norm.cu) and the staged ones (block_norm_tma.cuh).
#pragma once

#include "launch.h"

namespace rmsn {

// Where a unit's rows meet the gate's rows.  Unit u of U owns the rows
// [u R / U, (u + 1) R / U); gate row q owns rows_per_gate rows.  The pieces
// in which both are constant are the segments: each step from one segment to
// the next raises u or q (or both), so u + q numbers the segments without a
// clash, and below U + gate_rows.  Each segment has its own partial row of A.
// Where rows start anywhere in 16 bytes there are `period` classes of them, the
// rows c + period i of each over its own U / period units: unit u is of class
// u mod period, and the classes' segments follow one another.
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
  float* p_a;      // [units + period * gate rows, hidden] partial rows of A
  int64_t rows;
  int64_t rows_per_gate;
  int hidden;
  float a, b, off;
  int period;      // classes of rows the units are of (row_period), else 1
};

// Whether rows that start anywhere in 16 bytes are worth the staged kernels'
// start, over block_norm.cu's loops over single elements.  (bf16; loops /
// staged.)  Forward: 256 x 4097 9.6 / 10.0 us, 1024 x 4097 15.2 / 11.9, 1024 x
// 8191 27.8 / 21.5, 4096 x 257 9.1 / 15.0, 4096 x 1001 17.3 / 18.4, 16000 x 1001
// 58.5 / 55.0, 16000 x 4097 174 / 117; gates of several rows, which both read
// an element at a time: 4096 x 4097 48 / 59.
inline bool block_fwd_odd_pays(int64_t rows, int64_t rows_per_gate, int hidden) {
  return hidden >= 64 && rows >= 128 && rows_per_gate == rows &&
         rows * hidden >= (hidden > 1024 ? 1 << 21 : 1 << 22);
}

// Backward: 64 x 4097 8.7 / 13.0 us, 256 x 4097 18.5 / 14.8, 1024 x 257 13.0 /
// 9.4, 1024 x 1001 23.3 / 15.1, 4096 x 4097 176 / 45, 16000 x 8191 1484 / 329.  A
// unit's rows are of every gate row, of each an eighth of its rows: 4096 x 1001
// with 64, 16 and 4 gate rows 78 / 109, 78 / 52 and 78 / 42; 4096 x 4097 195 /
// 365, 201 / 155, 191 / 92.
inline bool block_bwd_odd_pays(int64_t rows, int64_t rows_per_gate, int hidden) {
  return hidden >= 64 && rows >= 128 && rows * hidden >= 1 << 18 &&
         (rows_per_gate == rows ||
          (rows_per_gate >= 256 && rows_per_gate * hidden >= 1 << 18));
}

// Staged kernels (block_fwd_tma.cu, block_bwd_tma.cu; block_bwd_odd.cu for rows
// that start anywhere in 16 bytes).  Each returns false, having enqueued
// nothing, where the sizes or the alignment do not suit it; otherwise true
// with the launch status in *err.  The backward sets p's partial rows and
// *units, for the sums that follow.
bool try_launch_block_fwd_tma(int dtype, int res_dtype, const BlockFwdArgs& a, cudaStream_t s,
                              cudaError_t* err);
bool try_launch_block_bwd_tma(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p,
                              int* units, cudaStream_t s, cudaError_t* err);
bool try_launch_block_bwd_odd(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p,
                              int* units, cudaStream_t s, cudaError_t* err);
// Bounded waits of theirs that ran out.
cudaError_t read_block_fwd_wait_timeouts(unsigned int* out);
cudaError_t read_block_bwd_tma_wait_timeouts(unsigned int* out);
cudaError_t read_block_bwd_odd_wait_timeouts(unsigned int* out);
cudaError_t read_block_wait_timeouts(unsigned int* out);  // their sum

// The partial rows of `units` units in the caller's workspace.
inline void place_partials(const BlockBwdArgs& a, int units, BlockBwdParams& p) {
  p.p_next = a.partial;
  p.p_post = a.partial + (int64_t)units * a.hidden;
  p.p_a = a.partial + 2 * (int64_t)units * a.hidden;
}

}  // namespace rmsn
