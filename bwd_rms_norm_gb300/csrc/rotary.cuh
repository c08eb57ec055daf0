// The head norm and rotation's arguments, and what its kernels share: a
// token's angles.
#pragma once

#include "cluster_launch.cuh"
#include "common.cuh"
#include "launch.h"
#include "rms_norm.h"

namespace rmsn {

// A tensor of heads [batch, tokens, heads, dim], strides in elements.
struct HeadView {
  char* p;
  int64_t sb, st, sh;
};

// One of the two tensors of a call, queries or keys.
struct RotarySide {
  HeadView in, out;      // forward: v and y; backward: v and dv
  HeadView dy;           // backward
  const void* gamma;
  float* rstd;           // [batch * tokens, heads]
  float* dgamma;         // backward
  float* partial;        // backward: [CTAs of this side, dim], unless `direct`
  int heads;
  int ctas;              // backward: CTAs that take this side
};

struct RotaryParams {
  RotarySide side[2];    // queries, keys (heads 0: none)
  const void* inv_freq;
  const void* positions; // NULL: the token's index
  int64_t pos_stride;    // between batch entries
  int freq64, pos64;
  int all, tokens;       // batch * tokens, tokens of a batch entry
  int dim, half;         // half: pairs
  int interleaved;
  float eps, off;
  bool vec_ok;           // 16-byte aligned rows in every tensor of heads
  bool direct;           // backward: a side's CTAs are a cluster, which adds up their sums
};

// inv_freq in turns a position, in units of 2^-64 turns: the product with a
// position, modulo 2^64, is the angle modulo a turn.  1 / (2 pi) goes in as two
// doubles, so that the turns are off by 2^-63 or so a position, not by the 2^-54
// of one product.
__device__ __forceinline__ uint64_t fixed_turns(const RotaryParams& p, int i) {
  constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
  const double f = p.freq64 ? static_cast<const double*>(p.inv_freq)[i]
                            : (double)static_cast<const float*>(p.inv_freq)[i];
  const double t = f * kHigh, rest = fma(f, kHigh, -t) + f * kLow;
  const double part = t - rint(t);  // exact
  return (uint64_t)((long long)(part * 0x1p64)) + (uint64_t)((long long)(rest * 0x1p64));
}

// (cos, sin) of a position's angle, from the upper 32 bits of its turn (low by less
// than 2^-32 of one) as an fp32 part of a half turn (off by 2^-25 of one at most,
// which is 2^6 times as much).
__device__ __forceinline__ float2 turn_of(uint64_t fixed, int64_t position) {
  const int part = (int)((fixed * (uint64_t)position) >> 32);
  float2 cs;
  sincospif((float)part * 0x1p-31f, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ int64_t position_of(const RotaryParams& p, int b, int t) {
  if (!p.positions) return t;
  const int64_t at = b * p.pos_stride + t;
  return p.pos64 ? static_cast<const int64_t*>(p.positions)[at]
                 : static_cast<const int32_t*>(p.positions)[at];
}

__device__ __forceinline__ int64_t row_at(const HeadView& v, int b, int t, int h) {
  return b * v.sb + t * v.st + h * v.sh;
}

// Few rows: the sums of the gammas' gradients stay inside a cluster of CTAs for
// each side, without workspace, partial rows and a second kernel.  It is the calls
// that gain: 256 x (8+8) x 64 fp32 11.9 us with partial rows, 7.2 so, 64 x (32+8) x
// 128 bf16 11.8 and 8.7.  In a graph, where a launch costs little, the clusters'
// passes over the rows take longer but for the fewest: 4.8 and 6.9 us, 5.5 and 8.6;
// 8 x (32+8) x 128 5.2 and 4.8.
inline bool few_rows(int64_t all, int64_t q_heads, int64_t k_heads, int64_t dim) {
  const int64_t rows = all * (q_heads > k_heads ? q_heads : k_heads);
  return rows <= 2048 && rows * dim <= 1 << 18;
}

// The CTAs of a side, where they are a cluster.
inline int cluster_of(int64_t rows, int64_t rows_a_cta, int sms) {
  int n = 1;
  while (n < kMaxCluster && 2 * n <= sms && n * rows_a_cta < rows) n *= 2;
  return n;
}

// Adds up the CTAs' sums, `mine` [dim] in each one's shared memory, in the order
// of the cluster's CTAs.
__device__ __forceinline__ void add_cluster(const float* mine, float* dgamma, int dim, int ctas) {
  __syncthreads();
  cluster_sync();
  if (cta_rank() == 0)
    for (int j = threadIdx.x; j < dim; j += blockDim.x) {
      float part[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        part[c] = c < ctas ? __uint_as_float(ld_peer(mine + j, c)) : 0.f;
      float v = part[0];
#pragma unroll
      for (int c = 1; c < kMaxCluster; ++c) v += part[c];
      dgamma[j] = v;
    }
  cluster_sync();  // no CTA leaves while its sums are read
}

// Shares `most` CTAs between queries and keys by their costs, at least one each,
// and places their partial rows; a CTA has `rows_a_cta` rows at least.
inline void share_ctas(RotaryParams& p, int64_t most, int64_t rows_a_cta, int64_t q_cost,
                       int64_t k_cost) {
  if (most > RMSN_ROTARY_MAX_PARTIALS) most = RMSN_ROTARY_MAX_PARTIALS;
  if (most < 2) most = 2;
  int64_t left = most;
  for (int i = 1; i >= 0; --i) {
    RotarySide& s = p.side[i];
    if (s.heads == 0) continue;
    int64_t n = i == 1 ? most * k_cost / (q_cost + k_cost) : left;
    if (n < 1) n = 1;
    if (i == 1 && n >= most) n = most - 1;
    left -= n;
    const int64_t useful = ((int64_t)p.all * s.heads + rows_a_cta - 1) / rows_a_cta;
    s.ctas = (int)(n < useful ? n : useful);
  }
  p.side[1].partial = p.side[0].partial + (int64_t)p.side[0].ctas * p.dim;
}

// The backward's CTAs, of `most` at once; returns the size of their clusters.
// q_cost, k_cost: of a token's queries and of its keys.
inline int place_ctas(RotaryParams& p, int64_t most, int64_t rows_a_cta, int sms, int64_t q_cost,
                      int64_t k_cost) {
  if (!p.direct) {
    share_ctas(p, most, rows_a_cta, q_cost, k_cost);
    return 1;
  }
  const int heads = p.side[0].heads > p.side[1].heads ? p.side[0].heads : p.side[1].heads;
  const int n = cluster_of((int64_t)p.all * heads, rows_a_cta, sms);
  for (RotarySide& s : p.side) s.ctas = s.heads > 0 ? n : 0;
  return n;
}

// Kernels of rows of 16-byte vectors (rotary_vec.cu).  Each returns false,
// having enqueued nothing, where the sizes or the alignment do not suit it;
// otherwise true with the launch status in *err.
bool try_launch_rotary_fwd_vec(int dtype, const RotaryParams& p, cudaStream_t s, cudaError_t* err);
bool try_launch_rotary_bwd_vec(int dtype, RotaryParams& p, cudaStream_t s, cudaError_t* err);

}  // namespace rmsn
