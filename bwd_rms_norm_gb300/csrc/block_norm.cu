// Block norm for sm_103a: the norms after and before a transformer block
// fused with the block's gate and the scaled residual sum.
//
//   z = x * rstd_post * w1                      w1 = gamma_post + offset
//   r = a * res + b * gate_q * z                (z = x without a post norm)
//   y = r * rstd_next * w2                      w2 = gamma_next + offset
//
// rstd_post = 1/sqrt(mean(x^2) + eps), rstd_next = 1/sqrt(mean(r^2) + eps);
// row i uses gate row q = i / rows_per_gate.  Every product and sum is fp32
// and r, y are rounded once, at their stores: y is formed from the fp32 r,
// not from the rounded one.
//
// The backward, from dy (of y) and dr (of r):
//   D       = dr + rstd_next * (dy w2 - rh * c1),  rh = r * rstd_next,
//             c1 = mean(dy w2 rh)
//   dres    = a * D
//   dx      = rstd_post * (w D - xh * c2),  xh = x * rstd_post,
//             w = b gate w1,  c2 = mean(w D xh)
//   A_q     = b * sum over the rows of gate row q of D * xh
//   dgate_q = w1 * A_q,  dgamma_post = sum_q gate_q * A_q,
//   dgamma_next = sum dy * rh
// (without a post norm xh = x, w1 = 1 and dx = w D).  D is linear in c1, so
// c2 follows from sums that need no c1,
//   S1 = sum dy w2 rh,  S2 = sum w xh (dr + rstd_next dy w2),
//   S3 = sum w xh rh:   c1 = S1 / H,  c2 = (S2 - rstd_next c1 S3) / H,
// and a row takes one round of reductions instead of two.
//
// The gate's and the post norm's gradients share the accumulator A: one
// fp32 sum a column serves both, whatever the number of gate rows.
#include "block_norm.cuh"
#include "common.cuh"
#include "launch.h"
#include "rms_norm.h"

namespace rmsn {
namespace {

// ---------------------------------------------------------------------------
// any alignment, rows of up to 1024 NC columns (backward 512 NC): single
// elements, consecutive lanes on consecutive ones, a thread's columns of the
// row in registers.  Bound by the instructions an element: 8192 x 4097 bf16
// forward 66 us, backward 139 us, where the staged kernels take 50 and 82 for
// 4096 columns.
// ---------------------------------------------------------------------------
// Columns tid, tid + blockDim, ... of a CTA whose threads own up to NC each.
template <int NC, typename F>
__device__ __forceinline__ void each_col(int hidden, F f) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int j = threadIdx.x + k * blockDim.x;
    if (j < hidden) f(k, j);
  }
}

template <typename T, typename TS, int NC>
__global__ void __launch_bounds__(1024) block_fwd_cols(
    const T* __restrict__ x, const TS* __restrict__ res, const T* __restrict__ gamma_post,
    const T* __restrict__ gate, const T* __restrict__ gamma_next, TS* __restrict__ res_out,
    T* __restrict__ y, float* __restrict__ rstd_post, float* __restrict__ rstd_next,
    int64_t rows, int64_t rows_per_gate, int hidden, float a, float b, float eps, float off) {
  __shared__ float red[64];
  pdl_trigger();
  pdl_wait();
  int parity = 0;
  auto sum = [&](float v) {
    v = block_sum(v, red, parity);
    parity ^= 1;
    return v;
  };
  // the root mean square's inverse of v, rescaled where the squares overflow
  auto rstd = [&](const float (&v)[NC]) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) ss = fmaf(v[k], v[k], ss);
    ss = sum(ss);
    if (!isinf(ss)) return rstd_of(ss / (float)hidden, eps);
    float s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const float t = v[k] * kOverflowScale;
      s2 = fmaf(t, t, s2);
    }
    return rstd_rescaled(sum(s2), hidden, eps);
  };
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t at = row * hidden;
    const T* gr = gate == nullptr ? nullptr : gate + row / rows_per_gate * hidden;
    float v[NC], r[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) v[k] = r[k] = 0.f;
    each_col<NC>(hidden, [&](int k, int j) {
      v[k] = Traits<T>::to_f(x[at + j]);
      r[k] = Traits<TS>::to_f(res[at + j]);
    });
    float rs1 = 1.f;
    if (gamma_post != nullptr) {
      rs1 = rstd(v);
      if (threadIdx.x == 0) rstd_post[row] = rs1;
    }
    each_col<NC>(hidden, [&](int k, int j) {
      float w = b;
      if (gr != nullptr) w *= Traits<T>::to_f(gr[j]);
      if (gamma_post != nullptr) w *= Traits<T>::to_f(gamma_post[j]) + off;
      r[k] = fmaf(w, v[k] * rs1, a * r[k]);
      res_out[at + j] = Traits<TS>::from_f(r[k]);
    });
    if (gamma_next == nullptr) continue;
    const float rs2 = rstd(r);
    if (threadIdx.x == 0) rstd_next[row] = rs2;
    each_col<NC>(hidden, [&](int k, int j) {
      y[at + j] = Traits<T>::from_f((r[k] * rs2) * (Traits<T>::to_f(gamma_next[j]) + off));
    });
  }
}

// ---------------------------------------------------------------------------
// any width and alignment: single elements, a row's values read again (from
// L1 / L2) after its reductions
// ---------------------------------------------------------------------------
constexpr int kLoopThreads = 256;

template <typename T, typename TS>
__global__ void __launch_bounds__(kLoopThreads) block_fwd_loop(
    const T* __restrict__ x, const TS* __restrict__ res, const T* __restrict__ gamma_post,
    const T* __restrict__ gate, const T* __restrict__ gamma_next, TS* __restrict__ res_out,
    T* __restrict__ y, float* __restrict__ rstd_post, float* __restrict__ rstd_next,
    int64_t rows, int64_t rows_per_gate, int hidden, float a, float b, float eps, float off) {
  __shared__ float red[64];
  pdl_trigger();
  pdl_wait();
  int parity = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * hidden;
    const TS* sr = res + row * hidden;
    const T* gr = gate == nullptr ? nullptr : gate + row / rows_per_gate * hidden;
    float rs1 = 1.f;
    if (gamma_post != nullptr) {
      float ss = 0.f;
      for (int j = threadIdx.x; j < hidden; j += kLoopThreads) {
        const float v = Traits<T>::to_f(xr[j]);
        ss = fmaf(v, v, ss);
      }
      ss = block_sum(ss, red, parity);
      parity ^= 1;
      rs1 = rstd_of(ss / (float)hidden, eps);
      if (isinf(ss)) {  // see kOverflowScale
        ss = block_sum(scaled_sum_sq(xr, threadIdx.x, kLoopThreads, hidden), red, parity);
        parity ^= 1;
        rs1 = rstd_rescaled(ss, hidden, eps);
      }
      if (threadIdx.x == 0) rstd_post[row] = rs1;
    }
    auto stream = [&](int j) {
      float w = b;
      if (gr != nullptr) w *= Traits<T>::to_f(gr[j]);
      if (gamma_post != nullptr) w *= Traits<T>::to_f(gamma_post[j]) + off;
      return fmaf(w, Traits<T>::to_f(xr[j]) * rs1, a * Traits<TS>::to_f(sr[j]));
    };
    float ss = 0.f;
    for (int j = threadIdx.x; j < hidden; j += kLoopThreads) {
      const float r = stream(j);
      ss = fmaf(r, r, ss);
      res_out[row * hidden + j] = Traits<TS>::from_f(r);
    }
    if (gamma_next == nullptr) continue;
    ss = block_sum(ss, red, parity);
    parity ^= 1;
    float rs2 = rstd_of(ss / (float)hidden, eps);
    if (isinf(ss)) {
      float s2 = 0.f;
      for (int j = threadIdx.x; j < hidden; j += kLoopThreads) {
        const float t = stream(j) * kOverflowScale;
        s2 = fmaf(t, t, s2);
      }
      s2 = block_sum(s2, red, parity);
      parity ^= 1;
      rs2 = rstd_rescaled(s2, hidden, eps);
    }
    if (threadIdx.x == 0) rstd_next[row] = rs2;
    for (int j = threadIdx.x; j < hidden; j += kLoopThreads)
      y[row * hidden + j] =
          Traits<T>::from_f((stream(j) * rs2) * (Traits<T>::to_f(gamma_next[j]) + off));
  }
}

// Sum of three values over the CTA (as block_sum; `red` holds 2 x 32 float4).
__device__ __forceinline__ float3 block_sum3(float a, float b, float c, float4* red, int parity) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nwarps = (blockDim.x + 31) >> 5;
  a = warp_sum(a);
  b = warp_sum(b);
  c = warp_sum(c);
  float4* slot = red + 32 * parity;
  if (lane == 0) slot[warp] = make_float4(a, b, c, 0.f);
  __syncthreads();
  float3 s = make_float3(0.f, 0.f, 0.f);
  for (int w = 0; w < nwarps; ++w) {
    s.x += slot[w].x;
    s.y += slot[w].y;
    s.z += slot[w].z;
  }
  return s;
}

template <typename T, typename TS>
__global__ void __launch_bounds__(kLoopThreads) block_bwd_loop(const BlockBwdParams p) {
  __shared__ float4 red[64];
  pdl_trigger();
  pdl_wait();
  const T* dy = static_cast<const T*>(p.dy);
  const TS* dr = static_cast<const TS*>(p.dr);
  const T* x = static_cast<const T*>(p.x);
  const TS* r = static_cast<const TS*>(p.r);
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gate = static_cast<const T*>(p.gate);
  const T* gamma_next = static_cast<const T*>(p.gamma_next);
  const int hidden = p.hidden;
  const int64_t u = blockIdx.x;
  const int64_t r0 = u * p.rows / gridDim.x, r1 = (u + 1) * p.rows / gridDim.x;
  const bool sums = gamma_post != nullptr || gate != nullptr;
  int parity = 0;
  float* pn = p.p_next + u * hidden;
  float* pp = p.p_post + u * hidden;
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t q = row / p.rows_per_gate;
    const bool seg_first = row == r0 || row == q * p.rows_per_gate;
    const bool seg_last = row + 1 == r1 || row + 1 == (q + 1) * p.rows_per_gate;
    float* pa = p.p_a + (u + q) * hidden;
    const T* gr = gate == nullptr ? nullptr : gate + q * hidden;
    const int64_t at = row * hidden;
    const float rs1 = gamma_post != nullptr ? p.rstd_post[row] : 1.f;
    const float rs2 = gamma_next != nullptr ? p.rstd_next[row] : 0.f;
    auto weight = [&](int j) {
      float w = p.b;
      if (gr != nullptr) w *= Traits<T>::to_f(gr[j]);
      if (gamma_post != nullptr) w *= Traits<T>::to_f(gamma_post[j]) + p.off;
      return w;
    };
    float s1 = 0.f, s2 = 0.f, s3 = 0.f;
    for (int j = threadIdx.x; j < hidden; j += kLoopThreads) {
      const float wx = weight(j) * (Traits<T>::to_f(x[at + j]) * rs1);
      float t = dr != nullptr ? Traits<TS>::to_f(dr[at + j]) : 0.f;
      if (gamma_next != nullptr) {
        const float rh = Traits<TS>::to_f(r[at + j]) * rs2;
        const float g = Traits<T>::to_f(dy[at + j]) * (Traits<T>::to_f(gamma_next[j]) + p.off);
        s1 = fmaf(g, rh, s1);
        s3 = fmaf(wx, rh, s3);
        t = fmaf(rs2, g, t);
      }
      s2 = fmaf(wx, t, s2);
    }
    const float3 s = block_sum3(s1, s2, s3, red, parity);
    parity ^= 1;
    const float c1 = s.x / (float)hidden;
    const float c2 = gamma_post != nullptr ? fmaf(-rs2 * c1, s.z, s.y) / (float)hidden : 0.f;
    for (int j = threadIdx.x; j < hidden; j += kLoopThreads) {
      const float xh = Traits<T>::to_f(x[at + j]) * rs1;
      float d = dr != nullptr ? Traits<TS>::to_f(dr[at + j]) : 0.f;
      if (gamma_next != nullptr) {
        const float rh = Traits<TS>::to_f(r[at + j]) * rs2;
        const float gy = Traits<T>::to_f(dy[at + j]);
        const float g = gy * (Traits<T>::to_f(gamma_next[j]) + p.off);
        d = fmaf(rs2, fmaf(-rh, c1, g), d);
        pn[j] = fmaf(gy, rh, row == r0 ? 0.f : pn[j]);
      }
      static_cast<TS*>(p.dres)[at + j] = Traits<TS>::from_f(p.a * d);
      static_cast<T*>(p.dx)[at + j] = Traits<T>::from_f(rs1 * fmaf(-xh, c2, weight(j) * d));
      if (sums) {
        const float acc = fmaf(p.b * d, xh, seg_first ? 0.f : pa[j]);
        pa[j] = acc;
        if (seg_last && gamma_post != nullptr && p.rows_per_gate < p.rows)
          pp[j] = fmaf(Traits<T>::to_f(gr[j]), acc, q == r0 / p.rows_per_gate ? 0.f : pp[j]);
      }
    }
  }
}

// The backward with a thread's sums over the rows in registers; with HOLD the
// row's values too, without it they are read again (from L1) after the
// reduction.
template <typename T, typename TS, int NC, bool HOLD>
__global__ void __launch_bounds__(512) block_bwd_cols(const BlockBwdParams p) {
  __shared__ float4 red[64];
  pdl_trigger();
  pdl_wait();
  const T* dy = static_cast<const T*>(p.dy);
  const TS* dr = static_cast<const TS*>(p.dr);
  const T* x = static_cast<const T*>(p.x);
  const TS* r = static_cast<const TS*>(p.r);
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gate = static_cast<const T*>(p.gate);
  const T* gamma_next = static_cast<const T*>(p.gamma_next);
  const int hidden = p.hidden;
  const int64_t u = blockIdx.x;
  const int64_t r0 = u * p.rows / gridDim.x, r1 = (u + 1) * p.rows / gridDim.x;
  const bool post = gamma_post != nullptr, next = gamma_next != nullptr;
  constexpr int NH = HOLD ? NC : 1;
  float acc_n[NC], acc_a[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) acc_n[k] = acc_a[k] = 0.f;
  int parity = 0;
  for (int64_t seg0 = r0; seg0 < r1;) {
    const int64_t q = seg0 / p.rows_per_gate;
    const int64_t seg1 = (q + 1) * p.rows_per_gate < r1 ? (q + 1) * p.rows_per_gate : r1;
    auto weight = [&](int j) {
      float w = p.b;
      if (gate != nullptr) w *= Traits<T>::to_f(gate[q * hidden + j]);
      if (post) w *= Traits<T>::to_f(gamma_post[j]) + p.off;
      return w;
    };
    for (int64_t row = seg0; row < seg1; ++row) {
      const int64_t at = row * hidden;
      const float rs1 = post ? p.rstd_post[row] : 1.f, rs2 = next ? p.rstd_next[row] : 0.f;
      // x_hat, r_hat, dy, dr of a column
      auto read = [&](int j) {
        float4 v;
        v.x = Traits<T>::to_f(x[at + j]) * rs1;
        v.y = next ? Traits<TS>::to_f(r[at + j]) * rs2 : 0.f;
        v.z = next ? Traits<T>::to_f(dy[at + j]) : 0.f;
        v.w = dr != nullptr ? Traits<TS>::to_f(dr[at + j]) : 0.f;
        return v;
      };
      float4 held[NH];
      float s1 = 0.f, s2 = 0.f, s3 = 0.f;
      if (HOLD) each_col<NC>(hidden, [&](int k, int j) { held[HOLD ? k : 0] = read(j); });
      each_col<NC>(hidden, [&](int k, int j) {
        const float4 v = HOLD ? held[HOLD ? k : 0] : read(j);
        const float wx = weight(j) * v.x;
        const float g = next ? v.z * (Traits<T>::to_f(gamma_next[j]) + p.off) : 0.f;
        s1 = fmaf(g, v.y, s1);
        s2 = fmaf(wx, fmaf(rs2, g, v.w), s2);
        s3 = fmaf(wx, v.y, s3);
      });
      const float3 s = block_sum3(s1, s2, s3, red, parity);
      parity ^= 1;
      const float c1 = s.x / (float)hidden;
      const float c2 = post ? fmaf(-rs2 * c1, s.z, s.y) / (float)hidden : 0.f;
      each_col<NC>(hidden, [&](int k, int j) {
        const float4 v = HOLD ? held[HOLD ? k : 0] : read(j);
        const float g = next ? v.z * (Traits<T>::to_f(gamma_next[j]) + p.off) : 0.f;
        const float d = fmaf(rs2, fmaf(-v.y, c1, g), v.w);
        acc_n[k] = fmaf(v.z, v.y, acc_n[k]);
        acc_a[k] = fmaf(d, v.x, acc_a[k]);
        static_cast<TS*>(p.dres)[at + j] = Traits<TS>::from_f(p.a * d);
        static_cast<T*>(p.dx)[at + j] = Traits<T>::from_f(rs1 * fmaf(-v.x, c2, weight(j) * d));
      });
    }
    const bool first = q == r0 / p.rows_per_gate, several = p.rows_per_gate < p.rows;
    each_col<NC>(hidden, [&](int k, int j) {
      if (post || gate != nullptr) {
        const float v = p.b * acc_a[k];
        p.p_a[(u + q) * hidden + j] = v;
        if (post && several) {
          float* pp = p.p_post + u * hidden + j;
          *pp = fmaf(Traits<T>::to_f(gate[q * hidden + j]), v, first ? 0.f : *pp);
        }
      }
      if (next && seg1 == r1) p.p_next[u * hidden + j] = acc_n[k];
      acc_a[k] = 0.f;
    });
    seg0 = seg1;
  }
}

// The sums over the partial rows, in a fixed order: 16 lanes, each adding
// every 16th row, then the 16 lane sums in order (as dw_finalize), four
// columns a thread where rows are 16-byte aligned (VEC 4).  Jobs (blockIdx.y):
// the next norm's sums; with one gate row, or none, the sums of A, which give
// dgamma_post = gate A and dgate = w1 A; with several, the post norm's sums,
// and for each gate row those of A over its segments u_first + q ... u_last + q.
constexpr int kSumLanes = 16;

template <typename T, int VEC>
__global__ void __launch_bounds__(32 * kSumLanes) block_bwd_sums(
    const BlockBwdParams p, int units, float* __restrict__ dgamma_post, float* __restrict__ dgate,
    float* __restrict__ dgamma_next) {
  __shared__ float s[kSumLanes][32 * VEC];
  pdl_trigger();
  pdl_wait();
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int hidden = p.hidden;
  const int j0 = (blockIdx.x * 32 + tx) * VEC;
  const bool one = p.rows_per_gate >= p.rows;
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gate = static_cast<const T*>(p.gate);
  const int64_t jobs = 2 + (one || dgate == nullptr ? 0 : p.rows / p.rows_per_gate);
  for (int64_t job = blockIdx.y; job < jobs; job += gridDim.y) {
    const float* src = job == 0 ? p.p_next : one ? p.p_a : p.p_post;
    int64_t n = units, q = 0;
    if (job == 0 ? dgamma_next == nullptr
                 : dgamma_post == nullptr && (dgate == nullptr || (job == 1 && !one)))
      continue;
    if (job >= 2) {
      q = job - 2;
      // unit of row i: the largest u with floor(u R / U) <= i
      const int64_t first = ((q * p.rows_per_gate + 1) * units - 1) / p.rows;
      const int64_t last = ((q + 1) * p.rows_per_gate * units - 1) / p.rows;
      src = p.p_a + (first + q) * hidden;
      n = last - first + 1;
    }
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    if (j0 < hidden) {
#pragma unroll 8
      for (int64_t i = ty; i < n; i += kSumLanes) {
        if constexpr (VEC == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src + i * hidden + j0);
          acc[0] += v.x;
          acc[1] += v.y;
          acc[2] += v.z;
          acc[3] += v.w;
        } else {
          acc[0] += src[i * hidden + j0];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[ty][tx * VEC + k] = acc[k];
    __syncthreads();
    const int c = ty * 32 + tx, j = blockIdx.x * 32 * VEC + c;
    if (c < 32 * VEC && j < hidden) {
      float t = 0.f;
#pragma unroll
      for (int l = 0; l < kSumLanes; ++l) t += s[l][c];
      if (job == 0) {
        dgamma_next[j] = t;
      } else {
        const float w1 = gamma_post != nullptr ? Traits<T>::to_f(gamma_post[j]) + p.off : 1.f;
        const float g = gate != nullptr && one ? Traits<T>::to_f(gate[j]) : 1.f;
        if (job == 1 && dgamma_post != nullptr) dgamma_post[j] = t * g;
        if (dgate != nullptr && (one || job >= 2)) dgate[q * hidden + j] = t * w1;
      }
    }
    __syncthreads();
  }
}

template <typename T> constexpr int code();
template <> constexpr int code<float>() { return RMSN_F32; }
template <> constexpr int code<__nv_bfloat16>() { return RMSN_BF16; }
template <> constexpr int code<__half>() { return RMSN_F16; }

template <typename T, typename TS>
cudaError_t launch_fwd_t(const BlockFwdArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (try_launch_block_fwd_tma(code<T>(), code<TS>(), a, s, &e)) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto go = [&](auto kern, int threads) {
    const int64_t most = (int64_t)sm_count(dev) * max_blocks_per_sm((const void*)kern, threads, 0);
    return launch_kernel(kern, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(threads), 0, s,
                         1, static_cast<const T*>(a.x), static_cast<const TS*>(a.res),
                         static_cast<const T*>(a.gamma_post), static_cast<const T*>(a.gate),
                         static_cast<const T*>(a.gamma_next), static_cast<TS*>(a.res_out),
                         static_cast<T*>(a.y), a.rstd_post, a.rstd_next, a.rows, a.rows_per_gate,
                         a.hidden, a.res_scale, a.branch_scale, a.eps, a.offset ? 1.f : 0.f);
  };
  constexpr int NC = 8;
  if (a.hidden <= 1024 * NC)
    return go(block_fwd_cols<T, TS, NC>, ((a.hidden + NC - 1) / NC + 31) / 32 * 32);
  return go(block_fwd_loop<T, TS>, kLoopThreads);
}

template <typename T, typename TS>
cudaError_t launch_bwd_t(const BlockBwdArgs& a, cudaStream_t s, int* launches) {
  BlockBwdParams p;
  p.dy = a.dy;
  p.dr = a.dr;
  p.x = a.x;
  p.r = a.r;
  p.gamma_post = a.gamma_post;
  p.gate = a.gate;
  p.gamma_next = a.gamma_next;
  p.rstd_post = a.rstd_post;
  p.rstd_next = a.rstd_next;
  p.dx = a.dx;
  p.dres = a.dres;
  p.rows = a.rows;
  p.rows_per_gate = a.rows_per_gate;
  p.hidden = a.hidden;
  p.a = a.res_scale;
  p.b = a.branch_scale;
  p.off = a.offset ? 1.f : 0.f;
  int units = 0;
  cudaError_t e = cudaSuccess;
  if (!try_launch_block_bwd_tma(code<T>(), code<TS>(), a, p, &units, s, &e)) {
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kern, int threads) {
      int64_t most = (int64_t)sm_count(dev) * max_blocks_per_sm((const void*)kern, threads, 0);
      if (most > RMSN_BLOCK_MAX_PARTIALS) most = RMSN_BLOCK_MAX_PARTIALS;
      units = (int)(a.rows < most ? a.rows : most);
      place_partials(a, units, p);
      return launch_kernel(kern, dim3((unsigned)units), dim3(threads), 0, s, 1, p);
    };
    auto threads = [&](int nc) { return ((a.hidden + nc - 1) / nc + 31) / 32 * 32; };
    if (a.hidden <= 512 * 8)
      e = go(block_bwd_cols<T, TS, 8, true>, threads(8));
    else if (a.hidden <= 512 * 16)
      e = go(block_bwd_cols<T, TS, 16, false>, threads(16));
    else
      e = go(block_bwd_loop<T, TS>, kLoopThreads);
  }
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (a.dgamma_post == nullptr && a.dgate == nullptr && a.dgamma_next == nullptr)
    return cudaSuccess;
  const int64_t gates = a.rows / a.rows_per_gate;
  const int64_t jobs = 2 + (a.dgate != nullptr && gates > 1 ? gates : 0);
  const int vec = a.hidden % 4 == 0 ? 4 : 1;  // the partial rows start on 16 bytes
  const dim3 grid((unsigned)((a.hidden + 32 * vec - 1) / (32 * vec)),
                  (unsigned)(jobs < 65535 ? jobs : 65535));
  e = launch_kernel(vec == 4 ? block_bwd_sums<T, 4> : block_bwd_sums<T, 1>, grid,
                    dim3(32, kSumLanes), 0, s, 1, p, units, a.dgamma_post, a.dgate, a.dgamma_next);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace

cudaError_t launch_block_fwd(int dtype, int res_dtype, const BlockFwdArgs& a, cudaStream_t s) {
  if (dtype == RMSN_F32) return launch_fwd_t<float, float>(a, s);
  if (dtype == RMSN_BF16)
    return res_dtype == RMSN_F32 ? launch_fwd_t<__nv_bfloat16, float>(a, s)
                                 : launch_fwd_t<__nv_bfloat16, __nv_bfloat16>(a, s);
  return res_dtype == RMSN_F32 ? launch_fwd_t<__half, float>(a, s)
                               : launch_fwd_t<__half, __half>(a, s);
}

cudaError_t launch_block_bwd(int dtype, int res_dtype, const BlockBwdArgs& a, cudaStream_t s,
                             int* launches) {
  if (dtype == RMSN_F32) return launch_bwd_t<float, float>(a, s, launches);
  if (dtype == RMSN_BF16)
    return res_dtype == RMSN_F32 ? launch_bwd_t<__nv_bfloat16, float>(a, s, launches)
                                 : launch_bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s, launches);
  return res_dtype == RMSN_F32 ? launch_bwd_t<__half, float>(a, s, launches)
                               : launch_bwd_t<__half, __half>(a, s, launches);
}

}  // namespace rmsn
