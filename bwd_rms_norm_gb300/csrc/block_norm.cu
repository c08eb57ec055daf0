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
// any width and alignment: single elements, a row's values read again (from
// L1 / L2) after its reductions, the sums over the rows kept in the partial
// rows.  For what the staged kernels do not take: few or narrow odd rows
// (block_fwd_odd_pays), tensors that do not start on 16 bytes.
// ---------------------------------------------------------------------------

// HELD: columns of a row that stay in a thread's registers.
template <typename T, typename TS, int NT, int HELD>
__global__ void __launch_bounds__(NT) block_fwd_loop(
    const T* __restrict__ x, const TS* __restrict__ res, const T* __restrict__ gamma_post,
    const T* __restrict__ gate, const T* __restrict__ gamma_next, TS* __restrict__ res_out,
    T* __restrict__ y, float* __restrict__ rstd_post, float* __restrict__ rstd_next,
    int64_t rows, int64_t rows_per_gate, int hidden, float a, float b, float eps, float off) {
  __shared__ float red[64];
  pdl_trigger();
  pdl_wait();
  int parity = 0;
  // f(k, j) for the thread's columns that are held, g(j) for its others
  auto each = [&](auto f, auto g) {
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if ((int)threadIdx.x + k * NT < hidden) f(k, (int)threadIdx.x + k * NT);
    for (int j = threadIdx.x + HELD * NT; j < hidden; j += NT) g(j);
  };
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * hidden;
    const TS* sr = res + row * hidden;
    const T* gr = gate == nullptr ? nullptr : gate + row / rows_per_gate * hidden;
    float xv[HELD + 1], r[HELD + 1];
#pragma unroll
    for (int k = 0; k < HELD; ++k) xv[k] = r[k] = 0.f;
    float ss = 0.f;
    each([&](int k, int j) {
      xv[k] = Traits<T>::to_f(xr[j]);
      r[k] = a * Traits<TS>::to_f(sr[j]);
    }, [&](int j) {
      const float v = Traits<T>::to_f(xr[j]);
      ss = fmaf(v, v, ss);
    });
    float rs1 = 1.f;
    if (gamma_post != nullptr) {
#pragma unroll
      for (int k = 0; k < HELD; ++k) ss = fmaf(xv[k], xv[k], ss);
      ss = block_sum(ss, red, parity);
      parity ^= 1;
      rs1 = rstd_of(ss / (float)hidden, eps);
      if (isinf(ss)) {  // see kOverflowScale
        ss = block_sum(scaled_sum_sq(xr, threadIdx.x, NT, hidden), red, parity);
        parity ^= 1;
        rs1 = rstd_rescaled(ss, hidden, eps);
      }
      if (threadIdx.x == 0) rstd_post[row] = rs1;
    }
    auto weight = [&](int j) {
      float w = b;
      if (gr != nullptr) w *= Traits<T>::to_f(gr[j]);
      if (gamma_post != nullptr) w *= Traits<T>::to_f(gamma_post[j]) + off;
      return w;
    };
    auto stream = [&](int j) {
      return fmaf(weight(j), Traits<T>::to_f(xr[j]) * rs1, a * Traits<TS>::to_f(sr[j]));
    };
    ss = 0.f;
    auto put = [&](int j, float v) {
      ss = fmaf(v, v, ss);
      res_out[row * hidden + j] = Traits<TS>::from_f(v);
    };
    each([&](int k, int j) {
      r[k] = fmaf(weight(j), xv[k] * rs1, r[k]);
      put(j, r[k]);
    }, [&](int j) { put(j, stream(j)); });
    if (gamma_next == nullptr) continue;
    ss = block_sum(ss, red, parity);
    parity ^= 1;
    float rs2 = rstd_of(ss / (float)hidden, eps);
    if (isinf(ss)) {
      float s2 = 0.f;
      for (int j = threadIdx.x; j < hidden; j += NT) {
        const float t = stream(j) * kOverflowScale;
        s2 = fmaf(t, t, s2);
      }
      s2 = block_sum(s2, red, parity);
      parity ^= 1;
      rs2 = rstd_rescaled(s2, hidden, eps);
    }
    if (threadIdx.x == 0) rstd_next[row] = rs2;
    auto out = [&](int j, float v) {
      y[row * hidden + j] = Traits<T>::from_f((v * rs2) * (Traits<T>::to_f(gamma_next[j]) + off));
    };
    each([&](int k, int j) { out(j, r[k]); }, [&](int j) { out(j, stream(j)); });
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

template <typename T, typename TS, int NT>
__global__ void __launch_bounds__(NT) block_bwd_loop(const BlockBwdParams p) {
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
    for (int j = threadIdx.x; j < hidden; j += NT) {
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
    for (int j = threadIdx.x; j < hidden; j += NT) {
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

// The sums over the partial rows, in a fixed order: 16 lanes, each adding
// every 16th row, then the 16 lane sums in order (as dw_finalize), four
// columns a thread where rows are 16-byte aligned (VEC 4).  Jobs (blockIdx.y):
// the next norm's sums; with one gate row, or none, the sums of A, which give
// dgamma_post = gate A and dgate = w1 A; with several, the post norm's sums,
// and for each gate row those of A over its segments.  Where gate rows have
// few segments each (`serial`), a lane takes a gate row.
constexpr int kSumLanes = 16;

template <typename T, int VEC>
__global__ void __launch_bounds__(32 * kSumLanes) block_bwd_sums(
    const BlockBwdParams p, int units, bool serial, float* __restrict__ dgamma_post,
    float* __restrict__ dgate, float* __restrict__ dgamma_next) {
  __shared__ float s[kSumLanes][32 * VEC];
  pdl_trigger();
  pdl_wait();
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int hidden = p.hidden;
  const int j0 = (blockIdx.x * 32 + tx) * VEC;
  const bool one = p.rows_per_gate >= p.rows;
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gate = static_cast<const T*>(p.gate);
  const int64_t gates = p.rows / p.rows_per_gate, of = units / p.period;
  const int64_t per = serial ? kSumLanes : 1;  // gate rows a job
  const int64_t jobs = 2 + (one || dgate == nullptr ? 0 : (gates + per - 1) / per);
  auto weight = [&](int j) {
    return gamma_post != nullptr ? Traits<T>::to_f(gamma_post[j]) + p.off : 1.f;
  };
  for (int64_t job = blockIdx.y; job < jobs; job += gridDim.y) {
    if (job == 0 ? dgamma_next == nullptr
                 : dgamma_post == nullptr && (dgate == nullptr || (job == 1 && !one)))
      continue;
    const bool alone = serial && job >= 2;  // a lane a gate row
    const int64_t q = (job - 2) * per + (alone ? ty : 0);
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    auto add = [&](const float* src, int64_t n) {
      if (j0 >= hidden) return;
#pragma unroll 8
      for (int64_t i = alone ? 0 : ty; i < n; i += alone ? 1 : kSumLanes) {
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
    };
    if (job < 2) {
      add(job == 0 ? p.p_next : one ? p.p_a : p.p_post, units);
    } else if (q < gates) {
      // class c's rows are c + P i; its unit of i is the largest u with
      // floor(u n / U) <= i, n of its rows over U units
      for (int c = 0; c < p.period; ++c) {
        const int64_t n = (p.rows - c + p.period - 1) / p.period;
        auto from = [&](int64_t row) { return row <= c ? 0 : (row - c + p.period - 1) / p.period; };
        const int64_t lo = from(q * p.rows_per_gate), hi = from((q + 1) * p.rows_per_gate);
        if (lo >= hi) continue;
        const int64_t first = ((lo + 1) * of - 1) / n, last = (hi * of - 1) / n;
        add(p.p_a + (c * (of + gates - 1) + first + q) * hidden, last - first + 1);
      }
    }
    if (alone) {
      if (q < gates && j0 < hidden)
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] *= weight(j0 + k);
      if (q < gates && j0 < hidden) {
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(dgate + q * hidden + j0) =
              make_float4(acc[0], acc[1], acc[2], acc[3]);
        else
          dgate[q * hidden + j0] = acc[0];
      }
      continue;
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
        const float g = gate != nullptr && one ? Traits<T>::to_f(gate[j]) : 1.f;
        if (job == 1 && dgamma_post != nullptr) dgamma_post[j] = t * g;
        if (dgate != nullptr && (one || job >= 2)) dgate[(one ? 0 : q) * hidden + j] = t * weight(j);
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
  const int sms = sm_count(dev);
  auto go = [&](auto kern, int threads) {
    const int64_t most = (int64_t)sms * max_blocks_per_sm((const void*)kern, threads, 0);
    return launch_kernel(kern, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(threads), 0, s,
                         1, static_cast<const T*>(a.x), static_cast<const TS*>(a.res),
                         static_cast<const T*>(a.gamma_post), static_cast<const T*>(a.gate),
                         static_cast<const T*>(a.gamma_next), static_cast<TS*>(a.res_out),
                         static_cast<T*>(a.y), a.rstd_post, a.rstd_next, a.rows, a.rows_per_gate,
                         a.hidden, a.res_scale, a.branch_scale, a.eps, a.offset ? 1.f : 0.f);
  };
  // bf16, 128 / 256 / 1024 threads with nothing held: 64 x 1001 4.3, 3.7, 3.4
  // us; 64 x 8191 13.5, 11.1, 6.5; 4096 x 257 9.8, 15.4, 65; 4096 x 4097 53, 49,
  // 128.  Held / not: 1024 x 257 3.8 / 4.7, 1024 x 1001 5.0 / 7.6, 4096 x 1500
  // 29 / 32, but 4096 x 33 9.9 / 7.2 and 4096 x 4097 58 / 47.
  if (a.rows <= sms && a.hidden > 512) return go(block_fwd_loop<T, TS, 1024, 0>, 1024);
  if (a.hidden <= 128) return go(block_fwd_loop<T, TS, 128, 0>, 128);
  if (a.hidden <= 1024) return go(block_fwd_loop<T, TS, 128, 8>, 128);
  if (a.hidden <= 2048) return go(block_fwd_loop<T, TS, 256, 8>, 256);
  return go(block_fwd_loop<T, TS, 256, 0>, 256);
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
  p.period = 1;
  int units = 0;
  cudaError_t e = cudaSuccess;
  const bool odd = a.edge_ok && block_bwd_odd_pays(a.rows, a.rows_per_gate, a.hidden);
  if (!(a.vec_ok && try_launch_block_bwd_tma(code<T>(), code<TS>(), a, p, &units, s, &e)) &&
      !(odd && try_launch_block_bwd_odd(code<T>(), code<TS>(), a, p, &units, s, &e))) {
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
    // bf16, 128 / 512 threads: 64 x 257 5.9, 5.9 us; 4096 x 257 27, 54; 64 x
    // 1001 10.5, 7.1; 64 x 4097 29, 16; 1024 x 4097 with 64 gate rows 166, 60
    e = a.hidden <= 512 ? go(block_bwd_loop<T, TS, 128>, 128) : go(block_bwd_loop<T, TS, 512>, 512);
  }
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (a.dgamma_post == nullptr && a.dgate == nullptr && a.dgamma_next == nullptr)
    return cudaSuccess;
  const int64_t gates = a.rows / a.rows_per_gate;
  const int vec = a.hidden % 4 == 0 && reinterpret_cast<uintptr_t>(a.dgate) % 16 == 0 ? 4 : 1;
  // bf16 4096 x 4096, by lanes / serially: 4096 gate rows 1244 / 165 us, 64 62 /
  // 46; 4096 x 1024 with 16 gate rows 22.5 / 23.4
  const bool serial = 4 * gates >= units;
  const int64_t jobs = 2 + (a.dgate == nullptr || gates == 1 ? 0
                            : serial ? (gates + kSumLanes - 1) / kSumLanes : gates);
  const dim3 grid((unsigned)((a.hidden + 32 * vec - 1) / (32 * vec)),
                  (unsigned)(jobs < 65535 ? jobs : 65535));
  e = launch_kernel(vec == 4 ? block_bwd_sums<T, 4> : block_bwd_sums<T, 1>, grid,
                    dim3(32, kSumLanes), 0, s, 1, p, units, serial, a.dgamma_post, a.dgate,
                    a.dgamma_next);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace

cudaError_t read_block_wait_timeouts(unsigned int* out) {
  unsigned int n[3] = {0, 0, 0};
  cudaError_t e = read_block_fwd_wait_timeouts(&n[0]);
  if (e == cudaSuccess) e = read_block_bwd_tma_wait_timeouts(&n[1]);
  if (e == cudaSuccess) e = read_block_bwd_odd_wait_timeouts(&n[2]);
  *out = n[0] + n[1] + n[2];
  return e;
}

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
