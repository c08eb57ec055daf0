// Head norm and rotation: the RMS norms of queries and keys over each head's
// row and the rotation by the token's position, one pass over both.
#include <math.h>

#include "rotary.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHalf = RMSN_ROTARY_MAX_DIM / 2;

// The columns of pair i.
__device__ __forceinline__ int2 columns(const RotaryParams& p, int i) {
  return p.interleaved ? make_int2(2 * i, 2 * i + 1) : make_int2(i, i + p.half);
}

// rstd of a row of which this lane has the columns lane, lane + 32, ...
template <typename T>
__device__ __forceinline__ float row_rstd(const T* v, int lane, int n, float eps) {
  float s = 0.f;
  for (int j = lane; j < n; j += 32) {
    const float f = Traits<T>::to_f(v[j]);
    s = fmaf(f, f, s);
  }
  s = warp_sum(s);
  if (isinf(s)) return rstd_rescaled(warp_sum(scaled_sum_sq(v, lane, 32, n)), n, eps);
  return rstd_of(s / (float)n, eps);
}

// A warp a head's row, an element at a time: rows of any width and alignment.
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_fwd_any(const RotaryParams p) {
  __shared__ uint64_t turns[kMaxHalf];
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < p.half; i += kThreads) turns[i] = fixed_turns(p, i);
  __syncthreads();
  const int lane = threadIdx.x & 31, heads = p.side[0].heads + p.side[1].heads;
  const int64_t rows = (int64_t)p.all * heads;
  for (int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * kWarps) {
    const int token = (int)(r / heads), b = token / p.tokens, t = token % p.tokens;
    int h = (int)(r % heads);
    const bool keys = h >= p.side[0].heads;
    const RotarySide& s = p.side[keys];
    if (keys) h -= p.side[0].heads;
    const T* v = reinterpret_cast<const T*>(s.in.p) + row_at(s.in, b, t, h);
    T* y = reinterpret_cast<T*>(s.out.p) + row_at(s.out, b, t, h);
    const T* gamma = static_cast<const T*>(s.gamma);
    const float rs = row_rstd(v, lane, p.dim, p.eps);
    if (s.rstd && lane == 0) s.rstd[(int64_t)token * s.heads + h] = rs;
    auto u = [&](int j) {
      return Traits<T>::to_f(v[j]) * rs * (Traits<T>::to_f(gamma[j]) + p.off);
    };
    const int64_t pos = position_of(p, b, t);
    for (int i = lane; i < p.half; i += 32) {
      const float2 cs = turn_of(turns[i], pos);
      const int2 c = columns(p, i);
      const float a = u(c.x), d = u(c.y);
      y[c.x] = Traits<T>::from_f(a * cs.x - d * cs.y);
      y[c.y] = Traits<T>::from_f(d * cs.x + a * cs.y);
    }
    for (int j = 2 * p.half + lane; j < p.dim; j += 32) y[j] = Traits<T>::from_f(u(j));
  }
}

// A CTA's sums of du vh, which its warps have in `acc` [kWarps][dim], as its
// partial row, or in the first of acc's.
__device__ __forceinline__ void sum_warps(float* acc, float* partial, int dim) {
  __syncthreads();
  for (int j = threadIdx.x; j < dim; j += kThreads) {
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += acc[w * dim + j];
    (partial ? partial : acc)[j] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_bwd_any(const RotaryParams p) {
  __shared__ uint64_t turns[kMaxHalf];
  extern __shared__ float acc[];
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < p.half; i += kThreads) turns[i] = fixed_turns(p, i);
  for (int j = threadIdx.x; j < kWarps * p.dim; j += kThreads) acc[j] = 0.f;
  __syncthreads();
  const bool keys = (int)blockIdx.x >= p.side[0].ctas;
  const RotarySide& s = p.side[keys];
  const int cta = blockIdx.x - (keys ? p.side[0].ctas : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = (int64_t)p.all * s.heads;
  const T* gamma = static_cast<const T*>(s.gamma);
  float* mine = acc + warp * p.dim;
  for (int64_t r = (int64_t)cta * kWarps + warp; r < rows; r += (int64_t)s.ctas * kWarps) {
    const int token = (int)(r / s.heads), b = token / p.tokens, t = token % p.tokens;
    const int h = (int)(r % s.heads);
    const T* v = reinterpret_cast<const T*>(s.in.p) + row_at(s.in, b, t, h);
    const T* dy = reinterpret_cast<const T*>(s.dy.p) + row_at(s.dy, b, t, h);
    T* dv = reinterpret_cast<T*>(s.out.p) + row_at(s.out, b, t, h);
    const float rs = s.rstd[r];
    const int64_t pos = position_of(p, b, t);
    auto gain = [&](int j) { return Traits<T>::to_f(gamma[j]) + p.off; };
    auto vh = [&](int j) { return Traits<T>::to_f(v[j]) * rs; };
    auto du = [&](int i, int2 c) {  // dy's pair rotated back
      const float2 cs = turn_of(turns[i], pos);
      const float a = Traits<T>::to_f(dy[c.x]), d = Traits<T>::to_f(dy[c.y]);
      return make_float2(a * cs.x + d * cs.y, d * cs.x - a * cs.y);
    };
    float dot = 0.f;
    for (int i = lane; i < p.half; i += 32) {
      const int2 c = columns(p, i);
      const float2 d = du(i, c);
      const float m = d.x * vh(c.x), n = d.y * vh(c.y);
      mine[c.x] += m;
      mine[c.y] += n;
      dot = fmaf(m, gain(c.x), fmaf(n, gain(c.y), dot));
    }
    for (int j = 2 * p.half + lane; j < p.dim; j += 32) {
      const float m = Traits<T>::to_f(dy[j]) * vh(j);
      mine[j] += m;
      dot = fmaf(m, gain(j), dot);
    }
    const float mean = warp_sum(dot) / (float)p.dim;
    auto out = [&](int j, float d) {
      return Traits<T>::from_f(rs * (d * gain(j) - vh(j) * mean));
    };
    for (int i = lane; i < p.half; i += 32) {
      const int2 c = columns(p, i);
      const float2 d = du(i, c);
      const T a = out(c.x, d.x), e = out(c.y, d.y);  // dv may be v or dy
      dv[c.x] = a;
      dv[c.y] = e;
    }
    for (int j = 2 * p.half + lane; j < p.dim; j += 32)
      dv[j] = out(j, Traits<T>::to_f(dy[j]));
  }
  sum_warps(acc, p.direct ? nullptr : s.partial + (int64_t)cta * p.dim, p.dim);
  if (p.direct) add_cluster(acc, s.dgamma, p.dim, s.ctas);
}

// dgamma[j] = the sum of a side's partial rows: 32 lanes a column, each over
// every 32nd row, then the lanes in order.
constexpr int kSumLanes = 32;
__global__ void __launch_bounds__(32 * kSumLanes) rotary_sums(const RotaryParams p) {
  __shared__ float part[kSumLanes][33];
  pdl_wait();
  pdl_trigger();
  const RotarySide& s = p.side[blockIdx.y];
  const int j = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (j < p.dim)
#pragma unroll 4
    for (int r = threadIdx.y; r < s.ctas; r += kSumLanes) v += s.partial[(int64_t)r * p.dim + j];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && j < p.dim) {
    v = 0.f;
    for (int k = 0; k < kSumLanes; ++k) v += part[k][threadIdx.x];
    s.dgamma[j] = v;
  }
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

template <typename T>
cudaError_t launch_fwd_t(int dtype, const RotaryParams& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaSuccess;
  if (try_launch_rotary_fwd_vec(dtype, p, s, &e)) return e;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kern = rotary_fwd_any<T>;
  const int64_t rows = (int64_t)p.all * (p.side[0].heads + p.side[1].heads);
  const int64_t most = (int64_t)sm_count(dev) * max_blocks_per_sm((const void*)kern, kThreads, 0);
  return launch_kernel(kern, dim3((unsigned)least((rows + kWarps - 1) / kWarps, most)),
                       dim3(kThreads), 0, s, 1, p);
}

template <typename T>
cudaError_t launch_bwd_t(int dtype, RotaryParams& p, cudaStream_t s, int* launches) {
  int dev = 0;
  cudaError_t e = cudaSuccess;
  if (!try_launch_rotary_bwd_vec(dtype, p, s, &e)) {
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    constexpr auto kern = rotary_bwd_any<T>;
    const size_t smem = (size_t)kWarps * p.dim * sizeof(float);
    e = allow_launch<kern>(dev, kWarps * RMSN_ROTARY_MAX_DIM * sizeof(float));
    if (e != cudaSuccess) return e;
    const int sms = sm_count(dev);
    const int64_t most = (int64_t)sms * max_blocks_per_sm((const void*)kern, kThreads, smem);
    const int cluster =
        place_ctas(p, most, kWarps, sms, p.side[0].heads, p.side[1].heads);
    e = launch_kernel(kern, dim3((unsigned)(p.side[0].ctas + p.side[1].ctas)), dim3(kThreads),
                      smem, s, cluster, p);
  }
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (p.direct) return e;
  e = launch_kernel(rotary_sums, dim3((unsigned)((p.dim + 31) / 32), p.side[1].heads ? 2 : 1),
                    dim3(32, kSumLanes), 0, s, 1, p);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------

// An argument's memory: runs of `run` bytes at steps of its own, empty where
// it is not given.
struct Block {
  uintptr_t p = 0;
  int64_t size[3] = {1, 1, 1}, step[3] = {0, 0, 0}, run = 0;
  Block() = default;
  Block(const void* at, int64_t bytes) : p(reinterpret_cast<uintptr_t>(at)), run(at ? bytes : 0) {}
  Block(const rmsn_heads* v, int64_t batch, int64_t tokens, int64_t heads, int64_t dim, int bytes) {
    if (!v) return;
    p = reinterpret_cast<uintptr_t>(v->data);
    run = dim * bytes;
    const int64_t n[3] = {batch, tokens, heads};
    const int64_t st[3] = {v->batch_stride, v->token_stride, v->head_stride};
    for (int i = 0; i < 3; ++i) size[i] = n[i], step[i] = n[i] > 1 ? st[i] * bytes : 0;
  }
  int64_t extent() const {  // bytes from the first to behind the last
    int64_t n = run;
    for (int i = 0; i < 3; ++i) n += (size[i] - 1) * step[i];
    return n;
  }
  bool operator==(const Block& o) const {
    bool same = p == o.p && run == o.run;
    for (int i = 0; i < 3; ++i) same = same && size[i] == o.size[i] && step[i] == o.step[i];
    return same;
  }
};

// How far apart two arguments' runs can be: d bytes and lo to hi times each of `n`
// steps, the largest first.
struct Distances {
  int n = 0;
  int64_t step[6], lo[6], hi[6];
  void add(int64_t s, int64_t from, int64_t to) {
    if (s == 0 || from == to) return;
    int at = 0;
    while (at < n && step[at] > s) ++at;
    if (at == n || step[at] != s) {
      for (int i = n++; i > at; --i) step[i] = step[i - 1], lo[i] = lo[i - 1], hi[i] = hi[i - 1];
      step[at] = s, lo[at] = hi[at] = 0;
    }
    lo[at] += from, hi[at] += to;
  }
  // Whether one is above -below and under `above`; taken to be so where `looks` run out.
  bool between(int64_t d, int64_t below, int64_t above, int* looks, int at = 0) const {
    if (at == n) return -below < d && d < above;
    if (--*looks < 0) return true;
    int64_t least = d, most = d;  // with what the smaller steps add
    for (int i = at + 1; i < n; ++i) least += lo[i] * step[i], most += hi[i] * step[i];
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    int64_t j = floor_div(-below - most, step[at]) + 1, end = -floor_div(least - above, step[at]);
    if (j < lo[at]) j = lo[at];
    if (end > hi[at] + 1) end = hi[at] + 1;
    if (at + 1 == n) return j < end;
    for (; j < end; ++j)
      if (between(d + j * step[at], below, above, looks, at + 1)) return true;
    return false;
  }
};

// Whether two arguments share a byte.  Arguments whose steps lie within one another,
// as in any slice or transpose of contiguous memory, take a few looks.
bool meet(const Block& a, const Block& b) {
  if (a.run == 0 || b.run == 0) return false;
  if (a.p + (uintptr_t)a.extent() <= b.p || b.p + (uintptr_t)b.extent() <= a.p) return false;
  Distances way;
  for (int i = 0; i < 3; ++i) {
    way.add(a.step[i], 1 - a.size[i], 0);
    way.add(b.step[i], 0, b.size[i] - 1);
  }
  int looks = 4096;
  return way.between((int64_t)(b.p - a.p), b.run, a.run, &looks);
}

// Whether every element of an output has a place of its own.
bool own_places(const Block& a) {
  bool used[3] = {false, false, false};
  int64_t reach = a.run;
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && a.size[i] > 1 && (at < 0 || a.step[i] < a.step[at])) at = i;
    if (at < 0) break;
    used[at] = true;
    if (a.step[at] < reach) return false;
    reach += (a.size[at] - 1) * a.step[at];
  }
  return true;
}

struct Sizes {
  int64_t batch, tokens, heads[2], dim, rotary;
};

int check_sizes(const Sizes& z, int interleaved, int offset, int dtype) {
  if (dtype != RMSN_F32 && dtype != RMSN_BF16 && dtype != RMSN_F16) return RMSN_ERR_DTYPE;
  if (z.dim < 1 || z.dim > RMSN_ROTARY_MAX_DIM || z.rotary < 0 || z.rotary > z.dim || z.rotary % 2)
    return RMSN_ERR_SHAPE;
  if (z.batch < 0 || z.tokens < 0 || z.heads[0] < 1 || z.heads[1] < 0) return RMSN_ERR_SHAPE;
  for (int64_t n : {z.batch, z.tokens, z.heads[0], z.heads[1]})
    if (n > RMSN_MAX_ROWS) return RMSN_ERR_SHAPE;
  if (z.batch > 0 && z.tokens > RMSN_MAX_ROWS / z.batch) return RMSN_ERR_SHAPE;
  const int64_t all = z.batch * z.tokens, most = z.heads[0] + z.heads[1];
  if (all > 0 && most > RMSN_MAX_ROWS / all) return RMSN_ERR_SHAPE;
  if ((offset != 0 && offset != 1) || (interleaved != 0 && interleaved != 1)) return RMSN_ERR_ARG;
  return RMSN_OK;
}

// A tensor of heads: its strides, its alignment; *vec: rows of 16-byte vectors.
int check_view(const rmsn_heads* v, const Sizes& z, int64_t heads, int bytes, bool* vec) {
  if (!v || !v->data) return RMSN_ERR_NULL;
  if ((uintptr_t)v->data % bytes != 0) return RMSN_ERR_ALIGN;
  const int64_t n[3] = {z.batch, z.tokens, heads};
  const int64_t st[3] = {v->batch_stride, v->token_stride, v->head_stride};
  for (int i = 0; i < 3; ++i) {
    if (n[i] < 2) continue;
    if (st[i] < 0 || st[i] > ((int64_t)1 << 58) / n[i]) return RMSN_ERR_SHAPE;
    if (st[i] * bytes % 16 != 0) *vec = false;
  }
  if ((uintptr_t)v->data % 16 != 0 || z.dim * bytes % 16 != 0) *vec = false;
  return RMSN_OK;
}

HeadView view_of(const rmsn_heads* v, const Sizes& z, int64_t heads) {
  HeadView h{};
  if (!v) return h;
  h.p = static_cast<char*>(v->data);
  h.sb = z.batch > 1 ? v->batch_stride : 0;
  h.st = z.tokens > 1 ? v->token_stride : 0;
  h.sh = heads > 1 ? v->head_stride : 0;
  return h;
}

RotaryParams params_of(const Sizes& z, const void* inv_freq, int inv_freq_64,
                       const void* positions, int positions_64, int64_t positions_batch_stride,
                       int interleaved, int offset) {
  RotaryParams p{};
  p.inv_freq = inv_freq;
  p.freq64 = inv_freq_64 != 0;
  p.positions = positions;
  p.pos64 = positions_64 != 0;
  p.pos_stride = z.batch > 1 ? positions_batch_stride : 0;
  p.all = (int)(z.batch * z.tokens);
  p.tokens = (int)z.tokens;
  p.dim = (int)z.dim;
  p.half = (int)(z.rotary / 2);
  p.interleaved = interleaved;
  p.off = offset ? 1.f : 0.f;
  return p;
}

// The memory of what every call reads beside the tensors of heads.
int check_shared(const Sizes& z, const void* q_gamma, const void* k_gamma, const void* inv_freq,
                 int inv_freq_64, const void* positions, int positions_64,
                 int64_t positions_batch_stride, int bytes, Block (&ins)[4]) {
  if (!q_gamma || (z.heads[1] > 0 && !k_gamma) || (z.rotary > 0 && !inv_freq)) return RMSN_ERR_NULL;
  if ((inv_freq_64 != 0 && inv_freq_64 != 1) || (positions_64 != 0 && positions_64 != 1))
    return RMSN_ERR_ARG;
  const int fb = inv_freq_64 ? 8 : 4, pb = positions_64 ? 8 : 4;
  const int64_t pos_step = z.batch > 1 ? positions_batch_stride : 0;
  if (pos_step < 0 || pos_step > ((int64_t)1 << 58) / (z.batch > 0 ? z.batch : 1))
    return RMSN_ERR_SHAPE;
  if ((uintptr_t)q_gamma % bytes != 0 || (uintptr_t)k_gamma % bytes != 0 ||
      (uintptr_t)inv_freq % fb != 0 || (uintptr_t)positions % pb != 0)
    return RMSN_ERR_ALIGN;
  ins[0] = Block(q_gamma, z.dim * bytes);
  ins[1] = Block(z.heads[1] > 0 ? k_gamma : nullptr, z.dim * bytes);
  ins[2] = Block(z.rotary > 0 ? inv_freq : nullptr, z.rotary / 2 * fb);
  ins[3] = Block(positions, ((z.batch - 1) * pos_step + z.tokens) * pb);
  return RMSN_OK;
}

}  // namespace
}  // namespace rmsn

extern "C" {

int rms_norm_rotary_fwd(const rmsn_heads* q, const rmsn_heads* k, const void* q_gamma,
                        const void* k_gamma, const void* inv_freq, int inv_freq_64,
                        const void* positions, int positions_64, int64_t positions_batch_stride,
                        const rmsn_heads* q_out, const rmsn_heads* k_out, float* rstd_q,
                        float* rstd_k, int64_t batch, int64_t tokens, int64_t q_heads,
                        int64_t k_heads, int64_t head_dim, int64_t rotary_dim, int interleaved,
                        float eps, int offset, int dtype, void* stream) {
  using namespace rmsn;
  const Sizes z = {batch, tokens, {q_heads, k_heads}, head_dim, rotary_dim};
  int st = check_sizes(z, interleaved, offset, dtype);
  if (st != RMSN_OK) return st;
  if (!(eps >= 0.f) || isinf(eps)) return RMSN_ERR_EPS;
  begin_call();
  if (batch * tokens == 0) return RMSN_OK;
  const int bytes = dtype == RMSN_F32 ? 4 : 2;
  Block ins[4];
  st = check_shared(z, q_gamma, k_gamma, inv_freq, inv_freq_64, positions, positions_64,
                    positions_batch_stride, bytes, ins);
  if (st != RMSN_OK) return st;
  RotaryParams p = params_of(z, inv_freq, inv_freq_64, positions, positions_64,
                             positions_batch_stride, interleaved, offset);
  p.eps = eps;
  p.vec_ok = true;
  const rmsn_heads* in[2] = {q, k};
  const rmsn_heads* out[2] = {q_out, k_out};
  float* rstd[2] = {rstd_q, rstd_k};
  Block from[2], to[4];
  for (int i = 0; i < 2; ++i) {
    const int64_t h = z.heads[i];
    if (h == 0) continue;
    st = check_view(in[i], z, h, bytes, &p.vec_ok);
    if (st == RMSN_OK) st = check_view(out[i], z, h, bytes, &p.vec_ok);
    if (st != RMSN_OK) return st;
    if ((uintptr_t)rstd[i] % sizeof(float) != 0) return RMSN_ERR_ALIGN;
    from[i] = Block(in[i], batch, tokens, h, head_dim, bytes);
    to[i] = Block(out[i], batch, tokens, h, head_dim, bytes);
    to[2 + i] = Block(rstd[i], batch * tokens * h * (int64_t)sizeof(float));
    if (!own_places(to[i])) return RMSN_ERR_ARG;
    p.side[i] = RotarySide{view_of(in[i], z, h), view_of(out[i], z, h), HeadView{},
                           i == 0 ? q_gamma : k_gamma, rstd[i], nullptr, nullptr, (int)h, 0};
    if ((uintptr_t)p.side[i].gamma % 16 != 0) p.vec_ok = false;
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 2; ++j)
      if (!(i == j && to[i] == from[j]) && meet(to[i], from[j])) return RMSN_ERR_ARG;
    for (const Block& b : ins)
      if (meet(to[i], b)) return RMSN_ERR_ARG;
    for (int j = i + 1; j < 4; ++j)
      if (meet(to[i], to[j])) return RMSN_ERR_ARG;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == RMSN_F32    ? launch_fwd_t<float>(dtype, p, cs)
                        : dtype == RMSN_BF16 ? launch_fwd_t<__nv_bfloat16>(dtype, p, cs)
                                             : launch_fwd_t<__half>(dtype, p, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(1);
  return RMSN_OK;
}

size_t rms_norm_rotary_bwd_workspace_size(int64_t batch, int64_t tokens, int64_t q_heads,
                                          int64_t k_heads, int64_t head_dim) {
  using namespace rmsn;
  const Sizes z = {batch, tokens, {q_heads, k_heads}, head_dim, 0};
  if (check_sizes(z, 0, 0, RMSN_F32) != RMSN_OK || batch * tokens == 0 ||
      few_rows(batch * tokens, q_heads, k_heads, head_dim))
    return 0;
  return (size_t)least(batch * tokens * (q_heads + k_heads), RMSN_ROTARY_MAX_PARTIALS) *
         (size_t)head_dim * sizeof(float);
}

int rms_norm_rotary_bwd(const rmsn_heads* dq_out, const rmsn_heads* dk_out, const rmsn_heads* q,
                        const rmsn_heads* k, const void* q_gamma, const void* k_gamma,
                        const float* rstd_q, const float* rstd_k, const void* inv_freq,
                        int inv_freq_64, const void* positions, int positions_64,
                        int64_t positions_batch_stride, const rmsn_heads* dq, const rmsn_heads* dk,
                        float* dq_gamma, float* dk_gamma, int64_t batch, int64_t tokens,
                        int64_t q_heads, int64_t k_heads, int64_t head_dim, int64_t rotary_dim,
                        int interleaved, int offset, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  using namespace rmsn;
  const Sizes z = {batch, tokens, {q_heads, k_heads}, head_dim, rotary_dim};
  int st = check_sizes(z, interleaved, offset, dtype);
  if (st != RMSN_OK) return st;
  begin_call();
  if (!dq_gamma || (k_heads > 0 && !dk_gamma)) return RMSN_ERR_NULL;
  if ((uintptr_t)dq_gamma % sizeof(float) != 0 || (uintptr_t)dk_gamma % sizeof(float) != 0)
    return RMSN_ERR_ALIGN;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t sums = head_dim * (int64_t)sizeof(float);
  if (batch * tokens == 0) {
    cudaError_t e = cudaMemsetAsync(dq_gamma, 0, (size_t)sums, cs);
    if (e == cudaSuccess && k_heads > 0) e = cudaMemsetAsync(dk_gamma, 0, (size_t)sums, cs);
    return e == cudaSuccess ? RMSN_OK : cuda_fail(e);
  }
  const int bytes = dtype == RMSN_F32 ? 4 : 2;
  Block ins[4];
  st = check_shared(z, q_gamma, k_gamma, inv_freq, inv_freq_64, positions, positions_64,
                    positions_batch_stride, bytes, ins);
  if (st != RMSN_OK) return st;
  RotaryParams p = params_of(z, inv_freq, inv_freq_64, positions, positions_64,
                             positions_batch_stride, interleaved, offset);
  p.vec_ok = true;
  const rmsn_heads *up[2] = {dq_out, dk_out}, *in[2] = {q, k}, *out[2] = {dq, dk};
  const float* rstd[2] = {rstd_q, rstd_k};
  float* dgamma[2] = {dq_gamma, dk_gamma};
  Block from[2], grad[2], stat[2], to[5];
  for (int i = 0; i < 2; ++i) {
    const int64_t h = z.heads[i];
    if (h == 0) continue;
    for (const rmsn_heads* v : {up[i], in[i], out[i]}) {
      st = check_view(v, z, h, bytes, &p.vec_ok);
      if (st != RMSN_OK) return st;
    }
    if (!rstd[i]) return RMSN_ERR_NULL;
    if ((uintptr_t)rstd[i] % sizeof(float) != 0) return RMSN_ERR_ALIGN;
    from[i] = Block(in[i], batch, tokens, h, head_dim, bytes);
    grad[i] = Block(up[i], batch, tokens, h, head_dim, bytes);
    stat[i] = Block(rstd[i], batch * tokens * h * (int64_t)sizeof(float));
    to[i] = Block(out[i], batch, tokens, h, head_dim, bytes);
    to[2 + i] = Block(dgamma[i], sums);
    if (!own_places(to[i])) return RMSN_ERR_ARG;
    p.side[i] = RotarySide{view_of(in[i], z, h), view_of(out[i], z, h), view_of(up[i], z, h),
                           i == 0 ? q_gamma : k_gamma, const_cast<float*>(rstd[i]), dgamma[i],
                           nullptr, (int)h, 0};
    if ((uintptr_t)p.side[i].gamma % 16 != 0) p.vec_ok = false;
  }
  const size_t need =
      rms_norm_rotary_bwd_workspace_size(batch, tokens, q_heads, k_heads, head_dim);
  p.direct = need == 0;
  if (need > 0 && !workspace) return RMSN_ERR_NULL;
  if ((uintptr_t)workspace % 16 != 0) return RMSN_ERR_ALIGN;
  if (workspace_bytes < need) return RMSN_ERR_WORKSPACE;
  to[4] = Block(need > 0 ? workspace : nullptr, (int64_t)workspace_bytes);
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 2; ++j) {
      if (!(i == j && to[i] == from[j]) && meet(to[i], from[j])) return RMSN_ERR_ARG;
      if (!(i == j && to[i] == grad[j]) && meet(to[i], grad[j])) return RMSN_ERR_ARG;
      if (meet(to[i], stat[j])) return RMSN_ERR_ARG;
    }
    for (const Block& b : ins)
      if (meet(to[i], b)) return RMSN_ERR_ARG;
    for (int j = i + 1; j < 5; ++j)
      if (meet(to[i], to[j])) return RMSN_ERR_ARG;
  }
  p.side[0].partial = static_cast<float*>(workspace);
  int launches = 0;
  const cudaError_t e = dtype == RMSN_F32    ? launch_bwd_t<float>(dtype, p, cs, &launches)
                        : dtype == RMSN_BF16 ? launch_bwd_t<__nv_bfloat16>(dtype, p, cs, &launches)
                                             : launch_bwd_t<__half>(dtype, p, cs, &launches);
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(launches);
  return RMSN_OK;
}

}  // extern "C"
