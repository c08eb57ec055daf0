// The 2-norm over a list of gradients, and the list scaled down to a largest
// norm, for sm_103a.
//
//   norm   = sqrt(sum over every tensor and element of g^2)
//   factor = min(1, max_norm / (norm + eps)), 1 where an element is not finite
//   out_i  = round(g_i * factor)
//
// Two launches.  grad_squares reads the list once and leaves one sum a CTA;
// grad_scale (or grad_norm_final, where only the norm is wanted) adds those
// sums, every CTA in the same order, and writes the scaled list.
//
// Bound by HBM bandwidth: the list is read for the norm, and read again and
// written for the scaling.  The list is cut into chunks of at most
// kChunkElems elements of one tensor, which the CTAs take round-robin;
// grad_scale takes them from the last to the first, so that what grad_squares
// read last is still in L2: it reads the last kKeepBytes with the priority to
// stay there and the rest with the priority to leave, as grad_scale writes
// (250 M bf16 into fp32 338 -> 327 us, 20 M 37.0 -> 32.5 us).
//
// The pointers and sizes travel in the kernel's parameters (up to
// kMaxTable tensors a launch), so that a call copies nothing to the device
// and a captured call keeps its list.
//
// Numerics: a thread squares and adds the elements of its share of one chunk
// in fp32 (at most kChunkElems / kThreads of them).  Shares are added as pairs
// of fp32 values, a sum and what its roundings lost (Knuth's two-sum), to
// about 2^-45: the same in double cost 7 us a kernel and 11 us in front of the
// scaling (1216 CTAs adding 500 partial sums each), since an SM adds two
// doubles a cycle.  Squares of fp32 and bf16 values can leave the fp32 range
// although their root does not: a share whose fp32 sum is above 2^60 or below
// 2^-90 (fp16: cannot be) is summed again scaled by 2^-73 or 2^100 where its
// squares are lost, and goes to a sum in double beside the pair, which is
// looked at only where it is not zero.  A small share needs no second look once
// the thread's sum is 2^-20 or more, 2^70 times it: so the zeros of a list (an
// embedding's unused rows) are read once, but for those before a thread's first
// other element (a list of nothing else takes 1.2 to 1.45 times as long).  Telling
// zeros from small values in the first look cost every bf16 list 1 to 2 %.
#include <algorithm>
#include <new>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "rms_norm.h"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkElems = 16384;
constexpr int64_t kKeepBytes = 80 << 20;  // of 126 MB of L2
constexpr int kSmallTable = 32;
constexpr int kMaxTable = 1024;

// Tensors of one launch; chunks [first[i], first[i + 1]) are tensor i's.
template <int N>
struct GradTable {
  const void* in[N];
  void* out[N];
  int64_t numel[N];
  int first[N + 1];
  unsigned char in_type[N];
  unsigned char out_type[N];
  int count;
  int chunk;  // elements a chunk
  int keep;   // first chunk that is to stay in L2
};

template <int N>
__device__ __forceinline__ int find_tensor(const GradTable<N>& t, int c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Elements before p's next 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int h = (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T));
  return h < n ? h : n;
}

__device__ __forceinline__ uint4 ld_policy(const void* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

// This thread's fp32 sum of (scale * g)^2 over a chunk.
template <typename T>
__device__ __forceinline__ float chunk_squares(const T* __restrict__ p, int n, float scale,
                                               uint64_t policy) {
  constexpr int E = Traits<T>::kVec;
  constexpr int UN = 4;
  const int head = head_of(p, n);
  const int nvec = (n - head) / E;
  const T* body = p + head;
  float part[E];
#pragma unroll
  for (int e = 0; e < E; ++e) part[e] = 0.f;
#pragma unroll 1
  for (int v0 = threadIdx.x; v0 < nvec; v0 += UN * kThreads) {
    uint4 q[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int v = v0 + k * kThreads;
      q[k] = v < nvec ? ld_policy(body + (int64_t)v * E, policy) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      float f[E];
      unpack<T>(q[k], f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float s = f[e] * scale;
        part[e] = fmaf(s, s, part[e]);
      }
    }
  }
  // the elements before and after the vectors: fewer than 2 E
  const int rest = n - nvec * E;
  if ((int)threadIdx.x < rest) {
    const int i = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + nvec * E;
    const float s = Traits<T>::to_f(p[i]) * scale;
    part[0] = fmaf(s, s, part[0]);
  }
#pragma unroll
  for (int w = E / 2; w >= 1; w /= 2)
#pragma unroll
    for (int e = 0; e < w; ++e) part[e] += part[e + w];
  return part[0];
}

// A sum: hi + lo + extra.
struct GradSum {
  float hi, lo;
  double extra;
};

// hi + lo = the old sum + v, to the last bit of lo.
__device__ __forceinline__ void add_to(float& hi, float& lo, float v) {
  const float s = __fadd_rn(hi, v);
  const float b = __fadd_rn(s, -hi);
  lo += __fadd_rn(hi, -__fadd_rn(s, -b)) + __fadd_rn(v, -b);
  hi = s;
}

template <typename T>
__device__ __forceinline__ void add_chunk(GradSum& sum, const void* in, int64_t e0, int n,
                                          uint64_t policy) {
  constexpr bool wide = !std::is_same<T, __half>::value;  // of fp32's exponents
  const T* p = static_cast<const T*>(in) + e0;
  const float s = chunk_squares<T>(p, n, 1.f, policy);
  if (s <= 0x1p60f && s >= (wide ? 0x1p-90f : 0.f)) {
    add_to(sum.hi, sum.lo, s);
  } else if (!wide || isnan(s) || (s > 0x1p60f && !isinf(s))) {
    sum.extra += (double)s;
  } else if (s > 1.f || sum.hi < 0x1p-20f) {
    const float again = chunk_squares<T>(p, n, s < 1.f ? 0x1p100f : kOverflowScale, policy);
    if (again != 0.f) sum.extra += (double)again * (s < 1.f ? 0x1p-200 : 0x1p146);
  }
}

// The CTA's sum, the same in every thread, in a fixed order.
__device__ __forceinline__ GradSum block_sum_grads(GradSum v, GradSum* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, v.hi, m);
    v.lo += __shfl_xor_sync(0xffffffffu, v.lo, m);
    add_to(v.hi, v.lo, hi);
  }
  const unsigned any = __ballot_sync(0xffffffffu, !(v.extra == 0.0));
  if (any)
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v.extra += __shfl_xor_sync(0xffffffffu, v.extra, m);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  GradSum s = {0.f, 0.f, 0.0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const GradSum r = red[w];
    add_to(s.hi, s.lo, r.hi);
    s.lo += r.lo;
    if (!(r.extra == 0.0)) s.extra += r.extra;
  }
  return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 8) grad_squares(const __grid_constant__ GradTable<N> t,
                                                         GradSum* __restrict__ partial) {
  __shared__ GradSum red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int chunks = t.first[t.count];
  GradSum sum = {0.f, 0.f, 0.0};
  uint64_t stay, pass;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(stay));
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pass));
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint64_t policy = c >= t.keep ? stay : pass;
    const int i = find_tensor(t, c);
    const int64_t e0 = (int64_t)(c - t.first[i]) * t.chunk;
    const int64_t left = t.numel[i] - e0;
    const int n = left < t.chunk ? (int)left : t.chunk;
    if (t.in_type[i] == RMSN_F32)
      add_chunk<float>(sum, t.in[i], e0, n, policy);
    else if (t.in_type[i] == RMSN_BF16)
      add_chunk<__nv_bfloat16>(sum, t.in[i], e0, n, policy);
    else
      add_chunk<__half>(sum, t.in[i], e0, n, policy);
  }
  sum = block_sum_grads(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the CTAs' partial sums, the same bits in every CTA: nearest +
// rest, nearest its fp32 value.  `wide` is the norm where it is finite and
// nearest is not (16 values of 3e38), else 0.
struct GradNorm {
  float nearest, rest;
  double wide;
};

__device__ __forceinline__ GradNorm norm_of(const GradSum* __restrict__ partial, int nparts,
                                            GradSum* red) {
  GradSum sum = {0.f, 0.f, 0.0};
  for (int i = threadIdx.x; i < nparts; i += kThreads) {
    const GradSum p = partial[i];
    add_to(sum.hi, sum.lo, p.hi);
    sum.lo += p.lo;
    if (!(p.extra == 0.0)) sum.extra += p.extra;
  }
  sum = block_sum_grads(sum, red);
  if (!(sum.extra == 0.0)) {
    const double v = sqrt((double)sum.hi + (double)sum.lo + sum.extra);
    const float f = (float)v;
    if (isfinite(f)) return {f, (float)(v - (double)f), 0.0};
    return {f, 0.f, isfinite(v) ? v : 0.0};
  }
  // sqrt(s + e) = r + (s - r^2 + e) / (2 r), r = sqrt(s), the difference exact
  const float s = sum.hi + sum.lo, e = sum.lo - (s - sum.hi);
  if (!(s > 0.f)) return {s, 0.f, 0.0};
  const float r = sqrtf(s);
  const float d = (fmaf(-r, r, s) + e) / (2.f * r);
  const float f = r + d;
  return {f, d - (f - r), 0.0};
}

// What a gradient is multiplied by: by `by`, then by `post`, which is 1 unless
// the product of the two is below the normal fp32 numbers and would lose bits
// as one value (the gradients times it need not be).
struct Factor {
  float by, post;
};

// min(1, max_norm / (norm + eps)), 1 where an element (or a given norm) is not
// finite; the quotient corrected by what its division and the norm's rounding
// left, so that it is rounded once.  In double where norm + eps is beyond fp32
// or the quotient below its normal numbers.
__device__ __forceinline__ Factor factor_of(const GradNorm& n, float max_norm, float eps) {
  if (!isfinite(n.nearest) && n.wide == 0.0) return {1.f, 1.f};
  float hi = n.nearest, lo = n.rest;
  add_to(hi, lo, eps);
  const float d = hi + lo, rest = lo - (d - hi);
  double e;
  if (isfinite(d)) {
    if (!(d > max_norm || (d == max_norm && rest > 0.f))) return {1.f, 1.f};
    const float q = max_norm / d;
    const float f = q + (fmaf(-q, d, max_norm) - q * rest) / d;
    if (f >= 0x1p-126f) return {f, 1.f};
    e = (double)max_norm / ((double)d + (double)rest);
  } else {
    e = (double)max_norm / ((n.wide != 0.0 ? n.wide : (double)n.nearest + n.rest) + (double)eps);
    if (!(e < 1.0)) return {1.f, 1.f};
    if (e >= 0x1p-126) return {(float)e, 1.f};
  }
  return e < 0x1p-200 ? Factor{(float)(e * 0x1p149), 0x1p-149f}
                      : Factor{(float)(e * 0x1p100), 0x1p-100f};
}

__global__ void __launch_bounds__(kThreads) grad_norm_final(const GradSum* __restrict__ partial,
                                                            int nparts, float* __restrict__ norm) {
  __shared__ GradSum red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const GradNorm v = norm_of(partial, nparts, red);
  if (threadIdx.x == 0) *norm = v.nearest;
}

// out = round(in * factor) over a chunk: V elements an access where both
// sides can be aligned together, single elements, consecutive lanes on
// consecutive ones, where they cannot.
template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, int64_t e0, int n,
                                            float factor) {
  constexpr int V = 16 / sizeof(O) < 16 / sizeof(T) ? 16 / sizeof(O) : 16 / sizeof(T);
  using VT = typename std::conditional<sizeof(T) * V == 16, uint4, uint2>::type;
  constexpr int UN = 4;
  const T* p = static_cast<const T*>(in) + e0;
  O* o = static_cast<O*>(out) + e0;
  int head = (int)(((16 - ((uintptr_t)o & 15)) & 15) / sizeof(O));
  if (head > n) head = n;
  const bool vec = ((uintptr_t)(p + head) % sizeof(VT)) == 0;
  const int nvec = vec ? (n - head) / V : 0;
  auto put = [&](int v, const VT& q) {
    float f[V];
    if constexpr (sizeof(VT) == 16)
      unpack<T>(q, f);
    else
      unpack_h<T>(q, f);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] *= factor;
    st_vec_stream(o + head + (int64_t)v * V, pack<O>(f));
  };
  auto get = [&](int v) { return *reinterpret_cast<const VT*>(p + head + (int64_t)v * V); };
  int v0 = threadIdx.x;
#pragma unroll 1
  for (; v0 + (UN - 1) * kThreads < nvec; v0 += UN * kThreads) {
    VT q[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k) q[k] = get(v0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < UN; ++k) put(v0 + k * kThreads, q[k]);
  }
#pragma unroll 1
  for (; v0 < nvec; v0 += kThreads) put(v0, get(v0));
  const int rest = n - nvec * V;
  if (rest < 2 * V) {
    if ((int)threadIdx.x < rest) {
      const int i = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + nvec * V;
      o[i] = Traits<O>::from_f(Traits<T>::to_f(p[i]) * factor);
    }
  } else {  // no common alignment: nvec is 0
    constexpr int US = 8;
    int i0 = threadIdx.x;
#pragma unroll 1
    for (; i0 + (US - 1) * kThreads < n; i0 += US * kThreads) {
      T q[US];
#pragma unroll
      for (int k = 0; k < US; ++k) q[k] = p[i0 + k * kThreads];
#pragma unroll
      for (int k = 0; k < US; ++k)
        o[i0 + k * kThreads] = Traits<O>::from_f(Traits<T>::to_f(q[k]) * factor);
    }
#pragma unroll 1
    for (; i0 < n; i0 += kThreads) o[i0] = Traits<O>::from_f(Traits<T>::to_f(p[i0]) * factor);
  }
}

// The same with a factor of two parts, which few lists ever have: in the loops
// above its second product cost 1 to 3 % of the call.
__device__ __noinline__ void scale_chunk_by_parts(const void* in, int from, void* out, int to,
                                                  int64_t e0, int n, float by, float post) {
  for (int64_t i = e0 + threadIdx.x; i < e0 + n; i += kThreads) {
    const float g = from == RMSN_F32    ? static_cast<const float*>(in)[i]
                    : from == RMSN_BF16 ? Traits<__nv_bfloat16>::to_f(
                                              static_cast<const __nv_bfloat16*>(in)[i])
                                        : Traits<__half>::to_f(static_cast<const __half*>(in)[i]);
    const float v = g * by * post;
    if (to == RMSN_F32)
      static_cast<float*>(out)[i] = v;
    else if (to == RMSN_BF16)
      static_cast<__nv_bfloat16*>(out)[i] = Traits<__nv_bfloat16>::from_f(v);
    else
      static_cast<__half*>(out)[i] = Traits<__half>::from_f(v);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale(const __grid_constant__ GradTable<N> t,
                                                       const GradSum* __restrict__ partial,
                                                       int nparts,
                                                       const float* __restrict__ total_norm,
                                                       float max_norm, float eps,
                                                       float* __restrict__ norm) {
  __shared__ GradSum red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const GradNorm v = total_norm != nullptr ? GradNorm{*total_norm, 0.f, 0.0}
                                           : norm_of(partial, nparts, red);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = v.nearest;
  const Factor f = factor_of(v, max_norm, eps);
  const float factor = f.by;
  const int chunks = t.first[t.count];
  for (int c = chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = find_tensor(t, c);
    if (factor == 1.f && t.in[i] == t.out[i]) continue;  // in place: nothing changes
    const int64_t e0 = (int64_t)(c - t.first[i]) * t.chunk;
    const int64_t left = t.numel[i] - e0;
    const int n = left < t.chunk ? (int)left : t.chunk;
    const int from = t.in_type[i], to = t.out_type[i];
    if (f.post != 1.f)
      scale_chunk_by_parts(t.in[i], from, t.out[i], to, e0, n, factor, f.post);
    else if (from == RMSN_F32)
      scale_chunk<float, float>(t.in[i], t.out[i], e0, n, factor);
    else if (from == RMSN_BF16 && to == RMSN_F32)
      scale_chunk<__nv_bfloat16, float>(t.in[i], t.out[i], e0, n, factor);
    else if (from == RMSN_BF16)
      scale_chunk<__nv_bfloat16, __nv_bfloat16>(t.in[i], t.out[i], e0, n, factor);
    else if (to == RMSN_F32)
      scale_chunk<__half, float>(t.in[i], t.out[i], e0, n, factor);
    else
      scale_chunk<__half, __half>(t.in[i], t.out[i], e0, n, factor);
  }
}

// As launch_kernel, with the arguments by address: a table is up to 30 KB.
cudaError_t launch_table(const void* kern, int grid, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
  LaunchLog& log = launch_log();
  if (e == cudaSuccess && log.n < 4) log.kern[log.n++] = kern;
  return e;
}

// One call's list, its empty tensors left out as the tables are filled.
struct GradList {
  const void* const* in;
  void* const* out;  // NULL: the norm alone
  const int64_t* numel;
  const int* in_type;
  const int* out_type;
  int64_t count;
  float max_norm, eps;
  const float* total_norm;
  float* norm;
  GradSum* partial;
};

int elem_size(int dtype) { return dtype == RMSN_F32 ? 4 : 2; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Fills the next table from list position *at; returns its chunks.
template <int N>
int fill_table(const GradList& g, int chunk, int64_t* at, GradTable<N>& t) {
  t.count = 0;
  t.chunk = chunk;
  int64_t c = 0;
  for (; *at < g.count && t.count < N; ++*at) {
    const int64_t n = g.numel[*at];
    if (n == 0) continue;
    t.in[t.count] = g.in[*at];
    t.out[t.count] = g.out != nullptr ? g.out[*at] : nullptr;
    t.numel[t.count] = n;
    t.in_type[t.count] = (unsigned char)g.in_type[*at];
    t.out_type[t.count] = (unsigned char)(g.out_type != nullptr ? g.out_type[*at] : 0);
    t.first[t.count++] = (int)c;
    c += ceil_div(n, chunk);  // a list of 2^42 elements has 2^29 chunks
  }
  t.first[t.count] = (int)c;
  t.keep = (int)c;
  if (g.out != nullptr) {  // the scaling follows
    int64_t bytes = 0;
    for (int i = t.count - 1; i >= 0 && bytes < kKeepBytes; --i) {
      const int64_t chunk_bytes = (int64_t)chunk * elem_size(t.in_type[i]);
      const int64_t mine = t.first[i + 1] - t.first[i];
      const int64_t room = (kKeepBytes - bytes + chunk_bytes - 1) / chunk_bytes;
      t.keep -= (int)(mine < room ? mine : room);
      bytes += mine * chunk_bytes;
    }
  }
  return (int)c;
}

template <int N>
cudaError_t run_list(const GradList& g, int chunk, cudaStream_t s, int* launches) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(dev);
  GradTable<N> t;
  int nparts = 0;
  if (g.total_norm == nullptr) {
    const void* kern = (const void*)grad_squares<N>;
    int most = sms * max_blocks_per_sm(kern, kThreads, 0);
    if (most > RMSN_GRAD_MAX_PARTIALS) most = RMSN_GRAD_MAX_PARTIALS;
    for (int64_t at = 0; at < g.count;) {
      const int chunks = fill_table<N>(g, chunk, &at, t);
      if (chunks == 0) break;
      const int grid = chunks < most ? chunks : most;
      GradSum* slot = g.partial + nparts;
      void* args[] = {&t, &slot};
      e = launch_table(kern, grid, s, args);
      if (e != cudaSuccess) return e;
      *launches += 1;
      nparts += grid;
    }
  }
  if (g.out == nullptr) {
    e = launch_kernel(grad_norm_final, dim3(1), dim3(kThreads), 0, s, 1, (const GradSum*)g.partial,
                      nparts, g.norm);
    if (e == cudaSuccess) *launches += 1;
    return e;
  }
  const void* kern = (const void*)grad_scale<N>;
  const int most = sms * max_blocks_per_sm(kern, kThreads, 0);
  const GradSum* partial = g.partial;
  float max_norm = g.max_norm, eps = g.eps;
  float* norm = g.norm;
  const float* total = g.total_norm;
  for (int64_t at = 0; at < g.count;) {
    const int chunks = fill_table<N>(g, chunk, &at, t);
    if (chunks == 0 && norm == nullptr) break;
    const int grid = chunks < 1 ? 1 : chunks < most ? chunks : most;
    void* args[] = {&t, &partial, &nparts, &total, &max_norm, &eps, &norm};
    e = launch_table(kern, grid, s, args);
    if (e != cudaSuccess) return e;
    *launches += 1;
    norm = nullptr;
  }
  return cudaSuccess;
}

cudaError_t launch_list(const GradList& g, cudaStream_t s, int* launches) {
  int64_t total = 0;
  for (int64_t i = 0; i < g.count; ++i) total += g.numel[i];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // 16384 or 8192 elements, whichever gives the longest CTA less to do, a
  // chunk costing about 512 elements more than it has (4096 would be half a
  // batch of 16-bit loads: 30 M 16.5 -> 25.4 us for the norm); short lists in
  // smaller chunks, down to one access a thread.
  const int64_t ctas = 8 * sm_count(dev);
  int chunk = kChunkElems;
  if (ceil_div(ceil_div(total, chunk / 2), ctas) * (chunk / 2 + 512) <
      ceil_div(ceil_div(total, chunk), ctas) * (chunk + 512))
    chunk /= 2;
  while (chunk > 1024 && total / chunk < 2 * sm_count(dev)) chunk /= 2;
  return g.count <= kSmallTable ? run_list<kSmallTable>(g, chunk, s, launches)
                                : run_list<kMaxTable>(g, chunk, s, launches);
}

int check_list(const void* const* grads, const int64_t* numels, const int* dtypes, int64_t count) {
  if (count < 0) return RMSN_ERR_SHAPE;
  if (count > 0 && (!grads || !numels || !dtypes)) return RMSN_ERR_NULL;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (dtypes[i] != RMSN_F32 && dtypes[i] != RMSN_BF16 && dtypes[i] != RMSN_F16)
      return RMSN_ERR_DTYPE;
    if (numels[i] < 0 || numels[i] > RMSN_GRAD_MAX_ELEMENTS) return RMSN_ERR_SHAPE;
    total += numels[i];
    if (total > RMSN_GRAD_MAX_ELEMENTS) return RMSN_ERR_SHAPE;
    if (numels[i] > 0 && !grads[i]) return RMSN_ERR_NULL;
    if ((uintptr_t)grads[i] % elem_size(dtypes[i]) != 0) return RMSN_ERR_ALIGN;
  }
  return RMSN_OK;
}

struct Span {
  uintptr_t lo, hi;
  int64_t index;
  bool out;
};

// Whether an output shares bytes with another output, or with a gradient
// that is not its own in place: such a list has no order of results.
// *failed: no memory to look.
bool overlaps(const void* const* grads, const int64_t* numels, const int* dtypes,
              void* const* outs, const int* out_dtypes, int64_t count, bool* failed) {
  Span* spans = new (std::nothrow) Span[2 * (size_t)count + 1];
  *failed = spans == nullptr;
  if (*failed) return false;
  size_t n = 0;
  bool sorted = true;
  for (int64_t i = 0; i < count; ++i) {
    if (numels[i] == 0) continue;
    const uintptr_t a = (uintptr_t)grads[i], b = (uintptr_t)outs[i];
    const bool in_place = a == b && dtypes[i] == out_dtypes[i];
    if (!in_place) spans[n++] = Span{a, a + (uintptr_t)numels[i] * elem_size(dtypes[i]), i, false};
    spans[n++] = Span{b, b + (uintptr_t)numels[i] * elem_size(out_dtypes[i]), i, true};
  }
  for (size_t i = 1; i < n && sorted; ++i) sorted = spans[i - 1].lo <= spans[i].lo;
  if (!sorted)
    std::sort(spans, spans + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  // furthest ends so far of outputs and of gradients
  uintptr_t out_end = 0, any_end = 0;
  bool hit = false;
  for (size_t i = 0; i < n && !hit; ++i) {
    hit = spans[i].lo < (spans[i].out ? any_end : out_end);
    any_end = std::max(any_end, spans[i].hi);
    if (spans[i].out) out_end = std::max(out_end, spans[i].hi);
  }
  delete[] spans;
  return hit;
}

bool meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  return a && b && na && nb && p < q + nb && q < p + na;
}

// Whether `bytes` at p share memory with a tensor of the list.
bool in_list(const void* p, size_t bytes, const void* const* list, const int64_t* numels,
             const int* dtypes, int64_t count) {
  for (int64_t i = 0; i < count; ++i)
    if (meet(p, bytes, list[i], (size_t)numels[i] * elem_size(dtypes[i]))) return true;
  return false;
}

// Room for the partial sums of every launch, a table's tensors each.
size_t workspace_bytes_of(int64_t count) {
  const int64_t tables = count <= kMaxTable ? 1 : ceil_div(count, kMaxTable);
  return (size_t)tables * RMSN_GRAD_MAX_PARTIALS * sizeof(GradSum);
}

}  // namespace
}  // namespace rmsn

extern "C" {

size_t rms_norm_grad_workspace_size(int64_t count) {
  return count < 0 ? 0 : rmsn::workspace_bytes_of(count);
}

int rms_norm_grad_norm(const void* const* grads, const int64_t* numels, const int* dtypes,
                       int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                       void* stream) {
  using namespace rmsn;
  const int st = check_list(grads, numels, dtypes, count);
  if (st != RMSN_OK) return st;
  begin_call();
  if (!norm || !workspace) return RMSN_ERR_NULL;
  if ((uintptr_t)workspace % 16 != 0) return RMSN_ERR_ALIGN;
  if (workspace_bytes < workspace_bytes_of(count)) return RMSN_ERR_WORKSPACE;
  if (meet(norm, sizeof(float), workspace, workspace_bytes) ||
      in_list(norm, sizeof(float), grads, numels, dtypes, count) ||
      in_list(workspace, workspace_bytes, grads, numels, dtypes, count))
    return RMSN_ERR_ARG;
  GradList g = {grads, nullptr, numels, dtypes, nullptr, count, 0.f, 0.f, nullptr, norm,
                static_cast<GradSum*>(workspace)};
  int launches = 0;
  const cudaError_t e = launch_list(g, static_cast<cudaStream_t>(stream), &launches);
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(launches);
  return RMSN_OK;
}

int rms_norm_grad_clip(const void* const* grads, const int64_t* numels, const int* dtypes,
                       void* const* outs, const int* out_dtypes, int64_t count, float max_norm,
                       float eps, const float* total_norm, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream) {
  using namespace rmsn;
  int st = check_list(grads, numels, dtypes, count);
  if (st == RMSN_OK) st = check_list(const_cast<const void* const*>(outs), numels, out_dtypes, count);
  if (st != RMSN_OK) return st;
  for (int64_t i = 0; i < count; ++i)
    if (out_dtypes[i] != dtypes[i] && out_dtypes[i] != RMSN_F32) return RMSN_ERR_DTYPE;
  if (!(max_norm >= 0.f)) return RMSN_ERR_ARG;
  if (!(eps >= 0.f) || isinf(eps)) return RMSN_ERR_EPS;
  begin_call();
  if ((!norm && !total_norm) || (!workspace && !total_norm)) return RMSN_ERR_NULL;
  if ((uintptr_t)workspace % 16 != 0) return RMSN_ERR_ALIGN;
  if (!total_norm && workspace_bytes < workspace_bytes_of(count)) return RMSN_ERR_WORKSPACE;
  bool failed = false;
  if (overlaps(grads, numels, dtypes, outs, out_dtypes, count, &failed)) return RMSN_ERR_ARG;
  if (failed) return cuda_fail(cudaErrorMemoryAllocation);
  const void* const* written = const_cast<const void* const*>(outs);
  if (in_list(norm, sizeof(float), grads, numels, dtypes, count) ||
      in_list(norm, sizeof(float), written, numels, out_dtypes, count))
    return RMSN_ERR_ARG;
  if (total_norm) {  // the same address as norm's: it receives its own value
    if ((total_norm != norm && meet(norm, sizeof(float), total_norm, sizeof(float))) ||
        in_list(total_norm, sizeof(float), written, numels, out_dtypes, count))
      return RMSN_ERR_ARG;
  } else if (meet(norm, sizeof(float), workspace, workspace_bytes) ||
             in_list(workspace, workspace_bytes, grads, numels, dtypes, count) ||
             in_list(workspace, workspace_bytes, written, numels, out_dtypes, count)) {
    return RMSN_ERR_ARG;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  GradList g = {grads, outs, numels, dtypes, out_dtypes, count, max_norm, eps, total_norm, norm,
                static_cast<GradSum*>(workspace)};
  int launches = 0;
  cudaError_t e = cudaSuccess;
  if (count == 0) {  // nothing to scale: the norm of nothing, or the given one
    if (norm && total_norm)
      e = cudaMemcpyAsync(norm, total_norm, sizeof(float), cudaMemcpyDeviceToDevice, cs);
    else if (norm)
      e = cudaMemsetAsync(norm, 0, sizeof(float), cs);
  } else {
    e = launch_list(g, cs, &launches);
  }
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(launches);
  return RMSN_OK;
}

}  // extern "C"
