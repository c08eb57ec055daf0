// Staged block norm for sm_103a (the formulas are in block_norm.cu).
//
// Both directions are bound by HBM bandwidth: the forward moves 2 + 2 and the
// backward 4 + 2 rows for each row, against 20 to 30 instructions an element.
// What decides the speed is how many bytes an SM keeps in flight while the
// row's reductions, which nothing of the row can be written before, run.
//
// A persistent CTA per SM (or cluster of CTAs, for rows too wide for one)
// streams its rows with 1D bulk copies into a ring of shared-memory stages
// (full[s] when a stage has landed, empty[s] when its readers are done).
// Every wait is bounded (mbar.cuh); a warp whose wait ran out skips the rest
// of its rows but still reaches the CTA's and the cluster's barriers.
//
// fp32 arithmetic goes by pairs (the f32x2 instructions): with 16-bit rows the
// instructions an element count as much as its bytes.
#pragma once

#include <atomic>
#include <type_traits>

#include "block_norm.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "mbar.cuh"
#include "rms_norm.h"

namespace rmsn {
namespace {

__device__ unsigned int g_block_timeouts;

constexpr int kMaxWarps = 16;     // consumer warps of a CTA
constexpr int kMaxStages = 16;
constexpr int kMaxSplit = 16;      // CTAs a row is split over
constexpr int kSmemBudget = 224 * 1024;

// Stages of a CTA whose rows it brings into L2 before griddepcontrol.wait
// (prefetch_l2).  Back to back, none / 4: 4096 x 4096 bf16 forward 28.2 / 27.2
// us, backward 44.2 / 43.5; 8192 x 4096 fp32 forward 89.5 / 85.1; 4096 x 1024
// fp16 backward 19.2 / 18.0.
constexpr int kFirstStages = 4;

// Elements a thread loads at a time: 16 bytes of the narrower type, and 16 of
// the wider, so that neighbouring lanes' accesses to shared memory and to
// global memory are contiguous in both.
template <typename T, typename TS>
constexpr int kElems = sizeof(T) == 2 && sizeof(TS) == 2 ? 8 : 4;

// ---------------------------------------------------------------------------
// pairs of fp32 values in 64-bit registers
// ---------------------------------------------------------------------------
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float2 split(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float sum2(f32x2 v) {
  const float2 f = split(v);
  return f.x + f.y;
}

template <typename U>
__device__ __forceinline__ f32x2 widen(uint32_t w);

template <>
__device__ __forceinline__ f32x2 widen<__nv_bfloat16>(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <>
__device__ __forceinline__ f32x2 widen<__half>(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}

template <typename U>
__device__ __forceinline__ uint32_t narrow(f32x2 v);

template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(f32x2 v) {
  const float2 f = split(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <>
__device__ __forceinline__ uint32_t narrow<__half>(f32x2 v) {
  const float2 f = split(v);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// E = 2 N elements of type U at p, 8 or 16 bytes.
template <typename U, int N>
__device__ __forceinline__ void load_pairs(const U* p, f32x2 (&f)[N]) {
  if constexpr (sizeof(U) == 4) {
    static_assert(N == 2, "16 bytes");
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(p);
    f[0] = q.x;
    f[1] = q.y;
  } else if constexpr (N == 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    f[0] = widen<U>(q.x);
    f[1] = widen<U>(q.y);
    f[2] = widen<U>(q.z);
    f[3] = widen<U>(q.w);
  } else {
    static_assert(N == 2, "8 bytes");
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    f[0] = widen<U>(q.x);
    f[1] = widen<U>(q.y);
  }
}

template <typename U, int N>
__device__ __forceinline__ void store_pairs(U* p, const f32x2 (&f)[N]) {
  if constexpr (sizeof(U) == 4) {
    const float2 a = split(f[0]), b = split(f[1]);
    st_vec(p, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                         __float_as_uint(b.y)));
  } else if constexpr (N == 4) {
    st_vec(p, make_uint4(narrow<U>(f[0]), narrow<U>(f[1]), narrow<U>(f[2]), narrow<U>(f[3])));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(narrow<U>(f[0]), narrow<U>(f[1]));
  }
}

template <int N>
__device__ __forceinline__ float sum_pairs(f32x2 (&f)[N]) {
#pragma unroll
  for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) f[i] = add2(f[i], f[i + h]);
  return sum2(f[0]);
}

struct Ring {
  int stage;
  uint32_t phase;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// A bounded wait of a whole warp for phase `parity` of `bar`.  A try suspends
// the warp for some hundred cycles; between tries it does next to nothing (a
// look at the timer and the abort flag every 64 of them), since what waiting
// warps issue is taken from those that have work.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort) {
  unsigned long long t0 = 0;
  for (int i = 1;; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (i & 63) continue;
    if (*abort) return false;
    if (t0 == 0) {
      t0 = global_ns();
    } else if (global_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      atomicAdd(&g_block_timeouts, 1u);
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool done = mbar_try_wait(bar, parity);
  if (!done) done = wait_long(bar, parity, abort);
  return __all_sync(0xffffffffu, done);
}

// Waits for the last copies issued, the latest of each stage, before the CTA may exit.
__device__ void drain_ring(uint64_t* full, Ring pos, int64_t issued, int stages) {
  const int n = issued < stages ? (int)issued : stages;
  for (int k = 0; k < n; ++k) {
    if (pos.stage == 0) {
      pos.stage = stages - 1;
      pos.phase ^= 1u;
    } else {
      --pos.stage;
    }
    drain_phase_counted(&full[pos.stage], pos.phase, &g_block_timeouts);
  }
}

__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// A barrier that the CTAs of a cluster of cs arrive on.
__device__ __forceinline__ bool team_wait(int cs, uint64_t* bar, uint32_t parity,
                                          volatile int* abort) {
  if (cs == 1) return wait_all(bar, parity, abort);
  bool done = try_wait_cluster(bar, parity);
  if (!done) done = wait_cluster_counted(bar, parity, abort, &g_block_timeouts);
  return __all_sync(0xffffffffu, done);
}

__device__ __forceinline__ void st_peer4(float4* local, uint32_t peer, float4 v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(remote)
               : "r"(smem_u32(local)), "r"(peer));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// Three sums over the lanes at once: lanes exchange halves of the values as
// they add (6 shuffles, and 3 to spread the results, for 15).
__device__ __forceinline__ float3 warp_sum3(float a, float b, float c, int lane) {
  const bool hi = lane & 16;
  const float k0 = hi ? c : a, k1 = hi ? 0.f : b;
  const float s0 = hi ? a : c, s1 = hi ? b : 0.f;
  float u = k0 + __shfl_xor_sync(0xffffffffu, s0, 16);
  float w = k1 + __shfl_xor_sync(0xffffffffu, s1, 16);
  const bool mid = lane & 8;
  const float keep = mid ? w : u, send = mid ? u : w;
  float v = keep + __shfl_xor_sync(0xffffffffu, send, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return make_float3(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 8),
                     __shfl_sync(0xffffffffu, v, 16));
}

template <int N>
__device__ __forceinline__ void load_plane(const float4* plane, int nvec, int v, f32x2 (&f)[N]) {
#pragma unroll
  for (int q = 0; q < N / 2; ++q) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(plane + q * nvec + v);
    f[2 * q] = u.x;
    f[2 * q + 1] = u.y;
  }
}

template <int N>
__device__ __forceinline__ void store_plane(float4* plane, int nvec, int v,
                                            const f32x2 (&f)[N]) {
#pragma unroll
  for (int q = 0; q < N / 2; ++q)
    *reinterpret_cast<ulonglong2*>(plane + q * nvec + v) = make_ulonglong2(f[2 * q], f[2 * q + 1]);
}

// Rows of up to kNarrowGroups groups of columns take kNarrowLanes lanes, and
// a warp takes 32 / kNarrowLanes of them at a time: their reductions share
// their shuffles.
constexpr int kNarrowLanes = 8;
constexpr int kNarrowGroups = 64;

// ---------------------------------------------------------------------------
// rows that do not start on 16 bytes (EDGE)
// ---------------------------------------------------------------------------
// Row i of a tensor of odd width starts i H elements after a 16-byte boundary,
// which is s = i H mod A past one (A elements in 16 bytes of T), the same s for
// every P-th row, P = A / gcd(H, A).  A unit works on rows i = c (mod P) alone,
// so that its s is fixed: it copies from the boundary before a row to the one
// after, s columns and a few others too many, keeps its weights s columns
// later, and takes the row as an aligned one of `span` = s + H columns of
// which the first s do not count.  What was copied too much is set to zero in
// shared memory by the first to read the row, so that the loops over its
// columns are those of aligned rows but for the stores of its two ends.
__host__ __device__ inline int row_period(int hidden, int a) {
  int p = a;
  while (p > 1 && hidden % 2 == 0) {
    hidden /= 2;
    p /= 2;
  }
  return p;
}

// Columns of a row over `cs` CTAs, with up to a - 1 in front of it.
__host__ __device__ inline int row_part(int hidden, int a, int cs, bool edge) {
  return edge ? ((hidden + a - 1 + cs - 1) / cs + a - 1) / a * a : hidden / cs;
}

// A CTA's columns of its rows: [s, span) of the `pitch` that it keeps, column
// c of them being the row's col0 + c.
struct Part {
  int s, span, pitch, col0;
  __device__ Part(int hidden, int a, int cs, uint32_t rank, int cls, bool edge) {
    pitch = row_part(hidden, a, cs, edge);
    const int before = edge ? cls * hidden % a : 0;
    s = rank == 0 ? before : 0;
    col0 = (int)rank * pitch - before;
    const int left = hidden - col0;
    span = left < pitch ? left : pitch;
  }
  // whether columns [c, c + e) are all the row's
  __device__ __forceinline__ bool inner(int c, int e) const { return c >= s && c + e <= span; }
  __device__ __forceinline__ bool has(int c) const { return c >= s && c < span; }
};

// The columns of a row's groups that are not all its own: the A / E first
// groups and the last one, a column each for sixteen lanes (eight lanes take
// two).  -1: none.
template <int A, int E>
__device__ __forceinline__ int end_column(int i, int nvec, const Part& part) {
  const int c = i < 8 ? i : (nvec - 1) * E + i - 8;
  const bool there = i < 8 ? i < A : i - 8 < E && nvec > A / E;
  return there && !part.inner(c / E * E, E) ? c : -1;
}

// Weights g[c], g[c + 1], ..., where they are not the row's zero.
template <typename T, int N, bool EDGE>
__device__ __forceinline__ void load_weights(const T* g, int c, const Part& part, f32x2 (&f)[N]) {
  if constexpr (EDGE) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = c + 2 * i;
      f[i] = pair(part.has(k) ? Traits<T>::to_f(g[k]) : 0.f,
                  part.has(k + 1) ? Traits<T>::to_f(g[k + 1]) : 0.f);
    }
  } else {
    load_pairs<T, N>(g + c, f);
  }
}

// Stores the row's columns among c, c + 1, ... one by one.
template <typename U, int N>
__device__ __forceinline__ void store_ends(U* p, int c, const Part& part, const f32x2 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 v = split(f[i]);
    const int k = c + 2 * i;
    if (part.has(k)) p[k] = Traits<U>::from_f(v.x);
    if (part.has(k + 1)) p[k + 1] = Traits<U>::from_f(v.y);
  }
}

// One row's copy, `n` elements from element `from` of src on, where the tensor
// has `total`: at its end whole 16 bytes only (`whole` elements).  copy_tail
// fetches the row's elements behind them, before the barrier's arrive, and
// gives the copy's bytes.
template <typename U>
__device__ __forceinline__ int64_t whole(int64_t from, int n, int64_t total) {
  constexpr int a = 16 / sizeof(U);
  const int64_t left = total - from;
  return left >= n ? n : left / a * a;
}

template <typename U>
__device__ __forceinline__ void copy_row(unsigned char* dst, const U* src, int64_t from, int n,
                                         int64_t total, uint64_t* bar) {
  const int64_t m = whole<U>(from, n, total);
  if (m > 0) bulk_load(dst, src + from, (uint32_t)(m * sizeof(U)), bar);
}

template <typename U>
__device__ __forceinline__ uint32_t copy_tail(unsigned char* dst, const U* src, int64_t from,
                                              int n, int64_t total) {
  const int m = (int)whole<U>(from, n, total);
  if (m < n)
    for (int64_t k = m; from + k < total; ++k) reinterpret_cast<U*>(dst)[k] = src[from + k];
  return (uint32_t)(m * (int)sizeof(U));
}

constexpr int kSlack = 1024;  // static shared memory beside the kernels' structs

template <auto KERNEL>
struct Kern {
  static constexpr auto value = KERNEL;
};

// Lets KERNEL use `bytes` of dynamic shared memory and clusters of any size,
// once a device: as calls on every launch they cost 0.4 us of 3.9.
template <auto KERNEL>
cudaError_t allow(int dev, size_t bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const void* kern = reinterpret_cast<const void*>(KERNEL);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) e = allow_cluster(kern, kMaxSplit);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace
}  // namespace rmsn
