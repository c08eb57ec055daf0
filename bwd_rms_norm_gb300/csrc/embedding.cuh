// What the embedding's forward and backward share: the accesses to rows, the
// ids, the checks of arguments and the launches.
#pragma once

#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "rms_norm.h"

namespace rmsn {
namespace {

// Elements a lane takes at a time: 16 bytes of the narrower type.
template <typename T, typename U>
constexpr int kElems = sizeof(T) == 4 && sizeof(U) == 4 ? 4 : 8;

// A lane's E elements of a row from column c on: consecutive ones, of rows of
// whole 16-byte vectors (VEC), or every 32nd one.
template <bool VEC, int E, typename T>
__device__ __forceinline__ void load_row(const T* row, int c, int hidden, float (&f)[E]) {
  if constexpr (VEC) {
    constexpr int V = Traits<T>::kVec;
    if (c < hidden) {
#pragma unroll
      for (int k = 0; k < E / V; ++k) {
        float g[V];
        unpack<T>(*(reinterpret_cast<const uint4*>(row + c) + k), g);
#pragma unroll
        for (int i = 0; i < V; ++i) f[k * V + i] = g[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c + 32 * i < hidden) f[i] = Traits<T>::to_f(row[c + 32 * i]);
  }
}

template <bool VEC, int E, typename U>
__device__ __forceinline__ void store_row(U* row, int c, int hidden, const float (&f)[E]) {
  if constexpr (VEC) {
    constexpr int V = Traits<U>::kVec;
    if (c < hidden) {
#pragma unroll
      for (int k = 0; k < E / V; ++k) {
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = f[k * V + i];
        st_vec(reinterpret_cast<uint4*>(row + c) + k, pack<U>(g));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c + 32 * i < hidden) row[c + 32 * i] = Traits<U>::from_f(f[i]);
  }
}

// The first of a lane's columns in slab `slab` of 32 E columns.
template <bool VEC, int E>
__device__ __forceinline__ int first_column(int slab, int lane) {
  return slab * 32 * E + (VEC ? lane * E : lane);
}

struct Ids {
  const void* p;
  int wide;
  // the id of token t, -1 for one outside the table
  __device__ __forceinline__ int get(int64_t t, int64_t vocab) const {
    const int64_t id = wide ? static_cast<const int64_t*>(p)[t]
                            : (int64_t) static_cast<const int32_t*>(p)[t];
    return id >= 0 && id < vocab ? (int)id : -1;
  }
};

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int bytes_of(int dtype) { return dtype == RMSN_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == RMSN_F32 || dtype == RMSN_BF16 || dtype == RMSN_F16; }

// Warps for `units`, as many CTAs as fit at once at most.
template <typename K, typename... Args>
cudaError_t launch_units(K kern, int64_t units, cudaStream_t s, Args... args) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sm_count(dev) * max_blocks_per_sm((const void*)kern, kThreads, 0);
  return launch_kernel(kern, dim3((unsigned)least(ceil_div(units, kWarps), most)), dim3(kThreads),
                       0, s, 1, args...);
}

bool rows_ok(const void* p, int64_t hidden, int bytes) {
  return (uintptr_t)p % 16 == 0 && hidden * bytes % 16 == 0;
}

// f(T, U) of the types' values, for equal ones or where one is fp32.
template <typename F>
cudaError_t with_types(int t, int u, F f) {
  const float f32 = 0;
  const __nv_bfloat16 bf16{};
  const __half f16{};
  if (t == RMSN_F32) return u == RMSN_F32 ? f(f32, f32) : u == RMSN_BF16 ? f(f32, bf16) : f(f32, f16);
  if (t == RMSN_BF16) return u == RMSN_F32 ? f(bf16, f32) : f(bf16, bf16);
  return u == RMSN_F32 ? f(f16, f32) : f(f16, f16);
}

struct Span {
  uintptr_t lo, hi;
  Span(const void* p, size_t n)
      : lo(reinterpret_cast<uintptr_t>(p)), hi(p ? reinterpret_cast<uintptr_t>(p) + n : 0) {}
  bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

int check(int64_t tokens, int64_t vocab, int64_t hidden, float scale, int ids_64, int t, int u) {
  if (!known(t) || !known(u) || (t != u && t != RMSN_F32 && u != RMSN_F32)) return RMSN_ERR_DTYPE;
  if (tokens < 0 || tokens > RMSN_MAX_ROWS || vocab < 1 || vocab > RMSN_EMBEDDING_MAX_VOCAB ||
      hidden < 1 || hidden > RMSN_MAX_HIDDEN)
    return RMSN_ERR_SHAPE;
  if (!isfinite(scale) || (ids_64 != 0 && ids_64 != 1)) return RMSN_ERR_ARG;
  return RMSN_OK;
}

}  // namespace
}  // namespace rmsn
