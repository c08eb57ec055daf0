// Embedding: the rows of a table that a batch of tokens takes, scaled, and the
// table's gradient, summed over the tokens sorted by their id.
#include <math.h>

#include "cluster.cuh"
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

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A warp takes 32 E columns of a token's row.
template <typename T, typename U, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_rows(Ids ids, const T* __restrict__ weight,
                                                           U* __restrict__ y, int64_t tokens,
                                                           int64_t vocab, int hidden, float scale) {
  constexpr int E = kElems<T, U>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slabs = (hidden + 32 * E - 1) / (32 * E);
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < tokens * slabs;
       u += (int64_t)gridDim.x * kWarps) {
    const int64_t t = u / slabs;
    const int c = first_column<VEC, E>((int)(u % slabs), lane);
    const int id = ids.get(t, vocab);
    float f[E] = {};
    if (id >= 0) load_row<VEC, E>(weight + (int64_t)id * hidden, c, hidden, f);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = id >= 0 ? f[i] * scale : 0.f;
    store_row<VEC, E>(y + t * hidden, c, hidden, f);
  }
}

// ---------------------------------------------------------------------------
// backward: tokens sorted by id
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;   // of a digit

struct SortParams {
  Ids ids;
  int64_t tokens, vocab, padding_idx;
  uint32_t* key[2];    // ids and tokens, in turn the source and the target of a pass
  uint32_t* token[2];
  int passes, bits;    // digits, and bits of each
  int cluster;
  char* zero;          // the table, where it is to be cleared: `zeros` bytes
  int64_t zeros;
};

__device__ __forceinline__ uint32_t ld_peer(const uint32_t* local, uint32_t peer) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(peer));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Clears [p, p + n), over `ctas` CTAs of which this is number `cta`.
__device__ __forceinline__ void clear(char* p, int64_t n, int64_t cta, int64_t ctas) {
  const int64_t edge = (16 - (int64_t)(reinterpret_cast<uintptr_t>(p) & 15)) & 15;
  const int64_t head = edge < n ? edge : n, vecs = (n - head) / 16, tail = head + vecs * 16;
  if (cta == 0) {
    for (int64_t i = threadIdx.x; i < head; i += blockDim.x) p[i] = 0;
    for (int64_t i = tail + threadIdx.x; i < n; i += blockDim.x) p[i] = 0;
  }
  for (int64_t i = cta * blockDim.x + threadIdx.x; i < vecs; i += ctas * blockDim.x)
    st_vec(p + head + i * 16, make_uint4(0, 0, 0, 0));
}

// A stable radix sort of the tokens by id, by one cluster of CTAs: each of its
// warps has a run of consecutive entries, counts its digits, and, once the
// counts of the warps before it are known, puts its entries in their order
// behind theirs.  The other clusters of the launch clear the table meanwhile.
__global__ void __launch_bounds__(kSortThreads) embedding_sort(const SortParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t sums[32];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= p.cluster) {
    clear(p.zero, p.zeros, blockIdx.x - p.cluster, gridDim.x - p.cluster);
    return;
  }
  const int bins = 1 << p.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* count = smem + warp * bins;           // this warp's
  uint32_t* total = smem + kSortWarps * bins;     // the CTA's, read by its peers
  uint32_t* base = total + bins;
  const int rank = (int)cta_rank(), d = threadIdx.x;
  const int64_t share = ((p.tokens + p.cluster * kSortWarps - 1) / (p.cluster * kSortWarps) + 31)
                        / 32 * 32;
  const int64_t lo = (rank * kSortWarps + warp) * share;
  const int64_t hi = lo + share < p.tokens ? lo + share : p.tokens;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t* key_in = p.key[(pass & 1) ^ 1];
    const uint32_t* token_in = p.token[(pass & 1) ^ 1];
    auto key_at = [&](int64_t i) -> uint32_t {
      if (pass > 0) return __ldcg(key_in + i);
      const int id = p.ids.get(i, p.vocab);
      return id < 0 || id == p.padding_idx ? (uint32_t)p.vocab : (uint32_t)id;
    };
    // The lanes with this lane's digit; none for a lane behind the end.
    auto same = [&](bool in, uint32_t digit) {
      return __match_any_sync(0xffffffffu, in ? digit : 0xffffffffu);
    };
    for (int i = lane; i < bins; i += 32) count[i] = 0;
    __syncwarp();
    for (int64_t i = lo; i < hi; i += 32) {
      const bool in = i + lane < hi;
      const uint32_t digit = in ? (key_at(i + lane) >> shift) & (bins - 1) : 0;
      const uint32_t m = same(in, digit);
      if (in && lane == __ffs(m) - 1) count[digit] += __popc(m);
      __syncwarp();
    }
    __syncthreads();
    if (d < bins) {
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = smem[w * bins + d];
        smem[w * bins + d] = run;
        run += n;
      }
      total[d] = run;
    }
    cluster_sync();
    uint32_t before = 0, all = 0;
    if (d < bins)
      for (int c = 0; c < p.cluster; ++c) {
        const uint32_t n = ld_peer(total + d, c);
        before += c < rank ? n : 0;
        all += n;
      }
    // entries of smaller digits: an exclusive sum over the threads
    uint32_t sum = all;
    for (int k = 1; k < 32; k <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += n;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      uint32_t s = sums[lane], own = s;
      for (int k = 1; k < 32; k <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, s, k);
        if (lane >= k) s += n;
      }
      sums[lane] = s - own;
    }
    __syncthreads();
    if (d < bins) base[d] = sums[warp] + sum - all + before;
    __syncthreads();
    uint32_t* key_out = p.key[pass & 1];
    uint32_t* token_out = p.token[pass & 1];
    for (int64_t i = lo; i < hi; i += 32) {
      const bool in = i + lane < hi;
      const uint32_t key = in ? key_at(i + lane) : 0, digit = (key >> shift) & (bins - 1);
      const uint32_t m = same(in, digit);
      const uint32_t at = in ? base[digit] + count[digit] + __popc(m & ((1u << lane) - 1)) : 0;
      __syncwarp();
      if (in) {
        if (lane == __ffs(m) - 1) count[digit] += __popc(m);
        key_out[at] = key;
        token_out[at] = pass > 0 ? __ldcg(token_in + i + lane) : (uint32_t)(i + lane);
      }
      __syncwarp();
    }
    // the target is complete before it is read; the totals, before they change
    cluster_sync();
  }
}

// ---------------------------------------------------------------------------
// backward: sums over the tokens of an id
// ---------------------------------------------------------------------------
constexpr int kPiece = 32;   // sorted entries that a warp takes
constexpr int kAhead = 8;    // of their rows loaded at a time

struct SumParams {
  const void* dy;
  const uint32_t* key;
  const uint32_t* token;
  float* open;         // [pieces][2][hidden]: sums of ids that go on before / behind a piece
  void* dweight;
  int64_t tokens, vocab;
  int hidden, accumulate;
  float scale;
};

template <bool VEC, int E, typename U>
__device__ __forceinline__ void finish(const SumParams& p, uint32_t id, int c, float (&f)[E]) {
  U* row = static_cast<U*>(p.dweight) + (int64_t)id * p.hidden;
  float g[E] = {};
  if (p.accumulate) load_row<VEC, E>(row, c, p.hidden, g);
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = p.accumulate ? fmaf(f[i], p.scale, g[i]) : f[i] * p.scale;
  store_row<VEC, E>(row, c, p.hidden, f);
}

// A warp takes 32 E columns of a piece's rows: the sum of an id whose entries
// all are in the piece goes to the table, that of one that goes on before or
// behind it to the piece's open sums.
template <typename T, typename U, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_sums(const SumParams p) {
  constexpr int E = kElems<T, U>;
  pdl_wait();
  pdl_trigger();
  const T* dy = static_cast<const T*>(p.dy);
  const int lane = threadIdx.x & 31, slabs = (p.hidden + 32 * E - 1) / (32 * E);
  const int64_t pieces = (p.tokens + kPiece - 1) / kPiece;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < pieces * slabs;
       u += (int64_t)gridDim.x * kWarps) {
    const int64_t piece = u / slabs, at = piece * kPiece;
    const int c = first_column<VEC, E>((int)(u % slabs), lane);
    const uint32_t none = (uint32_t)p.vocab;
    const uint32_t key = at + lane < p.tokens ? p.key[at + lane] : none;
    const uint32_t token = at + lane < p.tokens ? p.token[at + lane] : 0;
    const uint32_t before = at > 0 ? p.key[at - 1] : none;
    const uint32_t behind = at + kPiece < p.tokens ? p.key[at + kPiece] : none;
    uint32_t next = __shfl_down_sync(0xffffffffu, key, 1);
    if (lane == 31) next = behind;
    const int n = __popc(__ballot_sync(0xffffffffu, key < none));  // they come first
    const uint32_t ends = __ballot_sync(0xffffffffu, key != next);
    bool open_left = n > 0 && before == __shfl_sync(0xffffffffu, key, 0);
    float sum[E] = {};
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      float f[kAhead][E] = {};
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t t = __shfl_sync(0xffffffffu, token, i0 + k);
        if (i0 + k < n) load_row<VEC, E>(dy + t * p.hidden, c, p.hidden, f[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k;
        if (i >= n) break;
#pragma unroll
        for (int j = 0; j < E; ++j) sum[j] += f[k][j];
        const bool end = ends >> i & 1;
        if (!end && i + 1 < kPiece) continue;
        if (open_left || !end)
          store_row<VEC, E>(p.open + (piece * 2 + (open_left ? 0 : 1)) * p.hidden, c, p.hidden,
                            sum);
        else
          finish<VEC, E, U>(p, __shfl_sync(0xffffffffu, key, i), c, sum);
        open_left = false;
#pragma unroll
        for (int j = 0; j < E; ++j) sum[j] = 0.f;
      }
    }
  }
}

// The ids that go on over several pieces: a warp takes 32 E columns of the one
// that begins in its piece and goes on behind it, if there is one, and adds the
// pieces' open sums in order.
template <typename U, int E, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_joins(const SumParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slabs = (p.hidden + 32 * E - 1) / (32 * E);
  const int64_t pieces = (p.tokens + kPiece - 1) / kPiece;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < (pieces - 1) * slabs;
       u += (int64_t)gridDim.x * kWarps) {
    const int64_t piece = u / slabs, at = piece * kPiece;
    const uint32_t id = p.key[at + kPiece];
    if (id >= (uint32_t)p.vocab || p.key[at + kPiece - 1] != id) continue;
    if (at > 0 && p.key[at] == id && p.key[at - 1] == id) continue;  // began before
    // the last piece that begins with the id: first a look at the next ones, then halving
    int64_t last = piece + 1, out = pieces;
    const int64_t look = piece + 2 + lane;
    const bool goes_on = look < pieces && p.key[look * kPiece] == id;
    const int more = __popc(__ballot_sync(0xffffffffu, goes_on));
    last += more;
    if (more < 32) out = last + 1;
    while (out - last > 1) {
      const int64_t mid = last + (out - last) / 2;
      if (p.key[mid * kPiece] == id) last = mid;
      else out = mid;
    }
    const int c = first_column<VEC, E>((int)(u % slabs), lane);
    float sum[E] = {};
    load_row<VEC, E>(p.open + (piece * 2 + 1) * p.hidden, c, p.hidden, sum);
    for (int64_t q = piece + 1; q <= last; q += kAhead) {
      float f[kAhead][E] = {};
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (q + k <= last) load_row<VEC, E>(p.open + (q + k) * 2 * p.hidden, c, p.hidden, f[k]);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j) sum[j] += f[k][j];
    }
    finish<VEC, E, U>(p, id, c, sum);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
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

int64_t padded(int64_t tokens) { return (tokens + 3) / 4 * 4; }

size_t workspace_of(int64_t tokens, int64_t hidden) {
  return 4 * (size_t)padded(tokens) * sizeof(uint32_t) +
         2 * (size_t)ceil_div(tokens, kPiece) * (size_t)hidden * sizeof(float);
}

cudaError_t launch_sort(SortParams p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(dev);
  p.cluster = 1;
  while (p.cluster < 8 && p.cluster * 2 <= sms &&
         p.cluster * kSortThreads < p.tokens)  // a token a thread, where there are few
    p.cluster *= 2;
  int bits = 1;
  while (((int64_t)1 << bits) <= p.vocab) ++bits;  // of the ids and of `vocab` itself
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  const size_t smem = (size_t)(kSortWarps + 2) * sizeof(uint32_t) << p.bits;
  auto kern = embedding_sort;
  const size_t most = (size_t)(kSortWarps + 2) * sizeof(uint32_t) << kMaxBits;
  e = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)most);
  if (e != cudaSuccess) return e;
  int64_t clear = p.zeros > 0 ? least(ceil_div(p.zeros, 64 << 10), sms) : 0;
  clear = ceil_div(clear, p.cluster) * p.cluster;
  return launch_kernel(kern, dim3((unsigned)(p.cluster + clear)), dim3(kSortThreads), smem, s,
                       p.cluster, p);
}

}  // namespace
}  // namespace rmsn

extern "C" {

int rms_norm_embedding_fwd(const void* ids, int ids_64, const void* weight, void* y,
                           int64_t tokens, int64_t vocab, int64_t hidden, float scale,
                           int weight_dtype, int y_dtype, void* stream) {
  using namespace rmsn;
  const int st = check(tokens, vocab, hidden, scale, ids_64, weight_dtype, y_dtype);
  if (st != RMSN_OK) return st;
  begin_call();
  if (tokens == 0) return RMSN_OK;
  if (!ids || !weight || !y) return RMSN_ERR_NULL;
  const int wb = bytes_of(weight_dtype), yb = bytes_of(y_dtype), ib = ids_64 ? 8 : 4;
  if ((uintptr_t)ids % ib != 0 || (uintptr_t)weight % wb != 0 || (uintptr_t)y % yb != 0)
    return RMSN_ERR_ALIGN;
  const Span out(y, (size_t)tokens * hidden * yb);
  if (out.meets(Span(weight, (size_t)vocab * hidden * wb)) ||
      out.meets(Span(ids, (size_t)tokens * ib)))
    return RMSN_ERR_ARG;
  const Ids of = {ids, ids_64};
  const cudaError_t e = with_types(weight_dtype, y_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using U = decltype(u);
    constexpr int E = kElems<T, U>;
    const bool vec = rows_ok(weight, hidden, wb) && rows_ok(y, hidden, yb) && hidden % E == 0;
    return launch_units(vec ? embedding_rows<T, U, true> : embedding_rows<T, U, false>,
                        tokens * ceil_div(hidden, 32 * E), static_cast<cudaStream_t>(stream), of,
                        static_cast<const T*>(weight), static_cast<U*>(y), tokens, vocab,
                        (int)hidden, scale);
  });
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(1);
  return RMSN_OK;
}

size_t rms_norm_embedding_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden) {
  using namespace rmsn;
  if (tokens == 0 || check(tokens, vocab, hidden, 1.f, 0, RMSN_F32, RMSN_F32) != RMSN_OK) return 0;
  return workspace_of(tokens, hidden);
}

int rms_norm_embedding_bwd(const void* dy, const void* ids, int ids_64, void* dweight,
                           int64_t tokens, int64_t vocab, int64_t hidden, float scale,
                           int64_t padding_idx, int accumulate, int dy_dtype, int dweight_dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
  using namespace rmsn;
  const int st = check(tokens, vocab, hidden, scale, ids_64, dy_dtype, dweight_dtype);
  if (st != RMSN_OK) return st;
  if (accumulate != 0 && accumulate != 1) return RMSN_ERR_ARG;
  begin_call();
  if (!dweight) return RMSN_ERR_NULL;
  const int tb = bytes_of(dy_dtype), ub = bytes_of(dweight_dtype), ib = ids_64 ? 8 : 4;
  if ((uintptr_t)dweight % ub != 0) return RMSN_ERR_ALIGN;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const size_t table = (size_t)vocab * hidden * ub;
  if (tokens == 0) {
    const cudaError_t e = accumulate ? cudaSuccess : cudaMemsetAsync(dweight, 0, table, cs);
    return e == cudaSuccess ? RMSN_OK : cuda_fail(e);
  }
  if (!dy || !ids || !workspace) return RMSN_ERR_NULL;
  if ((uintptr_t)workspace % 16 != 0 || (uintptr_t)ids % ib != 0 || (uintptr_t)dy % tb != 0)
    return RMSN_ERR_ALIGN;
  if (workspace_bytes < workspace_of(tokens, hidden)) return RMSN_ERR_WORKSPACE;
  const Span out(dweight, table), ws(workspace, workspace_bytes);
  const Span ins[] = {{dy, (size_t)tokens * hidden * tb}, {ids, (size_t)tokens * ib}};
  if (out.meets(ws)) return RMSN_ERR_ARG;
  for (const Span& i : ins)
    if (out.meets(i) || ws.meets(i)) return RMSN_ERR_ARG;
  uint32_t* w = static_cast<uint32_t*>(workspace);
  const int64_t n = padded(tokens);
  SortParams sort = {{ids, ids_64}, tokens, vocab, padding_idx, {w, w + n}, {w + 2 * n, w + 3 * n},
                     0, 0, 1, static_cast<char*>(dweight), accumulate ? 0 : (int64_t)table};
  cudaError_t e = launch_sort(sort, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  int bits = 1;
  while (((int64_t)1 << bits) <= vocab) ++bits;
  const int last = ((bits + kMaxBits - 1) / kMaxBits - 1) & 1;  // where the last pass wrote
  SumParams sum = {dy, sort.key[last], sort.token[last], reinterpret_cast<float*>(w + 4 * n),
                   dweight, tokens, vocab, (int)hidden, accumulate, scale};
  const int64_t pieces = ceil_div(tokens, kPiece);
  int launches = 1;
  e = with_types(dy_dtype, dweight_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using U = decltype(u);
    constexpr int E = kElems<T, U>;
    const bool vec = rows_ok(dy, hidden, tb) && rows_ok(dweight, hidden, ub) && hidden % E == 0;
    const int64_t slabs = ceil_div(hidden, 32 * E);
    cudaError_t r = launch_units(vec ? embedding_sums<T, U, true> : embedding_sums<T, U, false>,
                                 pieces * slabs, cs, sum);
    if (r != cudaSuccess) return r;
    ++launches;
    if (pieces > 1) {
      r = launch_units(vec ? embedding_joins<U, E, true> : embedding_joins<U, E, false>,
                       (pieces - 1) * slabs, cs, sum);
      if (r == cudaSuccess) ++launches;
    }
    return r;
  });
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(launches);
  return RMSN_OK;
}

}  // extern "C"
