// Embedding, backward: the table's gradient, summed over the tokens of each id
// in their order.
//
// Up to kFew tokens one kernel does it all: every CTA has the ids in shared
// memory, and the warp of an id's first token looks the others up.  Beyond, a
// cluster of CTAs sorts the tokens by id (embedding_sort); warps then sum pieces
// of up to 32 sorted entries (embedding_sums): an id whose entries all lie in a piece
// is done, of one that goes on the piece's part is kept as an open sum, and a
// third kernel adds those (embedding_joins).  No atomics: an element's order of
// additions is fixed by the ids.
//
// What bounds it is memory: dy is read once, and, unless the caller accumulates,
// every row of the table is written.  The rows without a token are cleared by
// warps of their own beside the sort, the sums and the joins, whose latencies
// this hides.
#include "cluster_launch.cuh"
#include "embedding.cuh"
#include "pairs.cuh"

namespace rmsn {
namespace {

// A lane's E elements of a row, as they were loaded.  VEC: runs of R elements, 8
// or 16 bytes of the narrower type, that lie 32 R columns apart, from column c
// on; else every 32nd one.
template <typename T, int E, int R, bool VEC>
struct Slice {
  static constexpr int N = E * sizeof(T) / 8;  // 8-byte words
  uint2 v[VEC ? N : 1];
  T e[VEC ? 1 : E];
  __device__ __forceinline__ void load(const T* row, int c, int hidden) {
    if constexpr (VEC) {
      constexpr int M = R * sizeof(T) / 8;     // words of a run
#pragma unroll
      for (int r = 0; r < E / R; ++r) {
        const int at = c + 32 * R * r;
        if constexpr (M == 1) {
          v[r] = at < hidden ? *reinterpret_cast<const uint2*>(row + at) : make_uint2(0, 0);
        } else {
#pragma unroll
          for (int k = 0; k < M / 2; ++k) {
            const uint4 q = at < hidden ? *(reinterpret_cast<const uint4*>(row + at) + k)
                                        : make_uint4(0, 0, 0, 0);
            v[r * M + 2 * k] = make_uint2(q.x, q.y);
            v[r * M + 2 * k + 1] = make_uint2(q.z, q.w);
          }
        }
      }
    } else if (c + 32 * (E - 1) < hidden) {  // all of them: no test for each
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = row[c + 32 * i];
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = c + 32 * i < hidden ? row[c + 32 * i] : Traits<T>::from_f(0.f);
    }
  }
  __device__ __forceinline__ void get(f32x2 (&f)[E / 2]) const {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) f[i] = pair(Traits<T>::to_f(e[2 * i]), Traits<T>::to_f(e[2 * i + 1]));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = pair(__uint_as_float(v[k].x), __uint_as_float(v[k].y));
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        f[2 * k] = widen<T>(v[k].x);
        f[2 * k + 1] = widen<T>(v[k].y);
      }
    }
  }
};

template <bool VEC, int E, int R, typename U>
__device__ __forceinline__ void store_slice(U* row, int c, int hidden, const f32x2 (&f)[E / 2]) {
  if constexpr (VEC) {
    constexpr int P = R / 2;                   // pairs of a run
#pragma unroll
    for (int r = 0; r < E / R; ++r) {
      const int at = c + 32 * R * r;
      if (at >= hidden) continue;
      if constexpr (sizeof(U) == 4) {
#pragma unroll
        for (int k = 0; k < P; k += 2) {
          const float2 a = split(f[r * P + k]), b = split(f[r * P + k + 1]);
          st_vec(row + at + 2 * k, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y),
                                              __float_as_uint(b.x), __float_as_uint(b.y)));
        }
      } else if constexpr (P == 4) {
        st_vec(row + at, make_uint4(narrow<U>(f[r * P]), narrow<U>(f[r * P + 1]),
                                    narrow<U>(f[r * P + 2]), narrow<U>(f[r * P + 3])));
      } else {
        *reinterpret_cast<uint2*>(row + at) = make_uint2(narrow<U>(f[r * P]), narrow<U>(f[r * P + 1]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 v = split(f[i]);
      if (c + 64 * i < hidden) row[c + 64 * i] = Traits<U>::from_f(v.x);
      if (c + 64 * i + 32 < hidden) row[c + 64 * i + 32] = Traits<U>::from_f(v.y);
    }
  }
}

// The first of a lane's columns in slab `slab` of 32 E columns.
template <int E, int R, bool VEC>
__device__ __forceinline__ int column(int slab, int lane) {
  return slab * 32 * E + (VEC ? lane * R : lane);
}

struct SumParams {
  const void* dy;
  Ids ids;
  const uint2* sorted;    // (id, token) in order, id `vocab` for those without a part
  int piece;              // sorted entries that a warp takes
  int look;               // pieces that a warp of the joins looks at
  float* open;            // [pieces][2][hidden]: sums of ids that go on before / behind a piece
  void* dweight;
  int64_t tokens, vocab, padding_idx;
  int64_t clear0, clear1; // rows of the table that this kernel's clearing warps look after
  int hidden, accumulate;
  float scale;
};

// A sum as the row of its id; `was`: that row, where the caller accumulates.
template <bool VEC, int E, int R, typename U>
__device__ __forceinline__ void finish(const SumParams& p, uint32_t id, int c,
                                       const Slice<U, E, R, VEC>& was, f32x2 (&f)[E / 2]) {
  const f32x2 scale = pair(p.scale, p.scale);
  if (p.accumulate) {
    f32x2 g[E / 2];
    was.get(g);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) f[i] = fma2(f[i], scale, g[i]);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) f[i] = mul2(f[i], scale);
  }
  store_slice<VEC, E, R>(static_cast<U*>(p.dweight) + (int64_t)id * p.hidden, c, p.hidden, f);
}

// ---------------------------------------------------------------------------
// rows without a token
// ---------------------------------------------------------------------------
constexpr int kBits = 4096;   // rows whose tokens are looked at together

// A warp clears those of `rows` rows, from `table` on, whose bit is not set, a
// run of them at a time, in 16-byte stores but for its ends.
template <typename U>
__device__ __forceinline__ void clear_unmarked(U* table, int hidden, const uint32_t* bits, int rows,
                                               int lane) {
  for (int r = 0; r < rows;) {
    const uint32_t w = bits[r >> 5] >> (r & 31);
    if (w & 1) {  // rows with tokens
      r += w == 0xffffffffu ? 32 : __ffs(~w) - 1;
      continue;
    }
    int e = r;    // rows without, up to e
    while (e < rows) {
      const uint32_t v = bits[e >> 5] >> (e & 31);
      if (v) {
        e += __ffs(v) - 1;
        break;
      }
      e = (e | 31) + 1;
    }
    if (e > rows) e = rows;
    U* to = table + (int64_t)r * hidden;
    int64_t n = (int64_t)(e - r) * hidden;
    constexpr int W = 16 / sizeof(U);
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(to) & 15)) & 15) / sizeof(U);
    if (head > n) head = n;
    if (lane < head) to[lane] = Traits<U>::from_f(0.f);
    to += head;
    n -= head;
    const int64_t vecs = n / W;
#pragma unroll 4
    for (int64_t i = lane; i < vecs; i += 32) st_vec(to + i * W, make_uint4(0, 0, 0, 0));
    if (vecs * W + lane < n) to[vecs * W + lane] = Traits<U>::from_f(0.f);
    r = e;
  }
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
// Where looking the tokens up takes less time than sorting them: 200 x 1024 bf16 added
// to fp32 4.8 us so, 14.4 sorted, 500 x 1024 8.3 and 15.2; 1000 x 1024 15.8 and 16.5,
// 1000 x 4096 22.0 and 17.9.
constexpr int kFew = 512;

template <typename T, typename U, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_few(const SumParams p) {
  constexpr int E = kElems<T, U>, A = 8;
  __shared__ int id[kFew];
  __shared__ unsigned short list[kWarps][kFew];
  __shared__ uint32_t bits[kWarps][kBits / 32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)p.tokens;
  for (int i = threadIdx.x; i < kFew; i += kThreads) {
    const int k = i < n ? p.ids.get(i, p.vocab) : -1;
    id[i] = k == p.padding_idx ? -1 : k;
  }
  __syncthreads();
  U* table = static_cast<U*>(p.dweight);
  if (!p.accumulate) {  // this warp's rows without a token
    const int64_t number = (int64_t)blockIdx.x * kWarps + warp, warps = (int64_t)gridDim.x * kWarps;
    const int64_t r0 = p.vocab * number / warps, r1 = p.vocab * (number + 1) / warps;
    for (int64_t base = r0; base < r1; base += kBits) {
      const int rows = (int)(r1 - base < kBits ? r1 - base : kBits);
      for (int i = lane; i < (rows + 31) / 32; i += 32) bits[warp][i] = 0;
      __syncwarp();
      for (int i = lane; i < n; i += 32) {
        const int64_t at = id[i] - base;
        if (id[i] >= 0 && at >= 0 && at < rows) atomicOr(&bits[warp][at >> 5], 1u << (at & 31));
      }
      __syncwarp();
      clear_unmarked(table + base * p.hidden, p.hidden, bits[warp], rows, lane);
      __syncwarp();
    }
  }
  const T* dy = static_cast<const T*>(p.dy);
  const int slabs = (p.hidden + 32 * E - 1) / (32 * E);
  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < (int64_t)n * slabs;
       u += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(u / slabs), k = id[t];
    if (k < 0) continue;
    bool first = true;
    for (int j = 0; j < t && first; j += 32)
      first = !__any_sync(0xffffffffu, j + lane < t && id[j + lane] == k);
    if (!first) continue;
    int count = 0;
    for (int j = t / 32 * 32; j < n; j += 32) {
      const bool mine = id[j + lane] == k;  // -1 behind the tokens
      const uint32_t m = __ballot_sync(0xffffffffu, mine);
      if (mine) list[warp][count + __popc(m & ((1u << lane) - 1))] = (unsigned short)(j + lane);
      count += __popc(m);
    }
    __syncwarp();
    const int c = column<E, E, VEC>((int)(u % slabs), lane);
    Slice<U, E, E, VEC> was;
    if (p.accumulate) was.load(table + (int64_t)k * p.hidden, c, p.hidden);
    f32x2 sum[E / 2] = {};
    for (int i0 = 0; i0 < count; i0 += A) {
      Slice<T, E, E, VEC> s[A];
#pragma unroll
      for (int i = 0; i < A; ++i)
        if (i0 + i < count) s[i].load(dy + (int64_t)list[warp][i0 + i] * p.hidden, c, p.hidden);
#pragma unroll
      for (int i = 0; i < A; ++i) {
        if (i0 + i >= count) break;
        f32x2 f[E / 2];
        s[i].get(f);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) sum[j] = add2(sum[j], f[j]);
      }
    }
    finish<VEC, E, E, U>(p, k, c, was, sum);
    __syncwarp();  // the list gives way to the next
  }
}

// ---------------------------------------------------------------------------
// tokens sorted by id
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortCluster = 16;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 10;  // of a digit: two bins a thread
constexpr int kHeld = 16;     // entries of a lane loaded at a time

struct SortParams {
  Ids ids;
  int64_t tokens, vocab, padding_idx;
  uint2* items[2];     // (id, token), in turn the source and the target of a pass
  int passes, bits;    // digits, and bits of each
  int cluster;
  char* zero;          // the rows of the table that this kernel clears: `zeros` bytes
  int64_t zeros;
};

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
// behind theirs.  The launch's other clusters clear rows of the table meanwhile.
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
    const bool odd = pass & 1;
    const uint2* from_items = odd ? p.items[0] : p.items[1];
    // This lane's next entries, all of their loads under way together.
    uint2 item[kHeld];
    uint32_t peers[kHeld];
    auto take = [&](int64_t from) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        if (from + 32 * k >= hi) break;
        const int64_t i = from + 32 * k + lane;
        item[k] = make_uint2(0, 0);
        if (i >= hi) continue;
        if (pass > 0) {
          item[k] = __ldcg(from_items + i);  // another CTA's: not through this SM's L1
        } else {
          const int id = p.ids.get(i, p.vocab);
          item[k].x = id < 0 || id == p.padding_idx ? (uint32_t)p.vocab : (uint32_t)id;
          item[k].y = (uint32_t)i;
        }
      }
    };
    // The lanes with this lane's digit; a lane behind the end has none.
    auto same = [&](bool in, uint32_t digit) {
      return __match_any_sync(0xffffffffu, in ? digit : 0xffffffffu);
    };
    for (int i = lane; i < bins; i += 32) count[i] = 0;
    __syncwarp();
    for (int64_t from = lo; from < hi; from += 32 * kHeld) {
      take(from);
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        if (from + 32 * k >= hi) break;
        const bool in = from + 32 * k + lane < hi;
        const uint32_t digit = (item[k].x >> shift) & (bins - 1), m = same(in, digit);
        if (in && lane == __ffs(m) - 1) count[digit] += __popc(m);
        peers[k] = m;
        __syncwarp();
      }
    }
    __syncthreads();
    // the thread's two bins, 2 d and 2 d + 1, of at least two
    uint2 before = make_uint2(0, 0), all = make_uint2(0, 0);
    if (2 * d < bins) {
      uint2 run = make_uint2(0, 0);
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        uint2* at = reinterpret_cast<uint2*>(smem + w * bins) + d;
        const uint2 n = *at;
        *at = run;
        run.x += n.x;
        run.y += n.y;
      }
      reinterpret_cast<uint2*>(total)[d] = run;
    }
    cluster_sync();
    if (2 * d < bins) {
      uint32_t n[2][kSortCluster];
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        n[0][c] = c < p.cluster ? ld_peer(total + 2 * d, c) : 0;
        n[1][c] = c < p.cluster ? ld_peer(total + 2 * d + 1, c) : 0;
      }
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        before.x += c < rank ? n[0][c] : 0;
        before.y += c < rank ? n[1][c] : 0;
        all.x += n[0][c];
        all.y += n[1][c];
      }
    }
    // entries of smaller digits: an exclusive sum over the threads
    const uint32_t own = all.x + all.y;
    uint32_t sum = own;
    for (int k = 1; k < 32; k <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += n;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      uint32_t s = lane < kSortWarps ? sums[lane] : 0;
      const uint32_t mine = s;
      for (int k = 1; k < 32; k <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, s, k);
        if (lane >= k) s += n;
      }
      sums[lane] = s - mine;
    }
    __syncthreads();
    if (2 * d < bins) {
      const uint32_t smaller = sums[warp] + sum - own;
      reinterpret_cast<uint2*>(base)[d] = make_uint2(smaller + before.x, smaller + all.x + before.y);
    }
    __syncthreads();
    uint2* to_items = odd ? p.items[1] : p.items[0];
    for (int64_t from = lo; from < hi; from += 32 * kHeld) {
      const bool held = share <= 32 * kHeld;  // they are there
      if (!held) take(from);
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        if (from + 32 * k >= hi) break;
        const bool in = from + 32 * k + lane < hi;
        const uint32_t digit = (item[k].x >> shift) & (bins - 1);
        const uint32_t m = held ? peers[k] : same(in, digit);
        const uint32_t at = in ? base[digit] + count[digit] + __popc(m & ((1u << lane) - 1)) : 0;
        __syncwarp();
        if (in) {
          if (lane == __ffs(m) - 1) count[digit] += __popc(m);
          to_items[at] = item[k];
        }
        __syncwarp();
      }
    }
    // the target is complete before it is read; the totals, before they change
    cluster_sync();
  }
}

// The first i of [lo, hi) with test(i), hi where there is none, by a whole warp;
// from one i on the test holds.
template <typename F>
__device__ __forceinline__ int64_t first_of(int64_t lo, int64_t hi, int lane, F test) {
  while (lo < hi) {
    const int64_t at = lo + (hi - lo) * (lane + 1) / 33;
    const int below = __popc(__ballot_sync(0xffffffffu, !test(at)));
    const int64_t next = __shfl_sync(0xffffffffu, at, below < 32 ? below : 31);
    const int64_t prev = __shfl_sync(0xffffffffu, at, below > 0 ? below - 1 : 0);
    if (below > 0) lo = prev + 1;
    if (below < 32) hi = next;
  }
  return lo;
}

// The first of the sorted ids that is not below `id`.
__device__ __forceinline__ int64_t first_not_below(const SumParams& p, uint32_t id, int lane) {
  return first_of(0, p.tokens, lane, [&](int64_t i) { return p.sorted[i].x >= id; });
}

// One of `warps` warps clears its part of the rows [clear0, clear1) that no
// token has.  bits: kBits / 32 words of shared memory.  The parts are even in rows
// and 32nds of their tokens together, which a warp goes through: by rows alone the
// one of the most frequent ids ends last (89591 tokens of 142402 ids, 384 columns
// 203 us, 95 so).
template <typename U>
__device__ __forceinline__ void clear_rows(const SumParams& p, uint32_t* bits, int64_t number,
                                           int64_t warps, int lane) {
  const int64_t rows_all = p.clear1 - p.clear0;
  if (rows_all <= 0) return;
  const int64_t j0 = first_not_below(p, (uint32_t)p.clear0, lane) / 32;
  const int64_t j1 = first_not_below(p, (uint32_t)p.clear1, lane) / 32, all = rows_all + j1 - j0;
  // the least number of rows that makes x with the 32nds below the next row
  auto split = [&](int64_t x) {
    const int64_t least = x - (j1 - j0) > 0 ? x - (j1 - j0) : 0;
    return p.clear0 + first_of(least, x < rows_all ? x : rows_all, lane, [&](int64_t i) {
      const int64_t j = x - i;
      return j <= 0 || (int64_t)p.sorted[(j0 + j - 1) * 32].x < p.clear0 + i;
    });
  };
  const int64_t r0 = split(all * number / warps), r1 = split(all * (number + 1) / warps);
  for (int64_t base = r0; base < r1; base += kBits) {
    const int rows = (int)(r1 - base < kBits ? r1 - base : kBits);
    const uint32_t end = (uint32_t)(base + rows);
    for (int i = lane; i < (rows + 31) / 32; i += 32) bits[i] = 0;
    __syncwarp();
    // eight of a lane's ids under way together: frequent ones have thousands of tokens
    for (int64_t i = first_not_below(p, (uint32_t)base, lane) + lane;; i += 256) {
      uint32_t key[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        key[k] = i + 32 * k < p.tokens ? p.sorted[i + 32 * k].x : 0xffffffffu;
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // of equal neighbours one
        const uint32_t before = __shfl_up_sync(0xffffffffu, key[k], 1);
        const uint32_t at = key[k] - (uint32_t)base;
        if (key[k] < end && (lane == 0 || key[k] != before))
          atomicOr(&bits[at >> 5], 1u << (at & 31));
      }
      if (!__all_sync(0xffffffffu, key[7] < end)) break;
    }
    __syncwarp();
    clear_unmarked(static_cast<U*>(p.dweight) + base * p.hidden, p.hidden, bits, rows, lane);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// sums over the tokens of an id
// ---------------------------------------------------------------------------
constexpr int kPiece = 32;                 // sorted entries that a warp takes at most
constexpr int kSumThreads = kThreads + 32; // and a warp that clears
constexpr int kSumCtas = 2;                // an SM

// A warp takes 32 E columns of a piece's rows: the sum of an id whose entries
// all are in the piece goes to the table, that of one that goes on before or
// behind it to the piece's open sums.
template <typename T, typename U, int E, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumThreads, kSumCtas) embedding_sums(const SumParams p) {
  constexpr int R = kElems<T, U>, A = (ACC ? 32 : 64) / E;  // rows loaded at a time
  __shared__ uint32_t bits[kBits / 32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == kWarps) {
    if constexpr (!ACC) clear_rows<U>(p, bits, blockIdx.x, gridDim.x, lane);
    return;
  }
  const T* dy = static_cast<const T*>(p.dy);
  const U* table = static_cast<const U*>(p.dweight);
  const int slabs = (p.hidden + 32 * E - 1) / (32 * E);
  const int64_t pieces = (p.tokens + p.piece - 1) / p.piece;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < pieces * slabs;
       u += (int64_t)gridDim.x * kWarps) {
    const int64_t piece = u / slabs, at = piece * p.piece;
    const int c = column<E, R, VEC>((int)(u - piece * slabs), lane);
    const uint32_t none = (uint32_t)p.vocab;
    const bool in = lane < p.piece && at + lane < p.tokens;
    const uint2 item = in ? p.sorted[at + lane] : make_uint2(none, 0);
    const uint32_t key = item.x, token = item.y;
    const uint32_t before = at > 0 ? p.sorted[at - 1].x : none;
    const uint32_t behind = at + p.piece < p.tokens ? p.sorted[at + p.piece].x : none;
    uint32_t next = __shfl_down_sync(0xffffffffu, key, 1);
    if (lane == p.piece - 1) next = behind;
    const int n = __popc(__ballot_sync(0xffffffffu, key < none));  // they come first
    const uint32_t ends = __ballot_sync(0xffffffffu, key != next);
    const bool open_left = n > 0 && before == __shfl_sync(0xffffffffu, key, 0);
    // entries whose id is done with them: ends, but of the id that began before
    const uint32_t done = open_left ? ends & (ends - 1) : ends;
    bool left = open_left;
    f32x2 sum[E / 2] = {};
    for (int i0 = 0; i0 < n; i0 += A) {
      Slice<T, E, R, VEC> s[A];
      Slice<U, E, R, VEC> was[ACC ? A : 1];
#pragma unroll
      for (int k = 0; k < A; ++k) {
        const int64_t t = __shfl_sync(0xffffffffu, token, i0 + k);
        if (i0 + k < n) s[k].load(dy + t * p.hidden, c, p.hidden);
        if constexpr (ACC) {
          const int64_t id = __shfl_sync(0xffffffffu, key, i0 + k);
          if (i0 + k < n && (done >> (i0 + k) & 1)) was[k].load(table + id * p.hidden, c, p.hidden);
        }
      }
#pragma unroll
      for (int k = 0; k < A; ++k) {
        const int i = i0 + k;
        if (i >= n) break;
        f32x2 f[E / 2];
        s[k].get(f);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) sum[j] = add2(sum[j], f[j]);
        const bool end = ends >> i & 1;
        if (!end && i + 1 < p.piece) continue;
        if (left || !end)
          store_slice<VEC, E, R>(p.open + (piece * 2 + (left ? 0 : 1)) * p.hidden, c, p.hidden,
                                 sum);
        else
          finish<VEC, E, R, U>(p, __shfl_sync(0xffffffffu, key, i), c, was[ACC ? k : 0], sum);
        left = false;
#pragma unroll
        for (int j = 0; j < E / 2; ++j) sum[j] = 0;
      }
    }
  }
}

constexpr int kJoinCtas = 3, kJoinAhead = 8;  // CTAs an SM, open sums loaded at a time
constexpr int kLong = 32;                     // pieces of an id that a CTA's warps share

// The open sums of the pieces [from, to), added in order to sum.
template <bool VEC>
__device__ __forceinline__ void add_open(const SumParams& p, int64_t from, int64_t to, int c,
                                         f32x2 (&sum)[2]) {
  for (int64_t q = from; q < to; q += kJoinAhead) {
    Slice<float, 4, 4, VEC> s[kJoinAhead];
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k)
      if (q + k < to) s[k].load(p.open + (q + k) * 2 * p.hidden, c, p.hidden);
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      if (q + k >= to) break;
      f32x2 f[2];
      s[k].get(f);
      sum[0] = add2(sum[0], f[0]);
      sum[1] = add2(sum[1], f[1]);
    }
  }
}

// The ids that go on over several pieces: a warp looks at p.look pieces (32 at
// most), takes 128 columns of each id that begins in one and goes on behind it,
// and adds the pieces' open sums in order.  TEAM, for narrow rows: all warps of
// a CTA look at the same pieces and share the ids; one of many pieces they add
// together, a run of them each, and then their sums in order.
template <typename U, bool VEC, bool TEAM>
__global__ void __launch_bounds__(kSumThreads, kJoinCtas) embedding_joins(const SumParams p) {
  constexpr int E = 4;
  __shared__ uint32_t bits[kBits / 32];
  __shared__ float4 part[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == kWarps) {
    if (!p.accumulate) clear_rows<U>(p, bits, blockIdx.x, gridDim.x, lane);
    return;
  }
  // of the warps that add, not of the one that clears
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  const U* table = static_cast<const U*>(p.dweight);
  const int slabs = (p.hidden + 32 * E - 1) / (32 * E);
  const int64_t pieces = (p.tokens + p.piece - 1) / p.piece;
  const int64_t looks = (pieces - 1 + p.look - 1) / p.look;
  for (int64_t u = TEAM ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp; u < looks * slabs;
       u += TEAM ? gridDim.x : (int64_t)gridDim.x * kWarps) {
    const int64_t look = u / slabs, mine = look * p.look + lane;
    const int c = column<E, E, VEC>((int)(u - look * slabs), lane);
    uint32_t key = (uint32_t)p.vocab;  // of the id that begins in piece `mine` and goes on
    if (lane < p.look && mine + 1 < pieces) {
      const int64_t at = mine * p.piece;
      const uint32_t id = p.sorted[at + p.piece].x, end = p.sorted[at + p.piece - 1].x;
      const uint32_t first = p.sorted[at].x, before = at > 0 ? p.sorted[at - 1].x : (uint32_t)p.vocab;
      if (end == id && !(first == id && before == id)) key = id;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, key < (uint32_t)p.vocab);
    for (int turn = 0; todo; todo &= todo - 1, ++turn) {
      const int who = __ffs(todo) - 1;
      const int64_t piece = look * p.look + who;
      const uint32_t id = __shfl_sync(0xffffffffu, key, who);
      // pieces behind this one that begin with the id: a look at the next ones, then halving
      const int64_t ahead = piece + 2 + lane;
      const bool goes_on = ahead < pieces && p.sorted[ahead * p.piece].x == id;
      const int more = __popc(__ballot_sync(0xffffffffu, goes_on));
      int64_t end = piece + 2 + more;
      if (more == 32) {
        int64_t out = pieces + 1;  // the last such piece is end - 1, and before out - 1
        while (out - end > 1) {
          const int64_t mid = end + (out - end) / 2;
          if (p.sorted[(mid - 1) * p.piece].x == id) end = mid;
          else out = mid;
        }
      }
      const bool together = TEAM && end - piece - 1 >= kLong;  // the same for every warp
      if (TEAM && !together && turn % kWarps != warp) continue;
      const bool last = !together || warp == 0;        // the warp that has the sum
      Slice<U, E, E, VEC> was;
      if (last && p.accumulate) was.load(table + (int64_t)id * p.hidden, c, p.hidden);
      f32x2 sum[2] = {};
      if (last) {
        Slice<float, E, E, VEC> s;
        s.load(p.open + (piece * 2 + 1) * p.hidden, c, p.hidden);
        s.get(sum);
      }
      const int64_t n = end - piece - 1;
      add_open<VEC>(p, piece + 1 + (together ? n * warp / kWarps : 0),
                    piece + 1 + (together ? n * (warp + 1) / kWarps : n), c, sum);
      if (together) {
        const float2 a = split(sum[0]), b = split(sum[1]);
        part[warp][lane] = make_float4(a.x, a.y, b.x, b.y);
        sync();
        if (warp == 0)
          for (int w = 1; w < kWarps; ++w) {
            const float4 f = part[w][lane];
            sum[0] = add2(sum[0], pair(f.x, f.y));
            sum[1] = add2(sum[1], pair(f.z, f.w));
          }
        sync();  // the sums give way to the next id's
      }
      if (last) finish<VEC, E, E, U>(p, id, c, was, sum);
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
int64_t padded(int64_t tokens) { return (tokens + 1) / 2 * 2; }

// Elements of a row that a lane of the sums takes: two vectors of a wide row, whose
// joins a warp takes by itself.  Of bf16 rows added to fp32, 8192 x 2048 take 36.1 us
// with one vector and 33.3 with two, 32768 x 2048 82.1 and 76.1; 8192 x 512 19.9 and
// 26.2, 32768 x 768 48.1 and 50.4.  (Rows of 1024 itself are better off with one: 22.7
// and 28.7, 51.8 and 53.2.)
bool wide(int64_t hidden) { return hidden >= 1024; }

// Entries of a piece: fewer where there would be fewer pieces than warps, as joining
// them costs less than an idle SM does.  With 8, 16 and 32 of them 600 x 4096 bf16
// added to fp32 takes 17.2, 21.3 and 28.5 us, 8192 x 4096 53.1, 46.9 and 45.7, 32768 x
// 4096 165, 124 and 114.  The bounds (16 warps of a GB300's 152 SMs, and 512 pieces
// whatever the width) are numbers and not the device's SMs: a row's terms are added in
// an order that neither the GPU nor an SM budget changes.
int piece_of(int64_t tokens, int64_t hidden) {
  const int64_t slabs = ceil_div(hidden, wide(hidden) ? 512 : 256);
  int piece = kPiece;
  while (piece > 8 && ceil_div(tokens, piece) < 512 && ceil_div(tokens, piece) * slabs < 2432)
    piece /= 2;
  return piece;
}

size_t workspace_of(int64_t tokens, int64_t hidden) {
  if (tokens <= kFew) return 0;
  return 2 * (size_t)padded(tokens) * sizeof(uint2) +
         2 * (size_t)ceil_div(tokens, piece_of(tokens, hidden)) * (size_t)hidden * sizeof(float);
}

// Bits of the ids and of `vocab` itself.
int bits_of(int64_t vocab) {
  int bits = 1;
  while (((int64_t)1 << bits) <= vocab) ++bits;
  return bits;
}

cudaError_t launch_sort(SortParams& p, int sms, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  p.cluster = 1;
  while (p.cluster < kSortCluster && p.cluster * 2 <= sms &&
         p.cluster * kSortThreads < p.tokens)  // a token a thread, where there are few
    p.cluster *= 2;
  const int bits = bits_of(p.vocab);
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  const size_t smem = (size_t)(kSortWarps + 2) * sizeof(uint32_t) << p.bits;
  const size_t most = (size_t)(kSortWarps + 2) * sizeof(uint32_t) << kMaxBits;
  if (e == cudaSuccess) e = allow_launch<embedding_sort>(dev, most);
  if (e != cudaSuccess) return e;
  // the other SMs clear; whole clusters, one at least
  int64_t clear = p.zeros > 0 ? least(ceil_div(p.zeros, 64 << 10), sms - p.cluster) : 0;
  if (p.zeros > 0 && clear < 1) clear = 1;
  clear = ceil_div(clear, p.cluster) * p.cluster;
  return launch_kernel(embedding_sort, dim3((unsigned)(p.cluster + clear)), dim3(kSortThreads),
                       smem, s, p.cluster, p);
}

// Where the rows are cleared: as many bytes beside the sort, which takes longer
// for more tokens, and beside the joins as those take time, the rest beside the
// sums.  With 64 MB beside any sort and 100 beside the joins 89591 tokens of 142402
// ids of 384 columns take 90 us, 86 so; 11826 of 23462 of 4075 111 and 107; 600 of
// 50000 of 768 33.1 and 32.3; 32768 of 32000 of 4096 bf16 111 and 113.
constexpr int64_t kClearSort = 40 << 20, kClearToken = 1024, kClearJoins = 64 << 20;

template <typename T, typename U, bool VEC>
cudaError_t launch_sums(SortParams& sort, SumParams& p, cudaStream_t s, int* launches) {
  constexpr int E = kElems<T, U>;
  p.piece = piece_of(p.tokens, p.hidden);
  const int64_t pieces = ceil_div(p.tokens, p.piece), row = (int64_t)p.hidden * sizeof(U);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(dev);
  if (p.tokens <= kFew) {
    auto kern = embedding_few<T, U, VEC>;
    const int64_t work = ceil_div(p.tokens * ceil_div(p.hidden, 32 * E), kWarps);
    const int64_t rows = p.accumulate ? 0 : ceil_div(p.vocab * row, 32 << 10);
    const int64_t ctas = work > rows ? work : rows;
    const int64_t most = (int64_t)sms * max_blocks_per_sm((const void*)kern, kThreads, 0);
    e = launch_kernel(kern, dim3((unsigned)least(ctas, most)), dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess) ++*launches;
    return e;
  }
  // Beside the sums the first rows are cleared, beside the joins the next ones, and
  // beside the sort the last, with the tokens' among them: where ids go by
  // frequency those are few there.
  const int64_t sorts = least((kClearSort + p.tokens * kClearToken) / row, p.vocab);
  const int64_t rest = p.vocab - sorts;
  const int64_t joins = least(kClearJoins / row, rest);
  sort.zero = static_cast<char*>(p.dweight) + rest * row;
  sort.zeros = p.accumulate ? 0 : sorts * row;
  e = launch_sort(sort, sms, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  p.sorted = sort.items[(sort.passes - 1) & 1];  // where the last pass wrote
  p.clear0 = 0;
  p.clear1 = rest - joins;
  constexpr int W = VEC ? 2 * E : E;
  const bool two = VEC && wide(p.hidden);
  auto sums = p.accumulate ? two ? embedding_sums<T, U, W, VEC, true>
                                 : embedding_sums<T, U, E, VEC, true>
                           : two ? embedding_sums<T, U, W, VEC, false>
                                 : embedding_sums<T, U, E, VEC, false>;
  auto launch = [&](auto kern, int64_t units, int64_t clears) {
    const int64_t most = (int64_t)sms * max_blocks_per_sm((const void*)kern, kSumThreads, 0);
    int64_t ctas = ceil_div(units, kWarps);
    if (clears > ctas) ctas = clears;
    return launch_kernel(kern, dim3((unsigned)least(ctas, most)), dim3(kSumThreads), 0, s, 1, p);
  };
  auto clears = [&]() {
    return p.accumulate ? 0 : ceil_div((p.clear1 - p.clear0) * row, 64 << 10);
  };
  e = launch(sums, pieces * ceil_div(p.hidden, 32 * (two ? W : E)), clears());
  if (e != cudaSuccess) return e;
  ++*launches;
  p.clear0 = rest - joins;
  p.clear1 = rest;
  if (pieces > 1) {
    const bool team = !wide(p.hidden);
    const int64_t slabs = ceil_div(p.hidden, 128);
    const int64_t lookers = (int64_t)sms * kJoinCtas * (team ? 1 : kWarps);
    p.look = (int)least(ceil_div((pieces - 1) * slabs, lookers), 32);
    const int64_t units = ceil_div(pieces - 1, p.look) * slabs;
    e = team ? launch(embedding_joins<U, VEC, true>, units * kWarps, clears())
             : launch(embedding_joins<U, VEC, false>, units, clears());
    if (e == cudaSuccess) ++*launches;
  }
  return e;
}

}  // namespace
}  // namespace rmsn

extern "C" {

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
  const size_t need = workspace_of(tokens, hidden);
  if (!dy || !ids || (need > 0 && !workspace)) return RMSN_ERR_NULL;
  if ((uintptr_t)workspace % 16 != 0 || (uintptr_t)ids % ib != 0 || (uintptr_t)dy % tb != 0)
    return RMSN_ERR_ALIGN;
  if (workspace_bytes < need) return RMSN_ERR_WORKSPACE;
  const Span out(dweight, table), ws(need > 0 ? workspace : nullptr, workspace_bytes);
  const Span ins[] = {{dy, (size_t)tokens * hidden * tb}, {ids, (size_t)tokens * ib}};
  if (out.meets(ws)) return RMSN_ERR_ARG;
  for (const Span& i : ins)
    if (out.meets(i) || ws.meets(i)) return RMSN_ERR_ARG;
  uint2* w = static_cast<uint2*>(workspace);
  const int64_t n = padded(tokens);
  SortParams sort = {{ids, ids_64}, tokens, vocab, padding_idx, {w, w + n}, 0, 0, 1,
                     nullptr, 0};
  SumParams sum = {dy, {ids, ids_64}, nullptr, 0, 0, reinterpret_cast<float*>(w + 2 * n),
                   dweight, tokens, vocab, padding_idx, 0, 0, (int)hidden, accumulate, scale};
  int launches = 0;
  const cudaError_t e = with_types(dy_dtype, dweight_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using U = decltype(u);
    const bool vec =
        rows_ok(dy, hidden, tb) && rows_ok(dweight, hidden, ub) && hidden % kElems<T, U> == 0;
    return vec ? launch_sums<T, U, true>(sort, sum, cs, &launches)
               : launch_sums<T, U, false>(sort, sum, cs, &launches);
  });
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(launches);
  return RMSN_OK;
}

}  // extern "C"
