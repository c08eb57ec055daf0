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
constexpr int kMaxSplit = 8;      // CTAs a row is split over
constexpr int kSmemBudget = 224 * 1024;

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

// A team's waits are short: a few tries before the bounded wait with its
// timer and its sleeps.
constexpr int kTries = 64;

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool done = false;
  for (int i = 0; i < kTries && !done; ++i) done = mbar_try_wait(bar, parity);
  if (!done) done = wait_phase_counted(bar, parity, abort, &g_block_timeouts);
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

// A team's exchange of one sum (or three) of a row over its warps in every
// CTA of the cluster: `slots` [depth][cs * wpt], `bars` [depth].
struct Team {
  int wpt, cs;         // warps a team, CTAs a row
  int tw, lane;        // this warp in the team, this lane
  uint32_t rank;       // this CTA in the cluster
  volatile int* abort;
};

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

__device__ __forceinline__ bool team_wait(const Team& t, uint64_t* bar, uint32_t parity) {
  if (t.cs == 1) return wait_all(bar, parity, t.abort);
  bool done = false;
  for (int i = 0; i < kTries && !done; ++i) done = try_wait_cluster(bar, parity);
  if (!done) done = wait_cluster_counted(bar, parity, t.abort, &g_block_timeouts);
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

// Posts the warp's parts (the same in every lane) in its slot and arrives.
__device__ __forceinline__ void post3(const Team& t, float4* slot, uint64_t* bar, float4 v) {
  if (t.cs == 1) {
    if (t.lane == 0) {
      slot[t.tw] = v;
      mbar_arrive(bar);
    }
  } else if (t.lane < t.cs) {
    st_peer4(slot + t.rank * t.wpt + t.tw, t.lane, v);
    mbar_arrive_peer(bar, t.lane);
  }
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

__device__ __forceinline__ float3 total3(const Team& t, const float4* slot) {
  const int n = t.cs * t.wpt;
  float a = 0.f, b = 0.f, c = 0.f;
  for (int i = t.lane; i < n; i += 32) {
    const float4 q = slot[i];
    a += q.x;
    b += q.y;
    c += q.z;
  }
  return warp_sum3(a, b, c, t.lane);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A producer warp and teams of `wpt` warps.  A team takes whole stages (of
// one row, or several narrow ones) and carries each row through its three
// passes over shared memory: sum of squares of x; r, stored and kept in fp32
// in place of x and res (together they have its size), and its sum of
// squares; y.  With a warp a row there is nothing to wait for but the copy,
// and the other teams' rows cover the latencies of one; teams are made wider
// where there are few rows, or where a ring of wide rows holds few.  The
// weights w = b gate w1 and w2 stand in shared memory in fp32, in planes of
// four elements of every group of E, so that a warp reads contiguous bytes; a
// gate of several rows is read from global memory instead, where the rows of
// a sequence find it in L1.
struct BlockFwdParams {
  const void* x;
  const void* res;
  const void* gamma_post;
  const void* gate;
  const void* gamma_next;
  void* res_out;
  void* y;
  float* rstd_post;
  float* rstd_next;
  int64_t rows;
  int64_t rows_per_gate;
  int hidden;
  float a, b, eps, off;
  int teams, wpt, cs, stages, stage_rows, stride;  // stride: bytes a stage
};

constexpr int kFwdTeams = 12;

struct FwdShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t red[2];                                // across a cluster
  float slot[2][kMaxWarps * kMaxSplit];
  int abort;
};

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

template <typename T, typename TS, bool POST, bool NEXT>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1), 1) block_fwd_tma(const BlockFwdParams p) {
  constexpr int E = kElems<T, TS>, N = E / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ FwdShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages, cs = p.cs, K = p.stage_rows;
  const int cols = p.hidden / cs, nvec = cols / E;
  const uint32_t rank = cs > 1 ? cta_rank() : 0u;
  const int col0 = (int)rank * cols;
  const int64_t unit = blockIdx.x / cs, units = gridDim.x / cs;
  // stage k of a unit holds the rows [(k units + unit) K, + K): the grid
  // streams one window of consecutive rows
  const int64_t blocks = (p.rows + K - 1) / K;
  const int nst = blocks > unit ? (int)((blocks - unit + units - 1) / units) : 0;
  float4* plane1 = reinterpret_cast<float4*>(smem);
  float4* plane2 = plane1 + cols / 4;
  unsigned char* ring = reinterpret_cast<unsigned char*>(NEXT ? plane2 + cols / 4 : plane2);
  if ((int)threadIdx.x < stages) {
    mbar_init(&sh.full[threadIdx.x], 1);
    mbar_init(&sh.empty[threadIdx.x], p.wpt);
  }
  if (threadIdx.x < 2) mbar_init(&sh.red[threadIdx.x], cs * p.wpt);
  if (threadIdx.x == 0) sh.abort = 0;
  fence_mbar_init();
  __syncthreads();
  if (cs > 1) cluster_sync();
  pdl_trigger();
  pdl_wait();
  volatile int* abort = &sh.abort;
  const uint32_t xbytes = (uint32_t)(cols * sizeof(T)), sbytes = (uint32_t)(cols * sizeof(TS));
  const int res_at = K * (int)xbytes;
  auto issue = [&](int k, int stage) {
    const int64_t row = (k * units + unit) * K;
    const uint32_t n = (uint32_t)(p.rows - row < K ? p.rows - row : K);
    unsigned char* st = ring + (size_t)stage * p.stride;
    const int64_t at = row * p.hidden + col0;  // K is 1 where cs > 1
    mbar_arrive_expect_tx(&sh.full[stage], n * (xbytes + sbytes));
    bulk_load(st, static_cast<const T*>(p.x) + at, n * xbytes, &sh.full[stage]);
    bulk_load(st + res_at, static_cast<const TS*>(p.res) + at, n * sbytes, &sh.full[stage]);
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < stages && k < nst; ++k) issue(k, k);
  const T* gate = static_cast<const T*>(p.gate);
  const bool gate_each = gate != nullptr && p.rows_per_gate < p.rows;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    f32x2 w[N], f[N];
    const f32x2 off = pair(p.off, p.off), b = pair(p.b, p.b);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = b;
    if (POST) {
      load_pairs<T, N>(static_cast<const T*>(p.gamma_post) + col0 + v * E, f);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = mul2(w[i], add2(f[i], off));
    }
    if (gate != nullptr && !gate_each) {
      load_pairs<T, N>(gate + col0 + v * E, f);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = mul2(w[i], f[i]);
    }
    store_plane<N>(plane1, nvec, v, w);
    if (NEXT) {
      load_pairs<T, N>(static_cast<const T*>(p.gamma_next) + col0 + v * E, f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = add2(f[i], off);
      store_plane<N>(plane2, nvec, v, f);
    }
  }
  __syncthreads();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, k = stages;
      uint32_t phase = 0;
      for (; k < nst; ++k) {
        if (!wait_phase_counted(&sh.empty[stage], phase, abort, &g_block_timeouts)) break;
        issue(k, stage);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // every copy has landed before the CTA may exit
      const int issued = k < nst ? k : nst;
      drain_ring(sh.full, Ring{issued % stages, (uint32_t)(issued / stages) & 1u}, issued, stages);
    }
    __syncwarp();
  } else {
    const int team = (warp - 1) / p.wpt, tw = (warp - 1) % p.wpt;
    const Team t{p.wpt, cs, tw, lane, rank, abort};
    const int tt = tw * 32 + lane, threads = p.wpt * 32;
    const float inv = 1.f / (float)p.hidden;
    bool ok = true;
    uint32_t turn = 0;  // exchanges of this team: slots and barriers are used in turn
    auto over_team = [&](float v) {
      v = warp_sum(v);
      if (threads == 32 && cs == 1) return v;
      const uint32_t d = turn & 1u, parity = (turn >> 1) & 1u;
      ++turn;
      float* slot = sh.slot[d] + team * p.wpt;
      if (cs == 1) {
        if (lane == 0) slot[tw] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(threads) : "memory");
      } else {
        if (lane < cs) {
          st_peer(slot + rank * p.wpt + tw, lane, v);
          mbar_arrive_peer(&sh.red[d], lane);
        }
        ok = ok && team_wait(t, &sh.red[d], parity);
      }
      float s = 0.f;
      for (int i = lane; i < cs * p.wpt; i += 32) s += slot[i];
      return warp_sum(s);
    };
    const f32x2 a2 = pair(p.a, p.a);
    int stage = team;
    uint32_t phase = 0;
    for (int k = team; k < nst; k += p.teams) {
      ok = ok && wait_all(&sh.full[stage], phase, abort);
      const int64_t row0 = (k * units + unit) * K;
      const int n = (int)(p.rows - row0 < K ? p.rows - row0 : K);
      unsigned char* st = ring + (size_t)stage * p.stride;
      for (int q = 0; q < n; ++q) {
        const int64_t row = row0 + q;
        T* sx = reinterpret_cast<T*>(st) + q * cols;
        TS* sr = reinterpret_cast<TS*>(st + res_at) + q * cols;
        float rs1 = 1.f;
        if (POST) {
          f32x2 part[N];
#pragma unroll
          for (int i = 0; i < N; ++i) part[i] = 0;
#pragma unroll 4
          for (int v = tt; v < nvec; v += threads) {
            f32x2 x[N];
            load_pairs<T, N>(sx + v * E, x);
#pragma unroll
            for (int i = 0; i < N; ++i) part[i] = fma2(x[i], x[i], part[i]);
          }
          const float ss = over_team(sum_pairs<N>(part));
          rs1 = rsqrtf(fmaf(ss, inv, p.eps));
          if (isinf(ss)) {  // the squares overflowed (kOverflowScale)
            float again = 0.f;
            for (int j = tt; j < cols; j += threads) {
              const float f = Traits<T>::to_f(sx[j]) * kOverflowScale;
              again = fmaf(f, f, again);
            }
            rs1 = rstd_rescaled(over_team(again), p.hidden, p.eps);
          }
          if (tt == 0 && rank == 0 && ok) p.rstd_post[row] = rs1;
        }
        const f32x2 rs = pair(rs1, rs1);
        const T* grow = gate_each ? gate + row / p.rows_per_gate * p.hidden + col0 : nullptr;
        TS* out = static_cast<TS*>(p.res_out) + row * p.hidden + col0;
        f32x2 part[N];
#pragma unroll
        for (int i = 0; i < N; ++i) part[i] = 0;
#pragma unroll 2
        for (int v = tt; v < nvec; v += threads) {
          f32x2 x[N], r[N], w[N];
          load_pairs<T, N>(sx + v * E, x);
          load_pairs<TS, N>(sr + v * E, r);
          load_plane<N>(plane1, nvec, v, w);
          if (gate_each) {
            f32x2 g[N];
            load_pairs<T, N>(grow + v * E, g);
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = mul2(w[i], g[i]);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (POST) x[i] = mul2(x[i], rs);
            r[i] = fma2(w[i], x[i], mul2(a2, r[i]));
            if (NEXT) part[i] = fma2(r[i], r[i], part[i]);
          }
          if (ok) store_pairs<TS, N>(out + v * E, r);
          if (NEXT) {
            if constexpr (N == 4) {
              *reinterpret_cast<ulonglong2*>(sx + v * E) = make_ulonglong2(r[0], r[1]);
              *reinterpret_cast<ulonglong2*>(sr + v * E) = make_ulonglong2(r[2], r[3]);
            } else {
              *reinterpret_cast<ulonglong2*>(sr + v * E) = make_ulonglong2(r[0], r[1]);
            }
          }
        }
        if (!NEXT) continue;
        auto kept = [&](int v, f32x2 (&r)[N]) {
          const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(sr + v * E);
          if constexpr (N == 4) {
            const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(sx + v * E);
            r[0] = lo.x;
            r[1] = lo.y;
            r[2] = hi.x;
            r[3] = hi.y;
          } else {
            r[0] = hi.x;
            r[1] = hi.y;
          }
        };
        const float ss = over_team(sum_pairs<N>(part));
        float rs2 = rsqrtf(fmaf(ss, inv, p.eps));
        if (isinf(ss)) {
          const f32x2 scale = pair(kOverflowScale, kOverflowScale);
#pragma unroll
          for (int i = 0; i < N; ++i) part[i] = 0;
          for (int v = tt; v < nvec; v += threads) {
            f32x2 r[N];
            kept(v, r);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              r[i] = mul2(r[i], scale);
              part[i] = fma2(r[i], r[i], part[i]);
            }
          }
          rs2 = rstd_rescaled(over_team(sum_pairs<N>(part)), p.hidden, p.eps);
        }
        if (tt == 0 && rank == 0 && ok) p.rstd_next[row] = rs2;
        const f32x2 rn = pair(rs2, rs2);
        T* yr = static_cast<T*>(p.y) + row * p.hidden + col0;
#pragma unroll 4
        for (int v = tt; v < nvec; v += threads) {
          f32x2 r[N], w[N];
          kept(v, r);
          load_plane<N>(plane2, nvec, v, w);
#pragma unroll
          for (int i = 0; i < N; ++i) r[i] = mul2(mul2(r[i], rn), w[i]);
          if (ok) store_pairs<T, N>(yr + v * E, r);
        }
      }
      // r was written where the next copy will land
      if (NEXT) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
      stage += p.teams;
      if (stage >= stages) {
        stage -= stages;
        phase ^= 1u;
      }
    }
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while a peer may write to its slots
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// All warps are in teams; a team works on one row, and a stage holds one row
// a team.  A thread owns the same 8 or 16 columns of every row: their weights
// and their fp32 sums over the rows stay in its registers (which is why no
// warp is set aside for the copies: 16 warps have 128 registers a thread, 17
// have 96).  The reductions never stop a team: a warp posts its part of a
// row's sums to a slot, of every CTA of the cluster, arrives on the row's
// barrier (red), and takes the row up again after the sums of the next one:
//   A(i + 1): the three sums of row i + 1 -> red
//   B(i): wait for red of row i; dx and dresidual, read again from its stage
// Slots and barriers are four deep: a warp posts row i + 4 only after a wait
// that every reader of row i has passed.  The stage of row i - 1 is filled
// again by thread 0 between A(i + 1) and B(i), when the other warps are
// through with it (before A(i + 1) where there are two stages, and it is the
// one that A(i + 1) reads).
constexpr int kDepth = 4;

struct BwdShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t red[kMaxWarps][kDepth];
  float4 slot[kDepth][kMaxWarps * kMaxSplit];
  int64_t fill_row;   // thread 0's: the next row to copy,
  int64_t issued;     // the copies issued, and the stage of the next one
  Ring fill;
  int abort;
};

struct BwdShape {
  int teams, wpt, cs, stages, stride;
  bool read_x;  // x is wanted: a post norm or the gate's gradient
};

// Where the arrays of a stage begin.
struct BwdStage {
  int r, dy, dr, bytes;  // offsets; x is at 0
};

template <typename T, typename TS>
__host__ __device__ inline BwdStage bwd_stage(int teams, int cols, bool x, bool next, bool dr) {
  BwdStage s;
  const int t = teams * cols * (int)sizeof(T), ts = teams * cols * (int)sizeof(TS);
  s.r = x ? t : 0;
  s.dy = s.r + (next ? ts : 0);
  s.dr = s.dy + (next ? t : 0);
  s.bytes = s.dr + (dr ? ts : 0);
  return s;
}

template <typename T, typename TS, bool POST, bool NEXT, int NV>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    block_bwd_tma(const BlockBwdParams p, const BwdShape sp) {
  constexpr int E = kElems<T, TS>, N = E / 2;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ BwdShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = sp.teams, stages = sp.stages, cs = sp.cs;
  const int cols = p.hidden / cs;
  const uint32_t rank = cs > 1 ? cta_rank() : 0u;
  const int64_t unit = blockIdx.x / cs, units = gridDim.x / cs;
  const int64_t r0 = unit * p.rows / units, r1 = (unit + 1) * p.rows / units;
  const bool has_dr = p.dr != nullptr, has_x = sp.read_x;
  for (int i = threadIdx.x; i < kMaxStages + kMaxWarps; i += blockDim.x) {
    if (i < stages) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], K * sp.wpt);
    }
    if (i >= kMaxStages)
      for (int d = 0; d < kDepth; ++d) mbar_init(&sh.red[i - kMaxStages][d], cs * sp.wpt);
  }
  if (threadIdx.x == 0) {
    sh.abort = 0;
    sh.fill_row = r0;
    sh.issued = 0;
    sh.fill = Ring{0, 0u};
  }
  fence_mbar_init();
  __syncthreads();
  if (cs > 1) cluster_sync();
  pdl_trigger();
  pdl_wait();
  volatile int* abort = &sh.abort;
  const BwdStage at = bwd_stage<T, TS>(K, cols, has_x, NEXT, has_dr);

  // Thread 0: the copies of the next stage, if there are rows left.  A stage
  // never crosses from one gate row to the next.
  auto fill = [&]() {
    const int64_t row = sh.fill_row;
    if (row >= r1) return;
    Ring pos = sh.fill;
    if (sh.issued >= stages &&
        !wait_phase_counted(&sh.empty[pos.stage], pos.phase ^ 1u, abort, &g_block_timeouts)) {
      sh.fill_row = r1;
      return;
    }
    const int64_t seg = (row / p.rows_per_gate + 1) * p.rows_per_gate;
    const int64_t end = seg < r1 ? seg : r1;
    const uint32_t n = (uint32_t)(end - row < K ? end - row : K);
    const uint32_t tb = n * (uint32_t)(cols * sizeof(T)), sb = n * (uint32_t)(cols * sizeof(TS));
    unsigned char* st = ring + (size_t)pos.stage * sp.stride;
    uint64_t* full = &sh.full[pos.stage];
    const int64_t from = row * p.hidden + (int64_t)rank * cols;  // K is 1 where cs > 1
    mbar_arrive_expect_tx(full, (has_x ? tb : 0) + (NEXT ? tb + sb : 0) + (has_dr ? sb : 0));
    if (has_x) bulk_load(st, static_cast<const T*>(p.x) + from, tb, full);
    if (NEXT) {
      bulk_load(st + at.r, static_cast<const TS*>(p.r) + from, sb, full);
      bulk_load(st + at.dy, static_cast<const T*>(p.dy) + from, tb, full);
    }
    if (has_dr) bulk_load(st + at.dr, static_cast<const TS*>(p.dr) + from, sb, full);
    pos.next(stages);
    sh.fill = pos;
    sh.issued += 1;
    sh.fill_row = row + n;
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < stages; ++k) fill();

  const int team = warp / sp.wpt;
  const Team t{sp.wpt, cs, warp % sp.wpt, lane, rank, abort};
  const bool alone = sp.wpt == 1 && cs == 1;  // a warp's sums need no exchange
  const int tt = t.tw * 32 + lane, threads = sp.wpt * 32;
  const int nvec = cols / E, col0 = (int)rank * cols;
  const float inv = 1.f / (float)p.hidden;
  const bool want_a = POST || p.gate != nullptr;
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gate = static_cast<const T*>(p.gate);
  const f32x2 off = pair(p.off, p.off), a2 = pair(p.a, p.a);
  f32x2 w[NV][N], w2[NV][N], acc_n[NV][N], acc_a[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = tt + j * threads;
#pragma unroll
    for (int i = 0; i < N; ++i) w2[j][i] = 0;
    if (NEXT && v < nvec) load_pairs<T, N>(static_cast<const T*>(p.gamma_next) + col0 + v * E, w2[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w2[j][i] = add2(w2[j][i], off);
      acc_n[j][i] = 0;
      acc_a[j][i] = 0;
    }
  }
  bool ok = true;
  Ring pos_a{0, 0u}, pos_b{0, 0u};
  uint32_t posted = 0, taken = 0;  // rows of this team whose sums were posted, used
  uint32_t steps = 0;              // stages that went through A
  const bool early = stages < 3;   // the next stage is the one just left

  for (int64_t seg0 = r0; seg0 < r1;) {
    const int64_t q = seg0 / p.rows_per_gate;
    const int64_t seg1 = (q + 1) * p.rows_per_gate < r1 ? (q + 1) * p.rows_per_gate : r1;
    const int nrows = (int)(seg1 - seg0) - team;  // row i of this team: i K < nrows
    const int nst = (int)((seg1 - seg0 + K - 1) / K);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tt + j * threads;
      f32x2 f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[j][i] = pair(p.b, p.b);
      if (v >= nvec) continue;
      if (POST) {
        load_pairs<T, N>(gamma_post + col0 + v * E, f);
#pragma unroll
        for (int i = 0; i < N; ++i) w[j][i] = mul2(w[j][i], add2(f[i], off));
      }
      if (gate != nullptr) {
        load_pairs<T, N>(gate + q * p.hidden + col0 + v * E, f);
#pragma unroll
        for (int i = 0; i < N; ++i) w[j][i] = mul2(w[j][i], f[i]);
      }
    }
    const float* stat1 = p.rstd_post + seg0 + team;
    const float* stat2 = p.rstd_next + seg0 + team;
    // the row statistics, loaded a row ahead of their use
    float rs1_a = 1.f, rs2_a = 0.f;
    if (POST && nrows > 0) rs1_a = __ldg(stat1);
    if (NEXT && nrows > 0) rs2_a = __ldg(stat2);
    float rs1_n = 1.f, rs2_n = 0.f;
    float3 own = make_float3(0.f, 0.f, 0.f);  // a lone warp's sums of the row in A
    auto sums = [&](int i) {  // A
      if (early && steps >= 2 && threadIdx.x == 0) fill();
      ok = ok && wait_all(&sh.full[pos_a.stage], pos_a.phase, abort);
      rs1_n = rs1_a;
      rs2_n = rs2_a;
      if ((i + 1) * K < nrows) {
        if (POST) rs1_a = __ldg(stat1 + (i + 1) * K);
        if (NEXT) rs2_a = __ldg(stat2 + (i + 1) * K);
      }
      if (ok && i * K < nrows) {
        const unsigned char* st = ring + (size_t)pos_a.stage * sp.stride;
        const T* sx = reinterpret_cast<const T*>(st) + team * cols;
        const TS* sr = reinterpret_cast<const TS*>(st + at.r) + team * cols;
        const T* sdy = reinterpret_cast<const T*>(st + at.dy) + team * cols;
        const TS* sdr = reinterpret_cast<const TS*>(st + at.dr) + team * cols;
        const f32x2 rs1 = pair(rs1_n, rs1_n), rs2 = pair(rs2_n, rs2_n);
        f32x2 s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int v = tt + j * threads;
          if (v >= nvec) continue;
          f32x2 x[N], d[N];
          if (POST) {
#pragma unroll
            for (int k = 0; k < N; ++k) d[k] = 0;
            load_pairs<T, N>(sx + v * E, x);
            if (has_dr) load_pairs<TS, N>(sdr + v * E, d);
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = mul2(w[j][k], mul2(x[k], rs1));
          }
          if (NEXT) {
            f32x2 r[N], dy[N];
            load_pairs<TS, N>(sr + v * E, r);
            load_pairs<T, N>(sdy + v * E, dy);
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const f32x2 rh = mul2(r[k], rs2), g = mul2(dy[k], w2[j][k]);
              s1 = fma2(g, rh, s1);
              if (POST) {
                s3 = fma2(x[k], rh, s3);
                d[k] = fma2(rs2, g, d[k]);
              }
            }
          }
          if (POST)
#pragma unroll
            for (int k = 0; k < N; ++k) s2 = fma2(x[k], d[k], s2);
        }
        if (POST && NEXT)
          own = warp_sum3(sum2(s1), sum2(s2), sum2(s3), lane);
        else
          own = make_float3(NEXT ? warp_sum(sum2(s1)) : 0.f, POST ? warp_sum(sum2(s2)) : 0.f, 0.f);
        if (!alone)
          post3(t, sh.slot[posted % kDepth] + team * sp.wpt * cs, &sh.red[team][posted % kDepth],
                make_float4(own.x, own.y, own.z, 0.f));
        ++posted;
      }
      pos_a.next(stages);
      if (!early && steps >= 2 && threadIdx.x == 0) fill();
      ++steps;
      __syncwarp();
    };
    sums(0);
    for (int i = 0; i < nst; ++i) {
      const f32x2 rs1 = pair(rs1_n, rs1_n), rs2 = pair(rs2_n, rs2_n);
      float3 s = own;
      if (i + 1 < nst) sums(i + 1);
      if (ok && i * K < nrows) {  // B
        if (!alone) {
          ok = team_wait(t, &sh.red[team][taken % kDepth], (taken / kDepth) & 1u);
          s = total3(t, sh.slot[taken % kDepth] + team * sp.wpt * cs);
        }
        ++taken;
        const float rs2f = split(rs2).x;
        const float c1f = s.x * inv;
        const float c2f = POST ? fmaf(-rs2f * c1f, s.z, s.y) * inv : 0.f;
        const f32x2 c1 = pair(-c1f, -c1f), c2 = pair(-c2f, -c2f);
        const unsigned char* st = ring + (size_t)pos_b.stage * sp.stride;
        const T* sx = reinterpret_cast<const T*>(st) + team * cols;
        const TS* sr = reinterpret_cast<const TS*>(st + at.r) + team * cols;
        const T* sdy = reinterpret_cast<const T*>(st + at.dy) + team * cols;
        const TS* sdr = reinterpret_cast<const TS*>(st + at.dr) + team * cols;
        const int64_t to = (seg0 + team + (int64_t)i * K) * p.hidden + col0;
        T* dx = static_cast<T*>(p.dx) + to;
        TS* dres = static_cast<TS*>(p.dres) + to;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int v = tt + j * threads;
          if (v >= nvec) continue;
          f32x2 x[N], d[N];
#pragma unroll
          for (int k = 0; k < N; ++k) x[k] = d[k] = 0;
          if (has_dr) load_pairs<TS, N>(sdr + v * E, d);
          if (NEXT) {
            f32x2 r[N], dy[N];
            load_pairs<TS, N>(sr + v * E, r);
            load_pairs<T, N>(sdy + v * E, dy);
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const f32x2 rh = mul2(r[k], rs2);
              d[k] = fma2(rs2, fma2(c1, rh, mul2(dy[k], w2[j][k])), d[k]);
              acc_n[j][k] = fma2(dy[k], rh, acc_n[j][k]);
            }
          }
          if (has_x) load_pairs<T, N>(sx + v * E, x);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            if (POST) x[k] = mul2(x[k], rs1);
            acc_a[j][k] = fma2(d[k], x[k], acc_a[j][k]);
            const f32x2 g = mul2(w[j][k], d[k]);
            x[k] = POST ? mul2(rs1, fma2(c2, x[k], g)) : g;
            d[k] = mul2(a2, d[k]);
          }
          store_pairs<T, N>(dx + v * E, x);
          store_pairs<TS, N>(dres + v * E, d);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[pos_b.stage]);
      pos_b.next(stages);
    }

    // the segment's sum of A, and after the last one that of dgamma_next: a
    // thread's own columns, or its columns of the teams' sums, added in turn
    const bool first = q == r0 / p.rows_per_gate, last = seg1 == r1;
    float* pa = p.p_a + (unit + q) * p.hidden + col0;
    float* pp = p.p_post + unit * p.hidden + col0;
    float* pn = p.p_next + unit * p.hidden + col0;
    auto put_a = [&](int c, float v) {
      v *= p.b;
      if (gate != nullptr) {
        pa[c] = v;
        v *= Traits<T>::to_f(gate[q * p.hidden + col0 + c]);
      }
      if (POST) pp[c] = first ? v : pp[c] + v;
    };
    auto put_n = [&](int c, float v) { pn[c] = v; };
    auto flush = [&](f32x2 (&acc)[NV][N], auto put) {
      f32x2* comb = reinterpret_cast<f32x2*>(ring + (size_t)stages * sp.stride);
      if (K > 1)
        for (int m = 0; m < K; ++m) {
          if (team == m)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              const int v = tt + j * threads;
              if (v >= nvec) continue;
#pragma unroll
              for (int k = 0; k < N; ++k)
                comb[v * N + k] = m == 0 ? acc[j][k] : add2(comb[v * N + k], acc[j][k]);
            }
          __syncthreads();
        }
      if (K > 1)
        for (int c = threadIdx.x; c < cols; c += blockDim.x)
          put(c, reinterpret_cast<const float*>(comb)[c]);
      else
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int v = tt + j * threads;
          if (v >= nvec) continue;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float2 f = split(acc[j][k]);
            put(v * E + 2 * k, f.x);
            put(v * E + 2 * k + 1, f.y);
          }
        }
      if (K > 1) __syncthreads();
    };
    if (want_a) flush(acc_a, put_a);
    if (NEXT && last) flush(acc_n, put_n);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) acc_a[j][k] = 0;
    seg0 = seg1;
  }
  // after a wait that ran out copies may still be on their way
  if (threadIdx.x == 0 && *abort) drain_ring(sh.full, sh.fill, sh.issued, stages);
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while a peer may write to its slots
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int kSlack = 1024;  // static shared memory beside the kernels' structs

// The forward's teams and stages for `rows` rows on `sms` SMs.  The row is
// split over as few CTAs as leave two stages beside the weights.
struct FwdShape {
  int teams, wpt, cs, stages, stage_rows, stride;
  size_t smem;
};

bool fwd_shape(int64_t rows, int hidden, int sms, int row_elem, int planes, int align, int elems,
               FwdShape* s) {
  const int budget = kSmemBudget - (int)sizeof(FwdShared) - kSlack;
  for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
    if (hidden % (align * cs) != 0) return false;
    const int cols = hidden / cs, row = cols * row_elem, over = planes * cols * 4;
    if (over + 2 * ((row + 127) / 128 * 128) > budget) continue;
    s->cs = cs;
    const int64_t mine = (rows * cs + sms - 1) / sms;  // rows a CTA, about
    const int most = (cols / elems + 31) / 32;         // warps a row can use
    s->stage_rows = 1;
    if (cs > 1 || mine <= 2) {
      s->wpt = most < kMaxWarps ? most : kMaxWarps;
      s->teams = 1;
    } else {
      s->wpt = 1;
      while (s->wpt < kMaxWarps && cols > 4096 * s->wpt) s->wpt *= 2;
      // narrow rows: several to a stage, as long as every team has its own
      while (s->stage_rows * row < 8192 && mine >= 2 * kFwdTeams * s->stage_rows) s->stage_rows *= 2;
      s->teams = kMaxWarps / s->wpt < kFwdTeams ? kMaxWarps / s->wpt : kFwdTeams;
    }
    s->stride = (s->stage_rows * row + 127) / 128 * 128;
    s->stages = (budget - over) / s->stride;
    if (s->stages > kMaxStages) s->stages = kMaxStages;
    if (s->teams > s->stages) s->teams = s->stages;
    s->stages -= s->stages % s->teams;  // a stage is always the same team's
    s->smem = (size_t)over + (size_t)s->stages * s->stride;
    return true;
  }
  return false;
}

// The backward's teams and stages: all warps busy and three stages, with 16
// columns a thread or else 8 (one row a stage), over as few CTAs as can be.
struct BwdPick {
  int teams, wpt, cs, stages, stride, nv8;  // nv8: groups of 8 columns a thread
  size_t smem;
};

template <typename F>
bool bwd_pick(int hidden, int align, F stage_bytes, BwdPick* out) {
  const int budget = kSmemBudget - (int)sizeof(BwdShared) - kSlack;
  for (int least = 3; least >= 2; --least)
    for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
      if (hidden % (align * cs) != 0) break;
      const int cols = hidden / cs;
      for (int nv8 = cols < 512 ? 1 : 2; nv8 >= 1; --nv8) {
        BwdPick s;
        s.cs = cs;
        s.nv8 = nv8;
        s.wpt = (cols + nv8 * 256 - 1) / (nv8 * 256);
        if (s.wpt > kMaxWarps) continue;
        for (s.teams = cs > 1 ? 1 : kMaxWarps / s.wpt; s.teams >= 1; --s.teams) {
          if (s.teams * s.wpt < kMaxWarps / 2 + 1 && nv8 == 2 && 2 * s.wpt <= kMaxWarps) break;
          const int comb = s.teams > 1 ? cols * 4 : 0;
          s.stride = (stage_bytes(s.teams, cols) + 127) / 128 * 128;
          s.stages = (budget - comb) / s.stride;
          if (s.stages > kMaxStages) s.stages = kMaxStages;
          if (s.stages < least) continue;
          s.smem = (size_t)s.stages * s.stride + comb;
          *out = s;
          return true;
        }
      }
    }
  return false;
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)bytes);
}

template <typename T, typename TS, bool POST, bool NEXT>
bool try_fwd(const BlockFwdArgs& a, cudaStream_t s, cudaError_t* err) {
  constexpr int E = kElems<T, TS>;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return true;
  const int sms = sm_count(dev);
  FwdShape sh;
  if (!fwd_shape(a.rows, a.hidden, sms, (int)(sizeof(T) + sizeof(TS)), NEXT ? 2 : 1,
                 16 / (int)sizeof(T), E, &sh))
    return false;
  BlockFwdParams p;
  p.x = a.x;
  p.res = a.res;
  p.gamma_post = a.gamma_post;
  p.gate = a.gate;
  p.gamma_next = a.gamma_next;
  p.res_out = a.res_out;
  p.y = a.y;
  p.rstd_post = a.rstd_post;
  p.rstd_next = a.rstd_next;
  p.rows = a.rows;
  p.rows_per_gate = a.rows_per_gate;
  p.hidden = a.hidden;
  p.a = a.res_scale;
  p.b = a.branch_scale;
  p.eps = a.eps;
  p.off = a.offset ? 1.f : 0.f;
  p.teams = sh.teams;
  p.wpt = sh.wpt;
  p.cs = sh.cs;
  p.stages = sh.stages;
  p.stage_rows = sh.stage_rows;
  p.stride = sh.stride;
  auto kern = block_fwd_tma<T, TS, POST, NEXT>;
  *err = allow_smem(kern, sh.smem);
  if (*err != cudaSuccess) return true;
  int64_t units = sms / sh.cs;
  const int64_t blocks = (a.rows + sh.stage_rows - 1) / sh.stage_rows;
  if (units > blocks) units = blocks;
  if (units < 1) units = 1;
  *err = launch_kernel(kern, dim3((unsigned)(units * sh.cs)), dim3(32 * (1 + sh.teams * sh.wpt)),
                       sh.smem, s, sh.cs, p);
  return true;
}

template <typename T, typename TS, bool POST, bool NEXT>
bool try_bwd(const BlockBwdArgs& a, BlockBwdParams& p, int* units, cudaStream_t s,
             cudaError_t* err) {
  constexpr int E = kElems<T, TS>;
  BwdShape sp;
  sp.read_x = POST || a.gate != nullptr;
  const bool dr = a.dr != nullptr, x = sp.read_x;
  BwdPick sh;
  if (!bwd_pick(a.hidden, 16 / (int)sizeof(T),
                [=](int k, int cols) { return bwd_stage<T, TS>(k, cols, x, NEXT, dr).bytes; }, &sh))
    return false;
  sp.teams = sh.teams;
  sp.wpt = sh.wpt;
  sp.cs = sh.cs;
  sp.stages = sh.stages;
  sp.stride = sh.stride;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return true;
  int64_t n = sm_count(dev) / sh.cs;
  if (n < 1) n = 1;
  if (n > RMSN_BLOCK_MAX_PARTIALS) n = RMSN_BLOCK_MAX_PARTIALS;
  if (n > a.rows) n = a.rows;
  *units = (int)n;
  place_partials(a, *units, p);
  auto go = [&](auto kern) {
    *err = allow_smem(kern, sh.smem);
    if (*err != cudaSuccess) return;
    *err = launch_kernel(kern, dim3((unsigned)(n * sh.cs)), dim3(32 * sh.teams * sh.wpt), sh.smem,
                         s, sh.cs, p, sp);
  };
  if (sh.nv8 == 1)
    go(block_bwd_tma<T, TS, POST, NEXT, 8 / E>);
  else
    go(block_bwd_tma<T, TS, POST, NEXT, 16 / E>);
  return true;
}

template <typename T, typename TS>
bool fwd_of(const BlockFwdArgs& a, cudaStream_t s, cudaError_t* err) {
  if (a.gamma_post == nullptr) return try_fwd<T, TS, false, true>(a, s, err);
  if (a.gamma_next == nullptr) return try_fwd<T, TS, true, false>(a, s, err);
  return try_fwd<T, TS, true, true>(a, s, err);
}

template <typename T, typename TS>
bool bwd_of(const BlockBwdArgs& a, BlockBwdParams& p, int* units, cudaStream_t s,
            cudaError_t* err) {
  if (a.gamma_post == nullptr) return try_bwd<T, TS, false, true>(a, p, units, s, err);
  if (a.gamma_next == nullptr) return try_bwd<T, TS, true, false>(a, p, units, s, err);
  return try_bwd<T, TS, true, true>(a, p, units, s, err);
}

}  // namespace

bool try_launch_block_fwd_tma(int dtype, int res_dtype, const BlockFwdArgs& a, cudaStream_t s,
                              cudaError_t* err) {
  if (!a.vec_ok) return false;
  if (dtype == RMSN_F32) return fwd_of<float, float>(a, s, err);
  if (dtype == RMSN_BF16)
    return res_dtype == RMSN_F32 ? fwd_of<__nv_bfloat16, float>(a, s, err)
                                 : fwd_of<__nv_bfloat16, __nv_bfloat16>(a, s, err);
  return res_dtype == RMSN_F32 ? fwd_of<__half, float>(a, s, err)
                               : fwd_of<__half, __half>(a, s, err);
}

bool try_launch_block_bwd_tma(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p,
                              int* units, cudaStream_t s, cudaError_t* err) {
  if (!a.vec_ok) return false;
  if (dtype == RMSN_F32) return bwd_of<float, float>(a, p, units, s, err);
  if (dtype == RMSN_BF16)
    return res_dtype == RMSN_F32 ? bwd_of<__nv_bfloat16, float>(a, p, units, s, err)
                                 : bwd_of<__nv_bfloat16, __nv_bfloat16>(a, p, units, s, err);
  return res_dtype == RMSN_F32 ? bwd_of<__half, float>(a, p, units, s, err)
                               : bwd_of<__half, __half>(a, p, units, s, err);
}

cudaError_t read_block_wait_timeouts(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_block_timeouts, sizeof(unsigned int));
}

}  // namespace rmsn
