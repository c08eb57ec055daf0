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
constexpr int kMaxSplit = 16;      // CTAs a row is split over
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
  int lanes;  // of a warp on a row: 32, or kNarrowLanes where wpt is 1
};

// Rows of up to kNarrowGroups groups of columns take kNarrowLanes lanes, and
// a warp takes 32 / kNarrowLanes of them at a time: their reductions share
// their shuffles.
constexpr int kNarrowLanes = 8;
constexpr int kNarrowGroups = 64;

struct FwdShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t red[kMaxWarps][2];                     // a team's, across a cluster
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
  if ((int)threadIdx.x < p.teams)
    for (int d = 0; d < 2; ++d) mbar_init(&sh.red[threadIdx.x][d], cs * p.wpt);
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
    const int lanes = p.lanes, threads = p.wpt * 32;
    const int tt = tw * 32 + (lane & (lanes - 1)), step = lanes < 32 ? lanes : threads;
    const int at_once = 32 / lanes, sub = lane / lanes;  // rows a warp takes at a time
    const float inv = 1.f / (float)p.hidden;
    bool ok = true;
    uint32_t turn = 0;  // exchanges of this team: slots and barriers are used in turn
    auto over_team = [&](float v) {  // the sum over the row's lanes
      if (lanes == 32) {
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
      }
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      if (threads == 32 && cs == 1) return v;
      const uint32_t d = turn & 1u, parity = (turn >> 1) & 1u;
      ++turn;
      float* slot = sh.slot[d] + team * p.wpt * cs;
      if (cs == 1) {
        if (lane == 0) slot[tw] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(threads) : "memory");
      } else {
        if (lane < cs) {
          st_peer(slot + rank * p.wpt + tw, lane, v);
          mbar_arrive_peer(&sh.red[team][d], lane);
        }
        ok = ok && team_wait(cs, &sh.red[team][d], parity, abort);
      }
      float s = 0.f;
      for (int i = lane; i < cs * p.wpt; i += 32) s += slot[i];
      return warp_sum(s);
    };
    const f32x2 a2 = pair(p.a, p.a);
    // f for each of the thread's groups of columns, four at a time; the usual
    // steps are constants of the addresses
    auto by = [&](auto f, auto step_of) {
      constexpr int S = decltype(step_of)::value;
      int v = tt;
      for (; v + 3 * S < nvec; v += 4 * S) {
#pragma unroll
        for (int u = 0; u < 4; ++u) f(v + S * u);
      }
      for (; v < nvec; v += S) f(v);
    };
    auto each = [&](auto f) {
      if (step == 32)
        by(f, std::integral_constant<int, 32>{});
      else if (step == 128)
        by(f, std::integral_constant<int, 128>{});
      else if (step == kNarrowLanes)
        by(f, std::integral_constant<int, kNarrowLanes>{});
      else
        for (int v = tt; v < nvec; v += step) f(v);
    };
    int stage = team;
    uint32_t phase = 0;
    for (int k = team; k < nst; k += p.teams) {
      ok = ok && wait_all(&sh.full[stage], phase, abort);
      const int64_t row0 = (k * units + unit) * K;
      const int n = (int)(p.rows - row0 < K ? p.rows - row0 : K);
      unsigned char* st = ring + (size_t)stage * p.stride;
      for (int q0 = 0; q0 < n; q0 += at_once) {
        // every lane takes part in the shuffles; those past the last row work
        // on the stage's first row and write nothing
        const int qt = q0 + sub;
        const bool mine = qt < n && ok;
        const int q = qt < n ? qt : 0;
        const int64_t row = row0 + q;
        T* sx = reinterpret_cast<T*>(st) + q * cols;
        TS* sr = reinterpret_cast<TS*>(st + res_at) + q * cols;
        float rs1 = 1.f;
        if (POST) {
          f32x2 part[N];
#pragma unroll
          for (int i = 0; i < N; ++i) part[i] = 0;
          each([&](int v) {
            f32x2 x[N];
            load_pairs<T, N>(sx + v * E, x);
#pragma unroll
            for (int i = 0; i < N; ++i) part[i] = fma2(x[i], x[i], part[i]);
          });
          const float ss = over_team(sum_pairs<N>(part));
          rs1 = rsqrtf(fmaf(ss, inv, p.eps));
          if (__any_sync(0xffffffffu, isinf(ss))) {  // squares overflowed (kOverflowScale)
            float again = 0.f;
            for (int j = tt; j < cols; j += step) {
              const float f = Traits<T>::to_f(sx[j]) * kOverflowScale;
              again = fmaf(f, f, again);
            }
            again = over_team(again);
            if (isinf(ss)) rs1 = rstd_rescaled(again, p.hidden, p.eps);
          }
          if (tt == 0 && rank == 0 && mine) p.rstd_post[row] = rs1;
        }
        const f32x2 rs = pair(rs1, rs1);
        const T* grow = gate_each ? gate + row / p.rows_per_gate * p.hidden + col0 : nullptr;
        TS* out = static_cast<TS*>(p.res_out) + row * p.hidden + col0;
        f32x2 part[N];
#pragma unroll
        for (int i = 0; i < N; ++i) part[i] = 0;
        each([&](int v) {
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
          if (mine) store_pairs<TS, N>(out + v * E, r);
          if (NEXT && mine) {
            if constexpr (N == 4) {
              *reinterpret_cast<ulonglong2*>(sx + v * E) = make_ulonglong2(r[0], r[1]);
              *reinterpret_cast<ulonglong2*>(sr + v * E) = make_ulonglong2(r[2], r[3]);
            } else {
              *reinterpret_cast<ulonglong2*>(sr + v * E) = make_ulonglong2(r[0], r[1]);
            }
          }
        });
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
        if (__any_sync(0xffffffffu, isinf(ss))) {
          const f32x2 scale = pair(kOverflowScale, kOverflowScale);
#pragma unroll
          for (int i = 0; i < N; ++i) part[i] = 0;
          for (int v = tt; v < nvec; v += step) {
            f32x2 r[N];
            kept(v, r);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              r[i] = mul2(r[i], scale);
              part[i] = fma2(r[i], r[i], part[i]);
            }
          }
          const float again = over_team(sum_pairs<N>(part));
          if (isinf(ss)) rs2 = rstd_rescaled(again, p.hidden, p.eps);
        }
        if (tt == 0 && rank == 0 && mine) p.rstd_next[row] = rs2;
        const f32x2 rn = pair(rs2, rs2);
        T* yr = static_cast<T*>(p.y) + row * p.hidden + col0;
        each([&](int v) {
          f32x2 r[N], w[N];
          kept(v, r);
          load_plane<N>(plane2, nvec, v, w);
#pragma unroll
          for (int i = 0; i < N; ++i) r[i] = mul2(mul2(r[i], rn), w[i]);
          if (mine) store_pairs<T, N>(yr + v * E, r);
        });
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
// Three roles, which meet at per-stage mbarriers:
//   producer (warp 0)   copies a stage's rows (one, or several narrow ones):
//                       x, r, dy and dr                          -> full[s]
//   reducers            a warp takes every `reducers`-th stage: the three sums
//                       of each row, c1 and c2 into the row's slot -> red[s]
//                       (over a cluster the CTAs' parts of a row are exchanged
//                       first, through slots of every CTA)
//   appliers            teams of `wpt` warps, a row of the stage each: dx and
//                       dresidual; a thread owns the same 8 or 16 columns of
//                       every row, whose weights and fp32 sums over the rows
//                       stay in its registers                    -> empty[s]
// A row's sums are taken by one warp because sums exchanged between all the
// warps of a CTA, every row, cost more than the sums: with 16 warps on a row
// (each warp its columns, parts posted to slots and taken up a row later)
// 16384 x 8192 bf16 took 530 to 600 us.  The reducers' weights stand in shared
// memory as in the forward.
constexpr int kBwdStages = 8;
constexpr int kBwdRows = 32;      // rows of a stage, at most
constexpr int kBwdWarps = 16;     // 128 registers a thread

struct BwdShared {
  uint64_t full[kBwdStages];
  uint64_t red[kBwdStages];
  uint64_t empty[kBwdStages];
  uint64_t parts[kBwdStages];
  float4 stat[kBwdStages][kBwdRows];          // c1, c2, rstd_post, rstd_next
  float4 part[2][kBwdStages][kMaxSplit];      // of the cluster's CTAs
  int abort;
};

struct BwdShape {
  int reducers, teams, wpt, cs, stages, stage_rows, stride;
  int lanes;    // of a reducer on a row (kNarrowLanes: as in the forward)
  bool read_x;  // x is wanted: a post norm or the gate's gradient
};

// Where the arrays of a stage begin.
struct BwdStage {
  int r, dy, dr, bytes;  // offsets; x is at 0
};

template <typename T, typename TS>
__host__ __device__ inline BwdStage bwd_stage(int rows, int cols, bool x, bool next, bool dr) {
  BwdStage s;
  const int t = rows * cols * (int)sizeof(T), ts = rows * cols * (int)sizeof(TS);
  s.r = x ? t : 0;
  s.dy = s.r + (next ? ts : 0);
  s.dr = s.dy + (next ? t : 0);
  s.bytes = s.dr + (dr ? ts : 0);
  return s;
}

// The stages of a unit's rows, in order: n rows from `row` (counted from the
// unit's first) on, of gate row q; a stage never crosses from one gate row to
// the next.
struct Walk {
  int row, n, end, total, most;
  int64_t q, rows_per_gate;
  __device__ Walk(int64_t r0, int64_t r1, int64_t rpg, int stage_rows)
      : row(0), n(0), total((int)(r1 - r0)), most(stage_rows), q(r0 / rpg), rows_per_gate(rpg) {
    const int64_t left = (q + 1) * rpg - r0;
    end = left < total ? (int)left : total;
  }
  __device__ __forceinline__ bool next() {
    row += n;
    if (row >= total) return false;
    if (row == end) {
      ++q;
      end = rows_per_gate < total - end ? end + (int)rows_per_gate : total;
    }
    n = end - row < most ? end - row : most;
    return true;
  }
};

template <typename T, typename TS, bool POST, bool NEXT, bool DR, int NV>
__global__ void __launch_bounds__(32 * kBwdWarps, 1)
    block_bwd_tma(const BlockBwdParams p, const BwdShape sp) {
  constexpr int E = kElems<T, TS>, N = E / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ BwdShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = sp.stages, cs = sp.cs, K = sp.stage_rows, reducers = sp.reducers;
  const int applier_warps = sp.teams * sp.wpt;
  const int cols = p.hidden / cs, nvec = cols / E;
  const uint32_t rank = cs > 1 ? cta_rank() : 0u;
  const int col0 = (int)rank * cols;
  const int64_t unit = blockIdx.x / cs, units = gridDim.x / cs;
  const int64_t r0 = unit * p.rows / units, r1 = (unit + 1) * p.rows / units;
  const bool has_x = POST || sp.read_x;
  float4* plane1 = reinterpret_cast<float4*>(smem);
  float4* plane2 = POST ? plane1 + cols / 4 : plane1;
  unsigned char* ring = reinterpret_cast<unsigned char*>(NEXT ? plane2 + cols / 4 : plane2);
  if ((int)threadIdx.x < stages) {
    mbar_init(&sh.full[threadIdx.x], 1);
    mbar_init(&sh.red[threadIdx.x], 1);
    mbar_init(&sh.empty[threadIdx.x], 1 + applier_warps);
    mbar_init(&sh.parts[threadIdx.x], cs);
  }
  if (threadIdx.x == 0) sh.abort = 0;
  fence_mbar_init();
  __syncthreads();
  if (cs > 1) cluster_sync();
  pdl_trigger();
  pdl_wait();
  volatile int* abort = &sh.abort;
  const BwdStage at = bwd_stage<T, TS>(K, cols, has_x, NEXT, DR);
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gamma_next = static_cast<const T*>(p.gamma_next);
  const T* gate = static_cast<const T*>(p.gate);
  const bool gate_each = gate != nullptr && p.rows_per_gate < p.rows;
  const f32x2 off = pair(p.off, p.off);
  Walk walk(r0, r1, p.rows_per_gate, K);
  Ring pos{0, 0u};

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      while (walk.next()) {
        if (issued >= stages &&
            !wait_phase_counted(&sh.empty[pos.stage], pos.phase ^ 1u, abort, &g_block_timeouts))
          break;
        const uint32_t tb = (uint32_t)(walk.n * cols) * (uint32_t)sizeof(T);
        const uint32_t sb = (uint32_t)(walk.n * cols) * (uint32_t)sizeof(TS);
        unsigned char* st = ring + (size_t)pos.stage * sp.stride;
        uint64_t* full = &sh.full[pos.stage];
        const int64_t from = (r0 + walk.row) * p.hidden + col0;  // K is 1 where cs > 1
        mbar_arrive_expect_tx(full, (has_x ? tb : 0) + (NEXT ? tb + sb : 0) + (DR ? sb : 0));
        if (has_x) bulk_load(st, static_cast<const T*>(p.x) + from, tb, full);
        if (NEXT) {
          bulk_load(st + at.r, static_cast<const TS*>(p.r) + from, sb, full);
          bulk_load(st + at.dy, static_cast<const T*>(p.dy) + from, tb, full);
        }
        if (DR) bulk_load(st + at.dr, static_cast<const TS*>(p.dr) + from, sb, full);
        pos.next(stages);
        ++issued;
      }
      drain_ring(sh.full, pos, issued, stages);
    }
    __syncwarp();
  } else if (warp <= reducers) {
    // The reducers' weights: w (without a gate of several rows, which is read
    // from global memory, where L1 holds it) and w2.
    for (int v = threadIdx.x - 32; v < nvec; v += 32 * reducers) {
      f32x2 f[N], g[N];
      if (POST) {
        load_pairs<T, N>(gamma_post + col0 + v * E, f);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = mul2(pair(p.b, p.b), add2(f[i], off));
        if (gate != nullptr && !gate_each) {
          load_pairs<T, N>(gate + col0 + v * E, g);
#pragma unroll
          for (int i = 0; i < N; ++i) f[i] = mul2(f[i], g[i]);
        }
        store_plane<N>(plane1, nvec, v, f);
      }
      if (NEXT) {
        load_pairs<T, N>(gamma_next + col0 + v * E, f);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = add2(f[i], off);
        store_plane<N>(plane2, nvec, v, f);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"r"(32 * reducers) : "memory");
    const float inv = 1.f / (float)p.hidden;
    const int d = warp - 1, lanes = sp.lanes, at_once = 32 / lanes, sub = lane / lanes;
    bool more = walk.next();
    for (int i = 0; i < d && more; ++i) {
      more = walk.next();
      pos.next(stages);
    }
    uint32_t turn = 0;
    while (more) {
      // lane i: the statistics of the stage's row i
      const int64_t row = r0 + walk.row + (lane < walk.n ? lane : 0);
      const float rs1_l = POST ? __ldg(p.rstd_post + row) : 1.f;
      const float rs2_l = NEXT ? __ldg(p.rstd_next + row) : 0.f;
      if (!wait_all(&sh.full[pos.stage], pos.phase, abort)) break;
      const unsigned char* st = ring + (size_t)pos.stage * sp.stride;
      const T* grow = gate_each ? gate + walk.q * p.hidden + col0 : nullptr;
      bool ok = true;
      for (int q0 = 0; q0 < walk.n; q0 += at_once) {
        // lanes past the stage's rows work on its first one, for the shuffles
        const bool mine = q0 + sub < walk.n;
        const int q = mine ? q0 + sub : 0;
        const T* sx = reinterpret_cast<const T*>(st) + q * cols;
        const TS* sr = reinterpret_cast<const TS*>(st + at.r) + q * cols;
        const T* sdy = reinterpret_cast<const T*>(st + at.dy) + q * cols;
        const TS* sdr = reinterpret_cast<const TS*>(st + at.dr) + q * cols;
        const float rs1f = __shfl_sync(0xffffffffu, rs1_l, q);
        const float rs2f = __shfl_sync(0xffffffffu, rs2_l, q);
        const f32x2 rs2 = pair(rs2f, rs2f);
        f32x2 s1 = 0, s2 = 0, s3 = 0;  // S1, and S2 and S3 over rstd_post
        auto add = [&](int v) {
          f32x2 x[N], dv[N];
          if (POST) {
            f32x2 w[N];
            load_pairs<T, N>(sx + v * E, x);
            load_plane<N>(plane1, nvec, v, w);
            if (gate_each) {
              f32x2 g[N];
              load_pairs<T, N>(grow + v * E, g);
#pragma unroll
              for (int k = 0; k < N; ++k) w[k] = mul2(w[k], g[k]);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = mul2(w[k], x[k]);
            if (DR) load_pairs<TS, N>(sdr + v * E, dv);
          }
          if (NEXT) {
            f32x2 r[N], dy[N], w2[N];
            load_pairs<TS, N>(sr + v * E, r);
            load_pairs<T, N>(sdy + v * E, dy);
            load_plane<N>(plane2, nvec, v, w2);
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const f32x2 rh = mul2(r[k], rs2), g = mul2(dy[k], w2[k]);
              s1 = fma2(g, rh, s1);
              if (POST) {
                s3 = fma2(x[k], rh, s3);
                dv[k] = DR ? fma2(rs2, g, dv[k]) : mul2(rs2, g);
              }
            }
          }
          if (POST)
#pragma unroll
            for (int k = 0; k < N; ++k) s2 = fma2(x[k], dv[k], s2);
        };
        float3 s;
        if (lanes < 32) {
          int v = lane & (kNarrowLanes - 1);
          for (; v + 3 * kNarrowLanes < nvec; v += 4 * kNarrowLanes) {
#pragma unroll
            for (int u = 0; u < 4; ++u) add(v + kNarrowLanes * u);
          }
          for (; v < nvec; v += kNarrowLanes) add(v);
          s = make_float3(sum2(s1), sum2(s2), sum2(s3));
#pragma unroll
          for (int m = kNarrowLanes / 2; m >= 1; m /= 2) {
            if (NEXT) s.x += __shfl_xor_sync(0xffffffffu, s.x, m);
            if (POST) s.y += __shfl_xor_sync(0xffffffffu, s.y, m);
            if (POST && NEXT) s.z += __shfl_xor_sync(0xffffffffu, s.z, m);
          }
        } else {
          int v = lane;
          for (; v + 96 < nvec; v += 128) {
#pragma unroll
            for (int u = 0; u < 4; ++u) add(v + 32 * u);
          }
          for (; v < nvec; v += 32) add(v);
          if (POST && NEXT)
            s = warp_sum3(sum2(s1), sum2(s2), sum2(s3), lane);
          else
            s = make_float3(NEXT ? warp_sum(sum2(s1)) : 0.f, POST ? warp_sum(sum2(s2)) : 0.f, 0.f);
        }
        if (cs > 1) {
          // parts of every CTA, added in their order; the slots of a stage are
          // used in turn, so that none is written before it was read
          float4* slot = sh.part[turn & 1u][pos.stage];
          if (lane < cs) {
            st_peer4(slot + rank, lane, make_float4(s.x, s.y, s.z, 0.f));
            mbar_arrive_peer(&sh.parts[pos.stage], lane);
          }
          ok = team_wait(cs, &sh.parts[pos.stage], pos.phase, abort);
          s = make_float3(0.f, 0.f, 0.f);
          for (int i = 0; i < cs; ++i) {
            const float4 f = slot[i];
            s.x += f.x;
            s.y += f.y;
            s.z += f.z;
          }
        }
        const float c1 = s.x * inv;
        const float c2 = POST ? fmaf(-rs2f * c1, s.z, s.y) * (rs1f * inv) : 0.f;
        if ((lane & (lanes - 1)) == 0 && mine)
          sh.stat[pos.stage][q] = make_float4(-c1, -c2, rs1f, rs2f);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.red[pos.stage]);
        mbar_arrive(&sh.empty[pos.stage]);
      }
      // the reducer's next stage is `reducers` on; its turns count the ring's rounds
      const int before = pos.stage;
      for (int i = 0; i < reducers && more; ++i) {
        more = walk.next();
        pos.next(stages);
      }
      if (pos.stage <= before) ++turn;
    }
    __syncwarp();
  } else {
    const int aw = warp - 1 - reducers;
    const int team = aw / sp.wpt, tt = (aw % sp.wpt) * 32 + lane, threads = sp.wpt * 32;
    const bool want_a = POST || gate != nullptr;
    const f32x2 a2 = pair(p.a, p.a);
    unsigned char* dx = reinterpret_cast<unsigned char*>(
        static_cast<T*>(p.dx) + r0 * p.hidden + col0);
    unsigned char* dres = reinterpret_cast<unsigned char*>(
        static_cast<TS*>(p.dres) + r0 * p.hidden + col0);
    const uint32_t tbytes = (uint32_t)(cols * (int)sizeof(T)), sbytes = (uint32_t)(cols * (int)sizeof(TS));
    const uint32_t hbytes_t = (uint32_t)(p.hidden * (int)sizeof(T));
    const uint32_t hbytes_s = (uint32_t)(p.hidden * (int)sizeof(TS));
    // The thread's first columns; threads past the row take its last ones and
    // store nothing.
    int e0[NV];
    f32x2 w[NV][N], w2[NV][N], acc_n[NV][N], acc_a[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tt + j * threads;
      e0[j] = (v < nvec ? v : nvec - 1) * E;
#pragma unroll
      for (int i = 0; i < N; ++i) w2[j][i] = 0;
      if (NEXT) load_pairs<T, N>(gamma_next + col0 + e0[j], w2[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        w2[j][i] = add2(w2[j][i], off);
        acc_n[j][i] = 0;
        acc_a[j][i] = 0;
      }
    }
    bool ok = true;
    bool more = walk.next();
    while (more) {
      const int64_t q = walk.q;
#pragma unroll
      for (int j = 0; j < NV; ++j) {  // the weights of the segment
        f32x2 f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[j][i] = pair(p.b, p.b);
        if (POST) {
          load_pairs<T, N>(gamma_post + col0 + e0[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) w[j][i] = mul2(w[j][i], add2(f[i], off));
        }
        if (gate != nullptr) {
          load_pairs<T, N>(gate + q * p.hidden + col0 + e0[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) w[j][i] = mul2(w[j][i], f[i]);
        }
      }
      for (; more && walk.q == q; more = walk.next()) {
        ok = ok && wait_all(&sh.red[pos.stage], pos.phase, abort) &&
             wait_all(&sh.full[pos.stage], pos.phase, abort);
        const unsigned char* st = ring + (uint32_t)(pos.stage * sp.stride);
        for (int k = team; k < walk.n && ok; k += sp.teams) {
          const float4 stat = sh.stat[pos.stage][k];
          const f32x2 c1 = pair(stat.x, stat.x), c2 = pair(stat.y, stat.y);
          const f32x2 rs1 = pair(stat.z, stat.z), rs2 = pair(stat.w, stat.w);
          const uint32_t row = (uint32_t)(walk.row + k);
          const unsigned char* rt = st + (uint32_t)k * tbytes;
          const unsigned char* rs = st + (uint32_t)k * sbytes;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            f32x2 x[N], dv[N];
            if (DR) load_pairs<TS, N>(reinterpret_cast<const TS*>(rs + at.dr) + e0[j], dv);
            if (NEXT) {
              f32x2 r[N], dy[N];
              load_pairs<TS, N>(reinterpret_cast<const TS*>(rs + at.r) + e0[j], r);
              load_pairs<T, N>(reinterpret_cast<const T*>(rt + at.dy) + e0[j], dy);
#pragma unroll
              for (int i = 0; i < N; ++i) {
                const f32x2 rh = mul2(r[i], rs2);
                const f32x2 g = fma2(c1, rh, mul2(dy[i], w2[j][i]));
                dv[i] = DR ? fma2(rs2, g, dv[i]) : mul2(rs2, g);
                acc_n[j][i] = fma2(dy[i], rh, acc_n[j][i]);
              }
            }
            if (has_x) load_pairs<T, N>(reinterpret_cast<const T*>(rt) + e0[j], x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              if (POST) x[i] = mul2(x[i], rs1);
              if (has_x) acc_a[j][i] = fma2(dv[i], x[i], acc_a[j][i]);
              const f32x2 g = mul2(w[j][i], dv[i]);
              x[i] = POST ? mul2(rs1, fma2(c2, x[i], g)) : g;
              dv[i] = mul2(a2, dv[i]);
            }
            if (tt + j * threads < nvec) {
              store_pairs<T, N>(reinterpret_cast<T*>(dx + (uint64_t)row * hbytes_t) + e0[j], x);
              store_pairs<TS, N>(reinterpret_cast<TS*>(dres + (uint64_t)row * hbytes_s) + e0[j], dv);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[pos.stage]);
        pos.next(stages);
      }

      // the segment's sum of A, and after the last one that of dgamma_next: a
      // thread's own columns, or its columns of the teams' sums, added in turn
      const bool first = q == r0 / p.rows_per_gate;
      float* pa = p.p_a + (unit + q) * p.hidden + col0;
      float* pp = p.p_post + unit * p.hidden + col0;
      float* pn = p.p_next + unit * p.hidden + col0;
      // With one gate row the sums of A give dgamma_post too (block_bwd_sums).
      auto put_a = [&](int c, float4 v) {
        v = make_float4(v.x * p.b, v.y * p.b, v.z * p.b, v.w * p.b);
        *reinterpret_cast<float4*>(pa + c) = v;
        if (POST && gate_each) {
          f32x2 f[2], g[2] = {pair(v.x, v.y), pair(v.z, v.w)};
          load_pairs<T, 2>(gate + q * p.hidden + col0 + c, f);
          const float2 lo = split(mul2(f[0], g[0])), hi = split(mul2(f[1], g[1]));
          float4 s = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<float4*>(pp + c);
          s = make_float4(s.x + lo.x, s.y + lo.y, s.z + hi.x, s.w + hi.y);
          *reinterpret_cast<float4*>(pp + c) = s;
        }
      };
      auto put_n = [&](int c, float4 v) { *reinterpret_cast<float4*>(pn + c) = v; };
      const int me = aw * 32 + lane, all = applier_warps * 32;
      auto flush = [&](auto& acc, auto put) {
        f32x2* comb = reinterpret_cast<f32x2*>(ring + (size_t)stages * sp.stride);
        if (sp.teams == 1) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = tt + j * threads;
            if (v >= nvec) continue;
#pragma unroll
            for (int k = 0; k < N; k += 2) {
              const float2 f = split(acc[j][k]), g = split(acc[j][k + 1]);
              put(v * E + 2 * k, make_float4(f.x, f.y, g.x, g.y));
            }
          }
          return;
        }
        for (int m = 0; m < sp.teams; ++m) {
          if (team == m)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              const int v = tt + j * threads;
              if (v >= nvec) continue;
#pragma unroll
              for (int k = 0; k < N; ++k)
                comb[v * N + k] = m == 0 ? acc[j][k] : add2(comb[v * N + k], acc[j][k]);
            }
          asm volatile("bar.sync 2, %0;" ::"r"(all) : "memory");
        }
        for (int c = 4 * me; c < cols; c += 4 * all)
          put(c, *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(comb) + c));
        asm volatile("bar.sync 2, %0;" ::"r"(all) : "memory");
      };
      if (want_a) flush(acc_a, put_a);
      if (NEXT && !more) flush(acc_n, put_n);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) acc_a[j][k] = 0;
    }
  }
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
  int teams, wpt, cs, stages, stage_rows, stride, lanes, ctas;  // ctas: on an SM
  size_t smem;
};

bool fwd_shape(int64_t rows, int hidden, int sms, int row_elem, int planes, bool post, int align,
               int elems, FwdShape* s) {
  for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
    if (hidden % (align * cs) != 0) return false;
    const int cols = hidden / cs, row = cols * row_elem, over = planes * cols * 4;
    const int64_t mine = (rows * cs + sms - 1) / sms;            // rows an SM, about
    const int groups = cols / elems, most = (groups + 31) / 32;  // warps a row can use
    // Narrow rows in two CTAs an SM, of which one starts while the other
    // ends: 4096 x 1024 fp16 14.0 -> 10.0 us, 32768 x 512 bf16 29.0 -> 27.0
    // (4096 columns: 28.1 -> 31.3).
    s->ctas = cs == 1 && cols <= 1024 && mine > 4 ? 2 : 1;
    const int budget = kSmemBudget / s->ctas - (int)sizeof(FwdShared) - kSlack;
    int stages = (budget - over) / ((row + 127) / 128 * 128);
    if (stages < 2) continue;
    s->cs = cs;
    s->stage_rows = 1;
    s->lanes = 32;
    if (mine <= 2) {  // few rows: all the warps on one
      s->wpt = most < kMaxWarps ? most : kMaxWarps;
      s->teams = 1;
    } else if (s->ctas == 2 || (post && stages >= 8)) {
      // A warp a row, without exchanges, as many as the ring has stages (16
      // on an SM): 4096 x 4096 bf16 with both norms 28.1 us, 30.0 with 4
      // teams of four warps.
      s->wpt = 1;
      s->teams = kMaxWarps / s->ctas;
      // several narrow rows to a stage, as long as every team has its own
      while (s->stage_rows * row < 8192 && mine >= 2 * s->ctas * s->teams * s->stage_rows)
        s->stage_rows *= 2;
      if (groups <= kNarrowGroups && s->stage_rows > 1) s->lanes = kNarrowLanes;
    } else {
      // Teams of four warps leave more of a short ring to the copies, and have
      // one exchange a row without the post norm: 16384 x 8192 bf16 175 us,
      // 194 with teams of two; 4096 x 4096 without the post norm 24.1 us,
      // 25.6 with a warp a row.  fp32 rows have twice the time: two teams,
      // 8192 x 4096 85 us against 89 with four; 16-bit rows under an fp32
      // stream, whose ring holds three stages, teams of two warps: 16384 x
      // 8192 251 us against 266.
      s->wpt = row_elem == 6 ? 2 : 4;
      s->teams = row_elem == 8 ? 2 : 4;
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

// The backward's roles and stages, over as few CTAs as leave three stages
// (else two) beside the reducers' weights.
template <typename F>
bool bwd_pick(int64_t rows, int hidden, int sms, int align, int elems, int planes, F stage_bytes,
              BwdShape* s, int* nv8, size_t* smem) {
  const int budget = kSmemBudget - (int)sizeof(BwdShared) - kSlack;
  for (int least = 3; least >= 2; --least)
    for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
      if (hidden % (align * cs) != 0) break;
      const int cols = hidden / cs;
      *nv8 = cols < 512 ? 1 : 2;
      s->cs = cs;
      s->wpt = (cols + *nv8 * 256 - 1) / (*nv8 * 256);
      if (s->wpt > kBwdWarps - 3) continue;
      s->teams = cs > 1 || s->wpt > 4 ? 1 : 8 / s->wpt;
      // narrow rows: as many to a stage as make it a wide row's, if there are
      // enough of them for every CTA to fill its ring
      s->stage_rows = s->teams;
      while (cs == 1 && 2 * s->stage_rows <= kBwdRows && 2 * s->stage_rows * cols <= 4096 &&
             rows >= (int64_t)8 * s->stage_rows * sms)
        s->stage_rows *= 2;
      s->lanes = cs == 1 && cols / elems <= kNarrowGroups && s->stage_rows > 1 ? kNarrowLanes : 32;
      const int over = planes * cols * 4 + (s->teams > 1 ? cols * 4 : 0);
      s->stride = (stage_bytes(s->stage_rows, cols) + 127) / 128 * 128;
      s->stages = (budget - over) / s->stride;
      if (s->stages > kBwdStages) s->stages = kBwdStages;
      if (s->stages < least) continue;
      s->reducers = kBwdWarps - 1 - s->teams * s->wpt;
      if (s->reducers > s->stages) s->reducers = s->stages;
      s->stages -= s->stages % s->reducers;  // a stage is always the same reducer's
      *smem = (size_t)s->stages * s->stride + over;
      return true;
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
                 POST, 16 / (int)sizeof(T), E, &sh))
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
  p.lanes = sh.lanes;
  auto kern = block_fwd_tma<T, TS, POST, NEXT>;
  *err = allow_smem(kern, sh.smem);
  if (*err == cudaSuccess) *err = allow_cluster((const void*)kern, sh.cs);
  if (*err != cudaSuccess) return true;
  const int threads = 32 * (1 + sh.teams * sh.wpt);
  int64_t units = sh.cs == 1 ? (int64_t)sms * sh.ctas : max_clusters((const void*)kern, threads, sh.smem, sh.cs, sms);
  const int64_t blocks = (a.rows + sh.stage_rows - 1) / sh.stage_rows;
  if (units > blocks) units = blocks;
  if (units < 1) units = 1;
  *err = launch_kernel(kern, dim3((unsigned)(units * sh.cs)), dim3(threads), sh.smem, s,
                       sh.cs, p);
  return true;
}

template <typename T, typename TS, bool POST, bool NEXT>
bool try_bwd(const BlockBwdArgs& a, BlockBwdParams& p, int* units, cudaStream_t s,
             cudaError_t* err) {
  constexpr int E = kElems<T, TS>;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return true;
  const int sms = sm_count(dev);
  BwdShape sp;
  sp.read_x = POST || a.gate != nullptr;
  const bool dr = a.dr != nullptr, x = sp.read_x;
  int nv8 = 0;
  size_t smem = 0;
  if (!bwd_pick(a.rows, a.hidden, sms, 16 / (int)sizeof(T), E, (POST ? 1 : 0) + (NEXT ? 1 : 0),
                [=](int k, int cols) { return bwd_stage<T, TS>(k, cols, x, NEXT, dr).bytes; }, &sp,
                &nv8, &smem))
    return false;
  auto go = [&](auto kern) {
    *err = allow_smem(kern, smem);
    if (*err == cudaSuccess) *err = allow_cluster((const void*)kern, sp.cs);
    if (*err != cudaSuccess) return;
    const int threads = 32 * (1 + sp.reducers + sp.teams * sp.wpt);
    int64_t n = sp.cs == 1 ? sms : max_clusters((const void*)kern, threads, smem, sp.cs, sms);
    if (n < 1) n = 1;
    if (n > RMSN_BLOCK_MAX_PARTIALS) n = RMSN_BLOCK_MAX_PARTIALS;
    if (n > a.rows) n = a.rows;
    *units = (int)n;
    place_partials(a, *units, p);
    *err = launch_kernel(kern, dim3((unsigned)(n * sp.cs)), dim3(threads), smem, s, sp.cs, p, sp);
  };
  if (dr || !NEXT) {
    if (nv8 == 1)
      go(block_bwd_tma<T, TS, POST, NEXT, true, 8 / E>);
    else
      go(block_bwd_tma<T, TS, POST, NEXT, true, 16 / E>);
  } else {
    if (nv8 == 1)
      go(block_bwd_tma<T, TS, POST, true, false, 8 / E>);
    else
      go(block_bwd_tma<T, TS, POST, true, false, 16 / E>);
  }
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
