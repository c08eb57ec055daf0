// Staged block norm for sm_103a (the formulas are in block_norm.cu).
//
// Both directions are bound by HBM bandwidth: the forward moves 2 + 2 and the
// backward 4 + 2 rows for each row, against 20 to 30 instructions an element.
// What decides the speed is how many bytes an SM keeps in flight while the
// row's reductions, which nothing of the row can be written before, run.
//
// A persistent CTA per SM (or cluster of CTAs, for rows too wide for one)
// streams its rows with 1D bulk copies into a ring of shared-memory stages
// (producer: warp 0, one thread; full[s] when a stage has landed) and all its
// other warps are consumers, in teams: a team of H / 8 or H / 16 threads works
// on one row, and a stage holds one row a team, so that narrow rows fill the
// CTA as wide ones do.  A thread owns the same columns of every row; their
// weights, and in the backward their fp32 sums over rows, stay in its
// registers.
//
// The reductions never stop a team.  A warp puts its part of a row's sums
// into a slot and arrives on the row's barrier (red), of every CTA of the
// cluster; before it waits for that barrier it does other work:
//   forward   B(i): r of row i, its sum of squares -> red2
//             A(i + 1): sum of squares of x of the next row -> red1
//             C(i): wait red2, y of row i (r kept in registers from B)
//             and B(i + 1) waits for red1, which C(i) has covered
//   backward  A(i + 1): the three sums of the next row -> red
//             B(i): wait red, dx and dresidual of row i, read again from its stage
// Slots and red barriers of the forward are two deep and those of the
// backward four deep: a warp writes those of row i + 2 (i + 4) only after a
// wait that every reader of row i has passed.
//
// Every wait is bounded (mbar.cuh); a consumer whose wait ran out skips the
// rest of its rows but still reaches the CTA's and the cluster's barriers.
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

template <typename U, int E>
__device__ __forceinline__ void load_elems(const U* p, float (&f)[E]) {
  if constexpr (E * sizeof(U) == 16) {
    unpack<U>(*reinterpret_cast<const uint4*>(p), f);
  } else {
    static_assert(E * sizeof(U) == 8, "8 or 16 bytes");
    unpack_h<U>(*reinterpret_cast<const uint2*>(p), f);
  }
}

template <typename U, int E>
__device__ __forceinline__ void store_elems(U* p, const float (&f)[E]) {
  if constexpr (E * sizeof(U) == 16)
    st_vec(p, pack<U>(f));
  else
    *reinterpret_cast<uint2*>(p) = pack_h<U>(f);
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

// Posts the warp's part v (the same in every lane) in slot and arrives.
__device__ __forceinline__ void post(const Team& t, float* slot, uint64_t* bar, float v) {
  if (t.cs == 1) {
    if (t.lane == 0) {
      slot[t.tw] = v;
      mbar_arrive(bar);
    }
  } else if (t.lane < t.cs) {
    st_peer(slot + t.rank * t.wpt + t.tw, t.lane, v);
    mbar_arrive_peer(bar, t.lane);
  }
}

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

// Sum of a team's parts, in the same order in every thread.
__device__ __forceinline__ float total(const Team& t, const float* slot) {
  const int n = t.cs * t.wpt;
  float v = 0.f;
  for (int i = t.lane; i < n; i += 32) v += slot[i];
  return warp_sum(v);
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
  int teams, wpt, cs, stages, stride;  // stride: bytes a stage
};

struct FwdShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t red1[kMaxWarps][2];   // of a team: sum x^2 of a row
  uint64_t red2[kMaxWarps][2];   // sum r^2
  uint64_t redx[kMaxWarps][2];   // the same sums again, rescaled
  float slot1[2][kMaxWarps * kMaxSplit];
  float slot2[2][kMaxWarps * kMaxSplit];
  float slotx[2][kMaxWarps * kMaxSplit];
  int abort;
};

template <typename T, typename TS, bool POST, bool NEXT, int NV>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1)) block_fwd_tma(const BlockFwdParams p) {
  constexpr int E = kElems<T, TS>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ FwdShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = p.teams, stages = p.stages, cs = p.cs;
  const int cols = p.hidden / cs;
  const uint32_t rank = cs > 1 ? cta_rank() : 0u;
  const int64_t unit = blockIdx.x / cs, units = gridDim.x / cs;
  // stage k of a unit holds the rows [(k units + unit) K, + K): the grid
  // streams one window of consecutive rows
  const int64_t blocks = (p.rows + K - 1) / K;
  const int64_t nst = blocks > unit ? (blocks - unit + units - 1) / units : 0;
  for (int i = threadIdx.x; i < kMaxStages + kMaxWarps; i += blockDim.x) {
    if (i < stages) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], K * p.wpt);
    }
    if (i >= kMaxStages) {
      const int t = i - kMaxStages;
      for (int d = 0; d < 2; ++d) {
        mbar_init(&sh.red1[t][d], cs * p.wpt);
        mbar_init(&sh.red2[t][d], cs * p.wpt);
        mbar_init(&sh.redx[t][d], cs * p.wpt);
      }
    }
  }
  if (threadIdx.x == 0) sh.abort = 0;
  fence_mbar_init();
  __syncthreads();
  if (cs > 1) cluster_sync();
  pdl_trigger();
  pdl_wait();
  volatile int* abort = &sh.abort;
  const uint32_t xbytes = (uint32_t)(cols * sizeof(T)), sbytes = (uint32_t)(cols * sizeof(TS));
  const int res_at = K * (int)xbytes;

  if (warp == 0) {
    if (lane == 0) {
      Ring pos{0, 0u};
      int64_t k = 0;
      for (; k < nst; ++k) {
        if (k >= stages &&
            !wait_phase_counted(&sh.empty[pos.stage], pos.phase ^ 1u, abort, &g_block_timeouts))
          break;
        const int64_t row = (k * units + unit) * K;
        const uint32_t n = (uint32_t)(p.rows - row < K ? p.rows - row : K);
        unsigned char* st = ring + (size_t)pos.stage * p.stride;
        const int64_t at = row * p.hidden + (int64_t)rank * cols;  // K is 1 where cs > 1
        mbar_arrive_expect_tx(&sh.full[pos.stage], n * (xbytes + sbytes));
        bulk_load(st, static_cast<const T*>(p.x) + at, n * xbytes, &sh.full[pos.stage]);
        bulk_load(st + res_at, static_cast<const TS*>(p.res) + at, n * sbytes,
                  &sh.full[pos.stage]);
        pos.next(stages);
      }
      drain_ring(sh.full, pos, k, stages);
    }
    __syncwarp();
  } else {
    const int team = (warp - 1) / p.wpt;
    Team t{p.wpt, cs, (warp - 1) % p.wpt, lane, rank, abort};
    const bool alone = p.wpt == 1 && cs == 1;  // a warp's sums need no exchange
    const int tt = t.tw * 32 + lane, threads = p.wpt * 32;
    const int nvec = cols / E, col0 = (int)rank * cols;
    const float inv = 1.f / (float)p.hidden;
    float* slot1[2] = {sh.slot1[0] + team * p.wpt, sh.slot1[1] + team * p.wpt};
    float* slot2[2] = {sh.slot2[0] + team * p.wpt, sh.slot2[1] + team * p.wpt};
    float* slotx[2] = {sh.slotx[0] + team * p.wpt, sh.slotx[1] + team * p.wpt};
    float w[NV][E], w2[NV][E], r[NV][E];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tt + j * threads;
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 0.f;
      if (NEXT && v < nvec) load_elems<T, E>(static_cast<const T*>(p.gamma_next) + col0 + v * E, f);
#pragma unroll
      for (int e = 0; e < E; ++e) w2[j][e] = f[e] + p.off;
    }
    int64_t gate_row = -1;
    uint32_t xphase[2] = {0u, 0u};
    float ss1 = 0.f;  // a lone warp's sum of squares of the next row
    bool ok = true;
    Ring pos{0, 0u};
    // A: the stage's row of this team, if it has one
    auto sum_x = [&](int64_t k, const Ring& at) {
      ok = ok && wait_all(&sh.full[at.stage], at.phase, abort);
      if (!POST || !ok || (k * units + unit) * K + team >= p.rows) return;
      const T* sx = reinterpret_cast<const T*>(ring + (size_t)at.stage * p.stride) + team * cols;
      float part[E];
#pragma unroll
      for (int e = 0; e < E; ++e) part[e] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = tt + j * threads;
        if (v >= nvec) continue;
        float f[E];
        load_elems<T, E>(sx + v * E, f);
#pragma unroll
        for (int e = 0; e < E; ++e) part[e] = fmaf(f[e], f[e], part[e]);
      }
#pragma unroll
      for (int h = E / 2; h >= 1; h /= 2)
#pragma unroll
        for (int e = 0; e < h; ++e) part[e] += part[e + h];
      ss1 = warp_sum(part[0]);
      if (!alone) post(t, slot1[k & 1], &sh.red1[team][k & 1], ss1);
    };
    // the rescaled sums of a row whose squares overflowed (kOverflowScale)
    auto again = [&](int which, float part) {
      float s = warp_sum(part);
      if (alone) return s;
      post(t, slotx[which], &sh.redx[team][which], s);
      ok = team_wait(t, &sh.redx[team][which], xphase[which]);
      xphase[which] ^= 1u;
      return total(t, slotx[which]);
    };
    if (nst > 0) sum_x(0, pos);
    for (int64_t k = 0; k < nst; ++k) {
      const int64_t row = (k * units + unit) * K + team;
      const uint32_t parity = (uint32_t)(k >> 1) & 1u;
      Ring after = pos;
      after.next(stages);
      const bool mine = ok && row < p.rows;
      float ss2 = 0.f;
      if (mine) {
        const unsigned char* st = ring + (size_t)pos.stage * p.stride;
        const T* sx = reinterpret_cast<const T*>(st) + team * cols;
        const TS* sr = reinterpret_cast<const TS*>(st + res_at) + team * cols;
        float rs1 = 1.f;
        if (POST) {
          float ss = ss1;
          if (!alone) {
            ok = team_wait(t, &sh.red1[team][k & 1], parity);
            ss = total(t, slot1[k & 1]);
          }
          rs1 = rstd_of(ss * inv, p.eps);
          if (isinf(ss) && ok) {
            float part = 0.f;
            for (int v = tt; v < nvec; v += threads) {
              float f[E];
              load_elems<T, E>(sx + v * E, f);
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const float q = f[e] * kOverflowScale;
                part = fmaf(q, q, part);
              }
            }
            rs1 = rstd_rescaled(again(0, part), p.hidden, p.eps);
          }
          if (tt == 0 && rank == 0) p.rstd_post[row] = rs1;
        }
        const int64_t q = row / p.rows_per_gate;
        if (q != gate_row) {  // the weights of the row's gate
          gate_row = q;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = tt + j * threads;
            float f[E], g[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
              f[e] = 1.f - p.off;
              g[e] = 1.f;
            }
            if (POST && v < nvec)
              load_elems<T, E>(static_cast<const T*>(p.gamma_post) + col0 + v * E, f);
            if (p.gate != nullptr && v < nvec)
              load_elems<T, E>(static_cast<const T*>(p.gate) + q * p.hidden + col0 + v * E, g);
#pragma unroll
            for (int e = 0; e < E; ++e) w[j][e] = p.b * g[e] * (f[e] + p.off);
          }
        }
        float part[E];
#pragma unroll
        for (int e = 0; e < E; ++e) part[e] = 0.f;
        TS* out = static_cast<TS*>(p.res_out) + row * p.hidden + col0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int v = tt + j * threads;
          if (v >= nvec) continue;
          float f[E], g[E];
          load_elems<T, E>(sx + v * E, f);
          load_elems<TS, E>(sr + v * E, g);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            r[j][e] = fmaf(w[j][e], f[e] * rs1, p.a * g[e]);
            part[e] = fmaf(r[j][e], r[j][e], part[e]);
          }
          store_elems<TS, E>(out + v * E, r[j]);
        }
        if (NEXT) {
#pragma unroll
          for (int h = E / 2; h >= 1; h /= 2)
#pragma unroll
            for (int e = 0; e < h; ++e) part[e] += part[e + h];
          ss2 = warp_sum(part[0]);
          if (!alone) post(t, slot2[k & 1], &sh.red2[team][k & 1], ss2);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[pos.stage]);
      if (k + 1 < nst) sum_x(k + 1, after);
      if (NEXT && mine && ok) {
        float ss = ss2;
        if (!alone) {
          ok = team_wait(t, &sh.red2[team][k & 1], parity);
          ss = total(t, slot2[k & 1]);
        }
        float rs2 = rstd_of(ss * inv, p.eps);
        if (isinf(ss) && ok) {
          float part = 0.f;
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (tt + j * threads < nvec)
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const float q = r[j][e] * kOverflowScale;
                part = fmaf(q, q, part);
              }
          rs2 = rstd_rescaled(again(1, part), p.hidden, p.eps);
        }
        if (tt == 0 && rank == 0) p.rstd_next[row] = rs2;
        T* out = static_cast<T*>(p.y) + row * p.hidden + col0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int v = tt + j * threads;
          if (v >= nvec) continue;
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = (r[j][e] * rs2) * w2[j][e];
          store_elems<T, E>(out + v * E, o);
        }
      }
      pos = after;
    }
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while a peer may write to its slots
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
constexpr int kDepth = 4;

struct BwdShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t red[kMaxWarps][kDepth];
  float4 slot[kDepth][kMaxWarps * kMaxSplit];
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
__global__ void __launch_bounds__(32 * (kMaxWarps + 1), 1)
    block_bwd_tma(const BlockBwdParams p, const BwdShape sp) {
  constexpr int E = kElems<T, TS>;
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
  if (threadIdx.x == 0) sh.abort = 0;
  fence_mbar_init();
  __syncthreads();
  if (cs > 1) cluster_sync();
  pdl_trigger();
  pdl_wait();
  volatile int* abort = &sh.abort;
  const BwdStage at = bwd_stage<T, TS>(K, cols, has_x, NEXT, has_dr);

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t tb = (uint32_t)(cols * sizeof(T)), sb = (uint32_t)(cols * sizeof(TS));
      const uint32_t row_bytes =
          (has_x ? tb : 0) + (NEXT ? tb + sb : 0) + (has_dr ? sb : 0);
      Ring pos{0, 0u};
      int64_t issued = 0;
      // a stage never crosses from one gate row to the next
      for (int64_t row = r0; row < r1;) {
        const int64_t seg = (row / p.rows_per_gate + 1) * p.rows_per_gate;
        const int64_t end = seg < r1 ? seg : r1;
        const uint32_t n = (uint32_t)(end - row < K ? end - row : K);
        if (issued >= stages &&
            !wait_phase_counted(&sh.empty[pos.stage], pos.phase ^ 1u, abort, &g_block_timeouts))
          break;
        unsigned char* st = ring + (size_t)pos.stage * sp.stride;
        uint64_t* full = &sh.full[pos.stage];
        const int64_t from = row * p.hidden + (int64_t)rank * cols;  // K is 1 where cs > 1
        mbar_arrive_expect_tx(full, n * row_bytes);
        if (has_x) bulk_load(st, static_cast<const T*>(p.x) + from, n * tb, full);
        if (NEXT) {
          bulk_load(st + at.r, static_cast<const TS*>(p.r) + from, n * sb, full);
          bulk_load(st + at.dy, static_cast<const T*>(p.dy) + from, n * tb, full);
        }
        if (has_dr) bulk_load(st + at.dr, static_cast<const TS*>(p.dr) + from, n * sb, full);
        pos.next(stages);
        ++issued;
        row += n;
      }
      drain_ring(sh.full, pos, issued, stages);
    }
    __syncwarp();
  } else {
    const int team = (warp - 1) / sp.wpt;
    Team t{sp.wpt, cs, (warp - 1) % sp.wpt, lane, rank, abort};
    const bool alone = sp.wpt == 1 && cs == 1;
    const int tt = t.tw * 32 + lane, threads = sp.wpt * 32;
    const int nvec = cols / E, col0 = (int)rank * cols;
    const float inv = 1.f / (float)p.hidden;
    const bool want_a = POST || p.gate != nullptr;
    const T* gamma_post = static_cast<const T*>(p.gamma_post);
    const T* gate = static_cast<const T*>(p.gate);
    float w[NV][E], w2[NV][E], acc_n[NV][E], acc_a[NV][E];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = tt + j * threads;
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 0.f;
      if (NEXT && v < nvec) load_elems<T, E>(static_cast<const T*>(p.gamma_next) + col0 + v * E, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w2[j][e] = f[e] + p.off;
        acc_n[j][e] = 0.f;
        acc_a[j][e] = 0.f;
      }
    }
    bool ok = true;
    Ring pos_a{0, 0u}, pos_b{0, 0u};
    uint32_t posted = 0, taken = 0;  // rows of this team whose sums were posted, used
    float3 own = make_float3(0.f, 0.f, 0.f);  // a lone warp's sums of the row in A
    float rs1_a = 1.f, rs2_a = 0.f, rs1_b = 1.f, rs2_b = 0.f;
    float3 sums_b = own;

    for (int64_t seg0 = r0; seg0 < r1;) {
      const int64_t q = seg0 / p.rows_per_gate;
      const int64_t seg1 = (q + 1) * p.rows_per_gate < r1 ? (q + 1) * p.rows_per_gate : r1;
      const int nst = (int)((seg1 - seg0 + K - 1) / K);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = tt + j * threads;
        float f[E], g[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          f[e] = 1.f - p.off;
          g[e] = 1.f;
        }
        if (POST && v < nvec) load_elems<T, E>(gamma_post + col0 + v * E, f);
        if (gate != nullptr && v < nvec)
          load_elems<T, E>(gate + q * p.hidden + col0 + v * E, g);
#pragma unroll
        for (int e = 0; e < E; ++e) w[j][e] = p.b * g[e] * (f[e] + p.off);
      }
      auto row_of = [&](int i) { return seg0 + (int64_t)i * K + team; };
      auto stats = [&](int i) {  // the row statistics, loaded a row ahead of their use
        const int64_t row = row_of(i);
        if (row < seg1) {
          if (POST) rs1_a = __ldg(p.rstd_post + row);
          if (NEXT) rs2_a = __ldg(p.rstd_next + row);
        }
      };
      float rs1_n = 1.f, rs2_n = 0.f;
      auto sums = [&](int i) {  // A
        ok = ok && wait_all(&sh.full[pos_a.stage], pos_a.phase, abort);
        rs1_n = rs1_a;
        rs2_n = rs2_a;
        if (i + 1 < nst) stats(i + 1);
        if (ok && row_of(i) < seg1) {
          const unsigned char* st = ring + (size_t)pos_a.stage * sp.stride;
          const T* sx = reinterpret_cast<const T*>(st) + team * cols;
          const TS* sr = reinterpret_cast<const TS*>(st + at.r) + team * cols;
          const T* sdy = reinterpret_cast<const T*>(st + at.dy) + team * cols;
          const TS* sdr = reinterpret_cast<const TS*>(st + at.dr) + team * cols;
          float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = tt + j * threads;
            if (v >= nvec) continue;
            float x[E], r[E], dy[E], d[E];
            if (POST) load_elems<T, E>(sx + v * E, x);
            if (NEXT) {
              load_elems<TS, E>(sr + v * E, r);
              load_elems<T, E>(sdy + v * E, dy);
            }
            if (POST) {
              if (has_dr) {
                load_elems<TS, E>(sdr + v * E, d);
              } else {
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = 0.f;
              }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
              float rh = 0.f, g = 0.f;
              if (NEXT) {
                rh = r[e] * rs2_n;
                g = dy[e] * w2[j][e];
                s1 = fmaf(g, rh, s1);
              }
              if (POST) {
                const float wx = w[j][e] * (x[e] * rs1_n);
                s2 = fmaf(wx, NEXT ? fmaf(rs2_n, g, d[e]) : d[e], s2);
                if (NEXT) s3 = fmaf(wx, rh, s3);
              }
            }
          }
          if (POST && NEXT)
            own = warp_sum3(s1, s2, s3, lane);
          else
            own = make_float3(NEXT ? warp_sum(s1) : 0.f, POST ? warp_sum(s2) : 0.f, 0.f);
          if (!alone)
            post3(t, sh.slot[posted % kDepth] + team * sp.wpt * cs, &sh.red[team][posted % kDepth],
                  make_float4(own.x, own.y, own.z, 0.f));
          ++posted;
        }
        pos_a.next(stages);
      };
      stats(0);
      sums(0);
      for (int i = 0; i < nst; ++i) {
        rs1_b = rs1_n;
        rs2_b = rs2_n;
        sums_b = own;
        if (i + 1 < nst) sums(i + 1);
        const int64_t row = row_of(i);
        if (ok && row < seg1) {  // B
          float3 s = sums_b;
          if (!alone) {
            ok = team_wait(t, &sh.red[team][taken % kDepth], (taken / kDepth) & 1u);
            s = total3(t, sh.slot[taken % kDepth] + team * sp.wpt * cs);
          }
          ++taken;
          const float c1 = s.x * inv;
          const float c2 = POST ? fmaf(-rs2_b * c1, s.z, s.y) * inv : 0.f;
          const unsigned char* st = ring + (size_t)pos_b.stage * sp.stride;
          const T* sx = reinterpret_cast<const T*>(st) + team * cols;
          const TS* sr = reinterpret_cast<const TS*>(st + at.r) + team * cols;
          const T* sdy = reinterpret_cast<const T*>(st + at.dy) + team * cols;
          const TS* sdr = reinterpret_cast<const TS*>(st + at.dr) + team * cols;
          T* dx = static_cast<T*>(p.dx) + row * p.hidden + col0;
          TS* dres = static_cast<TS*>(p.dres) + row * p.hidden + col0;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = tt + j * threads;
            if (v >= nvec) continue;
            float x[E], r[E], dy[E], d[E], o[E];
            if (has_x) {
              load_elems<T, E>(sx + v * E, x);
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e) x[e] = 0.f;
            }
            if (has_dr) {
              load_elems<TS, E>(sdr + v * E, d);
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e) d[e] = 0.f;
            }
            if (NEXT) {
              load_elems<TS, E>(sr + v * E, r);
              load_elems<T, E>(sdy + v * E, dy);
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const float rh = r[e] * rs2_b;
                d[e] = fmaf(rs2_b, fmaf(-rh, c1, dy[e] * w2[j][e]), d[e]);
                acc_n[j][e] = fmaf(dy[e], rh, acc_n[j][e]);
              }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float xh = POST ? x[e] * rs1_b : x[e];
              acc_a[j][e] = fmaf(d[e], xh, acc_a[j][e]);
              o[e] = POST ? rs1_b * fmaf(-xh, c2, w[j][e] * d[e]) : w[j][e] * d[e];
              d[e] *= p.a;
            }
            store_elems<T, E>(dx + v * E, o);
            store_elems<TS, E>(dres + v * E, d);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[pos_b.stage]);
        pos_b.next(stages);
      }

      // the segment's sum of A, and after the last one that of dgamma_next:
      // a thread's own columns, or its columns of the teams' sums
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
      if (K == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int v = tt + j * threads;
          if (v >= nvec) continue;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (want_a) put_a(v * E + e, acc_a[j][e]);
            if (NEXT && last) pn[v * E + e] = acc_n[j][e];
            acc_a[j][e] = 0.f;
          }
        }
      } else {
        float* comb = reinterpret_cast<float*>(ring + (size_t)stages * sp.stride);
        const int consumers = blockDim.x - 32;
        auto join = [&](float (&acc)[NV][E], auto put) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = tt + j * threads;
            if (v >= nvec) continue;
#pragma unroll
            for (int e = 0; e < E; e += 4)
              *reinterpret_cast<float4*>(comb + team * cols + v * E + e) =
                  make_float4(acc[j][e], acc[j][e + 1], acc[j][e + 2], acc[j][e + 3]);
          }
          asm volatile("bar.sync 1, %0;" ::"r"(consumers) : "memory");
          for (int c = threadIdx.x - 32; c < cols; c += consumers) {
            float v = 0.f;
            for (int m = 0; m < K; ++m) v += comb[m * cols + c];
            put(c, v);
          }
          asm volatile("bar.sync 1, %0;" ::"r"(consumers) : "memory");
        };
        if (want_a) join(acc_a, put_a);
        if (NEXT && last) join(acc_n, [&](int c, float v) { pn[c] = v; });
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) acc_a[j][e] = 0.f;
      }
      seg0 = seg1;
    }
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while a peer may write to its slots
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Threads and stages for rows of `hidden` elements, `unit_bytes(k, cols)` the
// bytes of a stage of k rows of cols columns and `extra` those beside the
// ring.  The row is split over as few CTAs as leave `want` stages (else 2).
struct Shape {
  int teams, wpt, cs, stages, stride, nv8;  // nv8: groups of 8 columns a thread
  size_t smem;
};

template <typename F, typename X>
bool pick_shape(int hidden, int want, F unit_bytes, X extra, int budget, Shape* out) {
  for (int least = want; least >= 2; least -= want > 2 ? want - 2 : 1) {
    for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
      if (hidden % (8 * cs) != 0) break;
      const int cols = hidden / cs;
      if (cols > 16 * 32 * kMaxWarps) continue;
      Shape s;
      s.cs = cs;
      s.nv8 = cols <= 8 * 32 * kMaxWarps ? 1 : 2;
      s.wpt = (cols / 8 + s.nv8 * 32 - 1) / (s.nv8 * 32);
      s.teams = cs > 1 ? 1 : kMaxWarps / s.wpt;
      s.stride = (unit_bytes(s.teams, cols) + 127) / 128 * 128;
      const int over = s.teams > 1 ? extra(s.teams, cols) : 0;
      s.stages = (budget - over) / s.stride;
      if (s.stages > kMaxStages) s.stages = kMaxStages;
      if (s.stages < least) continue;
      s.smem = (size_t)s.stages * s.stride + over;
      *out = s;
      return true;
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
  Shape sh;
  if (!pick_shape(a.hidden, 3,
                  [](int k, int cols) { return k * cols * (int)(sizeof(T) + sizeof(TS)); },
                  [](int, int) { return 0; }, kSmemBudget - (int)sizeof(FwdShared), &sh))
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
  p.stride = sh.stride;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return true;
  auto go = [&](auto kern) {
    *err = allow_smem(kern, sh.smem);
    if (*err != cudaSuccess) return;
    const int threads = 32 * (1 + sh.teams * sh.wpt);
    const int64_t occ = max_blocks_per_sm((const void*)kern, threads, sh.smem);
    int64_t units = sm_count(dev) * occ / sh.cs;
    const int64_t blocks = (a.rows + sh.teams - 1) / sh.teams;
    if (units > blocks) units = blocks;
    if (units < 1) units = 1;
    *err = launch_kernel(kern, dim3((unsigned)(units * sh.cs)), dim3(threads), sh.smem, s, sh.cs,
                         p);
  };
  if (sh.nv8 == 1)
    go(block_fwd_tma<T, TS, POST, NEXT, 8 / E>);
  else
    go(block_fwd_tma<T, TS, POST, NEXT, 16 / E>);
  return true;
}

template <typename T, typename TS, bool POST, bool NEXT>
bool try_bwd(const BlockBwdArgs& a, BlockBwdParams& p, int* units, cudaStream_t s,
             cudaError_t* err) {
  constexpr int E = kElems<T, TS>;
  BwdShape sp;
  sp.read_x = POST || a.gate != nullptr;
  const bool dr = a.dr != nullptr, x = sp.read_x;
  Shape sh;
  if (!pick_shape(a.hidden, 3,
                  [=](int k, int cols) { return bwd_stage<T, TS>(k, cols, x, NEXT, dr).bytes; },
                  [](int k, int cols) { return k * cols * 4; }, kSmemBudget - (int)sizeof(BwdShared),
                  &sh))
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
    const int threads = 32 * (1 + sh.teams * sh.wpt);
    *err = launch_kernel(kern, dim3((unsigned)(n * sh.cs)), dim3(threads), sh.smem, s, sh.cs, p,
                         sp);
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
