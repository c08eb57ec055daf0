// Backward of the staged block norm (block_norm_tma.cuh, formulas in
// block_norm.cu), for block_bwd_tma.cu and block_bwd_odd.cu.
#pragma once

#include "block_norm_tma.cuh"

namespace rmsn {
namespace {

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

// The stages of a unit's rows, in order.  The unit's rows are c + P i for i in
// [i0, i1) (c 0 and P 1 where rows are aligned); a stage is the n of them from
// i0 + `at` on, all of gate row q.
struct Walk {
  int at, n, end, total, most, c, p;
  int64_t q, i0, rows_per_gate;
  __device__ Walk(int64_t i0, int64_t i1, int64_t rpg, int stage_rows, int c, int p)
      : at(0), n(0), total((int)(i1 - i0)), most(stage_rows), c(c), p(p),
        q((c + i0 * p) / rpg), i0(i0), rows_per_gate(rpg) {
    end = end_of();
  }
  __device__ __forceinline__ int64_t row(int k) const { return c + (i0 + at + k) * p; }
  __device__ int end_of() const {  // where gate row q ends
    const int64_t i = ((q + 1) * rows_per_gate - c + p - 1) / p - i0;
    return i < total ? (int)i : total;
  }
  __device__ __forceinline__ bool next() {
    at += n;
    if (at >= total) return false;
    if (at == end) {
      ++q;
      end = end_of();
    }
    n = end - at < most ? end - at : most;
    return true;
  }
};

template <typename T, typename TS, bool POST, bool NEXT, bool DR, int NV, bool EDGE>
__global__ void __launch_bounds__(32 * kBwdWarps, 1)
    block_bwd_tma(const BlockBwdParams p, const BwdShape sp) {
  constexpr int E = kElems<T, TS>, N = E / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ BwdShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = sp.stages, cs = sp.cs, K = sp.stage_rows, reducers = sp.reducers;
  const int applier_warps = sp.teams * sp.wpt;
  constexpr int A = 16 / sizeof(T);
  const uint32_t rank = cs > 1 ? cta_rank() : 0u;
  const int64_t unit = blockIdx.x / cs, units = gridDim.x / cs;
  const int P = EDGE ? p.period : 1;
  const int cls = EDGE ? (int)(unit % P) : 0;
  const Part part(p.hidden, A, cs, rank, cls, EDGE);
  const int pitch = part.pitch, col0 = part.col0;
  const int nvec = EDGE ? (part.span + E - 1) / E : pitch / E;
  // the unit's share of the rows of its class
  const int64_t ours = EDGE ? (p.rows - cls + P - 1) / P : p.rows;
  const int64_t of = EDGE ? units / P : units, idx = EDGE ? unit / P : unit;
  const int64_t i0 = idx * ours / of, i1 = (idx + 1) * ours / of;
  const bool has_x = POST || sp.read_x;
  if (!EDGE && threadIdx.x == 0) {  // the first rows into L2 (prefetch_l2)
    int64_t n = K * kFirstStages;
    if (n > i1 - i0) n = i1 - i0;
    for (int64_t i = i0; i < i0 + n; i += cs == 1 ? n : 1) {  // consecutive, or this CTA's part
      const int64_t from = i * p.hidden + col0;
      const uint32_t m = (uint32_t)((cs == 1 ? n : 1) * pitch);
      if (has_x) prefetch_l2(static_cast<const T*>(p.x) + from, m * (uint32_t)sizeof(T));
      if (NEXT) prefetch_l2(static_cast<const TS*>(p.r) + from, m * (uint32_t)sizeof(TS));
      if (NEXT) prefetch_l2(static_cast<const T*>(p.dy) + from, m * (uint32_t)sizeof(T));
      if (DR) prefetch_l2(static_cast<const TS*>(p.dr) + from, m * (uint32_t)sizeof(TS));
    }
  }
  float4* plane1 = reinterpret_cast<float4*>(smem);
  float4* plane2 = POST ? plane1 + pitch / 4 : plane1;
  unsigned char* ring = reinterpret_cast<unsigned char*>(NEXT ? plane2 + pitch / 4 : plane2);
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
  const BwdStage at = bwd_stage<T, TS>(K, pitch, has_x, NEXT, DR);
  const T* gamma_post = static_cast<const T*>(p.gamma_post);
  const T* gamma_next = static_cast<const T*>(p.gamma_next);
  const T* gate = static_cast<const T*>(p.gate);
  const bool gate_each = gate != nullptr && p.rows_per_gate < p.rows;
  const f32x2 off = pair(p.off, p.off);
  const uint32_t tpitch = (uint32_t)(pitch * (int)sizeof(T));
  const uint32_t spitch = (uint32_t)(pitch * (int)sizeof(TS));
  Walk walk(i0, i1, p.rows_per_gate, K, cls, P);
  Ring pos{0, 0u};

  if (warp == 0) {
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    const TS* r = static_cast<const TS*>(p.r);
    const TS* dr = static_cast<const TS*>(p.dr);
    int issued = 0;
    while (walk.next()) {
      bool go = true;
      if (issued >= stages && lane == 0)
        go = wait_phase_counted(&sh.empty[pos.stage], pos.phase ^ 1u, abort, &g_block_timeouts);
      if (!__shfl_sync(0xffffffffu, go, 0)) break;
      if (EDGE) __syncwarp();  // lane 0's wait comes before every lane's stores
      unsigned char* st = ring + (size_t)pos.stage * sp.stride;
      uint64_t* full = &sh.full[pos.stage];
      if constexpr (!EDGE) {  // consecutive rows; K is 1 where cs > 1
        if (lane == 0) {
          const uint32_t tb = (uint32_t)walk.n * tpitch, sb = (uint32_t)walk.n * spitch;
          const int64_t from = walk.row(0) * p.hidden + col0;
          mbar_arrive_expect_tx(full, (has_x ? tb : 0) + (NEXT ? tb + sb : 0) + (DR ? sb : 0));
          if (has_x) bulk_load(st, x + from, tb, full);
          if (NEXT) {
            bulk_load(st + at.r, r + from, sb, full);
            bulk_load(st + at.dy, dy + from, tb, full);
          }
          if (DR) bulk_load(st + at.dr, dr + from, sb, full);
        }
      } else {  // a lane a row
        const int64_t all = p.rows * p.hidden, from = walk.row(lane) * p.hidden + col0;
        const int m = (part.span + A - 1) / A * A;
        unsigned char* stt = st + lane * tpitch;
        unsigned char* sts = st + lane * spitch;
        uint32_t bytes = 0;
        if (lane < walk.n) {
          if (has_x) bytes += copy_tail(stt, x, from, m, all);
          if (NEXT) bytes += copy_tail(sts + at.r, r, from, m, all);
          if (NEXT) bytes += copy_tail(stt + at.dy, dy, from, m, all);
          if (DR) bytes += copy_tail(sts + at.dr, dr, from, m, all);
        }
        bytes = __reduce_add_sync(0xffffffffu, bytes);
        __syncwarp();  // every lane's tails come before lane 0's arrival
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (lane < walk.n) {
          if (has_x) copy_row(stt, x, from, m, all, full);
          if (NEXT) copy_row(sts + at.r, r, from, m, all, full);
          if (NEXT) copy_row(stt + at.dy, dy, from, m, all, full);
          if (DR) copy_row(sts + at.dr, dr, from, m, all, full);
        }
      }
      pos.next(stages);
      ++issued;
    }
    if (lane == 0) drain_ring(sh.full, pos, issued, stages);
    __syncwarp();
  } else if (warp <= reducers) {
    // The reducers' weights: w (without a gate of several rows, which is read
    // from global memory, where L1 holds it) and w2.
    for (int v = threadIdx.x - 32; v < nvec; v += 32 * reducers) {
      f32x2 f[N], g[N];
      if (POST) {
        load_weights<T, N, EDGE>(gamma_post + col0, v * E, part, f);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = mul2(pair(p.b, p.b), add2(f[i], off));
        if (gate != nullptr && !gate_each) {
          load_weights<T, N, EDGE>(gate + col0, v * E, part, g);
#pragma unroll
          for (int i = 0; i < N; ++i) f[i] = mul2(f[i], g[i]);
        }
        store_plane<N>(plane1, nvec, v, f);
      }
      if (NEXT) {
        load_weights<T, N, EDGE>(gamma_next + col0, v * E, part, f);
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
      const int64_t row = walk.row(lane < walk.n ? lane : 0);
      const float rs1_l = POST ? __ldg(p.rstd_post + row) : 1.f;
      const float rs2_l = NEXT ? __ldg(p.rstd_next + row) : 0.f;
      if (!wait_all(&sh.full[pos.stage], pos.phase, abort)) break;
      unsigned char* st = ring + (size_t)pos.stage * sp.stride;
      const T* grow = gate_each ? gate + walk.q * p.hidden + col0 : nullptr;
      bool ok = true;
      for (int q0 = 0; q0 < walk.n; q0 += at_once) {
        // lanes past the stage's rows work on its first one, for the shuffles
        const bool mine = q0 + sub < walk.n;
        const int q = mine ? q0 + sub : 0;
        T* sx = reinterpret_cast<T*>(st) + q * pitch;
        TS* sr = reinterpret_cast<TS*>(st + at.r) + q * pitch;
        T* sdy = reinterpret_cast<T*>(st + at.dy) + q * pitch;
        TS* sdr = reinterpret_cast<TS*>(st + at.dr) + q * pitch;
        if (EDGE) {  // for the appliers too
          if (mine)
            for (int i = lane & (lanes - 1); i < 16; i += lanes) {
              const int c = end_column<A, E>(i, nvec, part);
              if (c < 0 || part.has(c)) continue;
              if (has_x) sx[c] = Traits<T>::from_f(0.f);
              if (NEXT) sr[c] = Traits<TS>::from_f(0.f);
              if (NEXT) sdy[c] = Traits<T>::from_f(0.f);
              if (DR) sdr[c] = Traits<TS>::from_f(0.f);
            }
          __syncwarp();
        }
        const float rs1f = __shfl_sync(0xffffffffu, rs1_l, q);
        const float rs2f = __shfl_sync(0xffffffffu, rs2_l, q);
        const f32x2 rs2 = pair(rs2f, rs2f);
        // S1, and S2 and S3 over rstd_post: a multiplication an element less
        // (16384 x 8192 bf16 305 us, 316 with it).  Rows of very large or small
        // x, whose products could leave fp32's range, take it (`far`); what
        // rows beside them are multiplied by is 1.
        f32x2 s1 = 0, s2 = 0, s3 = 0;
        const bool far = POST && !(rs1f >= 0x1p-16f && rs1f <= 0x1p16f);
        auto add_to = [&](int v, auto scaled) {
          f32x2 x[N], dv[N];
          if (POST) {
            f32x2 w[N];
            load_pairs<T, N>(sx + v * E, x);
            load_plane<N>(plane1, nvec, v, w);
            if (gate_each) {
              f32x2 g[N];
              load_weights<T, N, EDGE>(grow, v * E, part, g);
#pragma unroll
              for (int k = 0; k < N; ++k) w[k] = mul2(w[k], g[k]);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
              if constexpr (decltype(scaled)::value) {
                const float by = far ? rs1f : 1.f;
                x[k] = mul2(x[k], pair(by, by));
              }
              x[k] = mul2(w[k], x[k]);
            }
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
        auto add = [&](int v) { add_to(v, std::false_type{}); };
        float3 s;
        if (__any_sync(0xffffffffu, far)) {
#pragma unroll 1
          for (int v = lane & (lanes - 1); v < nvec; v += lanes) add_to(v, std::true_type{});
          s = make_float3(sum2(s1), sum2(s2), sum2(s3));
#pragma unroll 1
          for (int m = lanes / 2; m >= 1; m /= 2) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, m);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, m);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, m);
          }
        } else if (lanes < 32) {
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
        const float c2 = POST ? fmaf(-rs2f * c1, s.z, s.y) * (far ? inv : rs1f * inv) : 0.f;
        if ((lane & (lanes - 1)) == 0 && mine)
          sh.stat[pos.stage][q] = make_float4(-c1, -c2, rs1f, rs2f);
      }
      if (!ok) break;
      // the rows' ends were written where the next copy will land
      if (EDGE) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
        static_cast<T*>(p.dx) + (cls + i0 * P) * p.hidden + col0);
    unsigned char* dres = reinterpret_cast<unsigned char*>(
        static_cast<TS*>(p.dres) + (cls + i0 * P) * p.hidden + col0);
    const uint32_t hbytes_t = (uint32_t)(P * p.hidden * (int)sizeof(T));  // to the next row
    const uint32_t hbytes_s = (uint32_t)(P * p.hidden * (int)sizeof(TS));
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
      if (NEXT) load_weights<T, N, EDGE>(gamma_next + col0, e0[j], part, w2[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        w2[j][i] = add2(w2[j][i], off);
        acc_n[j][i] = 0;
        acc_a[j][i] = 0;
      }
    }
    bool ok = true;
    bool more = walk.next();
    const int64_t first_q = walk.q;
    // the partial row of A for gate row q: a class's units and gate rows
    // number its segments, as units and gate rows do where there is one class
    const int64_t gates = p.rows / p.rows_per_gate;
    auto a_row = [&](int64_t q) { return cls * (of + gates - 1) + idx + q; };
    while (more) {
      const int64_t q = walk.q;
#pragma unroll
      for (int j = 0; j < NV; ++j) {  // the weights of the segment
        f32x2 f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[j][i] = pair(p.b, p.b);
        if (POST) {
          load_weights<T, N, EDGE>(gamma_post + col0, e0[j], part, f);
#pragma unroll
          for (int i = 0; i < N; ++i) w[j][i] = mul2(w[j][i], add2(f[i], off));
        }
        if (gate != nullptr) {
          load_weights<T, N, EDGE>(gate + q * p.hidden + col0, e0[j], part, f);
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
          const uint32_t row = (uint32_t)(walk.at + k);
          const unsigned char* rt = st + (uint32_t)k * tpitch;
          const unsigned char* rs = st + (uint32_t)k * spitch;
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
            T* dxr = reinterpret_cast<T*>(dx + (uint64_t)row * hbytes_t);
            TS* dresr = reinterpret_cast<TS*>(dres + (uint64_t)row * hbytes_s);
            if (tt + j * threads < nvec) {
              if (!EDGE || part.inner(e0[j], E)) {
                store_pairs<T, N>(dxr + e0[j], x);
                store_pairs<TS, N>(dresr + e0[j], dv);
              } else {
                store_ends<T, N>(dxr, e0[j], part, x);
                store_ends<TS, N>(dresr, e0[j], part, dv);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[pos.stage]);
        pos.next(stages);
      }

      // the segment's sum of A, and after the last one that of dgamma_next: a
      // thread's own columns, or its columns of the teams' sums, added in turn
      const bool first = q == first_q;
      float* pa = p.p_a + a_row(q) * p.hidden + col0;
      float* pp = p.p_post + unit * p.hidden + col0;
      float* pn = p.p_next + unit * p.hidden + col0;
      // With one gate row the sums of A give dgamma_post too (block_bwd_sums).
      auto put4 = [&](float* to, int c, const f32x2& lo, const f32x2& hi) {
        const f32x2 f[2] = {lo, hi};
        if constexpr (EDGE) {  // partial rows start anywhere
          store_ends<float, 2>(to, c, part, f);
        } else {
          store_pairs<float, 2>(to + c, f);
        }
      };
      auto put_a = [&](int c, f32x2 lo, f32x2 hi) {
        const f32x2 b2 = pair(p.b, p.b);
        lo = mul2(lo, b2);
        hi = mul2(hi, b2);
        put4(pa, c, lo, hi);
        if (POST && gate_each) {
          f32x2 f[2], s[2] = {0, 0};
          load_weights<T, 2, EDGE>(gate + q * p.hidden + col0, c, part, f);
          if (!first) load_weights<float, 2, EDGE>(p.p_post + unit * p.hidden + col0, c, part, s);
          put4(pp, c, add2(s[0], mul2(f[0], lo)), add2(s[1], mul2(f[1], hi)));
        }
      };
      auto put_n = [&](int c, const f32x2& lo, const f32x2& hi) { put4(pn, c, lo, hi); };
      const int me = aw * 32 + lane, all = applier_warps * 32;
      auto flush = [&](auto& acc, auto put) {
        f32x2* comb = reinterpret_cast<f32x2*>(ring + (size_t)stages * sp.stride);
        if (sp.teams == 1) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = tt + j * threads;
            if (v >= nvec) continue;
#pragma unroll
            for (int k = 0; k < N; k += 2) put(v * E + 2 * k, acc[j][k], acc[j][k + 1]);
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
        for (int c = 4 * me; c < nvec * E; c += 4 * all) put(c, comb[c / 2], comb[c / 2 + 1]);
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

// The backward's roles and stages, over as few CTAs as leave three stages, or
// four where the row's sums are exchanged (else one less), beside the reducers'
// weights, and three reducers beside the appliers.  (8192 rows, bf16: 6656
// columns with two reducers 149 us, over two CTAs 113; 12288 over two with three
// stages 269, over four with four 218; but 6144 over one with three 108, over two
// 109, and 3584 fp32 96 and 108.)
template <typename F>
bool bwd_pick(int64_t rows, int hidden, int sms, int align, int elems, int planes,
              bool edge, F stage_bytes, BwdShape* s, int* nv8, size_t* smem) {
  const int budget = kSmemBudget - (int)sizeof(BwdShared) - kSlack;
  for (int least = 3; least >= 2; --least)
    for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
      const int cols = row_part(hidden, align, cs, edge);
      if (edge ? (cs - 1) * cols >= hidden : hidden % (align * cs) != 0) break;
      *nv8 = cols < 512 ? 1 : 2;
      s->cs = cs;
      s->wpt = (cols + *nv8 * 256 - 1) / (*nv8 * 256);
      if (s->wpt > kBwdWarps - 4) continue;
      // Teams share a stage, which then is as many rows: up to 48 KB of them
      // (fp32, 32768 x 2048 336 -> 206 us with one team), and only where a CTA
      // has two such stages or more, or its rows would wait for one reducer
      // (256 x 1024 fp32 9.2 -> 7.5 us, 2048 x 512 bf16 12.5 -> 10.7).
      s->teams = cs > 1 || s->wpt > 4 ? 1 : 8 / s->wpt;
      while (s->teams > 1 && (stage_bytes(s->teams, cols) > 48 * 1024 ||
                              rows <= (int64_t)2 * s->teams * sms))
        s->teams /= 2;
      // narrow rows: as many to a stage as make it a wide row's (40 KB: fp32,
      // 65536 x 512 128 -> 108 us against 64 KB), if there are enough of them
      // for every CTA to fill its ring
      s->stage_rows = s->teams;
      while (cs == 1 && 2 * s->stage_rows <= kBwdRows &&
             stage_bytes(2 * s->stage_rows, cols) <= 40 * 1024 &&
             rows >= (int64_t)8 * s->stage_rows * sms)
        s->stage_rows *= 2;
      s->lanes = cs == 1 && cols / elems <= kNarrowGroups && s->stage_rows > 1 ? kNarrowLanes : 32;
      const int over = planes * cols * 4 + (s->teams > 1 ? cols * 4 : 0);
      s->stride = (stage_bytes(s->stage_rows, cols) + 127) / 128 * 128;
      s->stages = (budget - over) / s->stride;
      if (s->stages > kBwdStages) s->stages = kBwdStages;
      if (s->stages < (cs > 1 ? least + 1 : least)) continue;
      s->reducers = kBwdWarps - 1 - s->teams * s->wpt;
      if (s->reducers > s->stages) s->reducers = s->stages;
      s->stages -= s->stages % s->reducers;  // a stage is always the same reducer's
      *smem = (size_t)s->stages * s->stride + over;
      return true;
    }
  return false;
}

template <typename T, typename TS, bool POST, bool NEXT, bool EDGE>
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
  if (!bwd_pick(a.rows, a.hidden, sms, 16 / (int)sizeof(T), E, (POST ? 1 : 0) + (NEXT ? 1 : 0), EDGE,
                [=](int k, int cols) { return bwd_stage<T, TS>(k, cols, x, NEXT, dr).bytes; }, &sp,
                &nv8, &smem))
    return false;
  const int period = EDGE ? row_period(a.hidden, 16 / (int)sizeof(T)) : 1;
  if (EDGE && sms / sp.cs < period) return false;  // an SM budget below a unit for each class
  p.period = period;
  auto go = [&](auto which) {
    constexpr auto kern = decltype(which)::value;
    *err = allow<kern>(dev, kSmemBudget - sizeof(BwdShared));
    if (*err != cudaSuccess) return;
    const int threads = 32 * (1 + sp.reducers + sp.teams * sp.wpt);
    int64_t n = sp.cs == 1 ? sms : max_clusters((const void*)kern, threads, smem, sp.cs, sms);
    if (n < p.period) n = p.period;  // (fewer fit at once: they wait their turn)
    if (n > RMSN_BLOCK_MAX_PARTIALS) n = RMSN_BLOCK_MAX_PARTIALS;
    if (n > a.rows) n = a.rows;
    n -= n % p.period;  // a unit's rows are of one class, at least one each
    *units = (int)n;
    place_partials(a, *units, p);
    *err = launch_kernel(kern, dim3((unsigned)(n * sp.cs)), dim3(threads), smem, s, sp.cs, p, sp);
  };
  if (dr || !NEXT) {
    if (nv8 == 1)
      go(Kern<block_bwd_tma<T, TS, POST, NEXT, true, 8 / E, EDGE>>{});
    else
      go(Kern<block_bwd_tma<T, TS, POST, NEXT, true, 16 / E, EDGE>>{});
  } else {
    if (nv8 == 1)
      go(Kern<block_bwd_tma<T, TS, POST, true, false, 8 / E, EDGE>>{});
    else
      go(Kern<block_bwd_tma<T, TS, POST, true, false, 16 / E, EDGE>>{});
  }
  return true;
}

template <typename T, typename TS, bool EDGE>
bool bwd_parts(const BlockBwdArgs& a, BlockBwdParams& p, int* units, cudaStream_t s,
               cudaError_t* err) {
  if (a.gamma_post == nullptr) return try_bwd<T, TS, false, true, EDGE>(a, p, units, s, err);
  if (a.gamma_next == nullptr) return try_bwd<T, TS, true, false, EDGE>(a, p, units, s, err);
  return try_bwd<T, TS, true, true, EDGE>(a, p, units, s, err);
}

template <bool EDGE>
bool bwd_types(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p, int* units,
               cudaStream_t s, cudaError_t* err) {
  using bf16 = __nv_bfloat16;
  if (dtype == RMSN_F32) return bwd_parts<float, float, EDGE>(a, p, units, s, err);
  if (dtype == RMSN_BF16)
    return res_dtype == RMSN_F32 ? bwd_parts<bf16, float, EDGE>(a, p, units, s, err)
                                 : bwd_parts<bf16, bf16, EDGE>(a, p, units, s, err);
  return res_dtype == RMSN_F32 ? bwd_parts<__half, float, EDGE>(a, p, units, s, err)
                               : bwd_parts<__half, __half, EDGE>(a, p, units, s, err);
}

}  // namespace
}  // namespace rmsn
