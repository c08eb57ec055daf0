// Forward of the staged block norm (block_norm_tma.cuh, formulas in block_norm.cu).
#include "block_norm_tma.cuh"

namespace rmsn {
namespace {

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
  int lanes;   // of a warp on a row: 32, or kNarrowLanes where wpt is 1
  int period;  // of the rows' alignment (EDGE), else 1
};

struct FwdShared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t red[kMaxWarps][2];                     // a team's, across a cluster
  float slot[2][kMaxWarps * kMaxSplit];
  int abort;
};

template <typename T, typename TS, bool POST, bool NEXT, bool EDGE>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1), 1) block_fwd_tma(const BlockFwdParams p) {
  constexpr int E = kElems<T, TS>, N = E / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ FwdShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages, cs = p.cs, K = p.stage_rows;
  constexpr int A = 16 / sizeof(T);
  const uint32_t rank = cs > 1 ? cta_rank() : 0u;
  const int64_t unit = blockIdx.x / cs, units = gridDim.x / cs;
  const int P = EDGE ? p.period : 1;
  const int cls = EDGE ? (int)(unit % P) : 0;
  const Part part(p.hidden, A, cs, rank, cls, EDGE);
  const int pitch = part.pitch, col0 = part.col0;
  const int nvec = EDGE ? (part.span + E - 1) / E : pitch / E;
  // Block b of K rows: rows first, first + P, ..., all of one class (unit count
  // and P agree: a unit's blocks k units + unit are of its class)
  const int64_t blocks = (int64_t)P * ((p.rows + (int64_t)P * K - 1) / ((int64_t)P * K));
  const int nst = blocks > unit ? (int)((blocks - unit + units - 1) / units) : 0;
  auto first_row = [&](int k) {
    const int64_t b = k * units + unit;
    return EDGE ? cls + (int64_t)P * K * (b / P) : b * K;
  };
  auto rows_from = [&](int64_t first) {
    const int64_t left = EDGE ? (p.rows - first + P - 1) / P : p.rows - first;
    return left < 0 ? 0 : left < K ? (int)left : K;
  };
  if (!EDGE && threadIdx.x == 0)  // the first rows into L2 (prefetch_l2)
    for (int k = 0; k < kFirstStages && k < nst; ++k) {
      const int64_t first = first_row(k), at = first * p.hidden + col0;
      const uint32_t n = (uint32_t)(rows_from(first) * pitch);
      prefetch_l2(static_cast<const T*>(p.x) + at, n * (uint32_t)sizeof(T));
      prefetch_l2(static_cast<const TS*>(p.res) + at, n * (uint32_t)sizeof(TS));
    }
  float4* plane1 = reinterpret_cast<float4*>(smem);
  float4* plane2 = plane1 + pitch / 4;
  unsigned char* ring = reinterpret_cast<unsigned char*>(NEXT ? plane2 + pitch / 4 : plane2);
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
  const uint32_t xbytes = (uint32_t)(pitch * sizeof(T)), sbytes = (uint32_t)(pitch * sizeof(TS));
  const int res_at = K * (int)xbytes;
  const T* x = static_cast<const T*>(p.x);
  const TS* res = static_cast<const TS*>(p.res);
  auto issue = [&](int k, int stage) {
    const int64_t first = first_row(k);
    const int n = rows_from(first);
    unsigned char* st = ring + (size_t)stage * p.stride;
    uint64_t* full = &sh.full[stage];
    if constexpr (!EDGE) {  // consecutive rows; K is 1 where cs > 1
      if (lane != 0) return;
      const int64_t at = first * p.hidden + col0;
      mbar_arrive_expect_tx(full, (uint32_t)n * (xbytes + sbytes));
      bulk_load(st, x + at, (uint32_t)n * xbytes, full);
      bulk_load(st + res_at, res + at, (uint32_t)n * sbytes, full);
    } else {  // a lane a row
      const int64_t all = p.rows * p.hidden, at = (first + (int64_t)lane * P) * p.hidden + col0;
      const int m = (part.span + A - 1) / A * A;
      unsigned char* sx = st + lane * xbytes;
      unsigned char* sr = st + res_at + lane * sbytes;
      uint32_t bytes = 0;
      if (lane < n) bytes = copy_tail(sx, x, at, m, all) + copy_tail(sr, res, at, m, all);
      bytes = __reduce_add_sync(0xffffffffu, bytes);
      __syncwarp();  // every lane's tails come before lane 0's arrival
      if (lane == 0) mbar_arrive_expect_tx(full, bytes);
      __syncwarp();
      if (lane < n) {
        copy_row(sx, x, at, m, all, full);
        copy_row(sr, res, at, m, all, full);
      }
    }
  };
  if (warp == 0)
    for (int k = 0; k < stages && k < nst; ++k) issue(k, k);
  const T* gate = static_cast<const T*>(p.gate);
  const bool gate_each = !EDGE && gate != nullptr && p.rows_per_gate < p.rows;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    f32x2 w[N], f[N];
    const f32x2 off = pair(p.off, p.off), b = pair(p.b, p.b);
    const int c = v * E;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = b;
    if (POST) {
      load_weights<T, N, EDGE>(static_cast<const T*>(p.gamma_post) + col0, c, part, f);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = mul2(w[i], add2(f[i], off));
    }
    if (gate != nullptr && !gate_each) {
      load_weights<T, N, EDGE>(gate + col0, c, part, f);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = mul2(w[i], f[i]);
    }
    store_plane<N>(plane1, nvec, v, w);
    if (NEXT) {
      load_weights<T, N, EDGE>(static_cast<const T*>(p.gamma_next) + col0, c, part, f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = add2(f[i], off);
      store_plane<N>(plane2, nvec, v, f);
    }
  }
  __syncthreads();

  if (warp == 0) {
    int stage = 0, k = stages;
    uint32_t phase = 0;
    for (; k < nst; ++k) {
      bool go = true;
      if (lane == 0) go = wait_phase_counted(&sh.empty[stage], phase, abort, &g_block_timeouts);
      if (!__shfl_sync(0xffffffffu, go, 0)) break;
      if (EDGE) __syncwarp();  // lane 0's wait comes before every lane's stores
      issue(k, stage);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // every copy has landed before the CTA may exit
    const int issued = k < nst ? k : nst;
    if (lane == 0)
      drain_ring(sh.full, Ring{issued % stages, (uint32_t)(issued / stages) & 1u}, issued, stages);
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
      const int64_t row0 = first_row(k);
      const int n = rows_from(row0);
      unsigned char* st = ring + (size_t)stage * p.stride;
      for (int q0 = 0; q0 < n; q0 += at_once) {
        // every lane takes part in the shuffles; those past the last row work
        // on the stage's first row and write nothing
        const int qt = q0 + sub;
        const bool mine = qt < n && ok;
        const int q = qt < n ? qt : 0;
        const int64_t row = row0 + (int64_t)q * P;
        T* sx = reinterpret_cast<T*>(st) + q * pitch;
        TS* sr = reinterpret_cast<TS*>(st + res_at) + q * pitch;
        // f(c) for the columns of a row's ends, a lane each (end_column); the
        // warp that reads and writes their groups takes them
        auto ends = [&](auto f) {
          if (!EDGE) return;
          __syncwarp();
          if (mine)
            for (int i = lane & (lanes - 1); i < 16; i += lanes) {
              const int c = end_column<A, E>(i, nvec, part);
              if (c >= 0 && (lanes < 32 || c / E % step / 32 == tw)) f(c);
            }
          __syncwarp();
        };
        ends([&](int c) {
          if (part.has(c)) return;
          sx[c] = Traits<T>::from_f(0.f);
          sr[c] = Traits<TS>::from_f(0.f);
        });
        float rs1 = 1.f;
        if (POST) {
          f32x2 sums[N];
#pragma unroll
          for (int i = 0; i < N; ++i) sums[i] = 0;
          each([&](int v) {
            f32x2 x[N];
            load_pairs<T, N>(sx + v * E, x);
#pragma unroll
            for (int i = 0; i < N; ++i) sums[i] = fma2(x[i], x[i], sums[i]);
          });
          const float ss = over_team(sum_pairs<N>(sums));
          // The approximate root (2 ulp) of a mean by 1 / H, well inside the
          // error of the sum; the loops and rms_norm_fwd divide and round the
          // root correctly, which here every row waits for twice: 4096 x 4096
          // bf16 28.3 us, 28.8 with it.
          rs1 = rsqrtf(fmaf(ss, inv, p.eps));
          if (__any_sync(0xffffffffu, isinf(ss))) {  // squares overflowed (kOverflowScale)
            float again = 0.f;
            for (int j = tt; j < part.span; j += step) {
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
        f32x2 sums[N];
#pragma unroll
        for (int i = 0; i < N; ++i) sums[i] = 0;
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
            if (NEXT) sums[i] = fma2(r[i], r[i], sums[i]);
          }
          if (mine && (!EDGE || part.inner(v * E, E))) store_pairs<TS, N>(out + v * E, r);
          if ((NEXT || EDGE) && mine) {
            if constexpr (N == 4) {
              *reinterpret_cast<ulonglong2*>(sx + v * E) = make_ulonglong2(r[0], r[1]);
              *reinterpret_cast<ulonglong2*>(sr + v * E) = make_ulonglong2(r[2], r[3]);
            } else {
              *reinterpret_cast<ulonglong2*>(sr + v * E) = make_ulonglong2(r[0], r[1]);
            }
          }
        });
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
        auto kept_at = [&](int c) {
          const int at = c % E;
          if constexpr (N == 4)
            return reinterpret_cast<const float*>(at < 4 ? (const void*)(sx + c - at)
                                                         : (const void*)(sr + c - at))[at & 3];
          else
            return reinterpret_cast<const float*>(sr + c - at)[at];
        };
        ends([&](int c) {
          if (part.has(c)) out[c] = Traits<TS>::from_f(kept_at(c));
        });
        if (!NEXT) continue;
        const float ss = over_team(sum_pairs<N>(sums));
        float rs2 = rsqrtf(fmaf(ss, inv, p.eps));
        if (__any_sync(0xffffffffu, isinf(ss))) {
          const f32x2 scale = pair(kOverflowScale, kOverflowScale);
#pragma unroll
          for (int i = 0; i < N; ++i) sums[i] = 0;
          for (int v = tt; v < nvec; v += step) {
            f32x2 r[N];
            kept(v, r);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              r[i] = mul2(r[i], scale);
              sums[i] = fma2(r[i], r[i], sums[i]);
            }
          }
          const float again = over_team(sum_pairs<N>(sums));
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
          if (mine && (!EDGE || part.inner(v * E, E))) store_pairs<T, N>(yr + v * E, r);
        });
        ends([&](int c) {
          if (part.has(c)) {
            const float w = reinterpret_cast<const float*>(
                plane2)[(c % E / 4 * nvec + c / E) * 4 + c % 4];
            yr[c] = Traits<T>::from_f(kept_at(c) * rs2 * w);
          }
        });
      }
      // r was written where the next copy will land
      if (NEXT || EDGE) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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

// The forward's teams and stages for `rows` rows on `sms` SMs.  The row is
// split over as few CTAs as leave two stages beside the weights.  (The times
// that compare shapes were taken without kFirstStages, which takes about 1 us
// off each.)
struct FwdShape {
  int teams, wpt, cs, stages, stage_rows, stride, lanes, ctas;  // ctas: on an SM
  size_t smem;
};

bool fwd_shape(int64_t rows, int hidden, int sms, int row_elem, int planes, bool post, int align,
               int elems, bool edge, FwdShape* s) {
  for (int cs = 1; cs <= kMaxSplit; cs *= 2) {
    const int cols = row_part(hidden, align, cs, edge), row = cols * row_elem;
    if (edge ? (cs - 1) * cols >= hidden : hidden % (align * cs) != 0) return false;
    const int over = planes * cols * 4;
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
      // Rows of 12 KB and more (x and res): ten at once, not what the ring
      // holds: 32768 x 4096 bf16 179 -> 168 us, 32768 x 3584 162 -> 146, 32768
      // x 2048 bf16 under fp32 138 -> 132, 4096 x 4096 the same; narrower ones
      // lose by it (65536 x 2048 168 -> 188), and odd ones (32768 x 4097 230 ->
      // 236).
      if (!edge && row >= 12 * 1024) s->teams = 10;
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

template <typename T, typename TS, bool POST, bool NEXT, bool EDGE>
bool try_fwd(const BlockFwdArgs& a, cudaStream_t s, cudaError_t* err) {
  constexpr int E = kElems<T, TS>;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return true;
  const int sms = sm_count(dev);
  FwdShape sh;
  if (!fwd_shape(a.rows, a.hidden, sms, (int)(sizeof(T) + sizeof(TS)), NEXT ? 2 : 1,
                 POST, 16 / (int)sizeof(T), E, EDGE, &sh))
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
  p.period = EDGE ? row_period(a.hidden, 16 / (int)sizeof(T)) : 1;
  constexpr auto kern = block_fwd_tma<T, TS, POST, NEXT, EDGE>;
  *err = allow<kern>(dev, kSmemBudget - sizeof(FwdShared));
  if (*err != cudaSuccess) return true;
  const int threads = 32 * (1 + sh.teams * sh.wpt);
  int64_t units = sh.cs == 1 ? (int64_t)sms * sh.ctas
                             : max_clusters((const void*)kern, threads, sh.smem, sh.cs, sms);
  const int64_t span = (int64_t)p.period * sh.stage_rows;
  const int64_t blocks = p.period * ((a.rows + span - 1) / span);
  if (units < p.period) return false;  // an SM budget below the period
  units -= units % p.period;           // a unit's blocks are of one class
  if (units > blocks) units = blocks;
  *err = launch_kernel(kern, dim3((unsigned)(units * sh.cs)), dim3(threads), sh.smem, s,
                       sh.cs, p);
  return true;
}

template <typename T, typename TS, bool EDGE>
bool fwd_parts(const BlockFwdArgs& a, cudaStream_t s, cudaError_t* err) {
  if (a.gamma_post == nullptr) return try_fwd<T, TS, false, true, EDGE>(a, s, err);
  if (a.gamma_next == nullptr) return try_fwd<T, TS, true, false, EDGE>(a, s, err);
  return try_fwd<T, TS, true, true, EDGE>(a, s, err);
}

template <typename T, typename TS>
bool fwd_of(const BlockFwdArgs& a, cudaStream_t s, cudaError_t* err) {
  if (a.vec_ok && fwd_parts<T, TS, false>(a, s, err)) return true;
  return a.edge_ok && block_fwd_odd_pays(a.rows, a.rows_per_gate, a.hidden) &&
         fwd_parts<T, TS, true>(a, s, err);
}

}  // namespace

bool try_launch_block_fwd_tma(int dtype, int res_dtype, const BlockFwdArgs& a, cudaStream_t s,
                              cudaError_t* err) {
  if (dtype == RMSN_F32) return fwd_of<float, float>(a, s, err);
  if (dtype == RMSN_BF16)
    return res_dtype == RMSN_F32 ? fwd_of<__nv_bfloat16, float>(a, s, err)
                                 : fwd_of<__nv_bfloat16, __nv_bfloat16>(a, s, err);
  return res_dtype == RMSN_F32 ? fwd_of<__half, float>(a, s, err)
                               : fwd_of<__half, __half>(a, s, err);
}

cudaError_t read_block_fwd_wait_timeouts(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_block_timeouts, sizeof(unsigned int));
}

}  // namespace rmsn
