// Head norm and rotation of rows of 16-byte vectors: a group of G lanes has a
// head's row, two vectors a lane, 32 / G heads a warp at a time.
#include <type_traits>

#include "pairs.cuh"
#include "rotary.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Where a pair's columns are.
enum Mode {
  kHalves = 0,      // (i, i + half) of whole vectors: a lane's first vector is paired with its second
  kNeighbours = 1,  // (2 i, 2 i + 1): inside a vector
  kApart = 2        // (i, i + half), half not of whole vectors: through shared memory
};

// PART, of a row of which some columns do not rotate: those lie beside other columns
// all the same, and take nothing from them, not 0 times a value that may not be finite.
// Kernels of their own, as the selects cost a row that rotates as a whole 2 to 4 %
// (32768 x (64+8) x 128 bf16 forward 205 and 210 us, with neighbours paired 203 and 211).

// The columns of a lane's two vectors; dim where it has none.
template <int V, int MODE>
struct Lane {
  int a, b;
  __device__ __forceinline__ Lane(const RotaryParams& p, int l) {
    const int n = p.dim / V;
    int va, vb;
    if constexpr (MODE == kHalves) {
      const int paired = p.half / V;
      va = l < paired ? l : 2 * l;            // 2 paired + 2 (l - paired)
      vb = l < paired ? l + paired : 2 * l + 1;
    } else {
      const int per = (n + 1) / 2;
      va = l < per ? l : n;
      vb = l < per ? l + per : n;
    }
    a = va < n ? va * V : p.dim;
    b = vb < n ? vb * V : p.dim;
  }
};

// Lanes that a row takes.
int lanes_of(const RotaryParams& p, int v, int mode) {
  const int n = p.dim / v;
  if (mode != kHalves) return (n + 1) / 2;
  const int paired = p.half / v;
  return paired + (n - 2 * paired + 1) / 2;
}

// Every pair's (cos, sin) of a token's angles, in the warp's shared memory.
__device__ __forceinline__ void find_angles(const RotaryParams& p, const uint64_t* turns,
                                            float2* cs, int64_t position, int lane) {
  __syncwarp();
  for (int i = lane; i < p.half; i += 32) cs[i] = turn_of(turns[i], position);
  __syncwarp();
}

// A token's angles of this lane's columns.
template <int V, int MODE>
struct Angles {
  float c[V], s[V];  // kHalves: of the pairs a ..; kNeighbours: a / 2 .., b / 2 ..
  __device__ __forceinline__ void take(const RotaryParams& p, const uint64_t* turns, float2* cs,
                                       int64_t position, const Lane<V, MODE>& at, int lane) {
    find_angles(p, turns, cs, position, lane);
    if constexpr (MODE != kApart) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        int i;
        if constexpr (MODE == kHalves) i = at.a + k;
        else i = k < V / 2 ? at.a / 2 + k : at.b / 2 + k - V / 2;
        const float2 v = i < p.half ? cs[i] : make_float2(1.f, 0.f);
        c[k] = v.x;
        s[k] = v.y;
      }
    }
  }
  // The lane's columns turned, by SIGN times the angle.
  template <int SIGN, bool PART>
  __device__ __forceinline__ void turn(const RotaryParams& p, const float2* cs, float* row,
                                       const Lane<V, MODE>& at, float (&x)[V], float (&y)[V]) const {
    if constexpr (MODE == kHalves) {
      if (PART && at.a >= p.half) return;  // all of a lane's columns rotate, or none
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float u = x[k], w = y[k], t = SIGN * s[k];
        x[k] = u * c[k] - w * t;
        y[k] = w * c[k] + u * t;
      }
    } else if constexpr (MODE == kNeighbours) {
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float u = x[k], w = x[k + 1], t = SIGN * s[k / 2];
        if (!PART || at.a + k < 2 * p.half) {
          x[k] = u * c[k / 2] - w * t;
          x[k + 1] = w * c[k / 2] + u * t;
        }
        const float d = y[k], e = y[k + 1], r = SIGN * s[(V + k) / 2];
        if (!PART || at.b + k < 2 * p.half) {
          y[k] = d * c[(V + k) / 2] - e * r;
          y[k + 1] = e * c[(V + k) / 2] + d * r;
        }
      }
    } else {
      __syncwarp();
      if (at.a < p.dim) put(row + at.a, x);
      if (at.b < p.dim) put(row + at.b, y);
      __syncwarp();
      if (p.half % 4 == 0) {
        turn_runs<SIGN, 4>(p, cs, row, at.a, x);
        turn_runs<SIGN, 4>(p, cs, row, at.b, y);
      } else if (p.half % 2 == 0) {
        turn_runs<SIGN, 2>(p, cs, row, at.a, x);
        turn_runs<SIGN, 2>(p, cs, row, at.b, y);
      } else {
        turn_runs<SIGN, 1>(p, cs, row, at.a, x);
        turn_runs<SIGN, 1>(p, cs, row, at.b, y);
      }
    }
  }
  static __device__ __forceinline__ void put(float* to, const float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < V; k += 4)
      *reinterpret_cast<float4*>(to + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  }
  // Columns j .. of values v, by runs of R that lie in one half or behind both
  // (29315 x (64+16) x 96 bf16 of which 24 rotate: single columns 487 us, runs of
  // four 235).
  template <int SIGN, int R>
  static __device__ __forceinline__ void turn_runs(const RotaryParams& p, const float2* cs,
                                                   const float* row, int j, float (&v)[V]) {
    struct alignas(4 * R) Values { float f[R]; };
    struct alignas(R == 1 ? 8 : 16) Turns { float2 t[R]; };
#pragma unroll
    for (int k = 0; k < V; k += R) {
      const int at = j + k;
      if (at >= 2 * p.half) break;
      const bool first = at < p.half;
      const int i = first ? at : at - p.half;
      const Values other = *reinterpret_cast<const Values*>(row + (first ? at + p.half : i));
      const Turns turns = *reinterpret_cast<const Turns*>(cs + i);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float t = first ? -SIGN * turns.t[r].y : SIGN * turns.t[r].y;
        v[k + r] = v[k + r] * turns.t[r].x + other.f[r] * t;
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ uint4 load_at(const T* row, int c, int dim, bool in) {
  return in && c < dim ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
}

// A vector's values by pairs.
template <typename T, int E>
__device__ __forceinline__ void unpack2(const uint4& v, f32x2 (&f)[E]) {
  if constexpr (E == 2) {
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
  } else {
    f[0] = widen<T>(v.x);
    f[1] = widen<T>(v.y);
    f[2] = widen<T>(v.z);
    f[3] = widen<T>(v.w);
  }
}

__device__ __forceinline__ f32x2 swapped(f32x2 v) {
  const float2 f = split(v);
  return pair(f.y, f.x);
}

// The forward's factors of a lane's columns x (of its first vector) and y, with
// x', y' the pairs' other columns: gain and angle in one,
//   kHalves:     x <- x a - y b,   y <- y c + x d
//   kNeighbours: x <- x a + x' b,  y <- y c + y' d
//   kApart:      x <- x a,  y <- y c, and then the angle
template <int V, int MODE>
struct Factors {
  static constexpr int E = V / 2;
  f32x2 a[E], b[E], c[E], d[E];
  template <typename T>
  __device__ __forceinline__ void take(const RotaryParams& p, const RotarySide& s, const float2* cs,
                                       const Lane<V, MODE>& at) {
    const T* gamma = static_cast<const T*>(s.gamma);
    unpack2<T>(load_at(gamma, at.a, p.dim, true), a);
    unpack2<T>(load_at(gamma, at.b, p.dim, true), c);
    const f32x2 off = pair(p.off, p.off);
    const float2 none = make_float2(1.f, 0.f);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const f32x2 ga = add2(a[k], off), gb = add2(c[k], off);
      if constexpr (MODE == kApart) {
        a[k] = ga;
        c[k] = gb;
      } else if constexpr (MODE == kHalves) {
        const int i = at.a + 2 * k;
        const bool in = i < p.half;
        const float2 u = in ? cs[i] : none, v = in ? cs[i + 1] : none;
        const f32x2 cos = pair(u.x, v.x), sin = pair(u.y, v.y);
        a[k] = mul2(ga, cos);
        b[k] = mul2(gb, pair(-u.y, -v.y));
        c[k] = mul2(gb, cos);
        d[k] = mul2(ga, sin);
      } else {
        const int i = at.a / 2 + k, j = at.b / 2 + k;
        const float2 u = i < p.half ? cs[i] : none, v = j < p.half ? cs[j] : none;
        a[k] = mul2(ga, pair(u.x, u.x));
        b[k] = mul2(swapped(ga), pair(-u.y, u.y));
        c[k] = mul2(gb, pair(v.x, v.x));
        d[k] = mul2(swapped(gb), pair(-v.y, v.y));
      }
    }
  }
  template <bool PART>
  __device__ __forceinline__ void apply(const RotaryParams& p, const Lane<V, MODE>& at,
                                        f32x2 (&x)[E], f32x2 (&y)[E]) const {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const f32x2 u = mul2(x[k], a[k]), v = mul2(y[k], c[k]);
      if constexpr (MODE == kHalves) {
        const bool in = !PART || at.a < p.half;
        const f32x2 w = in ? fma2(y[k], b[k], u) : u;
        y[k] = in ? fma2(x[k], d[k], v) : v;
        x[k] = w;
      } else if constexpr (MODE == kNeighbours) {
        x[k] = !PART || at.a + 2 * k < 2 * p.half ? fma2(swapped(x[k]), b[k], u) : u;
        y[k] = !PART || at.b + 2 * k < 2 * p.half ? fma2(swapped(y[k]), d[k], v) : v;
      } else {
        x[k] = u;
        y[k] = v;
      }
    }
  }
};

// A row's columns turned through shared memory (MODE kApart).
template <int E, int MODE>
__device__ __forceinline__ void turn_apart(const RotaryParams& p, const float2* cs, float* row,
                                           const Lane<2 * E, MODE>& at, f32x2 (&x)[E],
                                           f32x2 (&y)[E]) {
  float u[2 * E], v[2 * E];
#pragma unroll
  for (int k = 0; k < E; ++k) {
    const float2 a = split(x[k]), b = split(y[k]);
    u[2 * k] = a.x, u[2 * k + 1] = a.y, v[2 * k] = b.x, v[2 * k + 1] = b.y;
  }
  Angles<2 * E, MODE>().template turn<1, false>(p, cs, row, at, u, v);
#pragma unroll
  for (int k = 0; k < E; ++k) {
    x[k] = pair(u[2 * k], u[2 * k + 1]);
    y[k] = pair(v[2 * k], v[2 * k + 1]);
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = G / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

template <typename T, int V>
__device__ __forceinline__ void gains(const RotarySide& s, int c, int dim, float off,
                                      float (&g)[V]) {
  unpack<T>(load_at(static_cast<const T*>(s.gamma), c, dim, true), g);
#pragma unroll
  for (int k = 0; k < V; ++k) g[k] += off;
}

// Shared memory of a CTA.
template <int V, int G, int MODE>
struct Shared {
  uint64_t turns[G * V];
  alignas(16) float2 cs[kWarps][G * V];
  alignas(16) float row[MODE == kApart ? kWarps : 1][MODE == kApart ? 32 / G : 1][MODE == kApart ? 2 * G * V : 1];
};

// A warp takes a token's heads [h0, h0 + per_unit) of one side, `kSteps` times
// 32 / G of them at a time: their loads are under way together, and while the
// token's angles are found.
constexpr int kSteps = 4;

template <typename T, int G, int MODE, bool PART>
__global__ void __launch_bounds__(kThreads, 2)
    rotary_fwd_vec(const __grid_constant__ RotaryParams p, int per_unit) {
  constexpr int V = Traits<T>::kVec, HPS = 32 / G;
  __shared__ Shared<V, G, MODE> sh;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < p.half; i += kThreads) sh.turns[i] = fixed_turns(p, i);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / G;
  const Lane<V, MODE> at(p, lane % G);
  float* row = sh.row[MODE == kApart ? warp : 0][MODE == kApart ? group : 0];
  const int uq = (p.side[0].heads + per_unit - 1) / per_unit;
  const int uk = (p.side[1].heads + per_unit - 1) / per_unit;
  // The units of queries come first: with a token's units side by side a warp's
  // stride can give it queries' alone, or keys' (32768 x (64+8) x 128 bf16 270
  // us, 213 so).
  const uint32_t first_k = (uint32_t)p.all * uq;
  const float inv_n = 1.f / (float)p.dim;
  // units are fewer than rows, and those fewer than 2^31
  for (uint32_t u = blockIdx.x * kWarps + warp; u < first_k + (uint32_t)p.all * uk;
       u += gridDim.x * kWarps) {
    const bool keys = u >= first_k;
    const uint32_t v = keys ? u - first_k : u, n = keys ? uk : uq;
    const int token = v / n, b = token / p.tokens, t = token - b * p.tokens;
    const RotarySide& s = p.side[keys];
    const int first = (v - token * n) * per_unit;
    const int end = first + per_unit < s.heads ? first + per_unit : s.heads;
    const T* in = reinterpret_cast<const T*>(s.in.p) + row_at(s.in, b, t, 0);
    T* out = reinterpret_cast<T*>(s.out.p) + row_at(s.out, b, t, 0);
    float* rstd = s.rstd ? s.rstd + (int64_t)token * s.heads : nullptr;
    Factors<V, MODE> factors;
    for (int h0 = first; h0 < end; h0 += kSteps * HPS) {
      uint4 va[kSteps], vb[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int h = h0 + i * HPS + group;
        va[i] = load_at(in + h * s.in.sh, at.a, p.dim, h < end);
        vb[i] = load_at(in + h * s.in.sh, at.b, p.dim, h < end);
      }
      if (h0 == first) {
        find_angles(p, sh.turns, sh.cs[warp], position_of(p, b, t), lane);
        factors.template take<T>(p, s, sh.cs[warp], at);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (h0 + i * HPS >= end) break;
        const int h = h0 + i * HPS + group;
        f32x2 x[V / 2], y[V / 2];
        unpack2<T>(va[i], x);
        unpack2<T>(vb[i], y);
        f32x2 squares = mul2(x[0], x[0]);
#pragma unroll
        for (int k = 1; k < V / 2; ++k) squares = fma2(x[k], x[k], squares);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) squares = fma2(y[k], y[k], squares);
        const float ss = group_sum<G>(sum2(squares));
        float rs = __frsqrt_rn(fmaf(ss, inv_n, p.eps));
        if (__any_sync(0xffffffffu, isinf(ss))) {  // the squares are beyond fp32
          const f32x2 down = pair(kOverflowScale, kOverflowScale);
          squares = 0;
#pragma unroll
          for (int k = 0; k < V / 2; ++k) {
            const f32x2 c = mul2(x[k], down), d = mul2(y[k], down);
            squares = fma2(c, c, fma2(d, d, squares));
          }
          const float s2 = group_sum<G>(sum2(squares));
          if (isinf(ss)) rs = rstd_rescaled(s2, p.dim, p.eps);
        }
        if (rstd && lane % G == 0 && h < end) rstd[h] = rs;
        const f32x2 r = pair(rs, rs);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          x[k] = mul2(x[k], r);
          y[k] = mul2(y[k], r);
        }
        factors.template apply<PART>(p, at, x, y);
        if constexpr (MODE == kApart) turn_apart(p, sh.cs[warp], row, at, x, y);
        if (h < end && at.a < p.dim) store_pairs(out + h * s.out.sh + at.a, x);
        if (h < end && at.b < p.dim) store_pairs(out + h * s.out.sh + at.b, y);
      }
    }
  }
}

// The backward: a CTA has one side, so that its sums of du vh stay in registers.
constexpr int kBwdSteps = 2;

template <typename T, int G, int MODE, bool PART>
__global__ void __launch_bounds__(kThreads, 2)
    rotary_bwd_vec(const __grid_constant__ RotaryParams p, int per_unit) {
  constexpr int V = Traits<T>::kVec, HPS = 32 / G;
  __shared__ Shared<V, G, MODE> sh;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < p.half; i += kThreads) sh.turns[i] = fixed_turns(p, i);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / G;
  const Lane<V, MODE> at(p, lane % G);
  float* row = sh.row[MODE == kApart ? warp : 0][MODE == kApart ? group : 0];
  const bool keys = (int)blockIdx.x >= p.side[0].ctas;
  const RotarySide& s = p.side[keys];
  const int cta = blockIdx.x - (keys ? p.side[0].ctas : 0);
  const int ut = (s.heads + per_unit - 1) / per_unit;
  const float inv_n = 1.f / (float)p.dim;
  float ga[V], gb[V], da[V] = {}, db[V] = {};
  gains<T>(s, at.a, p.dim, p.off, ga);
  gains<T>(s, at.b, p.dim, p.off, gb);
  for (uint32_t u = cta * kWarps + warp; u < (uint32_t)p.all * ut; u += s.ctas * kWarps) {
    const int token = u / (uint32_t)ut, b = token / p.tokens, t = token - b * p.tokens;
    const int first = (u - (uint32_t)token * ut) * per_unit;
    const int end = first + per_unit < s.heads ? first + per_unit : s.heads;
    const T* in = reinterpret_cast<const T*>(s.in.p) + row_at(s.in, b, t, 0);
    const T* dy = reinterpret_cast<const T*>(s.dy.p) + row_at(s.dy, b, t, 0);
    T* out = reinterpret_cast<T*>(s.out.p) + row_at(s.out, b, t, 0);
    const float* rstd = s.rstd + (int64_t)token * s.heads;
    Angles<V, MODE> angles;
    for (int h0 = first; h0 < end; h0 += kBwdSteps * HPS) {
      uint4 va[kBwdSteps], vb[kBwdSteps], wa[kBwdSteps], wb[kBwdSteps];
      float rs[kBwdSteps];
#pragma unroll
      for (int i = 0; i < kBwdSteps; ++i) {
        const int h = h0 + i * HPS + group;
        va[i] = load_at(in + h * s.in.sh, at.a, p.dim, h < end);
        vb[i] = load_at(in + h * s.in.sh, at.b, p.dim, h < end);
        wa[i] = load_at(dy + h * s.dy.sh, at.a, p.dim, h < end);
        wb[i] = load_at(dy + h * s.dy.sh, at.b, p.dim, h < end);
        rs[i] = h < end ? rstd[h] : 0.f;
      }
      if (h0 == first) angles.take(p, sh.turns, sh.cs[warp], position_of(p, b, t), at, lane);
#pragma unroll
      for (int i = 0; i < kBwdSteps; ++i) {
        if (h0 + i * HPS >= end) break;
        const int h = h0 + i * HPS + group;
        float x[V], y[V], dx[V], dz[V];
        unpack<T>(wa[i], dx);
        unpack<T>(wb[i], dz);
        angles.template turn<-1, PART>(p, sh.cs[warp], row, at, dx, dz);
        unpack<T>(va[i], x);
        unpack<T>(vb[i], y);
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x[k] *= rs[i];
          y[k] *= rs[i];
          da[k] = fmaf(dx[k], x[k], da[k]);
          db[k] = fmaf(dz[k], y[k], db[k]);
          dx[k] *= ga[k];
          dz[k] *= gb[k];
          dot = fmaf(dx[k], x[k], fmaf(dz[k], y[k], dot));
        }
        const float mean = group_sum<G>(dot) * inv_n;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          dx[k] = rs[i] * (dx[k] - x[k] * mean);
          dz[k] = rs[i] * (dz[k] - y[k] * mean);
        }
        if (h < end && at.a < p.dim) st_vec(out + h * s.out.sh + at.a, pack<T>(dx));
        if (h < end && at.b < p.dim) st_vec(out + h * s.out.sh + at.b, pack<T>(dz));
      }
    }
  }
  // the groups of a warp, then the warps of the CTA
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int m = G; m < 32; m <<= 1) {
      da[k] += __shfl_xor_sync(0xffffffffu, da[k], m);
      db[k] += __shfl_xor_sync(0xffffffffu, db[k], m);
    }
  __syncthreads();  // the angles give way to the sums
  auto sums = reinterpret_cast<float(*)[2 * G * V]>(sh.cs);
  static_assert(sizeof(sh.cs) == kWarps * 2 * G * V * sizeof(float), "a warp's sums");
  if (group == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (at.a < p.dim) sums[warp][at.a + k] = da[k];
      if (at.b < p.dim) sums[warp][at.b + k] = db[k];
    }
  }
  __syncthreads();
  static_assert(sizeof(sh.turns) == 2 * G * V * sizeof(float), "a CTA's sums");
  float* to = p.direct ? reinterpret_cast<float*>(sh.turns) : s.partial + (int64_t)cta * p.dim;
  for (int j = threadIdx.x; j < p.dim; j += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w][j];
    to[j] = v;
  }
  if (p.direct) add_cluster(to, s.dgamma, p.dim, s.ctas);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename T>
int mode_of(const RotaryParams& p) {
  if (p.interleaved || p.half == 0) return kNeighbours;
  return p.half % Traits<T>::kVec == 0 ? kHalves : kApart;
}

// Heads of a unit: all of a side's `heads`, unless that leaves warps without one.
int heads_per_unit(int64_t tokens, int heads, int hps, int steps, int64_t warps) {
  int n = (heads + hps - 1) / hps;               // steps
  while (n > 1 && tokens * ((heads + n * hps - 1) / (n * hps)) < 2 * warps) n = (n + 1) / 2;
  if (n > steps) n = (n + steps - 1) / steps * steps;
  return n * hps;
}

template <typename T, int G, int MODE, bool PART>
cudaError_t launch_fwd_g(const RotaryParams& p, cudaStream_t s) {
  auto kern = rotary_fwd_vec<T, G, MODE, PART>;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sm_count(dev) * max_blocks_per_sm((const void*)kern, kThreads, 0);
  const int per = heads_per_unit(p.all, p.side[0].heads, 32 / G, kSteps, most * kWarps);
  const int64_t units = (int64_t)p.all * ((p.side[0].heads + per - 1) / per +
                                          (p.side[1].heads + per - 1) / per);
  const int64_t ctas = (units + kWarps - 1) / kWarps;
  return launch_kernel(kern, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kThreads), 0, s, 1,
                       p, per);
}

template <typename T, int G, int MODE, bool PART>
cudaError_t launch_bwd_g(RotaryParams& p, cudaStream_t s) {
  constexpr auto kern = rotary_bwd_vec<T, G, MODE, PART>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = allow_launch<kern>(dev, 0);
  if (e != cudaSuccess) return e;
  constexpr int hps = 32 / G;
  const int sms = sm_count(dev);
  const int64_t most = (int64_t)sms * max_blocks_per_sm((const void*)kern, kThreads, 0);
  const int per = heads_per_unit(p.all, p.side[0].heads, hps, kBwdSteps,
                                 (p.direct ? 2 * kMaxCluster : most) * kWarps);
  // a unit costs its steps and about one more for its angles (shared by heads alone
  // the keys' CTAs end last: 4096 x (32+8) x 128 bf16 30.5 us, 29.7
  // so; 16384 x (32+8) x 64 69 and 56)
  const auto cost = [&](int heads) {
    return (int64_t)((heads + hps - 1) / hps + (heads + per - 1) / per);
  };
  const int cluster =
      place_ctas(p, most, kWarps * hps, sms, cost(p.side[0].heads), cost(p.side[1].heads));
  return launch_kernel(kern, dim3((unsigned)(p.side[0].ctas + p.side[1].ctas)), dim3(kThreads), 0,
                       s, cluster, p, per);
}

// f(G, MODE, PART) of the kernel for a row's lanes.
template <typename T, typename F>
bool with_kernel(const RotaryParams& p, F f) {
  const int mode = mode_of<T>(p), lanes = lanes_of(p, Traits<T>::kVec, mode);
  auto by_mode = [&](auto g) {
    auto by_part = [&](auto m) {
      if (2 * p.half < p.dim) f(g, m, std::true_type{});
      else f(g, m, std::false_type{});
    };
    if (mode == kHalves) by_part(std::integral_constant<int, kHalves>{});
    else if (mode == kNeighbours) by_part(std::integral_constant<int, kNeighbours>{});
    else f(g, std::integral_constant<int, kApart>{}, std::false_type{});
    return true;
  };
  if (lanes <= 4) return by_mode(std::integral_constant<int, 4>{});
  if (lanes <= 8) return by_mode(std::integral_constant<int, 8>{});
  if (lanes <= 16) return by_mode(std::integral_constant<int, 16>{});
  if (lanes <= 32) return by_mode(std::integral_constant<int, 32>{});
  return false;
}

template <typename F>
bool with_type(int dtype, F f) {
  if (dtype == RMSN_F32) return f(float{});
  if (dtype == RMSN_BF16) return f(__nv_bfloat16{});
  return f(__half{});
}

}  // namespace

bool try_launch_rotary_fwd_vec(int dtype, const RotaryParams& p, cudaStream_t s, cudaError_t* err) {
  return p.vec_ok && with_type(dtype, [&](auto t) {
    using T = decltype(t);
    return with_kernel<T>(p, [&](auto g, auto m, auto part) {
      *err = launch_fwd_g<T, decltype(g)::value, decltype(m)::value, decltype(part)::value>(p, s);
    });
  });
}

bool try_launch_rotary_bwd_vec(int dtype, RotaryParams& p, cudaStream_t s, cudaError_t* err) {
  return p.vec_ok && with_type(dtype, [&](auto t) {
    using T = decltype(t);
    return with_kernel<T>(p, [&](auto g, auto m, auto part) {
      *err = launch_bwd_g<T, decltype(g)::value, decltype(m)::value, decltype(part)::value>(p, s);
    });
  });
}

}  // namespace rmsn
