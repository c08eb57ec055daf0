// Embedding, forward: the rows of a table that a batch of tokens takes, scaled.
#include "embedding.cuh"

namespace rmsn {
namespace {

// A warp takes K times 32 E columns of a token's row, all loads under way together:
// kWide times where that leaves kWideWarps units an SM of rows cut so, else one.
// Large batches gain (32768 x 4096 bf16 80.9 us by ones, 79.5; 32768 x 1024 21.1 and
// 20.4), the smallest lose warps (256 x 1024 2.1 us by ones, 2.6 by fours).  Columns
// left over cost a warp (8192 x 1088 8.8 by ones, 10.0), and batches between would
// gain too (2048 x 1024 3.6 us by ones, as the rule has it, 2.7 by fours).
constexpr int kWide = 4, kWideWarps = 32;

template <typename T, typename U, bool VEC, int K>
__global__ void __launch_bounds__(kThreads) embedding_rows(Ids ids, const T* weight, U* y,
                                                           int64_t tokens, int64_t vocab,
                                                           int hidden, float scale) {
  constexpr int E = kElems<T, U>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slabs = (hidden + 32 * E * K - 1) / (32 * E * K);
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < tokens * slabs;
       u += (int64_t)gridDim.x * kWarps) {
    const int64_t t = u / slabs;
    const int c = first_column<VEC, E>((int)(u - t * slabs) * K, lane);
    const int id = ids.get(t, vocab);
    float f[K][E] = {};
    if (id >= 0) {
      const T* row = weight + (int64_t)id * hidden;
#pragma unroll
      for (int k = 0; k < K; ++k) load_row<VEC, E>(row, c + k * 32 * E, hidden, f[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < E; ++i) f[k][i] = id >= 0 ? f[k][i] * scale : 0.f;
      store_row<VEC, E>(y + t * hidden, c + k * 32 * E, hidden, f[k]);
    }
  }
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
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  e = with_types(weight_dtype, y_dtype, [&](auto t, auto u) {
    using T = decltype(t);
    using U = decltype(u);
    constexpr int E = kElems<T, U>;
    const bool vec = rows_ok(weight, hidden, wb) && rows_ok(y, hidden, yb) && hidden % E == 0;
    const auto launch = [&](auto kern, int k) {
      return launch_units(kern, tokens * ceil_div(hidden, 32 * E * k),
                          static_cast<cudaStream_t>(stream), of, static_cast<const T*>(weight),
                          static_cast<U*>(y), tokens, vocab, (int)hidden, scale);
    };
    constexpr int K = kWide;
    if (vec && tokens * (hidden / (32 * E * K)) >= (int64_t)kWideWarps * sm_count(dev))
      return launch(embedding_rows<T, U, true, K>, K);
    return vec ? launch(embedding_rows<T, U, true, 1>, 1)
               : launch(embedding_rows<T, U, false, 1>, 1);
  });
  if (e != cudaSuccess) return cuda_fail(e);
  set_last_launches(1);
  return RMSN_OK;
}

}  // extern "C"
