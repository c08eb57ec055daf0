// The staged block norm's backward, aligned rows.
#include "block_bwd_tma.cuh"

namespace rmsn {

bool try_launch_block_bwd_tma(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p,
                              int* units, cudaStream_t s, cudaError_t* err) {
  return bwd_types<false>(dtype, res_dtype, a, p, units, s, err);
}

cudaError_t read_block_bwd_tma_wait_timeouts(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_block_timeouts, sizeof(unsigned int));
}

}  // namespace rmsn
