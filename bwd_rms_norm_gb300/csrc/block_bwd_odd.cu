// The staged block norm's backward, rows that start anywhere in 16 bytes.
#include "block_bwd_tma.cuh"

namespace rmsn {

bool try_launch_block_bwd_odd(int dtype, int res_dtype, const BlockBwdArgs& a, BlockBwdParams& p,
                              int* units, cudaStream_t s, cudaError_t* err) {
  return bwd_types<true>(dtype, res_dtype, a, p, units, s, err);
}

cudaError_t read_block_bwd_odd_wait_timeouts(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_block_timeouts, sizeof(unsigned int));
}

}  // namespace rmsn
