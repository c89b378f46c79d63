// norm_layer_bwd.cu -- residual add + layer norm in front of a block, backward:
//   n = (s - mean) rstd,  a = w d_out,  r = d_s + rstd (a - mean(a) - n mean(a n)),
//   d_residual = r,  d_x = scale r,  d_w = sum_rows d_out n,  d_b = sum_rows d_out,
//   d_scale = sum_rows r x
// A row is read once and its two sums are formed together over its threads.
#include "norm_add_bwd.cuh"

namespace ssm {

cudaError_t launch_add_layer_norm_bwd(const AddNormBwd& a, int io, int res_io, bool vec, int sms,
                                      cudaStream_t st) {
  return launch_add_norm_bwd_of<true>(a, io, res_io, vec, sms, st);
}

}  // namespace ssm
