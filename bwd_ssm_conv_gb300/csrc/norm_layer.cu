// norm_layer.cu -- residual add + layer norm in front of a block, forward:
//   s = residual + scale x,  out = w (s - mean) rstd + b,  rstd = (mean((s - mean)^2) + eps)^-1/2
// The row stays in registers between its two sums, that of s and, with the mean known, that of the
// squares of what is left: E[s^2] - mean^2 would lose what a mean far from zero leaves of the digits.
#include "norm_add.cuh"

namespace ssm {

cudaError_t launch_add_layer_norm_fwd(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                      cudaStream_t st) {
  return launch_add_norm_fwd_of<true>(a, io, res_io, vec, sms, st);
}

}  // namespace ssm
