// norm_layer.cu -- residual add + layer norm in front of a block, forward:
//   s = residual + scale x,  out = w (s - mean) rstd + b,  rstd = (mean((s - mean)^2) + eps)^-1/2
// The row stays in registers between its two sums, that of s and, with the mean known, that of the
// squares of what is left: E[s^2] - mean^2 would lose what a mean far from zero leaves of the digits.
//
// Memory bounds it; with two sums of a row one after the other it is the loads in flight that have to cover
// them, so rows of up to 8192 columns are copied ahead to shared memory (kRing), which the RMSNorm's forward with
// its one sum goes without.  GB300: 32768 x 768 bf16 with an fp32 stream and both saved 48 us (45 at the rate of a
// copy), 16384 x 1024 all bf16 24 (20).  Odd widths (single columns, no copies ahead): 2047 x 1003 fp32 9.5 us,
// bound by instructions, a load and a store for every 4 bytes.
#include "norm_add.cuh"

namespace ssm {

cudaError_t launch_add_layer_norm_fwd(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                      cudaStream_t st) {
  return launch_add_norm_fwd_of<true>(a, io, res_io, vec, sms, st);
}

}  // namespace ssm
