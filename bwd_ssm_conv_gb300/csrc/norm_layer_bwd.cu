// norm_layer_bwd.cu -- residual add + layer norm in front of a block, backward:
//   n = (s - mean) rstd,  a = w d_out,  r = d_s + rstd (a - mean(a) - n mean(a n)),
//   d_residual = r,  d_x = scale r,  d_w = sum_rows d_out n,  d_b = sum_rows d_out,
//   d_scale = sum_rows r x
// A row is read once, copied ahead to shared memory, and its two sums are formed together over its threads.
// Memory bounds it.  GB300: 32768 x 768 bf16 with an fp32 stream, d_s and d_scale 77 us (67 at the rate of a copy)
// and 7 us for the column sums' join; 16384 x 1024 all bf16 33 (25) and 7; 2047 x 1003 fp32 in single columns
// 14.7 and 5, bound by instructions.
// Each pair of types in a file of its own, as they take the compiler a minute each.
#include "norm_add_bwd.cuh"

namespace ssm {

cudaError_t launch_add_layer_norm_bwd(const AddNormBwd& a, int io, int res_io, bool vec, int sms,
                                      cudaStream_t st) {
  if (io == SSM_F32) return add_layer_norm_bwd_f32(a, vec, sms, st);
  if (res_io == SSM_F32) return add_layer_norm_bwd_mixed(a, vec, sms, st);
  return bwd_types<true, __nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
}

}  // namespace ssm
