// norm_add_bwd.cu -- residual add + RMSNorm in front of a block, backward:
//   n = s rstd,  r = d_s + rstd (w d_out - n mean(w d_out n)),
//   d_residual = r,  d_x = scale r,  d_w = sum_rows d_out n,  d_scale = sum_rows r x
// A row of up to 4096 columns is read once, copied to shared memory (rows.cuh; one or two rows ahead,
// none for fp32 rows of two chunks per thread, which fill it), and its one sum formed over its threads.
// A thread's columns are fixed, so the column sums stay in registers over a block's rows; the blocks'
// sums are added by column_sums_kernel (norm_plan.cu).
// Memory traffic bounds it: 32768 rows of 768 columns, bf16 with an fp32 stream, the stream from 8
// bits, d_scale: 59 us for 378 MB, with the column sums and inputs and outputs beyond L2 65 (GB300).  It
// took 106 us with plain loads, 251 us with the next row loaded ahead into registers (which spill), and
// 77 us copied ahead past L1, where the two halves of an fp32 chunk each fetched their sector.
// Wider rows are read with plain loads, beyond 8192 columns by threads that hold 32 columns each and
// spill 2.0 KB (single columns 1.0 KB beyond 4096, 3.7 KB beyond 8192): all in bf16, 8192 x 5120
// takes 236 us of 63, 4096 x 8192 130 of 50, 2048 x 16384 334 of 50.
#include "norm_add_bwd.cuh"

namespace ssm {

cudaError_t launch_add_norm_bwd(const AddNormBwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st) {
  if (io == SSM_F32) return bwd_types<false, float, float>(a, vec, sms, st);
  if (res_io == SSM_F32) return bwd_types<false, __nv_bfloat16, float>(a, vec, sms, st);
  return bwd_types<false, __nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
}

}  // namespace ssm
