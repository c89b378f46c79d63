// norm_add.cu -- residual add + RMSNorm in front of a block, forward:
//   s = residual + scale x,  out = w s rstd,  rstd = (mean(s^2) + eps)^-1/2
// A row is read once into registers, its one sum formed over the row's threads and its results
// written, so that the kernel is bound by the memory traffic of its operands: 32768 rows of 768
// columns, bf16 with an fp32 stream, scale and the stream's 8-bit checkpoint take 51 us for 328 MB
// (GB300; 57 with inputs and outputs from call to call beyond L2, 5.7 TB/s of 6.7 measured for a copy; 70
// while w and scale were loaded as single values).  Four chunks per thread (2048, 4096 and 8192 columns)
// spill 88 - 104 bytes of registers per thread, rows beyond 8192 columns 400 - 620: 8192 x 4096, all in
// bf16, takes 55 us of 40, 2048 x 16384 89 of 40.
// The stream is formed with the product and the sum rounded one after the other, so that it holds
// the same bits as an unfused add does.
#include "norm_add.cuh"

namespace ssm {

cudaError_t launch_add_norm_fwd(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st) {
  return launch_add_norm_fwd_of<false>(a, io, res_io, vec, sms, st);
}

}  // namespace ssm
