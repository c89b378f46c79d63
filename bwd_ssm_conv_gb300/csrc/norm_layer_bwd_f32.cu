// norm_layer_bwd_f32.cu -- the layer norm's backward (norm_layer_bwd.cu), everything in fp32.
#include "norm_add_bwd.cuh"

namespace ssm {

cudaError_t add_layer_norm_bwd_f32(const AddNormBwd& a, bool vec, int sms, cudaStream_t st) {
  return bwd_types<true, float, float>(a, vec, sms, st);
}

}  // namespace ssm
