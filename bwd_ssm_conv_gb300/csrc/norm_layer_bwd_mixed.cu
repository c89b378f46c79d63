// norm_layer_bwd_mixed.cu -- the layer norm's backward (norm_layer_bwd.cu), bf16 activations and an fp32 stream.
#include "norm_add_bwd.cuh"

namespace ssm {

cudaError_t add_layer_norm_bwd_mixed(const AddNormBwd& a, bool vec, int sms, cudaStream_t st) {
  return bwd_types<true, __nv_bfloat16, float>(a, vec, sms, st);
}

}  // namespace ssm
