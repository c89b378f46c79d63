// block.cuh -- launchers of the operators around the scan (norm_add.cu, norm_gated.cu, ckpt8.cu,
// wgrad8.cu), called by the C ABI in block_api.cu, and what the norms' kernels share.
#pragma once

#include <cuda_runtime.h>

#include "kernels.cuh"
#include "rows.cuh"

namespace ssm {

// ---- the norms' launches ----------------------------------------------------------------------
// The kernel instances: columns of an access, accesses per thread, most threads of a block and
// blocks of that size that the registers leave room for.
enum NormVariant { kVec1, kVec1Wide, kVec2, kVec2Wide, kVec3, kVec4, kVec4Wide, kOne2, kOne4,
                   kOne8, kOne8Wide, kOne32 };
#define SSM_NORM_CASES(LAUNCH)                        \
    case ssm::kVec1: LAUNCH(8, 1, 256, 4); break;      \
    case ssm::kVec1Wide: LAUNCH(8, 1, 1024, 1); break; \
    case ssm::kVec2: LAUNCH(8, 2, 256, 2); break;      \
    case ssm::kVec4Wide: LAUNCH(8, 4, 1024, 1); break; \
    case ssm::kOne2: LAUNCH(1, 2, 128, 4); break;      \
    case ssm::kOne8: LAUNCH(1, 8, 512, 1); break;      \
    case ssm::kOne8Wide: LAUNCH(1, 8, 1024, 1); break; \
    default: LAUNCH(1, 32, 1024, 1); break;
#define SSM_NORM_FWD_SWITCH(variant, LAUNCH)           \
  switch (variant) {                                   \
    case ssm::kVec3: LAUNCH(8, 3, 256, 2); break;      \
    case ssm::kVec4: LAUNCH(8, 4, 256, 2); break;      \
    case ssm::kOne4: LAUNCH(1, 4, 256, 4); break;      \
    SSM_NORM_CASES(LAUNCH)                             \
  }
#define SSM_NORM_BWD_SWITCH(variant, LAUNCH)           \
  switch (variant) {                                   \
    case ssm::kVec2Wide: LAUNCH(8, 2, 512, 1); break;  \
    case ssm::kOne4: LAUNCH(1, 4, 256, 3); break;      \
    SSM_NORM_CASES(LAUNCH)                             \
  }
// Threads per SM of a launch's blocks, which all fit at once (registers: the instances above).
inline int norm_threads_per_sm(NormVariant v, bool backward) {
  switch (v) {
    case kVec1: return 768;
    case kOne4: return backward ? 768 : 1024;
    case kVec1Wide: case kVec4Wide: case kOne8Wide: case kOne32: return 1024;
    default: return 512;
  }
}
// The plan of a launch.
struct NormShape {
  NormVariant variant;
  RowPlan plan;
};
NormShape norm_shape(long long rows, int group, int groups, bool vec, int sms, bool backward);

// A backward's column sums: each block's own over its rows, [nbx][cols], then their sum.
size_t column_sums_bytes(long long rows, int group, int groups, int sms, int sums);
// out0 and out1 (either may be NULL) from part [sums][n][cols], in that order.
cudaError_t launch_column_sums(const float* part, int n, int cols, float* out0, float* out1,
                               cudaStream_t st);

inline size_t slots_bytes(const RowPlan& p, int vec, int nj) {
  return p.rpb > 1 ? sizeof(float) * (size_t)p.threads * vec * nj : 0;
}

// Adds a block's rpb rows' column sums in order and stores them at part[blockIdx.x][col].  Every
// thread of the block calls it.
template <int VEC, int NJ>
__device__ __forceinline__ void store_partial(float (&v)[NJ][VEC], const RowPlan& pl,
                                              const RowPos& pos, const int (&col)[NJ],
                                              const bool (&okc)[NJ], int cols, float* part,
                                              float* slots) {
  if (pl.rpb > 1) {
    __syncthreads();  // the area may still be read for an earlier sum
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
      for (int i = 0; i < VEC; i++) slots[(j * VEC + i) * blockDim.x + threadIdx.x] = v[j][i];
    __syncthreads();
    if (pos.slot != 0) return;
    const int step = pl.tpr * pl.gpb;  // threads of one row
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
      for (int i = 0; i < VEC; i++)
        for (int s = 1; s < pl.rpb; s++)
          v[j][i] += slots[(j * VEC + i) * blockDim.x + threadIdx.x + s * step];
  }
#pragma unroll
  for (int j = 0; j < NJ; j++)
    if (okc[j]) st_cols(part + (long long)blockIdx.x * cols + col[j], v[j]);
}

// ---- add_norm -----------------------------------------------------------------------------------
struct AddNormFwd {
  int rows, cols;
  float eps;
  const void* x;
  const void* residual;
  const float* scale;
  const float* w;
  void* out;
  void* res_out;
  float* rstd;
  int ld_x, ld_residual, ld_out, ld_res_out;
  int8_t *res_q, *x_q, *out_q;
  uint8_t *res_e, *x_e, *out_e;
};
struct AddNormBwd {
  int rows, cols;
  const void* d_out;
  const void* d_res_out;
  const void* res;
  const void* x;
  int ld_d_out, ld_d_res_out, ld_res, ld_x;
  const int8_t *res_q, *x_q;
  const uint8_t *res_e, *x_e;
  const float* rstd_in;
  const float* scale;
  const float* w;
  void* d_res;
  void* d_x;
  int ld_d_res, ld_d_x;
  float* d_w;
  float* d_scale;
  float* part;
};
// vec: widths, strides and pointers allow 8 columns at a time
cudaError_t launch_add_norm_fwd(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st);
cudaError_t launch_add_norm_bwd(const AddNormBwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st);

// ---- gated_norm ---------------------------------------------------------------------------------
struct GatedNormFwd {
  int rows, cols, group, norm_first;
  float eps;
  const void* y;
  const void* z;
  const float* w;
  void* out;
  int ld_y, ld_z, ld_out;
  float* rstd;
  int8_t *y_q, *z_q, *out_q;  // y's and z's: both or neither
  uint8_t *y_e, *z_e, *out_e;
};
struct GatedNormBwd {
  int rows, cols, group, norm_first;
  const void* d_out;
  const void* y;
  const void* z;
  int ld_d_out, ld_y, ld_z;
  const int8_t *y_q, *z_q;
  const uint8_t *y_e, *z_e;
  const float* rstd_in;
  const float* w;
  void* d_y;
  void* d_z;
  int ld_d_y, ld_d_z;
  float* d_w;
  float* part;
};
cudaError_t launch_gated_norm_fwd(const GatedNormFwd& a, int io, bool vec, int sms,
                                  cudaStream_t st);
cudaError_t launch_gated_norm_bwd(const GatedNormBwd& a, int io, bool vec, int sms,
                                  cudaStream_t st);

// ---- 8-bit checkpoints ----------------------------------------------------------------------------
cudaError_t launch_ckpt8_save(const void* x, long long ld, int8_t* q, uint8_t* e, long long rows,
                              int cols, int io, int sms, cudaStream_t st);
cudaError_t launch_ckpt8_load(const int8_t* q, const uint8_t* e, void* out, long long ld,
                              long long rows, int cols, int io, int sms, cudaStream_t st);
struct Wgrad {
  const void* g;
  long long ld_g;
  const int8_t* q;
  const uint8_t* e;
  float* d_W;
  long long tokens;
  int m, k, io, accumulate, no_wait;
};
size_t wgrad_ws_bytes(long long tokens, int m, int k, int io, bool aligned, int sms);
size_t wgrad_ws_bytes(const Wgrad& a, int sms);  // what this call needs: at most the above
cudaError_t launch_wgrad(const Wgrad& a, void* ws, int sms, cudaStream_t st);
// The tensor-core kernel (wgrad8_tc.cu): g as `terms` bf16 planes [tokens] x ld_g, q with rows of ld_q
// bytes.  part: the splits' tiles, [splits][m][k], or NULL with one split.
int wgrad_tc_splits(long long tokens, int terms, int m, int k, int sms);
cudaError_t launch_wgrad_tc(const void* g, long long ld_g, int terms, const int8_t* q,
                            long long ld_q, const Wgrad& a, float* part, int splits, int* status,
                            cudaStream_t st);

}  // namespace ssm
