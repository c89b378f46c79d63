// norm_plan.cu -- how the norms' launches are laid out, and the sums over rows that their
// backwards share.
#include "block.cuh"

namespace ssm {

namespace {

constexpr int kFewRows = 4;  // rows per SM below which a row is spread over more threads

// out[c] = sum_b part[b][c]: 32 columns x 32 slices per block, every slice in order, then the
// slices in order.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ part, int n,
                                                           int cols, float* __restrict__ out) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int b = threadIdx.y; b < n; b += 32) v += __ldg(part + (long long)b * cols + c);
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i++) t += s[i][threadIdx.x];
    out[c] = t;
  }
}

}  // namespace

NormShape norm_shape(long long rows, int group, int groups, bool vec, int sms, bool backward) {
  NormShape s{};
  int nj, per_sm;
  if (vec) {
    const int nch = group / 8;
    const bool few = rows * groups < (long long)kFewRows * sms;
    if (nch <= 32 || (few && nch <= 1024)) {
      s.variant = kVec8x1, nj = 1;
    } else if (nch <= 512 && (backward || nch <= 64)) {
      s.variant = kVec8x2, nj = 2;
    } else if (nch <= 1024) {
      s.variant = kVec8x4, nj = 4;
    } else {
      s.variant = kVec8x4Wide, nj = 4;
    }
    const int tpr = row_threads(nch, nj, 8);
    per_sm = tpr <= 128 ? 8 : (tpr <= 256 ? 6 : 2);
    s.plan = row_plan(rows, group, groups, tpr, 128, per_sm, sms);
  } else {
    nj = group <= 64 ? 2 : (group <= 8192 ? 8 : 32);
    s.variant = nj == 2 ? kOne2 : (nj == 8 ? kOne8 : kOne32);
    const int tpr = row_threads(group, nj, 1);
    per_sm = tpr <= 128 ? 8 : (tpr <= 256 ? 6 : 2);
    s.plan = row_plan(rows, group, groups, tpr, 128, per_sm, sms);
  }
  return s;
}

size_t column_sums_bytes(long long rows, int group, int groups, int sms, int sums) {
  // the larger of the two layouts: which one a call takes depends on its pointers and strides
  int n = norm_shape(rows, group, groups, false, sms, true).plan.nbx;
  if (group % 8 == 0) {
    const int v = norm_shape(rows, group, groups, true, sms, true).plan.nbx;
    if (v > n) n = v;
  }
  return sizeof(float) * (size_t)sums * n * group * groups;
}

cudaError_t launch_column_sums(const float* part, int n, int cols, float* out, cudaStream_t st) {
  column_sums_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, st>>>(part, n, cols, out);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace ssm
