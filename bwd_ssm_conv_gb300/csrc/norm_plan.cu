// norm_plan.cu -- how the norms' launches are laid out, and the sums over rows that their
// backwards share.
#include <stdlib.h>

#include "block.cuh"

namespace ssm {

namespace {

// Groups per SM below which a group is spread over as many threads as it has chunks: one chunk each
// is the shortest chain (16 rows of 1536 columns, gated: 2.5 us).
constexpr int kFewRows = 4;

// out[c] = sum_b part[b][c]: a block sums 32 columns (blockIdx.x) of one of the sums (blockIdx.y),
// 8 threads x 4 columns across and 128 slices of the rows, every slice in order, then the slices in
// order.  Its launch is set up while the kernel that writes `part` runs (which gives no early signal, so
// that this one starts at its end) and it waits here for that one's results: 2 - 3 us less per
// backward than an ordinary launch (8192 x 512 fp32, forward and backward: 34.9 and 37.6 us).
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* part, int n, int cols,
                                                           float* out0, float* out1,
                                                           float* out2) {
  __shared__ float s[128][33];
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, c = blockIdx.x * 32 + 4 * tx;
  int nth = blockIdx.y;  // of the outputs that are given
  float* out = out0 && nth-- == 0 ? out0 : out1 && nth-- == 0 ? out1 : out2;
  part += (long long)blockIdx.y * n * cols;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v[4] = {};
  if (cols % 4 == 0) {
    if (c < cols) {
#pragma unroll 4
      for (int b = ty; b < n; b += 128) {
        const float4 p = *reinterpret_cast<const float4*>(part + (long long)b * cols + c);
        v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
      }
    }
  } else {
#pragma unroll 4
    for (int b = ty; b < n; b += 128)
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (c + i < cols) v[i] += part[(long long)b * cols + c + i];
  }
#pragma unroll
  for (int i = 0; i < 4; i++) s[ty][4 * tx + i] = v[i];
  __syncthreads();
  // 32 threads per column: 4 slices each, then over the warp
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  float t = (s[4 * l][w] + s[4 * l + 1][w]) + (s[4 * l + 2][w] + s[4 * l + 3][w]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if (l == 0 && blockIdx.x * 32 + w < cols) out[blockIdx.x * 32 + w] = t;
}

}  // namespace

NormShape norm_shape(long long rows, int group, int groups, bool vec, int sms, bool backward) {
  NormShape s{};
  int nj;
  if (vec) {
    const int nch = group / 8;
    const bool few = rows * groups < (long long)kFewRows * sms;
    if (nch <= 32 || (few && nch <= 1024)) {
      nj = 1, s.variant = nch <= 256 ? kVec1 : kVec1Wide;
    } else if (nch > 1024) {
      nj = 4, s.variant = kVec4Wide;
    } else if (backward && nch > 512) {
      nj = 2, s.variant = kVec2Wide;
    } else {
      // Of 4, 3 and 2 chunks per thread (2 and 1 in the backward, which keeps more of each) the one
      // that leaves the fewest threads without a chunk: on 32768 rows of 1536 bf16 columns from and to
      // 8 bits the forward takes 68 us with 3, 75 with 2, 86 with 4 and 92 with 1, the backward 96 with
      // 2 and 106 with 1; add_norm's backward of 32768 x 768 65 with 1 and 72 with 2.
      // Among equals the forward takes the one nearest to two warps per row (add_norm of bf16 rows and an
      // fp32 stream, 2 and 4 chunks: 16384 x 512 20.5 and 22.6 us, 16384 x 1024 36.8 and 39.3; both
      // bf16, 8192 x 2048: 32.2 and 30.4), the backward the larger, whose fewer rows at a time leave
      // fewer column sums to add (8192 x 512 fp32, 2 and 1: 22.6 and 22.7 us with them).
      int best = -1, from64 = 0;
      nj = 2;
      for (int k = backward ? 2 : 4; k >= (backward ? 1 : 2); k--) {
        const int tpr = row_threads(nch, k, 8), idle = tpr * k - nch, off = abs(tpr - 64);
        if (tpr <= 256 && (best < 0 || idle < best || (!backward && idle == best && off < from64)))
          nj = k, best = idle, from64 = off;
      }
      s.variant = nj == 1 ? kVec1 : (nj == 2 ? kVec2 : (nj == 3 ? kVec3 : kVec4));
    }
    s.plan = row_plan(rows, group, groups, row_threads(nch, nj, 8), 128,
                      norm_threads_per_sm(s.variant, backward), sms);
  } else {
    nj = group <= 64 ? 2 : (group <= 1024 ? 4 : (group <= 8192 ? 8 : 32));
    s.variant = nj == 2   ? kOne2
                : nj == 4 ? kOne4
                : nj == 8 ? (group <= 4096 ? kOne8 : kOne8Wide)
                          : kOne32;
    s.plan = row_plan(rows, group, groups, row_threads(group, nj, 1), 128,
                      norm_threads_per_sm(s.variant, backward), sms);
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

cudaError_t launch_column_sums(const float* part, int n, int cols, float* out0, float* out1,
                               float* out2, cudaStream_t st) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((cols + 31) / 32, (out0 ? 1 : 0) + (out1 ? 1 : 0) + (out2 ? 1 : 0));
  c.blockDim = dim3(1024);
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, column_sums_kernel, part, n, cols, out0, out1, out2);
  count_launches(1);
  return e;
}

}  // namespace ssm
