// wgrad8.cu -- d_W[i][j] (+)= sum_t g[t][i] X[t][j] with X read from its 8-bit checkpoint: the
// general kernel, in fp32 arithmetic, for any size, stride and type.
//
// A block forms a 64 x 64 tile of d_W over a range of tokens, 4 x 4 values per thread, from
// tiles of 16 tokens staged in shared memory as fp32.  Where the tiles alone leave SMs idle the
// tokens are split over blocks; the splits' tiles go to the workspace and are added in order.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

__device__ __forceinline__ float as_f(float v) { return v; }
__device__ __forceinline__ float as_f(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename IO>
__global__ void __launch_bounds__(kThreads) wgrad8_kernel(const Wgrad a, float* part,
                                                          long long per_split) {
  __shared__ float sg[kDepth][kTile + 4], sx[kDepth][kTile + 4];
  const int tid = threadIdx.x, i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const long long t_begin = blockIdx.z * per_split;
  const long long t_end = t_begin + per_split < a.tokens ? t_begin + per_split : a.tokens;
  const int nb = (a.k + 31) / 32;
  const int ti = tid / 16, tj = tid % 16;
  float acc[4][4] = {};
  for (long long t0 = t_begin; t0 < t_end; t0 += kDepth) {
#pragma unroll
    for (int r = 0; r < kDepth * kTile / kThreads; r++) {
      const int at = tid + r * kThreads, tt = at / kTile, c = at % kTile;
      const long long t = t0 + tt;
      float gv = 0.0f, xv = 0.0f;
      if (t < t_end) {
        if (i0 + c < a.m) gv = as_f(((const IO*)a.g)[t * a.ld_g + i0 + c]);
        if (j0 + c < a.k)
          xv = (float)a.q[t * a.k + j0 + c] * block_step(a.e[t * nb + (j0 + c) / 32]);
      }
      sg[tt][c] = gv;
      sx[tt][c] = xv;
    }
    __syncthreads();
#pragma unroll
    for (int tt = 0; tt < kDepth; tt++) {
      const float4 gv = *reinterpret_cast<const float4*>(&sg[tt][4 * ti]);
      const float4 xv = *reinterpret_cast<const float4*>(&sx[tt][4 * tj]);
      const float gs[4] = {gv.x, gv.y, gv.z, gv.w}, xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int u = 0; u < 4; u++)
#pragma unroll
        for (int v = 0; v < 4; v++) acc[u][v] = fmaf(gs[u], xs[v], acc[u][v]);
    }
    __syncthreads();
  }
  float* dst = part ? part + (long long)blockIdx.z * a.m * a.k : a.d_W;
#pragma unroll
  for (int u = 0; u < 4; u++)
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int i = i0 + 4 * ti + u, j = j0 + 4 * tj + v;
      if (i < a.m && j < a.k) {
        const long long at = (long long)i * a.k + j;
        dst[at] = !part && a.accumulate ? dst[at] + acc[u][v] : acc[u][v];
      }
    }
}

__global__ void wgrad8_sum_kernel(const float* __restrict__ part, int splits, long long n,
                                  float* d_W, int accumulate) {
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    float v = 0.0f;
    for (int s = 0; s < splits; s++) v += __ldg(part + s * n + i);
    d_W[i] = accumulate ? d_W[i] + v : v;
  }
}

// Splits of the tokens: enough for two blocks per SM, at least 256 tokens each.
int splits_of(long long tokens, int m, int k, int sms) {
  const long long tiles = (long long)((m + kTile - 1) / kTile) * ((k + kTile - 1) / kTile);
  long long s = (2LL * sms + tiles - 1) / tiles, most = (tokens + 255) / 256;
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}

}  // namespace

size_t wgrad_ws_bytes(long long tokens, int m, int k, int io, int sms) {
  // the larger of the two kernels': which one a call takes depends on its pointers and strides
  int s = splits_of(tokens, m, k, sms);
  if (io == SSM_BF16) {
    const int t = wgrad_tc_splits(tokens, m, k, sms);
    if (t > s) s = t;
  }
  return kStatusBytes + (s > 1 ? sizeof(float) * (size_t)s * m * k : 0);
}

cudaError_t launch_wgrad(const Wgrad& a, void* ws, int sms, cudaStream_t st) {
  const bool tc = wgrad_tc_applies(a);
  const int s = tc ? wgrad_tc_splits(a.tokens, a.m, a.k, sms) : splits_of(a.tokens, a.m, a.k, sms);
  float* part = s > 1 ? (float*)((char*)ws + kStatusBytes) : nullptr;
  if (tc) {
    if (cudaError_t e = launch_wgrad_tc(a, part, s, (int*)ws, st)) return e;
  } else {
    const long long per = ((a.tokens + s - 1) / s + kDepth - 1) / kDepth * kDepth;
    const dim3 grid((a.k + kTile - 1) / kTile, (a.m + kTile - 1) / kTile, s);
    if (a.io == SSM_F32)
      wgrad8_kernel<float><<<grid, kThreads, 0, st>>>(a, part, per);
    else
      wgrad8_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, part, per);
    count_launches(1);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  if (part) {
    const long long n = (long long)a.m * a.k, b = (n + 255) / 256;
    wgrad8_sum_kernel<<<(int)(b < 8LL * sms ? b : 8LL * sms), 256, 0, st>>>(part, s, n, a.d_W,
                                                                          a.accumulate);
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace ssm
