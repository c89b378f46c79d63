// wgrad8.cu -- d_W[i][j] (+)= sum_t g[t][i] X[t][j] with X read from its 8-bit checkpoint: what
// happens around the tensor-core kernel of wgrad8_tc.cu.
//   before  operands that it cannot read as they are go to the workspace in a form that it can:
//           fp32 g as three bf16 terms, rows that are not 16-byte aligned with their rows padded
//   after   where the tokens are split over blocks, the splits' tiles are added in order
// The copies read and write each value once.  8189 tokens x 64 x 512, fp32 g (GB300): 16.7 us, a chain
// of three kernels, each set up while the one before it runs (one after the other, with the status word
// cleared by a copy of its own: 20.5).  8192 x 2048 x 1024: 94 us, 1100 TFLOP/s of bf16 products for
// 367 of fp32 (a library fp32 product: 61).  Padding: 8192 x 1000 x 1008 in bf16 26 us, x 1001 50.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 256;

// A call's first kernel clears its status word; the tensor-core kernel may be set up meanwhile (it
// waits where it needs the copies).
__device__ __forceinline__ void first_of_call(int* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  asm volatile("griddepcontrol.launch_dependents;");
}
__global__ void clear_status_kernel(int* status) { first_of_call(status); }

// A thread pads 8 columns of a row of bf16 g.
__global__ void __launch_bounds__(kThreads) pad_g_kernel(const __nv_bfloat16* g, long long ld,
                                                         __nv_bfloat16* out, int m, int m8,
                                                         long long n, int* status) {
  first_of_call(status);
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const long long t = i / (m8 / 8);
    const int c = (int)(i - t * (m8 / 8)) * 8;
    const __nv_bfloat16* p = g + t * ld + c;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t lo = c + 2 * j < m ? __bfloat16_as_ushort(p[2 * j]) : 0u;
      const uint32_t hi = c + 2 * j + 1 < m ? __bfloat16_as_ushort(p[2 * j + 1]) : 0u;
      w[j] = lo | hi << 16;
    }
    *reinterpret_cast<uint4*>(out + t * m8 + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// fp32 as three bf16 terms: 8 leading bits of the 24, the next 8 and the last 8, cut off rather than
// rounded, so that the terms' sum is the value exactly (above the smallest normal numbers).  What is
// not finite stays so in the first term.
__device__ __forceinline__ void three_bf16(float v, uint32_t (&h)[3]) {
  const uint32_t b = __float_as_uint(v);
  h[0] = b >> 16, h[1] = h[2] = 0u;
  if ((b & 0x7f800000u) == 0x7f800000u) {
    if (b & 0x7fffffu) h[0] = 0x7fc0u;
    return;
  }
  const float r = v - __uint_as_float(b & 0xffff0000u);
  const uint32_t rb = __float_as_uint(r);
  h[1] = rb >> 16;
  h[2] = __float_as_uint(r - __uint_as_float(rb & 0xffff0000u)) >> 16;
}

// A thread splits 8 columns of a row of fp32 g into planes [3][tokens][m8].
template <bool VEC>
__global__ void __launch_bounds__(kThreads) split_g_kernel(const float* g, long long ld,
                                                           __nv_bfloat16* out, long long plane,
                                                           int m, int m8, long long n,
                                                           int* status) {
  first_of_call(status);
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const long long t = i / (m8 / 8);
    const int c = (int)(i - t * (m8 / 8)) * 8;
    const float* p = g + t * ld + c;
    float v[8];
    if constexpr (VEC) {
      Cols<float, 8> x;
      x.load(p);
      x.get(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = c + j < m ? p[j] : 0.0f;
    }
    uint32_t w[3][4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t a[3], b[3];
      three_bf16(v[2 * j], a);
      three_bf16(v[2 * j + 1], b);
#pragma unroll
      for (int r = 0; r < 3; r++) w[r][j] = a[r] | b[r] << 16;
    }
#pragma unroll
    for (int r = 0; r < 3; r++)
      *reinterpret_cast<uint4*>(out + r * plane + t * m8 + c) =
          make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
  }
}

// A thread pads 16 columns of a row of q.
__global__ void __launch_bounds__(kThreads) pad_q_kernel(const int8_t* q, int8_t* out, int k,
                                                         int k16, long long n, int* status) {
  first_of_call(status);
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const long long t = i / (k16 / 16);
    const int c = (int)(i - t * (k16 / 16)) * 16;
    const uint8_t* p = (const uint8_t*)q + t * k + c;
    uint32_t w[4] = {};
#pragma unroll
    for (int j = 0; j < 16; j++)
      if (c + j < k) w[j / 4] |= (uint32_t)p[j] << (8 * (j % 4));
    *reinterpret_cast<uint4*>(out + t * k16 + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// d_W (+)= the splits' tiles: a block adds 32 x VEC values in kThreads / 32 slices of the splits, every
// slice in order, then the slices in order (`slices` of them: one where the splits are few).
template <int VEC>
__global__ void __launch_bounds__(kThreads) wgrad8_sum_kernel(const float* part, int splits,
                                                              int slices, long long n, float* d_W,
                                                              int accumulate) {
  __shared__ float s[kThreads / 32][32 * VEC + 1];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  // slices == 1: every warp takes 32 x VEC values of its own
  const long long i = (slices == 1 ? (long long)blockIdx.x * (kThreads / 32) + y : blockIdx.x) *
                          (32LL * VEC) + x * VEC;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the tiles are complete
  float v[VEC] = {};
  if (i < n) {
#pragma unroll 4
    for (int t = slices == 1 ? 0 : y; t < splits; t += slices) {
      if constexpr (VEC == 4) {
        const float4 p = *reinterpret_cast<const float4*>(part + t * n + i);
        v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
      } else {
        v[0] += part[t * n + i];
      }
    }
  }
  if (slices > 1) {
#pragma unroll
    for (int j = 0; j < VEC; j++) s[y][x * VEC + j] = v[j];
    __syncthreads();
    if (y != 0) return;
    for (int t = 1; t < slices; t++)
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] += s[t][x * VEC + j];
  }
  if (i < n)
#pragma unroll
    for (int j = 0; j < VEC; j++) d_W[i + j] = accumulate ? d_W[i + j] + v[j] : v[j];
}

int blocks_of(long long n, int sms) {
  const long long b = (n + kThreads - 1) / kThreads;
  return (int)(b < 16LL * sms ? b : 16LL * sms);
}

// The workspace after the status word: g's copy, q's copy, the splits' tiles.
struct Plan {
  int terms, splits, m8, k16;
  bool copy_g, copy_q;
  size_t g, q, part, bytes;
};
Plan plan_of(long long tokens, int m, int k, int io, bool aligned_g, bool aligned_q, int sms) {
  Plan p{};
  p.terms = io == SSM_F32 ? 3 : 1;
  p.m8 = (m + 7) / 8 * 8;
  p.k16 = (k + 15) / 16 * 16;
  p.copy_g = io == SSM_F32 || p.m8 != m || !aligned_g;
  p.copy_q = p.k16 != k || !aligned_q;
  p.splits = wgrad_tc_splits(tokens, p.terms, m, k, sms);
  p.g = kStatusBytes;
  p.q = p.g + (p.copy_g ? align_up((size_t)p.terms * tokens * p.m8 * 2, 256) : 0);
  p.part = p.q + (p.copy_q ? align_up((size_t)tokens * p.k16, 256) : 0);
  p.bytes = p.part + (p.splits > 1 ? sizeof(float) * (size_t)p.splits * m * k : 0);
  return p;
}

}  // namespace

// Each operand is copied for its own sake only: what is not 16-byte aligned costs a pass over itself, and
// fp32 g, which is copied in any case, may lie anywhere.
static Plan plan_of(const Wgrad& a, int sms) {
  const size_t row = (size_t)a.ld_g * (a.io == SSM_F32 ? 4 : 2);
  return plan_of(a.tokens, a.m, a.k, a.io, (uintptr_t)a.g % 16 == 0 && row % 16 == 0,
                 (uintptr_t)a.q % 16 == 0, sms);
}

size_t wgrad_ws_bytes(long long tokens, int m, int k, int io, bool aligned, int sms) {
  return plan_of(tokens, m, k, io, aligned, aligned, sms).bytes;
}
size_t wgrad_ws_bytes(const Wgrad& a, int sms) { return plan_of(a, sms).bytes; }

cudaError_t launch_wgrad(const Wgrad& a, void* ws, int sms, cudaStream_t st) {
  const Plan p = plan_of(a, sms);
  char* w = (char*)ws;
  int* status = (int*)ws;
  const void* g = a.g;
  long long ld_g = a.ld_g, ld_q = a.k;
  const int8_t* q = a.q;
  if (p.copy_g) {
    __nv_bfloat16* out = (__nv_bfloat16*)(w + p.g);
    const long long n = a.tokens * (p.m8 / 8);
    if (a.io == SSM_F32) {
      const bool vec = p.m8 == a.m && a.ld_g % 8 == 0 && (uintptr_t)a.g % 32 == 0;
      auto kernel = vec ? split_g_kernel<true> : split_g_kernel<false>;
      kernel<<<blocks_of(n, sms), kThreads, 0, st>>>((const float*)a.g, a.ld_g, out,
                                                     a.tokens * p.m8, a.m, p.m8, n, status);
    } else {
      pad_g_kernel<<<blocks_of(n, sms), kThreads, 0, st>>>((const __nv_bfloat16*)a.g, a.ld_g, out,
                                                           a.m, p.m8, n, status);
    }
    count_launches(1);
    if (cudaError_t e = cudaGetLastError()) return e;
    g = out;
    ld_g = p.m8;
  }
  if (p.copy_q) {
    int8_t* out = (int8_t*)(w + p.q);
    const long long n = a.tokens * (p.k16 / 16);
    pad_q_kernel<<<blocks_of(n, sms), kThreads, 0, st>>>(a.q, out, a.k, p.k16, n, status);
    count_launches(1);
    if (cudaError_t e = cudaGetLastError()) return e;
    q = out;
    ld_q = p.k16;
  }
  if (!p.copy_g && !p.copy_q) {
    clear_status_kernel<<<1, 32, 0, st>>>(status);
    count_launches(1);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  float* part = p.splits > 1 ? (float*)(w + p.part) : nullptr;
  if (cudaError_t e = launch_wgrad_tc(g, ld_g, p.terms, q, ld_q, a, part, p.splits, status, st))
    return e;
  if (!part) return cudaSuccess;
  const long long n = (long long)a.m * a.k;
  const bool vec = n % 4 == 0;
  const int slices = p.splits >= 16 ? kThreads / 32 : 1;
  const long long per = (vec ? 128 : 32) * (slices == 1 ? kThreads / 32 : 1);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)((n + per - 1) / per));
  c.blockDim = dim3(kThreads);
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&c, vec ? wgrad8_sum_kernel<4> : wgrad8_sum_kernel<1>,
                            (const float*)part, p.splits, slices, n, a.d_W, a.accumulate);
}

}  // namespace ssm
