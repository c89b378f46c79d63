// head_few.cu -- the forward for a few rows (tokens as they come): Z = h W^T with every row of W read once,
// by plain fp32 arithmetic.  W's bytes bound it; a tensor-core tile would be all but empty, its rows would
// have to be packed first, and fp32 W split into planes.  768 columns, 32768 words, in a graph with the kernel
// that joins the sums (GB300), here and by the tensor cores:
//   bf16  1 row 16.1 us, 2 20.0, 4 25.3; tensor cores 23.7 for any number up to 256; reading W 7.4
//   fp32  1 row 23.6 us, 2 25.4, 4 29.8, 8 41.3; tensor cores 87.5; reading W 14.9
// so that up to 2 rows come here, 8 in fp32.
//
// h lies in shared memory as fp32.  A warp takes 4 words at a time, a lane every 32nd chunk of 8 columns
// of each, which leaves 4 to 32 sums of words and rows to add over the lanes: at each step the lanes keep
// half of them and give the other half away, until each has one, the logit of one word and row.
// A lane keeps the maximum and the sum of the exponentials of what comes its way.
// The logits of the rows' own words (or entries) are computed by themselves, a warp each.
#include "head.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 2;  // as the registers leave room for
constexpr int kWarps = kThreads / 32;
constexpr int kWords = 4;  // whose loads are in flight together

struct FewArgs {
  const void* h;
  long long ld_h;
  const void* w;
  long long ld_w;
  const int64_t* target;
  const uint8_t* valid;
  int* idx;
  HeadState* state;
  int* pos;
  float2* stats;  // [blocks][ld_stats]
  float* zt;
  long long ignore, ld_stats;
  int rows, cols, vocab, entries;
  float scale;
};

// 8 columns, or what is left of them, as fp32.
template <typename IO, bool VEC> struct Chunk {
  Cols<IO, VEC ? 8 : 1> c[VEC ? 1 : 8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (VEC ? 1 : 8); i++) c[i].zero();
  }
  __device__ __forceinline__ void load(const IO* p, int left) {  // the rest stays as it is
    if constexpr (VEC) {
      c[0].load(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (i < left) c[i].load(p + i);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (VEC) {
      c[0].get(v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float x[1];
        c[i].get(x);
        v[i] = x[0];
      }
    }
  }
};

// This lane's chunks of N words, U of them at a time, those past the row's end as zeros.
template <typename IO, bool VEC, int R, int N> struct Words {
  static constexpr int U = R == 1 && sizeof(IO) == 2 ? 3 : 2;
  Chunk<IO, VEC> x[U][N];
  __device__ __forceinline__ void load(const FewArgs& a, int padded, const int (&words)[N], int c0) {
#pragma unroll
    for (int j = 0; j < N; j++) {
      const IO* p = (const IO*)a.w + words[j] * a.ld_w;
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int c = c0 + 256 * u + 8 * (threadIdx.x & 31);
        x[u][j].zero();
        if (c < padded) x[u][j].load(p + c, a.cols - c);
      }
    }
  }
  // sum[j][r] += over them of words j and row r of h [R][padded] in shared memory
  __device__ __forceinline__ void add(const float* h, int padded, int c0, float (&sum)[N][R]) const {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int c = min(c0 + 256 * u + 8 * (int)(threadIdx.x & 31), padded - 8);
      float v[N][8];
#pragma unroll
      for (int j = 0; j < N; j++) x[u][j].get(v[j]);
#pragma unroll
      for (int r = 0; r < R; r++) {
        const float4 h0 = *reinterpret_cast<const float4*>(h + r * padded + c),
                     h1 = *reinterpret_cast<const float4*>(h + r * padded + c + 4);
        const float hv[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
        for (int j = 0; j < N; j++)
#pragma unroll
          for (int i = 0; i < 8; i++) sum[j][r] = fmaf(v[j][i], hv[i], sum[j][r]);
      }
    }
  }
};

template <typename IO, bool VEC, int R>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) head_few_kernel(const FewArgs a) {
  extern __shared__ __align__(16) float h[];  // [R][padded], then the warps' sums
  __shared__ int kind[R];
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int padded = (a.cols + 7) / 8 * 8;
  // A warp's words lie together, as many as the others' or one more.
  const long long warps = (long long)gridDim.x * kWarps, me = (long long)blockIdx.x * kWarps + warp;
  const int from = (int)(me * a.vocab / warps), to = (int)((me + 1) * a.vocab / warps);
  // its first ones are on their way while the rows are looked at: W is nobody's result in this call
  Words<IO, VEC, R, kWords> batch;
  int words[kWords];
#pragma unroll
  for (int i = 0; i < kWords; i++) words[i] = max(min(from + i, to - 1), 0);
  batch.load(a, padded, words, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x < R) {  // which rows count: each block sees for itself
    const int t = threadIdx.x;
    int pos = kIgnored, word = kNoEntry;
    if (t < a.rows) {
      if (a.target) {
        const int64_t y = a.target[t];
        if (y != a.ignore) {
          pos = y >= 0 && y < a.vocab ? t : kBadRow;
          if (pos == t) word = (int)y;
        }
      } else {
        pos = a.valid[t] == 1 ? t : a.valid[t] == 2 ? kBadRow : kIgnored;
      }
      if (blockIdx.x == 0) {
        a.pos[t] = pos;
        if (a.target) a.idx[t] = word;
      }
    }
    kind[t] = pos;
    const bool bad = __any_sync((1u << R) - 1u, pos == kBadRow);
    if (blockIdx.x == 0 && t == 0) a.state->status = bad ? SSM_ERR_INVALID_ARG : SSM_OK;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * padded; i += kThreads) {
    const int r = i / padded, c = i - r * padded;
    h[i] = r < a.rows && kind[r] >= 0 && c < a.cols ? ld((const IO*)a.h + r * a.ld_h + c) : 0.0f;
  }
  __syncthreads();

  constexpr int W = kWords;      // words of a warp at a time
  constexpr int N = W * R;       // sums: number j * R + r is word j's of row r
  constexpr int kSame = 32 / N;  // lanes that end with the same one
  const int mine = lane / kSame;
  float top = -INFINITY, total = 0.0f;
  for (int w0 = from; w0 < to; w0 += W) {
    float d[W][R] = {}, s[N];
    for (int c0 = 0; c0 < padded; c0 += 256 * batch.U) {
      if (w0 > from || c0 > 0) batch.load(a, padded, words, c0);
      batch.add(h, padded, c0, d);
    }
#pragma unroll
    for (int i = 0; i < W; i++) {
      words[i] = min(w0 + W + i, to - 1);
#pragma unroll
      for (int r = 0; r < R; r++) s[i * R + r] = d[i][r];
    }
#pragma unroll
    for (int off = 16, n = N / 2; off > 0; off >>= 1, n >>= 1) {
      if (n == 0) s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
#pragma unroll
      for (int i = 0; i < n; i++) {
        const bool up = lane & off;
        const float give = up ? s[i] : s[i + n], keep = up ? s[i + n] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    }
    if (w0 + mine / R < to && lane % kSame == 0) {
      const float above = fmaxf(top, s[0]), base = above == -INFINITY ? 0.0f : above;
      total = total * ex2((top - base) * a.scale) + ex2((s[0] - base) * a.scale);
      top = above;
    }
  }
  // over the lanes of a row, then the warps
#pragma unroll
  for (int off = 16; off >= R * kSame; off >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, top, off), u = __shfl_xor_sync(0xffffffffu, total, off);
    const float above = fmaxf(top, t), base = above == -INFINITY ? 0.0f : above;
    total = total * ex2((top - base) * a.scale) + u * ex2((t - base) * a.scale);
    top = above;
  }
  // the entries' logits, from the last warp on, which has the fewest words
  for (long long i = warps - 1 - me; i < a.rows * a.entries; i += warps) {
    const int row = (int)(i / a.entries);
    const int word = kind[row] < 0 ? kNoEntry : a.target ? (int)a.target[row] : a.idx[i];
    if (word == kNoEntry) continue;
    const int one[1] = {word};
    Words<IO, VEC, 1, 1> x;
    float d[1][1] = {};
    for (int c0 = 0; c0 < padded; c0 += 256 * x.U) {
      x.load(a, padded, one, c0);
      x.add(h + row * padded, padded, c0, d);
    }
    float v = d[0][0];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0) a.zt[i] = v;
  }
  float2* sums = reinterpret_cast<float2*>(h + R * padded);
  if (mine < R && lane % kSame == 0) sums[warp * R + mine] = make_float2(top, total);
  __syncthreads();
  if (threadIdx.x < R && (int)threadIdx.x < a.rows) {
    top = -INFINITY, total = 0.0f;
    for (int w = 0; w < kWarps; w++) {
      const float2 v = sums[w * R + threadIdx.x];
      const float above = fmaxf(top, v.x), base = above == -INFINITY ? 0.0f : above;
      total = total * ex2((top - base) * a.scale) + v.y * ex2((v.x - base) * a.scale);
      top = above;
    }
    a.stats[blockIdx.x * a.ld_stats + threadIdx.x] = make_float2(top, total);
  }
}

int rows_of(long long rows) { return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8; }
size_t smem_of(int R, int cols) { return sizeof(float) * R * pad8(cols) + sizeof(float2) * kWarps * R; }

template <typename IO, bool VEC, int R>
cudaError_t launch(const FewArgs& a, int blocks, bool first, cudaStream_t st) {
  auto kernel = head_few_kernel<IO, VEC, R>;
  const size_t smem = smem_of(R, a.cols);
  if (smem > 40 * 1024) {
    // asked for once per device (the first 64 remember it)
    static std::atomic<unsigned long long> asked{0};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(asked.load(std::memory_order_relaxed) & bit)) {
      if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)kFewSmem))
        return e;
      asked.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = first ? 0 : 1;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, a);
  count_launches(1);
  return e;
}
template <typename IO, bool VEC>
cudaError_t launch(const FewArgs& a, int blocks, bool first, cudaStream_t st) {
  switch (rows_of(a.rows)) {
    case 1: return launch<IO, VEC, 1>(a, blocks, first, st);
    case 2: return launch<IO, VEC, 2>(a, blocks, first, st);
    case 4: return launch<float, VEC, 4>(a, blocks, first, st);  // fp32 only (head_few)
    default: return launch<float, VEC, 8>(a, blocks, first, st);
  }
}

}  // namespace

bool head_few(long long rows, int cols, int io) {
  return rows <= (io == SSM_F32 ? 8 : 2) && smem_of(rows_of(rows), cols) <= kFewSmem;
}
int head_few_blocks(int sms) { return kBlocksPerSm * sms; }

cudaError_t launch_head_few(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                            const void* h, long long ld_h, const void* w, long long ld_w, int* idx,
                            const HeadRows& r, float2* stats, float* zt, int sms, cudaStream_t st) {
  FewArgs a{h, ld_h, w, ld_w, target, valid, idx, r.state, r.pos, stats, zt, d.ignore_index,
            pad_rows(d.rows), (int)d.rows, d.cols, d.vocab, d.entries ? d.entries : 1,
            d.entries ? kLog2e / d.temperature : kLog2e};
  const size_t size = d.io == SSM_F32 ? 4 : 2;
  const bool vec = d.cols % 8 == 0 && ld_w % 8 == 0 && (uintptr_t)w % (8 * size) == 0;
  const int blocks = head_few_blocks(sms);
  const bool first = valid == nullptr;
  if (d.io == SSM_F32)
    return vec ? launch<float, true>(a, blocks, first, st) : launch<float, false>(a, blocks, first, st);
  return vec ? launch<__nv_bfloat16, true>(a, blocks, first, st) :
               launch<__nv_bfloat16, false>(a, blocks, first, st);
}

}  // namespace ssm
