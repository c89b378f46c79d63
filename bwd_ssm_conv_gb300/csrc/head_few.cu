// head_few.cu -- a few rows (tokens as they come): Z = h W^T with every row of W read once, by plain fp32
// arithmetic; the forward, and below it the backward.  W's bytes bound both; a tensor-core tile would be all
// but empty, its rows would have to be packed first, and fp32 W split into planes.  768 columns, 32768 words,
// us in a graph (GB300), with the kernel that joins the blocks' sums, and by the tensor cores (TC):
//              1 row     2     4     8    TC   W's bytes (the backward's: and d_W's)
//   bf16 fwd    16.1  20.0  25.3     -  23.7    7.4
//   bf16 bwd    33.4  40.7  52.2  99.5    58   14.9
//   fp32 fwd    23.6  25.4  29.8  41.3  87.5   14.9
//   fp32 bwd    45.8  48.4  55.5  97.5   166   29.8
// so that bf16 rows come here up to 2 in the forward and 4 in the backward, fp32 rows up to 8.
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
  const int* idx;  // a teacher's
  HeadState* state;
  int* pos;
  float2* stats;  // [blocks][ld_stats]
  float* zt;
  long long ignore, ld_stats;
  int rows, cols, vocab, entries;
  float scale;
  // backward
  const float* p;
  const float* lse;
  const float* d_loss;
  float tau, inv_tau, inv_tau_rest;
  void* d_w;
  int vec_w, groups;
  float* h_part;  // [blocks][rows][padded cols]
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

// Which rows count, and their target: each block sees for itself, the first one writes down the former.
template <int R>
__device__ __forceinline__ void look_at_rows(const FewArgs& a, int (&kind)[R], int (&target)[R]) {
  if (threadIdx.x >= R) return;
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
    if (blockIdx.x == 0) a.pos[t] = pos;
  }
  kind[t] = pos;
  target[t] = word;
  const bool bad = __any_sync((1u << R) - 1u, pos == kBadRow);
  if (blockIdx.x == 0 && t == 0) a.state->status = bad ? SSM_ERR_INVALID_ARG : SSM_OK;
}
// Their h as fp32, zeros for rows that do not count.
template <typename IO, int R>
__device__ __forceinline__ void stage_rows(const FewArgs& a, const int (&kind)[R], int padded, float* h) {
  for (int i = threadIdx.x; i < R * padded; i += kThreads) {
    const int r = i / padded, c = i - r * padded;
    h[i] = r < a.rows && kind[r] >= 0 && c < a.cols ? ld((const IO*)a.h + r * a.ld_h + c) : 0.0f;
  }
}
// Sums of N = kWords R over the lanes: each ends with one, number lane / kSame, which is word / R's of row % R.
template <int R> struct Spread {
  static constexpr int N = kWords * R, kSame = 32 / N;
  static __device__ __forceinline__ float over_lanes(const float (&d)[kWords][R]) {
    float s[N];
#pragma unroll
    for (int i = 0; i < kWords; i++)
#pragma unroll
      for (int r = 0; r < R; r++) s[i * R + r] = d[i][r];
#pragma unroll
    for (int off = 16, n = N / 2; off > 0; off >>= 1, n >>= 1) {
      if (n == 0) s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
#pragma unroll
      for (int i = 0; i < n; i++) {
        const bool up = threadIdx.x & off;
        const float give = up ? s[i] : s[i + n], keep = up ? s[i + n] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    }
    return s[0];
  }
};

template <typename IO, bool VEC, int R>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) head_few_kernel(const FewArgs a) {
  extern __shared__ __align__(16) float h[];  // [R][padded], then the warps' sums
  __shared__ int kind[R], target[R];
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
  look_at_rows<R>(a, kind, target);
  __syncthreads();
  stage_rows<IO, R>(a, kind, padded, h);
  __syncthreads();

  constexpr int kSame = Spread<R>::kSame;
  const int mine = lane / kSame;
  HeadSum sum{-INFINITY, 0.0f};
  for (int w0 = from; w0 < to; w0 += kWords) {
    float d[kWords][R] = {};
    for (int c0 = 0; c0 < padded; c0 += 256 * batch.U) {
      if (w0 > from || c0 > 0) batch.load(a, padded, words, c0);
      batch.add(h, padded, c0, d);
    }
#pragma unroll
    for (int i = 0; i < kWords; i++) words[i] = min(w0 + kWords + i, to - 1);
    const float z = Spread<R>::over_lanes(d);
    if (w0 + mine / R < to && lane % kSame == 0) sum = join(sum, {z, 0.0f}, a.scale);
  }
  // over the lanes of a row, then the warps
#pragma unroll
  for (int off = 16; off >= R * kSame; off >>= 1)
    sum = join(sum, {__shfl_xor_sync(0xffffffffu, sum.top, off), __shfl_xor_sync(0xffffffffu, sum.rest, off)},
               a.scale);
  // the entries' logits, from the last warp on, which has the fewest words
  for (long long i = warps - 1 - me; i < a.rows * a.entries; i += warps) {
    const int row = (int)(i / a.entries);
    const int word = kind[row] < 0 ? kNoEntry : a.target ? target[row] : a.idx[i];
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
  if (mine < R && lane % kSame == 0) sums[warp * R + mine] = make_float2(sum.top, sum.rest);
  __syncthreads();
  if (threadIdx.x < R && (int)threadIdx.x < a.rows) {
    sum = {-INFINITY, 0.0f};
    for (int w = 0; w < kWarps; w++) {
      const float2 v = sums[w * R + threadIdx.x];
      sum = join(sum, {v.x, v.y}, a.scale);
    }
    a.stats[blockIdx.x * a.ld_stats + threadIdx.x] = make_float2(sum.top, sum.rest);
  }
}

// The backward in one pass over W: a block takes 32 words at a time, a warp 4 of them for Z and from it
// G = (q - p) d_loss tau of every word and row; then a thread takes 8 columns of some of the words (read
// again, from the cache) and writes G^T h there, and adds G W to its sums of d_h, which lie in shared memory,
// one set for each group of threads that covers a row.  The groups' sums are added in order at the end, the
// blocks' by head_few_sum_kernel.  Reading W and writing d_W bound it.
template <typename IO, bool VEC, int R>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) head_few_bwd_kernel(const FewArgs a) {
  constexpr int kBatch = kWarps * kWords;
  extern __shared__ __align__(16) float h[];  // [R][padded], then the groups' sums [groups][R][padded]
  __shared__ int kind[R], target[R];
  __shared__ float G[kBatch][R];
  __shared__ float lse[R], up[R];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int padded = (a.cols + 7) / 8 * 8, chunks = padded / 8;
  const int from = (int)((long long)blockIdx.x * a.vocab / gridDim.x),
            to = (int)((long long)(blockIdx.x + 1) * a.vocab / gridDim.x);
  look_at_rows<R>(a, kind, target);
  __syncthreads();
  stage_rows<IO, R>(a, kind, padded, h);
  float* sums = h + R * padded;
  for (int i = threadIdx.x; i < a.groups * R * padded; i += kThreads) sums[i] = 0.0f;
  if (threadIdx.x < R) {
    const bool counts = kind[threadIdx.x] >= 0;
    lse[threadIdx.x] = counts ? a.lse[threadIdx.x] : 0.0f;
    up[threadIdx.x] = counts ? a.d_loss[threadIdx.x] * a.tau : 0.0f;
  }
  __syncthreads();
  const int mine = lane / Spread<R>::kSame, row = mine % R;
  const int* list = a.target ? &target[row] : a.idx + (long long)row * a.entries;
  const bool counts = row < a.rows && kind[row] >= 0;
  const int per = (kThreads / a.groups), group = threadIdx.x / per, first = threadIdx.x - group * per;
  for (int b0 = from; b0 < to; b0 += kBatch) {
    const int w0 = b0 + warp * kWords;
    if (w0 < to) {
      int words[kWords];
#pragma unroll
      for (int i = 0; i < kWords; i++) words[i] = min(w0 + i, to - 1);
      float d[kWords][R] = {};
      Words<IO, VEC, R, kWords> batch;
      for (int c0 = 0; c0 < padded; c0 += 256 * batch.U) {
        batch.load(a, padded, words, c0);
        batch.add(h, padded, c0, d);
      }
      const float z = Spread<R>::over_lanes(d);
      const int word = w0 + mine / R;
      if (lane % Spread<R>::kSame == 0) {
        float g = 0.0f;
        if (counts && word < to) {
          // at most 1; a NaN stays one
          const float x = fmaf(z, a.inv_tau, fmaf(z, a.inv_tau_rest, -lse[row])) * kLog2e;
          g = ex2(x > 0.0f ? 0.0f : x);
          int lo = 0, hi = a.entries;  // the list is in order
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (list[mid] < word) lo = mid + 1;
            else hi = mid;
          }
          float p = 0.0f;
          for (; lo < a.entries && list[lo] == word; lo++)
            p += a.p ? a.p[(long long)row * a.entries + lo] : 1.0f;
          g = (g - p) * up[row];
        }
        G[warp * kWords + mine / R][row] = g;
      }
    }
    __syncthreads();
    const int n = min(kBatch, to - b0);
    if (group < a.groups)
      for (int c = first; c < chunks; c += per) {
        constexpr int H = R > 4 ? 1 : R;  // rows whose h stays in registers
        float hv[H][8], dh[R][8] = {};
        const auto take = [&](int r, float (&x)[8]) {
          const float4 *p = reinterpret_cast<const float4*>(h + r * padded + 8 * c), u = p[0], t = p[1];
          x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = t.x, x[5] = t.y, x[6] = t.z, x[7] = t.w;
        };
        if (H == R)
#pragma unroll
          for (int r = 0; r < H; r++) take(r, hv[r]);
#pragma unroll(H == R ? 2 : 1)
        for (int w = group; w < n; w += a.groups) {
          Chunk<IO, VEC> x;
          x.zero();
          x.load((const IO*)a.w + (b0 + w) * a.ld_w + 8 * c, a.cols - 8 * c);
          float v[8], o[8] = {};
          x.get(v);
#pragma unroll
          for (int r = 0; r < R; r++) {
            const float g = G[w][r];
            if (H < R) take(r, hv[0]);
#pragma unroll
            for (int i = 0; i < 8; i++) {
              dh[r][i] = fmaf(g, v[i], dh[r][i]);
              o[i] = fmaf(g, hv[H < R ? 0 : r][i], o[i]);
            }
          }
          if (a.d_w) {
            IO* to_w = (IO*)a.d_w + (long long)(b0 + w) * a.cols + 8 * c;
            if (VEC && a.vec_w) {
              st_cols(to_w, o);
            } else {
#pragma unroll
              for (int i = 0; i < 8; i++)
                if (8 * c + i < a.cols) st(to_w + i, o[i]);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
          for (int i = 0; i < 8; i++) sums[(group * R + r) * padded + 8 * c + i] += dh[r][i];
      }
    __syncthreads();
  }
  if (!a.h_part) return;
  for (int i = threadIdx.x; i < a.rows * padded; i += kThreads) {
    float v = 0.0f;
    for (int g = 0; g < a.groups; g++) v += sums[g * R * padded + i];
    a.h_part[(long long)blockIdx.x * a.rows * padded + i] = v;
  }
}

// d_h of a row's 32 columns: 8 threads x 4 columns across, 32 slices of the blocks' sums, each in order, then
// the slices in order.
template <typename IO>
__global__ void __launch_bounds__(kThreads) head_few_sum_kernel(const float* part, int n, int rows,
                                                                int cols, int padded, const int* pos,
                                                                IO* d_h, long long ld) {
  __shared__ float s[32][33];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3, c = blockIdx.x * 32 + 4 * x, row = blockIdx.y;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < padded) {
#pragma unroll 10
    for (int b = y; b < n; b += 32) {
      const float4 p =
          *reinterpret_cast<const float4*>(part + ((long long)b * rows + row) * padded + c);
      v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
    }
  }
  s[y][4 * x] = v.x, s[y][4 * x + 1] = v.y, s[y][4 * x + 2] = v.z, s[y][4 * x + 3] = v.w;
  __syncthreads();
  const int col = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || col >= cols) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i++) t += s[i][threadIdx.x];
  const int at = pos[row];
  st(d_h + row * ld + col, at >= 0 ? t : at == kIgnored ? 0.0f : __uint_as_float(0x7fc00000u));
}

int rows_of(long long rows) { return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8; }
size_t smem_of(int R, int cols) { return sizeof(float) * R * pad8(cols) + sizeof(float2) * kWarps * R; }
// Groups of threads that each cover a row's chunks, in the backward.
int groups_of(int R, int cols) {
  const int chunks = pad8(cols) / 8;
  int groups = kThreads / chunks > 1 ? kThreads / chunks : 1;
  while (groups > 1 && sizeof(float) * (groups + 1) * R * pad8(cols) > kFewSmem) groups /= 2;
  return groups > 16 ? 16 : groups;
}
size_t smem_bwd_of(int R, int cols) {
  return sizeof(float) * (groups_of(R, cols) + 1) * R * pad8(cols);
}

template <auto Kernel> cudaError_t launch(const FewArgs& a, size_t smem, int blocks, bool first,
                                          cudaStream_t st) {
  if (smem > 40 * 1024) {
    // asked for once per device (the first 64 remember it)
    static std::atomic<unsigned long long> asked{0};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(asked.load(std::memory_order_relaxed) & bit)) {
      if (cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  const cudaError_t e = cudaLaunchKernelEx(&c, Kernel, a);
  count_launches(1);
  return e;
}
template <typename IO, bool VEC>
cudaError_t launch_fwd(const FewArgs& a, int blocks, bool first, cudaStream_t st) {
  const int R = rows_of(a.rows);
  const size_t smem = smem_of(R, a.cols);
  if (R == 1) return launch<head_few_kernel<IO, VEC, 1>>(a, smem, blocks, first, st);
  if constexpr (sizeof(IO) == 4) {
    if (R == 8) return launch<head_few_kernel<IO, VEC, 8>>(a, smem, blocks, first, st);
    if (R == 4) return launch<head_few_kernel<IO, VEC, 4>>(a, smem, blocks, first, st);
  }
  return launch<head_few_kernel<IO, VEC, 2>>(a, smem, blocks, first, st);
}
template <typename IO, bool VEC>
cudaError_t launch_bwd(const FewArgs& a, int blocks, bool first, cudaStream_t st) {
  const int R = rows_of(a.rows);
  const size_t smem = smem_bwd_of(R, a.cols);
  if (R == 1) return launch<head_few_bwd_kernel<IO, VEC, 1>>(a, smem, blocks, first, st);
  if (R == 2) return launch<head_few_bwd_kernel<IO, VEC, 2>>(a, smem, blocks, first, st);
  if constexpr (sizeof(IO) == 4)
    if (R == 8) return launch<head_few_bwd_kernel<IO, VEC, 8>>(a, smem, blocks, first, st);
  return launch<head_few_bwd_kernel<IO, VEC, 4>>(a, smem, blocks, first, st);
}
template <typename IO, bool VEC>
cudaError_t launch_all(const FewArgs& a, bool backward, int blocks, bool first, cudaStream_t st) {
  return backward ? launch_bwd<IO, VEC>(a, blocks, first, st) :
                    launch_fwd<IO, VEC>(a, blocks, first, st);
}
cudaError_t launch_few(const ssm_head_desc& d, const FewArgs& a, bool backward, int sms,
                       cudaStream_t st) {
  const size_t size = d.io == SSM_F32 ? 4 : 2;
  const bool vec = d.cols % 8 == 0 && a.ld_w % 8 == 0 && (uintptr_t)a.w % (8 * size) == 0;
  const int blocks = head_few_blocks(sms);
  const bool first = a.valid == nullptr;
  if (d.io == SSM_F32)
    return vec ? launch_all<float, true>(a, backward, blocks, first, st) :
                 launch_all<float, false>(a, backward, blocks, first, st);
  return vec ? launch_all<__nv_bfloat16, true>(a, backward, blocks, first, st) :
               launch_all<__nv_bfloat16, false>(a, backward, blocks, first, st);
}
FewArgs few_args(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid, const void* h,
                 long long ld_h, const void* w, long long ld_w, const HeadLists& lists,
                 const HeadRows& r) {
  FewArgs a{h, ld_h, w, ld_w, target, valid, lists.idx, r.state, r.pos};
  a.ignore = d.ignore_index;
  a.rows = (int)d.rows, a.cols = d.cols, a.vocab = d.vocab, a.entries = d.entries ? d.entries : 1;
  a.scale = d.entries ? kLog2e / d.temperature : kLog2e;
  a.p = lists.p;
  return a;
}

}  // namespace

bool head_few(long long rows, int cols, int io, bool backward) {
  const int R = rows_of(rows);
  return rows <= (io == SSM_F32 ? 8 : backward ? 4 : 2) &&
         (backward ? smem_bwd_of(R, cols) : smem_of(R, cols)) <= kFewSmem;
}
int head_few_blocks(int sms) { return kBlocksPerSm * sms; }

cudaError_t launch_head_few(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                            const void* h, long long ld_h, const void* w, long long ld_w,
                            const HeadLists& lists, const HeadRows& r, float2* stats, float* zt, int sms,
                            cudaStream_t st) {
  FewArgs a = few_args(d, target, valid, h, ld_h, w, ld_w, lists, r);
  a.stats = stats;
  a.zt = zt;
  a.ld_stats = pad_rows(d.rows);
  return launch_few(d, a, false, sms, st);
}

cudaError_t launch_head_few_bwd(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                                const void* h, long long ld_h, const void* w, long long ld_w,
                                const HeadLists& lists, const HeadRows& r, const float* lse,
                                const float* d_loss, float* h_part, void* d_h, long long ld_d_h,
                                void* d_w, int sms, cudaStream_t st) {
  FewArgs a = few_args(d, target, valid, h, ld_h, w, ld_w, lists, r);
  const size_t size = d.io == SSM_F32 ? 4 : 2;
  const double inv = d.entries ? 1.0 / d.temperature : 1.0;
  a.lse = lse, a.d_loss = d_loss;
  a.tau = d.entries ? d.temperature : 1.0f;
  a.inv_tau = (float)inv, a.inv_tau_rest = (float)(inv - a.inv_tau);
  a.h_part = h_part;
  a.d_w = d_w;
  a.vec_w = d.cols % 8 == 0 && (uintptr_t)d_w % (8 * size) == 0;
  a.groups = groups_of(rows_of(d.rows), d.cols);
  if (cudaError_t e = launch_few(d, a, true, sms, st)) return e;
  if (!d_h) return cudaSuccess;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((d.cols + 31) / 32, (unsigned)d.rows);
  c.blockDim = dim3(kThreads);
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  count_launches(1);
  const int n = head_few_blocks(sms), padded = pad8(d.cols);
  if (d.io == SSM_F32)
    return cudaLaunchKernelEx(&c, head_few_sum_kernel<float>, (const float*)h_part, n, a.rows, d.cols,
                              padded, (const int*)r.pos, (float*)d_h, ld_d_h);
  return cudaLaunchKernelEx(&c, head_few_sum_kernel<__nv_bfloat16>, (const float*)h_part, n, a.rows,
                            d.cols, padded, (const int*)r.pos, (__nv_bfloat16*)d_h, ld_d_h);
}

}  // namespace ssm
