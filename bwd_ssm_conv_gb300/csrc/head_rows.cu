// head_rows.cu -- the head's loss: what happens to rows before and after the products of head_tc.cu.
// Every kernel here reads and writes its operands once; all but the first of a call are set up while the
// kernel before them runs.
#include "head.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void early_launch() {
  asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void wait_for_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float nan_() { return __uint_as_float(0x7fc00000u); }

// ---- a teacher's entries ------------------------------------------------------------------------
// A warp per row.  An entry's place is the number of entries before it, counted.
template <typename T>
__global__ void __launch_bounds__(kThreads) head_entries_kernel(const int64_t* t_idx, const T* t_logit,
                                                                long long rows, int k, int vocab,
                                                                float tau, int* idx, float* p,
                                                                float* known, uint8_t* valid) {
  constexpr int N = SSM_MAX_HEAD_ENTRIES / 32;
  __shared__ int keys[kThreads / 32][SSM_MAX_HEAD_ENTRIES];
  early_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kThreads / 32) + warp;
  if (row >= rows) return;
  int* key = keys[warp];
  float t[N];
  bool here[N], bad = false, odd = false;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; j++) {
    const int i = lane + 32 * j;
    here[j] = false;
    t[j] = -INFINITY;
    if (i < k) {
      const int64_t word = t_idx[row * k + i];
      here[j] = word >= 0 && word < vocab;
      bad = bad || word >= vocab;
      if (here[j]) t[j] = ld(t_logit + row * k + i) / tau;
      key[i] = here[j] ? (int)word : kNoEntry;
      odd = odd || t[j] != t[j];
      top = fmaxf(top, t[j]);
    }
  }
  __syncwarp();
  top = warp_max(top);
  bad = __any_sync(0xffffffffu, bad);
  odd = __any_sync(0xffffffffu, odd);  // a NaN is a loss of NaN, not an entry that is not there
  const bool some = odd || top > -INFINITY;
  float e[N], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    e[j] = here[j] && some ? expf(t[j] - top) : 0.0f;
    sum += e[j];
  }
  sum = warp_sum(sum);
  const float log_sum = logf(sum);
  float kn = 0.0f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    e[j] = some ? e[j] / sum : 0.0f;
    if (!(e[j] == 0.0f)) kn += e[j] * (t[j] - top - log_sum);
    const int i = lane + 32 * j;
    if (i < k) {
      const int mine = key[i];
      int place = 0;
      for (int o = 0; o < k; o++) place += key[o] < mine || (key[o] == mine && o < i);
      idx[row * k + place] = mine;
      p[row * k + place] = e[j];
    }
  }
  kn = warp_sum(kn);
  if (lane == 0) {
    known[row] = kn;
    valid[row] = bad ? 2 : some ? 1 : 0;
  }
}

// ---- which rows count -----------------------------------------------------------------------------
// One block steps over the rows, 4 per thread, and numbers those that have a loss; in the backward it
// also finds the largest |d_loss| of theirs.
constexpr int kBeginThreads = 1024, kBeginRows = 4;
__global__ void __launch_bounds__(kBeginThreads) head_begin_kernel(const int64_t* target,
                                                                   const uint8_t* valid,
                                                                   long long rows, int vocab,
                                                                   long long ignore, float tau,
                                                                   const float* d_loss, int* idx,
                                                                   HeadRows r) {
  __shared__ int sums[2][32];
  __shared__ float tops[32];
  early_launch();
  wait_for_before();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int total = 0, half = 0;
  bool bad = false;
  float top = 0.0f;
  for (long long base = 0; base < rows; base += kBeginThreads * kBeginRows, half ^= 1) {
    const long long t0 = base + (long long)threadIdx.x * kBeginRows;
    int pos[kBeginRows], n = 0;
#pragma unroll
    for (int i = 0; i < kBeginRows; i++) {
      pos[i] = kIgnored;
      if (t0 + i >= rows) continue;
      if (target) {
        const int64_t y = target[t0 + i];
        const bool in = y >= 0 && y < vocab;
        if (y != ignore) pos[i] = in ? 0 : kBadRow;
        idx[t0 + i] = pos[i] == 0 ? (int)y : kNoEntry;
      } else {
        const int v = valid[t0 + i];
        pos[i] = v == 1 ? 0 : v == 2 ? kBadRow : kIgnored;
      }
      n += pos[i] == 0;
      bad = bad || pos[i] == kBadRow;
      if (pos[i] == 0 && d_loss) {
        const float g = fabsf(d_loss[t0 + i]);
        if (g < INFINITY) top = fmaxf(top, g);
      }
    }
    int before = n;  // within the warp, then the block
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += o;
    }
    if (lane == 31) sums[half][warp] = before;
    before -= n;
    __syncthreads();
    int all = sums[half][lane], upto = all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += o;
    }
    before += __shfl_sync(0xffffffffu, upto - all, warp) + total;
    total += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
    for (int i = 0; i < kBeginRows; i++)
      if (t0 + i < rows) {
        if (pos[i] == 0) {
          pos[i] = before++;
          r.src[pos[i]] = (int)(t0 + i);
        }
        r.pos[t0 + i] = pos[i];
      }
  }
  const int padded = ((total > 0 ? total : 1) + 63) / 64 * 64;
  for (int i = total + threadIdx.x; i < padded; i += kBeginThreads) r.src[i] = -1;
  top = warp_max(top);
  if (lane == 0) tops[warp] = top;
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    top = warp_max(tops[lane]);
    if (lane == 0) {
      r.state->status = bad ? SSM_ERR_INVALID_ARG : SSM_OK;
      r.state->count = total;
      if (!(top > 0.0f)) top = 1.0f;
      r.state->g_top = top;
      r.state->scale = top * tau;
    }
  }
}

// ---- rows as the products read them ---------------------------------------------------------------
// A value as PLANES bf16 terms, each rounded from what the ones before leave: three hold all 24 bits.
// What is not finite stays so in the first.
template <int PLANES> __device__ __forceinline__ void split(float v, float (&term)[PLANES]) {
  if constexpr (PLANES == 1) {
    term[0] = v;
  } else {
    const bool finite = fabsf(v) < INFINITY;
    term[0] = __bfloat162float(__float2bfloat16_rn(v));
    if (finite && !(fabsf(term[0]) < INFINITY))  // rounded past the largest bf16 number
      term[0] = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    const float rest = finite ? v - term[0] : 0.0f;
    term[1] = __bfloat162float(__float2bfloat16_rn(rest));
    term[2] = rest - term[1];
  }
}
// 8 columns of a row of x to their place in each plane.
template <typename IO, int PLANES, bool VEC>
__device__ __forceinline__ void copy8(const IO* x, int left, __nv_bfloat16* out, long long plane) {
  if constexpr (PLANES == 1 && VEC) {
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(x);
  } else {
    float v[8], term[8][PLANES];
    if constexpr (VEC) {
      Cols<IO, 8> c;
      c.load(x);
      c.get(v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = i < left ? ld(x + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) split<PLANES>(v[i], term[i]);
#pragma unroll
    for (int p = 0; p < PLANES; p++) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; i++) w[i] = bf16x2_rn(term[2 * i][p], term[2 * i + 1][p]);
      *reinterpret_cast<uint4*>(out + p * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// A warp per packed row, or per row of zeros past them.
template <typename IO, int PLANES, bool VEC>
__global__ void __launch_bounds__(kThreads) head_pack_kernel(const IO* h, long long ld_h, int cols,
                                                             int padded_cols, long long plane,
                                                             const float* lse, const float* d_loss,
                                                             HeadRows r) {
  early_launch();
  wait_for_before();
  const int count = r.state->count, lane = threadIdx.x & 31;
  const int rows = ((count > 0 ? count : 1) + 63) / 64 * 64;
  const int step = gridDim.x * (kThreads / 32);
  for (int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); row < rows; row += step) {
    __nv_bfloat16* out = r.h + (long long)row * padded_cols;
    const int from = row < count ? r.src[row] : -1;
    if (from < 0) {
      for (int c = 8 * lane; c < padded_cols; c += 256)
#pragma unroll
        for (int p = 0; p < PLANES; p++)
          *reinterpret_cast<uint4*>(out + p * plane + c) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const IO* x = h + from * ld_h;
#pragma unroll 4
      for (int c = 8 * lane; c < padded_cols; c += 256)
        copy8<IO, PLANES, VEC>(x + c, cols - c, out + c, plane);
    }
    if (lse && lane == 0) {
      r.rl[row] = from < 0 ? 0.0f : lse[from] * kLog2e;
      r.rg[row] = from < 0 ? 0.0f : d_loss[from] / r.state->g_top;
    }
  }
}

// A thread copies 8 columns of a row of W at a time.
template <typename IO, int PLANES, bool VEC>
__global__ void __launch_bounds__(kThreads) head_copy_w_kernel(const IO* w, long long ld_w, int rows,
                                                               int cols, int padded_cols,
                                                               __nv_bfloat16* out) {
  early_launch();
  const int chunks = padded_cols / 8;
  const long long n = (long long)rows * chunks, plane = (long long)rows * padded_cols;
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const int row = (int)(i / chunks), c = (int)(i - (long long)row * chunks) * 8;
    copy8<IO, PLANES, VEC>(w + row * ld_w + c, cols - c, out + (long long)row * padded_cols + c,
                           plane);
  }
  wait_for_before();  // this one does not end ahead of the kernel before
}

// ---- loss -------------------------------------------------------------------------------------------
struct Sum {  // of the exponentials 2^((z - top) scale)
  float top, sum;
};
__device__ __forceinline__ Sum join(const Sum& a, const Sum& b, float scale) {
  const float top = fmaxf(a.top, b.top), at = top == -INFINITY ? 0.0f : top;
  return {top, a.sum * ex2((a.top - at) * scale) + b.sum * ex2((b.top - at) * scale)};
}
// A block joins 32 rows' sums: 32 slices of the tiles, each in order, then the slices in a tree.
__global__ void __launch_bounds__(1024) head_loss_kernel(const float2* stats, int n_stats,
                                                         long long ld, const float* zt,
                                                         const float* p, const float* known,
                                                         long long rows, int entries, float scale,
                                                         float tau, HeadRows r, float* loss,
                                                         float* lse) {
  __shared__ float2 part[32][33];
  early_launch();
  wait_for_before();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long long first = (long long)blockIdx.x * 32;
  const int pos = first + x < rows ? r.pos[first + x] : kIgnored;
  Sum s{-INFINITY, 0.0f};
  if (pos >= 0)
#pragma unroll 4
    for (int i = y; i < n_stats; i += 32) {
      const float2 v = stats[i * ld + pos];
      s = join(s, {v.x, v.y}, scale);
    }
  part[y][x] = make_float2(s.top, s.sum);
  __syncthreads();
  const long long row = first + y;  // a warp per row from here
  if (row >= rows) return;
  const float2 v = part[x][y];
  s = {v.x, v.y};
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    // the same order in both lanes
    const Sum o{__shfl_xor_sync(0xffffffffu, s.top, off), __shfl_xor_sync(0xffffffffu, s.sum, off)};
    s = x & off ? join(o, s, scale) : join(s, o, scale);
  }
  const int at = r.pos[row];
  // loss from distances to the largest logit: a loss near 0 keeps its digits
  const float log_sum = logf(s.sum);
  float l = 0.0f;
  if (at >= 0)
    for (int j = x; j < entries; j += 32) {
      const float pj = p ? p[row * entries + j] : 1.0f;
      if (!(pj == 0.0f)) l += pj * ((s.top - zt[row * entries + j]) / tau + log_sum);
    }
  l = warp_sum(l);
  if (x != 0) return;
  float whole = s.top / tau + log_sum;
  if (known && at >= 0) l = (l + known[row]) * (tau * tau);
  if (at < 0) l = whole = 0.0f;
  if (at == kBadRow || r.state->status == SSM_ERR_TIMEOUT) l = whole = nan_();
  loss[row] = l;
  if (lse) lse[row] = whole;
}

// ---- gradients ----------------------------------------------------------------------------------------
// 8 columns at a time: the splits' sums in order, times what G lacks.
__device__ __forceinline__ void sum8(const float* part, int splits, long long step, float scale,
                                     float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < splits; s++) {
    Cols<float, 8> c;
    c.load(part + s * step);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] += c.a[i];
  }
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] *= scale;
}
template <typename IO, bool VEC>
__device__ __forceinline__ void put8(IO* out, int left, const float (&v)[8]) {
  if constexpr (VEC) {
    st_cols(out, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < left) st(out + i, v[i]);
  }
}

template <typename IO, bool VEC>
__global__ void __launch_bounds__(kThreads) head_finish_kernel(const float* part, int splits,
                                                               long long step, long long rows,
                                                               int cols, int padded_cols, HeadRows r,
                                                               IO* d_h, long long ld, IO* d_w,
                                                               long long n_w) {
  early_launch();
  wait_for_before();
  const bool lost = r.state->status == SSM_ERR_TIMEOUT;
  const float scale = r.state->scale;
  const int chunks = padded_cols / 8;
  const long long n = rows * chunks, stride = (long long)gridDim.x * kThreads,
                  mine = blockIdx.x * (long long)kThreads + threadIdx.x;
  if (d_h)
    for (long long i = mine; i < n; i += stride) {
      const long long row = i / chunks;
      const int c = (int)(i - row * chunks) * 8, at = r.pos[row];
      float v[8];
      if (at >= 0) sum8(part + (long long)at * padded_cols + c, splits, step, scale, v);
      if (at < 0 || lost)
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = at == kIgnored && !lost ? 0.0f : nan_();
      put8<IO, VEC>(d_h + row * ld + c, cols - c, v);
    }
  if (lost && d_w)
    for (long long i = mine; i < n_w; i += stride) st(d_w + i, nan_());
}

template <typename IO, bool VEC>
__global__ void __launch_bounds__(kThreads) head_sum_w_kernel(const float* part, int per_split,
                                                              long long step, int rows, int cols,
                                                              int padded_cols, HeadRows r, IO* d_w) {
  early_launch();
  wait_for_before();
  const float scale = r.state->scale;
  const int stages = ((r.state->count > 0 ? r.state->count : 1) + kHeadBlock - 1) / kHeadBlock;
  const int splits = (stages + per_split - 1) / per_split;  // those that had rows
  const int chunks = padded_cols / 8;
  const long long n = (long long)rows * chunks;
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const int row = (int)(i / chunks), c = (int)(i - (long long)row * chunks) * 8;
    float v[8];
    sum8(part + (long long)row * padded_cols + c, splits, step, scale, v);
    put8<IO, VEC>(d_w + (long long)row * cols + c, cols - c, v);
  }
}

// A launch that is set up while the kernel before it runs.
template <typename... P, typename... A>
cudaError_t go(void (*kernel)(P...), long long blocks, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3(threads);
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
  count_launches(1);
  return e;
}
long long at_most(long long blocks, int sms) {
  const long long most = 16LL * sms;
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}
bool vec_rows(const void* p, long long ld, int cols, int io) {
  const size_t size = io == SSM_F32 ? 4 : 2;
  return cols % 8 == 0 && ld % 8 == 0 && (uintptr_t)p % (8 * size) == 0;
}

}  // namespace

cudaError_t launch_head_entries(const ssm_head_desc& d, const int64_t* t_idx, const void* t_logit,
                                int* idx, float* p, float* known, uint8_t* valid, cudaStream_t st) {
  const unsigned blocks = (unsigned)((d.rows + kThreads / 32 - 1) / (kThreads / 32));
  if (d.entry_io == SSM_F32)
    head_entries_kernel<<<blocks, kThreads, 0, st>>>(t_idx, (const float*)t_logit, d.rows, d.entries,
                                                     d.vocab, d.temperature, idx, p, known, valid);
  else
    head_entries_kernel<<<blocks, kThreads, 0, st>>>(t_idx, (const __nv_bfloat16*)t_logit, d.rows,
                                                     d.entries, d.vocab, d.temperature, idx, p,
                                                     known, valid);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_head_begin(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                              const float* d_loss, int* idx, const HeadRows& r, bool first,
                              cudaStream_t st) {
  const float tau = d.entries ? d.temperature : 1.0f;
  if (!first)
    return go(head_begin_kernel, 1, kBeginThreads, st, target, valid, d.rows, d.vocab,
              d.ignore_index, tau, d_loss, idx, r);
  head_begin_kernel<<<1, kBeginThreads, 0, st>>>(target, valid, d.rows, d.vocab, d.ignore_index, tau,
                                                 d_loss, idx, r);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_head_pack(const ssm_head_desc& d, const void* h, long long ld_h,
                             const float* lse, const float* d_loss, const HeadRows& r, int sms,
                             cudaStream_t st) {
  const long long rows = pad_rows(d.rows), blocks = at_most(rows / (kThreads / 32), sms);
  const int padded = pad8(d.cols);
  const bool vec = vec_rows(h, ld_h, d.cols, d.io);
  if (d.io == SSM_F32)
    return go(vec ? head_pack_kernel<float, 3, true> : head_pack_kernel<float, 3, false>, blocks,
              kThreads, st, (const float*)h, ld_h, d.cols, padded, rows * padded, lse, d_loss, r);
  return go(vec ? head_pack_kernel<__nv_bfloat16, 1, true> : head_pack_kernel<__nv_bfloat16, 1, false>,
            blocks, kThreads, st, (const __nv_bfloat16*)h, ld_h, d.cols, padded, rows * padded, lse,
            d_loss, r);
}

cudaError_t launch_head_copy_w(const ssm_head_desc& d, const void* w, long long ld_w,
                               __nv_bfloat16* out, int sms, cudaStream_t st) {
  const int padded = pad8(d.cols);
  const long long blocks = at_most(((long long)d.vocab * (padded / 8) + kThreads - 1) / kThreads, sms);
  const bool vec = vec_rows(w, ld_w, d.cols, d.io);
  if (d.io == SSM_F32)
    return go(vec ? head_copy_w_kernel<float, 3, true> : head_copy_w_kernel<float, 3, false>, blocks,
              kThreads, st, (const float*)w, ld_w, d.vocab, d.cols, padded, out);
  return go(vec ? head_copy_w_kernel<__nv_bfloat16, 1, true> :
                  head_copy_w_kernel<__nv_bfloat16, 1, false>,
            blocks, kThreads, st, (const __nv_bfloat16*)w, ld_w, d.vocab, d.cols, padded, out);
}

cudaError_t launch_head_loss(const ssm_head_desc& d, const float2* stats, int n_stats,
                             const float* zt, const float* p, const float* known,
                             const HeadRows& r, float* loss, float* lse, cudaStream_t st) {
  const float tau = d.entries ? d.temperature : 1.0f;
  return go(head_loss_kernel, (d.rows + 31) / 32, 1024, st, stats, n_stats, pad_rows(d.rows), zt, p,
            known, d.rows, d.entries ? d.entries : 1, kLog2e / tau, tau, r, loss, lse);
}

cudaError_t launch_head_finish(const ssm_head_desc& d, const float* part, int splits,
                               const HeadRows& r, void* d_h, long long ld_d_h, void* d_w, int sms,
                               cudaStream_t st) {
  const int padded = pad8(d.cols);
  const long long step = pad_rows(d.rows) * padded, n_w = (long long)d.vocab * d.cols;
  const long long blocks = at_most(d_h ? (d.rows * (padded / 8) + kThreads - 1) / kThreads : sms, sms);
  const bool vec = vec_rows(d_h, ld_d_h, d.cols, d.io);
  if (d.io == SSM_F32)
    return go(vec ? head_finish_kernel<float, true> : head_finish_kernel<float, false>, blocks,
              kThreads, st, part, splits, step, d.rows, d.cols, padded, r, (float*)d_h, ld_d_h,
              (float*)d_w, n_w);
  return go(vec ? head_finish_kernel<__nv_bfloat16, true> : head_finish_kernel<__nv_bfloat16, false>,
            blocks, kThreads, st, part, splits, step, d.rows, d.cols, padded, r,
            (__nv_bfloat16*)d_h, ld_d_h, (__nv_bfloat16*)d_w, n_w);
}

cudaError_t launch_head_sum_w(const ssm_head_desc& d, const float* part, int per_split, int n_part,
                              const HeadRows& r, void* d_w, int v0, int n, int sms,
                              cudaStream_t st) {
  const int padded = pad8(d.cols);
  const long long step = (long long)n_part * padded,
                  blocks = at_most(((long long)n * (padded / 8) + kThreads - 1) / kThreads, sms);
  const long long at = (long long)v0 * d.cols;
  const bool vec = vec_rows(d_w, d.cols, d.cols, d.io);
  if (d.io == SSM_F32)
    return go(vec ? head_sum_w_kernel<float, true> : head_sum_w_kernel<float, false>, blocks, kThreads,
              st, part, per_split, step, n, d.cols, padded, r, (float*)d_w + at);
  return go(vec ? head_sum_w_kernel<__nv_bfloat16, true> : head_sum_w_kernel<__nv_bfloat16, false>,
            blocks, kThreads, st, part, per_split, step, n, d.cols, padded, r,
            (__nv_bfloat16*)d_w + at);
}

}  // namespace ssm
