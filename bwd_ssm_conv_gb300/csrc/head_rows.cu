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
// A warp per row.  An entry's place in the order is the number of smaller keys, counted: a key is the word
// and, behind it, the entry's number, so that no two are alike.  A logit's distance to the row's largest is
// formed before it is divided by tau: t / tau of 7e6 (7 at 1e-6) would be good to half a unit.  4096 rows of 64
// entries take 8 - 9 us (GB300), 333 of 17 4.3, most of it a start, an end and the chain of one row.
template <typename T>
__global__ void __launch_bounds__(kThreads) head_entries_kernel(const int64_t* t_idx, const T* t_logit,
                                                                long long rows, int k, int vocab,
                                                                float tau, int shift,
                                                                HeadLists lists, uint8_t* valid) {
  constexpr int N = SSM_MAX_HEAD_ENTRIES / 32, kBits = 7, kNone = SSM_MAX_HEAD_VOCAB << kBits;
  static_assert(SSM_MAX_HEAD_ENTRIES == 1 << kBits, "an entry's number in its key");
  __shared__ int4 keys[kThreads / 32][SSM_MAX_HEAD_ENTRIES / 4];
  __shared__ int parts[kThreads / 32][kHeadParts];
  early_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kThreads / 32) + warp;
  if (row >= rows) return;
  int* key = reinterpret_cast<int*>(keys[warp]);
  int* part = parts[warp];
  part[2 * lane] = part[2 * lane + 1] = 0;
  float t[N];
  int word[N], mine[N], place[N];
  bool bad = false, odd = false;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; j++) {
    const int i = lane + 32 * j;
    word[j] = -1;
    t[j] = -INFINITY;
    place[j] = 0;
    mine[j] = 0x7fffffff;
    if (i < k) {
      const int64_t w = t_idx[row * k + i];
      bad = bad || w >= vocab;
      if (w >= 0 && w < vocab) word[j] = (int)w;
      const float x = ld(t_logit + row * k + i);
      if (word[j] >= 0) t[j] = x;
      mine[j] = word[j] >= 0 ? word[j] << kBits | i : kNone + i;
      odd = odd || t[j] != t[j];
      top = fmaxf(top, t[j]);
    }
    key[i] = mine[j];
  }
  __syncwarp();
  // sorted, and counted by parts of the vocabulary
#pragma unroll
  for (int j = 0; j < N; j++)
    if (word[j] >= 0) atomicAdd(&part[word[j] >> shift], 1);
  for (int o = 0; o < (k + 3) / 4; o++) {
    const int4 x = keys[warp][o];
#pragma unroll
    for (int j = 0; j < N; j++)
      if (32 * j < k)
        place[j] += (x.x < mine[j]) + (x.y < mine[j]) + (x.z < mine[j]) + (x.w < mine[j]);
  }
  top = warp_max(top);
  bad = __any_sync(0xffffffffu, bad);
  odd = __any_sync(0xffffffffu, odd);  // a NaN is a loss of NaN, not an entry that is not there
  const bool some = odd || top > -INFINITY;
  float e[N], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    t[j] = (t[j] - top) / tau;
    e[j] = word[j] >= 0 && some ? expf(t[j]) : 0.0f;
    sum += e[j];
  }
  sum = warp_sum(sum);
  const float log_sum = logf(sum);
  float kn = 0.0f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    e[j] = some ? e[j] / sum : 0.0f;
    if (!(e[j] == 0.0f)) kn += e[j] * (t[j] - log_sum);
    if (lane + 32 * j < k) {
      lists.idx[row * k + place[j]] = word[j] >= 0 ? word[j] : kNoEntry;
      lists.p[row * k + place[j]] = e[j];
    }
  }
  kn = warp_sum(kn);
  __syncwarp();
  const int a = part[2 * lane], b = part[2 * lane + 1];
  int before = a + b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += o;
  }
  before -= a + b;
  reinterpret_cast<uchar2*>(lists.table + row * kHeadParts)[lane] =
      make_uchar2((unsigned char)before, (unsigned char)(before + a));
  if (lane == 0) {
    lists.known[row] = kn;
    valid[row] = bad ? 2 : some ? 1 : 0;
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

// ---- which rows count, and their copies --------------------------------------------------------------
// A block takes `per_block` rows.  It looks at every row, which costs less than a launch of its own for a
// count, so that it knows where its own go, and packs them, a warp per row; the last one also the rows
// of zeros past them.  The blocks behind copy W.  GB300, a start and an end of 4 us among them: 8192 x 768 bf16
// 13 us, 4096 x 768 8; 1021 x 515 fp32 with W of 10007 words into three planes 13.5 (52 MB, 8 at the rate of a copy).
constexpr int kRowThreads = 512;
struct RowsArgs {
  const int64_t* target;
  const uint8_t* valid;
  long long rows, ignore;
  int vocab, cols, padded_cols, per_block, row_blocks;
  float tau;
  const void* h;
  long long ld_h;
  const float* lse;
  const float* d_loss;
  const void* w;
  long long ld_w;
  __nv_bfloat16* w_out;
  int* idx;
  HeadRows r;
  HeadTiles tiles;
};
enum RowKind { kCounts, kNone, kBad };
// said: a row's target, or what `valid` holds of it.
__device__ __forceinline__ int kind_of(const RowsArgs& a, int64_t said) {
  if (a.target) return said == a.ignore ? kNone : said >= 0 && said < a.vocab ? kCounts : kBad;
  return said == 1 ? kCounts : said == 2 ? kBad : kNone;
}

template <typename IO, int PLANES, bool VEC_H, bool VEC_W>
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const RowsArgs a) {
  constexpr int kWarps = kRowThreads / 32;
  __shared__ int ints[3][kWarps];
  __shared__ float tops[kWarps];
  early_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const HeadRows& r = a.r;
  if ((int)blockIdx.x >= a.row_blocks) {
    const int chunks = a.padded_cols / 8, copiers = gridDim.x - a.row_blocks;
    const long long n = (long long)a.vocab * chunks, plane = (long long)a.vocab * a.padded_cols;
    for (long long i = (blockIdx.x - a.row_blocks) * (long long)kRowThreads + threadIdx.x;
         i < n; i += (long long)copiers * kRowThreads) {
      const int row = (int)(i / chunks), c = (int)(i - (long long)row * chunks) * 8;
      copy8<IO, PLANES, VEC_W>((const IO*)a.w + row * a.ld_w + c, a.cols - c,
                               a.w_out + (long long)row * a.padded_cols + c, plane);
    }
    wait_for_before();  // this one does not end ahead of the kernel before
    return;
  }
  wait_for_before();
  const long long first = (long long)blockIdx.x * a.per_block;
  int all = 0, before = 0, bad = 0;
  float top = 0.0f;
  constexpr int kBatch = 8;  // rows of a thread whose loads are in flight together
  for (long long t0 = threadIdx.x; t0 < a.rows; t0 += kBatch * kRowThreads) {
    int64_t said[kBatch];
    float g[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const long long t = t0 + i * kRowThreads < a.rows ? t0 + i * kRowThreads : t0;
      said[i] = a.target ? a.target[t] : a.valid[t];
      g[i] = a.d_loss ? fabsf(a.d_loss[t]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const long long t = t0 + i * kRowThreads;
      const int kind = t < a.rows ? kind_of(a, said[i]) : kNone;
      all += kind == kCounts;
      before += kind == kCounts && t < first;
      bad |= kind == kBad;
      if (kind == kCounts && g[i] < INFINITY) top = fmaxf(top, g[i]);
    }
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  top = warp_max(top);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) ints[0][warp] = all, ints[1][warp] = before, ints[2][warp] = bad, tops[warp] = top;
  __syncthreads();
  all = before = bad = 0, top = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    all += ints[0][w], before += ints[1][w], bad |= ints[2][w];
    top = fmaxf(top, tops[w]);
  }
  if (!(top > 0.0f)) top = 1.0f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    r.state->status = bad ? SSM_ERR_INVALID_ARG : SSM_OK;
    r.state->count = all;
    r.state->scale = top * a.tau;
    r.state->tile = head_tile(a.tiles, all > 0 ? all : 1);
  }
  // its own rows' places, kRowThreads of them at a time
  const int mine = before;
  for (int base = 0; base < a.per_block; base += kRowThreads) {
    const long long t = first + base + threadIdx.x;
    const bool own = base + (int)threadIdx.x < a.per_block && t < a.rows;
    const int64_t said = own ? (a.target ? a.target[t] : a.valid[t]) : 0;
    const int kind = own ? kind_of(a, said) : kNone;
    const unsigned votes = __ballot_sync(0xffffffffu, kind == kCounts);
    __syncthreads();  // the counts before may still be read
    if (lane == 0) ints[0][warp] = __popc(votes);
    __syncthreads();
    int at = before + __popc(votes & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      if (w < warp) at += ints[0][w];
      before += ints[0][w];
    }
    if (own) {
      r.pos[t] = kind == kCounts ? at : kind == kBad ? kBadRow : kIgnored;
      if (kind == kCounts) r.src[at] = (int)t;
      if (a.target) a.idx[t] = kind == kCounts ? (int)said : kNoEntry;
    }
  }
  __syncthreads();
  const bool last = (int)blockIdx.x == a.row_blocks - 1;
  const int padded = ((all > 0 ? all : 1) + 63) / 64 * 64, end = last ? padded : before;
  const long long plane = (a.rows + 63) / 64 * 64 * a.padded_cols;
  for (int row = mine + warp; row < end; row += kWarps) {
    __nv_bfloat16* out = r.h + (long long)row * a.padded_cols;
    const int from = row < before ? r.src[row] : -1;
    if (from < 0) {
      if (lane == 0) r.src[row] = -1;
      for (int c = 8 * lane; c < a.padded_cols; c += 256)
#pragma unroll
        for (int p = 0; p < PLANES; p++)
          *reinterpret_cast<uint4*>(out + p * plane + c) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const IO* x = (const IO*)a.h + from * a.ld_h;
#pragma unroll 4
      for (int c = 8 * lane; c < a.padded_cols; c += 256)
        copy8<IO, PLANES, VEC_H>(x + c, a.cols - c, out + c, plane);
    }
    if (a.lse && lane == 0) {
      r.rl[row] = from < 0 ? 0.0f : a.lse[from];
      r.rg[row] = from < 0 ? 0.0f : a.d_loss[from] / top;
    }
  }
}

// ---- loss -------------------------------------------------------------------------------------------
// A block of 1024 threads joins X rows' sums: 1024 / X slices of the tiles, each in order, then the slices,
// a few per lane of a row's warp in order, then a tree.  X is 32, or 4 where that many rows do not fill the
// SMs and the chain of loads is what counts.  4096 rows of 32768 words 9 us, 1021 of 10007 6 (GB300).
template <int X>
__global__ void __launch_bounds__(1024) head_loss_kernel(const float2* stats, int n_stats,
                                                         long long ld, const float* zt,
                                                         const float* p, const float* known,
                                                         long long rows, int entries, int vocab,
                                                         float scale, float tau, HeadRows r, float* loss,
                                                         float* lse) {
  constexpr int Y = 1024 / X;
  __shared__ float2 part[Y][X + 1];
  early_launch();
  wait_for_before();
  if (n_stats == 0) n_stats = 2 * ((vocab + r.state->tile - 1) / r.state->tile);
  const int x = threadIdx.x % X, y = threadIdx.x / X;
  const long long first = (long long)blockIdx.x * X;
  const int pos = first + x < rows ? r.pos[first + x] : kIgnored;
  HeadSum s{-INFINITY, 0.0f};
  if (pos >= 0)
#pragma unroll 4
    for (int i = y; i < n_stats; i += Y) {
      const float2 v = stats[i * ld + pos];
      s = join(s, {v.x, v.y}, scale);
    }
  part[y][x] = make_float2(s.top, s.rest);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = first + warp;  // a warp per row from here
  if (warp >= X || row >= rows) return;
  s = {-INFINITY, 0.0f};
#pragma unroll
  for (int i = lane; i < Y; i += 32) {
    const float2 v = part[i][warp];
    s = join(s, {v.x, v.y}, scale);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    // the same order in both lanes
    const HeadSum o{__shfl_xor_sync(0xffffffffu, s.top, off),
                    __shfl_xor_sync(0xffffffffu, s.rest, off)};
    s = lane & off ? join(o, s, scale) : join(s, o, scale);
  }
  const int at = r.pos[row];
  // loss from distances to the largest logit and the sum beside it: a loss near 0 keeps its digits
  const float log_sum = log1pf(s.rest);
  float l = 0.0f;
  if (at >= 0)
    for (int j = lane; j < entries; j += 32) {
      const float pj = p ? p[row * entries + j] : 1.0f;
      if (!(pj == 0.0f)) l += pj * ((s.top - zt[row * entries + j]) / tau + log_sum);
    }
  l = warp_sum(l);
  if (lane != 0) return;
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
#pragma unroll 8
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

struct FinishArgs {
  HeadRows r;
  const float* h_part;
  int h_splits;
  long long h_step, rows;
  void* d_h;
  long long ld_h;
  const float* w_part;
  int w_per, words, g_stages;
  long long w_step;
  void* d_w;        // the first of the words
  void* all_w;      // the whole of d_W where this is the call's last kernel
  long long n_w;
  int cols, padded_cols, last;
};
// A thread takes 8 columns of a row at a time, first of d_h's rows, then of d_W's.  Reads of the splits' sums
// bound it: 18 us for 8192 x 768 of two pieces (GB300).
template <typename IO, bool VEC_H, bool VEC_W>
__global__ void __launch_bounds__(kThreads) head_finish_kernel(const FinishArgs a) {
  early_launch();
  wait_for_before();
  const HeadState state = *a.r.state;
  const bool lost = a.last && state.status == SSM_ERR_TIMEOUT;
  const int chunks = a.padded_cols / 8;
  // without sums of d_h only rows without a loss are left to do, if there are any
  const long long n_h = a.d_h && (a.h_part || lost || state.count < a.rows) ? a.rows * chunks : 0,
                  n = n_h + (a.w_part ? (long long)a.words * chunks : 0),
                  stride = (long long)gridDim.x * kThreads,
                  first = blockIdx.x * (long long)kThreads + threadIdx.x;
  const int stages = ((state.count > 0 ? state.count : 1) + kHeadBlock - 1) / kHeadBlock * a.g_stages;
  for (long long i = first; i < n; i += stride) {
    float v[8];
    if (i < n_h) {
      const long long row = i / chunks;
      const int c = (int)(i - row * chunks) * 8, at = a.r.pos[row];
      if (at >= 0 && !lost) {
        if (!a.h_part) continue;
        sum8(a.h_part + (long long)at * a.padded_cols + c, a.h_splits, a.h_step, state.scale, v);
      }
      if (at < 0 || lost)
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = at == kIgnored && !lost ? 0.0f : nan_();
      put8<IO, VEC_H>((IO*)a.d_h + row * a.ld_h + c, a.cols - c, v);
    } else {
      const long long row = (i - n_h) / chunks;
      const int c = (int)(i - n_h - row * chunks) * 8;
      const int splits = (stages + a.w_per - 1) / a.w_per;  // those that had rows
      sum8(a.w_part + row * a.padded_cols + c, splits, a.w_step, state.scale, v);
      if (lost)
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = nan_();
      put8<IO, VEC_W>((IO*)a.d_w + row * a.cols + c, a.cols - c, v);
    }
  }
  if (lost && a.all_w)
    for (long long i = first; i < a.n_w; i += stride) st((IO*)a.all_w + i, nan_());
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
                                const HeadLists& lists, uint8_t* valid, cudaStream_t st) {
  const unsigned blocks = (unsigned)((d.rows + kThreads / 32 - 1) / (kThreads / 32));
  const int shift = head_part_shift(d.vocab);
  if (d.entry_io == SSM_F32)
    head_entries_kernel<<<blocks, kThreads, 0, st>>>(t_idx, (const float*)t_logit, d.rows, d.entries,
                                                     d.vocab, d.temperature, shift, lists, valid);
  else
    head_entries_kernel<<<blocks, kThreads, 0, st>>>(t_idx, (const __nv_bfloat16*)t_logit, d.rows,
                                                     d.entries, d.vocab, d.temperature, shift, lists,
                                                     valid);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_head_rows(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                             const void* h, long long ld_h, const float* lse, const float* d_loss,
                             const void* w, long long ld_w, int* idx, const HeadRows& r,
                             __nv_bfloat16* w_out, const HeadTiles& tiles, int sms, cudaStream_t st) {
  RowsArgs a{target, valid, d.rows, d.ignore_index, d.vocab, d.cols, pad8(d.cols)};
  // at most 256 blocks, as each looks at every row (8192 x 512 fp32: 128 13.5 us, 256 12.3, 512 16.6)
  const long long per = (d.rows + 255) / 256;
  a.per_block = per < kRowThreads / 32 ? kRowThreads / 32 : (int)per;
  a.row_blocks = (int)((d.rows + a.per_block - 1) / a.per_block);
  a.tau = d.entries ? d.temperature : 1.0f;
  a.h = h, a.ld_h = ld_h, a.lse = lse, a.d_loss = d_loss;
  a.w = w, a.ld_w = ld_w, a.w_out = w_out;
  a.idx = idx, a.r = r, a.tiles = tiles;
  const long long chunks = (long long)d.vocab * (a.padded_cols / 8);
  const long long copiers = w_out ? at_most((chunks + kRowThreads - 1) / kRowThreads, sms) : 0;
  const bool vec_h = vec_rows(h, ld_h, d.cols, d.io), vec_w = vec_rows(w, ld_w, d.cols, d.io);
  void (*kernel)(RowsArgs);
  if (d.io == SSM_F32)
    kernel = vec_h ? (vec_w ? head_rows_kernel<float, 3, true, true> :
                              head_rows_kernel<float, 3, true, false>) :
                     (vec_w ? head_rows_kernel<float, 3, false, true> :
                              head_rows_kernel<float, 3, false, false>);
  else  // W that can be copied in chunks is not copied
    kernel = vec_h ? head_rows_kernel<__nv_bfloat16, 1, true, false> :
                     head_rows_kernel<__nv_bfloat16, 1, false, false>;
  if (valid) return go(kernel, a.row_blocks + copiers, kRowThreads, st, a);
  kernel<<<(unsigned)(a.row_blocks + copiers), kRowThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_head_loss(const ssm_head_desc& d, const float2* stats, int n_stats,
                             const float* zt, const HeadLists& lists, const HeadRows& r,
                             float* loss, float* lse, int sms,
                             cudaStream_t st) {
  const float tau = d.entries ? d.temperature : 1.0f;
  const int x = d.rows > 4 * sms ? 32 : 4;
  return go(x == 32 ? head_loss_kernel<32> : head_loss_kernel<4>, (d.rows + x - 1) / x, 1024, st, stats,
            n_stats, pad_rows(d.rows), zt, lists.p, lists.known, d.rows, d.entries ? d.entries : 1,
            d.vocab, kLog2e / tau, tau, r, loss, lse);
}

cudaError_t launch_head_finish(const ssm_head_desc& d, const HeadRows& r, const float* h_part,
                               int h_splits, void* d_h, long long ld_d_h, const float* w_part,
                               int w_per, int piece, void* d_w, int v0, int n, bool last, int sms,
                               cudaStream_t st) {
  FinishArgs a{r};
  const size_t size = d.io == SSM_F32 ? 4 : 2;
  a.cols = d.cols, a.padded_cols = pad8(d.cols), a.last = last;
  a.h_part = h_part, a.h_splits = h_splits, a.h_step = pad_rows(d.rows) * a.padded_cols;
  a.rows = d.rows, a.d_h = d_h, a.ld_h = ld_d_h;
  a.g_stages = head_g_terms(d) == 2 ? 2 : 1;
  a.w_part = w_part, a.w_per = w_per, a.words = n, a.w_step = (long long)piece * a.padded_cols;
  a.d_w = (char*)d_w + (size_t)v0 * d.cols * size;
  a.all_w = d_w, a.n_w = (long long)d.vocab * d.cols;
  const long long work = ((d_h ? d.rows : 0) + (w_part ? n : 0)) * (a.padded_cols / 8);
  const long long blocks = at_most(work ? (work + kThreads - 1) / kThreads : sms, sms);
  const bool vec_h = vec_rows(d_h, ld_d_h, d.cols, d.io), vec_w = vec_rows(d_w, d.cols, d.cols, d.io);
  void (*kernel)(FinishArgs);
#define SSM_PICK(IO)                                                                             \
  vec_h ? (vec_w ? head_finish_kernel<IO, true, true> : head_finish_kernel<IO, true, false>) :   \
          (vec_w ? head_finish_kernel<IO, false, true> : head_finish_kernel<IO, false, false>)
  if (d.io == SSM_F32) kernel = SSM_PICK(float);
  else kernel = SSM_PICK(__nv_bfloat16);
#undef SSM_PICK
  return go(kernel, blocks, kThreads, st, a);
}

}  // namespace ssm
