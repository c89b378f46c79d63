// head_tc.cu -- the head's products on the tensor cores.  One kernel, three uses:
//   kLogits  Z = h W^T, of which a tile leaves only what its row needs: the maximum, the sum of the
//            exponentials beside it, and the logits of the row's entries
//   kGrad    Z again, turned into G = (softmax - p) d_loss, a piece of the vocabulary at a time
//   kOut     d_h = G W (sums over the vocabulary), d_W = G^T h (sums over the rows)
//
// A pair of CTAs (tcgen05 cta_group::2) forms a 256 x 256 tile, 64 steps of the sum per stage: each CTA
// holds 128 rows of A and 128 columns of B.  An operand is staged as it lies: [row][64 of the sum]
// (K-major) or [64 of the sum][64 columns] slabs (MN-major), both from 64 x 64 boxes with the 128-byte
// swizzle, so that neither G nor W nor h is ever transposed.  Pairs step over the tiles; two
// accumulators in tensor memory (four where tiles are 128 columns wide) take turns, so that a tile's results
// are taken out under the products of the next.
//   warp 0      one thread copies the tiles by TMA (past the ends they read as 0)
//   warp 1      one thread of the first CTA issues the MMAs; the second CTA's passes on that its copies
//               have landed
//   warps 4-11  take the results out: thread = row, 128 of its columns each
// fp32 operands are three bf16 planes each, staged one after the other (1, 0, 2) in slots of their own:
// six products per step over 64 of the sum (of planes 1 1, 1 0, 0 1, 2 0, 0 2, 0 0; the rest is below 2^-24
// of a product), whose slots come free in between, so that a slot's next copy has more than a step's time.
// The tensor cores truncate when they add, by the size of the sum: small products come before the large one,
// and the sums are taken out every 64 columns and added in registers.
//
// GB300, us of a launch by itself and its rate (cuBLAS's bf16 product of 8192^3 on this GPU: 1908 TFLOP/s):
//                                  kLogits        kGrad          kOut
//   7370 x 768, 50000 words bf16   292  1940      2 x 164  1730  2 x 333  1700
//   16384 x 1024, 32768 bf16       537  2050      2 x 298  1850  2 x 593  1850
//   3891 x 768, 32768 bf16         116  1690      132      1480  220      1780
//   684 x 515, 10007 fp32           40  1030       50       850   87       970  (six products counted)
//   300 x 256, 5003 fp32            14   330       18       260   18       510
// G in two terms (SSM_HEAD_FINE_G): a stage for each, the smaller one first, with the other operand copied again;
// the backward of 8192 x 768 over 50000 words 1.08 -> 2.13 ms, of 16384 x 1024 over 32768 1.86 -> 3.59.
// The tensor cores bound it, back to back the power limit (1500 - 1650 TFLOP/s).  kGrad's stores are what it is
// slower by (with fp32 few products run meanwhile); fp32 of few rows lacks whole tiles (768 of rows, 640 of
// columns for 684 and 515), a stage in nine and even rounds of tiles.  Z's tiles may be of 256, 192 or 128 columns
// (head_tile): with 256 and 128 alone 300 x 256 takes 15 and 20 us.  kOut with tiles of d_h and of d_W in one
// launch has one end with idle SMs instead of two, and four accumulators instead of two for 128 columns spare fp32 5 %
// (684 x 515) to 13 % (8192 x 512 over 256 words).
#include "head.cuh"
#include "pair.cuh"

namespace ssm {

namespace {

enum Use { kLogits, kGrad, kOut };

constexpr int kThreads = 384;
constexpr int kSumWarps = 8;
constexpr uint32_t kSlab = 64 * 128;          // a box of 64 x 64 bf16
constexpr uint32_t kOperand = 2 * kSlab;      // 128 rows or columns of a CTA
constexpr uint32_t kTmCols = 2 * kHeadTile;
constexpr int kRegsFew = 64, kRegsSum = 216;  // PLANES = 3: 128 x 64 + 256 x 216 <= 384 x 168

// Shared memory of a CTA: slots of A's and B's part of a stage (one plane of it), then, only where results
// are stored at any width, 32 x 32 values of each warp that takes them out, rows 33 apart (Taker::store).
// Without those a block of the small kernels before and behind fits beside it, so that either starts under the
// other's end.
constexpr int kSlots = 6;
constexpr uint32_t kSlot = 2 * kOperand, kAtTurn = kSlots * kSlot;
constexpr uint32_t kTurn = kSumWarps * 32 * 33 * 4, kSmem = kAtTurn + 1024;

// Stages between two emptyings of the accumulator: as the tensor cores truncate when they add, by up to 2^-23 of
// the sum for each 16 terms.  Errors of lse and of d_W against 64 bits (plain fp32: 2e-7, 6.6e-7 and up):
//   fp32, 1021 x 515 over 10007 words: every 2 stages 3.2e-7 and 6.4e-7, every stage 0.7e-7 and 3.5e-7, for
//     5 % of the time
//   bf16, lse and the loss (medians over random sizes of 700 - 1024 and 1025 - 2048 columns; plain fp32 1.9e-7 and
//     3e-7): every 16 stages 5.9e-7 and 6.8e-7, 8 3.2e-7 and 3.5e-7, 4 1.6e-7 and 1.8e-7.  Forward
//     of 7370 x 768 over 50000 words at 16, 8 and 4: 293, 306 and 347 us, 16384 x 1024 over 32768 590, 601 and 664;
//     with few tiles (as where their widths are chosen) 4 cost nothing (64 x 768 over 32768 words 29.0, 29.0 and
//     27.3, 1021 x 512 over 10000 28.2, 29.0 and 27.0).
//   G of bf16 operands is rounded far more coarsely: its logits every 16 stages, as one sum up to 1024 columns.
// The sums of bf16 gradients, over any number of rows or words, are emptied every 64 stages (4096 terms), which
// leaves 1.5e-5 of a sum of one sign, 1/128 of the result's own rounding and less; all at once 65536 rows lost 2.4e-4.
// It costs 0.4 % at most (8192 x 768 over 50000 words 1493 -> 1499 us; every 16 stages 1523).
constexpr int kSegmentLogits = 8, kSegmentFew = 4, kSegmentGrad = 16, kSegmentOut = 64;

// A product of a launch.
struct Job {
  CUtensorMap a, b;
  int a_mn, b_mn;      // how the operands lie
  int m_fixed;         // rows of the result; 0: the packed rows
  int n, tile_n;       // columns of the result, and of a tile (256 or 128; 0: the state's, 192 too)
  int k_fixed;         // length of the sum; 0: the packed rows
  int a_terms;         // log2 of A's terms with bf16 operands: a stage for each, the smaller one first
  int per_split;       // stages of a split of the sum (each of A's terms has its own)
  int b_row0;          // first row of b's in the tensor
  int m_first;         // unit order: m fastest (else n)
  // kOut: the splits' sums or, where there is one split, the result
  float* part;
  long long part_rows;
  int ld_part, add;
  void* out;
  long long ld_out;
  int vec_out;
  const int* to_row;   // out's row of each of the result's; NULL: the same
};

struct TcArgs {
  Job job[2];
  int jobs;
  HeadState* state;
  int no_wait;
  int segment;  // bf16 operands: stages between two emptyings
  // kLogits, kGrad
  float scale;         // log2(e) / tau
  float inv_tau, inv_tau_rest;
  int v0, vocab;       // the word of column 0
  int entries;
  const int* src;
  const int* idx;
  const uint8_t* table;
  int part_shift;
  const float* p;
  float2* stats;
  float* zt;
  long long ld_stats;
  const float *rl, *rg;
  __nv_bfloat16* g;
  long long ld_g, plane_g;
  int fine;            // G in two terms with bf16 operands
  int io;
};

// Matrix descriptors: 128-byte swizzle.  K-major: rows of 128 bytes, 8 of them 1024 bytes apart; 16 of the
// sum are 32 bytes.  MN-major: slabs of 64 columns, kSlab apart, rows of 128 bytes; 16 of the sum are
// 2048 bytes.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, bool mn) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn ? kSlab >> 4 : 1u) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// A bounded wait that also ends where another part of the pair has given up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const int* bad) {
  const uint32_t addr = smem_u32(bar);
  for (uint32_t i = 0; i < kSpinLimit; i++) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if (*reinterpret_cast<const volatile int*>(bad)) return false;
  }
  return false;
}
// Tells both CTAs.
__device__ __forceinline__ void give_up(int* bad) {
#pragma unroll
  for (int cta = 0; cta < 2; cta++) {
    uint32_t a = smem_u32(bad);
    asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(cta));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(1u) : "memory");
  }
}

__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8]) {  // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The smaller one, NaN if either is one.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// v[i], i known to the thread only: halving.
__device__ __forceinline__ float pick(const float (&v)[32], int i) {
  float s[16];
#pragma unroll
  for (int j = 0; j < 16; j++) s[j] = i & 16 ? v[j + 16] : v[j];
#pragma unroll
  for (int n = 8; n > 0; n >>= 1)
#pragma unroll
    for (int j = 0; j < n; j++) s[j] = i & n ? s[j + n] : s[j];
  return s[0];
}

// What becomes of a row's columns of a tile's half, 32 at a time (chunk c).
template <int USE, int PLANES> struct Taker {
  const TcArgs& a;
  const Job& job;
  const int row, col0, width;  // of the result: its row, and its columns
  const bool row_ok;
  float* turn;  // this warp's
  // kLogits, kGrad
  int e, next, src;  // the row's next entry, from this thread's first column on
  float top = -INFINITY, rest = 0.0f, rl = 0.0f, rg = 0.0f;
  // kOut
  float* dst = nullptr;
  float scale = 1.0f;

  __device__ __forceinline__ Taker(const TcArgs& a, const Job& job, int row, int col0, int width, int rows,
                                   int split, float* turn)
      : a(a), job(job), row(row), col0(col0), width(width), row_ok(row < rows), turn(turn) {
    if constexpr (USE != kOut) {
      src = row_ok ? a.src[row] : -1;
      e = 0, next = kNoEntry;
      if (src >= 0 && a.v0 + col0 < a.vocab) find(a.v0 + col0);
      if constexpr (USE == kGrad)
        if (row_ok) rl = PLANES == 1 ? a.rl[row] * kLog2e : a.rl[row], rg = a.rg[row];
    } else {
      if (job.part) dst = job.part + ((long long)split * job.part_rows + row) * job.ld_part + col0;
      else scale = a.state->scale;
    }
  }

  // The first entry from `word` on of the row's list, which is in order: between the places that the row's
  // table has for the word's part of the vocabulary, by halving.  (Halving all of 64 entries, 8 reads per
  // row and tile, and looking at 8 and 8 of them at once, took 110 and 143 us for the logits of 4096 x 768
  // over 32768 words.)
  __device__ __forceinline__ void find(int word) {
    const int* list = a.idx + (long long)src * a.entries;
    int lo = 0, hi = a.entries;
    if (a.table) {
      const uint8_t* t = a.table + (long long)src * kHeadParts;
      const int part = word >> a.part_shift;
      lo = t[part];
      if (part + 1 < kHeadParts) hi = t[part + 1];
    }
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (list[mid] < word) lo = mid + 1;
      else hi = mid;
    }
    e = lo;
    if (e < a.entries) next = list[e];
  }

  __device__ __forceinline__ void chunk(int c, float (&v)[32]) {
    if constexpr (USE == kLogits) {
      const int word = a.v0 + col0 + 32 * c;
      if (word + 32 > a.vocab) {
#pragma unroll
        for (int i = 0; i < 32; i++)
          if (word + i >= a.vocab) v[i] = -INFINITY;
      }
      float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < 32; i++) m[i & 3] = fmaxf(m[i & 3], v[i]);
      const float above = fmaxf(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
      const float at = above == -INFINITY ? 0.0f : above;
      const float one = above > top ? 1.0f : 0.0f;  // the largest so far is among these
      const float f = ex2((top - at) * a.scale);
      rest = fmaf(rest, f, one * f);
      top = above;
      // The distance first: logits may be so large that a product's rounding is not small.
      f2_t s[4] = {};
      const f2_t off = f2_pack(-at, -at), scale = f2_pack(a.scale, a.scale);
#pragma unroll
      for (int i = 0; i < 16; i++)
        s[i & 3] = f2_add(s[i & 3], f2_ex2(f2_mul(f2_add(f2_pack(v[2 * i], v[2 * i + 1]), off), scale)));
      float s0, s1;
      f2_unpack(f2_add(f2_add(s[0], s[1]), f2_add(s[2], s[3])), s0, s1);
      float here = s0 + s1 - one;
      // Where it is nearly all of them, the others by themselves (there is no second one like it then): next to it they
      // would lose up to 6 roundings of 2^-24, which is 6e-6 of a sum of 2^-4.  Forward of 8192 x 768 over 50000 words
      // with three rows in five of that kind 307 -> 311 us, 333 x 256 over 5003 fp32 25.3 -> 26.9.
      if (one > 0.0f && here < 0.0625f) {
        here = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++) here += v[i] == at ? 0.0f : ex2((v[i] - at) * a.scale);
      }
      rest += here;
      while (next < word + 32) {
        a.zt[(long long)src * a.entries + e] = pick(v, next - word);
        advance();
      }
    } else if constexpr (USE == kGrad) {
      const int word = a.v0 + col0 + 32 * c;
      // At most 1, also where logits are so large that roundings are not small.  With fp32 operands the
      // distance z / tau - lse is formed first (1 / tau in two terms): a product rounded at lse log2(e) would
      // be the largest error of G.
#pragma unroll
      for (int i = 0; i < 32; i++) {
        const float x = PLANES == 1 ? fmaf(v[i], a.scale, -rl) :
                                      fmaf(v[i], a.inv_tau, fmaf(v[i], a.inv_tau_rest, -rl)) * kLog2e;
        v[i] = ex2(min_nan(x, 0.0f));
      }
      // In braces: nvcc 13.0.88 drops an unrolled loop (`#pragma unroll`, whatever the optimisation level) that
      // comes next behind a discarded `if constexpr (...) while (...)` without them, here the products with rg.
      if constexpr (PLANES > 1) {
        while (next < word + 32) {
          const float p = prob();
          const int at = next - word;
#pragma unroll
          for (int i = 0; i < 32; i++) v[i] -= i == at ? p : 0.0f;
          advance();
        }
      }
      const f2_t rg2 = f2_pack(rg, rg);
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        f2_unpack(f2_mul(f2_pack(v[i], v[i + 1]), rg2), v[i], v[i + 1]);
      // past the vocabulary, and in the rows of zeros past the packed ones, whatever W holds
      const int left = src < 0 ? 0 : a.vocab - word;
      if (left < 32) {
#pragma unroll
        for (int i = 0; i < 32; i++)
          if (i >= left) v[i] = 0.0f;
      }
      if (!row_ok || col0 + 32 * c >= job.n) return;  // tiles of 192 go past a piece's end
      __nv_bfloat16* g = a.g + (long long)row * a.ld_g + col0 + 32 * c;
#pragma unroll
      for (int r = 0; r < PLANES; r++) {
#pragma unroll
        for (int b = 0; b < 2; b++) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const int j = 16 * b + 2 * i;
            w[i] = bf16x2_rn(v[j], v[j + 1]);
            if (r + 1 < PLANES) {
              v[j] -= __uint_as_float(w[i] << 16);
              v[j + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
          }
          st_global32(g + r * a.plane_g + 16 * b, w);
          if (PLANES == 1 && a.fine) {  // what is left of them; v stays
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const int j = 16 * b + 2 * i;
              w[i] = bf16x2_rn(v[j] - __uint_as_float(w[i] << 16),
                               v[j + 1] - __uint_as_float(w[i] & 0xffff0000u));
            }
            st_global32(g + a.plane_g + 16 * b, w);
          }
        }
      }
      if constexpr (PLANES == 1) {  // cheaper than a subtraction from each: over what was stored for the word
        while (next < word + 32) {
          const int at = next - word;
          float p = 0.0f;
          for (; next == word + at; advance()) p += prob();
          const float x = pick(v, at) - p * rg;
          const __nv_bfloat16 first = __float2bfloat16_rn(x);
          g[at] = first;
          if (a.fine) g[a.plane_g + at] = __float2bfloat16_rn(x - __bfloat162float(first));
        }
      }
    } else if (job.part) {
      if (!row_ok) return;
#pragma unroll
      for (int b = 0; b < 4; b++) {
        if (col0 + 32 * c + 8 * b >= job.ld_part) break;
        float* to = dst + 32 * c + 8 * b;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = v[8 * b + i];
        if (job.add) {
          Cols<float, 8> was;
          was.load(to);
#pragma unroll
          for (int i = 0; i < 8; i++) o[i] += was.a[i];
        }
        st_cols(to, o);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; i++) v[i] *= scale;
      if (a.io == SSM_BF16) store((__nv_bfloat16*)job.out, c, v);
      else store((float*)job.out, c, v);
    }
  }
  __device__ __forceinline__ float prob() const {
    return a.p ? a.p[(long long)src * a.entries + e] : 1.0f;
  }
  __device__ __forceinline__ void advance() {
    e++;
    next = e < a.entries ? a.idx[(long long)src * a.entries + e] : kNoEntry;
  }
  // Rows of any width are turned around first, so that a warp stores 32 columns of one row at a time: as
  // single values down a column 10007 x 515 fp32 took 76 us in all.
  template <typename T> __device__ __forceinline__ void store(T* out, int c, const float (&v)[32]) {
    const int first = col0 + 32 * c;
    const int mine = row_ok ? (job.to_row ? job.to_row[row] : row) : -1;
    if (job.vec_out) {
      T* to = out + mine * job.ld_out + first;
#pragma unroll
      for (int b = 0; b < 4; b++)
        if (mine >= 0 && first + 8 * b < job.n) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; i++) o[i] = v[8 * b + i];
          st_cols(to + 8 * b, o);
        }
    } else {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int i = 0; i < 32; i++) turn[33 * lane + i] = v[i];
      __syncwarp();
#pragma unroll 8
      for (int i = 0; i < 32; i++) {
        const int at = __shfl_sync(0xffffffffu, mine, i);
        if (at >= 0 && first + lane < job.n) st(out + at * job.ld_out + first + lane, turn[33 * i + lane]);
      }
      __syncwarp();
    }
  }
  __device__ __forceinline__ void done() {
    if constexpr (USE == kLogits)
      if (row_ok)
        a.stats[(long long)((a.v0 + col0) / width) * a.ld_stats + row] =
            make_float2(top, rest);
  }
};

// The units of a launch: each product's tiles, and ranges of its sum; the first product's come first.
struct Unit {
  int job, mt, nt, split, begin, iters, tile_n;
};
struct Units {
  int m[2], n[2], stages[2], rows[2], total[2], tile_n[2];
  __device__ __forceinline__ Units(const TcArgs& a, int count) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      total[j] = 0;
      if (j >= a.jobs) continue;
      const Job& b = a.job[j];
      rows[j] = b.m_fixed ? b.m_fixed : count;
      tile_n[j] = b.tile_n ? b.tile_n : a.state->tile;
      m[j] = (rows[j] + kHeadTile - 1) / kHeadTile;
      n[j] = (b.n + tile_n[j] - 1) / tile_n[j];
      const int k = b.k_fixed ? b.k_fixed : count;
      stages[j] = (k + kHeadBlock - 1) / kHeadBlock << b.a_terms;
      total[j] = m[j] * n[j] * ((stages[j] + b.per_split - 1) / b.per_split);
    }
  }
  __device__ __forceinline__ int all() const { return total[0] + total[1]; }
  __device__ __forceinline__ Unit of(const TcArgs& a, int u) const {
    Unit x;
    x.job = u >= total[0];
    const Job& b = a.job[x.job];
    if (x.job) u -= total[0];
    const int mj = x.job ? m[1] : m[0], nj = x.job ? n[1] : n[0],
              sj = x.job ? stages[1] : stages[0];
    x.split = u / (mj * nj);
    const int t = u - x.split * (mj * nj);
    if (b.m_first) x.nt = t / mj, x.mt = t - x.nt * mj;
    else x.mt = t / nj, x.nt = t - x.mt * nj;
    x.begin = x.split * b.per_split;
    x.iters = sj - x.begin < b.per_split ? sj - x.begin : b.per_split;
    x.tile_n = x.job ? tile_n[1] : tile_n[0];
    return x;
  }
};

// SEG: sums are taken out in between (without it the kernel has half the registers).
template <int USE, int PLANES, bool SEG>
__global__ void __launch_bounds__(kThreads, 1) head_tc_kernel(const __grid_constant__ TcArgs a) {
  constexpr int S = kSlots;
  const int kSeg = !SEG ? 1 << 30 : PLANES > 1 ? 1 : a.segment;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t here[S], there[S], empty[S], ready[4], drained[4], last;
  __shared__ uint32_t tbase;
  __shared__ int bad;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to the compiler as uniform
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int i = 0; i < S; i++) {
      mbar_init(&here[i], 1);
      mbar_init(&there[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int b = 0; b < 4; b++) {
      mbar_init(&ready[b], 1);
      mbar_init(&drained[b], 2 * kSumWarps);
    }
    mbar_init(&last, 1);
    bad = 0;
    fence_barrier_init();
    for (int j = 0; j < a.jobs; j++) {
      prefetch_tmap(&a.job[j].a);
      prefetch_tmap(&a.job[j].b);
    }
  }
  __syncwarp();
  if (warp == 1) Mma<2>::alloc(&tbase, kTmCols);
  tmem_fence_before_sync();
  __syncthreads();
  sync_tile<2>();
  tmem_fence_after_sync();
  const uint32_t tm = tbase;
  asm volatile("griddepcontrol.launch_dependents;");
  wait_for_copies();
  const int count = a.state->count > 0 ? a.state->count : 1;
  const Units units(a, count);
  const int n_units = units.all();
  // Accumulators: two of up to 256 columns or four of 128 (both products' tiles are alike), by turns.
  const int acc_log = units.tile_n[0] > kHeadTile / 2 ? 1 : 2, acc_mask = (1 << acc_log) - 1;
  const uint32_t acc_cols = kTmCols >> acc_log;

  if (warp < 4) {
    if constexpr (PLANES > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      Ring<S> r;
      int it = 0;
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += pairs) {
        const Unit x = units.of(a, u);
        const Job& b = a.job[x.job];
        const int half = x.tile_n / 2;  // columns of B here
        const int m0 = x.mt * kHeadTile + rank * (kHeadTile / 2), n0 = x.nt * x.tile_n + rank * half;
        const bool a_mn = b.a_mn, b_mn = b.b_mn;
        const uint32_t bytes = kOperand + (half > 64 ? 2 : 1) * kSlab;  // of 96 columns all of the second slab
        for (int stage = x.begin; stage < x.begin + x.iters && ok; stage++) {
          const int k = stage >> b.a_terms;
#pragma unroll
          for (int i = 0; i < PLANES; i++, it++, r.next()) {
            const int p = PLANES == 1 ? 0 : i == 0 ? 1 : i == 1 ? 0 : 2;
            const int pa = PLANES == 1 ? b.a_terms & ~stage : p;
            if (it >= S) ok = ok && wait_for(&empty[r.s], r.phase ^ 1, &bad);
            if (!ok) break;
            if (elect_one()) {
              mbar_expect_tx(&here[r.s], bytes);
              unsigned char* to = smem + r.s * kSlot;
#pragma unroll
              for (int c = 0; c < 2; c++) {
                tma_load_3d(to + c * kSlab, &b.a, a_mn ? m0 + 64 * c : 64 * k,
                            a_mn ? 64 * k : m0 + 64 * c, pa, &here[r.s]);
                if (64 * c < half)
                  tma_load_3d(to + kOperand + c * kSlab, &b.b, b_mn ? n0 + 64 * c : 64 * k,
                              b.b_row0 + (b_mn ? 64 * k : n0 + 64 * c), p, &here[r.s]);
              }
            }
            __syncwarp();
          }
        }
      }
      // the copies in flight land, and the first CTA's word that their slots are free arrives, before the
      // block may end
      for (int j = it > S ? it - S : 0; j < it; j++) {
        if (!mbar_wait(&here[j % S], (j / S) & 1)) break;
        if (ok) ok = wait_for(&empty[j % S], (j / S) & 1, &bad);
      }
      if (!ok) give_up(&bad);
    } else if (warp == 1 && rank == 0) {
      Ring<S> r;
      int seg = 0;  // counted over the units
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += pairs) {
        const Unit x = units.of(a, u);
        const int iters = x.iters;
        const bool a_mn = a.job[x.job].a_mn, b_mn = a.job[x.job].b_mn;
        const uint32_t idesc = idesc_bf16(kHeadTile, x.tile_n, a_mn, b_mn);
        const uint64_t da0 = desc_of(smem_u32(smem), a_mn),
                       db0 = desc_of(smem_u32(smem) + kOperand, b_mn);
        const uint32_t sa = a_mn ? 2048 >> 4 : 32 >> 4, sb = b_mn ? 2048 >> 4 : 32 >> 4;
        for (int it = 0; it < iters && ok; seg++) {
          const uint32_t d = tm + (seg & acc_mask) * acc_cols;
          const int end = iters - it < kSeg ? iters : it + kSeg;
          if (seg > acc_mask)
            ok = wait_for(&drained[seg & acc_mask], ((seg >> acc_log) - 1) & 1, &bad);
          bool first = true;
          // the product of slot i's A and slot j's B
          const auto mul = [&](int i, int j, bool add) {
            const uint64_t da = da0 + (uint32_t)(i * (kSlot >> 4)), db = db0 + (uint32_t)(j * (kSlot >> 4));
#pragma unroll
            for (int kk = 0; kk < kHeadBlock / 16; kk++)
              Mma<2>::mma(idesc, d, da + sa * kk, db + sb * kk, add || kk > 0);
          };
          for (; it < end && ok; it++, first = false) {
            int slot[PLANES];
#pragma unroll
            for (int i = 0; i < PLANES && ok; i++, r.next()) {
              slot[i] = r.s;
              ok = wait_for(&here[r.s], r.phase, &bad) && wait_for(&there[r.s], r.phase, &bad);
              tmem_fence_after_sync();
              if (ok && elect_one()) {
                if (PLANES == 1) {
                  mul(slot[0], slot[0], !first);
                  Mma<2>::commit(&empty[slot[0]]);
                } else if (i == 0) {  // plane 1
                  mul(slot[0], slot[0], !first);
                } else if (i == 1) {  // plane 0
                  mul(slot[0], slot[i], true);
                  mul(slot[i], slot[0], true);
                  Mma<2>::commit(&empty[slot[0]]);
                } else {  // plane 2, then the leading product
                  mul(slot[i], slot[1], true);
                  mul(slot[1], slot[i], true);
                  Mma<2>::commit(&empty[slot[i]]);
                  mul(slot[1], slot[1], true);
                  Mma<2>::commit(&empty[slot[1]]);
                }
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          if (elect_one()) Mma<2>::commit(&ready[seg & acc_mask]);
          __syncwarp();
        }
      }
      if (!ok) give_up(&bad);
    } else if (warp == 1) {
      Ring<S> r;
      const uint32_t first_there = bar_of_first<2>(there);
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += pairs) {
        const int slots = units.of(a, u).iters * PLANES;
        for (int it = 0; it < slots && ok; it++, r.next()) {
          ok = wait_for(&here[r.s], r.phase, &bad);
          if (ok && elect_one()) mbar_arrive_first<2>(first_there + 8 * r.s);
          __syncwarp();
        }
      }
      if (!ok) give_up(&bad);
    }
  } else {
    if constexpr (PLANES > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSum));
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = tm + ((uint32_t)(32 * quad) << 16);
    float* turn = reinterpret_cast<float*>(smem + kAtTurn) + (warp - 4) * 32 * 33;
    const uint32_t first_drained = bar_of_first<2>(drained);
    int seg = 0;
    bool ok = !a.no_wait;
    for (int u = pair; u < n_units && ok; u += pairs) {
      const Unit x = units.of(a, u);
      const int iters = x.iters, width = x.tile_n / 2, chunks = width / 32;
      const uint32_t tacc = lanes + width * half;
      // the rows that a sum over rows reads: zeros past the packed ones
      const int rows_here = x.job ? units.rows[1] : units.rows[0];
      const int rows = USE == kGrad ? (rows_here + 63) / 64 * 64 : rows_here;
      Taker<USE, PLANES> taker(a, a.job[x.job],
                               x.mt * kHeadTile + rank * (kHeadTile / 2) + 32 * quad + lane,
                               x.nt * x.tile_n + width * half, width, rows, x.split, turn);
      if constexpr (!SEG) {
        ok = wait_for(&ready[seg & acc_mask], (seg >> acc_log) & 1, &bad);
        __syncwarp();
        tmem_fence_after_sync();
        if (!ok) break;
        const uint32_t t = tacc + (seg & acc_mask) * acc_cols;
#pragma unroll 1
        for (int c = 0; c < chunks; c++) {
          float v[32];
          tmem_ld32(t + 32 * c, v);
          if (c == chunks - 1) {
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_first<2>(first_drained + 8 * (seg & acc_mask));
          }
          taker.chunk(c, v);
          __syncwarp();
        }
        seg++;
      } else {
        // The first stretch of a sum is loaded in place, which is half of what these warps would do for sums of two
        // (fp32, with one for each stage, is 3 % slower so).
        float acc[4][32];
        if constexpr (PLANES > 1) {
#pragma unroll
          for (int c = 0; c < 4; c++)
#pragma unroll
            for (int i = 0; i < 32; i++) acc[c][i] = 0.0f;
        }
        for (int it = 0; it < iters && ok; it += kSeg, seg++) {
          ok = wait_for(&ready[seg & acc_mask], (seg >> acc_log) & 1, &bad);
          __syncwarp();
          tmem_fence_after_sync();
          if (!ok) break;
          const uint32_t t = tacc + (seg & acc_mask) * acc_cols;
#pragma unroll
          for (int c = 0; c < 4; c++) {
            if (c >= chunks) break;
            if (PLANES == 1 && it == 0) {
              tmem_ld32(t + 32 * c, acc[c]);
            } else {
              float v[32];
              tmem_ld32(t + 32 * c, v);
#pragma unroll
              for (int i = 0; i < 32; i++) acc[c][i] += v[i];
            }
          }
          tmem_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_first<2>(first_drained + 8 * (seg & acc_mask));
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          if (c >= chunks) break;
          taker.chunk(c, acc[c]);
          __syncwarp();
        }
      }
      taker.done();
    }
    if (!ok) give_up(&bad);
  }
  __syncwarp();
  __syncthreads();
  sync_tile<2>();  // what either CTA gave up is known to both
  const bool gave_up = *reinterpret_cast<volatile int*>(&bad);
  if (warp == 1 && rank == 0 && gave_up) {
    // Perhaps with MMAs in flight: they read the shared memory and write the tensor memory of both CTAs,
    // so they complete first.
    if (elect_one()) Mma<2>::commit_here(&last);
    __syncwarp();
    mbar_wait(&last, 0);
  }
  sync_tile<2>();
  if (warp == 1) {
    tmem_fence_after_sync();
    Mma<2>::dealloc(tm, kTmCols);
  }
  if (tid == 0 && gave_up) atomicExch(&a.state->status, SSM_ERR_TIMEOUT);
}

template <int USE, int PLANES, bool SEG>
cudaError_t launch(const TcArgs& t, int sms, cudaStream_t st) {
  auto kernel = head_tc_kernel<USE, PLANES, SEG>;
  bool turn = false;
  for (int j = 0; j < t.jobs; j++)
    turn = turn || (USE == kOut && !t.job[j].part && !t.job[j].vec_out);
  // asked for once per device (the first 64 remember it)
  static std::atomic<unsigned long long> asked{0};
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(kSmem + kTurn)))
      return e;
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(sms / 2 * 2);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem + (turn ? kTurn : 0);
  c.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, t);
  count_launches(1);
  return e;
}
template <int USE> cudaError_t launch(const ssm_head_desc& d, const TcArgs& t, int sms, cudaStream_t st) {
  if (d.io == SSM_F32) return launch<USE, 3, true>(t, sms, st);
  for (int j = 0; j < t.jobs; j++)
    if (t.job[j].per_split > t.segment) return launch<USE, 1, true>(t, sms, st);
  return launch<USE, 1, false>(t, sms, st);
}

bool encode(CUtensorMap* map, const HeadMatrix& x, int planes) {
  return encode_tmap_3d(map, x.p, 2, x.cols, x.rows, planes, x.ld, planes > 1 ? x.plane : x.ld, 64,
                        64, 1, 128);
}
int planes_of(const ssm_head_desc& d) { return d.io == SSM_F32 ? 3 : 1; }

TcArgs args_of(const ssm_head_desc& d, const HeadRows& r, const HeadLists& lists) {
  TcArgs t{};
  t.jobs = 1;
  t.state = r.state;
  t.no_wait = (d.flags & SSM_DEBUG_NO_WAIT) != 0;
  t.scale = d.entries ? kLog2e / d.temperature : kLog2e;
  const double inv = d.entries ? 1.0 / d.temperature : 1.0;
  t.inv_tau = (float)inv;
  t.inv_tau_rest = (float)(inv - t.inv_tau);
  t.vocab = d.vocab;
  t.entries = d.entries ? d.entries : 1;
  t.src = r.src;
  t.idx = lists.idx;
  t.table = lists.table;
  t.part_shift = head_part_shift(d.vocab);
  t.p = lists.p;
  t.io = d.io;
  return t;
}
// Z of the words from v0 on.
bool logits_job(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w, int v0, int n, Job& j) {
  j.n = n;
  j.k_fixed = d.cols;
  j.per_split = (d.cols + kHeadBlock - 1) / kHeadBlock;
  j.b_row0 = v0;
  j.m_first = 1;
  return encode(&j.a, h, planes_of(d)) && encode(&j.b, w, planes_of(d));
}

}  // namespace

cudaError_t launch_head_logits(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w,
                               const HeadRows& r, const HeadLists& lists, const HeadTiles& tiles,
                               float2* stats, float* zt, int sms, cudaStream_t st) {
  TcArgs t = args_of(d, r, lists);
  t.segment = tiles.words ? kSegmentFew : kSegmentLogits;
  if (!logits_job(d, h, w, 0, d.vocab, t.job[0])) return cudaErrorInvalidValue;
  t.stats = stats;
  t.ld_stats = h.rows;
  t.zt = zt;
  return launch<kLogits>(d, t, sms, st);
}

cudaError_t launch_head_grad(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w,
                             const HeadRows& r, const HeadLists& lists, __nv_bfloat16* g, int v0, int n,
                             int sms, cudaStream_t st) {
  TcArgs t = args_of(d, r, lists);
  if (!logits_job(d, h, w, v0, n, t.job[0])) return cudaErrorInvalidValue;
  t.segment = kSegmentGrad;
  t.v0 = v0;
  t.rl = r.rl;
  t.rg = r.rg;
  t.g = g;
  t.ld_g = n;
  t.plane_g = h.rows * n;
  t.fine = head_g_terms(d) == 2;
  return launch<kGrad>(d, t, sms, st);
}

cudaError_t launch_head_out(const ssm_head_desc& d, const HeadMatrix& g, const HeadMatrix& h,
                            const HeadMatrix& w, const HeadRows& r, const HeadOut& o, int v0, int n,
                            bool add, int sms, cudaStream_t st) {
  TcArgs t = args_of(d, r, {});
  t.jobs = 0;
  t.segment = kSegmentOut;
  const int planes = planes_of(d), terms = head_g_terms(d), padded = pad8(d.cols);
  const size_t size = d.io == SSM_F32 ? 4 : 2;
  if (o.d_w) {
    Job& j = t.job[t.jobs++];
    if (!encode(&j.a, g, terms) || !encode(&j.b, h, planes)) return cudaErrorInvalidValue;
    j.a_mn = j.b_mn = 1;
    j.a_terms = terms == 2;
    j.m_fixed = n;
    j.n = d.cols;
    j.tile_n = o.w.tile_n;
    j.per_split = o.w.per;
    j.part = o.w_part;
    j.part_rows = g.cols;
    j.ld_part = padded;
    j.out = (char*)o.d_w + (size_t)v0 * d.cols * size;
    j.ld_out = d.cols;
    j.vec_out = d.cols % 8 == 0 && (uintptr_t)o.d_w % (8 * size) == 0;
  }
  if (o.h_part || o.d_h) {
    Job& j = t.job[t.jobs++];
    if (!encode(&j.a, g, terms) || !encode(&j.b, w, planes)) return cudaErrorInvalidValue;
    j.b_mn = 1;
    j.a_terms = terms == 2;
    j.n = d.cols;
    j.tile_n = o.h.tile_n;
    j.k_fixed = g.cols;
    j.per_split = o.h.per;
    j.b_row0 = v0;
    j.part = o.h_part;
    j.part_rows = g.rows;
    j.ld_part = padded;
    j.add = add;
    j.out = o.d_h;
    j.ld_out = o.ld_d_h;
    j.vec_out = d.cols % 8 == 0 && o.ld_d_h % 8 == 0 && (uintptr_t)o.d_h % (8 * size) == 0;
    j.to_row = r.src;
  }
  if (t.jobs == 2 && o.h_first) {
    const Job j = t.job[0];
    t.job[0] = t.job[1], t.job[1] = j;
  }
  return launch<kOut>(d, t, sms, st);
}

}  // namespace ssm
