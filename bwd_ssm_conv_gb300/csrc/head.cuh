// head.cuh -- launchers of the head and its loss, called by the C ABI in head_api.cu: head_rows.cu holds
// what happens to rows (which of them count, copies, the sums over the vocabulary's tiles, d_h),
// head_tc.cu the products.
//
// Rows that have a loss are packed: row r of the packed ones is row src[r] of the call, pos[] is the
// inverse.  Everything between the calls' arguments and results goes by packed rows, `count` of them, a
// number that only the device knows; zeros fill up to a multiple of 64 (at least 64), so that sums over
// rows need not stop inside a tile.
#pragma once

#include <math.h>

#include "kernels.cuh"
#include "rows.cuh"
#include "ssm_head.h"

namespace ssm {

constexpr int kHeadTile = 256;   // rows and columns of a pair of CTAs' tile
constexpr int kHeadBlock = 64;   // of a sum, per stage
constexpr int kIgnored = -1, kBadRow = -2;  // in pos[]
constexpr int kNoEntry = 0x7fffffff;        // fills a row's list of entries

// The workspace's first bytes.
struct HeadState {
  int status;
  int count;     // packed rows
  float scale;   // what G lacks between the products: tau times the largest finite |d_loss| of theirs (1: none)
  int tile;      // columns of a tile of Z
};

struct HeadRows {  // of a call, on the device
  HeadState* state;
  int* pos;  // [rows]
  int* src;  // [padded rows], -1 past the packed ones
  float *rl, *rg;  // backward, [padded rows]: lse, d_loss over the largest
  __nv_bfloat16* h;  // [planes][padded rows][padded cols]
};

// What the rows say, by rows of the call: their words in order ([rows][entries], ended by kNoEntry where
// there are fewer; one target) and, of a teacher, p, sum p log p, and for each of kHeadParts equal parts
// of the vocabulary how many of the row's words lie before it.
constexpr int kHeadParts = 64;
struct HeadLists {
  int* idx;
  float* p;
  float* known;
  uint8_t* table;
};
inline int head_part_shift(int vocab) {  // a part's words, as a power of two
  int shift = 0;
  while (((vocab - 1) >> shift) >= kHeadParts) shift++;
  return shift;
}

// Sums of the exponentials 2^((z - top) scale) of a row's words, without the one of the largest logit itself,
// which is 1: next to it the others of a loss near 0 would lose their digits.
struct HeadSum {
  float top, rest;
};
__device__ __forceinline__ HeadSum join(const HeadSum& a, const HeadSum& b, float scale) {
  const bool second = b.top > a.top;
  const HeadSum &hi = second ? b : a, &lo = second ? a : b;
  const float f = ex2((lo.top - (hi.top == -INFINITY ? 0.0f : hi.top)) * scale);  // 0 where lo has no words
  return {hi.top, hi.rest + fmaf(f, lo.rest, f)};
}

// Z's tiles are 256, 192 or 128 words wide: what takes the fewest rounds of the pairs of CTAs, in time, for the
// rows that count.
struct HeadTiles {
  int words;     // of a launch; 0: tiles of 256
  int pairs;
  float cost[3]; // of a tile of 256, 192 and 128
};
__host__ __device__ inline int head_tile(const HeadTiles& t, int rows) {
  int best = kHeadTile;
  float least = 0.0f;
  if (t.words)
    for (int i = 0; i < 3; i++) {
      const int tile = kHeadTile - 64 * i,
                units = (rows + kHeadTile - 1) / kHeadTile * ((t.words + tile - 1) / tile);
      const float time = (float)((units + t.pairs - 1) / t.pairs) * t.cost[i];
      if (i == 0 || time < least) least = time, best = tile;
    }
  return best;
}

// bf16 terms of G between the products.  With bf16 operands a second one leaves d_h and d_W with their own rounding.
// A tile's rows get it in any case, as reading W and writing d_W is most of their time (768 columns, 32768 words,
// us with one and two: 5 to 64 rows 62 and 69, 256 69 and 81, 512 86 and 118, 1024 123 and 192).
inline int head_g_terms(const ssm_head_desc& d) {
  return d.io == SSM_F32 ? 3 : d.rows <= kHeadTile || d.flags & SSM_HEAD_FINE_G ? 2 : 1;
}
inline int pad8(int n) { return (n + 7) / 8 * 8; }
inline long long pad_rows(long long rows) { return (rows + 63) / 64 * 64; }

// ---- head_rows.cu ---------------------------------------------------------------------------------
// A teacher's entries as lists, and in valid[row] whether the row has a loss (1), or is bad (2).
cudaError_t launch_head_entries(const ssm_head_desc& d, const int64_t* t_idx, const void* t_logit,
                                const HeadLists& lists, uint8_t* valid, cudaStream_t st);
// Which rows count, from `valid` or from the targets (whose words go to idx), their h packed (and, given
// lse, rl and rg); W with padded rows, fp32 as three planes, to w_out where that is given.
cudaError_t launch_head_rows(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                             const void* h, long long ld_h, const float* lse, const float* d_loss,
                             const void* w, long long ld_w, int* idx, const HeadRows& r,
                             __nv_bfloat16* w_out, const HeadTiles& tiles, int sms, cudaStream_t st);
// Loss and lse from the tiles' sums (n_stats of them; 0: two for each of the state's tiles); zt: the entries'
// logits [rows][entries or 1].
cudaError_t launch_head_loss(const ssm_head_desc& d, const float2* stats, int n_stats,
                             const float* zt, const HeadLists& lists, const HeadRows& r,
                             float* loss, float* lse, int sms,
                             cudaStream_t st);
// What the gradients' sums lack: d_h from the splits' sums [splits][padded rows][padded cols], and
// rows v0 .. v0 + n of d_W from theirs [splits][piece][padded cols], either where given (d_h without its sums:
// only the rows that were not written).  `last`: of the
// call; where a wait of it gave up, d_h and all of d_w are filled with NaN.
cudaError_t launch_head_finish(const ssm_head_desc& d, const HeadRows& r, const float* h_part,
                               int h_splits, void* d_h, long long ld_d_h, const float* w_part,
                               int w_per, int piece, void* d_w, int v0, int n, bool last, int sms,
                               cudaStream_t st);

// ---- head_few.cu ----------------------------------------------------------------------------------
// A few rows, unpacked (pos[row] is row).  The forward: what head_rows and head_logits do together, with
// stats [blocks][padded rows].  The backward: d_w, and d_h by way of its sums h_part [blocks][rows][padded cols]
// (either NULL: not wanted).
constexpr size_t kFewSmem = 72 * 1024;  // of a block
bool head_few(long long rows, int cols, int io, bool backward);
int head_few_blocks(int sms);
cudaError_t launch_head_few(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                            const void* h, long long ld_h, const void* w, long long ld_w,
                            const HeadLists& lists, const HeadRows& r, float2* stats, float* zt, int sms,
                            cudaStream_t st);
cudaError_t launch_head_few_bwd(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                                const void* h, long long ld_h, const void* w, long long ld_w,
                                const HeadLists& lists, const HeadRows& r, const float* lse,
                                const float* d_loss, float* h_part, void* d_h, long long ld_d_h,
                                void* d_w, int sms, cudaStream_t st);

// ---- head_tc.cu -----------------------------------------------------------------------------------
struct HeadMatrix {  // [planes][rows][cols], rows ld elements apart
  const __nv_bfloat16* p;
  long long rows, ld, plane;
  int cols;
};
// How a product with G is cut: columns of a tile (256 or 128), splits of the sum and their stages (two for
// each 64 of the sum where G has two terms).
struct HeadCut {
  int tile_n, splits, per;
};
// The sums of the vocabulary's tiles, stats [2 tiles][padded rows] (HeadSum), and the entries' logits.
cudaError_t launch_head_logits(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w,
                               const HeadRows& r, const HeadLists& lists, const HeadTiles& tiles,
                               float2* stats, float* zt, int sms, cudaStream_t st);
// G of the words v0 .. v0 + n (n a multiple of 256; 0 past the vocabulary): g [terms][padded rows][n].
cudaError_t launch_head_grad(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w,
                             const HeadRows& r, const HeadLists& lists, __nv_bfloat16* g, int v0, int n,
                             int sms, cudaStream_t st);
// The two products with G of the words v0 .. v0 + n, in one launch:
//   h_part [splits][padded rows][padded cols] (+)= G W, the piece's words split, or without it rows src[]
//   of d_h (with one split and one piece),
//   rows v0 .. v0 + n of d_W = G^T h, or with w_part [splits][piece][padded cols] the splits' sums.
struct HeadOut {
  HeadCut h, w;
  bool h_first;  // the units of d_h before those of d_W
  float* h_part;
  float* w_part;
  void* d_w;
  void* d_h;
  long long ld_d_h;
};
cudaError_t launch_head_out(const ssm_head_desc& d, const HeadMatrix& g, const HeadMatrix& h,
                            const HeadMatrix& w, const HeadRows& r, const HeadOut& o, int v0, int n,
                            bool add, int sms, cudaStream_t st);

}  // namespace ssm
