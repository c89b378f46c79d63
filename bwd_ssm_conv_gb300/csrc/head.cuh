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
  float g_top;   // the largest finite |d_loss| of theirs (1 where there is none)
  float scale;   // what G lacks between the products: g_top tau
};

struct HeadRows {  // of a call, on the device
  HeadState* state;
  int* pos;  // [rows]
  int* src;  // [padded rows], -1 past the packed ones
  float *rl, *rg;  // backward, [padded rows]: lse log2(e), d_loss / g_top
  __nv_bfloat16* h;  // [planes][padded rows][padded cols]
};

inline int pad8(int n) { return (n + 7) / 8 * 8; }
inline long long pad_rows(long long rows) { return (rows + 63) / 64 * 64; }

// ---- head_rows.cu ---------------------------------------------------------------------------------
// Teacher entries: each row's in order of the vocabulary (idx, ended by kNoEntry where there are fewer), with
// p, sum p log p in known[row], and in valid[row] whether the row has a loss (1), or is bad (2).
cudaError_t launch_head_entries(const ssm_head_desc& d, const int64_t* t_idx, const void* t_logit,
                                int* idx, float* p, float* known, uint8_t* valid, cudaStream_t st);
// Which rows count: from `valid`, or from the targets (whose words go to idx).
cudaError_t launch_head_begin(const ssm_head_desc& d, const int64_t* target, const uint8_t* valid,
                              const float* d_loss, int* idx, const HeadRows& r, bool first,
                              cudaStream_t st);
// Packs h's rows (and rl, rg, given lse).
cudaError_t launch_head_pack(const ssm_head_desc& d, const void* h, long long ld_h,
                             const float* lse, const float* d_loss, const HeadRows& r, int sms,
                             cudaStream_t st);
// W with padded rows, fp32 as three planes.
cudaError_t launch_head_copy_w(const ssm_head_desc& d, const void* w, long long ld_w,
                               __nv_bfloat16* out, int sms, cudaStream_t st);
// Loss and lse from the tiles' sums; zt: the entries' logits [rows][entries or 1].
cudaError_t launch_head_loss(const ssm_head_desc& d, const float2* stats, int n_stats,
                             const float* zt, const float* p, const float* known,
                             const HeadRows& r, float* loss, float* lse, cudaStream_t st);
// d_h from the splits' sums [splits][padded rows][padded cols].  Where a wait of the call gave up, d_h and
// d_w are filled with NaN.
cudaError_t launch_head_finish(const ssm_head_desc& d, const float* part, int splits,
                               const HeadRows& r, void* d_h, long long ld_d_h, void* d_w, int sms,
                               cudaStream_t st);
// Rows v0 .. v0 + n of d_W from the splits' sums [splits][n_part][padded cols].
cudaError_t launch_head_sum_w(const ssm_head_desc& d, const float* part, int per_split, int n_part,
                              const HeadRows& r, void* d_w, int v0, int n, int sms,
                              cudaStream_t st);

// ---- head_tc.cu -----------------------------------------------------------------------------------
struct HeadMatrix {  // [planes][rows][cols], rows ld elements apart
  const __nv_bfloat16* p;
  long long rows, ld, plane;
  int cols;
};
// The sums of the vocabulary's tiles, stats [2 tiles][padded rows], and the entries' logits.
cudaError_t launch_head_logits(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w,
                               const HeadRows& r, const int* idx, float2* stats, float* zt, int sms,
                               cudaStream_t st);
// G of the words v0 .. v0 + n (n a multiple of 256; 0 past the vocabulary): g [planes][padded rows][n].
cudaError_t launch_head_grad(const ssm_head_desc& d, const HeadMatrix& h, const HeadMatrix& w,
                             const HeadRows& r, const int* idx, const float* p, __nv_bfloat16* g,
                             int v0, int n, int sms, cudaStream_t st);
// part [splits][padded rows][padded cols] (+)= G W over a piece, its words split over `splits`.
cudaError_t launch_head_dh(const ssm_head_desc& d, const HeadMatrix& g, const HeadMatrix& w,
                           const HeadRows& r, float* part, int splits, int per_split, int v0,
                           bool add, int sms, cudaStream_t st);
// Rows v0 .. v0 + n of d_W = G^T h, or with part the splits' sums.
cudaError_t launch_head_dw(const ssm_head_desc& d, const HeadMatrix& g, const HeadMatrix& h,
                           const HeadRows& r, void* d_w, float* part, int splits, int per_split,
                           int v0, int n, int sms, cudaStream_t st);

}  // namespace ssm
