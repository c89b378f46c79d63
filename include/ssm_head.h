/*
 * ssm_head.h -- C ABI of the head and its loss (libssm_gb300.so): the logits z = h W^T over a vocabulary
 * are formed in pieces, used and dropped, in the forward and again in the backward.
 *
 *   head_ce       loss = lse - z_target,               lse = log sum_v exp(z_v)
 *   head_distill  from a teacher's logits t at `entries` words i of the vocabulary (its largest, say):
 *                 p = softmax(t / tau) over the row's entries,  q = softmax(z / tau) over the vocabulary,
 *                 lse = log sum_v exp(z_v / tau)
 *                 loss = tau^2 sum_j p_j (log p_j - log q_{i_j})
 *   backward      G = d loss / d z:  (softmax(z) - onehot(target)) d_loss,  tau (q - p) d_loss
 *                 d_h = G W,  d_W = G^T h
 *
 * Layouts: h and d_h [rows][cols], W [vocab][cols] (io), rows `ld_*` elements apart (0 means cols; at
 * least cols otherwise, those of W below 2^40 bytes); d_W [vocab][cols] (io) contiguous; target int64
 * [rows]; t_idx int64 and t_logit (entry_io) [rows][entries], loss, lse and d_loss fp32 [rows], all
 * contiguous.
 *
 * Rows without a loss: a target of ignore_index; a row without an entry.  Their loss, lse and gradient are
 * 0 and h is not read there, whatever it holds; they cost no product.  An entry with t_idx below 0 is not
 * there; one whose logit is -infinity has p = 0.  The same word twice adds up.  Any other target or entry
 * outside the vocabulary is recorded as SSM_ERR_INVALID_ARG in the status word, and the row's loss, lse and
 * d_h are NaN, without a part in d_W.
 *
 * Ownership, streams and errors are those of ssm.h: caller-owned device pointers, nothing allocated or
 * synchronised, work enqueued on `stream`, argument errors found on the host before anything is
 * enqueued.  Outputs are overwritten and overlap neither inputs nor each other.  The first word of the
 * workspace is a status word, read with ssm_scan_status; where a bounded wait gave up (SSM_ERR_TIMEOUT
 * there), every output of the call is NaN.  Sums run in a fixed order: results are bitwise reproducible.
 *
 * Arithmetic: products on the tensor cores with fp32 sums, fp32 operands as three bf16 terms each
 * (six products, which leave out 2^-24 of a product and less).  The tensor cores truncate as they
 * add, up to 2^-23 of the sum for each 16 terms: sums are taken out every 64 terms with fp32 operands,
 * with bf16 ones those of the logits every 512 or 256 (the backward's every 1024) and those of the gradients
 * every 4096, and added with rounding to nearest, so that long sums lose no more than short ones.  With bf16 operands G,
 * divided by the largest |d_loss|, is rounded to bf16 between the products (2^-8 of each of its values), which
 * gives d_h and d_W an error of the size of their own rounding; up to 256 rows, and with SSM_HEAD_FINE_G any
 * number, it is kept in two bf16 terms (2^-16), which leaves d_h and d_W with their own rounding and takes twice the
 * time where rows are many.  A few rows
 * (bf16: 2 in the forward, 4 in the backward; fp32: 8) are fp32 arithmetic throughout, G too, where they lie in the
 * shared memory of a block: rows (as a power of two) * cols up to 18000 in the forward, 9216 in the backward.
 * lse is an fp32 number, so that the backward's softmax is good to 2^-24 |lse| of its values: for logits over tau
 * of 16, 1e-6, which shows in d_h and d_W of fp32 where softmax and target are nearly alike.  The forward carries the
 * sum beside the largest exponential by itself: a loss near 0 is as good as its logits.
 * An infinite weight gives infinite logits with bf16 operands and with a few rows, and NaN with more fp32 rows, whose
 * lower terms may be 0 or of the other sign there.
 */
#ifndef SSM_HEAD_GB300_H
#define SSM_HEAD_GB300_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_HEAD_FINE_G 2u /* of a descriptor's flags */
#define SSM_MAX_HEAD_ENTRIES 128 /* teacher entries of a row (SSM_ERR_UNSUPPORTED beyond) */
#define SSM_MAX_HEAD_COLS 65536
#define SSM_MAX_HEAD_VOCAB (1 << 22)
#define SSM_MAX_HEAD_ROWS (1 << 24)    /* and rows * vocab up to 2^40 */
#define SSM_MAX_HEAD_TEMPERATURE 1e6f  /* and 1e-6 at least (SSM_ERR_UNSUPPORTED beyond) */

typedef struct {
  long long rows; /* tokens, >= 1 */
  int cols;       /* channels of h */
  int vocab;
  int io;         /* ssm_dtype of h, W and their gradients */
  int entries;    /* head_distill: teacher entries of a row, >= 1; head_ce: 0 */
  int entry_io;   /* head_distill: ssm_dtype of t_logit */
  float temperature;      /* head_distill: tau > 0, finite */
  long long ignore_index; /* head_ce: the target of a row without a loss */
  unsigned flags; /* SSM_HEAD_FINE_G: the backward of more than 256 bf16 rows keeps G in two terms as that of fewer;
                     ssm.h's SSM_DEBUG_NO_WAIT, for tests of the error path only: the warps that take
                     the sums out give up at once, as if the bound of their wait had run out (the kernels of
                     a few rows wait for nothing) */
} ssm_head_desc;

/* Bytes of scratch of a call on the current device (at least 256; 0 if the arguments are invalid): a copy of
 * h (three times its bf16 size with fp32), one of W with fp32 or rows that are not aligned, and
 *   forward   rows * vocab / 16 bytes of sums (twice that up to 5 tiles of 256 x 256 for
 *             each pair of SMs, which may be narrower ones; next to none for a few rows)
 *   backward  a piece of G, 512 MiB at most (or 256 words of it; the flags count), and fp32 sums of d_h and perhaps of d_W,
 *             up to 64 of them where there are few rows; for a few rows 2 sums of d_h per SM.
 * grads: 0 for the forward, else bits 1 (d_h wanted) and 2 (d_W wanted) of the backward.  aligned: W's rows
 * (pointer and ld_w * element size) are 16-byte aligned; fp32 W may lie anywhere. */
size_t ssm_head_workspace_size(const ssm_head_desc* desc, int grads, int aligned);

/* Forward.  Required: everything but lse. */
int ssm_head_ce_fwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                    long long ld_w, const int64_t* target, float* loss, float* lse, void* ws,
                    size_t ws_bytes, void* stream);
int ssm_head_distill_fwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                         long long ld_w, const int64_t* t_idx, const void* t_logit, float* loss,
                         float* lse, void* ws, size_t ws_bytes, void* stream);

/* Backward.  lse: the forward's.  One of d_h and d_w may be NULL. */
int ssm_head_ce_bwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                    long long ld_w, const int64_t* target, const float* lse, const float* d_loss,
                    void* d_h, long long ld_d_h, void* d_w, void* ws, size_t ws_bytes,
                    void* stream);
int ssm_head_distill_bwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                         long long ld_w, const int64_t* t_idx, const void* t_logit,
                         const float* lse, const float* d_loss, void* d_h, long long ld_d_h,
                         void* d_w, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
