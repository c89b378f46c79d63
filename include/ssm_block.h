/*
 * ssm_block.h -- C ABI of the operators around the scan in a Mamba block (libssm_gb300.so):
 * the norms before and after it and 8-bit activation checkpoints.
 *
 *   add_norm    s   = residual + scale * x            (residual and scale optional)
 *               out = w * s * rstd,   rstd = 1 / sqrt(mean(s^2) + eps)
 *   add_layer_norm
 *               s   = residual + scale * x            (residual and scale optional)
 *               out = w * (s - mean) * rstd + b,   rstd = 1 / sqrt(mean((s - mean)^2) + eps)
 *   gated_norm  per group of columns:
 *               v   = y * silu(z),  out = w * v * rstd(v)              (gate first, the default)
 *               out = w * y * rstd(y) * silu(z)                        (SSM_NORM_FIRST)
 *   ckpt8       an activation held as int8 values with one power-of-two scale per 32 columns
 *   wgrad       d_W[m][k] = sum_t g[t][m] * X[t][k], X read from its 8-bit checkpoint
 *
 * Layouts: row-major; a row is a token, `cols` channels each.  Activations may be strided by
 * row: `ld_*` is the row stride in elements (0 means cols; at least cols otherwise), so that a
 * tensor may be a slice of a wider one (the gate's half of an input projection).  Parameters w,
 * b, scale and their gradients are fp32 [cols]; mean and rstd are fp32 [rows][cols / group].
 *
 * 8-bit checkpoints ("ckpt8"): q int8 [rows][cols] and e uint8 [rows][ceil(cols / 32)], both
 * contiguous.  Block j of a row holds columns 32 j .. 32 j + 31.  With E = floor(log2(max |v|))
 * over the block, raised to -120 where it is less (or the block is zero),
 *   e = E + 127,   q = round-to-nearest-even(v * 2^(6 - E)) limited to -127 .. 127,
 * and the value kept is q * 2^(E - 6): exact in bf16 and in fp32.  The error of a kept value is
 * at most 2^(E - 7), i.e. max |v| / 128 of its block (2^(E - 6) where |v| > 127 2^(E-6)).  A block
 * that holds an infinity or a NaN is kept as e = 255, q = 0 and reads back as NaN throughout.  A save
 * writes e of 7 .. 255; everything that reads a checkpoint takes any byte below 255 as q 2^(e - 133),
 * so that one filled with zeros holds zeros.
 *
 * Ownership, streams and errors are those of ssm.h: caller-owned device pointers, nothing
 * allocated or synchronised, work enqueued on `stream`, argument errors found on the host before
 * anything is enqueued.  Outputs are overwritten.  Inputs and outputs must not overlap, except
 * that an output may be the same tensor (pointer and stride) as an input of its own type of the
 * norms' forward or backward, element for element (res_out = residual, d_x = d_out, ...).
 * Row statistics and sums over rows are fp32 (the weight gradient's as it says below); a value is
 * rounded to the I/O type once, where it is stored.  Sums run in a fixed order: results are bitwise
 * reproducible.
 */
#ifndef SSM_BLOCK_GB300_H
#define SSM_BLOCK_GB300_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_MAX_NORM_COLS 32768 /* columns of a row of the norms (SSM_ERR_UNSUPPORTED beyond) */
#define SSM_MAX_NORM_ROWS 0x7ff00000 /* rows of the norms; their strides: below 2^31 elements */
#define SSM_CKPT8_BLOCK 32      /* columns that share a scale */

enum {
  SSM_NORM_FIRST = 1u,      /* gated_norm: norm of y, then the gate */
  SSM_WGRAD_ACCUMULATE = 1u /* wgrad: add to d_W instead of overwriting it */
  /* wgrad also takes ssm.h's SSM_DEBUG_NO_WAIT, for tests of the error path only: the warps that take the
     sums out give up at once, as if the bound of their wait had run out */
};

typedef struct {
  long long rows; /* tokens, >= 1 */
  int cols;       /* channels, 1 .. SSM_MAX_NORM_COLS */
  int group;      /* columns per norm, a divisor of cols; 0 means cols */
  int io;         /* ssm_dtype of the activations */
  int res_io;     /* add_norm: ssm_dtype of the residual stream (residual, res_out and their
                     gradients): SSM_F32, or the same as io */
  unsigned flags; /* gated_norm: SSM_NORM_FIRST */
  float eps;      /* > 0, finite */
} ssm_norm_desc;

/* ---- residual add + RMSNorm (before a block) ---------------------------------------------
 * Forward.  Required: desc, x, out.  Optional (NULL): residual (s = scale * x), scale, w,
 * res_out (s in the stream's type), rstd, and the 8-bit checkpoints (each a pair of pointers,
 * both or neither): res_q / res_e of s as res_out stores it (what ssm_add_norm_bwd reads), x_q /
 * x_e of x (what it reads for d_scale), out_q / out_e of out as stored (what ssm_ckpt8_wgrad
 * reads for the projection that follows).  out is normalised from s before its rounding to the
 * stream's type. */
int ssm_add_norm_fwd(const ssm_norm_desc* desc, const void* x, long long ld_x,
                     const void* residual, long long ld_residual, const float* scale,
                     const float* w, void* out, long long ld_out, void* res_out,
                     long long ld_res_out, float* rstd, int8_t* res_q, uint8_t* res_e, int8_t* x_q,
                     uint8_t* x_e, int8_t* out_q, uint8_t* out_e, void* stream);

/* Bytes of scratch the norms' backward needs for `sums` column sums (add_norm: 1, or 2 with
 * d_scale; add_layer_norm: one for each of d_w, d_b and d_scale; gated_norm: 1) on the current device; 0 if
 * the arguments are invalid. */
size_t ssm_norm_bwd_workspace_size(const ssm_norm_desc* desc, int sums);

/* Backward.  Required: d_out, rstd (the forward's), and s as either res (the forward's res_out)
 * or res_q / res_e.  Optional: d_res_out (the gradient that reaches s past the norm; NULL =
 * zero), scale, w (as in the forward), x or x_q / x_e (required with d_scale).  Outputs, each
 * optional: d_res (stream type), d_x (I/O type), d_w, d_scale (requires scale).
 *   n = s rstd,  r = d_res_out + rstd (w d_out - n mean(w d_out n)),
 *   d_res = r,  d_x = scale r,  d_w = sum_rows d_out n,  d_scale = sum_rows r x */
int ssm_add_norm_bwd(const ssm_norm_desc* desc, const void* d_out, long long ld_d_out,
                     const void* d_res_out, long long ld_d_res_out, const void* res,
                     long long ld_res, const int8_t* res_q, const uint8_t* res_e, const void* x,
                     long long ld_x, const int8_t* x_q, const uint8_t* x_e, const float* rstd,
                     const float* scale, const float* w, void* d_res, long long ld_d_res,
                     void* d_x, long long ld_d_x, float* d_w, float* d_scale, void* ws,
                     size_t ws_bytes, void* stream);

/* ---- residual add + layer norm (before a block, or before the head) -------------------------
 * As ssm_add_norm_fwd, with an optional b, and mean and rstd as two optional outputs. */
int ssm_add_layer_norm_fwd(const ssm_norm_desc* desc, const void* x, long long ld_x,
                           const void* residual, long long ld_residual, const float* scale,
                           const float* w, const float* b, void* out, long long ld_out,
                           void* res_out, long long ld_res_out, float* mean, float* rstd,
                           int8_t* res_q, uint8_t* res_e, int8_t* x_q, uint8_t* x_e, int8_t* out_q,
                           uint8_t* out_e, void* stream);

/* As ssm_add_norm_bwd; mean and rstd (the forward's) are both required, d_b is optional.
 *   n = (s - mean) rstd,  a = w d_out,  r = d_res_out + rstd (a - mean(a) - n mean(a n)),
 *   d_res = r,  d_x = scale r,  d_w = sum_rows d_out n,  d_b = sum_rows d_out,
 *   d_scale = sum_rows r x */
int ssm_add_layer_norm_bwd(const ssm_norm_desc* desc, const void* d_out, long long ld_d_out,
                           const void* d_res_out, long long ld_d_res_out, const void* res,
                           long long ld_res, const int8_t* res_q, const uint8_t* res_e,
                           const void* x, long long ld_x, const int8_t* x_q, const uint8_t* x_e,
                           const float* mean, const float* rstd, const float* scale,
                           const float* w, void* d_res, long long ld_d_res, void* d_x,
                           long long ld_d_x, float* d_w, float* d_b, float* d_scale, void* ws,
                           size_t ws_bytes, void* stream);

/* ---- gated RMSNorm (after the scan) --------------------------------------------------------
 * Forward.  Required: y, z, out.  Optional: w, rstd, checkpoints of y, z and out, each by itself (a
 * pair of pointers, both or neither). */
int ssm_gated_norm_fwd(const ssm_norm_desc* desc, const void* y, long long ld_y, const void* z,
                       long long ld_z, const float* w, void* out, long long ld_out, float* rstd,
                       int8_t* y_q, uint8_t* y_e, int8_t* z_q, uint8_t* z_e, int8_t* out_q,
                       uint8_t* out_e, void* stream);

/* Backward.  Required: d_out, rstd (the forward's), y or y_q / y_e, z or z_q / z_e (both tensors
 * or both checkpoints), d_y and d_z.  Optional: w, d_w.
 *   gate first: n = y silu(z) rstd,  dv = rstd (w d_out - n mean(w d_out n)),
 *               d_y = dv silu(z),  d_z = dv y silu'(z),  d_w = sum_rows d_out n
 *   norm first: n = y rstd,  dn = w d_out silu(z),
 *               d_y = rstd (dn - n mean(dn n)),  d_z = w d_out n silu'(z),
 *               d_w = sum_rows d_out n silu(z) */
int ssm_gated_norm_bwd(const ssm_norm_desc* desc, const void* d_out, long long ld_d_out,
                       const void* y, long long ld_y, const int8_t* y_q, const uint8_t* y_e,
                       const void* z, long long ld_z, const int8_t* z_q, const uint8_t* z_e,
                       const float* rstd, const float* w, void* d_y, long long ld_d_y, void* d_z,
                       long long ld_d_z, float* d_w, void* ws, size_t ws_bytes, void* stream);

/* ---- 8-bit activation checkpoints ----------------------------------------------------------
 * Save: x [rows][cols] (io) -> q, e.  Load: q, e -> out [rows][cols] (io). */
int ssm_ckpt8_save(const void* x, long long ld_x, int8_t* q, uint8_t* e, long long rows, int cols,
                   int io, void* stream);
int ssm_ckpt8_load(const int8_t* q, const uint8_t* e, void* out, long long ld_out, long long rows,
                   int cols, int io, void* stream);

/* Weight gradient of a projection from its input's checkpoint:
 *   d_W[i][j] (+)= sum_{t < tokens} g[t][i] * X[t][j],   i < m, j < k
 * g [tokens][m] (io), X = the ckpt8 (q [tokens][k], e [tokens][ceil(k / 32)]), d_W [m][k] fp32
 * contiguous; tokens up to 2^29.  It runs on the tensor cores: kept values and bf16 g are bf16 numbers,
 * fp32 g is split into three exactly, so that every product is exact.  Sums are fp32, truncated by
 * the tensor cores within 1024 tokens (64 additions) and rounded to nearest between them: about
 * (64 + tokens / 2048) 2^-23 of sum |g X| off at worst, (64 + 3 tokens / 2048) 2^-23 with fp32 g.
 * Workspace: ssm_ckpt8_wgrad_workspace_size bytes (at least 256: its first word is a status word,
 * read with ssm_scan_status).  Where a bounded wait gave up (SSM_ERR_TIMEOUT there), the tiles of d_W that
 * it concerns are NaN.  aligned: the rows of g (pointer and ld_g * element size; fp32 g may lie
 * anywhere) and q's pointer are 16-byte aligned; 0 asks for room for copies that are.  Each of the two is
 * copied only where it is not aligned itself; with bf16 g, m a multiple of 8 and k of 16 an aligned call
 * needs no copies. */
size_t ssm_ckpt8_wgrad_workspace_size(long long tokens, int m, int k, int io, int aligned);
int ssm_ckpt8_wgrad(const void* g, long long ld_g, const int8_t* q, const uint8_t* e, float* d_W,
                    long long tokens, int m, int k, int io, unsigned flags, void* ws,
                    size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
