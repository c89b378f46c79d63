// block_api.cu -- the extern "C" entry points of include/ssm_block.h: argument validation on the
// host, then the launch.  Nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "block.cuh"
#include "ssm_block.h"

namespace {

constexpr long long kMaxTotal = 1LL << 40;
constexpr long long kMaxWgrad = 1LL << 38;  // elements of g and of X there
constexpr long long kMaxTokens = 1LL << 29;  // of the weight gradient
constexpr long long kMaxStride = 0x7fffffff;  // of the norms' rows
constexpr int kMaxDim = 1 << 20;  // m and k of the weight gradient, columns of a checkpoint

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t io_size(int io) { return io == SSM_BF16 ? 2 : (io == SSM_F32 ? 4 : 0); }

// SMs of the current device, asked for once per device (the answer never changes).
int num_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// An activation argument: its stride resolved (0: cols), its alignment checked, and whether 8
// columns at a time can be read from every row of it.
struct Rows {
  int cols;
  bool ok, vec;
  void arg(const void* p, long long& ld, int io) {
    if (!p) return;
    if (ld == 0) ld = cols;
    const size_t sz = io_size(io);
    if (ld < cols || !aligned(p, sz)) ok = false;
    if (ld % 8 != 0 || !aligned(p, 8 * sz)) vec = false;
  }
  void kept(const void* q, const void* e) {  // both or neither
    if ((q == nullptr) != (e == nullptr)) ok = false;
    if (q && !aligned(q, 8)) vec = false;
  }
  void f32(const void* p) {  // a parameter or its gradient
    if (p && !aligned(p, 4)) ok = false;
    if (p && !aligned(p, 16)) vec = false;
  }
};

int norm_check(const ssm_norm_desc* d, bool add, int* group) {
  if (!d || d->rows <= 0 || d->cols <= 0 || d->group < 0 || !io_size(d->io))
    return SSM_ERR_INVALID_ARG;
  *group = d->group ? d->group : d->cols;
  if (*group > d->cols || d->cols % *group != 0) return SSM_ERR_INVALID_ARG;
  if (!(d->eps > 0.0f) || isinf(d->eps)) return SSM_ERR_INVALID_ARG;
  if (add) {
    if (d->flags || *group != d->cols) return SSM_ERR_INVALID_ARG;
    if (d->res_io != SSM_F32 && d->res_io != d->io) return SSM_ERR_INVALID_ARG;
  } else if (d->flags & ~(unsigned)SSM_NORM_FIRST) {
    return SSM_ERR_INVALID_ARG;
  }
  if (d->cols > SSM_MAX_NORM_COLS || d->rows > SSM_MAX_NORM_ROWS) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

bool ld_fits(long long ld, long long rows) { return ld <= kMaxTotal / rows; }

int status_of(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

}  // namespace

extern "C" {

int ssm_add_norm_fwd(const ssm_norm_desc* desc, const void* x, long long ld_x,
                     const void* residual, long long ld_residual, const float* scale,
                     const float* w, void* out, long long ld_out, void* res_out,
                     long long ld_res_out, float* rstd, int8_t* res_q, uint8_t* res_e, int8_t* x_q,
                     uint8_t* x_e, int8_t* out_q, uint8_t* out_e, void* stream) {
  int group;
  int rc = norm_check(desc, true, &group);
  if (rc != SSM_OK) return rc;
  if (!x || !out) return SSM_ERR_INVALID_ARG;
  const int io = desc->io, rio = desc->res_io;
  Rows r{desc->cols, true, desc->cols % 8 == 0};
  r.arg(x, ld_x, io);
  r.arg(residual, ld_residual, rio);
  r.arg(out, ld_out, io);
  r.arg(res_out, ld_res_out, rio);
  r.kept(res_q, res_e);
  r.kept(x_q, x_e);
  r.kept(out_q, out_e);
  r.f32(scale);
  r.f32(w);
  if (!r.ok || (rstd && !aligned(rstd, 4))) return SSM_ERR_INVALID_ARG;
  for (long long ld : {ld_x, ld_residual, ld_out, ld_res_out})
    if (ld > kMaxStride) return SSM_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  ssm::AddNormFwd a{(int)desc->rows, desc->cols, desc->eps, x, residual, scale, w, out, res_out,
                    rstd, (int)ld_x, (int)ld_residual, (int)ld_out, (int)ld_res_out, res_q, x_q,
                    out_q, res_e, x_e, out_e};
  return status_of(ssm::launch_add_norm_fwd(a, io, rio, r.vec, sms, (cudaStream_t)stream));
}

size_t ssm_norm_bwd_workspace_size(const ssm_norm_desc* desc, int sums) {
  int group;
  if (sums < 0 || sums > 2) return 0;
  if (norm_check(desc, false, &group) != SSM_OK && norm_check(desc, true, &group) != SSM_OK)
    return 0;
  const int sms = num_sms();
  if (sms <= 0) return 0;
  return 256 + ssm::column_sums_bytes(desc->rows, group, desc->cols / group, sms, sums);
}

int ssm_add_norm_bwd(const ssm_norm_desc* desc, const void* d_out, long long ld_d_out,
                     const void* d_res_out, long long ld_d_res_out, const void* res,
                     long long ld_res, const int8_t* res_q, const uint8_t* res_e, const void* x,
                     long long ld_x, const int8_t* x_q, const uint8_t* x_e, const float* rstd,
                     const float* scale, const float* w, void* d_res, long long ld_d_res,
                     void* d_x, long long ld_d_x, float* d_w, float* d_scale, void* ws,
                     size_t ws_bytes, void* stream) {
  int group;
  int rc = norm_check(desc, true, &group);
  if (rc != SSM_OK) return rc;
  if (!d_out || !rstd || (!d_res && !d_x && !d_w && !d_scale)) return SSM_ERR_INVALID_ARG;
  if ((res != nullptr) == (res_q != nullptr)) return SSM_ERR_INVALID_ARG;  // one of the two
  if (x && x_q) return SSM_ERR_INVALID_ARG;
  if (d_scale && (!scale || (!x && !x_q))) return SSM_ERR_INVALID_ARG;
  const int io = desc->io, rio = desc->res_io;
  Rows r{desc->cols, true, desc->cols % 8 == 0};
  r.arg(d_out, ld_d_out, io);
  r.arg(d_res_out, ld_d_res_out, rio);
  r.arg(res, ld_res, rio);
  r.arg(x, ld_x, io);
  r.arg(d_res, ld_d_res, rio);
  r.arg(d_x, ld_d_x, io);
  r.kept(res_q, res_e);
  r.kept(x_q, x_e);
  r.f32(scale);
  r.f32(w);
  if (!r.ok || !aligned(rstd, 4) || (d_w && !aligned(d_w, 4)) || (d_scale && !aligned(d_scale, 4)))
    return SSM_ERR_INVALID_ARG;
  for (long long ld : {ld_d_out, ld_d_res_out, ld_res, ld_x, ld_d_res, ld_d_x})
    if (ld > kMaxStride) return SSM_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  const int sums = (d_w ? 1 : 0) + (d_scale ? 1 : 0);
  if (sums && (!ws || !aligned(ws, 256) ||
               ws_bytes < 256 + ssm::column_sums_bytes(desc->rows, group, 1, sms, sums)))
    return SSM_ERR_WORKSPACE;
  ssm::AddNormBwd a{(int)desc->rows, desc->cols, d_out, d_res_out, res, x, (int)ld_d_out,
                    (int)ld_d_res_out, (int)ld_res, (int)ld_x, res_q, x_q, res_e, x_e, rstd, scale,
                    w, d_res, d_x, (int)ld_d_res, (int)ld_d_x, d_w, d_scale,
                    sums ? (float*)((char*)ws + 256) : nullptr};
  return status_of(ssm::launch_add_norm_bwd(a, io, rio, r.vec, sms, (cudaStream_t)stream));
}

int ssm_gated_norm_fwd(const ssm_norm_desc* desc, const void* y, long long ld_y, const void* z,
                       long long ld_z, const float* w, void* out, long long ld_out, float* rstd,
                       int8_t* y_q, uint8_t* y_e, int8_t* z_q, uint8_t* z_e, int8_t* out_q,
                       uint8_t* out_e, void* stream) {
  int group;
  int rc = norm_check(desc, false, &group);
  if (rc != SSM_OK) return rc;
  if (!y || !z || !out) return SSM_ERR_INVALID_ARG;
  const int io = desc->io, cols = desc->cols;
  Rows r{cols, true, group % 8 == 0};
  r.arg(y, ld_y, io);
  r.arg(z, ld_z, io);
  r.arg(out, ld_out, io);
  r.kept(y_q, y_e);
  r.kept(z_q, z_e);
  r.kept(out_q, out_e);
  r.f32(w);
  if (!r.ok || (rstd && !aligned(rstd, 4))) return SSM_ERR_INVALID_ARG;
  for (long long ld : {ld_y, ld_z, ld_out})
    if (ld > kMaxStride) return SSM_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const int norm_first = (desc->flags & SSM_NORM_FIRST) ? 1 : 0;
  ssm::GatedNormFwd a{(int)desc->rows, cols, group, norm_first, desc->eps, y, z, w, out, (int)ld_y,
                      (int)ld_z, (int)ld_out, rstd, y_q, z_q, out_q, y_e, z_e, out_e};
  // Blocks of 32 columns that straddle groups belong to no group's threads, and the norm's kernel
  // keeps y and z together or not at all (a branch for each costs the pair 0.8 % of 32768 x 1536):
  // such checkpoints are saved by their own kernel, the inputs' before out is written.
  const bool straddle = group != cols && group % SSM_CKPT8_BLOCK != 0;
  if (straddle || !y_q != !z_q) {
    a.y_q = a.z_q = nullptr;
    cudaError_t e = cudaSuccess;
    if (y_q) e = ssm::launch_ckpt8_save(y, ld_y, y_q, y_e, desc->rows, cols, io, sms, st);
    if (e == cudaSuccess && z_q)
      e = ssm::launch_ckpt8_save(z, ld_z, z_q, z_e, desc->rows, cols, io, sms, st);
    if (e != cudaSuccess) return SSM_ERR_CUDA;
  }
  if (straddle) a.out_q = nullptr;
  cudaError_t e = ssm::launch_gated_norm_fwd(a, io, r.vec, sms, st);
  if (e == cudaSuccess && straddle && out_q)
    e = ssm::launch_ckpt8_save(out, ld_out, out_q, out_e, desc->rows, cols, io, sms, st);
  return status_of(e);
}

int ssm_gated_norm_bwd(const ssm_norm_desc* desc, const void* d_out, long long ld_d_out,
                       const void* y, long long ld_y, const int8_t* y_q, const uint8_t* y_e,
                       const void* z, long long ld_z, const int8_t* z_q, const uint8_t* z_e,
                       const float* rstd, const float* w, void* d_y, long long ld_d_y, void* d_z,
                       long long ld_d_z, float* d_w, void* ws, size_t ws_bytes, void* stream) {
  int group;
  int rc = norm_check(desc, false, &group);
  if (rc != SSM_OK) return rc;
  if (!d_out || !rstd || !d_y || !d_z) return SSM_ERR_INVALID_ARG;
  const bool kept = y_q != nullptr;
  if (kept ? (y || z || !z_q) : (!y || !z || z_q)) return SSM_ERR_INVALID_ARG;
  const int io = desc->io, cols = desc->cols;
  Rows r{cols, true, group % 8 == 0};
  r.arg(d_out, ld_d_out, io);
  r.arg(y, ld_y, io);
  r.arg(z, ld_z, io);
  r.arg(d_y, ld_d_y, io);
  r.arg(d_z, ld_d_z, io);
  r.kept(y_q, y_e);
  r.kept(z_q, z_e);
  r.f32(w);
  if (!r.ok || !aligned(rstd, 4) || (d_w && !aligned(d_w, 4))) return SSM_ERR_INVALID_ARG;
  for (long long ld : {ld_d_out, ld_y, ld_z, ld_d_y, ld_d_z})
    if (ld > kMaxStride) return SSM_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  if (d_w && (!ws || !aligned(ws, 256) ||
              ws_bytes < 256 + ssm::column_sums_bytes(desc->rows, group, cols / group, sms, 1)))
    return SSM_ERR_WORKSPACE;
  ssm::GatedNormBwd a{(int)desc->rows, cols, group, (desc->flags & SSM_NORM_FIRST) ? 1 : 0, d_out, y, z,
                      (int)ld_d_out, (int)ld_y, (int)ld_z, y_q, z_q, y_e, z_e, rstd, w, d_y, d_z,
                      (int)ld_d_y, (int)ld_d_z,
                      d_w, d_w ? (float*)((char*)ws + 256) : nullptr};
  return status_of(ssm::launch_gated_norm_bwd(a, io, r.vec, sms, (cudaStream_t)stream));
}

static int ckpt8_check(const void* act, long long& ld, const void* q, const void* e,
                       long long rows, int cols, int io) {
  if (!act || !q || !e || rows <= 0 || cols <= 0 || !io_size(io)) return SSM_ERR_INVALID_ARG;
  if (ld == 0) ld = cols;
  if (ld < cols || !aligned(act, io_size(io))) return SSM_ERR_INVALID_ARG;
  if (cols > kMaxDim || !ld_fits(ld, rows)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

int ssm_ckpt8_save(const void* x, long long ld_x, int8_t* q, uint8_t* e, long long rows, int cols,
                   int io, void* stream) {
  int rc = ckpt8_check(x, ld_x, q, e, rows, cols, io);
  if (rc != SSM_OK) return rc;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  return status_of(
      ssm::launch_ckpt8_save(x, ld_x, q, e, rows, cols, io, sms, (cudaStream_t)stream));
}

int ssm_ckpt8_load(const int8_t* q, const uint8_t* e, void* out, long long ld_out, long long rows,
                   int cols, int io, void* stream) {
  int rc = ckpt8_check(out, ld_out, q, e, rows, cols, io);
  if (rc != SSM_OK) return rc;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  return status_of(
      ssm::launch_ckpt8_load(q, e, out, ld_out, rows, cols, io, sms, (cudaStream_t)stream));
}

static int wgrad_check(long long tokens, int m, int k, int io) {
  if (tokens <= 0 || m <= 0 || k <= 0 || !io_size(io)) return SSM_ERR_INVALID_ARG;
  if (m > kMaxDim || k > kMaxDim || tokens > kMaxTokens || tokens > kMaxWgrad / m ||
      tokens > kMaxWgrad / k)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

size_t ssm_ckpt8_wgrad_workspace_size(long long tokens, int m, int k, int io, int aligned) {
  if (wgrad_check(tokens, m, k, io) != SSM_OK) return 0;
  const int sms = num_sms();
  return sms <= 0 ? 0 : ssm::wgrad_ws_bytes(tokens, m, k, io, aligned != 0, sms);
}

int ssm_ckpt8_wgrad(const void* g, long long ld_g, const int8_t* q, const uint8_t* e, float* d_W,
                    long long tokens, int m, int k, int io, unsigned flags, void* ws,
                    size_t ws_bytes, void* stream) {
  int rc = wgrad_check(tokens, m, k, io);
  if (rc != SSM_OK) return rc;
  if (!g || !q || !e || !d_W || (flags & ~(unsigned)(SSM_WGRAD_ACCUMULATE | SSM_DEBUG_NO_WAIT)))
    return SSM_ERR_INVALID_ARG;
  if (ld_g == 0) ld_g = m;
  if (ld_g < m || !aligned(g, io_size(io)) || !aligned(d_W, 4)) return SSM_ERR_INVALID_ARG;
  if (ld_g > kMaxWgrad / tokens) return SSM_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  ssm::Wgrad a{g, ld_g, q, e, d_W, tokens, m, k, io, (flags & SSM_WGRAD_ACCUMULATE) ? 1 : 0,
               (flags & SSM_DEBUG_NO_WAIT) ? 1 : 0};
  if (!ws || !aligned(ws, 256) ||
      ws_bytes < ssm::wgrad_ws_bytes(a, sms))
    return SSM_ERR_WORKSPACE;
  return status_of(ssm::launch_wgrad(a, ws, sms, (cudaStream_t)stream));
}

}  // extern "C"
