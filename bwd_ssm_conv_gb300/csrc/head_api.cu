// head_api.cu -- the extern "C" entry points of include/ssm_head.h: argument validation on the host, the
// layout of the workspace and the order of the launches.  Nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "head.cuh"

namespace {

using namespace ssm;

constexpr long long kMaxTotal = 1LL << 40;  // elements between a tensor's first and last row
constexpr long long kMaxPiece = 256LL << 20;  // bytes of G at a time (a tile's columns at least)

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

// Splits of a sum of `stages` stages over `tiles` tiles' pairs of CTAs: the number that the slowest pair
// needs least time with, in stages (half a microsecond and less), where a split costs its tiles' way to
// memory and back besides.
struct Split {
  int splits, per;
};
Split split_of(long long tiles, int stages, double part_bytes, int sms) {
  const long long pairs = sms / 2 > 0 ? sms / 2 : 1;
  constexpr double kStageBytes = 1.5e6;  // that memory moves in a stage's time
  constexpr int kUnit = 3;               // stages that a unit costs by itself
  Split best{1, stages};
  double least = 0.0;
  for (int s = 1; s <= 64 && s <= stages; s++) {
    const int per = (stages + s - 1) / s;
    if ((stages + per - 1) / per != s) continue;
    const double time = (double)((tiles * s + pairs - 1) / pairs) * (per + kUnit) +
                        (s > 1 ? 2.0 * s * part_bytes / kStageBytes : 0.0);
    if (s == 1 || time < least) least = time, best = {s, per};
  }
  return best;
}

// The workspace, by bytes from its start.
struct Plan {
  size_t pos, src, idx, p, known, valid, rl, rg, h, w, stats, zt, g, dh, dw, bytes;
  int planes, tiles, piece, pieces;
  Split s_h, s_w;
};
Plan plan_of(const ssm_head_desc& d, int grads, bool copy_w, int sms) {
  Plan p{};
  const long long T = d.rows, Tp = pad_rows(T), n_e = d.entries ? d.entries : 1;
  const int Dp = pad8(d.cols);
  p.planes = d.io == SSM_F32 ? 3 : 1;
  p.tiles = (d.vocab + kHeadTile - 1) / kHeadTile;
  size_t at = 256;
  const auto take = [&](size_t n) {
    const size_t was = at;
    at += align_up(n, 256);
    return was;
  };
  p.pos = take(4 * T);
  p.src = take(4 * Tp);
  p.idx = take(4 * T * n_e);
  if (d.entries) {
    p.p = take(4 * T * n_e);
    p.known = take(4 * T);
    p.valid = take(T);
  }
  p.h = take((size_t)2 * p.planes * Tp * Dp);
  if (copy_w) p.w = take((size_t)2 * p.planes * d.vocab * Dp);
  if (!grads) {
    p.stats = take((size_t)8 * 2 * p.tiles * Tp);
    p.zt = take(4 * T * n_e);
  } else {
    p.rl = take(4 * Tp);
    p.rg = take(4 * Tp);
    // pieces of the vocabulary, alike
    long long most = kMaxPiece / (2 * p.planes * Tp) / kHeadTile;
    if (most < 1) most = 1;
    p.pieces = (int)((p.tiles + most - 1) / most);
    p.piece = (p.tiles + p.pieces - 1) / p.pieces * kHeadTile;
    p.pieces = (d.vocab + p.piece - 1) / p.piece;
    p.g = take((size_t)2 * p.planes * Tp * p.piece);
    const long long rows = (T + kHeadTile - 1) / kHeadTile,
                    cols = (d.cols + kHeadTile - 1) / kHeadTile;
    if (grads & 1) {
      p.s_h = split_of(rows * cols, p.piece / kHeadBlock, 4.0 * Tp * Dp, sms);
      p.dh = take((size_t)4 * p.s_h.splits * Tp * Dp);
    }
    if (grads & 2) {
      p.s_w = split_of(p.piece / kHeadTile * cols, (int)(Tp / kHeadBlock), 4.0 * p.piece * Dp, sms);
      if (p.s_w.splits > 1) p.dw = take((size_t)4 * p.s_w.splits * p.piece * Dp);
    }
  }
  p.bytes = at;
  return p;
}

int check(const ssm_head_desc* d, bool distill) {
  if (!d || d->rows <= 0 || d->cols <= 0 || d->vocab <= 0 || !io_size(d->io))
    return SSM_ERR_INVALID_ARG;
  if (d->flags & ~(unsigned)SSM_DEBUG_NO_WAIT) return SSM_ERR_INVALID_ARG;
  if (distill) {
    if (d->entries <= 0 || !io_size(d->entry_io)) return SSM_ERR_INVALID_ARG;
    if (!(d->temperature > 0.0f) || isinf(d->temperature)) return SSM_ERR_INVALID_ARG;
    if (d->entries > SSM_MAX_HEAD_ENTRIES) return SSM_ERR_UNSUPPORTED;
  } else if (d->entries) {
    return SSM_ERR_INVALID_ARG;
  }
  if (d->rows > SSM_MAX_HEAD_ROWS || d->cols > SSM_MAX_HEAD_COLS || d->vocab > SSM_MAX_HEAD_VOCAB)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// One call, its arguments as they come.
struct Call {
  const ssm_head_desc* desc;
  const void* h;
  long long ld_h;
  const void* w;
  long long ld_w;
  const int64_t* target;  // or
  const int64_t* t_idx;
  const void* t_logit;
  float* loss;  // forward
  float* lse_out;
  const float* lse;  // backward
  const float* d_loss;
  void* d_h;
  long long ld_d_h;
  void* d_w;
  void* ws;
  size_t ws_bytes;
  void* stream;
};

int run(Call c, bool distill, bool backward) {
  if (const int rc = check(c.desc, distill)) return rc;
  const ssm_head_desc& d = *c.desc;
  const size_t size = io_size(d.io);
  if (!c.h || !c.w || (distill ? !c.t_idx || !c.t_logit : !c.target)) return SSM_ERR_INVALID_ARG;
  if (backward ? !c.lse || !c.d_loss || (!c.d_h && !c.d_w) : !c.loss) return SSM_ERR_INVALID_ARG;
  if (c.ld_h == 0) c.ld_h = d.cols;
  if (c.ld_w == 0) c.ld_w = d.cols;
  if (c.ld_d_h == 0) c.ld_d_h = d.cols;
  if (c.ld_h < d.cols || c.ld_w < d.cols || c.ld_d_h < d.cols) return SSM_ERR_INVALID_ARG;
  for (const void* p : {c.h, c.w, (const void*)c.d_h, (const void*)c.d_w})
    if (p && !aligned(p, size)) return SSM_ERR_INVALID_ARG;
  for (const void* p : {(const void*)c.loss, (const void*)c.lse_out, (const void*)c.lse,
                        (const void*)c.d_loss})
    if (p && !aligned(p, 4)) return SSM_ERR_INVALID_ARG;
  for (const int64_t* p : {c.target, c.t_idx})
    if (p && !aligned(p, 8)) return SSM_ERR_INVALID_ARG;
  if (distill && !aligned(c.t_logit, io_size(d.entry_io))) return SSM_ERR_INVALID_ARG;
  if (c.ld_h > kMaxTotal / d.rows || c.ld_d_h > kMaxTotal / d.rows || c.ld_w > kMaxTotal / d.vocab)
    return SSM_ERR_UNSUPPORTED;
  const int sms = num_sms();
  if (sms <= 0) return SSM_ERR_CUDA;
  const bool copy_w =
      d.io == SSM_F32 || !aligned(c.w, 16) || c.ld_w * size % 16 != 0;
  const int grads = backward ? (c.d_h ? 1 : 0) | (c.d_w ? 2 : 0) : 0;
  const Plan p = plan_of(d, grads, copy_w, sms);
  if (!c.ws || !aligned(c.ws, 256) || c.ws_bytes < p.bytes) return SSM_ERR_WORKSPACE;

  cudaStream_t st = (cudaStream_t)c.stream;
  char* ws = (char*)c.ws;
  const long long Tp = pad_rows(d.rows);
  const int Dp = pad8(d.cols);
  int* idx = (int*)(ws + p.idx);
  float* prob = d.entries ? (float*)(ws + p.p) : nullptr;
  float* known = d.entries ? (float*)(ws + p.known) : nullptr;
  uint8_t* valid = d.entries ? (uint8_t*)(ws + p.valid) : nullptr;
  HeadRows r{(HeadState*)ws, (int*)(ws + p.pos), (int*)(ws + p.src), (float*)(ws + p.rl),
             (float*)(ws + p.rg), (__nv_bfloat16*)(ws + p.h)};
#define SSM_DO(call) \
  if ((call) != cudaSuccess) return SSM_ERR_CUDA
  if (distill) SSM_DO(launch_head_entries(d, c.t_idx, c.t_logit, idx, prob, known, valid, st));
  SSM_DO(launch_head_begin(d, c.target, valid, backward ? c.d_loss : nullptr, idx, r, !distill, st));
  SSM_DO(launch_head_pack(d, c.h, c.ld_h, backward ? c.lse : nullptr, c.d_loss, r, sms, st));
  const HeadMatrix h{r.h, Tp, Dp, Tp * Dp, d.cols};
  HeadMatrix w{(const __nv_bfloat16*)c.w, d.vocab, c.ld_w, 0, d.cols};
  if (copy_w) {
    __nv_bfloat16* to = (__nv_bfloat16*)(ws + p.w);
    SSM_DO(launch_head_copy_w(d, c.w, c.ld_w, to, sms, st));
    w = {to, d.vocab, Dp, (long long)d.vocab * Dp, d.cols};
  }
  if (!backward) {
    float2* stats = (float2*)(ws + p.stats);
    float* zt = (float*)(ws + p.zt);
    SSM_DO(launch_head_logits(d, h, w, r, idx, stats, zt, sms, st));
    SSM_DO(launch_head_loss(d, stats, 2 * p.tiles, zt, prob, known, r, c.loss, c.lse_out, st));
    return SSM_OK;
  }
  __nv_bfloat16* gp = (__nv_bfloat16*)(ws + p.g);
  float *dh = (float*)(ws + p.dh), *dw = p.dw ? (float*)(ws + p.dw) : nullptr;
  const HeadMatrix g{gp, Tp, p.piece, Tp * p.piece, p.piece};
  for (int i = 0; i < p.pieces; i++) {
    const int v0 = i * p.piece, n = d.vocab - v0 < p.piece ? d.vocab - v0 : p.piece;
    SSM_DO(launch_head_grad(d, h, w, r, idx, prob, gp, v0, p.piece, sms, st));
    if (c.d_w) {
      SSM_DO(launch_head_dw(d, g, h, r, c.d_w, dw, p.s_w.splits, p.s_w.per, v0, n, sms, st));
      if (dw)
        SSM_DO(launch_head_sum_w(d, dw, p.s_w.per, p.piece, r, c.d_w, v0, n, sms, st));
    }
    if (c.d_h)
      SSM_DO(launch_head_dh(d, g, w, r, dh, p.s_h.splits, p.s_h.per, v0, i > 0, sms, st));
  }
  SSM_DO(launch_head_finish(d, dh, p.s_h.splits, r, c.d_h, c.ld_d_h, c.d_w, sms, st));
#undef SSM_DO
  return SSM_OK;
}

}  // namespace

extern "C" {

size_t ssm_head_workspace_size(const ssm_head_desc* desc, int grads, int aligned_w) {
  if (grads < 0 || grads > 3 || !desc || check(desc, desc->entries != 0) != SSM_OK) return 0;
  const int sms = num_sms();
  if (sms <= 0) return 0;
  return plan_of(*desc, grads, desc->io == SSM_F32 || !aligned_w, sms).bytes;
}

int ssm_head_ce_fwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                    long long ld_w, const int64_t* target, float* loss, float* lse, void* ws,
                    size_t ws_bytes, void* stream) {
  Call c{desc, h, ld_h, w, ld_w, target};
  c.loss = loss, c.lse_out = lse;
  c.ws = ws, c.ws_bytes = ws_bytes, c.stream = stream;
  return run(c, false, false);
}

int ssm_head_distill_fwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                         long long ld_w, const int64_t* t_idx, const void* t_logit, float* loss,
                         float* lse, void* ws, size_t ws_bytes, void* stream) {
  Call c{desc, h, ld_h, w, ld_w, nullptr, t_idx, t_logit};
  c.loss = loss, c.lse_out = lse;
  c.ws = ws, c.ws_bytes = ws_bytes, c.stream = stream;
  return run(c, true, false);
}

int ssm_head_ce_bwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                    long long ld_w, const int64_t* target, const float* lse, const float* d_loss,
                    void* d_h, long long ld_d_h, void* d_w, void* ws, size_t ws_bytes,
                    void* stream) {
  Call c{desc, h, ld_h, w, ld_w, target};
  c.lse = lse, c.d_loss = d_loss, c.d_h = d_h, c.ld_d_h = ld_d_h, c.d_w = d_w;
  c.ws = ws, c.ws_bytes = ws_bytes, c.stream = stream;
  return run(c, false, true);
}

int ssm_head_distill_bwd(const ssm_head_desc* desc, const void* h, long long ld_h, const void* w,
                         long long ld_w, const int64_t* t_idx, const void* t_logit,
                         const float* lse, const float* d_loss, void* d_h, long long ld_d_h,
                         void* d_w, void* ws, size_t ws_bytes, void* stream) {
  Call c{desc, h, ld_h, w, ld_w, nullptr, t_idx, t_logit};
  c.lse = lse, c.d_loss = d_loss, c.d_h = d_h, c.ld_d_h = ld_d_h, c.d_w = d_w;
  c.ws = ws, c.ws_bytes = ws_bytes, c.stream = stream;
  return run(c, true, true);
}

}  // extern "C"
