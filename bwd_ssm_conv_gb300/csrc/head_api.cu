// head_api.cu -- the extern "C" entry points of include/ssm_head.h: argument validation on the host, the
// layout of the workspace and the order of the launches.  Nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "head.cuh"

namespace {

using namespace ssm;

constexpr long long kMaxTotal = 1LL << 40;  // elements between a tensor's first and last row
constexpr long long kMaxStride = 1LL << 40;  // bytes between two rows that TMA copies: below this
constexpr long long kMaxLogits = 1LL << 40;  // rows times words: tiles are counted in 32 bits
// Bytes of G at a time (a tile's columns at least).  Fewer and larger pieces leave fewer ends of launches with
// idle SMs: 16384 x 1024 over 32768 words 2.97 ms at 96 MiB, 2.76 at 256, 2.64 at 512, 2.66 at 1024.
constexpr long long kMaxPiece = 512LL << 20;

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

// ---- how the products are cut ---------------------------------------------------------------------
// Costs are in stages, the time of a 256 x 256 tile's step over 64 of the sum (six products for fp32).
constexpr long long kFewRounds = 5;  // of tiles on the pairs of CTAs: below, their widths and splits are chosen
double unit_cost(int io) { return io == SSM_F32 ? 0.7 : 3.0; }           // of a unit by itself
double stage_bytes(int io) { return io == SSM_F32 ? 9.0e6 : 1.5e6; }     // that memory moves meanwhile
double tile_cost(int tile_n, int io) {
  if (tile_n == kHeadTile) return 1.0;
  if (tile_n == 192) return io == SSM_F32 ? 0.8 : 0.85;
  return io == SSM_F32 ? 0.55 : 0.65;
}

// Units of one or two kinds are dealt out to the pairs of CTAs in turn, the first kind first: the time of
// the pair with the most to do.
double dealt(long long n0, double c0, long long n1, double c1, long long pairs) {
  double most = 0.0;
  const auto of = [&](long long p) {  // pair p's units: those u with u % pairs == p
    const long long a = p < n0 ? (n0 - 1 - p) / pairs + 1 : 0,
                    b = p < n0 + n1 ? (n0 + n1 - 1 - p) / pairs + 1 : 0;
    const double time = (double)a * c0 + (double)(b - a) * c1;
    if (time > most) most = time;
  };
  of(0);
  of(n0 % pairs);
  if (n0 % pairs) of(n0 % pairs - 1);
  const long long end = (n0 + n1) % pairs;
  of(end ? end - 1 : pairs - 1);
  return most;
}

// Tiles of Z: narrower ones where there are few, as the last round then leaves a good part of the pairs idle.
// The sums' warps of fp32 kGrad store G while no products run.
HeadTiles tiles_of(long long rows, int cols, int words, int io, bool grad, int sms) {
  const int pairs = sms / 2 > 0 ? sms / 2 : 1, stages = (cols + kHeadBlock - 1) / kHeadBlock;
  HeadTiles t{words, pairs};
  if ((rows + kHeadTile - 1) / kHeadTile * ((words + kHeadTile - 1) / kHeadTile) > kFewRounds * pairs)
    t.words = 0;
  for (int i = 0; i < 3; i++) {
    const int tile = kHeadTile - 64 * i;
    const double unit = io == SSM_F32 && grad ? 3.0 * tile / kHeadTile : unit_cost(io);
    t.cost[i] = (float)(stages * tile_cost(tile, io) + unit);
  }
  return t;
}

struct Cuts {
  HeadCut h, w;
  bool h_first;
};
// The two products with G: pairs of numbers of splits, and both widths, as far as more units than a few for
// each pair of CTAs could help.
Cuts cuts_of(long long rows, int cols, int piece, int io, bool fine, int grads, bool several, int sms) {
  const long long pairs = sms / 2 > 0 ? sms / 2 : 1, padded = pad_rows(rows);
  const int terms = fine ? 2 : 1;  // a stage for each
  const int st_h = piece / kHeadBlock * terms, st_w = (int)(padded / kHeadBlock) * terms;
  const long long m_h = (rows + kHeadTile - 1) / kHeadTile, m_w = piece / kHeadTile;
  const double mb_h = 4.0 * padded * pad8(cols), mb_w = 4.0 * piece * pad8(cols);
  const auto per_of = [](int stages, int splits) { return (stages + splits - 1) / splits; };
  Cuts best{};
  double least = -1.0;
  static constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64};
  const long long enough = kFewRounds * pairs;
  for (int tile : {256, 128}) {
    const long long n = (cols + tile - 1) / tile;
    if (tile == 128 && m_w * n > enough && m_h * n > enough) break;
    for (int sw : kSplits) {
      if (sw > 1 && (!(grads & 2) || sw > st_w || m_w * n * sw > enough)) break;
      const int pw = per_of(st_w, sw);
      if (per_of(st_w, pw) != sw) continue;
      for (int sh : kSplits) {
        if (sh > 1 && (!(grads & 1) || sh > st_h || m_h * n * sh > enough)) break;
        const int ph = per_of(st_h, sh);
        if (per_of(st_h, ph) != sh) continue;
        const long long nw = grads & 2 ? m_w * n * sw : 0, nh = grads & 1 ? m_h * n * sh : 0;
        const double cw = pw * tile_cost(tile, io) + unit_cost(io),
                     ch = ph * tile_cost(tile, io) + unit_cost(io);
        const bool h_first = ch > cw;
        double time = h_first ? dealt(nh, ch, nw, cw, pairs) : dealt(nw, cw, nh, ch, pairs);
        // the splits' sums: written and read, those of d_h once for each piece and under its products
        if ((grads & 1) && (several || sh > 1))
          time += sh * mb_h * (several ? 1.0 : 2.0) / stage_bytes(io);
        if (sw > 1) time += 2.0 * sw * mb_w / stage_bytes(io);
        if (least < 0.0 || time < least)
          least = time, best = {{tile, sh, ph}, {tile, sw, pw}, h_first};
      }
    }
  }
  return best;
}

// The workspace, by bytes from its start.
struct Plan {
  size_t pos, src, idx, p, known, table, valid, rl, rg, h, w, stats, zt, g, dh, dw, bytes;
  int planes, n_stats, piece, pieces;
  bool few;
  HeadTiles tiles;
  Cuts cuts;
};
Plan make_plan(const ssm_head_desc& d, int grads, bool copy_w, int sms) {
  Plan p{};
  const long long T = d.rows, Tp = pad_rows(T), n_e = d.entries ? d.entries : 1;
  const int Dp = pad8(d.cols);
  p.planes = d.io == SSM_F32 ? 3 : 1;
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
    p.table = take(kHeadParts * T);
    p.valid = take(T);
  }
  p.few = head_few(T, d.cols, d.io, grads != 0);
  if (p.few && grads) {
    if (grads & 1) p.dh = take((size_t)4 * head_few_blocks(sms) * T * Dp);
    p.bytes = at;
    return p;
  }
  if (p.few) {
    p.n_stats = head_few_blocks(sms);
    p.stats = take((size_t)8 * p.n_stats * Tp);
    p.zt = take(4 * T * n_e);
    p.bytes = at;
    return p;
  }
  p.h = take((size_t)2 * p.planes * Tp * Dp);
  if (copy_w) p.w = take((size_t)2 * p.planes * d.vocab * Dp);
  if (!grads) {
    p.tiles = tiles_of(T, d.cols, d.vocab, d.io, false, sms);
    const int narrow = p.tiles.words ? kHeadTile / 2 : kHeadTile;
    p.stats = take((size_t)8 * 2 * ((d.vocab + narrow - 1) / narrow) * Tp);
    p.zt = take(4 * T * n_e);
  } else {
    p.rl = take(4 * Tp);
    p.rg = take(4 * Tp);
    // pieces of the vocabulary, alike
    const int tiles = (d.vocab + kHeadTile - 1) / kHeadTile;
    const int terms = head_g_terms(d);
    long long most = kMaxPiece / (2 * terms * Tp) / kHeadTile;
    if (most < 1) most = 1;
    p.pieces = (int)((tiles + most - 1) / most);
    p.piece = (tiles + p.pieces - 1) / p.pieces * kHeadTile;
    p.pieces = (d.vocab + p.piece - 1) / p.piece;
    p.g = take((size_t)2 * terms * Tp * p.piece);
    p.tiles = tiles_of(T, d.cols, p.piece, d.io, true, sms);
    p.cuts = cuts_of(T, d.cols, p.piece, d.io, terms == 2, grads, p.pieces > 1, sms);
    if ((grads & 1) && (p.pieces > 1 || p.cuts.h.splits > 1))
      p.dh = take((size_t)4 * p.cuts.h.splits * Tp * Dp);
    if ((grads & 2) && p.cuts.w.splits > 1)
      p.dw = take((size_t)4 * p.cuts.w.splits * p.piece * Dp);
  }
  p.bytes = at;
  return p;
}

// The plan of sizes, which a call needs twice (workspace and launches) and a training loop again and again:
// the thread's last few are kept (deciding on the cuts takes the host several us).
Plan plan_of(const ssm_head_desc& d, int grads, bool copy_w, int sms) {
  struct Known {
    long long rows;
    int cols, vocab, io, entries, terms, grads, copy_w, sms;
    Plan plan;
  };
  constexpr int kPlans = 8;
  static thread_local Known known[kPlans];
  static thread_local int next = 0;
  for (const Known& k : known)
    if (k.sms == sms && k.rows == d.rows && k.cols == d.cols && k.vocab == d.vocab && k.io == d.io &&
        k.entries == d.entries && k.terms == head_g_terms(d) && k.grads == grads && k.copy_w == (int)copy_w)
      return k.plan;
  Known& k = known[next];
  next = (next + 1) % kPlans;
  k = {d.rows, d.cols, d.vocab, d.io, d.entries, head_g_terms(d), grads, (int)copy_w, sms,
       make_plan(d, grads, copy_w, sms)};
  return k.plan;
}

int check(const ssm_head_desc* d, bool distill) {
  if (!d || d->rows <= 0 || d->cols <= 0 || d->vocab <= 0 || !io_size(d->io))
    return SSM_ERR_INVALID_ARG;
  if (d->flags & ~(SSM_DEBUG_NO_WAIT | SSM_HEAD_FINE_G)) return SSM_ERR_INVALID_ARG;
  if (distill) {
    if (d->entries <= 0 || !io_size(d->entry_io)) return SSM_ERR_INVALID_ARG;
    if (!(d->temperature > 0.0f) || isinf(d->temperature)) return SSM_ERR_INVALID_ARG;
    if (d->entries > SSM_MAX_HEAD_ENTRIES || d->temperature < 1.0f / SSM_MAX_HEAD_TEMPERATURE ||
        d->temperature > SSM_MAX_HEAD_TEMPERATURE)
      return SSM_ERR_UNSUPPORTED;
  } else if (d->entries) {
    return SSM_ERR_INVALID_ARG;
  }
  if (d->rows > SSM_MAX_HEAD_ROWS || d->cols > SSM_MAX_HEAD_COLS || d->vocab > SSM_MAX_HEAD_VOCAB)
    return SSM_ERR_UNSUPPORTED;
  if (d->rows > kMaxLogits / d->vocab) return SSM_ERR_UNSUPPORTED;
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
  if (c.ld_h > kMaxTotal / d.rows || c.ld_d_h > kMaxTotal / d.rows || c.ld_w > kMaxTotal / d.vocab ||
      c.ld_w >= kMaxStride / (long long)size)
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
  HeadLists lists{(int*)(ws + p.idx)};
  if (d.entries) {
    lists.p = (float*)(ws + p.p);
    lists.known = (float*)(ws + p.known);
    lists.table = (uint8_t*)(ws + p.table);
  }
  uint8_t* valid = d.entries ? (uint8_t*)(ws + p.valid) : nullptr;
  HeadRows r{(HeadState*)ws, (int*)(ws + p.pos), (int*)(ws + p.src), (float*)(ws + p.rl),
             (float*)(ws + p.rg), (__nv_bfloat16*)(ws + p.h)};
#define SSM_DO(call) \
  if ((call) != cudaSuccess) return SSM_ERR_CUDA
  if (distill) SSM_DO(launch_head_entries(d, c.t_idx, c.t_logit, lists, valid, st));
  float2* stats = (float2*)(ws + p.stats);
  float* zt = (float*)(ws + p.zt);
  if (p.few && backward) {
    float* h_part = c.d_h ? (float*)(ws + p.dh) : nullptr;
    SSM_DO(launch_head_few_bwd(d, c.target, valid, c.h, c.ld_h, c.w, c.ld_w, lists, r, c.lse, c.d_loss,
                               h_part, c.d_h, c.ld_d_h, c.d_w, sms, st));
    return SSM_OK;
  }
  if (p.few) {
    SSM_DO(launch_head_few(d, c.target, valid, c.h, c.ld_h, c.w, c.ld_w, lists, r, stats, zt, sms, st));
    SSM_DO(launch_head_loss(d, stats, p.n_stats, zt, lists, r, c.loss, c.lse_out, sms, st));
    return SSM_OK;
  }
  __nv_bfloat16* w_out = copy_w ? (__nv_bfloat16*)(ws + p.w) : nullptr;
  SSM_DO(launch_head_rows(d, c.target, valid, c.h, c.ld_h, backward ? c.lse : nullptr,
                          backward ? c.d_loss : nullptr, c.w, c.ld_w, lists.idx, r, w_out, p.tiles,
                          sms, st));
  const HeadMatrix h{r.h, Tp, Dp, Tp * Dp, d.cols};
  const HeadMatrix w = copy_w ? HeadMatrix{w_out, d.vocab, Dp, (long long)d.vocab * Dp, d.cols} :
                                HeadMatrix{(const __nv_bfloat16*)c.w, d.vocab, c.ld_w, 0, d.cols};
  if (!backward) {
    SSM_DO(launch_head_logits(d, h, w, r, lists, p.tiles, stats, zt, sms, st));
    SSM_DO(launch_head_loss(d, stats, p.n_stats, zt, lists, r, c.loss, c.lse_out, sms, st));
    return SSM_OK;
  }
  __nv_bfloat16* gp = (__nv_bfloat16*)(ws + p.g);
  const HeadMatrix g{gp, Tp, p.piece, Tp * p.piece, p.piece};
  const HeadOut out{p.cuts.h, p.cuts.w, p.cuts.h_first, p.dh ? (float*)(ws + p.dh) : nullptr,
                    p.dw ? (float*)(ws + p.dw) : nullptr, c.d_w, p.dh ? nullptr : c.d_h, c.ld_d_h};
  for (int i = 0; i < p.pieces; i++) {
    const int v0 = i * p.piece, n = d.vocab - v0 < p.piece ? d.vocab - v0 : p.piece;
    const bool last = i == p.pieces - 1;
    SSM_DO(launch_head_grad(d, h, w, r, lists, gp, v0, p.piece, sms, st));
    SSM_DO(launch_head_out(d, g, h, w, r, out, v0, n, i > 0, sms, st));
    if (last || out.w_part)
      SSM_DO(launch_head_finish(d, r, out.h_part, p.cuts.h.splits, last ? c.d_h : nullptr, c.ld_d_h,
                                out.w_part, p.cuts.w.per, p.piece, c.d_w, v0, n, last, sms, st));
  }
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
