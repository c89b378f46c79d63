// norm_add.cuh -- the forward kernel of both norms in front of a block (norm_add.cu: RMSNorm,
// norm_layer.cu: layer norm).
#pragma once

#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

// KEPT: there may be checkpoints to write.
template <bool LAYER, bool KEPT, typename IO, typename RES, int VEC, int NJ, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) add_norm_fwd_kernel(const AddNormFwd a,
                                                                  const RowPlan pl) {
  // The layer norm's rows of up to 8192 columns are copied ahead to shared memory (rows.cuh).
  constexpr bool kRing = LAYER && VEC == 8 && MAXT <= 256;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int cols = a.cols, nb = (cols + 31) / 32;
  const float inv = 1.0f / (float)cols;
  bool okc[NJ];
  int col[NJ];
  float w[NJ][VEC], sc[NJ][VEC];
  float bias[LAYER ? NJ : 1][VEC];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < cols;
    ld_param<VEC>(a.w, col[j], okc[j], w[j]);
    ld_param<VEC>(a.scale, col[j], okc[j], sc[j]);
    if constexpr (LAYER) ld_param<VEC>(a.b, col[j], okc[j], bias[j], 0.0f);
  }
  // Single columns are loaded one row ahead (rows.cuh).
  typedef Operand<IO, VEC, NJ, kRing, false> Act;
  typedef Operand<RES, VEC, NJ, kRing, false> Res;
  const uint32_t at = shared_addr(ring) + 16 * threadIdx.x, act = Act::slot_bytes(blockDim.x),
                 bytes = act + Res::slot_bytes(blockDim.x);
  Act x1{a.x, nullptr, nullptr, a.ld_x, at};
  Res r1{a.residual, nullptr, nullptr, a.ld_residual, at + act};
  auto ahead = [&](int r, int slot) {
    if constexpr (Act::kAhead || kRing) {
      if (r < a.rows) {
        x1.issue(slot * bytes, r, col, okc, cols);
        r1.issue(slot * bytes, r, col, okc, cols);
      } else {
        x1.clear(slot * bytes, okc, true);
        r1.clear(slot * bytes, okc, true);
      }
      if constexpr (kRing) cp_async_commit();
    }
  };
  const int step = gridDim.x * pl.rpb;  // rows stay below 2^31 - step
  const int more = kRing ? pl.slots - 1 : 1;  // rows ahead
  int half = 0, slot = 0;
  if constexpr (kRing) {
    for (int i = 0; i < pl.slots; i++) {
      x1.clear(i * bytes, okc, false);
      r1.clear(i * bytes, okc, false);
    }
  }
  for (int i = 0; i < more; i++) ahead(blockIdx.x * pl.rpb + pos.slot + i * step, i);
  for (int base = blockIdx.x * pl.rpb; base < a.rows; base += step, half ^= 1) {
    const int row = base + pos.slot;
    const bool rok = row < a.rows;
    float s[NJ][VEC];
    Cols<IO, VEC> xr[NJ];
    Cols<RES, VEC> rr[NJ];
    const uint32_t here = slot * bytes;  // this row's place in the ring
    if constexpr (kRing) {
      ahead(row + more * step, slot == 0 ? more : slot - 1);
      cp_async_wait(more);
      slot = slot == more ? 0 : slot + 1;
    } else if constexpr (Act::kAhead) {
      x1.advance();
      r1.advance();
      ahead(row + step, 0);
    } else {
#pragma unroll
      for (int j = 0; j < NJ; j++) {
        xr[j].zero();
        rr[j].zero();
        if (rok && okc[j]) {
          xr[j].load((const IO*)a.x + (long long)row * a.ld_x + col[j]);
          if (a.residual)
            rr[j].load((const RES*)a.residual + (long long)row * a.ld_residual + col[j]);
        }
      }
    }
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      float xv[VEC], rv[VEC];
      if constexpr (Act::kAhead || kRing) {
        x1.get(here, j, true, row, col[j], cols, 7u, xv);
        r1.get(here, j, true, row, col[j], cols, 7u, rv);
      } else {
        xr[j].get(xv);
        rr[j].get(rv);
      }
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        s[j][i] = __fadd_rn(rv[i], __fmul_rn(sc[j][i], xv[i]));
        sq = LAYER ? sq + s[j][i] : fmaf(s[j][i], s[j][i], sq);
      }
    }
    float mean = 0.0f;
    if constexpr (LAYER) {  // the squares of what is left once the mean is known: two sums of the row
      mean = row_sum(sq, pl.tpr, part, 0) * inv;
      sq = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; j++)
#pragma unroll
        for (int i = 0; i < VEC; i++) {
          const float t = okc[j] ? s[j][i] - mean : 0.0f;
          sq = fmaf(t, t, sq);
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum(sq, pl.tpr, part, LAYER ? 1 : half) * inv + a.eps);
    if (rok && pos.ok && pos.lane == 0) {
      if (a.rstd) a.rstd[row] = rstd;
      if (LAYER && a.mean) a.mean[row] = mean;
    }
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float o[VEC];
      Cols<IO, VEC> oc;
      Cols<RES, VEC> stored;
#pragma unroll
      for (int i = 0; i < VEC; i++)
        // columns that the thread does not have stay zeros: an 8-bit block counts them
        o[i] = !LAYER ? w[j][i] * (s[j][i] * rstd) :
               okc[j] ? fmaf(w[j][i], (s[j][i] - mean) * rstd, bias[j][i]) : 0.0f;
      to_cols(o, oc);
      to_cols(s[j], stored);
      if (ok) {
        st_cols((IO*)a.out + (long long)row * a.ld_out + col[j], oc);
        if (a.res_out) st_cols((RES*)a.res_out + (long long)row * a.ld_res_out + col[j], stored);
      }
      const long long q = (long long)row * cols + col[j],
                      e = (long long)row * nb + (int)((unsigned)col[j] / 32);
      if (KEPT && a.res_q) {
        float kept[VEC];
        stored.get(kept);
        store_ckpt8<VEC>(kept, ok, a.res_q + q, a.res_e + e);
      }
      if (KEPT && a.x_q) {
        float xv[VEC];
        if constexpr (Act::kAhead || kRing) x1.get(here, j, true, row, col[j], cols, 7u, xv);
        else xr[j].get(xv);
        store_ckpt8<VEC>(xv, ok, a.x_q + q, a.x_e + e);
      }
      if (KEPT && a.out_q) {
        oc.get(o);
        store_ckpt8<VEC>(o, ok, a.out_q + q, a.out_e + e);
      }
    }
  }
}

template <bool LAYER, typename IO, typename RES, int VEC, int NJ, int MAXT, int MINB>
cudaError_t fwd_launch(const AddNormFwd& a, RowPlan pl, int per_sm, cudaStream_t st) {
  constexpr bool kRing = LAYER && VEC == 8 && MAXT <= 256;
  const uint32_t slot = Operand<IO, VEC, NJ, kRing>::slot_bytes(pl.threads) +
                        Operand<RES, VEC, NJ, kRing>::slot_bytes(pl.threads);
  pl.slots = ring_slots(slot, pl.threads, per_sm);
  const size_t smem = (size_t)pl.slots * slot;
  if constexpr (LAYER && VEC == 1)
    if (!a.res_q && !a.x_q && !a.out_q)
      return launch_rows<add_norm_fwd_kernel<LAYER, false, IO, RES, VEC, NJ, MAXT, MINB>>(a, pl, smem,
                                                                                        st);
  return launch_rows<add_norm_fwd_kernel<LAYER, true, IO, RES, VEC, NJ, MAXT, MINB>>(a, pl, smem, st);
}
template <bool LAYER, typename IO, typename RES>
cudaError_t fwd_types(const AddNormFwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.cols, 1, vec, sms, false);
  const RowPlan& p = s.plan;
  cudaError_t e;
#define SSM_LAUNCH(VEC, NJ, MAXT, MINB) \
  e = fwd_launch<LAYER, IO, RES, VEC, NJ, MAXT, MINB>(a, p, norm_threads_per_sm(s.variant, false), st)
  SSM_NORM_FWD_SWITCH(s.variant, SSM_LAUNCH)
#undef SSM_LAUNCH
  count_launches(1);
  return e;
}

template <bool LAYER>
cudaError_t launch_add_norm_fwd_of(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                   cudaStream_t st) {
  if (io == SSM_F32) return fwd_types<LAYER, float, float>(a, vec, sms, st);
  if (res_io == SSM_F32) return fwd_types<LAYER, __nv_bfloat16, float>(a, vec, sms, st);
  return fwd_types<LAYER, __nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
}

}  // namespace

}  // namespace ssm
