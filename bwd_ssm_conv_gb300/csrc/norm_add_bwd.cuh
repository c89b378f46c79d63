// norm_add_bwd.cuh -- the backward kernel of both norms in front of a block (norm_add_bwd.cu: RMSNorm,
// norm_layer_bwd.cu: layer norm).
#pragma once

#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

// KEPT: s or x may be checkpoints.
template <bool LAYER, bool KEPT, typename IO, typename RES, int VEC, int NJ, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) add_norm_bwd_kernel(const AddNormBwd a,
                                                                  const RowPlan pl) {
  extern __shared__ __align__(16) unsigned char ring[];  // at the end: the slots' column sums
  __shared__ float part[2][32];
  __shared__ float part2[LAYER ? 2 : 1][32];  // the layer norm's other sum
  const RowPos pos = row_pos(pl);
  const int cols = a.cols, nb = (cols + 31) / 32;
  const float inv = 1.0f / (float)cols;
  bool okc[NJ];
  int col[NJ];
  float w[NJ][VEC], dw[NJ][VEC], ds[NJ][VEC];
  float db[LAYER ? NJ : 1][VEC];
  constexpr bool kHoldScale = LAYER && VEC == 1 && NJ <= 4;
  float hold[kHoldScale ? NJ : 1];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < cols;
    ld_param<VEC>(a.w, col[j], okc[j], w[j]);
#pragma unroll
    for (int i = 0; i < VEC; i++) dw[j][i] = ds[j][i] = 0.0f;
    if constexpr (LAYER)
#pragma unroll
      for (int i = 0; i < VEC; i++) db[j][i] = 0.0f;
    if constexpr (kHoldScale) {
      float one[1];
      ld_param<1>(a.scale, col[j], okc[j], one);
      hold[j] = one[0];
    }
  }
  typedef Operand<IO, VEC, NJ, (VEC == 8 && MAXT <= 256), KEPT> Act;
  typedef Operand<RES, VEC, NJ, (VEC == 8 && MAXT <= 256), KEPT> Res;
  const uint32_t act = Act::slot_bytes(blockDim.x), res = Res::slot_bytes(blockDim.x);
  const uint32_t at = shared_addr(ring) + 16 * threadIdx.x, bytes = 2 * act + 2 * res;
  const bool want_ds = a.d_scale != nullptr;
  Act d{a.d_out, nullptr, nullptr, a.ld_d_out, at};
  Act x{want_ds ? a.x : nullptr, want_ds ? a.x_q : nullptr, a.x_e, a.ld_x, at + act};
  Res sv{a.res, a.res_q, a.res_e, a.ld_res, at + 2 * act};
  Res up{a.d_res_out, nullptr, nullptr, a.ld_d_res_out, at + 2 * act + res};
  const int step = gridDim.x * pl.rpb;  // rows stay below 2^31 - step
  int row = blockIdx.x * pl.rpb + pos.slot;
  auto issue = [&](int r, int slot) {
    const uint32_t s = slot * bytes;
    if (r < a.rows) {
      d.issue(s, r, col, okc, cols);
      sv.issue(s, r, col, okc, cols);
      up.issue(s, r, col, okc, cols);
      x.issue(s, r, col, okc, cols);
    } else {  // adds nothing to the column sums
      d.clear(s, okc, true);
      sv.clear(s, okc, true);
      up.clear(s, okc, true);
      x.clear(s, okc, true);
    }
    cp_async_commit();
  };
  // what a row needs besides: read one row ahead
  float rstd_next = 0.0f, mean_next = 0.0f;
  uint32_t es_next[NJ], ex_next[NJ];
  auto small = [&](int r) {
    const bool rok = r < a.rows;
    rstd_next = rok ? a.rstd_in[r] : 0.0f;
    if constexpr (LAYER) mean_next = rok ? a.mean_in[r] : 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      es_next[j] = sv.scale(rok && okc[j], r, col[j], nb);
      ex_next[j] = x.scale(rok && okc[j], r, col[j], nb);
    }
  };
  for (int i = 0; i < pl.slots; i++) {
    d.clear(i * bytes, okc, false);
    x.clear(i * bytes, okc, false);
    sv.clear(i * bytes, okc, false);
    up.clear(i * bytes, okc, false);
  }
  const int ahead = pl.slots - 1;
  for (int i = 0; i < ahead; i++) issue(row + i * step, i);
  small(row);
  int half = 0, slot = 0;
  for (int base = blockIdx.x * pl.rpb; base < a.rows; base += step, row += step, half ^= 1) {
    const bool rok = row < a.rows;
    const float rstd = rstd_next, mean = mean_next;
    uint32_t es[NJ], ex[NJ];
#pragma unroll
    for (int j = 0; j < NJ; j++) es[j] = es_next[j], ex[j] = ex_next[j];
    small(row + step);
    d.advance();
    x.advance();
    sv.advance();
    up.advance();
    issue(row + ahead * step, slot == 0 ? ahead : slot - 1);
    cp_async_wait(ahead);
    const uint32_t s = slot * bytes;
    slot = slot == ahead ? 0 : slot + 1;
    float wd[NJ][VEC], sr[NJ][VEC], dot = 0.0f, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float dv[VEC];
      d.get(s, j, ok, row, col[j], cols, 7u, dv);
      sv.get(s, j, ok, row, col[j], cols, es[j], sr[j]);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        if constexpr (LAYER) sr[j][i] -= mean;
        const float n = sr[j][i] * rstd;
        dw[j][i] = fmaf(dv[i], n, dw[j][i]);
        wd[j][i] = w[j][i] * dv[i];
        if constexpr (LAYER) db[j][i] += dv[i], sum += wd[j][i];
        dot = fmaf(wd[j][i], n, dot);
      }
    }
    float off = 0.0f;
    if constexpr (LAYER) {
      row_sum2(dot, sum, pl.tpr, part, part2, half);
      off = -sum * inv;
    } else {
      dot = row_sum(dot, pl.tpr, part, half);
    }
    const float c = -dot * inv * rstd;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float r[VEC];
      up.get(s, j, ok, row, col[j], cols, 7u, r);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        const float t = LAYER ? wd[j][i] + off : wd[j][i];
        r[i] = fmaf(rstd, fmaf(sr[j][i], c, t), r[i]);
      }
      if (want_ds) {
        float xv[VEC];
        x.get(s, j, ok, row, col[j], cols, ex[j], xv);
#pragma unroll
        for (int i = 0; i < VEC; i++) ds[j][i] = fmaf(r[i], xv[i], ds[j][i]);
      }
      if (ok) {
        if (a.d_res) st_cols((RES*)a.d_res + (long long)row * a.ld_d_res + col[j], r);
        if (a.d_x) {
          if constexpr (kHoldScale) {
            r[0] *= hold[j];
          } else {
            float sc[VEC];
            ld_param<VEC>(a.scale, col[j], true, sc);
#pragma unroll
            for (int i = 0; i < VEC; i++) r[i] *= sc[i];
          }
          st_cols((IO*)a.d_x + (long long)row * a.ld_d_x + col[j], r);
        }
      }
    }
  }
  cp_async_wait(0);
  float* sums = a.part;  // of the outputs that are wanted, one after the other
  if (a.d_w) {
    store_partial<VEC, NJ>(dw, pl, pos, col, okc, cols, sums, (float*)ring);
    sums += (long long)pl.nbx * cols;
  }
  if constexpr (LAYER)
    if (a.d_b) {
      store_partial<VEC, NJ>(db, pl, pos, col, okc, cols, sums, (float*)ring);
      sums += (long long)pl.nbx * cols;
    }
  if (a.d_scale) store_partial<VEC, NJ>(ds, pl, pos, col, okc, cols, sums, (float*)ring);
}

template <bool LAYER, typename IO, typename RES, int VEC, int NJ, int MAXT, int MINB>
cudaError_t bwd_launch(const AddNormBwd& a, RowPlan pl, int per_sm, cudaStream_t st) {
  constexpr bool kRing = VEC == 8 && MAXT <= 256;
  const uint32_t slot = 2 * (Operand<IO, VEC, NJ, kRing>::slot_bytes(pl.threads) +
                             Operand<RES, VEC, NJ, kRing>::slot_bytes(pl.threads));
  pl.slots = VEC == 1 ? 2 : ring_slots(slot, pl.threads, per_sm);
  const size_t ring = (size_t)pl.slots * slot, sums = slots_bytes(pl, VEC, NJ);
  const size_t smem = ring > sums ? ring : sums;
  if constexpr (LAYER && VEC == 1)
    if (!a.res_q && !a.x_q)
      return launch_rows<add_norm_bwd_kernel<LAYER, false, IO, RES, VEC, NJ, MAXT, MINB>>(a, pl, smem,
                                                                                        st);
  return launch_rows<add_norm_bwd_kernel<LAYER, true, IO, RES, VEC, NJ, MAXT, MINB>>(a, pl, smem, st);
}

template <bool LAYER, typename IO, typename RES>
cudaError_t bwd_types(const AddNormBwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.cols, 1, vec, sms, true);
  count_launches(1);
  cudaError_t e;
#define SSM_LAUNCH(VEC, NJ, MAXT, MINB) \
  e = bwd_launch<LAYER, IO, RES, VEC, NJ, MAXT, MINB>(a, s.plan, norm_threads_per_sm(s.variant, true), st)
  SSM_NORM_BWD_SWITCH(s.variant, SSM_LAUNCH)
#undef SSM_LAUNCH
  if (e != cudaSuccess || (!a.d_w && !a.d_b && !a.d_scale)) return e;
  return launch_column_sums(a.part, s.plan.nbx, a.cols, a.d_w, a.d_b, a.d_scale, st);
}


}  // namespace

}  // namespace ssm
