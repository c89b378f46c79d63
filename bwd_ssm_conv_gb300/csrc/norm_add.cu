// norm_add.cu -- residual add + RMSNorm in front of a block, forward and backward:
//   s = residual + scale x,  out = w s rstd,  rstd = (mean(s^2) + eps)^-1/2
//   n = s rstd,  r = d_s + rstd (w d_out - n mean(w d_out n)),
//   d_residual = r,  d_x = scale r,  d_w = sum_rows d_out n,  d_scale = sum_rows r x
// Both directions read a row once into registers, form its one sum over the row's threads and
// write its results, so each is bound by the memory traffic of its operands.  The stream is
// formed with the product and the sum rounded one after the other, so that it holds the same bits
// as an unfused add does.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

template <typename IO, typename RES, int VEC, int NJ, int MAXT>
__global__ void __launch_bounds__(MAXT) add_norm_fwd_kernel(const AddNormFwd a, const RowPlan pl) {
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int cols = a.cols, nb = (cols + 31) / 32;
  const float inv = 1.0f / (float)cols;
  bool okc[NJ];
  int col[NJ];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < cols;
  }
  int half = 0;
  for (long long base = (long long)blockIdx.x * pl.rpb; base < a.rows;
       base += (long long)gridDim.x * pl.rpb, half ^= 1) {
    const long long row = base + pos.slot;
    const bool rok = row < a.rows;
    float s[NJ][VEC];
    Cols<IO, VEC> xr[NJ];
    Cols<RES, VEC> rr[NJ];
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      xr[j].zero();
      rr[j].zero();
      if (rok && okc[j]) {
        xr[j].load((const IO*)a.x + row * a.ld_x + col[j]);
        if (a.residual) rr[j].load((const RES*)a.residual + row * a.ld_residual + col[j]);
      }
    }
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      float xv[VEC], rv[VEC], sc[VEC];
      xr[j].get(xv);
      rr[j].get(rv);
      ld_param<VEC>(a.scale, col[j], okc[j], sc);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        s[j][i] = __fadd_rn(rv[i], __fmul_rn(sc[i], xv[i]));
        sq = fmaf(s[j][i], s[j][i], sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum(sq, pl.tpr, part, half) * inv + a.eps);
    if (a.rstd && rok && pos.ok && pos.lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float w[VEC], o[VEC], kept[VEC];
      ld_param<VEC>(a.w, col[j], okc[j], w);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        o[i] = rounded<IO>(w[i] * (s[j][i] * rstd));
        kept[i] = rounded<RES>(s[j][i]);
      }
      if (ok) {
        st_cols((IO*)a.out + row * a.ld_out + col[j], o);
        if (a.res_out) st_cols((RES*)a.res_out + row * a.ld_res_out + col[j], kept);
      }
      const long long q = row * cols + col[j], e = row * nb + col[j] / 32;
      if (a.res_q) store_ckpt8<VEC>(kept, ok, a.res_q + q, a.res_e + e);
      if (a.x_q) {
        float xv[VEC];
        xr[j].get(xv);
        store_ckpt8<VEC>(xv, ok, a.x_q + q, a.x_e + e);
      }
      if (a.out_q) store_ckpt8<VEC>(o, ok, a.out_q + q, a.out_e + e);
    }
  }
}

// KEPT: s (and x, where d_scale is wanted from a checkpoint) is read from 8 bits.
template <typename IO, typename RES, int VEC, int NJ, int MAXT>
__global__ void __launch_bounds__(MAXT) add_norm_bwd_kernel(const AddNormBwd a, const RowPlan pl) {
  extern __shared__ float slots[];  // rpb > 1: the slots' column sums
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int cols = a.cols, nb = (cols + 31) / 32;
  const float inv = 1.0f / (float)cols;
  bool okc[NJ];
  int col[NJ];
  float w[NJ][VEC], dw[NJ][VEC], ds[NJ][VEC];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < cols;
    ld_param<VEC>(a.w, col[j], okc[j], w[j]);
#pragma unroll
    for (int i = 0; i < VEC; i++) dw[j][i] = ds[j][i] = 0.0f;
  }
  int half = 0;
  for (long long base = (long long)blockIdx.x * pl.rpb; base < a.rows;
       base += (long long)gridDim.x * pl.rpb, half ^= 1) {
    const long long row = base + pos.slot;
    const bool rok = row < a.rows;
    const float rstd = rok ? a.rstd_in[row] : 0.0f;
    Cols<IO, VEC> dr[NJ];
    float n[NJ][VEC];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      dr[j].zero();
      if (ok) dr[j].load((const IO*)a.d_out + row * a.ld_d_out + col[j]);
      if (a.res_q) {
        Kept<VEC> k;
        k.zero();
        if (ok) k.load(a.res_q + row * cols + col[j], a.res_e + row * nb + col[j] / 32);
        k.get(n[j]);
      } else {
        Cols<RES, VEC> k;
        k.zero();
        if (ok) k.load((const RES*)a.res + row * a.ld_res + col[j]);
        k.get(n[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      float d[VEC];
      dr[j].get(d);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        n[j][i] *= rstd;
        dw[j][i] = fmaf(d[i], n[j][i], dw[j][i]);
        dot = fmaf(w[j][i] * d[i], n[j][i], dot);
      }
    }
    const float mean = row_sum(dot, pl.tpr, part, half) * inv;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float d[VEC], r[VEC];
      dr[j].get(d);
      Cols<RES, VEC> up;
      up.zero();
      if (ok && a.d_res_out) up.load((const RES*)a.d_res_out + row * a.ld_d_res_out + col[j]);
      up.get(r);
#pragma unroll
      for (int i = 0; i < VEC; i++)
        r[i] = fmaf(rstd, fmaf(-n[j][i], mean, w[j][i] * d[i]), r[i]);
      if (a.d_scale) {
        float xv[VEC];
        if (a.x_q) {
          Kept<VEC> k;
          k.zero();
          if (ok) k.load(a.x_q + row * cols + col[j], a.x_e + row * nb + col[j] / 32);
          k.get(xv);
        } else {
          Cols<IO, VEC> k;
          k.zero();
          if (ok) k.load((const IO*)a.x + row * a.ld_x + col[j]);
          k.get(xv);
        }
#pragma unroll
        for (int i = 0; i < VEC; i++) ds[j][i] = fmaf(r[i], xv[i], ds[j][i]);
      }
      if (ok) {
        if (a.d_res) st_cols((RES*)a.d_res + row * a.ld_d_res + col[j], r);
        if (a.d_x) {
          float sc[VEC];
          ld_param<VEC>(a.scale, col[j], true, sc);
#pragma unroll
          for (int i = 0; i < VEC; i++) r[i] *= sc[i];
          st_cols((IO*)a.d_x + row * a.ld_d_x + col[j], r);
        }
      }
    }
  }
  if (a.d_w) store_partial<VEC, NJ>(dw, pos, pl, col, okc, cols, a.part, slots);
  if (a.d_scale)
    store_partial<VEC, NJ>(ds, pos, pl, col, okc, cols,
                           a.part + (a.d_w ? (long long)pl.nbx * cols : 0), slots);
}

template <typename IO, typename RES, int VEC, int NJ, int MAXT>
void fwd_launch(const AddNormFwd& a, const RowPlan& pl, cudaStream_t st) {
  add_norm_fwd_kernel<IO, RES, VEC, NJ, MAXT>
      <<<dim3(pl.nbx, pl.nby), pl.threads, 0, st>>>(a, pl);
}
template <typename IO, typename RES, int VEC, int NJ, int MAXT>
void bwd_launch(const AddNormBwd& a, const RowPlan& pl, cudaStream_t st) {
  const size_t smem = slots_bytes(pl, VEC, NJ);
  add_norm_bwd_kernel<IO, RES, VEC, NJ, MAXT>
      <<<dim3(pl.nbx, pl.nby), pl.threads, smem, st>>>(a, pl);
}

template <typename IO, typename RES>
cudaError_t fwd_types(const AddNormFwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.cols, 1, vec, sms, false);
  const RowPlan& p = s.plan;
  switch (s.variant) {
    case kVec8x1: fwd_launch<IO, RES, 8, 1, 1024>(a, p, st); break;
    case kVec8x2: fwd_launch<IO, RES, 8, 2, 256>(a, p, st); break;
    case kVec8x4: fwd_launch<IO, RES, 8, 4, 256>(a, p, st); break;
    case kVec8x4Wide: fwd_launch<IO, RES, 8, 4, 1024>(a, p, st); break;
    case kOne2: fwd_launch<IO, RES, 1, 2, 128>(a, p, st); break;
    case kOne8: fwd_launch<IO, RES, 1, 8, 1024>(a, p, st); break;
    default: fwd_launch<IO, RES, 1, 32, 1024>(a, p, st); break;
  }
  count_launches(1);
  return cudaGetLastError();
}
template <typename IO, typename RES>
cudaError_t bwd_types(const AddNormBwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.cols, 1, vec, sms, true);
  const RowPlan& p = s.plan;
  switch (s.variant) {
    case kVec8x1: bwd_launch<IO, RES, 8, 1, 1024>(a, p, st); break;
    case kVec8x2: bwd_launch<IO, RES, 8, 2, 256>(a, p, st); break;
    case kVec8x4: bwd_launch<IO, RES, 8, 4, 256>(a, p, st); break;
    case kVec8x4Wide: bwd_launch<IO, RES, 8, 4, 1024>(a, p, st); break;
    case kOne2: bwd_launch<IO, RES, 1, 2, 128>(a, p, st); break;
    case kOne8: bwd_launch<IO, RES, 1, 8, 1024>(a, p, st); break;
    default: bwd_launch<IO, RES, 1, 32, 1024>(a, p, st); break;
  }
  count_launches(1);
  if (cudaError_t e = cudaGetLastError()) return e;
  const float* part = a.part;
  if (a.d_w) {
    if (cudaError_t e = launch_column_sums(part, p.nbx, a.cols, a.d_w, st)) return e;
    part += (long long)p.nbx * a.cols;
  }
  if (a.d_scale) return launch_column_sums(part, p.nbx, a.cols, a.d_scale, st);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_add_norm_fwd(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st) {
  if (io == SSM_F32) return fwd_types<float, float>(a, vec, sms, st);
  if (res_io == SSM_F32) return fwd_types<__nv_bfloat16, float>(a, vec, sms, st);
  return fwd_types<__nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
}
cudaError_t launch_add_norm_bwd(const AddNormBwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st) {
  if (io == SSM_F32) return bwd_types<float, float>(a, vec, sms, st);
  if (res_io == SSM_F32) return bwd_types<__nv_bfloat16, float>(a, vec, sms, st);
  return bwd_types<__nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
}

}  // namespace ssm
