// norm_gated.cu -- the gated RMSNorm after the scan, forward and backward, per group of columns:
//   gate first:  v = y silu(z),  n = v rstd(v),  out = w n
//                dv = rstd (w d_out - n mean(w d_out n)),  d_y = dv silu(z),  d_z = dv y silu'(z)
//   norm first:  n = y rstd(y),  out = w n silu(z),  dn = w d_out silu(z)
//                d_y = rstd (dn - n mean(dn n)),  d_z = w d_out n silu'(z)
// As in norm_add.cu a group is read once into registers and its one sum formed over its threads.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

template <typename IO, int VEC, int NJ, int MAXT>
__global__ void __launch_bounds__(MAXT) gated_norm_fwd_kernel(const GatedNormFwd a,
                                                              const RowPlan pl) {
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int nb = (a.cols + 31) / 32;
  const float inv = 1.0f / (float)a.group;
  bool okc[NJ];
  int col[NJ];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < a.group;
    col[j] += pos.col0;
  }
  int half = 0;
  for (long long base = (long long)blockIdx.x * pl.rpb; base < a.rows;
       base += (long long)gridDim.x * pl.rpb, half ^= 1) {
    const long long row = base + pos.slot;
    const bool rok = row < a.rows;
    Cols<IO, VEC> yr[NJ], zr[NJ];
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      yr[j].zero();
      zr[j].zero();
      if (rok && okc[j]) {
        yr[j].load((const IO*)a.y + row * a.ld_y + col[j]);
        zr[j].load((const IO*)a.z + row * a.ld_z + col[j]);
      }
    }
    float v[NJ][VEC];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      yr[j].get(v[j]);
      if (!a.norm_first) {
        float z[VEC];
        zr[j].get(z);
#pragma unroll
        for (int i = 0; i < VEC; i++) v[j][i] *= siluf_(z[i]);
      }
#pragma unroll
      for (int i = 0; i < VEC; i++) sq = fmaf(v[j][i], v[j][i], sq);
    }
    const float rstd = 1.0f / sqrtf(row_sum(sq, pl.tpr, part, half) * inv + a.eps);
    if (a.rstd && rok && pos.ok && pos.lane == 0)
      a.rstd[row * pl.groups + pos.col0 / a.group] = rstd;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float w[VEC], o[VEC], z[VEC];
      ld_param<VEC>(a.w, col[j], okc[j], w);
      zr[j].get(z);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        o[i] = w[i] * (v[j][i] * rstd);
        if (a.norm_first) o[i] *= siluf_(z[i]);
        o[i] = rounded<IO>(o[i]);
      }
      if (ok) st_cols((IO*)a.out + row * a.ld_out + col[j], o);
      const long long q = row * a.cols + col[j], e = row * nb + col[j] / 32;
      if (a.y_q) {
        float y[VEC];
        yr[j].get(y);
        store_ckpt8<VEC>(y, ok, a.y_q + q, a.y_e + e);
      }
      if (a.z_q) store_ckpt8<VEC>(z, ok, a.z_q + q, a.z_e + e);
      if (a.out_q) store_ckpt8<VEC>(o, ok, a.out_q + q, a.out_e + e);
    }
  }
}

template <typename IO, int VEC, int NJ, int MAXT>
__global__ void __launch_bounds__(MAXT) gated_norm_bwd_kernel(const GatedNormBwd a,
                                                              const RowPlan pl) {
  extern __shared__ float slots[];
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int nb = (a.cols + 31) / 32;
  const float inv = 1.0f / (float)a.group;
  bool okc[NJ];
  int col[NJ];
  float w[NJ][VEC], dw[NJ][VEC];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < a.group;
    ld_param<VEC>(a.w, pos.col0 + col[j], okc[j], w[j]);
#pragma unroll
    for (int i = 0; i < VEC; i++) dw[j][i] = 0.0f;
  }
  int half = 0;
  for (long long base = (long long)blockIdx.x * pl.rpb; base < a.rows;
       base += (long long)gridDim.x * pl.rpb, half ^= 1) {
    const long long row = base + pos.slot;
    const bool rok = row < a.rows;
    const float rstd =
        rok && pos.ok ? a.rstd_in[row * pl.groups + pos.col0 / a.group] : 0.0f;
    Cols<IO, VEC> dr[NJ];
    float y[NJ][VEC], z[NJ][VEC];
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      const int c = pos.col0 + col[j];
      dr[j].zero();
      if (ok) dr[j].load((const IO*)a.d_out + row * a.ld_d_out + c);
      if (a.y_q) {
        Kept<VEC> ky, kz;
        ky.zero();
        kz.zero();
        if (ok) {
          ky.load(a.y_q + row * a.cols + c, a.y_e + row * nb + c / 32);
          kz.load(a.z_q + row * a.cols + c, a.z_e + row * nb + c / 32);
        }
        ky.get(y[j]);
        kz.get(z[j]);
      } else {
        Cols<IO, VEC> ky, kz;
        ky.zero();
        kz.zero();
        if (ok) {
          ky.load((const IO*)a.y + row * a.ld_y + c);
          kz.load((const IO*)a.z + row * a.ld_z + c);
        }
        ky.get(y[j]);
        kz.get(z[j]);
      }
    }
    // y becomes n; z stays
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      float d[VEC];
      dr[j].get(d);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        const float gate = siluf_(z[j][i]);
        const float n = a.norm_first ? y[j][i] * rstd : y[j][i] * gate * rstd;
        const float up = a.norm_first ? d[i] * gate : d[i];  // the gradient of w n
        dw[j][i] = fmaf(up, n, dw[j][i]);
        dot = fmaf(w[j][i] * up, n, dot);
      }
    }
    const float mean = row_sum(dot, pl.tpr, part, half) * inv;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      float d[VEC], dy[VEC], dz[VEC];
      dr[j].get(d);
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        const float sg = sigmoidf_(z[j][i]), gate = z[j][i] * sg;
        const float slope = sg * (1.0f + z[j][i] * (1.0f - sg));
        const float wd = w[j][i] * d[i];
        if (a.norm_first) {
          const float n = y[j][i] * rstd;
          dy[i] = rstd * fmaf(-n, mean, wd * gate);
          dz[i] = wd * n * slope;
        } else {
          const float n = y[j][i] * gate * rstd;
          const float dv = rstd * fmaf(-n, mean, wd);
          dy[i] = dv * gate;
          dz[i] = dv * y[j][i] * slope;
        }
      }
      if (rok && okc[j]) {
        st_cols((IO*)a.d_y + row * a.ld_d_y + pos.col0 + col[j], dy);
        st_cols((IO*)a.d_z + row * a.ld_d_z + pos.col0 + col[j], dz);
      }
    }
  }
  if (a.d_w) store_partial<VEC, NJ>(dw, pos, pl, col, okc, a.cols, a.part, slots);
}

template <typename IO, int VEC, int NJ, int MAXT>
void fwd_launch(const GatedNormFwd& a, const RowPlan& pl, cudaStream_t st) {
  gated_norm_fwd_kernel<IO, VEC, NJ, MAXT><<<dim3(pl.nbx, pl.nby), pl.threads, 0, st>>>(a, pl);
}
template <typename IO, int VEC, int NJ, int MAXT>
void bwd_launch(const GatedNormBwd& a, const RowPlan& pl, cudaStream_t st) {
  gated_norm_bwd_kernel<IO, VEC, NJ, MAXT>
      <<<dim3(pl.nbx, pl.nby), pl.threads, slots_bytes(pl, VEC, NJ), st>>>(a, pl);
}

template <typename IO>
cudaError_t fwd_types(const GatedNormFwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.group, a.cols / a.group, vec, sms, false);
  const RowPlan& p = s.plan;
  switch (s.variant) {
    case kVec8x1: fwd_launch<IO, 8, 1, 1024>(a, p, st); break;
    case kVec8x2: fwd_launch<IO, 8, 2, 256>(a, p, st); break;
    case kVec8x4: fwd_launch<IO, 8, 4, 256>(a, p, st); break;
    case kVec8x4Wide: fwd_launch<IO, 8, 4, 1024>(a, p, st); break;
    case kOne2: fwd_launch<IO, 1, 2, 128>(a, p, st); break;
    case kOne8: fwd_launch<IO, 1, 8, 1024>(a, p, st); break;
    default: fwd_launch<IO, 1, 32, 1024>(a, p, st); break;
  }
  count_launches(1);
  return cudaGetLastError();
}
template <typename IO>
cudaError_t bwd_types(const GatedNormBwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.group, a.cols / a.group, vec, sms, true);
  const RowPlan& p = s.plan;
  switch (s.variant) {
    case kVec8x1: bwd_launch<IO, 8, 1, 1024>(a, p, st); break;
    case kVec8x2: bwd_launch<IO, 8, 2, 256>(a, p, st); break;
    case kVec8x4: bwd_launch<IO, 8, 4, 256>(a, p, st); break;
    case kVec8x4Wide: bwd_launch<IO, 8, 4, 1024>(a, p, st); break;
    case kOne2: bwd_launch<IO, 1, 2, 128>(a, p, st); break;
    case kOne8: bwd_launch<IO, 1, 8, 1024>(a, p, st); break;
    default: bwd_launch<IO, 1, 32, 1024>(a, p, st); break;
  }
  count_launches(1);
  if (cudaError_t e = cudaGetLastError()) return e;
  return a.d_w ? launch_column_sums(a.part, p.nbx, a.cols, a.d_w, st) : cudaSuccess;
}

}  // namespace

cudaError_t launch_gated_norm_fwd(const GatedNormFwd& a, int io, bool vec, int sms,
                                  cudaStream_t st) {
  return io == SSM_F32 ? fwd_types<float>(a, vec, sms, st)
                       : fwd_types<__nv_bfloat16>(a, vec, sms, st);
}
cudaError_t launch_gated_norm_bwd(const GatedNormBwd& a, int io, bool vec, int sms,
                                  cudaStream_t st) {
  return io == SSM_F32 ? bwd_types<float>(a, vec, sms, st)
                       : bwd_types<__nv_bfloat16>(a, vec, sms, st);
}

}  // namespace ssm
