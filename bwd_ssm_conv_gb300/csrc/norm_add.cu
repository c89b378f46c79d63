// norm_add.cu -- residual add + RMSNorm in front of a block, forward:
//   s = residual + scale x,  out = w s rstd,  rstd = (mean(s^2) + eps)^-1/2
// A row is read once into registers, its one sum formed over the row's threads and its results
// written, so that the kernel is bound by the memory traffic of its operands: 32768 rows of 768
// columns, bf16 with an fp32 stream, scale and the stream's 8-bit checkpoint take 51 us for 328 MB
// (GB300; 57 with inputs and outputs from call to call beyond L2, 5.7 TB/s of 6.7 measured for a copy; 70
// while w and scale were loaded as single values).  Four chunks per thread (2048, 4096 and 8192 columns)
// spill 88 - 104 bytes of registers per thread, rows beyond 8192 columns 400 - 620: 8192 x 4096, all in
// bf16, takes 55 us of 40, 2048 x 16384 89 of 40.
// The stream is formed with the product and the sum rounded one after the other, so that it holds
// the same bits as an unfused add does.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

template <typename IO, typename RES, int VEC, int NJ, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) add_norm_fwd_kernel(const AddNormFwd a,
                                                                  const RowPlan pl) {
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int cols = a.cols, nb = (cols + 31) / 32;
  const float inv = 1.0f / (float)cols;
  bool okc[NJ];
  int col[NJ];
  float w[NJ][VEC], sc[NJ][VEC];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    col[j] = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && col[j] < cols;
    ld_param<VEC>(a.w, col[j], okc[j], w[j]);
    ld_param<VEC>(a.scale, col[j], okc[j], sc[j]);
  }
  // Single columns are loaded one row ahead (rows.cuh).
  typedef Operand<IO, VEC, NJ, false> Act;
  typedef Operand<RES, VEC, NJ, false> Res;
  Act x1{a.x, nullptr, nullptr, a.ld_x, 0};
  Res r1{a.residual, nullptr, nullptr, a.ld_residual, 0};
  auto ahead = [&](int r) {
    if constexpr (Act::kAhead) {
      if (r < a.rows) {
        x1.issue(0, r, col, okc, cols);
        r1.issue(0, r, col, okc, cols);
      } else {
        x1.clear(0, okc, true);
        r1.clear(0, okc, true);
      }
    }
  };
  const int step = gridDim.x * pl.rpb;  // rows stay below 2^31 - step
  int half = 0;
  ahead(blockIdx.x * pl.rpb + pos.slot);
  for (int base = blockIdx.x * pl.rpb; base < a.rows; base += step, half ^= 1) {
    const int row = base + pos.slot;
    const bool rok = row < a.rows;
    float s[NJ][VEC];
    Cols<IO, VEC> xr[NJ];
    Cols<RES, VEC> rr[NJ];
    if constexpr (Act::kAhead) {
      x1.advance();
      r1.advance();
      ahead(row + step);
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
      if constexpr (Act::kAhead) {
        x1.get(0, j, true, row, col[j], cols, 7u, xv);
        r1.get(0, j, true, row, col[j], cols, 7u, rv);
      } else {
        xr[j].get(xv);
        rr[j].get(rv);
      }
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        s[j][i] = __fadd_rn(rv[i], __fmul_rn(sc[j][i], xv[i]));
        sq = fmaf(s[j][i], s[j][i], sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum(sq, pl.tpr, part, half) * inv + a.eps);
    if (a.rstd && rok && pos.ok && pos.lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float o[VEC];
      Cols<IO, VEC> oc;
      Cols<RES, VEC> stored;
#pragma unroll
      for (int i = 0; i < VEC; i++) o[i] = w[j][i] * (s[j][i] * rstd);
      to_cols(o, oc);
      to_cols(s[j], stored);
      if (ok) {
        st_cols((IO*)a.out + (long long)row * a.ld_out + col[j], oc);
        if (a.res_out) st_cols((RES*)a.res_out + (long long)row * a.ld_res_out + col[j], stored);
      }
      const long long q = (long long)row * cols + col[j],
                      e = (long long)row * nb + (int)((unsigned)col[j] / 32);
      if (a.res_q) {
        float kept[VEC];
        stored.get(kept);
        store_ckpt8<VEC>(kept, ok, a.res_q + q, a.res_e + e);
      }
      if (a.x_q) {
        float xv[VEC];
        if constexpr (Act::kAhead) x1.get(0, j, true, row, col[j], cols, 7u, xv);
        else xr[j].get(xv);
        store_ckpt8<VEC>(xv, ok, a.x_q + q, a.x_e + e);
      }
      if (a.out_q) {
        oc.get(o);
        store_ckpt8<VEC>(o, ok, a.out_q + q, a.out_e + e);
      }
    }
  }
}

template <typename IO, typename RES, int VEC, int NJ, int MAXT, int MINB>
void fwd_launch(const AddNormFwd& a, const RowPlan& pl, cudaStream_t st) {
  add_norm_fwd_kernel<IO, RES, VEC, NJ, MAXT, MINB>
      <<<dim3(pl.nbx, pl.nby), pl.threads, 0, st>>>(a, pl);
}
template <typename IO, typename RES>
cudaError_t fwd_types(const AddNormFwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.cols, 1, vec, sms, false);
  const RowPlan& p = s.plan;
#define SSM_LAUNCH(VEC, NJ, MAXT, MINB) fwd_launch<IO, RES, VEC, NJ, MAXT, MINB>(a, p, st)
  SSM_NORM_FWD_SWITCH(s.variant, SSM_LAUNCH)
#undef SSM_LAUNCH
  count_launches(1);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_add_norm_fwd(const AddNormFwd& a, int io, int res_io, bool vec, int sms,
                                cudaStream_t st) {
  if (io == SSM_F32) return fwd_types<float, float>(a, vec, sms, st);
  if (res_io == SSM_F32) return fwd_types<__nv_bfloat16, float>(a, vec, sms, st);
  return fwd_types<__nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
}

}  // namespace ssm
