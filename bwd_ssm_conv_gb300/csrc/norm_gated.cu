// norm_gated.cu -- the gated RMSNorm after the scan, forward and backward, per group of columns:
//   gate first:  v = y silu(z),  n = v rstd(v),  out = w n
//                dv = rstd (w d_out - n mean(w d_out n)),  d_y = dv silu(z),  d_z = dv y silu'(z)
//   norm first:  n = y rstd(y),  out = w n silu(z),  dn = w d_out silu(z)
//                d_y = rstd (dn - n mean(dn n)),  d_z = w d_out n silu'(z)
// A group is read once, copied to shared memory (rows.cuh; ahead, but for fp32 rows of four chunks per
// thread, and with plain loads beyond 8192 columns, in the backward beyond 4096), and its one sum
// formed over its threads.  The sigmoid is taken once per value in each direction.
//
// What bounds them (32768 rows of 1536 bf16 columns, checkpoints of y and z, GB300):
//   forward   67 us, 406 MB: 6.1 TB/s of 6.7 measured for a copy, and 57 % of the issue slots.
//             Largest magnitudes of bf16 blocks taken two at a time, and one fused rounding per
//             value, brought 94 -> 74 us; rows and strides in 32 bits 74 -> 67 us.
//   backward  93 us, 406 MB at 4.4 TB/s: issue slots (58 % busy at 14 warps per SM, which wait for
//             their own results).  The rows read with plain loads took 191 us, the next row
//             loaded ahead into registers (which spill) 252 us, copied ahead 134 us; fewer chunks per
//             thread (norm_shape) and all blocks resident 108 us, 32-bit rows and strides 93 us,
//             pairs of values per instruction 90 us; 1 us goes to scale bytes below 7 (block_step).
//             One chunk per thread, for twice the warps, takes 10 us more.
// Beyond 4096 columns the backward spills 1.2 KB per thread (single columns 0.7 - 3.0 KB): bf16,
// 4096 x 8192 139 us of 50, 2048 x 16384 271 of 50.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

template <typename IO, int VEC, int NJ, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) gated_norm_fwd_kernel(const GatedNormFwd a,
                                                                    const RowPlan pl) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int nb = (a.cols + 31) / 32;
  const float inv = 1.0f / (float)a.group;
  const int grp = pos.col0 / a.group;
  bool okc[NJ];
  int col[NJ];
  float w[NJ][VEC];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    const int c = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && c < a.group;
    col[j] = pos.col0 + c;
    ld_param<VEC>(a.w, col[j], okc[j], w[j]);
  }
  typedef Operand<IO, VEC, NJ, (VEC == 8 && MAXT <= 256)> Op;
  typedef Packed<VEC> P;
  const uint32_t bytes = Op::slot_bytes(blockDim.x), at = shared_addr(ring) + 16 * threadIdx.x;
  Op y{a.y, nullptr, nullptr, a.ld_y, at}, z{a.z, nullptr, nullptr, a.ld_z, at + bytes};
  const int step = gridDim.x * pl.rpb;  // rows stay below 2^31 - step
  int row = blockIdx.x * pl.rpb + pos.slot;
  auto issue = [&](int r, int slot) {
    if (r < a.rows) {
      y.issue(slot * 2 * bytes, r, col, okc, a.cols);
      z.issue(slot * 2 * bytes, r, col, okc, a.cols);
    }
    cp_async_commit();
  };
  for (int i = 0; i < pl.slots; i++) {
    y.clear(i * 2 * bytes, okc, false);
    z.clear(i * 2 * bytes, okc, false);
  }
  const int ahead = pl.slots - 1;
  for (int i = 0; i < ahead; i++) issue(row + i * step, i);
  int half = 0, slot = 0;
  for (int base = blockIdx.x * pl.rpb; base < a.rows; base += step, row += step, half ^= 1) {
    const bool rok = row < a.rows;
    y.advance();
    z.advance();
    issue(row + ahead * step, slot == 0 ? ahead : slot - 1);
    cp_async_wait(ahead);
    const uint32_t s = slot * 2 * bytes;
    slot = slot == ahead ? 0 : slot + 1;
    const long long qrow = (long long)row * a.cols, erow = (long long)row * nb;
    float v[NJ][VEC];
    typename P::T sq = P::of(0.0f);
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float zv[VEC];
      y.get(s, j, ok, row, col[j], a.cols, 7u, v[j]);
      z.get(s, j, ok, row, col[j], a.cols, 7u, zv);
      if (a.y_q) {  // both checkpoints or neither (block_api.cu)
        const uint32_t ytop = y.top(s, j, v[j]), ztop = z.top(s, j, zv);
        const int blk = (int)((unsigned)col[j] / 32);
        store_ckpt8_top<VEC>(v[j], ytop, ok, a.y_q + qrow + col[j], a.y_e + erow + blk);
        store_ckpt8_top<VEC>(zv, ztop, ok, a.z_q + qrow + col[j], a.z_e + erow + blk);
      }
#pragma unroll
      for (int i = 0; i < P::N; i++) {
        typename P::T t = P::at(v[j], i);
        if (!a.norm_first) {
          const typename P::T z2 = P::at(zv, i);
          t = mul_(t, mul_(z2, sigmoid_(z2)));
          P::put(v[j], i, t);
        }
        sq = fma_(t, t, sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum(P::sum(sq), pl.tpr, part, half) * inv + a.eps);
    if (a.rstd && rok && pos.ok && pos.lane == 0)
      a.rstd[(long long)row * pl.groups + grp] = rstd;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float o[VEC], zv[VEC];
      if (a.norm_first) z.get(s, j, ok, row, col[j], a.cols, 7u, zv);
#pragma unroll
      for (int i = 0; i < P::N; i++) {
        typename P::T t = mul_(P::at(w[j], i), mul_(P::at(v[j], i), P::of(rstd)));
        if (a.norm_first) {
          const typename P::T z2 = P::at(zv, i);
          t = mul_(t, mul_(z2, sigmoid_(z2)));
        }
        P::put(o, i, t);
      }
      Cols<IO, VEC> oc;
      to_cols(o, oc);
      if (ok) st_cols((IO*)a.out + (long long)row * a.ld_out + col[j], oc);
      if (a.out_q) {
        oc.get(o);
        store_ckpt8<VEC>(o, ok, a.out_q + qrow + col[j],
                         a.out_e + erow + (int)((unsigned)col[j] / 32));
      }
    }
  }
}

template <typename IO, int VEC, int NJ, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) gated_norm_bwd_kernel(const GatedNormBwd a,
                                                                    const RowPlan pl) {
  extern __shared__ __align__(16) unsigned char ring[];  // at the end: the slots' column sums
  __shared__ float part[2][32];
  const RowPos pos = row_pos(pl);
  const int nb = (a.cols + 31) / 32;
  const float inv = 1.0f / (float)a.group;
  const int grp = pos.col0 / a.group;
  bool okc[NJ];
  int col[NJ];
  typedef Packed<VEC> P;
  typedef typename P::T T;
  T w[NJ][P::N], dw[NJ][P::N];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    const int c = (pos.lane + j * pl.tpr) * VEC;
    okc[j] = pos.ok && c < a.group;
    col[j] = pos.col0 + c;
    float wv[VEC];
    ld_param<VEC>(a.w, col[j], okc[j], wv);
#pragma unroll
    for (int i = 0; i < P::N; i++) w[j][i] = P::at(wv, i), dw[j][i] = P::of(0.0f);
  }
  typedef Operand<IO, VEC, NJ, (VEC == 8 && MAXT <= 256)> Op;
  const uint32_t bytes = Op::slot_bytes(blockDim.x), at = shared_addr(ring) + 16 * threadIdx.x;
  Op d{a.d_out, nullptr, nullptr, a.ld_d_out, at}, y{a.y, a.y_q, a.y_e, a.ld_y, at + bytes},
      z{a.z, a.z_q, a.z_e, a.ld_z, at + 2 * bytes};
  const int step = gridDim.x * pl.rpb;  // rows stay below 2^31 - step
  int row = blockIdx.x * pl.rpb + pos.slot;
  auto issue = [&](int r, int slot) {
    const uint32_t s = slot * 3 * bytes;
    if (r < a.rows) {
      d.issue(s, r, col, okc, a.cols);
      y.issue(s, r, col, okc, a.cols);
      z.issue(s, r, col, okc, a.cols);
    } else {  // adds nothing to the column sums
      d.clear(s, okc, true);
      y.clear(s, okc, true);
      z.clear(s, okc, true);
    }
    cp_async_commit();
  };
  // what a row needs besides: read one row ahead
  float rstd_next = 0.0f;
  uint32_t ey_next[NJ], ez_next[NJ];
  auto small = [&](int r) {
    const bool rok = r < a.rows;
    rstd_next = rok && pos.ok ? a.rstd_in[(long long)r * pl.groups + grp] : 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      ey_next[j] = y.scale(rok && okc[j], r, col[j], nb);
      ez_next[j] = z.scale(rok && okc[j], r, col[j], nb);
    }
  };
  for (int i = 0; i < pl.slots; i++) {
    d.clear(i * 3 * bytes, okc, false);
    y.clear(i * 3 * bytes, okc, false);
    z.clear(i * 3 * bytes, okc, false);
  }
  const int ahead = pl.slots - 1;
  for (int i = 0; i < ahead; i++) issue(row + i * step, i);
  small(row);
  int half = 0, slot = 0;
  for (int base = blockIdx.x * pl.rpb; base < a.rows; base += step, row += step, half ^= 1) {
    const bool rok = row < a.rows;
    const float rstd = rstd_next;
    uint32_t ey[NJ], ez[NJ];
#pragma unroll
    for (int j = 0; j < NJ; j++) ey[j] = ey_next[j], ez[j] = ez_next[j];
    small(row + step);
    d.advance();
    y.advance();
    z.advance();
    issue(row + ahead * step, slot == 0 ? ahead : slot - 1);
    cp_async_wait(ahead);
    const uint32_t s = slot * 3 * bytes;
    slot = slot == ahead ? 0 : slot + 1;
    // What the second pass needs of y and z, so that it does not unpack them again: g = silu(z),
    // m = n / rstd, b = y silu'(z) (gate first) or d_z already (norm first)
    T g[NJ][P::N], b[NJ][P::N], m[NJ][P::N], dot = P::of(0.0f);
    const T rs = P::of(rstd);
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float dv[VEC], yv[VEC], zv[VEC];
      d.get(s, j, ok, row, col[j], a.cols, 7u, dv);
      y.get(s, j, ok, row, col[j], a.cols, ey[j], yv);
      z.get(s, j, ok, row, col[j], a.cols, ez[j], zv);
#pragma unroll
      for (int i = 0; i < P::N; i++) {
        const T y2 = P::at(yv, i), z2 = P::at(zv, i), sg = sigmoid_(z2);
        const T dr = mul_(P::at(dv, i), rs);
        g[j][i] = mul_(z2, sg);
        b[j][i] = mul_(y2, fma_(g[j][i], fma_(sg, P::of(-1.0f), P::of(1.0f)), sg));
        m[j][i] = mul_(y2, g[j][i]);
        const T t = mul_(dr, m[j][i]);  // d_out times n and gate
        dw[j][i] = add_(dw[j][i], t);
        dot = fma_(w[j][i], t, dot);
        if (a.norm_first) m[j][i] = y2, b[j][i] = mul_(b[j][i], mul_(w[j][i], dr));
      }
    }
    const T c = P::of(-row_sum(P::sum(dot), pl.tpr, part, half) * inv * rstd);
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool ok = rok && okc[j];
      float dv[VEC], dy[VEC], dz[VEC];
      d.get(s, j, ok, row, col[j], a.cols, 7u, dv);
#pragma unroll
      for (int i = 0; i < P::N; i++) {
        T t = mul_(w[j][i], P::at(dv, i));
        if (a.norm_first) {
          P::put(dy, i, mul_(rs, fma_(m[j][i], c, mul_(t, g[j][i]))));
          P::put(dz, i, b[j][i]);
        } else {
          t = mul_(rs, fma_(m[j][i], c, t));
          P::put(dy, i, mul_(t, g[j][i]));
          P::put(dz, i, mul_(t, b[j][i]));
        }
      }
      if (ok) {
        st_cols((IO*)a.d_y + (long long)row * a.ld_d_y + col[j], dy);
        st_cols((IO*)a.d_z + (long long)row * a.ld_d_z + col[j], dz);
      }
    }
  }
  cp_async_wait(0);
  if (a.d_w) {
    float sums[NJ][VEC];
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
      for (int i = 0; i < P::N; i++) P::put(sums[j], i, dw[j][i]);
    store_partial<VEC, NJ>(sums, pl, pos, col, okc, a.cols, a.part, (float*)ring);
  }
}

template <typename IO, int VEC, int NJ, int MAXT, int MINB>
cudaError_t fwd_launch(const GatedNormFwd& a, RowPlan pl, int per_sm, cudaStream_t st) {
  const uint32_t slot = 2 * Operand<IO, VEC, NJ, (VEC == 8 && MAXT <= 256)>::slot_bytes(pl.threads);
  pl.slots = VEC == 1 ? 2 : ring_slots(slot, pl.threads, per_sm);
  return launch_rows<gated_norm_fwd_kernel<IO, VEC, NJ, MAXT, MINB>>(a, pl, pl.slots * slot, st);
}
template <typename IO, int VEC, int NJ, int MAXT, int MINB>
cudaError_t bwd_launch(const GatedNormBwd& a, RowPlan pl, int per_sm, cudaStream_t st) {
  const uint32_t slot = 3 * Operand<IO, VEC, NJ, (VEC == 8 && MAXT <= 256)>::slot_bytes(pl.threads);
  pl.slots = VEC == 1 ? 2 : ring_slots(slot, pl.threads, per_sm);
  const size_t ring = (size_t)pl.slots * slot, sums = slots_bytes(pl, VEC, NJ);
  return launch_rows<gated_norm_bwd_kernel<IO, VEC, NJ, MAXT, MINB>>(
      a, pl, ring > sums ? ring : sums, st);
}

template <typename IO>
cudaError_t fwd_types(const GatedNormFwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.group, a.cols / a.group, vec, sms, false);
  count_launches(1);
#define SSM_LAUNCH(VEC, NJ, MAXT, MINB) \
  return fwd_launch<IO, VEC, NJ, MAXT, MINB>(a, s.plan, norm_threads_per_sm(s.variant, false), st)
  SSM_NORM_FWD_SWITCH(s.variant, SSM_LAUNCH)
#undef SSM_LAUNCH
}
template <typename IO>
cudaError_t bwd_types(const GatedNormBwd& a, bool vec, int sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.rows, a.group, a.cols / a.group, vec, sms, true);
  count_launches(1);
  cudaError_t e;
#define SSM_LAUNCH(VEC, NJ, MAXT, MINB) \
  e = bwd_launch<IO, VEC, NJ, MAXT, MINB>(a, s.plan, norm_threads_per_sm(s.variant, true), st)
  SSM_NORM_BWD_SWITCH(s.variant, SSM_LAUNCH)
#undef SSM_LAUNCH
  if (e != cudaSuccess || !a.d_w) return e;
  return launch_column_sums(a.part, s.plan.nbx, a.cols, a.d_w, nullptr, nullptr, st);
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
