// ckpt8.cu -- 8-bit activation checkpoints: saving an activation and reading it back.  Pure
// streaming: a save reads the activation and writes 33/32 bytes per value, a load the reverse.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // chunks of VEC columns per thread

// A warp takes a segment of 32 VEC kUnroll columns of one row.
template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads) ckpt8_save_kernel(
    const IO* x, long long ld, int8_t* q, uint8_t* e, long long rows, long long cols,
    long long nb, long long segs) {
  const int lane = threadIdx.x & 31;
  const long long units = rows * segs;
  for (long long u = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5; u < units;
       u += (long long)gridDim.x * (kThreads / 32)) {
    const long long row = u / segs, c0 = (u - row * segs) * (32 * VEC * kUnroll) + lane * VEC;
    Cols<IO, VEC> r[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      const long long c = c0 + j * 32 * VEC;
      r[j].zero();
      if (c < cols) r[j].load(x + row * ld + c);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      const long long c = c0 + j * 32 * VEC;
      float v[VEC];
      r[j].get(v);
      store_ckpt8<VEC>(v, c < cols, q + row * cols + c, e + row * nb + c / 32);
    }
  }
}

template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads) ckpt8_load_kernel(
    const int8_t* q, const uint8_t* e, IO* out, long long ld, long long rows, long long cols,
    long long nb, long long segs) {
  const int lane = threadIdx.x & 31;
  const long long units = rows * segs;
  for (long long u = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5; u < units;
       u += (long long)gridDim.x * (kThreads / 32)) {
    const long long row = u / segs, c0 = (u - row * segs) * (32 * VEC * kUnroll) + lane * VEC;
    Kept<VEC> r[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      const long long c = c0 + j * 32 * VEC;
      r[j].zero();
      if (c < cols) r[j].load(q + row * cols + c, e + row * nb + c / 32);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      const long long c = c0 + j * 32 * VEC;
      float v[VEC];
      r[j].get(v);
      if (c < cols) st_cols(out + row * ld + c, v);
    }
  }
}

bool vec_ok(const void* act, long long ld, const void* q, int cols, int io) {
  const int bytes = io == SSM_F32 ? 32 : 16;
  return cols % 8 == 0 && ld % 8 == 0 && (uintptr_t)act % bytes == 0 && (uintptr_t)q % 8 == 0;
}

template <typename IO, int VEC>
cudaError_t save(const void* x, long long ld, int8_t* q, uint8_t* e, long long rows,
                 long long cols, int sms, cudaStream_t st) {
  // rows without gaps whose blocks are whole are one long row
  if (ld == cols && cols % 32 == 0) cols *= rows, ld = cols, rows = 1;
  const long long segs = (cols + 32 * VEC * kUnroll - 1) / (32 * VEC * kUnroll);
  const long long need = (rows * segs + kThreads / 32 - 1) / (kThreads / 32), most = sms * 32LL;
  ckpt8_save_kernel<IO, VEC><<<(int)(need < most ? need : most), kThreads, 0, st>>>(
      (const IO*)x, ld, q, e, rows, cols, (cols + 31) / 32, segs);
  count_launches(1);
  return cudaGetLastError();
}
template <typename IO, int VEC>
cudaError_t load(const int8_t* q, const uint8_t* e, void* out, long long ld, long long rows,
                 long long cols, int sms, cudaStream_t st) {
  if (ld == cols && cols % 32 == 0) cols *= rows, ld = cols, rows = 1;
  const long long segs = (cols + 32 * VEC * kUnroll - 1) / (32 * VEC * kUnroll);
  const long long need = (rows * segs + kThreads / 32 - 1) / (kThreads / 32), most = sms * 32LL;
  ckpt8_load_kernel<IO, VEC><<<(int)(need < most ? need : most), kThreads, 0, st>>>(
      q, e, (IO*)out, ld, rows, cols, (cols + 31) / 32, segs);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt8_save(const void* x, long long ld, int8_t* q, uint8_t* e, long long rows,
                              int cols, int io, int sms, cudaStream_t st) {
  const bool v = vec_ok(x, ld, q, cols, io);
  if (io == SSM_F32)
    return v ? save<float, 8>(x, ld, q, e, rows, cols, sms, st)
             : save<float, 1>(x, ld, q, e, rows, cols, sms, st);
  return v ? save<__nv_bfloat16, 8>(x, ld, q, e, rows, cols, sms, st)
           : save<__nv_bfloat16, 1>(x, ld, q, e, rows, cols, sms, st);
}

cudaError_t launch_ckpt8_load(const int8_t* q, const uint8_t* e, void* out, long long ld,
                              long long rows, int cols, int io, int sms, cudaStream_t st) {
  const bool v = vec_ok(out, ld, q, cols, io);
  if (io == SSM_F32)
    return v ? load<float, 8>(q, e, out, ld, rows, cols, sms, st)
             : load<float, 1>(q, e, out, ld, rows, cols, sms, st);
  return v ? load<__nv_bfloat16, 8>(q, e, out, ld, rows, cols, sms, st)
           : load<__nv_bfloat16, 1>(q, e, out, ld, rows, cols, sms, st);
}

}  // namespace ssm
