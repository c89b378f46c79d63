// ckpt8.cu -- 8-bit activation checkpoints: saving an activation and reading it back.  Pure
// streaming: a save reads the activation and writes 33/32 bytes per value, a load the reverse.
// 16384 x 2048 bf16 (GB300): 18.5 and 18.8 us for 102 MB each, 5.5 TB/s of 6.7 measured for a copy, with
// inputs and outputs beyond L2; a save and its load back to back 34, the load finding part of the
// checkpoint in L2 (35 while every segment's row was found by a 64-bit division).  Single columns,
// 16384 x 2047: 45 and 37 us.
#include "block.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // chunks of VEC columns per thread, all loaded before the first is used

// A warp takes a segment of 32 VEC kUnroll columns of one row: unit u is segment u % segs of row
// u / segs.  FLAT: rows without gaps between them are one long row, and nothing is divided.
template <bool FLAT, int VEC> struct Place {
  long long row, c0;
  __device__ __forceinline__ Place(long long u, unsigned segs, int lane) {
    if constexpr (FLAT) {
      row = 0;
      c0 = u * (32 * VEC * kUnroll) + lane * VEC;
    } else {
      row = (unsigned)u / segs;
      c0 = (long long)((unsigned)u - (unsigned)row * segs) * (32 * VEC * kUnroll) + lane * VEC;
    }
  }
};

template <typename IO, int VEC>
__device__ __forceinline__ uint32_t top_of(const Cols<IO, VEC>& c, const float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(IO) == 2) return block_top(c.a);
  else return block_top<VEC>(v);
}

template <typename IO, int VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) ckpt8_save_kernel(const IO* x, long long ld, int8_t* q,
                                                              uint8_t* e, long long cols,
                                                              long long nb, unsigned segs,
                                                              long long units) {
  const int lane = threadIdx.x & 31;
  for (long long u = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5; u < units;
       u += (long long)gridDim.x * (kThreads / 32)) {
    const Place<FLAT, VEC> at(u, segs, lane);
    const IO* xr = x + at.row * ld + at.c0;
    int8_t* qr = q + at.row * cols + at.c0;
    uint8_t* er = e + at.row * nb + at.c0 / 32;
    Cols<IO, VEC> r[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      r[j].zero();
      if (at.c0 + j * 32 * VEC < cols) r[j].load(xr + j * 32 * VEC);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      float v[VEC];
      r[j].get(v);
      store_ckpt8_top<VEC>(v, top_of<IO, VEC>(r[j], v), at.c0 + j * 32 * VEC < cols,
                           qr + j * 32 * VEC, er + j * VEC);
    }
  }
}

template <typename IO, int VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) ckpt8_load_kernel(const int8_t* q, const uint8_t* e,
                                                              IO* out, long long ld,
                                                              long long cols, long long nb,
                                                              unsigned segs, long long units) {
  const int lane = threadIdx.x & 31;
  for (long long u = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5; u < units;
       u += (long long)gridDim.x * (kThreads / 32)) {
    const Place<FLAT, VEC> at(u, segs, lane);
    IO* o = out + at.row * ld + at.c0;
    const int8_t* qr = q + at.row * cols + at.c0;
    const uint8_t* er = e + at.row * nb + at.c0 / 32;
    Kept<VEC> r[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      r[j].zero();
      if (at.c0 + j * 32 * VEC < cols) r[j].load(qr + j * 32 * VEC, er + j * VEC);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      float v[VEC];
      r[j].get(v);
      if (at.c0 + j * 32 * VEC < cols) st_cols(o + j * 32 * VEC, v);
    }
  }
}

bool vec_ok(const void* act, long long ld, const void* q, int cols, int io) {
  const int bytes = io == SSM_F32 ? 32 : 16;
  return cols % 8 == 0 && ld % 8 == 0 && (uintptr_t)act % bytes == 0 && (uintptr_t)q % 8 == 0;
}

// Calls launch(first row, rows, columns, stride, segments, units, flat) for the whole activation:
// once, unless the units of rows with gaps between them pass 32 bits.
template <int VEC, typename F>
cudaError_t for_rows(long long rows, long long cols, long long ld, F launch) {
  constexpr int kSeg = 32 * VEC * kUnroll;
  if (ld == cols && cols % 32 == 0) {  // no gaps, and blocks that end with their rows
    const long long n = rows * cols;
    return launch(0, n, n, (unsigned)1, (n + kSeg - 1) / kSeg, true);
  }
  const long long segs = (cols + kSeg - 1) / kSeg, most = 0x7fffffffLL / segs;
  for (long long r = 0; r < rows; r += most) {
    const long long n = rows - r < most ? rows - r : most;
    if (cudaError_t e = launch(r, cols, ld, (unsigned)segs, n * segs, false)) return e;
  }
  return cudaSuccess;
}
int blocks_of(long long units, int sms) {
  const long long need = (units + kThreads / 32 - 1) / (kThreads / 32), most = sms * 32LL;
  return (int)(need < most ? need : most);
}

template <typename IO, int VEC>
cudaError_t save(const void* x, long long ld, int8_t* q, uint8_t* e, long long rows,
                 long long cols, int sms, cudaStream_t st) {
  const long long nb = (cols + 31) / 32;
  return for_rows<VEC>(rows, cols, ld, [&](long long r, long long c, long long l, unsigned segs,
                                           long long units, bool flat) {
    auto kernel = flat ? ckpt8_save_kernel<IO, VEC, true> : ckpt8_save_kernel<IO, VEC, false>;
    kernel<<<blocks_of(units, sms), kThreads, 0, st>>>((const IO*)x + r * ld, l, q + r * cols,
                                                       e + r * nb, c, nb, segs, units);
    count_launches(1);
    return cudaGetLastError();
  });
}
template <typename IO, int VEC>
cudaError_t load(const int8_t* q, const uint8_t* e, void* out, long long ld, long long rows,
                 long long cols, int sms, cudaStream_t st) {
  const long long nb = (cols + 31) / 32;
  return for_rows<VEC>(rows, cols, ld, [&](long long r, long long c, long long l, unsigned segs,
                                           long long units, bool flat) {
    auto kernel = flat ? ckpt8_load_kernel<IO, VEC, true> : ckpt8_load_kernel<IO, VEC, false>;
    kernel<<<blocks_of(units, sms), kThreads, 0, st>>>(q + r * cols, e + r * nb,
                                                       (IO*)out + r * ld, l, c, nb, segs, units);
    count_launches(1);
    return cudaGetLastError();
  });
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
