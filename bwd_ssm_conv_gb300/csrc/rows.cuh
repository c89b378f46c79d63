// rows.cuh -- what the row-wise operators (norms, 8-bit checkpoints) share: vector loads and
// stores of a row's columns, sums over the threads of a row, and the 8-bit block format.
//
// A thread takes VEC consecutive columns at a time: 8 where widths, strides and pointers allow
// (one 16- or 32-byte access), else 1.
#pragma once

#include "common.cuh"
#include "ssm_block.h"

namespace ssm {

// ---- VEC columns of a row --------------------------------------------------------------------
template <typename IO, int VEC> struct Cols;  // the loaded bits, unpacked when they are used

template <> struct Cols<float, 1> {
  float a;
  __device__ __forceinline__ void load(const float* p) { a = *p; }
  __device__ __forceinline__ void zero() { a = 0.0f; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = a; }
};
template <> struct Cols<__nv_bfloat16, 1> {
  __nv_bfloat16 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *p; }
  __device__ __forceinline__ void zero() { a = __float2bfloat16_rn(0.0f); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __bfloat162float(a); }
};
template <> struct Cols<float, 8> {
  float a[8];
  __device__ __forceinline__ void load(const float* p) {  // 32-byte aligned
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]),
                   "=f"(a[6]), "=f"(a[7])
                 : "l"(p)
                 : "memory");
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; i++) a[i] = 0.0f;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = a[i];
  }
};
template <> struct Cols<__nv_bfloat16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {  // 16-byte aligned
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void st_cols(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void st_cols(__nv_bfloat16* p, const float (&v)[1]) {
  *p = __float2bfloat16_rn(v[0]);
}
__device__ __forceinline__ void st_cols(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void st_cols(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]),
                                            bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
}
// The value as the type stores it.
template <typename IO> __device__ __forceinline__ float rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ float rounded<__nv_bfloat16>(float v) {
  return __bfloat162float(__float2bfloat16_rn(v));
}
// fp32 parameters of VEC columns (1 where there are none).
template <int VEC>
__device__ __forceinline__ void ld_param(const float* p, int col, bool ok, float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; i++) v[i] = (ok && p) ? __ldg(p + col + i) : 1.0f;
}

// ---- the 8-bit block format (ssm_block.h) ------------------------------------------------------
// A block's 32 columns lie in 32 / VEC consecutive lanes.  The largest magnitude is taken as an
// unsigned comparison of the bits, which orders NaN above infinity above every finite value.
template <int VEC>
__device__ __forceinline__ uint32_t block_top(const float (&v)[VEC]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VEC; i++) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  if constexpr (VEC == 1) {
    top = __reduce_max_sync(0xffffffffu, top);
  } else {
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  }
  return top;
}
// E + 127 of a block, 255 where a value is not finite.
__device__ __forceinline__ uint32_t block_exp(uint32_t top) {
  const uint32_t x = top >> 23;  // E + 127 of a normal number; 0 for zero and subnormals
  return x < 7u ? 7u : x;        // E >= -120; 255 stays
}
// 2^(6 - E) and 2^(E - 6) from e = E + 127 in 7 .. 254 (both normal numbers).
__device__ __forceinline__ float block_up(uint32_t e) { return __uint_as_float((260u - e) << 23); }
__device__ __forceinline__ float block_step(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : (e - 6u) << 23);
}
// Four values of a block as bytes: v 2^(6 - E) lies within +-128, is limited to +-127 and rounded to
// the nearest even integer by adding 1.5 2^23, whose low byte is then the two's complement value.
__device__ __forceinline__ uint32_t quant_bits(float v, float up) {
  return __float_as_uint(fminf(fmaxf(v * up, -127.0f), 127.0f) + 12582912.0f);
}
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Quantises VEC columns of a row and stores them at q (and, in the block's first lane, *e).  Every
// lane of the warp calls it; lanes with !ok hold zeros and store nothing.
template <int VEC>
__device__ __forceinline__ void store_ckpt8(const float (&v)[VEC], bool ok, int8_t* q, uint8_t* e) {
  const uint32_t x = block_exp(block_top<VEC>(v));
  const float up = block_up(x);
  if (ok) {
    if constexpr (VEC == 1) {
      *q = x == 255u ? (int8_t)0 : (int8_t)(quant_bits(v[0], up) & 0xffu);
    } else {
      uint2 w;
      w.x = pack_low_bytes(quant_bits(v[0], up), quant_bits(v[1], up), quant_bits(v[2], up),
                           quant_bits(v[3], up));
      w.y = pack_low_bytes(quant_bits(v[4], up), quant_bits(v[5], up), quant_bits(v[6], up),
                           quant_bits(v[7], up));
      if (x == 255u) w = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(q) = w;
    }
    if ((threadIdx.x & (32 / VEC - 1)) == 0) *e = (uint8_t)x;
  }
}
// VEC columns of a checkpoint: the loaded bits, and their values.
template <int VEC> struct Kept;
template <> struct Kept<1> {
  int8_t q;
  uint8_t e;
  __device__ __forceinline__ void load(const int8_t* pq, const uint8_t* pe) { q = *pq; e = *pe; }
  __device__ __forceinline__ void zero() { q = 0; e = 7; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = (float)q * block_step(e); }
};
template <> struct Kept<8> {
  uint2 q;
  uint8_t e;
  __device__ __forceinline__ void load(const int8_t* pq, const uint8_t* pe) {  // 8-byte aligned
    q = *reinterpret_cast<const uint2*>(pq);
    e = *pe;
  }
  __device__ __forceinline__ void zero() { q = make_uint2(0u, 0u); e = 7; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const float step = block_step(e);
    const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};  // q + 128 in each byte
#pragma unroll
    for (int i = 0; i < 8; i++) {  // 2^23 + (q + 128) as a float, minus 2^23 + 128: exactly q
      const uint32_t b = __byte_perm(w[i >> 2], 0x4b000000u, 0x7650u + (i & 3));
      v[i] = (__uint_as_float(b) - 8388736.0f) * step;
    }
  }
};

// ---- how a row's threads are laid out ----------------------------------------------------------
// A row is `groups` groups of `group` columns.  tpr threads (a power of two up to 32, or whole
// warps) take a group: thread i of them columns VEC (i + j tpr), j < NJ.  A block holds gpb groups
// of rpb rows; blockIdx.y steps over the groups, blocks step over the rows by gridDim.x rpb.
struct RowPlan {
  int tpr, gpb, rpb;  // tpr > 32: gpb = rpb = 1
  int group, groups;
  int threads, nbx, nby;
};

struct RowPos {
  int slot, col0, lane;  // row within the block's rpb, first column of the group, thread in it
  bool ok;
};
__device__ __forceinline__ RowPos row_pos(const RowPlan& p) {
  RowPos r;
  const int s = (int)threadIdx.x / p.tpr;
  r.lane = (int)threadIdx.x - s * p.tpr;
  r.slot = s / p.gpb;
  const int g = blockIdx.y * p.gpb + (s - r.slot * p.gpb);
  r.col0 = g * p.group;
  r.ok = r.slot < p.rpb && g < p.groups;
  return r;
}

// Sum over a group's threads, the same bits in each of them.  Within a warp by xor shuffles; over
// warps through `part` (2 x 32 floats: consecutive calls alternate halves, so that one barrier per
// call is enough).  Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, int tpr, float (*part)[32], int half) {
  if (tpr <= 32) {
    for (int off = tpr >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[half][threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < tpr >> 5; w++) s += part[half][w];
  return s;
}

// ---- host: launch plans ---------------------------------------------------------------------
inline int round_up32(int v) { return (v + 31) / 32 * 32; }

// Threads of a row for groups of nch chunks at nj chunks per thread.
inline int row_threads(int nch, int nj, int vec) {
  const int t = (nch + nj - 1) / nj;
  if (t >= 32 || vec == 1) return round_up32(t);
  int p = 4;  // a block of the 8-bit format spans 4 threads of 8 columns
  while (p < t) p <<= 1;
  return p;
}

inline RowPlan row_plan(long long rows, int group, int groups, int tpr, int block, int per_sm,
                        int sms) {
  RowPlan p{};
  p.tpr = tpr;
  p.group = group;
  p.groups = groups;
  p.gpb = p.rpb = 1;
  if (tpr <= 32) {
    const int teams = block / tpr > 0 ? block / tpr : 1;
    p.gpb = groups < teams ? groups : teams;
    p.rpb = teams / p.gpb;
    if (p.rpb > rows) p.rpb = (int)rows;
  }
  p.threads = round_up32(p.tpr * p.gpb * p.rpb);
  p.nby = (groups + p.gpb - 1) / p.gpb;
  const long long need = (rows + p.rpb - 1) / p.rpb;
  const long long most = ((long long)sms * per_sm + p.nby - 1) / p.nby;
  p.nbx = (int)(need < most ? need : most);
  if (p.nbx < 1) p.nbx = 1;
  return p;
}

}  // namespace ssm
