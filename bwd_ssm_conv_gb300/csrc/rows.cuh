// rows.cuh -- what the row-wise operators (norms, 8-bit checkpoints) share: vector loads and
// stores of a row's columns, sums over the threads of a row, and the 8-bit block format.
//
// A thread takes VEC consecutive columns at a time: 8 where widths, strides and pointers allow
// (one 16- or 32-byte access), else 1.
#pragma once

#include <atomic>

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
// Values as the type stores them: rounded once, here.
__device__ __forceinline__ void to_cols(const float (&v)[1], Cols<float, 1>& c) { c.a = v[0]; }
__device__ __forceinline__ void to_cols(const float (&v)[1], Cols<__nv_bfloat16, 1>& c) {
  c.a = __float2bfloat16_rn(v[0]);
}
__device__ __forceinline__ void to_cols(const float (&v)[8], Cols<float, 8>& c) {
#pragma unroll
  for (int i = 0; i < 8; i++) c.a[i] = v[i];
}
__device__ __forceinline__ void to_cols(const float (&v)[8], Cols<__nv_bfloat16, 8>& c) {
  c.a = make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]),
                   bf16x2_rn(v[6], v[7]));
}
__device__ __forceinline__ void st_cols(float* p, const Cols<float, 1>& c) { *p = c.a; }
__device__ __forceinline__ void st_cols(__nv_bfloat16* p, const Cols<__nv_bfloat16, 1>& c) {
  *p = c.a;
}
__device__ __forceinline__ void st_cols(float* p, const Cols<float, 8>& c) { st_cols(p, c.a); }
__device__ __forceinline__ void st_cols(__nv_bfloat16* p, const Cols<__nv_bfloat16, 8>& c) {
  *reinterpret_cast<uint4*>(p) = c.a;
}
// fp32 parameters of VEC columns (`none` where there are none), 16-byte aligned for VEC = 8.
template <int VEC>
__device__ __forceinline__ void ld_param(const float* p, int col, bool ok, float (&v)[VEC],
                                         float none = 1.0f) {
#pragma unroll
  for (int i = 0; i < VEC; i++) v[i] = none;
  if (ok && p) {
    if constexpr (VEC == 1) {
      v[0] = __ldg(p + col);
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + col));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p + col) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  }
}

// A chunk's values for arithmetic: pairs of columns (one instruction for two) or the single one.
template <int VEC> struct Packed {
  typedef f2_t T;
  static constexpr int N = VEC / 2;
  static __device__ __forceinline__ T of(float v) { return f2_pack(v, v); }
  static __device__ __forceinline__ T at(const float (&v)[VEC], int i) {
    return f2_pack(v[2 * i], v[2 * i + 1]);
  }
  static __device__ __forceinline__ void put(float (&v)[VEC], int i, T x) {
    f2_unpack(x, v[2 * i], v[2 * i + 1]);
  }
  static __device__ __forceinline__ float sum(T x) {
    float a, b;
    f2_unpack(x, a, b);
    return a + b;
  }
};
template <> struct Packed<1> {
  typedef float T;
  static constexpr int N = 1;
  static __device__ __forceinline__ T of(float v) { return v; }
  static __device__ __forceinline__ T at(const float (&v)[1], int) { return v[0]; }
  static __device__ __forceinline__ void put(float (&v)[1], int, T x) { v[0] = x; }
  static __device__ __forceinline__ float sum(T x) { return x; }
};
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f2_t mul_(f2_t a, f2_t b) { return f2_mul(a, b); }
__device__ __forceinline__ f2_t add_(f2_t a, f2_t b) { return f2_add(a, b); }
__device__ __forceinline__ f2_t fma_(f2_t a, f2_t b, f2_t c) { return f2_fma(a, b, c); }
__device__ __forceinline__ float sigmoid_(float v) { return sigmoidf_(v); }
__device__ __forceinline__ f2_t sigmoid_(f2_t v) {
  float a, b;
  f2_unpack(f2_mul(v, f2_pack(-kLog2e, -kLog2e)), a, b);
  f2_unpack(f2_add(f2_pack(ex2(a), ex2(b)), f2_pack(1.0f, 1.0f)), a, b);
  return f2_pack(rcp_approx(a), rcp_approx(b));
}

// ---- the 8-bit block format (ssm_block.h) ------------------------------------------------------
// A block's 32 columns lie in 32 / VEC consecutive lanes.
// The larger magnitude, NaN if either is one (its sign is left undefined).
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The bits of the block's largest magnitude (0x7f800000 and above: not finite).
template <int VEC>
__device__ __forceinline__ uint32_t block_top(const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    return __reduce_max_sync(0xffffffffu, __float_as_uint(v[0]) & 0x7fffffffu);
  } else {
    float t = max_abs(max_abs(max_abs(v[0], v[1]), max_abs(v[2], v[3])),
                      max_abs(max_abs(v[4], v[5]), max_abs(v[6], v[7])));
    t = max_abs(t, __shfl_xor_sync(0xffffffffu, t, 1));
    t = max_abs(t, __shfl_xor_sync(0xffffffffu, t, 2));
    return __float_as_uint(t) & 0x7fffffffu;
  }
}
// E + 127 of a block, 255 where a value is not finite.
__device__ __forceinline__ uint32_t block_exp(uint32_t top) {
  const uint32_t x = top >> 23;  // E + 127 of a normal number; 0 for zero and subnormals
  return x < 7u ? 7u : x;        // E >= -120; 255 stays
}
// 2^(6 - E) from e = E + 127 in 7 .. 254, as a save makes it (a normal number).
__device__ __forceinline__ float block_up(uint32_t e) { return __uint_as_float((260u - e) << 23); }
// 2^(E - 6) = 2^(e - 133) from any e that a checkpoint may hold, by way of 2^(e - 127) (a subnormal
// number for e = 0); below 7, where a save writes none but a buffer filled with zeros does, it is
// subnormal.
__device__ __forceinline__ float block_step(uint32_t e) {
  const float f = __uint_as_float(max(e << 23, 0x00400000u)) * 0.015625f;
  return e == 255u ? __uint_as_float(0x7fc00000u) : f;
}
// A value as a byte: v 2^(6 - E), within +-128, is rounded to the nearest even integer by adding
// 1.5 2^23 (one rounding, the product being exact); the low byte is then the two's complement value.
// Only where the block's largest magnitude rounds up to 128 (its leading 8 bits are ones) does the
// limit of +-127 matter: kLimit.
template <bool kLimit> __device__ __forceinline__ uint32_t quant_bits(float v, float up) {
  if constexpr (kLimit) v = fminf(fmaxf(v * up, -127.0f), 127.0f), up = 1.0f;
  return __float_as_uint(fmaf(v, up, 12582912.0f));
}
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
template <bool kLimit> __device__ __forceinline__ uint2 quant8(const float (&v)[8], float up) {
  if constexpr (!kLimit) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 4; i++)
      f2_unpack(f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), f2_pack(up, up),
                       f2_pack(12582912.0f, 12582912.0f)),
                r[2 * i], r[2 * i + 1]);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; i++) b[i] = __float_as_uint(r[i]);
    return make_uint2(pack_low_bytes(b[0], b[1], b[2], b[3]),
                      pack_low_bytes(b[4], b[5], b[6], b[7]));
  }
  return make_uint2(pack_low_bytes(quant_bits<kLimit>(v[0], up), quant_bits<kLimit>(v[1], up),
                                   quant_bits<kLimit>(v[2], up), quant_bits<kLimit>(v[3], up)),
                    pack_low_bytes(quant_bits<kLimit>(v[4], up), quant_bits<kLimit>(v[5], up),
                                   quant_bits<kLimit>(v[6], up), quant_bits<kLimit>(v[7], up)));
}
// The same from 8 values as bf16 pairs, which hold the largest magnitude as they are.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t block_top(const uint4& v) {
  uint32_t t = max_abs2(max_abs2(v.x, v.y), max_abs2(v.z, v.w));
  t = max_abs2(t, __shfl_xor_sync(0xffffffffu, t, 1));
  t = max_abs2(t, __shfl_xor_sync(0xffffffffu, t, 2));
  const uint32_t lo = (t << 16) & 0x7fffffffu, hi = t & 0x7fff0000u;
  return lo > hi ? lo : hi;
}
// Quantises VEC columns of a row, whose block's largest magnitude is `top`, and stores them at q
// (and, in the block's first lane, *e).  Every lane of the warp calls it; lanes with !ok hold zeros
// and store nothing.
template <int VEC>
__device__ __forceinline__ void store_ckpt8_top(const float (&v)[VEC], uint32_t top, bool ok,
                                                int8_t* q, uint8_t* e) {
  const uint32_t x = block_exp(top);
  const float up = block_up(x);
  if constexpr (VEC == 1) {
    if (ok) *q = x == 255u ? (int8_t)0 : (int8_t)(quant_bits<true>(v[0], up) & 0xffu);
  } else {
    uint2 w;
    // rare: a block that holds 1.9921875 2^E (127.5 steps) or more, or what is not finite
    if (__any_sync(0xffffffffu, (top & 0x7fffffu) >= 0x7f0000u || x == 255u)) {
      w = quant8<true>(v, up);
      if (x == 255u) w = make_uint2(0u, 0u);
    } else {
      w = quant8<false>(v, up);
    }
    if (ok) *reinterpret_cast<uint2*>(q) = w;
  }
  if (ok && (threadIdx.x & (32 / VEC - 1)) == 0) *e = (uint8_t)x;
}
template <int VEC>
__device__ __forceinline__ void store_ckpt8(const float (&v)[VEC], bool ok, int8_t* q, uint8_t* e) {
  store_ckpt8_top<VEC>(v, block_top<VEC>(v), ok, q, e);
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
    const f2_t step2 = f2_pack(step, step), off = f2_pack(-8388736.0f, -8388736.0f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {  // 2^23 + (q + 128) as a float, minus 2^23 + 128: exactly q
      const uint32_t a = __byte_perm(w[i >> 2], 0x4b000000u, 0x7650u + (i & 3));
      const uint32_t b = __byte_perm(w[i >> 2], 0x4b000000u, 0x7651u + (i & 3));
      f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(a), __uint_as_float(b)), off), step2), v[i],
                v[i + 1]);
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
  int slots;  // rows in shared memory at a time (1 .. 3)
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

// Two such sums at once, in place.
__device__ __forceinline__ void row_sum2(float& v, float& u, int tpr, float (*part)[32],
                                         float (*part2)[32], int half) {
  if (tpr <= 32) {
    for (int off = tpr >> 1; off > 0; off >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, off);
      u += __shfl_xor_sync(0xffffffffu, u, off);
    }
    return;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, off);
    u += __shfl_xor_sync(0xffffffffu, u, off);
  }
  if ((threadIdx.x & 31) == 0) {
    part[half][threadIdx.x >> 5] = v;
    part2[half][threadIdx.x >> 5] = u;
  }
  __syncthreads();
  v = u = 0.0f;
  for (int w = 0; w < tpr >> 5; w++) v += part[half][w], u += part2[half][w];
}

// ---- rows ahead ---------------------------------------------------------------------------------
// In the backwards and the layer norm's forward a thread's own chunks of the rows to come are copied
// to shared memory while it works on the current one (cp.async, 8 columns at a time, RowPlan::slots
// rows in all).  It alone reads what it copied, so no barrier is needed, and it may read a row twice,
// before and after the row's sum, instead of holding it in registers.  With one slot (ring_slots) nothing is ahead: a row is copied as
// a whole and waited for.  Single columns (VEC = 1) are loaded one row ahead into registers instead, up
// to 8 per thread (20000 x 1001 fp32, add_norm: forward 59 us, backward 123; read where they are used
// 77 and 233); wider rows (and VEC = 8 without RING) are read where they are used (2000 x 12345 bf16
// forward, 32 columns per thread held ahead: add_norm 491 us, gated_norm 412; not: 232 and 185).

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same through L1, for a thread's two halves of a 32-byte sector: the second finds it there.
__device__ __forceinline__ void cp_async16_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most the newest n (0 .. 2) groups are pending.
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// One operand, a tensor t or (q given) its checkpoint, and a thread's NJ chunks of its rows.  Without KEPT
// there is no checkpoint, and nothing asks for one: for single columns that is a third of the instructions.
template <typename IO, int VEC, int NJ, bool RING, bool KEPT = true> struct Operand {
  static constexpr int kUnits = RING ? (int)sizeof(IO) / 2 : 0;  // 16 bytes per chunk and row
  const void* t;
  const int8_t* q;
  const uint8_t* e;
  int ld;
  uint32_t at;  // this thread's place in the first slot of the ring
  static constexpr bool kAhead = VEC == 1 && NJ <= 8;
  // single columns of this row and the next, as loaded: nothing waits for the next row's
  uint32_t cur[kAhead ? NJ : 1], next[kAhead ? NJ : 1];

  __device__ __forceinline__ bool kept() const { return KEPT && q; }
  __device__ __forceinline__ bool given() const { return t || kept(); }
  // Bytes that a block's threads need per slot of the ring.
  static __host__ __device__ constexpr uint32_t slot_bytes(int threads) {
    return 16u * kUnits * NJ * threads;
  }
  // The row that was asked for last becomes the current one.
  __device__ __forceinline__ void advance() {
    if constexpr (kAhead)
#pragma unroll
      for (int j = 0; j < NJ; j++) cur[j] = next[j];
  }
  // Starts the copies of a row; col: the thread's chunks, `s` the byte offset of the ring slot.
  __device__ __forceinline__ void issue(uint32_t s, int row, const int (&col)[NJ],
                                        const bool (&okc)[NJ], int cols) {
    if constexpr (kAhead) {
      const int8_t* pq = q + (long long)row * cols;
      const IO* pt = (const IO*)t + (long long)row * ld;
#pragma unroll
      for (int j = 0; j < NJ; j++) {
        next[j] = 0u;
        if (!okc[j] || !given()) continue;
        if (kept()) next[j] = (uint32_t)(int)pq[col[j]];
        else if constexpr (sizeof(IO) == 2) next[j] = reinterpret_cast<const uint16_t*>(pt)[col[j]];
        else next[j] = reinterpret_cast<const uint32_t*>(pt)[col[j]];
      }
    }
    if constexpr (RING) {
      const uint32_t unit = 16 * blockDim.x;
      if (kept()) {
        const int8_t* p = q + (long long)row * cols;
#pragma unroll
        for (int j = 0; j < NJ; j++)
          if (okc[j]) cp_async8(at + s + j * kUnits * unit, p + col[j]);
      } else if (t) {
        const IO* p = (const IO*)t + (long long)row * ld;
#pragma unroll
        for (int j = 0; j < NJ; j++)
          if (okc[j])
#pragma unroll
            for (int u = 0; u < kUnits; u++) {
              const uint32_t dst = at + s + (j * kUnits + u) * unit;
              const char* src = (const char*)(p + col[j]) + 16 * u;
              if constexpr (kUnits == 1) cp_async16(dst, src);
              else cp_async16_l1(dst, src);
            }
      }
    }
  }
  // Zeros in the slot at s: for the chunks that the thread does not have, which are never copied to
  // (so once is enough), or for all of them, where there is no row to copy.
  __device__ __forceinline__ void clear(uint32_t s, const bool (&okc)[NJ], bool all) {
    if constexpr (kAhead)
#pragma unroll
      for (int j = 0; j < NJ; j++) next[j] = 0u;
    if constexpr (RING) {
#pragma unroll
      for (int j = 0; j < NJ; j++)
        if (all || !okc[j] || !given())
#pragma unroll
          for (int u = 0; u < kUnits; u++)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             at + s + (j * kUnits + u) * 16 * blockDim.x),
                         "r"(0u)
                         : "memory");
    }
  }
  // The scale byte of a chunk (a checkpoint's; 7 otherwise).
  __device__ __forceinline__ uint32_t scale(bool ok, int row, int col, int nb) const {
    return kept() && ok ? e[(long long)row * nb + (int)((unsigned)col / 32)] : 7u;
  }
  // The largest magnitude's bits of the block that a tensor's chunk lies in; v holds its values.
  __device__ __forceinline__ uint32_t top(uint32_t s, int j, const float (&v)[VEC]) const {
    if constexpr (RING && sizeof(IO) == 2)
      return block_top(ld_shared16(at + s + j * kUnits * 16 * blockDim.x));
    else
      return block_top<VEC>(v);
  }
  // A chunk's values (x is its scale byte); zeros for a chunk that the thread does not have.
  __device__ __forceinline__ void get(uint32_t s, int j, bool ok, int row, int col, int cols,
                                      uint32_t x, float (&v)[VEC]) const {
    if constexpr (kAhead) {
      v[0] = kept() ? (float)(int)cur[j] * block_step(x) :
             __uint_as_float(sizeof(IO) == 2 ? cur[j] << 16 : cur[j]);
    } else if constexpr (VEC == 1) {
      Cols<IO, 1> c;
      c.zero();
      if (ok && t) c.load((const IO*)t + (long long)row * ld + col);
      c.get(v);
      if (ok && kept()) v[0] = (float)q[(long long)row * cols + col] * block_step(x);
    } else if constexpr (!RING) {
      if (!ok || !given()) {
#pragma unroll
        for (int i = 0; i < VEC; i++) v[i] = 0.0f;
      } else if (kept()) {
        Kept<8> k;
        k.q = *reinterpret_cast<const uint2*>(q + (long long)row * cols + col);
        k.e = (uint8_t)x;
        k.get(v);
      } else {
        Cols<IO, 8> c;
        c.load((const IO*)t + (long long)row * ld + col);
        c.get(v);
      }
    } else {
      const uint32_t unit = 16 * blockDim.x, a = at + s + j * kUnits * unit;
      const uint4 w = ld_shared16(a);
      if (kept()) {
        Kept<8> k;
        k.q = make_uint2(w.x, w.y);
        k.e = (uint8_t)x;
        k.get(v);
      } else if constexpr (sizeof(IO) == 2) {
        Cols<IO, 8> c;
        c.a = w;
        c.get(v);
      } else {
        const uint4 w2 = ld_shared16(a + unit);
        v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
        v[4] = __uint_as_float(w2.x), v[5] = __uint_as_float(w2.y);
        v[6] = __uint_as_float(w2.z), v[7] = __uint_as_float(w2.w);
      }
    }
  }
};

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

inline RowPlan row_plan(long long rows, int group, int groups, int tpr, int block, int per_sm_threads,
                        int sms) {
  RowPlan p{};
  p.tpr = tpr;
  p.group = group;
  p.groups = groups;
  p.gpb = p.rpb = p.slots = 1;
  if (tpr <= 32) {
    const int teams = block / tpr > 0 ? block / tpr : 1;
    p.gpb = groups < teams ? groups : teams;
    p.rpb = teams / p.gpb;
    if (p.rpb > rows) p.rpb = (int)rows;
  }
  p.threads = round_up32(p.tpr * p.gpb * p.rpb);
  p.nby = (groups + p.gpb - 1) / p.gpb;
  const long long need = (rows + p.rpb - 1) / p.rpb;
  // one round of blocks, each stepping over the rows
  const int per_sm = p.threads >= per_sm_threads ? 1 : per_sm_threads / p.threads;
  const long long most = ((long long)sms * per_sm + p.nby - 1) / p.nby;
  p.nbx = (int)(need < most ? need : most);
  if (p.nbx < 1) p.nbx = 1;
  return p;
}

// Rows in shared memory: as many, up to 3, as leave room for per_sm_threads threads on an SM.  One for
// fp32 rows of more than one chunk per thread in add_norm's backward (its four operands take 128 KB
// per row on an SM, those that a call does not have included) and of four in the gated forward; two
// or three else.
constexpr int kRingBytesPerSm = 208 * 1024;
constexpr int kRingBytesMost = 224 * 1024;  // of one block
inline int ring_slots(uint32_t slot_bytes, int threads, int per_sm_threads) {
  if (!slot_bytes) return 1;
  const int blocks = threads >= per_sm_threads ? 1 : per_sm_threads / threads;
  const int n = (int)(kRingBytesPerSm / ((long long)slot_bytes * blocks));
  return n < 1 ? 1 : (n > 3 ? 3 : n);
}
// Launches Kernel with `smem` bytes of dynamic shared memory.  More than 48 KB in all has to be asked
// for, once per kernel and device (the first 64 devices remember it).
template <auto Kernel, typename A>
inline cudaError_t launch_rows(const A& a, const RowPlan& p, size_t smem, cudaStream_t st) {
  if (smem > 40 * 1024) {  // with the static part, 48 KB at most without asking
    static std::atomic<unsigned long long> asked{0};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(asked.load(std::memory_order_relaxed) & bit)) {
      if (cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRingBytesMost))
        return e;
      asked.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  Kernel<<<dim3(p.nbx, p.nby), p.threads, smem, st>>>(a, p);
  return cudaGetLastError();
}

}  // namespace ssm
