// wgrad8_tc.cu -- d_W[i][j] (+)= sum_t g[t][i] X[t][j] on the tensor cores, with X read from its
// 8-bit checkpoint and g in bf16, or in fp32 as three bf16 terms (wgrad8.cu splits it).
//
// Both operands run along the tokens in memory's slow direction, so both are staged as they lie,
// [tokens][columns] with the columns contiguous (the MMA's MN-major form, 128-byte swizzle): no
// transposition anywhere.  A kept value q 2^(E-6) is exact in bf16, so the products are exact in
// fp32 and the result differs from an fp32 one by the order and rounding of its additions only.
//
// The sum runs over stages of 64 tokens; with three terms, over the tokens three times, g's terms one
// after the other and X again each time (its conversion costs nothing beside the MMAs).
//
// One or two CTAs (CG) form a 128 CG x 256 tile of d_W over a range of tokens, 64 tokens per stage.
// With two, each holds its 128 rows' g and half of X's columns, and the MMAs (cta_group::2, issued
// by the first CTA) read both halves: per MMA a CTA then converts and stores half as much X, and
// shared-memory traffic, which bounds one CTA, falls from 128 to 80 KB per stage.
//   warp 0       one thread copies q's tiles by TMA (past the ends they read as 0)
//   warp 1       one thread of the first CTA issues the MMAs (K 16; accumulators in tensor memory);
//                the second CTA's warp passes on that its g has landed
//   warp 3       one thread copies g's tiles by TMA
//   warps 4-11   empty the accumulators, and read the scales (whose rows are too short for TMA) a
//                segment of 1024 tokens ahead
//   warps 12-23  turn q into bf16, 16 columns at a time, and store it swizzled: three groups of four
//                warps take every third stage each, since a stage's conversion is a chain of
//                latencies (waits, loads, about 45 instructions per 16 columns, stores, a proxy
//                fence) longer than two stages' MMAs.  One group at a time with the accumulators in
//                the same warps took 108 us on 16384 x 4096 x 1024, two groups 108, three 87.
// q has a ring of its own beside that of g and the converted X: with one ring for both, the chain
// copy (1300 cycles) - conversion (950) - MMAs (560) of a slot bounds the rate.  The warps of one
// thread's work run as long as a stage's instructions take one after the other, so each waits for
// as few barriers as can be: a stage's `full` (the first CTA's) collects the bytes of its g, the
// word that the second CTA's has landed, and every converting warp's part; the MMAs' commit
// completes `empty`.
//
// The tensor cores truncate as they accumulate: over 16384 tokens that alone costs 1e-5 of the
// result.  The accumulator is therefore emptied every 1024 tokens (two of them alternate, so that
// the MMAs go on) into fp32 registers, added with rounding to nearest: 4e-7, less than a plain fp32
// product's 7e-7.  At the end they go to d_W or, where the tokens are split over blocks, to the
// workspace; wgrad8.cu then adds the splits in order.
//
// Measured (GB300): g 16384 x 4096, X 16384 x 1024: 88 us, 1565 TFLOP/s (82 % of the measured bf16
// peak on 128 of 152 SMs); MMAs alone 78 us.  g 32768 x 768, X 32768 x 1536: 52 us.
#include "block.cuh"
#include "pair.cuh"
#include "rows.cuh"

namespace ssm {

namespace {

constexpr int kTM = 128, kTN = 256, kTT = 64;  // rows per CTA, columns per tile, tokens per stage
constexpr int kGroupWarps = 4, kGroups = 3;  // warps that convert a stage, and stages at once
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (4 + kSumWarps + kGroups * kGroupWarps);
// Registers per thread: the first four warps', the adding ones' (which hold a 128 x 256 accumulator
// between them) and the converting ones': 128 x 32 + 256 x 152 + 384 x 48 = 768 x 80, what the block
// is launched with.
constexpr int kRegsFew = 32, kRegsSum = 152, kRegsConv = 48;
constexpr uint32_t kSlab = kTT * 128;  // 64 columns of bf16 x 64 tokens
constexpr uint32_t kBytesA = kTM / 64 * kSlab;
constexpr int kSegment = 16;  // stages between two emptyings of the accumulator
constexpr int kSegTokens = kSegment * kTT;
constexpr uint32_t kTmCols = 2 * kTN;

template <int CG> struct Lay {  // shared memory of a CTA
  static constexpr int NB = kTN / CG;  // X's columns here
  static constexpr int stages = CG == 1 ? 3 : 5;  // slots of both rings
  static constexpr uint32_t bytes_b = NB / 64 * kSlab, bytes_q = NB * kTT;  // of a stage
  static constexpr uint32_t stage = kBytesA + bytes_b, at_q = stages * stage;
  static constexpr int blocks = NB / 32;                                // scales of a row here
  static constexpr uint32_t scales = (uint32_t)kSegTokens * blocks * 2;  // of a segment, as bf16
  static constexpr uint32_t at_scales = at_q + stages * bytes_q;
  static constexpr uint32_t smem = at_scales + 2 * scales + 1024;
};

struct TcArgs {
  CUtensorMap g, q;
  const uint8_t* e;
  float* out;  // d_W, or the splits' partial tiles
  long long tokens;
  int stages, per_term, per_split;  // in all, of one term of g, of one split
  int m, k, nb, accumulate, vec_out, q_copied, no_wait;
  int* status;
};

// Matrix descriptor of a tile of 64-column slabs [64 tokens][128 bytes], MN-major, 128-byte swizzle:
// leading offset = next 64 columns, stride offset = next 8 tokens.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kSlab >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// The int8 values in bytes 0 and 2 of w as bf16, times the scale.  Below 0x43, the low 7 bits of a
// byte read as the bf16 number 128 + low, and its sign bit alone as 128 or 256; the difference of
// the two is the two's complement value, exactly.
__device__ __forceinline__ uint32_t two_bf16(uint32_t w, __nv_bfloat162 scale) {
  const uint32_t t = (w & 0x007f007fu) | 0x43004300u, c = (w & 0x00800080u) | 0x43004300u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                             *reinterpret_cast<const __nv_bfloat162*>(&c));
  r = __hmul2(r, scale);
  return *reinterpret_cast<uint32_t*>(&r);
}
// The steps 2^(e - 133) of the scale bytes in bits 0 .. 7 and 16 .. 23 as bf16, which holds each of
// them: as 2^(e - 127) (a subnormal number for e = 0, infinite for 255) times 2^-6, plus f - f for a NaN.
__device__ __forceinline__ uint32_t two_steps(uint32_t e2) {
  uint32_t f;
  asm("max.u16x2 %0, %1, %2;" : "=r"(f) : "r"(e2 << 7), "r"(0x00400040u));
  const uint32_t small = 0x3c803c80u;
  const __nv_bfloat162 f2 = *reinterpret_cast<const __nv_bfloat162*>(&f);
  const __nv_bfloat162 r =
      __hfma2(f2, *reinterpret_cast<const __nv_bfloat162*>(&small), __hsub2(f2, f2));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Four columns of a word leave in the order 0, 2, 1, 3 (taking every other byte saves moving them):
// place j of the tile holds column column_of(j), undone where the accumulator is stored.
__device__ __forceinline__ constexpr int column_of(int j) {
  return (j & ~3) | ((j & 1) << 1) | ((j & 2) >> 1);
}

// A converting thread (warp cw of its group): 16 columns of every kRowsOnce-th row.  8 lanes cover
// the 128 bytes of a row between two rows, 64 bytes of each: so both their loads and their stores
// (in the swizzle, neighbouring rows' even 16-byte chunks fall on different banks) hit every bank
// once.
template <int CG> struct Converter {
  using L = Lay<CG>;
  static constexpr int kRowsOnce = kGroupWarps * 32 / (L::NB / 16);  // rows of the group at once
  static_assert(kRowsOnce % 8 == 0, "the swizzle of a thread's rows");
  uint32_t q, b0, b1, scales;  // shared-memory addresses of this thread's part of the first slot

  __device__ __forceinline__ Converter(uint32_t smem, int cw, int lane) {
    const int part = CG == 1 ? (cw & 1) : 0;  // which 128 columns
    const int c = lane & 7, pair = lane >> 3;
    const int row0 = 4 * (CG == 1 ? cw >> 1 : cw) + 2 * (pair >> 1) + ((pair & 1) ^ (c >> 2));
    const uint32_t x = row0 & 7;  // also that of the thread's other rows: multiples of 8 apart
    const uint32_t b = smem + kBytesA + (2 * part + (c >> 2)) * kSlab + row0 * 128;
    b0 = b + (((2 * (c & 3)) ^ x) << 4);
    b1 = b + (((2 * (c & 3) + 1) ^ x) << 4);
    q = smem + L::at_q + row0 * L::NB + part * 128 + c * 16;
    scales = smem + L::at_scales + 2 * (row0 * L::blocks + part * 4 + (c >> 1));
  }
  // The stage in ring slot `slot` (a byte offset sb of g and X, sq of q), its scales sc bytes on.
  __device__ __forceinline__ void run(uint32_t sb, uint32_t sq, uint32_t sc) const {
    constexpr int kBatch = 4;  // rows whose loads are in flight together, before the stores
#pragma unroll
    for (int r0 = 0; r0 < kTT; r0 += kBatch * kRowsOnce) {
      uint4 u[kBatch];
      uint32_t e[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        e[i] = lds16(scales + sc + 2 * (r0 + i * kRowsOnce) * L::blocks);
        u[i] = lds128(q + sq + (r0 + i * kRowsOnce) * L::NB);
      }
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        const uint32_t at = sb + (r0 + i * kRowsOnce) * 128;
        const uint32_t s = __byte_perm(e[i], 0u, 0x1010u);
        const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&s);
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          v[2 * j] = two_bf16(w[j], scale);
          v[2 * j + 1] = two_bf16(w[j] >> 8, scale);
        }
        sts128(b0 + at, v[0], v[1], v[2], v[3]);
        sts128(b1 + at, v[4], v[5], v[6], v[7]);
      }
    }
  }
};

template <int CG>
__global__ void __launch_bounds__(kThreads, 1) wgrad8_tc_kernel(const __grid_constant__ TcArgs a) {
  using L = Lay<CG>;
  constexpr int S = L::stages;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[S], empty[S], g_here[S], q_here[S], q_empty[S];
  __shared__ uint64_t seg_done[2], drained[2], scaled[2];
  __shared__ uint32_t tbase;
  __shared__ int bad;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* scales = smem + L::at_scales;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to the compiler as uniform
  const int rank = CG == 1 ? 0 : (blockIdx.x & 1);
  const int m0 = (blockIdx.y * CG + rank) * kTM, n0 = (blockIdx.x / CG) * kTN;
  const int nq = n0 + rank * L::NB;  // first column of X staged here
  const int s_begin = blockIdx.z * a.per_split;  // its stages: s_begin ... s_begin + iters - 1
  const int iters = a.stages - s_begin < a.per_split ? a.stages - s_begin : a.per_split;
  const int segs = (iters + kSegment - 1) / kSegment;
  if (tid == 0) {
    for (int i = 0; i < S; i++) {
      mbar_init(&full[i], CG + CG * kGroupWarps);
      mbar_init(&empty[i], 1);
      mbar_init(&g_here[i], 1);
      mbar_init(&q_here[i], 1);
      mbar_init(&q_empty[i], kGroupWarps);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&seg_done[b], 1);
      mbar_init(&drained[b], CG * kSumWarps);
      mbar_init(&scaled[b], kSumWarps);
    }
    bad = 0;
    fence_barrier_init();
    prefetch_tmap(&a.g);
    prefetch_tmap(&a.q);
  }
  __syncwarp();
  if (warp == 1) Mma<CG>::alloc(&tbase, kTmCols);
  tmem_fence_before_sync();
  __syncthreads();
  sync_tile<CG>();
  tmem_fence_after_sync();
  const uint32_t tm = tbase;
  asm volatile("griddepcontrol.launch_dependents;");  // the kernel that adds the splits, if any

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      if (a.q_copied) wait_for_copies();
      Ring<S> r;
      int it = 0, st = s_begin % a.per_term;
      for (; it < iters; it++, st = st + 1 == a.per_term ? 0 : st + 1, r.next()) {
        if (it >= S && !mbar_wait(&q_empty[r.s], r.phase ^ 1)) {
          atomicExch(&bad, 1);
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(&q_here[r.s], L::bytes_q);
          tma_load_3d(smem + L::at_q + r.s * L::bytes_q, &a.q, nq, st * kTT, 0, &q_here[r.s]);
        }
        __syncwarp();
      }
      // the copies in flight land before the block may end
      for (int j = it > S ? it - S : 0; j < it; j++)
        if (!mbar_wait(&q_here[j % S], (j / S) & 1)) break;
    } else if (warp == 3) {
      uint64_t* here = rank == 0 ? full : g_here;
      wait_for_copies();
      Ring<S> r;
      int it = 0, term = s_begin / a.per_term, st = s_begin - term * a.per_term;
      for (; it < iters; it++, r.next()) {
        if (it >= S && !mbar_wait(&empty[r.s], r.phase ^ 1)) {
          atomicExch(&bad, 1);
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(&here[r.s], kBytesA);
#pragma unroll
          for (int c = 0; c < kTM / 64; c++)
            tma_load_3d(smem + r.s * L::stage + c * kSlab, &a.g, m0 + 64 * c, st * kTT, term,
                        &here[r.s]);
        }
        __syncwarp();
        if (++st == a.per_term) st = 0, term++;
      }
      for (int j = it > S ? it - S : 0; j < it; j++)
        if (!mbar_wait(&here[j % S], (j / S) & 1)) break;
    } else if (warp == 1 && rank == 0) {
      // Only the address in a descriptor's low word changes: 16 tokens on, 2048 bytes (>> 4: 128).
      Ring<S> r;
      const uint64_t desc0 = desc_mn(smem_u32(smem));
      constexpr uint32_t idesc = idesc_bf16(kTM * CG, kTN, true, true);
      int it = 0;
      for (int seg = 0; seg < segs; seg++) {
        const uint32_t d = tm + (seg & 1) * kTN;
        const int end = it + kSegment < iters ? it + kSegment : iters;
        bool ok = true;
        if (seg >= 2)  // this accumulator's previous segment has been taken out
          ok = mbar_wait(&drained[seg & 1], ((seg >> 1) - 1) & 1);
        bool first = true;
        for (; it < end && ok; it++, r.next(), first = false) {
          ok = mbar_wait(&full[r.s], r.phase);
          tmem_fence_after_sync();
          if (ok && elect_one()) {
            const uint64_t da = desc0 + (uint32_t)(r.s * (L::stage >> 4)), db = da + (kBytesA >> 4);
            Mma<CG>::mma(idesc, d, da, db, !first);
#pragma unroll
            for (int kk = 1; kk < kTT / 16; kk++)
              Mma<CG>::mma(idesc, d, da + 128 * kk, db + 128 * kk, true);
            Mma<CG>::commit(&empty[r.s]);
          }
          __syncwarp();
        }
        if (!ok) {
          atomicExch(&bad, 1);
          break;
        }
        if (elect_one()) Mma<CG>::commit(&seg_done[seg & 1]);
        __syncwarp();
      }
    } else if (warp == 1) {
      Ring<S> r;
      const uint32_t first_full = bar_of_first<CG>(full);
      for (int it = 0; it < iters; it++, r.next()) {
        if (!mbar_wait(&g_here[r.s], r.phase)) {
          atomicExch(&bad, 1);
          break;
        }
        if (elect_one()) mbar_arrive_first<CG>(first_full + 8 * r.s);
        __syncwarp();
      }
    }
  } else if (warp >= 4 + kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    const int cw = warp & 3, group = (warp - 4 - kSumWarps) >> 2;
    const uint32_t first_full = bar_of_first<CG>(full);
    const Converter<CG> conv(smem_u32(smem), cw, lane);
    uint32_t slot = group, phase = 0;
    if (slot >= S) slot -= S, phase ^= 1;
    bool ok = true;
    int seg = -1;
    for (int it = group; it < iters && ok; it += kGroups) {
      if (it / kSegment != seg) {
        seg = it / kSegment;
        ok = mbar_wait(&scaled[seg & 1], (seg >> 1) & 1);
      }
      if (it >= S) ok = ok && mbar_wait(&empty[slot], phase ^ 1);
      ok = ok && mbar_wait(&q_here[slot], phase);
      if (ok) {
        conv.run(slot * L::stage, slot * L::bytes_q,
                 (it % (2 * kSegment)) * (2 * kTT * L::blocks));
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_first<CG>(first_full + 8 * slot);
          mbar_arrive(&q_empty[slot]);
        }
      }
      slot += kGroups;
      if (slot >= S) slot -= S, phase ^= 1;
    }
    if (!ok) atomicExch(&bad, 1);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSum));
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tacc = tm + ((uint32_t)(32 * quad) << 16) + 128 * half;
    const uint32_t first_drained = bar_of_first<CG>(drained);
    float acc[128];  // row 32 quad + lane of this CTA's tile, columns 128 half ...
#pragma unroll
    for (int j = 0; j < 128; j++) acc[j] = 0.0f;
    // A word is the scale bytes of 128 columns of a row; 255 marks NaN, 7 fills what is not there.
    // The steps are stored as bf16.
    constexpr int W = L::blocks / 4, kBatch = kSegTokens * W / (32 * kSumWarps);
    const int blk0 = nq / 32;
    const bool words = a.nb % 4 == 0 && (uintptr_t)a.e % 4 == 0;
    auto load_scales = [&](int seg) {
      uint2* dst = reinterpret_cast<uint2*>(scales + (seg & 1) * L::scales);
      uint32_t v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; b++) {
        const int i = (tid - 128) + 32 * kSumWarps * b, blk = blk0 + 4 * (i % W);
        const int st = (s_begin + seg * kSegment + i / W / kTT) % a.per_term;
        const long long t = (long long)st * kTT + i / W % kTT;
        v[b] = 0x07070707u;
        if (t < a.tokens && blk < a.nb) {
          const uint8_t* p = a.e + t * a.nb + blk;
          if (words) {
            v[b] = *reinterpret_cast<const uint32_t*>(p);
          } else {
#pragma unroll
            for (int u = 0; u < 4; u++)
              if (blk + u < a.nb) v[b] = (v[b] & ~(0xffu << (8 * u))) | ((uint32_t)p[u] << (8 * u));
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; b++)
        dst[(tid - 128) + 32 * kSumWarps * b] =
            make_uint2(two_steps(__byte_perm(v[b], 0u, 0x4140)),
                       two_steps(__byte_perm(v[b], 0u, 0x4342)));
      __syncwarp();
      if (lane == 0) mbar_arrive(&scaled[seg & 1]);
    };
    load_scales(0);
    if (segs > 1) load_scales(1);
    bool ok = true;
    for (int seg = 0; seg < segs && ok; seg++) {
      ok = !a.no_wait && mbar_wait(&seg_done[seg & 1], (seg >> 1) & 1);
      __syncwarp();
      tmem_fence_after_sync();
      const uint32_t t = tacc + (seg & 1) * kTN;
#pragma unroll
      for (int c = 0; c < 32; c++) {
        float v[4];
        tmem_ld4(t + 4 * c, v);
#pragma unroll
        for (int j = 0; j < 4; j++) acc[4 * c + j] += v[j];
      }
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_first<CG>(first_drained + 8 * (seg & 1));
      if (ok && seg + 2 < segs) load_scales(seg + 2);  // this segment's half of the area is free
    }
    if (!ok) atomicExch(&bad, 1);
    const int i = m0 + 32 * quad + lane;
    float* dst = a.out + ((long long)blockIdx.z * a.m + i) * a.k;
    if (!ok && i < a.m) {  // what is missing reads as NaN, also where nobody looks at the status
#pragma unroll 1
      for (int j = n0 + 128 * half; j < n0 + 128 * (half + 1) && j < a.k; j++)
        dst[j] = __uint_as_float(0x7fc00000u);
    } else if (i < a.m) {
#pragma unroll
      for (int b = 0; b < 128; b += 8) {
        const int j = n0 + 128 * half + b;
        if (a.vec_out) {  // rows are multiples of 8 columns, 32-byte aligned
          if (j < a.k) {
            float o[8];
#pragma unroll
            for (int u = 0; u < 8; u++) o[column_of(u)] = acc[b + u];
            if (a.accumulate) {
              Cols<float, 8> was;
              was.load(dst + j);
#pragma unroll
              for (int u = 0; u < 8; u++) o[u] += was.a[u];
            }
            st_cols(dst + j, o);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 8; u++)
          {
            const int at = j + column_of(u);
            if (at < a.k) dst[at] = a.accumulate ? dst[at] + acc[b + u] : acc[b + u];
          }
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1 && rank == 0 && bad) {
    // Some wait has given up, perhaps with MMAs in flight: they read the shared memory and write the
    // tensor memory of both CTAs, so they complete first.  g_here is the second CTA's; free here.
    if (elect_one()) Mma<CG>::commit_here(&g_here[0]);
    __syncwarp();
    mbar_wait(&g_here[0], 0);
  }
  sync_tile<CG>();  // the other CTA may still arrive on barriers here
  if (warp == 1) {
    tmem_fence_after_sync();
    Mma<CG>::dealloc(tm, kTmCols);
  }
  if (tid == 0) {
    wait_for_copies();  // the kernel before clears the status; this one does not end ahead of it
    if (bad) record_status(a.status, SSM_ERR_TIMEOUT);
  }
}

// A tile of two CTAs where a row tile of one would be full.
int ctas_of(int m) { return m > kTM ? 2 : 1; }

template <int CG> cudaError_t launch(const TcArgs& t, int splits, cudaStream_t st) {
  auto kernel = wgrad8_tc_kernel<CG>;
  // asked for once per device (the first 64 remember it)
  static std::atomic<unsigned long long> asked{0};
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Lay<CG>::smem))
      return e;
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((t.k + kTN - 1) / kTN * CG, (t.m + kTM * CG - 1) / (kTM * CG), splits);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = Lay<CG>::smem;
  c.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = CG > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, t);
  count_launches(1);
  return e;
}

int per_split_of(int stages, int splits) { return (stages + splits - 1) / splits; }

}  // namespace

// Splits of the stages: as many as fill the SMs once, at least 4 stages each.
int wgrad_tc_splits(long long tokens, int terms, int m, int k, int sms) {
  const int cg = ctas_of(m);
  const long long tiles = (long long)((m + cg * kTM - 1) / (cg * kTM)) * ((k + kTN - 1) / kTN);
  const int stages = terms * (int)((tokens + kTT - 1) / kTT);
  long long s = sms / cg / tiles;
  const int most = (stages + 3) / 4;
  if (s > most) s = most;
  if (s < 1) s = 1;
  const int per = per_split_of(stages, (int)s);
  return (stages + per - 1) / per;  // none of them empty
}

// To be called right after a kernel of the same call that clears `status` and lets this one start
// early.  g: [terms][tokens] rows of ld_g elements, q: rows of ld_q bytes; both 16-byte aligned.
cudaError_t launch_wgrad_tc(const void* g, long long ld_g, int terms, const int8_t* q,
                            long long ld_q, const Wgrad& a, float* part, int splits, int* status,
                            cudaStream_t st) {
  const int cg = ctas_of(a.m);
  TcArgs t{};
  if (!encode_tmap_3d(&t.g, g, 2, a.m, a.tokens, terms, ld_g,
                      terms > 1 ? ld_g * a.tokens : ld_g, 64, kTT, 1, 128) ||
      !encode_tmap_3d(&t.q, q, 1, a.k, a.tokens, 1, ld_q, ld_q, kTN / cg, kTT, 1))
    return cudaErrorInvalidValue;
  t.e = a.e;
  t.out = part ? part : a.d_W;
  t.tokens = a.tokens;
  t.per_term = (int)((a.tokens + kTT - 1) / kTT);
  t.stages = terms * t.per_term;
  t.per_split = per_split_of(t.stages, splits);
  t.m = a.m;
  t.k = a.k;
  t.nb = (a.k + 31) / 32;
  t.accumulate = part ? 0 : a.accumulate;
  t.q_copied = q != a.q;
  t.no_wait = a.no_wait;
  t.vec_out = a.k % 8 == 0 && (uintptr_t)t.out % 32 == 0;
  t.status = status;
  return cg == 1 ? launch<1>(t, splits, st) : launch<2>(t, splits, st);
}

}  // namespace ssm
