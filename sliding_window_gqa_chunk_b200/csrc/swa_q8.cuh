// swa_q8.cuh - device pieces shared by the kernels of the 8-bit rolling cache:
// the two 8-bit formats and the rounding of one block of rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "swa_common.cuh"
#include "swa_internal.h"

namespace swa {
namespace q8 {

// Exponents of a block's scale: 2^-100 keeps every product and quotient with
// a scale or its inverse a normal fp32 number.
constexpr int kMinScaleExp = -100;

// Exponent e of the scale 2^e of a block whose largest magnitude has the bf16
// bits `amax` (sign cleared): the smallest e with amax <= top * 2^e.  With
// amax = (1 + m / 128) 2^E and top = (1 + M / 128) 2^T that is E - T, or one
// more if m > M: no rounding, no division.  0 for amax = 0.
template <int FMT>
__device__ __forceinline__ int scale_exp(uint32_t amax) {
  constexpr int T = FMT == SWA_Q8_E4M3 ? 8 : 6;       // 448 = 1.75 * 2^8, 127 = (127 / 64) * 2^6
  constexpr int M = FMT == SWA_Q8_E4M3 ? 96 : 126;
  if (amax == 0) return 0;
  const int E = (int)(amax >> 7) - 127;
  const int e = E - T + ((int)(amax & 127) > M ? 1 : 0);
  return e < kMinScaleExp ? kMinScaleExp : e;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four scaled values -> four 8-bit numbers, round to nearest even.  The scale
// brings every value into range, so nothing saturates (but infinities).
template <int FMT>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  if constexpr (FMT == SWA_Q8_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  } else {
    const uint32_t x = (uint32_t)__float2int_rn(a) & 255u, y = (uint32_t)__float2int_rn(b) & 255u;
    const uint32_t z = (uint32_t)__float2int_rn(c) & 255u, w = (uint32_t)__float2int_rn(d) & 255u;
    return x | (y << 8) | (z << 16) | (w << 24);
  }
}

// Bytes 0, 1 and 2, 3 of `w` as two f16 pairs; every 8-bit number of either
// format is exact in f16.  e4m3 is converted by instruction; a whole number x
// is made from the f16 bits of 1024 + (x + 128) by subtracting 1152.
template <int FMT>
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == SWA_Q8_E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    w ^= 0x80808080u;
    const __half2 off = __float2half2_rn(1152.f);
    const uint32_t a = prmt(w, 0x64646464u, 0x4140), b = prmt(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Largest magnitude (bf16 bits without sign) of the 8 bf16 in `x`.  Bits of
// magnitudes compare like the magnitudes.
__device__ __forceinline__ uint32_t amax8(const uint4& x) {
  uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                        __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// 8 bf16 times `inv` -> 8 8-bit numbers.
template <int FMT>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv) {
  uint2 y;
  y.x = pack4<FMT>(bf16_lo(x.x) * inv, bf16_hi(x.x) * inv, bf16_lo(x.y) * inv, bf16_hi(x.y) * inv);
  y.y = pack4<FMT>(bf16_lo(x.z) * inv, bf16_hi(x.z) * inv, bf16_lo(x.w) * inv, bf16_hi(x.w) * inv);
  return y;
}

// Rounds one block of `size` rows of K and of V (all THREADS threads of the CTA, and
// only when all of them come here).  k_row(i) / v_row(i) give row i in bf16; `dst` the
// block's first row in the ring.  `red` is 2 words of shared memory.  The rows stay in
// registers between the search for the largest magnitude and the rounding.
template <int D, int FMT, int THREADS, typename KRow, typename VRow>
__device__ __forceinline__ void round_block(KRow k_row, VRow v_row, int size, uint8_t* k_dst, uint8_t* v_dst,
                                            float* k_scale, float* v_scale, uint32_t* red) {
  constexpr int kVecs = D / 8;
  constexpr int kPer = (kQ8Block * kVecs + THREADS - 1) / THREADS;
  if (threadIdx.x < 2) red[threadIdx.x] = 0;
  __syncthreads();
  uint4 k[kPer], v[kPer];
  uint32_t ka = 0, va = 0;
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int i = threadIdx.x + n * THREADS, r = i / kVecs, c = i % kVecs;
    k[n] = v[n] = make_uint4(0, 0, 0, 0);
    if (r < size) {
      k[n] = reinterpret_cast<const uint4*>(k_row(r))[c];
      v[n] = reinterpret_cast<const uint4*>(v_row(r))[c];
    }
  }
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    ka = max(ka, amax8(k[n]));
    va = max(va, amax8(v[n]));
  }
  ka = __reduce_max_sync(0xffffffffu, ka);
  va = __reduce_max_sync(0xffffffffu, va);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&red[0], ka);
    atomicMax(&red[1], va);
  }
  __syncthreads();
  const int ke = scale_exp<FMT>(red[0]), ve = scale_exp<FMT>(red[1]);
  const float ki = exp2_int(-ke), vi = exp2_int(-ve);
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int i = threadIdx.x + n * THREADS;
    if (i >= size * kVecs) continue;
    reinterpret_cast<uint2*>(k_dst)[i] = quantise8<FMT>(k[n], ki);
    reinterpret_cast<uint2*>(v_dst)[i] = quantise8<FMT>(v[n], vi);
  }
  if (threadIdx.x == 0) {
    *k_scale = exp2_int(ke);
    *v_scale = exp2_int(ve);
  }
}

}  // namespace q8
}  // namespace swa
