// Block-scaled formats: the scale of a block, the 4-bit conversions and the scale layout.
//
// A block is 32 (MXFP4, MXFP8) or 16 (NVFP4) neighbours along the packed axis.
//   MX:  scale = 2^(c - 127), the smallest power of two with amax / scale <= the largest code
//        value (6 or 448), so no value saturates; x / scale is exact in fp32, and the one
//        rounding is the code's.
//   NV:  sb = E4M3(fp32(fp32(amax * s) / 6)) with s the tensor's fp32 scale; the codes are those of
//        fp32(x * fp32(s / sb)).  A block whose sb rounds to zero holds zeros.
// A block that holds an infinity or a NaN gets a NaN scale (and zero codes), so that whatever
// reads it is NaN too instead of a plausible number.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace te {

// Bits of |v| order like the values, infinities above every finite number and NaN above those.
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kF32Max = 3.4028234663852886e38f;

// The byte of one scale within its row of tiles, for blocks counted within a CTA's own tiles: tiles
// of 128 rows x 4 blocks, 512 bytes, in which the rows r, r + 32, r + 64, r + 96 are neighbours.  This is the order in which
// tcgen05.cp.32x128b hands a tile to tensor memory.
__device__ __forceinline__ uint32_t scale_offset(uint32_t row_in_tile, uint32_t block) {
  return (block >> 2) * 512 + (row_in_tile & 31) * 16 + (row_in_tile >> 5) * 4 + (block & 3);
}

// The same of any block of a row of tiles: 4 bytes a column, so past 32 bits from 2^30 columns on.
__device__ __forceinline__ int64_t scale_offset_wide(uint32_t row_in_tile, int64_t block) {
  return (block >> 2) * 512 + scale_offset(row_in_tile, uint32_t(block) & 3);
}

// Two fp32 -> two E2M1 codes in a byte (lo in the low half): nearest even, saturating to +-6.
// Eight fp32 -> eight codes, element 0 lowest.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight E2M1 codes -> exact fp32 pairs (through the exact conversion to f16).
__device__ __forceinline__ void unpack_e2m1x8(uint32_t w, f32x2 (&v)[4]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
}

// 2^(c - 127) of an E8M0 byte; NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t c) {
  const uint32_t bits = c == 0 ? 0x00400000u : c == 255 ? 0x7fc00000u : c << 23;
  return __uint_as_float(bits);
}

// A block's scale byte and the factor its values are multiplied by before the code's rounding.
struct BlockScale {
  uint32_t byte;
  float mul;
  bool bad;  // the block holds an infinity or a NaN
};

// t / 6 rounded as division rounds it, by Markstein's method (a quotient from the rounded
// reciprocal, corrected once by its exact remainder), for 0 <= t <= 2^100; below 2^-100 the result is
// only near, which its rounding to E4M3 does not see.
__device__ __forceinline__ float sixth(float t) {
  constexpr float y = 1.0f / 6.0f;
  const float q = t * y;
  return fmaf(fmaf(-6.0f, q, t), y, q);
}

// NVFP4's factors fp32(s / scale) by the scale's byte, made once by the threads of a CTA (a division
// a block costs as much as the rest of its packing).  Entry 0 is 0: such a block holds zeros.  A quotient
// past the largest float becomes that float: with an infinite factor a zero of the block would turn
// into NaN, and its code into the largest.
constexpr int kNvFactors = 128;
__device__ __forceinline__ void nv_factors(float* table, float s, int thread, int threads) {
  for (int i = thread; i < kNvFactors; i += threads) {
    const float f = i == 0 || i == 0x7f ? 0.0f : __fdiv_rn(s, unpack_e4m3x2(uint16_t(i)).x);
    table[i] = f > kF32Max ? kF32Max : f;
  }
}

// factors: nv_factors' table of s (NVFP4 only).
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, float s, const float* factors) {
  BlockScale r;
  r.bad = amax_bits >= kInfBits;
  if constexpr (FMT == TE_NVFP4) {
    const float t = fminf(__fmul_rn(__uint_as_float(amax_bits), s), 65536.0f);  // saturates far below
    const uint32_t sb = pack_e4m3x2(sixth(t), 0.0f) & 0xffu;
    r.byte = r.bad ? 0x7fu : sb;
    r.mul = factors[sb];
  } else {
    // 6 = 1.5 * 2^2 and 448 = 1.75 * 2^8: one more when the mantissa is above the top's
    constexpr int kTopExp = FMT == TE_MXFP4 ? 2 : 8;
    constexpr uint32_t kTopMant = FMT == TE_MXFP4 ? 0x400000u : 0x600000u;
    int c = int(amax_bits >> 23) - kTopExp + ((amax_bits & 0x7fffffu) > kTopMant ? 1 : 0);
    c = c < 0 ? 0 : c;
    r.byte = r.bad ? 255u : uint32_t(c);
    r.mul = __uint_as_float(uint32_t(254 - c) << 23);  // 2^(127 - c); c <= 253
  }
  return r;
}

// fp32 tensor scale of NVFP4 from the tensor's amax: the block scales of the largest block reach
// E4M3's largest value (1 when amax is 0 or not finite, FLT_MAX if the quotient overflows).
__device__ __forceinline__ float nv_scale_from_amax(float amax) {
  if (!(amax > 0.0f) || !isfinite(amax)) return 1.0f;
  const float s = __fdiv_rn(6.0f * kE4M3Max, amax);
  return isfinite(s) ? s : kF32Max;
}

// max(m, |a|, |b|), NaN if one is: the largest magnitude of two more values in one instruction.
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// 8 neighbours of T as fp32.  load: memory that nothing writes while the kernel runs; load_fresh: what the
// kernel before a programmatic dependent may still have been writing when this one began.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldg(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_fresh(const void* p) { u = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void to_smem(void* p) const { *static_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  }
  // the largest magnitude, NaN ignored
  __device__ __forceinline__ float amax() const {
    auto abs2 = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
    const __nv_bfloat162 t = __hmax2(__hmax2(abs2(u.x), abs2(u.y)), __hmax2(abs2(u.z), abs2(u.w)));
    return fmaxf(__low2float(t), __high2float(t));
  }
  // its bits, those of a NaN above all others
  __device__ __forceinline__ uint32_t amax_bits() const {
    float v[8];
    get(v);
    float m = max_abs3(v[0], v[1], v[2]);
    m = max_abs3(m, v[3], v[4]);
    m = max_abs3(m, v[5], v[6]);
    return __float_as_uint(max_abs3(m, v[7], 0.0f));
  }
};
template <>
struct Eight<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldg(static_cast<const uint4*>(p));
    b = __ldg(static_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void load_fresh(const void* p) {
    a = static_cast<const uint4*>(p)[0];
    b = static_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void to_smem(void* p) const {
    static_cast<uint4*>(p)[0] = a;
    static_cast<uint4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z);
    v[3] = __uint_as_float(a.w); v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  }
  __device__ __forceinline__ float amax() const {
    auto f = [](uint32_t w) { return fabsf(__uint_as_float(w)); };
    return fmaxf(fmaxf(fmaxf(f(a.x), f(a.y)), fmaxf(f(a.z), f(a.w))),
                 fmaxf(fmaxf(f(b.x), f(b.y)), fmaxf(f(b.z), f(b.w))));
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    float v[8];
    get(v);
    float m = max_abs3(v[0], v[1], v[2]);
    m = max_abs3(m, v[3], v[4]);
    m = max_abs3(m, v[5], v[6]);
    return __float_as_uint(max_abs3(m, v[7], 0.0f));
  }
};

// Codes of 8 neighbours: 4 bytes (x) of E2M1 or 8 bytes of E4M3.
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const BlockScale& b) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 p = mul2(f2(x[2 * i], x[2 * i + 1]), f2s(b.mul));
    v[2 * i] = f2lo(p);
    v[2 * i + 1] = f2hi(p);
  }
  uint2 r = make_uint2(0u, 0u);
  if (b.bad) return r;
  if constexpr (FMT == TE_MXFP8) {
    r.x = pack_e4m3x4(v[0], v[1], v[2], v[3]);
    r.y = pack_e4m3x4(v[4], v[5], v[6], v[7]);
  } else {
    r.x = pack_e2m1x8(v);
  }
  return r;
}

}  // namespace te
