// Conversions between e4m3 codes, f32 and packed bf16.
#pragma once
#include "common.cuh"

namespace mla {

// Two e4m3 codes (low byte first) as f32, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t pair) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(pair));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Four bf16 values of the query (two pairs) times s -> four hi codes and four lo codes, by
// integer arithmetic (with conversion instructions a query took as long or longer). The values are formed as y = 2^-8 2^e q in f16 (s = 2^(e - 8)): then e4m3's exponent
// field is f16's (bias 7 against 15) and a code is bits 13 to 7 of y, rounded to nearest even at bit
// 7, its sign bit 15; subnormals alike.
__device__ __forceinline__ void split4(uint32_t q01, uint32_t q23, float s, uint32_t* hi, uint32_t* lo) {
  auto scaled = [&](uint32_t q) {
    const __half2 h = __floats2half2_rn(__uint_as_float(q << 16) * s, __uint_as_float(q & 0xFFFF0000u) * s);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  auto rounded = [](uint32_t y) { return y + 0x003F003Fu + ((y >> 7) & 0x00010001u); };
  auto codes = [](uint32_t t0, uint32_t t1) {
    const uint32_t mag = __byte_perm(t0 << 1, t1 << 1, 0x7531), sign = __byte_perm(t0, t1, 0x7531);
    return (mag & 0x7F7F7F7Fu) | (sign & 0x80808080u);
  };
  auto rest = [](uint32_t y, uint32_t t) {             // 16 (y - hi), exactly: at most 4 bits left, cut off
    t &= 0xFF80FF80u;
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&t)),
                              __floats2half2_rn(16.f, 16.f));
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  const uint32_t y0 = scaled(q01), y1 = scaled(q23), t0 = rounded(y0), t1 = rounded(y1);
  *hi = codes(t0, t1);
  *lo = codes(rest(y0, t0), rest(y1, t1));             // (nothing to round but subnormals)
}

}  // namespace mla
