// Expansion of e4m3 codes in shared memory into the bf16 tiles that the MMAs read.
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

// Half a token row (32 dims, half 0 or 1) of a 64-dim chunk: the 32 codes times `scale` as bf16
// into a tile of 128-byte rows with the 128-byte swizzle. With kLow, what the rounding left over
// goes to that second tile as another bf16 (the two add up to the product within 2^-17 of it).
// Without a scale the codes are exact.
template <bool kScaled, bool kLow>
__device__ __forceinline__ void expand_codes_half_row(const uint4 (&code)[2], uint8_t* hi, uint8_t* lo, int row,
                                                      int half, float scale) {
#pragma unroll
  for (int ii = 0; ii < 2; ++ii) {
    const int i = 2 * half + ii;
    const uint32_t w[4] = {code[ii].x, code[ii].y, code[ii].z, code[ii].w};
    uint32_t h[8], l[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2 f = e4m3x2_to_f32(k ? w[j] >> 16 : w[j] & 0xFFFFu);
        if (kScaled) {
          f.x *= scale;
          f.y *= scale;
        }
        h[2 * j + k] = pack_bf16(f.x, f.y);
        if (kLow)
          l[2 * j + k] = pack_bf16(f.x - __uint_as_float(h[2 * j + k] << 16),
                                   f.y - __uint_as_float(h[2 * j + k] & 0xFFFF0000u));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = row * 128 + (((2 * i + k) ^ (row & 7)) << 4);
      *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
      if (kLow)
        *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[4 * k], l[4 * k + 1], l[4 * k + 2], l[4 * k + 3]);
    }
  }
}

// The codes of half a token row in a tile of 64-byte rows with the 64-byte swizzle.
__device__ __forceinline__ void load_codes_half_row(const uint8_t* codes, int row, int half, uint4 (&code)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    code[i] = *reinterpret_cast<const uint4*>(codes + row * 64 + (((2 * half + i) ^ ((row >> 1) & 3)) << 4));
}

}  // namespace mla
