// 4-bit weights: scales and element values.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "common.cuh"

namespace mla {
namespace mx4 {

// Scale byte e of a block whose largest magnitude has the fp32 bits `top`: the scale is 2^(e - 127), the
// power of two under `top` rounded to two significant bits, divided by 4 (so that `top` lies in [3.5, 7)
// scales and becomes 4 or 6). At most 2^125 (6 scales stay finite). A block that holds an infinity or
// NaN gets the scale NaN (255).
__device__ __forceinline__ int scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255;
  const int e = (int)((top + (1u << 21)) >> 23) - 2;
  return e < 0 ? 0 : (e > 252 ? 252 : e);
}
__device__ __forceinline__ float scale_value(int byte) {
  if (byte == 255) return __uint_as_float(0x7FFFFFFFu);
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)byte << 23);   // (2^-127: subnormal)
}
// 1 / scale of a byte up to 253 (NaN blocks: any).
__device__ __forceinline__ float inverse_scale(int byte) {
  return byte == 255 ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
}

// Where the scale of column n and block blk (of 32 rows) lies: tiles of 128 columns x 4 blocks, in the
// order in which the tensor cores take them (column n % 32 first, then n / 32, then the block).
__device__ __forceinline__ long long scale_at(int n, int blk, int groups) {
  return ((long long)(n / 128) * groups + blk / 4) * 512 + (n % 32) * 16 + (n % 128) / 32 * 4 + blk % 4;
}

// The two values of a byte (low nibble first).
__device__ __forceinline__ float2 values(uint8_t b) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1);
  return __half22float2(__half2(h));
}

}  // namespace mx4
}  // namespace mla
