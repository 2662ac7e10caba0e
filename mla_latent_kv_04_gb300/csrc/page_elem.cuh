// Reads of one cache row held in 32-bit words, per storage format: an element's value (without
// a per-tensor scale) and the dot product with an fp32 vector.
#pragma once
#include "common.cuh"

namespace mla {

template <typename CT> struct PageElem;
template <> struct PageElem<float> {
  __device__ __forceinline__ static float get(const uint32_t* row, int k, int) {
    return __uint_as_float(row[k]);
  }
  __device__ __forceinline__ static float dot(const uint32_t* row, const float* q, int D, int) {
    float acc = 0.f;
    for (int w = 0; w < D; ++w) acc = fmaf(q[w], __uint_as_float(row[w]), acc);
    return acc;
  }
};
template <> struct PageElem<bf16> {
  __device__ __forceinline__ static float get(const uint32_t* row, int k, int) {
    const uint32_t w = row[k >> 1];
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ static float dot(const uint32_t* row, const float* q, int D, int) {
    float acc = 0.f;
    for (int w = 0; w < D / 2; ++w) {
      const uint32_t v = row[w];
      acc = fmaf(q[2 * w], __uint_as_float(v << 16), acc);
      acc = fmaf(q[2 * w + 1], __uint_as_float(v & 0xFFFF0000u), acc);
    }
    return acc;
  }
};
template <> struct PageElem<uint8_t> {
  __device__ __forceinline__ static float get(const uint32_t* row, int k, int) {
    return fp8_to_f32((uint8_t)(row[k >> 2] >> (8 * (k & 3))));
  }
  __device__ __forceinline__ static float dot(const uint32_t* row, const float* q, int D, int) {
    float acc = 0.f;
    for (int w = 0; w < D / 4; ++w) {
      const uint32_t v = row[w];
#pragma unroll
      for (int b = 0; b < 4; ++b) acc = fmaf(q[4 * w + b], fp8_to_f32((uint8_t)(v >> (8 * b))), acc);
    }
    return acc;
  }
};
// Block-scaled fp8 rows: d_c e4m3 codes, d_c / 128 fp32 scales, d_r bf16 (k_pe).
struct E4m3B128 {};
template <> struct PageElem<E4m3B128> {
  __device__ __forceinline__ static float get(const uint32_t* row, int k, int d_c) {
    return fp8_to_f32((uint8_t)(row[k >> 2] >> (8 * (k & 3)))) * __uint_as_float(row[(d_c >> 2) + (k >> 7)]);
  }
  __device__ __forceinline__ static float dot(const uint32_t* row, const float* q, int D, int d_c) {
    float acc = 0.f;
    for (int blk = 0; blk < d_c / 128; ++blk) {
      float part = 0.f;
      for (int w = 32 * blk; w < 32 * blk + 32; ++w) {
        const uint32_t v = row[w];
#pragma unroll
        for (int b = 0; b < 4; ++b) part = fmaf(q[4 * w + b], fp8_to_f32((uint8_t)(v >> (8 * b))), part);
      }
      acc = fmaf(part, __uint_as_float(row[(d_c >> 2) + blk]), acc);
    }
    const uint32_t* kr = row + (d_c >> 2) + (d_c >> 7);
    for (int w = 0; w < (D - d_c) / 2; ++w) {
      const uint32_t v = kr[w];
      acc = fmaf(q[d_c + 2 * w], __uint_as_float(v << 16), acc);
      acc = fmaf(q[d_c + 2 * w + 1], __uint_as_float(v & 0xFFFF0000u), acc);
    }
    return acc;
  }
};

// Rotary element k of a row (without a per-tensor scale).
template <typename CT>
__device__ __forceinline__ float page_rope_elem(const uint32_t* row, int k, int d_c) {
  return PageElem<CT>::get(row, d_c + k, d_c);
}
template <>
__device__ __forceinline__ float page_rope_elem<E4m3B128>(const uint32_t* row, int k, int d_c) {
  const uint32_t w = row[(d_c >> 2) + (d_c >> 7) + (k >> 1)];
  return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
}

}  // namespace mla
