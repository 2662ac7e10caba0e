// 4-bit weights: e2m1 codes with one power of two per 32 elements of the summed dimension (the OCP
// microscaling layout of elements and scales), their values, and the product with them in SIMT form
// (the tensor-core form is mx4_tc.cu).
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

#include "internal.h"
#include "mx4.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace mla {
namespace {

constexpr int kTileN = 64, kTileK = 256;       // columns and rows of W that a block takes
constexpr int kThreads = 256;
constexpr int kRowWords = kTileK / 8 + 4;      // a column's codes in shared memory (128 bytes, padded)

// ======================================================================== quantisation
// Warp = one block of 32 rows x 64 columns, two columns a lane: W is read in rows, once; the codes of
// a column (16 bytes a warp) are put together in shared memory and written 128 bytes at a time.
// Bound by memory: 65536 x 5120 bf16 weights (671 MB in, 178 out) in 141 us, 6.0 TB/s; back to bf16 in 130.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const T* __restrict__ W, int K, int N,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  __shared__ uint32_t code_s[kTileN][kRowWords];
  __shared__ uint8_t scale_s[kTileN][kTileK / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kTileN, k0 = blockIdx.y * kTileK;
  const int kb = k0 + 32 * warp;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
#pragma unroll
  for (int half = 0; half < (kPair ? 1 : 2); ++half) {
    constexpr int kCols = kPair ? 2 : 1;
    const int c0 = kPair ? 2 * lane : lane + 32 * half;
    float v[kCols][32];
    uint32_t top[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) top[c] = 0u;
    if (kb < K && n0 + c0 < N) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const T* src = W + (long long)(kb + i) * N + n0 + c0;
        if constexpr (kPair && sizeof(T) == 2) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(src);
          v[0][i] = __uint_as_float(x << 16);
          v[kCols - 1][i] = __uint_as_float(x & 0xFFFF0000u);
        } else if constexpr (kPair) {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[0][i] = x.x;
          v[kCols - 1][i] = x.y;
        } else {
          v[0][i] = to_f32(*src);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[c][i] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
#pragma unroll
      for (int i = 0; i < 32; ++i) top[c] = max(top[c], __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
      const int byte = kb < K && n0 + c0 + c < N ? mx4::scale_byte(top[c]) : 127;
      const float inv = mx4::inverse_scale(byte);
      scale_s[c0 + c][warp] = (uint8_t)byte;
      uint32_t word[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        word[j] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 pair = make_float2(v[c][8 * j + 2 * i] * inv, v[c][8 * j + 2 * i + 1] * inv);
          word[j] |= (uint32_t)__nv_cvt_float2_to_fp4x2(pair, __NV_E2M1, cudaRoundNearest) << (8 * i);
        }
        code_s[c0 + c][4 * warp + j] = word[j];
      }
    }
  }
  __syncthreads();
  // 8 pieces of 16 bytes a column
  for (int i = threadIdx.x; i < kTileN * 8; i += kThreads) {
    const int n = i / 8, j = i % 8;
    if (n0 + n < N && k0 + 32 * j < K)
      *reinterpret_cast<uint4*>(codes + (long long)(n0 + n) * (K / 2) + k0 / 2 + 16 * j) =
          *reinterpret_cast<const uint4*>(&code_s[n][4 * j]);
  }
  // the scale tiles are whole: columns behind N and blocks behind K hold 1
  const int groups = (K + 127) / 128;
  if (threadIdx.x < kTileN * 2) {
    const int n = threadIdx.x / 2, j = threadIdx.x % 2, kg = k0 / 128 + j;
    if (kg < groups)
      *reinterpret_cast<uint32_t*>(scales + mx4::scale_at(n0 + n, kg * 4, groups)) =
          *reinterpret_cast<const uint32_t*>(&scale_s[n][4 * j]);
  }
}

// ======================================================================== values
// The same tiles the other way: codes in 16-byte pieces, W in rows. Every value is exact in bf16.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, int K,
                                                                  int N, T* __restrict__ W) {
  __shared__ uint32_t code_s[kTileN][kRowWords];
  __shared__ uint8_t scale_s[kTileN][kTileK / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kTileN, k0 = blockIdx.y * kTileK, groups = (K + 127) / 128;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  for (int i = threadIdx.x; i < kTileN * 8; i += kThreads) {
    const int n = i / 8, j = i % 8;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (n0 + n < N && k0 + 32 * j < K)
      x = *reinterpret_cast<const uint4*>(codes + (long long)(n0 + n) * (K / 2) + k0 / 2 + 16 * j);
    *reinterpret_cast<uint4*>(&code_s[n][4 * j]) = x;
  }
  if (threadIdx.x < kTileN * 2) {
    const int n = threadIdx.x / 2, j = threadIdx.x % 2, kg = k0 / 128 + j;
    if (kg < groups)
      *reinterpret_cast<uint32_t*>(&scale_s[n][4 * j]) =
          *reinterpret_cast<const uint32_t*>(scales + mx4::scale_at(n0 + n, kg * 4, groups));
  }
  __syncthreads();
  const int kb = k0 + 32 * warp;
  if (kb >= K) return;
#pragma unroll
  for (int half = 0; half < (kPair ? 1 : 2); ++half) {
    constexpr int kCols = kPair ? 2 : 1;
    const int c0 = kPair ? 2 * lane : lane + 32 * half;
    if (n0 + c0 >= N) continue;
    float scale[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) scale[c] = mx4::scale_value(scale_s[c0 + c][warp]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t word[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) word[c] = code_s[c0 + c][4 * warp + j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 y[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          y[c] = mx4::values((uint8_t)(word[c] >> (8 * i)));
          y[c].x *= scale[c];
          y[c].y *= scale[c];
        }
        T* dst = W + (long long)(kb + 8 * j + 2 * i) * N + n0 + c0;
        if constexpr (kPair && sizeof(T) == 2) {
          *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(y[0].x, y[kCols - 1].x);
          *reinterpret_cast<__nv_bfloat162*>(dst + N) = __floats2bfloat162_rn(y[0].y, y[kCols - 1].y);
        } else if constexpr (kPair) {
          *reinterpret_cast<float2*>(dst) = make_float2(y[0].x, y[kCols - 1].x);
          *reinterpret_cast<float2*>(dst + N) = make_float2(y[0].y, y[kCols - 1].y);
        } else {
          dst[0] = from_f32<T>(y[0].x);
          dst[N] = from_f32<T>(y[0].y);
        }
      }
    }
  }
}

// ======================================================================== product (SIMT)
// Warp per two columns and up to kR rows, eight elements of K a lane and step, so that codes and rows are read
// in order (64 rows x 4096 x 2048 in fp32: 125 us; with a block of 32 elements a lane 870); fp32 throughout.
constexpr int kR = 4;

// Eight elements of x, in one or two 16-byte loads where it starts at a multiple of 16 bytes.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
  if constexpr (kVec && sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else if constexpr (kVec) {
    const uint4 a = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(src[i]);
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(256) mx4_project_kernel(const T* __restrict__ x, const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int K, int N,
                                                          int rows, T* __restrict__ out) {
  const int n0 = 2 * (blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31, groups = (K + 127) / 128;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (n0 >= N) return;
  const int n1 = min(n0 + 1, N - 1);
  for (int r0 = blockIdx.y * kR; r0 < rows; r0 += gridDim.y * kR) {
    float acc[2][kR] = {};
    for (int k = 8 * lane; k < K; k += 256) {
      float w[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = c ? n1 : n0;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + (long long)n * (K / 2) + k / 2);
        const float scale = mx4::scale_value(scales[mx4::scale_at(n, k / 32, groups)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = mx4::values((uint8_t)(word >> (8 * i)));
          w[c][2 * i] = v.x * scale;
          w[c][2 * i + 1] = v.y * scale;
        }
      }
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r0 + r >= rows) break;
        float v[8];
        load8<T, kVec>(x + (long long)(r0 + r) * K + k, v);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[c][r] = fmaf(v[i], w[c][i], acc[c][r]);
      }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float s = warp_sum(acc[c][r]);
        if (lane == 0 && r0 + r < rows && n0 + c < N) out[(long long)(r0 + r) * N + n0 + c] = from_f32<T>(s);
      }
  }
}

// Two columns at a time: rows of an even length that start at a multiple of two elements.
template <typename T>
bool pairs(const void* W, int N) { return N % 2 == 0 && ((uintptr_t)W & (2 * sizeof(T) - 1)) == 0; }

dim3 tiles(int K, int N) {
  return dim3((unsigned)((N + 127) / 128 * (128 / kTileN)), (unsigned)((K + kTileK - 1) / kTileK), 1);
}

template <typename T>
cudaError_t quantize_t(const void* W, int K, int N, void* codes, void* scales, cudaStream_t s) {
  auto kern = pairs<T>(W, N) ? mx4_quantize_kernel<T, true> : mx4_quantize_kernel<T, false>;
  return launch_pdl(kern, tiles(K, N), kThreads, 0, s, (const T*)W, K, N, (uint8_t*)codes, (uint8_t*)scales);
}
template <typename T>
cudaError_t dequantize_t(const void* codes, const void* scales, int K, int N, void* W, cudaStream_t s) {
  auto kern = pairs<T>(W, N) ? mx4_dequantize_kernel<T, true> : mx4_dequantize_kernel<T, false>;
  return launch_pdl(kern, tiles(K, N), kThreads, 0, s, (const uint8_t*)codes, (const uint8_t*)scales, K, N, (T*)W);
}
template <typename T>
cudaError_t project_t(const void* x, const void* codes, const void* scales, int K, int N, int rows, void* out,
                      cudaStream_t s) {
  auto kern = ((uintptr_t)x & 15) == 0 ? mx4_project_kernel<T, true> : mx4_project_kernel<T, false>;
  return launch_pdl(kern, dim3((unsigned)((N + 15) / 16), (unsigned)std::min((rows + kR - 1) / kR, 32768), 1), 256, 0, s,
                    (const T*)x, (const uint8_t*)codes, (const uint8_t*)scales, K, N, rows, (T*)out);
}

}  // namespace

cudaError_t launch_mx4_quantize(mla_dtype act, const void* W, int K, int N, void* codes, void* scales,
                                cudaStream_t s) {
  return act == MLA_F32 ? quantize_t<float>(W, K, N, codes, scales, s) : quantize_t<bf16>(W, K, N, codes, scales, s);
}
cudaError_t launch_mx4_dequantize(mla_dtype act, const void* codes, const void* scales, int K, int N, void* W,
                                  cudaStream_t s) {
  return act == MLA_F32 ? dequantize_t<float>(codes, scales, K, N, W, s)
                        : dequantize_t<bf16>(codes, scales, K, N, W, s);
}
cudaError_t launch_mx4_project_simt(mla_dtype act, const void* x, const void* codes, const void* scales, int K,
                                    int N, int rows, void* out, cudaStream_t s) {
  return act == MLA_F32 ? project_t<float>(x, codes, scales, K, N, rows, out, s)
                        : project_t<bf16>(x, codes, scales, K, N, rows, out, s);
}

}  // namespace mla
