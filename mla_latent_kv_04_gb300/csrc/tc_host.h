// Host-side helpers of the kernels: tensor maps, the SM count, launches.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mla {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// 3-D map {d0 (contiguous), d1, d2}, byte strides of d1 and d2, box {b0, b1, 1}; out of range
// reads as zero. False if the driver refuses it (a base that is not 16-byte aligned, say).
inline bool tensor_map_3d(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle,
                          const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                          uint64_t s2, uint32_t b0, uint32_t b1) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {s1, s2};
  cuuint32_t box[3] = {b0, b1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool tensor_map_bf16(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2,
                            uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1) {
  return tensor_map_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, ptr, d0, d1, d2, s1,
                       s2, b0, b1);
}

// SMs of the current device.
inline int device_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

// Shared memory of one CTA (227 KB), static and dynamic together.
constexpr size_t kSmemPerCta = 232448;

// Lets a kernel with `fixed` bytes of static shared memory have more than 48 KB in all. The limit
// belongs to the kernel and not to a launch, so it goes to the most that any call may need: set to
// one call's need, another host thread could lower it between this call's setting and its launch.
template <typename K>
inline cudaError_t allow_smem(K kern, size_t dynamic, size_t fixed = 0) {
  if (dynamic + fixed <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSmemPerCta - fixed));
}

// A launch with programmatic serialization: it may start while the kernel before it in the stream ends, and
// waits for that one (griddepcontrol.wait) before it reads or writes.
void note_launch(int n);
template <typename K, typename... A>
inline cudaError_t launch_pdl(K kern, dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) note_launch(1);
  return e;
}

}  // namespace mla
