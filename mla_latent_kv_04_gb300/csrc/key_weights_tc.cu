// Accumulated attention weight of every cached token, on the tensor cores (bf16 cache, 64-token
// pages, d_c 512, d_r 64, a multiple of 16 heads up to 128).
//
// Per tile of 128 tokens (two pages) the scores of all heads are one product,
//   Z = X q_lat^T   (M = 128 tokens, N = heads, K = 576),
// tokens in the rows: a token's sum over heads is then a sum over the columns of one lane of
// tensor memory, in one thread's registers:
//   mass = sum_h exp2(c Z_h - log2(e) lse_h),   c = softmax scale * log2 e.
// q_lat is an operand as given (bf16), products are exact and sums fp32, so the weights are
// fp32 results.
//
// A run of tiles (key_runs.cuh) loads its request's query (H x 576) once; several query tokens are
// further columns as far as they fit. With more a run is passed over several times (the later passes
// read its pages from L2), each pass adding to the weights that the same thread wrote before: no
// atomics, one order of sums.
//
// Bound: the cache is read once, 147 KB a tile; the MMAs take a third of that time. 32 x 4096
// tokens take 28.5 us, 5.5 TB/s; four requests of 32K to 128K tokens 76 us, 6.1 TB/s.
#include <math.h>

#include "internal.h"
#include "key_runs.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace weigh {

constexpr int kD = 576, kChunks = 9;                   // 64 dims a chunk
constexpr int kStage = kTile * 64 * 2;                 // one chunk of a tile: 16 KB
constexpr int kStages = 5;
constexpr int kQChunk = 128 * 64 * 2;
constexpr int kOffRing = kChunks * kQChunk;            // the query first: 144 KB
constexpr int kOffLse = kOffRing + kStages * kStage;
constexpr int kOffBar = kOffLse + 512;
constexpr int kSmem = kOffBar + 256 + 1024;
static_assert(kSmem <= 232448 - 256, "dynamic shared memory per CTA");
constexpr int kThreads = 192;
enum { B_FULL = 0, B_EMPTY = kStages, B_QFULL = 2 * kStages, B_QEMPTY, B_ZFULL, B_ZFREE = B_ZFULL + 2,
       B_MEET = B_ZFREE + 2, B_TEAR, B_COUNT };

__global__ void __launch_bounds__(kThreads, 1)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_q,
                          const KeyWeightParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + kOffBar + 240);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + kOffBar + 244);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) ptx::mbar_init(bar(i), i >= B_ZFREE && i <= B_MEET ? 4 : 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_x);
    ptx::prefetch_tensormap(&tm_q);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 256);
    ptx::tmem_relinquish();
  }
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  // the scan's scratch is the query's place, not yet in use; a query's load costs about a tile
  Runs run = first_run(p, reinterpret_cast<int*>(basep), 1, 8);
  ptx::tc_fence_before();
  // the scratch is done with before the query's copy (through the async proxy) may land on it
  ptx::fence_proxy_async_smem();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  // a warp goes on, or gives up, as one
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = ptx::l2_policy_evict_first();
      uint32_t g = 0;
      bool ok = true;
      while (ok && run.next()) {
        for (int t = 0; ok && t < p.passes; ++t) {
          int y0 = run.row_of(2 * run.t0), y1 = run.row_of(2 * run.t0 + 1);
          for (int tile = run.t0; ok && tile < run.t1; ++tile) {
            const bool two = (long long)(2 * tile + 1) * 64 < run.S;
            int n0 = 0, n1 = 0;
            for (int c = 0; c < kChunks; ++c, ++g) {
              const uint32_t st = g % kStages;
              if (!(ok = wait(B_EMPTY + st, ((g / kStages) & 1) ^ 1))) break;
              const uint32_t dst = base + kOffRing + st * kStage, full = bar(B_FULL + st);
              ptx::mbar_arrive_expect_tx(full, two ? kStage : kStage / 2);
              if (p.passes > 1) {
                ptx::tma_load_3d(dst, &tm_x, 64 * c, y0, 0, full);
                if (two) ptx::tma_load_3d(dst + kStage / 2, &tm_x, 64 * c, y1, 0, full);
              } else {
                ptx::tma_load_3d_hint(dst, &tm_x, 64 * c, y0, 0, full, pol);
                if (two) ptx::tma_load_3d_hint(dst + kStage / 2, &tm_x, 64 * c, y1, 0, full, pol);
              }
              if (c == 0 && tile + 1 < run.t1) {       // the next tile's pages, ahead of need
                n0 = run.row_of(2 * tile + 2);
                n1 = run.row_of(2 * tile + 3);
              }
            }
            y0 = n0;
            y1 = n1;
          }
        }
      }
      if (*abort)
        for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i)
          drain_wait(bar(B_FULL + i % kStages), (i / kStages) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = ptx::idesc_bf16_f32(128, p.cols, false, false);
    uint32_t g = 0, q_iter = 0, z = 0;
    bool ok = true;
    while (ok && run.next()) {
      for (int t = 0; ok && t < p.passes; ++t, ++q_iter) {
        // the query of this run and token: B_QEMPTY says that the MMAs on the one before are done
        if (!(ok = wait_w(B_QEMPTY, (q_iter & 1) ^ 1))) break;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(bar(B_QFULL), kChunks * p.cols * 128);
          for (int c = 0; c < kChunks; ++c)
            ptx::tma_load_3d(base + c * kQChunk, &tm_q, 64 * c, 0, run.rb * p.passes + t, bar(B_QFULL));
        }
        __syncwarp();
        if (!(ok = wait_w(B_QFULL, q_iter & 1))) break;
        for (int tile = run.t0; ok && tile < run.t1; ++tile, ++z) {
          if (!(ok = wait_w(B_ZFREE + (z & 1), ((z >> 1) & 1) ^ 1))) break;
          for (int c = 0; c < kChunks; ++c, ++g) {
            const uint32_t st = g % kStages;
            if (!(ok = wait_w(B_FULL + st, (g / kStages) & 1))) break;
            ptx::tc_fence_after();
            const uint32_t x = base + kOffRing + st * kStage, q = base + c * kQChunk;
            if (ptx::elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ptx::mma_bf16_ss(tmem + 128 * (z & 1), ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                                 ptx::smem_desc(q + 32 * k, 16, 1024, ptx::kSwizzle128), idesc,
                                 (c || k) ? 1u : 0u);
              ptx::mma_commit(bar(B_EMPTY + st));
              if (c == kChunks - 1) {
                ptx::mma_commit(bar(B_ZFULL + (z & 1)));
                if (tile == run.t1 - 1) ptx::mma_commit(bar(B_QEMPTY));
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (*abort) {
      if (ptx::elect_one()) ptx::mma_commit(bar(B_TEAR));
      __syncwarp();
      drain_wait(bar(B_TEAR), 0);
      if (q_iter) drain_wait(bar(B_QFULL), (q_iter - 1) & 1);
      drain_wait(bar(B_QFULL), q_iter & 1);
    }
  } else {
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16);
    float* lse_s = reinterpret_cast<float*>(basep + kOffLse);
    uint32_t z = 0, meets = 0;
    bool ok = true;
    auto meet = [&]() {                                // the four warps (bounded, unlike a named barrier)
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_MEET));
      return wait_w(B_MEET, meets++ & 1);
    };
    while (ok && run.next()) {
      const int32_t* bt = p.block_table + (long long)run.rb * p.max_pages;
      const int S = run.S;
      float* w = p.weights + (long long)run.rb * p.max_pages * p.P;
      for (int t = 0; ok && t < p.passes; ++t) {
        const float* lse = p.lse + ((long long)run.rb * p.passes + t) * p.cols;
        if (!(ok = meet())) break;
        if (row < p.cols) lse_s[row] = lse[row] * kLog2e;
        if (!(ok = meet())) break;
        for (int tile = run.t0; tile < run.t1; ++tile, ++z) {
          if (!(ok = wait_w(B_ZFULL + (z & 1), (z >> 1) & 1))) break;
          ptx::tc_fence_after();
          const int j = tile * kTile + row, from = first_column(p, S, j, t);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          for (int h0 = 0; h0 < p.cols; h0 += 16) {
            uint32_t v[16];
            ptx::tmem_ld16(t_row + 128 * (z & 1) + h0, v);
            ptx::tmem_wait_ld();
            const bool sees = h0 >= from;              // (a query token's columns are a multiple of 16)
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 off = *reinterpret_cast<const float4*>(lse_s + h0 + j);
              const float e[4] = {ptx::ex2(fmaf(__uint_as_float(v[j]), p.scale_log2, -off.x)),
                                  ptx::ex2(fmaf(__uint_as_float(v[j + 1]), p.scale_log2, -off.y)),
                                  ptx::ex2(fmaf(__uint_as_float(v[j + 2]), p.scale_log2, -off.z)),
                                  ptx::ex2(fmaf(__uint_as_float(v[j + 3]), p.scale_log2, -off.w))};
#pragma unroll
              for (int k = 0; k < 4; ++k) sum[k] += sees ? e[k] : 0.f;
            }
            __syncwarp();                              // the next load is warp-wide
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(B_ZFREE + (z & 1)));
          if (j < S) {
            const int page = bt[j / 64];
            if (page >= 0 && page < p.num_pages) {
              const float mass = (sum[0] + sum[1]) + (sum[2] + sum[3]);
              if (t == 0) w[j] = (p.decay != 0.f && j < S - p.q_len) ? fmaf(p.decay, w[j], mass) : mass;
              else if (from < p.cols) w[j] += mass;
            }
          }
        }
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 256);
  }
}

}  // namespace weigh

bool key_weights_tc_supported(const mla_config* c, long long num_pages) {
  return c->act_dtype == MLA_BF16 && c->page_size == 64 && c->d_latent == 512 && c->d_rope == 64 &&
         c->num_heads % 16 == 0 && c->num_heads <= 128 && num_pages * 64 <= 0x7FFFFF00LL;
}

cudaError_t launch_key_weights_tc(mla_dtype cache, KeyWeightParams p, cudaStream_t s) {
  using namespace weigh;
  set_passes(p);
  if (cache != MLA_BF16) return launch_key_weights_fp8(cache, p, s);
  CUtensorMap x, q;
  const uint64_t rows = (uint64_t)p.num_pages * 64;
  if (!tensor_map_bf16(&x, p.cache, kD, rows, 1, kD * 2, rows * kD * 2, 64, 64) ||
      !tensor_map_bf16(&q, p.q_lat, kD, (uint64_t)p.cols, (uint64_t)p.batch * p.passes, kD * 2,
                       (uint64_t)p.cols * kD * 2, 64, (uint32_t)p.cols))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(key_weights_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid_size(p), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, key_weights_tc_kernel, x, q, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace mla
