// Expansion of a prefix's cached latents into per-head keys and values, on the tensor cores
// (bf16 activations, 64-token pages, d_c 512, d_r 64, d_n = d_v = 128; every cache format).
//
//   keys[h] = C W_UK[:, h],  values[h] = C W_UV[:, h]     (C: L x 512; 128 columns per head)
//
// A pair of CTAs takes 256 tokens and a head at a time, as one MMA over both (cta_group::2, M = 256
// tokens, N = 256: the head's keys and values): CTA r holds token rows 128 r .. of the tile, all
// 512 dims of them, resident in its shared memory (128 KB), and streams as its half of N the
// head's 512 x 128 slice of W_UK (r = 0) or W_UV (r = 1), 16 KB for every 512 MMA cycles. Its
// MMAs read 64 bytes of shared memory a cycle. (With one CTA per 128 x 128 tile and the token
// chunks multicast to the pair, 8192 tokens took 333 us: 128 bytes a cycle of operand reads plus
// the fill are more than shared memory gives.) The accumulators (256 columns) are double-buffered
// in tensor memory, so that the conversion to bf16 and the stores (through shared memory, by TMA,
// which leaves out rows behind L) overlap the next head's MMAs. The (token tile, head) units in
// this order are cut into one contiguous range per pair.
//
// fp8 caches: a tile's codes are read once, when the pair turns to it, and eight warps expand them
// into the resident bf16 rows; every head then finds them there (expanding them again for each
// head took 75 us instead of WXYZ for 1000 tokens). A per-tensor scale multiplies the fp32 sums
// (codes are exact in bf16); block scales multiply the codes and the product is rounded to bf16,
// which adds as much error as the rounding of the result does.
//
// Bound: the MMAs (4096 cycles for a tile of 256 x 256 x 512 on two SMs).
#include "fp8_tiles.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace expand {

constexpr int kTile = 256, kChunks = 8;                // tokens of a pair's tile; chunks of 64 dims
constexpr int kChunk = 128 * 64 * 2;                   // one CTA's half of a chunk in bf16: 16 KB
constexpr int kRing = 5;                               // weight chunks in flight
constexpr int kOffX = 0;                               // the resident tokens: 8 chunks of 128 x 64
constexpr int kOffOut = kChunks * kChunk;              // 2 KB of output staging per epilogue warp
constexpr int kOffRing = kOffOut + 8 * 2048;
constexpr int kOffBar = kOffRing + kRing * kChunk;
constexpr int kSmem = kOffBar + 512 + 1024;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kConvWarps = 8;
template <int kKind>
constexpr int kThreads = 384 + (kKind ? 32 * kConvWarps : 0);
// WFULL, XFULL and DFREE are used in the even CTA alone (its MMA warp waits for both CTAs); WEMPTY,
// XEMPTY and DFULL in each (the MMAs' commits go to both)
enum { B_WFULL = 0, B_WEMPTY = kRing, B_XFULL = 2 * kRing, B_XEMPTY = B_XFULL + kChunks,
       B_DFULL = B_XEMPTY + 1, B_DFREE = B_DFULL + 2, B_TEAR = B_DFREE + 2, B_COUNT };

struct Job {
  PrefixExpandParams p;
  int tiles;                                           // token tiles
  int pairs;
};

// kKind: 0 bf16 cache, 1 e4m3 with one scale, 2 e4m3 with block scales
template <int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<kKind>, 1)
    expand_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_wk,
                     const __grid_constant__ CUtensorMap tm_wv, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Job job) {
  extern __shared__ uint8_t smem_raw[];
  const PrefixExpandParams& p = job.p;
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + kOffBar + 496);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + kOffBar + 500);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank(), pair = blockIdx.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      int n = 1;
      if (kKind != 0 && i >= B_XFULL && i < B_XEMPTY) n = 2 * kConvWarps;   // both CTAs' converters
      if (i >= B_DFREE && i < B_TEAR) n = 16;                        // both CTAs' epilogue warps
      ptx::mbar_init(bar(i), n);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_x);
    ptx::prefetch_tensormap(rank ? &tm_wv : &tm_wk);
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  ptx::cluster_sync();                                 // both CTAs run, with their barriers set up
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  auto wait_w = [&](int i, uint32_t parity) {          // a warp goes on, or gives up, as one
    return __all_sync(0xffffffffu, bounded_wait<true>(bar(i), parity, abort, p.status)) != 0;
  };
  // the even CTA's barriers, as an address that both CTAs can signal
  auto lead = [&](int i) { return ptx::map_to_rank(bar(i), 0u); };
  const int units = p.H * job.tiles;
  const int u0 = (int)((long long)units * pair / job.pairs), u1 = (int)((long long)units * (pair + 1) / job.pairs);
  const int tile0 = u0 / p.H, h0 = u0 % p.H;
  // the page that holds token l (a multiple of 64): -1 behind the prefix or with a bad id
  auto page_of = [&](int l) {
    if (l >= p.L) return -1;
    const int page = p.table[l >> 6];
    return page >= 0 && page < p.num_pages ? page : -1;
  };

  if (warp == 0) {
    if (lane == 0) {                                   // this CTA's half of every weight chunk
      const CUtensorMap* tm = rank ? &tm_wv : &tm_wk;
      uint32_t g = 0;
      bool ok = true;
      for (int u = u0, h = h0; ok && u < u1; ++u) {
        for (int c = 0; c < kChunks; ++c, ++g) {
          const uint32_t st = g % kRing;
          if (!(ok = wait(B_WEMPTY + st, ((g / kRing) & 1) ^ 1))) break;
          const uint32_t dst = base + kOffRing + st * kChunk, full = lead(B_WFULL + st);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_WFULL + st), 2 * kChunk);
          ptx::tma_load_3d_pair(dst, tm, h * 128, 64 * c, 0, full);
          ptx::tma_load_3d_pair(dst + kChunk / 2, tm, h * 128 + 64, 64 * c, 0, full);
        }
        if (++h == p.H) h = 0;
      }
      if (*abort && rank == 0)
        for (uint32_t i = g > kRing ? g - kRing : 0; i < g; ++i)
          drain_wait(bar(B_WFULL + i % kRing), (i / kRing) & 1);
    }
  } else if (warp == 2) {
    if (kKind == 0 && lane == 0) {                     // the token tile, when it changes
      uint32_t n = 0;
      bool ok = true;
      for (int u = u0, tile = tile0; ok && u < u1; u = ++tile * p.H, ++n) {
        const int l = tile * kTile + 128 * rank;
        const int a = page_of(l), b = page_of(l + 64);
        // rows out of the tensor's range read as zero
        const int y0 = (a >= 0 ? a : p.num_pages) * 64, y1 = (b >= 0 ? b : p.num_pages) * 64;
        if (!(ok = wait(B_XEMPTY, (n & 1) ^ 1))) break;
        for (int c = 0; c < kChunks; ++c) {
          const uint32_t dst = base + kOffX + c * kChunk, full = lead(B_XFULL + c);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_XFULL + c), 2 * kChunk);
          ptx::tma_load_3d_pair(dst, &tm_x, 64 * c, y0, 0, full);
          ptx::tma_load_3d_pair(dst + kChunk / 2, &tm_x, 64 * c, y1, 0, full);
        }
      }
      if (*abort && n && rank == 0)
        for (int c = 0; c < kChunks; ++c) drain_wait(bar(B_XFULL + c), (n - 1) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(256, 256, false, true);
      uint32_t g = 0, z = 0, n = 0;
      bool ok = true;
      for (int u = u0, h = h0; ok && u < u1; ++u, ++z) {
        const bool first = u == u0 || h == 0;
        const bool last = u + 1 == u1 || h + 1 == p.H;
        if (++h == p.H) h = 0;
        if (!(ok = wait_w(B_DFREE + (z & 1), ((z >> 1) & 1) ^ 1))) break;
        for (int c = 0; c < kChunks; ++c, ++g) {
          const uint32_t st = g % kRing;
          if (first && !(ok = wait_w(B_XFULL + c, n & 1))) break;
          if (!(ok = wait_w(B_WFULL + st, (g / kRing) & 1))) break;
          ptx::tc_fence_after();
          const uint32_t x = base + kOffX + c * kChunk, w = base + kOffRing + st * kChunk;
          if (ptx::elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_bf16_ss_pair(tmem + 256 * (z & 1), ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                                    ptx::smem_desc(w + 2048 * k, kChunk / 2, 1024, ptx::kSwizzle128), kIdesc,
                                    (c || k) ? 1u : 0u);
            ptx::mma_commit_pair(bar(B_WEMPTY + st));
            if (c == kChunks - 1) {
              ptx::mma_commit_pair(bar(B_DFULL + (z & 1)));
              if (last) ptx::mma_commit_pair(bar(B_XEMPTY));
            }
          }
          __syncwarp();
        }
        if (last) ++n;
      }
      if (*abort) {
        if (ptx::elect_one()) ptx::mma_commit_pair(bar(B_TEAR));
        __syncwarp();
        drain_wait(bar(B_TEAR), 0);
      }
    }
  } else if (warp == 3) {
    // the rotary keys, every CTA an even share of the tokens: 8 elements a lane, 4 rows a step
    const int ctas = gridDim.x;
    const int l0 = (int)((long long)p.L * blockIdx.x / ctas), l1 = (int)((long long)p.L * (blockIdx.x + 1) / ctas);
    const int c8 = lane & 7;
    for (int l = l0 + (lane >> 3); l < l1; l += 4) {
      const int page = page_of(l);
      if (page < 0 && c8 == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (page >= 0) {
        const uint8_t* row = reinterpret_cast<const uint8_t*>(p.cache) + ((long long)page * 64 + (l & 63)) * p.row_bytes;
        if (kKind == 1) {
          const uint2 c = *reinterpret_cast<const uint2*>(row + 512 + 8 * c8);
          const uint32_t w[2] = {c.x, c.y};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = e4m3x2_to_f32((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
            o[i] = pack_bf16(f.x * p.cache_scale, f.y * p.cache_scale);
          }
          v = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          v = *reinterpret_cast<const uint4*>(row + (kKind == 0 ? 1024 : 528) + 16 * c8);
        }
      }
      reinterpret_cast<uint4*>(p.k_pe)[(long long)l * 8 + c8] = v;
    }
  } else if (warp < 12) {
    // epilogue: thread = token row; warps 4-7 the keys' 128 columns, 8-11 the values', 32 at a time
    // through 2 KB of staging (64-byte rows, 64-byte swizzle)
    const int quad = warp & 3, what = warp >= 8 ? 1 : 0;
    const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16) + 128 * what;
    const uint32_t stg = base + kOffOut + 2048 * (warp - 4);
    uint8_t* stgp = basep + kOffOut + 2048 * (warp - 4);
    const CUtensorMap* tm = what ? &tm_v : &tm_k;
    const float scale = kKind == 1 ? p.cache_scale : 1.f;
    const uint32_t free0 = lead(B_DFREE);
    uint32_t z = 0;
    for (int u = u0, h = h0, tile = tile0; u < u1; ++u, ++z) {
      const int l = tile * kTile + 128 * rank + 32 * quad;
      if (!__all_sync(0xffffffffu, wait(B_DFULL + (z & 1), (z >> 1) & 1))) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[2][32];
        ptx::tmem_ld32(t_row + 256 * (z & 1) + 64 * half, v[0]);
        ptx::tmem_ld32(t_row + 256 * (z & 1) + 64 * half + 32, v[1]);
        ptx::tmem_wait_ld();
        if (half == 1) {                               // (tensor memory alone was read: no release)
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote_relaxed(free0 + 8 * (z & 1), 0u);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (lane == 0) ptx::bulk_wait_read_all();    // the staging's previous store has read it
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = pack_bf16(__uint_as_float(v[q][8 * j + 2 * i]) * scale,
                               __uint_as_float(v[q][8 * j + 2 * i + 1]) * scale);
            *reinterpret_cast<uint4*>(stgp + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && l < p.L) {
            ptx::tma_store_3d(tm, 64 * half + 32 * q, l, h, stg);
            ptx::bulk_commit();
          }
        }
      }
      if (++h == p.H) {
        h = 0;
        ++tile;
      }
    }
    if (lane == 0) ptx::bulk_wait_all();
  } else if (kKind != 0) {
    // converters: two threads per token row, 32 dims of every chunk each
    const int row = (threadIdx.x - 384) & 127, half = (threadIdx.x - 384) >> 7;
    const uint32_t full0 = lead(B_XFULL);
    uint32_t n = 0;
    bool ok = true;
    for (int u = u0, tile = tile0; ok && u < u1; u = ++tile * p.H, ++n) {
      const int page = page_of(tile * kTile + 128 * rank + (row & 64));
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.cache) +
                           ((long long)(page < 0 ? 0 : page) * 64 + (row & 63)) * p.row_bytes;
      float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
      uint4 code[kChunks][2];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          code[c][i] = page >= 0 ? *reinterpret_cast<const uint4*>(src + 64 * c + 32 * half + 16 * i)
                                 : make_uint4(0u, 0u, 0u, 0u);
      if (kKind == 2 && page >= 0) sc = *reinterpret_cast<const float4*>(src + 512);
      if (!(ok = __all_sync(0xffffffffu, wait(B_XEMPTY, (n & 1) ^ 1)) != 0)) break;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const float s = (c >> 1) == 0 ? sc.x : ((c >> 1) == 1 ? sc.y : ((c >> 1) == 2 ? sc.z : sc.w));
        // rows 0-63 and 64-127 are two tiles of their own, one behind the other: the swizzle runs on
        expand_codes_half_row<kKind == 2, false>(code[c], basep + kOffX + c * kChunk, nullptr, row, half, s);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(full0 + 8 * c);
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();                                 // no copy, arrival or MMA of the pair is on its way
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

template <int kKind>
static cudaError_t run(const CUtensorMap& x, const CUtensorMap& wk, const CUtensorMap& wv, const CUtensorMap& k,
                       const CUtensorMap& v, const Job& job, cudaStream_t s) {
  auto kern = expand_tc_kernel<kKind>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * job.pairs), 1, 1);
  cfg.blockDim = dim3(kThreads<kKind>, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, x, wk, wv, k, v, job);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace expand

bool prefix_expand_tc_supported(const mla_config* c, long long num_pages) {
  return c->act_dtype == MLA_BF16 && c->page_size == 64 && c->d_latent == 512 && c->d_rope == 64 &&
         c->d_nope == 128 && c->d_v == 128 && num_pages * 64 <= 0x7FFFFF00LL;
}

cudaError_t launch_prefix_expand_tc(mla_dtype cache, const PrefixExpandParams& p, cudaStream_t s) {
  using namespace expand;
  Job job;
  job.p = p;
  job.tiles = (p.L + kTile - 1) / kTile;
  const long long units = (long long)p.H * job.tiles;
  const int most = device_sms() / 2 > 0 ? device_sms() / 2 : 1;
  job.pairs = (int)(units < most ? units : most);
  CUtensorMap x, wk, wv, k, v;
  const uint64_t rows = (uint64_t)p.num_pages * 64, H = (uint64_t)p.H, L = (uint64_t)p.L;
  const bool bf = cache == MLA_BF16;
  // (fp8 caches are read by the converters, not through the map)
  if (!tensor_map_3d(&x, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     bf ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, p.cache, 512, rows, 1,
                     (uint64_t)p.row_bytes, rows * p.row_bytes, 64, 64) ||
      !tensor_map_bf16(&wk, p.W_UK, H * 128, 512, 1, H * 256, H * 256 * 512, 64, 64) ||
      !tensor_map_bf16(&wv, p.W_UV, H * 128, 512, 1, H * 256, H * 256 * 512, 64, 64) ||
      !tensor_map_3d(&k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B, p.keys, 128, L, H, 256,
                     L * 256, 32, 32) ||
      !tensor_map_3d(&v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B, p.values, 128, L, H, 256,
                     L * 256, 32, 32))
    return cudaErrorInvalidValue;
  if (bf) return run<0>(x, wk, wv, k, v, job, s);
  if (cache == MLA_FP8_E4M3) return run<1>(x, wk, wv, k, v, job, s);
  return run<2>(x, wk, wv, k, v, job, s);
}

}  // namespace mla
