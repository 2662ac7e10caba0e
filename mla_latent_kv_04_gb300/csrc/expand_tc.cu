// Expansion of a prefix's cached latents into per-head keys and values, on the tensor cores
// (bf16 activations, 64-token pages, d_c 512, d_r 64, d_n = d_v = 128; every cache format).
//
//   keys[h] = C W_UK[:, h],  values[h] = C W_UV[:, h]     (C: L x 512; 128 columns per head)
//
// A pair of CTAs takes a head and 256 tokens at a time, as one MMA over both (cta_group::2, M =
// 256 tokens, N = 256: the head's keys and values): CTA r holds token rows 128 r .. of each
// chunk of 64 dims, and as its half of N the 512 x 128 slice of W_UK (r = 0) or W_UV (r = 1),
// resident in its shared memory (128 KB). So a CTA streams 16 KB for 512 MMA cycles, and its
// MMAs read 64 bytes of shared memory a cycle. (With one
// CTA per 128 x 128 tile and the token chunks multicast to the pair, 8192 tokens took 333 us
// instead of 191: 128 bytes a cycle of operand reads plus the fill are more than shared memory
// gives, and 5 chunks in flight covered half the latency.)
// The accumulators (256 columns) are double-buffered in tensor memory, so that the conversion
// to bf16 and the stores (through shared memory, by TMA, which leaves out rows behind L)
// overlap the next tile's MMAs. The (head, token tile) units in this order are cut into one
// contiguous range per pair.
//
// fp8 caches land as codes; eight converter warps expand them into the bf16 chunk that the
// MMAs read. A per-tensor scale multiplies the fp32 sums (codes are exact in bf16); block
// scales multiply the codes and the product is rounded to bf16, which adds as much error as the
// rounding of the result does.
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
constexpr int kOffW = 0;                               // the weight slice: 8 chunks of 64 x 128
constexpr int kOffOut = kChunks * kChunk;              // 4 KB of output staging per epilogue warp
constexpr int kOffRing = kOffOut + 4 * 4096;
constexpr int kRingBytes = 5 * kChunk;
constexpr int kOffBar = kOffRing + kRingBytes;
constexpr int kSmem = kOffBar + 512 + 1024;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
// bf16: 5 chunks in flight. fp8: 3 expanded chunks and 4 of codes (8 KB).
template <int kKind> struct Ring {
  static constexpr int kTiles = kKind ? 3 : 5;
  static constexpr int kRaw = 4;
  static constexpr int kOffRaw = kOffRing + 3 * kChunk;
  static constexpr int kThreads = kKind ? 512 : 256;
};
constexpr int kConvWarps = 8;
// FULL, WFULL and DFREE are used in the even CTA alone (its MMA thread waits for both CTAs);
// EMPTY, WEMPTY and DFULL in each (the MMAs' commits go to both)
enum { B_FULL = 0, B_EMPTY = 5, B_WFULL = 10, B_WEMPTY = 18, B_DFULL = 26, B_DFREE = 28, B_RAWFULL = 30,
       B_RAWEMPTY = 34, B_TEAR = 38, B_COUNT };

struct Job {
  PrefixExpandParams p;
  int tiles;                                           // token tiles
  int pairs;
};

template <int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Ring<kKind>::kThreads, 1)
    expand_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_wk,
                     const __grid_constant__ CUtensorMap tm_wv, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Job job) {
  using R = Ring<kKind>;
  extern __shared__ uint8_t smem_raw[];
  const PrefixExpandParams& p = job.p;
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + kOffBar + 496);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + kOffBar + 500);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank(), pair = blockIdx.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      int n = 1;
      if (kKind != 0 && i < B_EMPTY) n = 2 * kConvWarps;             // both CTAs' converter warps
      if (i >= B_DFREE && i < B_RAWFULL) n = 8;                      // both CTAs' epilogue warps
      if (i >= B_RAWEMPTY && i < B_TEAR) n = kConvWarps;
      ptx::mbar_init(bar(i), n);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_x);
    ptx::prefetch_tensormap(rank ? &tm_wv : &tm_wk);
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
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
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  // the even CTA's barriers, as an address that both CTAs can signal
  auto lead = [&](int i) { return ptx::map_to_rank(bar(i), 0u); };
  const int units = p.H * job.tiles;
  const int u0 = (int)((long long)units * pair / job.pairs), u1 = (int)((long long)units * (pair + 1) / job.pairs);
  const int h0 = u0 / job.tiles, tile0 = u0 % job.tiles;
  // the page that holds token l (a multiple of 64): -1 behind the prefix or with a bad id
  auto page_of = [&](int l) {
    if (l >= p.L) return -1;
    const int page = p.table[l >> 6];
    return page >= 0 && page < p.num_pages ? page : -1;
  };

  if (warp == 0) {
    if (lane == 0) {                                   // this CTA's token rows of every chunk
      constexpr uint32_t kSlots = kKind ? R::kRaw : R::kTiles, kBytes = kKind ? kChunk / 2 : kChunk;
      constexpr uint32_t kOff = kKind ? R::kOffRaw : kOffRing;
      constexpr int kEmptyBar = kKind ? B_RAWEMPTY : B_EMPTY;
      uint32_t g = 0;
      bool ok = true;
      int page[2] = {page_of(tile0 * kTile + 128 * rank), page_of(tile0 * kTile + 128 * rank + 64)};
      for (int u = u0, tile = tile0; ok && u < u1; ++u) {
        // rows out of the tensor's range read as zero
        const int y0 = (page[0] >= 0 ? page[0] : p.num_pages) * 64, y1 = (page[1] >= 0 ? page[1] : p.num_pages) * 64;
        if (++tile == job.tiles) tile = 0;
        for (int c = 0; c < kChunks; ++c, ++g) {
          const uint32_t st = g % kSlots;
          if (!(ok = wait(kEmptyBar + st, ((g / kSlots) & 1) ^ 1))) break;
          const uint32_t dst = base + kOff + st * kBytes;
          if (kKind == 0) {
            const uint32_t full = lead(B_FULL + st);
            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_FULL + st), 2 * kBytes);
            ptx::tma_load_3d_pair(dst, &tm_x, 64 * c, y0, 0, full);
            ptx::tma_load_3d_pair(dst + kBytes / 2, &tm_x, 64 * c, y1, 0, full);
          } else {
            ptx::mbar_arrive_expect_tx(bar(B_RAWFULL + st), kBytes);
            ptx::tma_load_3d(dst, &tm_x, 64 * c, y0, 0, bar(B_RAWFULL + st));
            ptx::tma_load_3d(dst + kBytes / 2, &tm_x, 64 * c, y1, 0, bar(B_RAWFULL + st));
          }
          if (c == 0) {                                // the next tile's pages, ahead of need
            page[0] = page_of(tile * kTile + 128 * rank);
            page[1] = page_of(tile * kTile + 128 * rank + 64);
          }
        }
      }
      if (*abort && (kKind != 0 || rank == 0))
        for (uint32_t i = g > kSlots ? g - kSlots : 0; i < g; ++i)
          drain_wait(bar((kKind ? B_RAWFULL : B_FULL) + i % kSlots), (i / kSlots) & 1);
    }
  } else if (warp == 2) {
    if (lane == 0) {                                   // the weight slice, when the head changes
      uint32_t n = 0;
      bool ok = true;
      for (int u = u0, h = h0; ok && u < u1; u = ++h * job.tiles, ++n) {
        for (int c = 0; c < kChunks; ++c) {
          if (!(ok = wait(B_WEMPTY + c, (n & 1) ^ 1))) break;
          const uint32_t dst = base + kOffW + c * kChunk, full = lead(B_WFULL + c);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_WFULL + c), 2 * kChunk);
          ptx::tma_load_3d_pair(dst, rank ? &tm_wv : &tm_wk, h * 128, 64 * c, 0, full);
          ptx::tma_load_3d_pair(dst + kChunk / 2, rank ? &tm_wv : &tm_wk, h * 128 + 64, 64 * c, 0, full);
        }
      }
      if (*abort && n && rank == 0)
        for (int c = 0; c < kChunks; ++c) drain_wait(bar(B_WFULL + c), (n - 1) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(256, 256, false, true);
      uint32_t g = 0, z = 0, n = 0;
      bool ok = true;
      for (int u = u0, tile = tile0; ok && u < u1; ++u, ++z) {
        const bool first = u == u0 || tile == 0;
        const bool last = u + 1 == u1 || tile + 1 == job.tiles;
        if (++tile == job.tiles) tile = 0;
        if (!(ok = bounded_wait<true>(bar(B_DFREE + (z & 1)), ((z >> 1) & 1) ^ 1, abort, p.status))) break;
        for (int c = 0; c < kChunks; ++c, ++g) {
          const uint32_t st = g % R::kTiles;
          if (first && !(ok = wait(B_WFULL + c, n & 1))) break;
          if (!(ok = bounded_wait<kKind != 0>(bar(B_FULL + st), (g / R::kTiles) & 1, abort, p.status))) break;
          ptx::tc_fence_after();
          const uint32_t x = base + kOffRing + st * kChunk, w = base + kOffW + c * kChunk;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::mma_bf16_ss_pair(tmem + 256 * (z & 1), ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                                  ptx::smem_desc(w + 2048 * k, kChunk / 2, 1024, ptx::kSwizzle128), kIdesc,
                                  (c || k) ? 1u : 0u);
          ptx::mma_commit_pair(bar(B_EMPTY + st));
          if (last) ptx::mma_commit_pair(bar(B_WEMPTY + c));
        }
        if (!ok) break;
        ptx::mma_commit_pair(bar(B_DFULL + (z & 1)));
        if (last) ++n;
      }
      if (*abort) {
        ptx::mma_commit_pair(bar(B_TEAR));
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
  } else if (warp < 8) {
    // epilogue: thread = token row; 64 columns at a time through 4 KB of staging
    const int quad = warp & 3, row = lane;
    const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t stg = base + kOffOut + 4096 * quad;
    uint8_t* stgp = basep + kOffOut + 4096 * quad;
    const float scale = kKind == 1 ? p.cache_scale : 1.f;
    const uint32_t free0 = lead(B_DFREE);
    uint32_t z = 0;
    for (int u = u0, h = h0, tile = tile0; u < u1; ++u, ++z) {
      const int l = tile * kTile + 128 * rank + 32 * quad;
      if (!__all_sync(0xffffffffu, wait(B_DFULL + (z & 1), (z >> 1) & 1))) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int part = 0; part < 4; ++part) {           // keys 0-63, 64-127, values 0-63, 64-127
        uint32_t a[32], b[32];
        ptx::tmem_ld32(t_row + 256 * (z & 1) + 64 * part, a);
        ptx::tmem_ld32(t_row + 256 * (z & 1) + 64 * part + 32, b);
        ptx::tmem_wait_ld();
        if (part == 3) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote(free0 + 8 * (z & 1));
        }
        if (lane == 0) ptx::bulk_wait_read_all();      // the staging's previous store has read it
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t* s = j < 4 ? a + 8 * j : b + 8 * (j - 4);
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack_bf16(__uint_as_float(s[2 * i]) * scale, __uint_as_float(s[2 * i + 1]) * scale);
          *reinterpret_cast<uint4*>(stgp + row * 128 + ((j ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && l < p.L) {
          ptx::tma_store_3d(part < 2 ? &tm_k : &tm_v, 64 * (part & 1), l, h, stg);
          ptx::bulk_commit();
        }
      }
      if (++tile == job.tiles) {
        tile = 0;
        ++h;
      }
    }
    if (lane == 0) ptx::bulk_wait_all();
  } else if (kKind != 0) {
    // converters: two threads per token row of the chunk, 32 dims each
    const int row = (threadIdx.x - 256) & 127, half = (threadIdx.x - 256) >> 7;
    const uint32_t full0 = lead(B_FULL);
    uint32_t g = 0;
    bool ok = true;
    for (int u = u0, tile = tile0; ok && u < u1; ++u) {
      float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (kKind == 2) {
        const int page = page_of(tile * kTile + 128 * rank + (row & 64));
        if (page >= 0)
          sc = *reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(p.cache) +
                                                ((long long)page * 64 + (row & 63)) * p.row_bytes + 512);
      }
      if (++tile == job.tiles) tile = 0;
      for (int c = 0; c < kChunks; ++c, ++g) {
        const uint32_t rs = g % R::kRaw, st = g % R::kTiles;
        if (!(ok = __all_sync(0xffffffffu, wait(B_RAWFULL + rs, (g / R::kRaw) & 1)) != 0)) break;
        if (!(ok = __all_sync(0xffffffffu, wait(B_EMPTY + st, ((g / R::kTiles) & 1) ^ 1)) != 0)) break;
        const float s = (c >> 1) == 0 ? sc.x : ((c >> 1) == 1 ? sc.y : ((c >> 1) == 2 ? sc.z : sc.w));
        // rows 0-63 and 64-127 are two tiles of their own, one behind the other: the swizzle runs on
        expand_codes_half_row<kKind == 2, false>(basep + R::kOffRaw + rs * (kChunk / 2),
                                                 basep + kOffRing + st * kChunk, nullptr, row, half, s);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive_remote(full0 + 8 * st);
          ptx::mbar_arrive(bar(B_RAWEMPTY + rs));
        }
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
  kern<<<2 * job.pairs, Ring<kKind>::kThreads, kSmem, s>>>(x, wk, wv, k, v, job);
  note_launch();
  return cudaGetLastError();
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
  if (!tensor_map_3d(&x, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     bf ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, p.cache, 512, rows, 1,
                     (uint64_t)p.row_bytes, rows * p.row_bytes, 64, 64) ||
      !tensor_map_bf16(&wk, p.W_UK, H * 128, 512, 1, H * 256, H * 256 * 512, 64, 64) ||
      !tensor_map_bf16(&wv, p.W_UV, H * 128, 512, 1, H * 256, H * 256 * 512, 64, 64) ||
      !tensor_map_bf16(&k, p.keys, 128, L, H, 256, L * 256, 64, 32) ||
      !tensor_map_bf16(&v, p.values, 128, L, H, 256, L * 256, 64, 32))
    return cudaErrorInvalidValue;
  if (bf) return run<0>(x, wk, wv, k, v, job, s);
  if (cache == MLA_FP8_E4M3) return run<1>(x, wk, wv, k, v, job, s);
  return run<2>(x, wk, wv, k, v, job, s);
}

}  // namespace mla
