// Expansion of a prefix's cached latents into per-head keys and values, on the tensor cores
// (bf16 activations, 64-token pages, d_c 512, d_r 64, d_n = d_v = 128; every cache format).
//
//   keys[h] = C W_UK[:, h],  values[h] = C W_UV[:, h]     (C: L x 512; 128 columns per head)
//
// A pair of CTAs takes 256 tokens at a time and goes through heads, a head's keys and then its
// values each as one MMA sequence over both CTAs (cta_group::2, M = 256 tokens, N = 128, K =
// 512). CTA r holds token rows 128 r .. of the tile, all 512 dims of them, in tensor memory (256
// columns, the A operand), and streams half of the N: 64 columns of the weight slice, 16 KB for
// every 128 dims and 512 MMA cycles, through a ring of 11 such chunks. The accumulators (128
// columns) are double-buffered in the rest of tensor memory, so that the conversion to bf16 and
// the stores (through shared memory, by TMA, which leaves out rows behind L) overlap the next
// MMAs.
//
// Why so: shared memory gives 128 bytes a cycle. With the tokens resident there as well, operands
// (64), weight fill (32) and results (32, in and out of the staging) took all of it, and 8192
// tokens took 189 us (126 without the stores); now the operands take 32. Chunks of 64 dims cost
// 197: a chunk's wait, commit and four MMA issues took longer than its 256 MMA cycles. One CTA per
// 128 x 128 tile with multicast token chunks took 333 us, clusters of two pairs that share the
// weights by multicast 205 (36 of them fit, not 38).
//
// Tokens come straight from the cache's rows, by eight warps, when the pair turns to a tile: bf16
// as they are, fp8 codes expanded once for all heads. A per-tensor scale multiplies the fp32 sums
// (codes are exact in bf16); block scales multiply the codes and the product is rounded to bf16,
// which adds as much error as the rounding of the result does.
//
// Bound: the MMAs (4096 cycles for 256 tokens and a head on two SMs): 8192 tokens take 165 to 175 us
// in a graph of such calls (1570 to 1670 TFLOP/s, as the power cap lets it), a call by itself 184.
#include "fp8_tiles.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace expand {

constexpr int kTile = 256, kChunks = 4;                // tokens of a pair's tile; chunks of 128 dims
constexpr int kChunk = 128 * 64 * 2;                   // 128 dims x 64 weight columns: 16 KB
constexpr int kRing = 11;
constexpr int kOffOut = kRing * kChunk;                // 2 x 2 KB of output staging per epilogue warp
constexpr int kOffBar = kOffOut + 8 * 4096;
constexpr int kSmem = kOffBar + 512 + 1024;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kThreads = 640;                          // 4 + 8 epilogue + 8 token-loading warps
constexpr uint32_t kColX = 256;                        // D: two buffers of 128, then the tokens
// WFULL, XFULL and DFREE are used in the even CTA alone (its MMA warp waits for both CTAs); WEMPTY,
// XEMPTY and DFULL in each (the MMAs' commits go to both)
enum { B_WFULL = 0, B_WEMPTY = kRing, B_XFULL = 2 * kRing, B_XEMPTY, B_DFULL, B_DFREE = B_DFULL + 2,
       B_TEAR = B_DFREE + 2, B_COUNT };
static_assert(B_COUNT * 8 <= 480, "barrier area");

struct Job {
  PrefixExpandParams p;
  int tiles;                                           // token tiles
  int pairs;
  int head_block;                                      // heads of a block (see Units)
};

// The (head, token tile) units in the order that the pairs' ranges cut: heads in blocks, in a block
// the tiles, in a tile the block's heads. With a bf16 cache and ranges of many heads a block is
// about a range: pairs that run at the same time are then near the same head, on different
// tiles, and read the same weights at about the same time (worth 4% at 8192 tokens).
// Otherwise a block is all heads: a pair changes its tile as seldom as can be.
struct Units {
  int H, tiles, block;
  int h, tile, h0, h1;                                 // the current unit; its block's heads
  __device__ Units(const Job& j, int u) : H(j.p.H), tiles(j.tiles), block(j.head_block) {
    const int per = tiles * block;
    h0 = u / per * block;
    h1 = min(H, h0 + block);
    const int in = u - h0 * tiles;
    tile = in / (h1 - h0);
    h = h0 + in % (h1 - h0);
  }
  __device__ bool row_start() const { return h == h0; }
  __device__ bool row_end() const { return h == h1 - 1; }
  __device__ void next() {
    if (++h < h1) return;
    h = h0;
    if (++tile < tiles) return;
    tile = 0;
    h = h0 = h1;
    h1 = min(H, h0 + block);
  }
};

// kKind: 0 bf16 cache, 1 e4m3 with one scale, 2 e4m3 with block scales
template <int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expand_tc_kernel(const __grid_constant__ CUtensorMap tm_wk, const __grid_constant__ CUtensorMap tm_wv,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const Job job) {
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
      if (i == B_XFULL) n = 16;                        // both CTAs' loading warps
      if (i >= B_DFREE && i < B_TEAR) n = 16;          // both CTAs' epilogue warps
      ptx::mbar_init(bar(i), n);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_wk);
    ptx::prefetch_tensormap(&tm_wv);
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
    return __all_sync(0xffffffffu, wait(i, parity)) != 0;
  };
  auto wait_lead = [&](int i, uint32_t parity) {       // for what the other CTA's threads arrived on
    return __all_sync(0xffffffffu, bounded_wait<true>(bar(i), parity, abort, p.status)) != 0;
  };
  // the even CTA's barriers, as an address that both CTAs can signal
  auto lead = [&](int i) { return ptx::map_to_rank(bar(i), 0u); };
  const int units = p.H * job.tiles;
  const int u0 = (int)((long long)units * pair / job.pairs), u1 = (int)((long long)units * (pair + 1) / job.pairs);
  // the page that holds token l: -1 behind the prefix or with a bad id
  auto page_of = [&](int l) {
    if (l >= p.L) return -1;
    const int page = p.table[l >> 6];
    return page >= 0 && page < p.num_pages ? page : -1;
  };

  if (warp == 0) {
    if (lane == 0) {                                   // this CTA's columns of every weight chunk
      uint32_t g = 0, st = 0, wrap = 0;
      bool ok = true;
      Units it(job, u0);
      for (int u = u0; ok && u < u1; ++u, it.next()) {
        const int x = it.h * 128 + 64 * rank;
        for (int i = 0; i < 2 * kChunks; ++i, ++g) {   // the keys' chunks, the values'
          if (!(ok = wait(B_WEMPTY + st, (wrap & 1) ^ 1))) break;
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_WFULL + st), 2 * kChunk);
          ptx::tma_load_3d_pair(base + st * kChunk, i < kChunks ? &tm_wk : &tm_wv, x, 128 * (i % kChunks), 0,
                                lead(B_WFULL + st));
          if (++st == kRing) {
            st = 0;
            ++wrap;
          }
        }
      }
      if (*abort && rank == 0)
        for (uint32_t i = g > kRing ? g - kRing : 0; i < g; ++i)
          drain_wait(bar(B_WFULL + i % kRing), (i / kRing) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(256, 128, false, true);
      uint32_t st = 0, wrap = 0, z = 0, n = 0;
      bool ok = true;
      Units it(job, u0);
      for (int u = u0; ok && u < u1; ++u, it.next()) {
        const bool first = u == u0 || it.row_start(), last = u + 1 == u1 || it.row_end();
        if (first && !(ok = wait_lead(B_XFULL, n++ & 1))) break;
        for (int kv = 0; ok && kv < 2; ++kv, ++z) {
          if (!(ok = wait_lead(B_DFREE + (z & 1), ((z >> 1) & 1) ^ 1))) break;
          for (int c = 0; c < kChunks; ++c) {
            if (!(ok = wait_w(B_WFULL + st, wrap & 1))) break;
            ptx::tc_fence_after();
            const uint32_t w = base + st * kChunk;
            if (ptx::elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                ptx::mma_bf16_ts_pair(tmem + 128 * (z & 1), tmem + kColX + 64 * c + 8 * k,
                                      ptx::smem_desc(w + 2048 * k, kChunk, 1024, ptx::kSwizzle128), kIdesc,
                                      (c || k) ? 1u : 0u);
              ptx::mma_commit_pair(bar(B_WEMPTY + st));
              if (c == kChunks - 1) {
                ptx::mma_commit_pair(bar(B_DFULL + (z & 1)));
                if (last && kv) ptx::mma_commit_pair(bar(B_XEMPTY));
              }
            }
            __syncwarp();
            if (++st == kRing) {
              st = 0;
              ++wrap;
            }
          }
        }
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
  } else if (warp >= 4 && warp < 12) {
    // epilogue: thread = token row, columns 64 part .., 32 at a time through two 2 KB buffers of
    // staging (64-byte rows, 64-byte swizzle)
    const int quad = warp & 3, part = warp >= 8 ? 1 : 0;
    const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16) + 64 * part;
    const uint32_t stg = base + kOffOut + 4096 * (warp - 4);
    uint8_t* stgp = basep + kOffOut + 4096 * (warp - 4);
    const float scale = kKind == 1 ? p.cache_scale : 1.f;
    const uint32_t free0 = lead(B_DFREE);
    uint32_t z = 0;
    bool ok = true;
    Units it(job, u0);
    for (int u = u0; ok && u < u1; ++u, it.next()) {
      const int l = it.tile * kTile + 128 * rank + 32 * quad;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++z) {
        if (!(ok = wait_w(B_DFULL + (z & 1), (z >> 1) & 1))) break;
        ptx::tc_fence_after();
        uint32_t v[2][32];
        ptx::tmem_ld32(t_row + 128 * (z & 1), v[0]);
        ptx::tmem_ld32(t_row + 128 * (z & 1) + 32, v[1]);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote_relaxed(free0 + 8 * (z & 1));   // (only tensor memory was read)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (lane == 0) ptx::bulk_wait_read_le1();    // this buffer's last store has read it
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = pack_bf16(__uint_as_float(v[q][8 * j + 2 * i]) * scale,
                               __uint_as_float(v[q][8 * j + 2 * i + 1]) * scale);
            *reinterpret_cast<uint4*>(stgp + 2048 * q + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (l < p.L) ptx::tma_store_3d(kv ? &tm_v : &tm_k, 64 * part + 32 * q, l, it.h, stg + 2048 * q);
            ptx::bulk_commit();
          }
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_all();
  } else if (warp >= 12) {
    // the pair's tokens into tensor memory: two threads per row, 256 dims each, 64 at a time
    const int t = threadIdx.x - 384, quad = warp & 3, row = 32 * quad + lane, half = t >> 7;
    const uint32_t t_x = tmem + ((uint32_t)(32 * quad) << 16) + kColX + 128 * half;
    const uint32_t full = lead(B_XFULL);
    constexpr int kVecs = kKind ? 4 : 8;               // 16-byte loads for 64 dims
    uint32_t n = 0;
    bool ok = true;
    Units it(job, u0);
    for (int u = u0; ok && u < u1; ++u, it.next()) {
      if (u != u0 && !it.row_start()) continue;
      // a warp's 32 tokens lie on one page, so that its lanes go one way to the warp-wide stores below
      // (rows behind the prefix, on its last page, are not written out)
      const int l = it.tile * kTile + 128 * rank + row, page = page_of(l - lane);
      const uint8_t* row_p = reinterpret_cast<const uint8_t*>(p.cache) +
                             ((long long)(page < 0 ? 0 : page) * 64 + (l & 63)) * p.row_bytes;
      const uint4* src = reinterpret_cast<const uint4*>(row_p + (kKind ? 256 : 512) * half);
      uint4 cur[kVecs], nxt[kVecs];
      float2 sc = make_float2(0.f, 0.f);
      auto load = [&](uint4 (&v)[kVecs], int b) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = page >= 0 ? src[kVecs * b + i] : make_uint4(0u, 0u, 0u, 0u);
      };
      load(cur, 0);
      if (kKind == 2 && page >= 0) sc = *reinterpret_cast<const float2*>(row_p + 512 + 8 * half);
      if (!(ok = wait_w(B_XEMPTY, (n & 1) ^ 1))) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b < 3) load(nxt, b + 1);
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kKind == 0) {
              o[4 * i + j] = w[j];
            } else {
              const float s = kKind == 2 ? (b < 2 ? sc.x : sc.y) : 1.f;
              const float2 f0 = e4m3x2_to_f32(w[j] & 0xFFFFu), f1 = e4m3x2_to_f32(w[j] >> 16);
              o[(8 * i + 2 * j) % 32] = pack_bf16(f0.x * s, f0.y * s);
              o[(8 * i + 2 * j + 1) % 32] = pack_bf16(f1.x * s, f1.y * s);
            }
          }
        }
        ptx::tmem_st32(t_x + 32 * b, o);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) cur[i] = nxt[i];
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote_relaxed(full);      // (only tensor memory was written)
      ++n;
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
static cudaError_t run(const CUtensorMap& wk, const CUtensorMap& wv, const CUtensorMap& k, const CUtensorMap& v,
                       Job job, cudaStream_t s) {
  auto kern = expand_tc_kernel<kKind>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  job.tiles = (job.p.L + kTile - 1) / kTile;
  const long long units = (long long)job.p.H * job.tiles;
  const int most = device_sms() / 2 > 0 ? device_sms() / 2 : 1;
  job.pairs = (int)(units < most ? units : most);
  const int range = (int)((units + job.pairs - 1) / job.pairs), rows = (range + job.p.H - 1) / job.p.H;
  job.head_block = kKind == 0 && range >= 32 ? (range + rows - 1) / rows : job.p.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * job.pairs), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, wk, wv, k, v, job);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace expand

bool prefix_expand_tc_supported(const mla_config* c) {
  return c->act_dtype == MLA_BF16 && c->page_size == 64 && c->d_latent == 512 && c->d_rope == 64 &&
         c->d_nope == 128 && c->d_v == 128;
}

cudaError_t launch_prefix_expand_tc(mla_dtype cache, const PrefixExpandParams& p, cudaStream_t s) {
  using namespace expand;
  Job job{};
  job.p = p;
  CUtensorMap wk, wv, k, v;
  const uint64_t H = (uint64_t)p.H, L = (uint64_t)p.L;
  if (!tensor_map_bf16(&wk, p.W_UK, H * 128, 512, 1, H * 256, H * 256 * 512, 64, 128) ||
      !tensor_map_bf16(&wv, p.W_UV, H * 128, 512, 1, H * 256, H * 256 * 512, 64, 128) ||
      !tensor_map_3d(&k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B, p.keys, 128, L, H, 256,
                     L * 256, 32, 32) ||
      !tensor_map_3d(&v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B, p.values, 128, L, H, 256,
                     L * 256, 32, 32))
    return cudaErrorInvalidValue;
  if (cache == MLA_BF16) return run<0>(wk, wv, k, v, job, s);
  return cache == MLA_FP8_E4M3 ? run<1>(wk, wv, k, v, job, s) : run<2>(wk, wv, k, v, job, s);
}

}  // namespace mla
