// Page scores on the tensor cores (bf16, d_c 512, d_r 64, up to 128 heads).
//
//   Z = q_lat K^T (M = heads, N = 128 pages, K = 576),  score_p = m_p sum_h 2^(c Z_hp) / L_h,
//   L_h = sum_p m_p 2^(c Z_hp),   c = softmax scale * log2 e, m_p the tokens of page p that the query sees.
// A cluster of up to 16 CTAs takes one query token; each CTA computes up to four tiles of 128 pages and
// keeps them in tensor memory (512 columns), so that nothing but the heads' maxima and sums, which the
// CTAs exchange through distributed shared memory, stands between the product and the scores. A head is
// a lane of tensor memory: its maximum and sum are a thread's own; the sum over heads is a butterfly of
// shuffles that leaves each lane one page. The pages' rows lie wherever the block table puts them: 256
// threads copy them 16 bytes at a time (cp.async), which takes 2 us a tile; gathered by the TMA, four rows
// an instruction, they took 8.
//
// Bound: latency of a tile's load and of the exchange, not bytes: 32 requests of 512 pages 10.6 us among calls
// (24 MB, which the copy rate moves in 3.5), 4 requests of 512 to 2048 pages with 2 query tokens each 15.3.
#include <math.h>

#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace pscore {

constexpr int kD = 576, kChunks = 9, kTile = 128;
constexpr int kTiles = 4;                      // of a CTA
constexpr int kMaxCluster = 16;                // above 8: where the GPU places such a cluster
constexpr int kChunk = 128 * 64 * 2;
constexpr int kStages = 4;
constexpr int kOffRing = kChunks * kChunk;     // the query first
constexpr int kOffCount = kOffRing + kStages * kChunk;     // [kTiles][128] tokens seen of each page
constexpr int kOffStat = kOffCount + kTiles * kTile * 4;   // [2][128] maxima and sums of the two column halves
constexpr int kOffHead = kOffStat + 2 * 128 * 8;           // [128] this CTA's (other CTAs read it)
constexpr int kOffBar = kOffHead + 128 * 8;
constexpr int kSmem = kOffBar + 128 + 1024;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kThreads = 320;
enum { B_FULL = 0, B_EMPTY = kStages, B_QFULL = 2 * kStages, B_ZFULL, B_TEAR = B_ZFULL + kTiles, B_COUNT };

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    page_scores_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const PageScoreParams p, int C) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + kOffBar + 8 * B_COUNT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + kOffBar + 8 * B_COUNT + 4);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = blockIdx.x / C, rank = blockIdx.x % C, b = g / p.q_len;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) ptx::mbar_init(bar(i), i < B_EMPTY ? 8 : 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_q);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int S = p.seq_lens[b];
  const bool bad = S < 0 || (S > 0 && S < p.q_len) || S > (long long)p.max_pages * 64;
  if (bad && rank == 0 && threadIdx.x == 0 && g % p.q_len == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  const int see = bad || S == 0 ? 0 : S - p.q_len + g % p.q_len + 1;
  const int pages = (see + 63) / 64, tiles = (pages + kTile - 1) / kTile;
  const int mine = tiles > rank ? (tiles - rank + C - 1) / C : 0;          // tiles rank, rank + C, ..
  // tokens seen of every page of these tiles (0: none, or a bad id), and the ids for the gathering warp
  float* count = reinterpret_cast<float*>(basep + kOffCount);
  const int32_t* bt = p.block_table + (long long)b * p.max_pages;
  for (int i = threadIdx.x; i < mine * kTile; i += kThreads) {
    const int pg = (rank + i / kTile * C) * kTile + i % kTile;
    float n = 0.f;
    if (pg < pages) {
      const int page = bt[pg];
      if (page >= 0 && page < p.num_pages) n = (float)min(64, see - pg * 64);
      else flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    }
    count[i] = n;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const uint64_t limit = p.test.limit_ns;
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status, limit); };
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  float2* head = reinterpret_cast<float2*>(basep + kOffHead);
  float* part = reinterpret_cast<float*>(basep + kOffRing);                // [4][kTiles][128], after the products
  const int quad = warp & 3, half = warp >= 6 ? 1 : 0, row = 32 * quad + lane;
  const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16) + 64 * half;
  float m = -INFINITY, l = 0.f;
  bool ok = true;

  if (warp == 0) {
    if (mine > 0) {
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(bar(B_QFULL), kChunks * p.H * 128);
        for (int c = 0; c < kChunks; ++c) ptx::tma_load_3d(base + c * kChunk, &tm_q, 64 * c, 0, g, bar(B_QFULL));
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    if (mine > 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(128, kTile, false, false);
      const uint64_t qd = ptx::smem_desc(base, 16, 1024, ptx::kSwizzle128);
      const uint64_t kd = ptx::smem_desc(base + kOffRing, 16, 1024, ptx::kSwizzle128);
      uint32_t st = 0, phase = 0;
      ok = wait_w(B_QFULL, 0);
      for (int i = 0; ok && i < mine; ++i) {
        for (int c = 0; c < kChunks; ++c) {
          if (!(ok = wait_w(B_FULL + st, phase))) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_bf16_ss(tmem + kTile * i, qd + (c * (kChunk >> 4) + 2 * k), kd + (st * (kChunk >> 4) + 2 * k), idesc,
                               k ? 1u : (c ? 1u : 0u));
            ptx::mma_commit(bar(B_EMPTY + st));
            if (c == kChunks - 1) ptx::mma_commit(bar(B_ZFULL + i));
          }
          __syncwarp();
          if (++st == kStages) {
            st = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort) {
        if (ptx::elect_one()) ptx::mma_commit(bar(B_TEAR));
        __syncwarp();
        drain_wait(bar(B_TEAR), 0, limit);
        drain_wait(bar(B_QFULL), 0, limit);
      }
    }
  } else {
    // the pages' rows, a chunk of 64 dims at a time, kStages - 1 chunks ahead of the one handed over: eight
    // threads a row, rows tid / 8 + 32 j. Behind the pages, or for a bad id, any row (its count is 0)
    const int tid = threadIdx.x - 64, unit = tid & 7, r0 = tid >> 3, total = mine * kChunks;
    const uint8_t* src[4];
    for (int n = 0; ok && n < total + kStages - 1; ++n) {
      const int c = n % kChunks;
      if (n < total) {
        if (c == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int pg = (rank + n / kChunks * C) * kTile + r0 + 32 * j;
            const int page = pg < pages ? bt[pg] : 0;
            src[j] = reinterpret_cast<const uint8_t*>(p.page_keys) +
                     (long long)(page >= 0 && page < p.num_pages ? page : 0) * (kD * 2) + 16 * unit;
          }
        }
        const uint32_t st = n % kStages;
        if (!(ok = wait_w(B_EMPTY + st, ((n / kStages) & 1) ^ 1))) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + 32 * j;
          cp_async16(base + kOffRing + st * kChunk + r * 128 + ((unit ^ (r & 7)) << 4), src[j] + 128 * c);
        }
      }
      cp_async_commit();
      if (n >= kStages - 1) {
        cp_async_wait<kStages - 1>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && (blockIdx.x != 0 || n - kStages + 1 != p.test.withhold - 1))
          ptx::mbar_arrive(bar(B_FULL + (n - kStages + 1) % kStages));
      }
    }
    cp_async_wait<0>();
    // a head's maximum and sum over 64 columns of every tile
    for (int i = 0; ok && i < mine; ++i) {
      if (!(ok = wait_w(B_ZFULL + i, 0))) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t v[32];
        ptx::tmem_ld32(t_row + kTile * i + c0, v);
        ptx::tmem_wait_ld();
        const float* n = count + i * kTile + 64 * half + c0;
        float top = m;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float z = n[j] > 0.f ? __uint_as_float(v[j]) * p.scale_log2 : -INFINITY;
          v[j] = __float_as_uint(z);
          top = fmaxf(top, z);
        }
        if (top > -INFINITY) {
          l *= ptx::ex2(m - top);              // (no column yet: l is 0)
          m = top;
        }
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float z = __uint_as_float(v[j]);
          s = fmaf(z == -INFINITY ? 0.f : ptx::ex2(z - m), n[j], s);
        }
        l += s;
        __syncwarp();                          // the next load is warp-wide
      }
    }
    reinterpret_cast<float2*>(basep + kOffStat)[128 * half + row] = make_float2(m, l);
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x < 128) {                     // both halves' columns
    const float2* stat = reinterpret_cast<const float2*>(basep + kOffStat);
    const float2 x = stat[threadIdx.x], y = stat[128 + threadIdx.x];
    const float top = fmaxf(x.x, y.x);
    head[threadIdx.x] = make_float2(top, (x.y > 0.f || x.y != x.y ? x.y * ptx::ex2(x.x - top) : 0.f) +
                                             (y.y > 0.f || y.y != y.y ? y.y * ptx::ex2(y.x - top) : 0.f));
  }
  __syncwarp();
  if (C > 1) ptx::cluster_sync();
  else __syncthreads();
  if (warp == 0 && C > 1) {                    // a CTA that gave up has no sums to share: nobody writes
    const uint32_t at = ptx::map_to_rank(ptx::smem_u32(const_cast<int*>(abort)), (uint32_t)(lane < C ? lane : 0));
    if (__any_sync(0xffffffffu, ptx::ld_dsmem_u32(at) != 0) && lane == 0) *abort = 1;
    __syncwarp();
  }
  if (warp >= 2) {
    // the head's over the cluster, in order of ranks
    float top = -INFINITY, sum = 0.f;
    if (C > 1) {
      float mm[kMaxCluster], ll[kMaxCluster];
      const uint32_t at = ptx::smem_u32(&head[row]);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        mm[r] = -INFINITY;
        ll[r] = 0.f;
        if (r < C) {
          const uint32_t a = ptx::map_to_rank(at, (uint32_t)r);
          mm[r] = ptx::ld_dsmem_f32(a);
          ll[r] = ptx::ld_dsmem_f32(a + 4);
        }
        top = fmaxf(top, mm[r]);
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (ll[r] != 0.f) sum = fmaf(ll[r], ptx::ex2(mm[r] - top), sum);
    } else {
      top = head[row].x;
      sum = head[row].y;
    }
    // NaN scores reach the sum (a maximum leaves them out); no page at all: weights of 0
    const float lse2 = sum == 0.f ? INFINITY : top + log2f(sum);
    for (int i = 0; i < mine && ok; ++i) {
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t v[32];
        ptx::tmem_ld32(t_row + kTile * i + c0, v);
        ptx::tmem_wait_ld();
        const float* n = count + i * kTile + 64 * half + c0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float e = ptx::ex2(fmaf(__uint_as_float(v[j]), p.scale_log2, -lse2)) * n[j];
          v[j] = __float_as_uint(row < p.H && n[j] > 0.f ? e : 0.f);
        }
        // sums over the warp's heads: lane j is left with column j
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int j = 0; j < o; ++j) {
            const uint32_t give = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
            v[j] = __float_as_uint(__uint_as_float(keep) + __uint_as_float(__shfl_xor_sync(0xffffffffu, give, o)));
          }
        }
        part[(quad * kTiles + i) * kTile + 64 * half + c0 + lane] = __uint_as_float(v[0]);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (!*abort) {
    float* out = p.scores + (long long)g * p.max_pages;
    for (int i = threadIdx.x; i < mine * kTile; i += kThreads) {
      const int pg = (rank + i / kTile * C) * kTile + i % kTile;
      if (pg < pages)
        out[pg] = (part[i] + part[kTiles * kTile + i]) + (part[2 * kTiles * kTile + i] + part[3 * kTiles * kTile + i]);
    }
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (C > 1) ptx::cluster_sync();              // the others have read this CTA's heads
}

}  // namespace pscore

using namespace pscore;

// The largest cluster that this GPU places, 8 or 16 CTAs (a GPC has to have room for one CTA an SM).
static int largest_cluster() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
  if (!cached[dev]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kMaxCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok =
        cudaFuncSetAttribute(page_scores_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
        cudaFuncSetAttribute(page_scores_tc_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, page_scores_tc_kernel, &cfg) == cudaSuccess && n > 0;
    if (!ok) (void)cudaGetLastError();
    cached[dev] = ok ? kMaxCluster : 8;
  }
  return cached[dev];
}

bool page_scores_tc_supported(const mla_config* c, int num_pages, int max_pages) {
  const int tiles = (max_pages + kTile - 1) / kTile;
  return c->act_dtype == MLA_BF16 && c->page_size == 64 && c->d_latent == 512 && c->d_rope == 64 &&
         c->num_heads <= 128 && num_pages > 0 &&
         (tiles <= kTiles * 8 || (tiles <= kTiles * kMaxCluster && largest_cluster() == kMaxCluster));
}

cudaError_t launch_page_scores_tc(const PageScoreParams& p, cudaStream_t s) {
  CUtensorMap q;
  if (!tensor_map_bf16(&q, p.q_lat, kD, (uint64_t)p.H, (uint64_t)p.groups, kD * 2, (uint64_t)p.H * kD * 2, 64,
                       (uint32_t)p.H))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(page_scores_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // as many CTAs a query as its tiles need, or as the GPU has room for; above 8 only for the need (4 requests of 32K
  // to 128K tokens, 2 query tokens each: 15.1 us with clusters of 8, two tiles a CTA, 24.3 with 16)
  const int tiles = (p.max_pages + kTile - 1) / kTile;
  int C = 1;
  while (C < 8 && C < tiles && (C * kTiles < tiles || (long long)p.groups * C * 2 <= device_sms())) C *= 2;
  if (C * kTiles < tiles) {
    C = kMaxCluster;
    e = cudaFuncSetAttribute(page_scores_tc_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.groups * C), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, page_scores_tc_kernel, q, p, C);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace mla
