// Accumulated attention weight of every cached token, on the tensor cores (bf16 activations, every
// cache format, 64-token pages, d_c 512, d_r 64, a multiple of 16 heads up to 128).
//
// Per tile of 128 tokens (two pages) the scores of all heads are one product,
//   Z = X q_lat^T   (M = 128 tokens, N = heads, K = 576),
// tokens in the rows: a token's sum over heads is then a sum over the columns of one lane of
// tensor memory, in one thread's registers:
//   mass = sum_h exp2(c Z_h - log2(e) lse_h),   c = softmax scale * log2 e.
// q_lat is an operand as given (bf16), products are exact and sums fp32, so the weights are
// fp32 results.
//
// Work: the tiles of all requests in order, cut into one contiguous range per CTA; a CTA's
// tiles of one request are a run, which loads the request's query (H x 576) once. With several
// query tokens a run is at most kRunMax tiles and is passed over once per query token (the
// later passes read its pages from L2), each pass adding to the weights that the same thread
// wrote before: no atomics, one order of sums.
//
// fp8 caches land as codes, which eight converter warps expand into the bf16 chunks that the MMAs
// read: exactly for a per-tensor scale (which multiplies the scores); a block-scaled code times
// its scale as the sum of two bf16 chunks (residual 2^-17 of it), both multiplied with the
// same query chunk, since one bf16 would leave 2^-9 in every term of a score.
//
// Bound: the cache is read once, 147 KB a tile (bf16); the MMAs take a third of that time.
#include <math.h>

#include "fp8_tiles.cuh"
#include "internal.h"
#include "prologue.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace weigh {

constexpr int kTile = 128, kD = 576, kChunks = 9;      // 64 dims a chunk
constexpr int kStage = kTile * 64 * 2;                 // one chunk of a tile: 16 KB
constexpr int kRingBytes = 5 * kStage;
constexpr int kQChunk = 128 * 64 * 2;
constexpr int kOffRing = kChunks * kQChunk;            // the query first: 144 KB
constexpr int kOffLse = kOffRing + kRingBytes;
constexpr int kOffBar = kOffLse + 512;
constexpr int kSmem = kOffBar + 256 + 1024;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kRunMax = 4;
constexpr int kConvWarps = 8;
// kKind 0: bf16 cache, 5 chunks in flight; 1: e4m3 with one scale, 2: block scales (3 expanded
// chunks and 4 of codes, 8 KB each)
template <int kKind> struct Ring {
  static constexpr uint32_t kTiles = kKind ? 3 : 5;
  static constexpr uint32_t kRaw = 4;
  static constexpr int kOffRaw = kOffRing + 3 * kStage;
  static constexpr int kThreads = 192 + (kKind ? 32 * kConvWarps : 0);
  static constexpr int kLoads = kKind == 2 ? 8 : kChunks;   // chunks of a tile that come by TMA
  static constexpr int kSteps = kKind == 2 ? 17 : kChunks;  // chunks that the MMAs read
};
enum { B_FULL = 0, B_EMPTY = 5, B_QFULL = 10, B_QEMPTY, B_ZFULL, B_ZFREE = B_ZFULL + 2,
       B_MEET = B_ZFREE + 2, B_RAWFULL, B_RAWEMPTY = B_RAWFULL + 4, B_TEAR = B_RAWEMPTY + 4, B_COUNT };
static_assert(B_COUNT * 8 <= 240, "barrier area");

__device__ __forceinline__ int request_tiles(const KeyWeightParams& p, int b) {
  const int S = p.seq_lens[b];
  if (S < p.q_len || S <= 0 || S > (long long)p.max_pages * p.P) return 0;
  return (S + kTile - 1) / kTile;
}

// A CTA's runs in order: tiles [t0, t1) of request b.
struct Runs {
  const KeyWeightParams* p;
  int b, at, tiles;            // next tile of request b, and how many it has
  long long left;              // tiles of the CTA's range still to come
  int limit, t0, t1, rb;
  __device__ bool next() {
    if (left <= 0) return false;
    while (at >= tiles) {
      tiles = request_tiles(*p, ++b);
      at = 0;
    }
    rb = b;
    t0 = at;
    int n = min(tiles - at, limit);
    if (n > left) n = (int)left;
    t1 = at + n;
    at = t1;
    left -= t1 - t0;
    return true;
  }
};

template <int kKind>
__global__ void __launch_bounds__(Ring<kKind>::kThreads, 1)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_q,
                          const KeyWeightParams p) {
  using R = Ring<kKind>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + kOffBar + 240);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + kOffBar + 244);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      int n = 1;
      if (i >= B_ZFREE && i <= B_MEET) n = 4;                        // the epilogue warps
      if (kKind && (i < B_EMPTY || (i >= B_RAWEMPTY && i < B_TEAR))) n = kConvWarps;
      ptx::mbar_init(bar(i), n);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_x);
    ptx::prefetch_tensormap(&tm_q);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 256);
    ptx::tmem_relinquish();
  }
  // the requests' tiles, summed up (the scan's scratch is the query's place, not yet in use)
  int* cu = reinterpret_cast<int*>(basep);             // [batch + 1]
  __shared__ int warp_tot[32], start[2];
  for (int b = threadIdx.x; b < p.batch; b += R::kThreads) {
    const int S = p.seq_lens[b];
    cu[b + 1] = request_tiles(p, b);
    if (blockIdx.x == 0 && S != 0 && cu[b + 1] == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  }
  if (threadIdx.x == 0) cu[0] = 0;
  __syncthreads();
  block_inclusive_scan(cu + 1, p.batch, warp_tot);
  const long long total = cu[p.batch];
  const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  if (threadIdx.x == 0 && u1 > u0) {
    const int b = last_at_most(cu, p.batch, u0);       // its last request with cu[b] <= u0: not empty
    start[0] = b;
    start[1] = (int)(u0 - cu[b]);
  }
  ptx::tc_fence_before();
  // the scratch is done with before the query's copy (through the async proxy) may land on it
  ptx::fence_proxy_async_smem();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  Runs run;
  run.p = &p;
  run.left = u1 - u0;
  run.limit = p.q_len > 1 ? kRunMax : 0x7FFFFFFF;
  run.b = run.left > 0 ? start[0] : 0;
  run.at = run.left > 0 ? start[1] : 0;
  run.tiles = run.left > 0 ? request_tiles(p, run.b) : 0;

  if (warp == 0) {
    if (lane == 0) {
      constexpr uint32_t kSlots = kKind ? R::kRaw : R::kTiles, kBytes = kKind ? kStage / 2 : kStage;
      constexpr int kFullBar = kKind ? B_RAWFULL : B_FULL, kEmptyBar = kKind ? B_RAWEMPTY : B_EMPTY;
      constexpr int kOff = kKind ? R::kOffRaw : kOffRing;
      const uint64_t pol = ptx::l2_policy_evict_first();
      uint32_t g = 0;
      bool ok = true;
      while (ok && run.next()) {
        const int32_t* bt = p.block_table + (long long)run.rb * p.max_pages;
        const int S = p.seq_lens[run.rb];
        // a page's first row; behind the request's last page, or for a bad id, any page's (those
        // tokens are not written)
        auto row_of = [&](int pg) {
          int page = (long long)pg * p.P < S ? bt[pg] : 0;
          if (page < 0 || page >= p.num_pages) {
            flag_status(p.status, MLA_ERR_DEVICE_GUARD);
            page = 0;
          }
          return page * p.P;
        };
        for (int t = 0; ok && t < p.q_len; ++t) {
          int y0 = row_of(2 * run.t0), y1 = row_of(2 * run.t0 + 1);
          for (int tile = run.t0; ok && tile < run.t1; ++tile) {
            const bool two = (long long)(2 * tile + 1) * p.P < S;
            int n0 = 0, n1 = 0;
            for (int c = 0; c < R::kLoads; ++c, ++g) {
              const uint32_t st = g % kSlots;
              if (!(ok = wait(kEmptyBar + st, ((g / kSlots) & 1) ^ 1))) break;
              const uint32_t dst = base + kOff + st * kBytes, full = bar(kFullBar + st);
              ptx::mbar_arrive_expect_tx(full, two ? kBytes : kBytes / 2);
              if (p.q_len > 1) {
                ptx::tma_load_3d(dst, &tm_x, 64 * c, y0, 0, full);
                if (two) ptx::tma_load_3d(dst + kBytes / 2, &tm_x, 64 * c, y1, 0, full);
              } else {
                ptx::tma_load_3d_hint(dst, &tm_x, 64 * c, y0, 0, full, pol);
                if (two) ptx::tma_load_3d_hint(dst + kBytes / 2, &tm_x, 64 * c, y1, 0, full, pol);
              }
              if (c == 0 && tile + 1 < run.t1) {       // the next tile's pages, ahead of need
                n0 = row_of(2 * tile + 2);
                n1 = row_of(2 * tile + 3);
              }
            }
            y0 = n0;
            y1 = n1;
          }
        }
      }
      if (*abort)
        for (uint32_t i = g > kSlots ? g - kSlots : 0; i < g; ++i)
          drain_wait(bar(kFullBar + i % kSlots), (i / kSlots) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(128, p.H, false, false);
      uint32_t g = 0, q_iter = 0, z = 0;
      bool ok = true;
      while (ok && run.next()) {
        for (int t = 0; ok && t < p.q_len; ++t, ++q_iter) {
          // the query of this run and token: all MMAs on the one before were issued by this
          // thread, and B_QEMPTY says they have completed
          if (!(ok = wait(B_QEMPTY, (q_iter & 1) ^ 1))) break;
          ptx::mbar_arrive_expect_tx(bar(B_QFULL), kChunks * p.H * 128);
          for (int c = 0; c < kChunks; ++c)
            ptx::tma_load_3d(base + c * kQChunk, &tm_q, 64 * c, 0, run.rb * p.q_len + t, bar(B_QFULL));
          if (!(ok = wait(B_QFULL, q_iter & 1))) break;
          for (int tile = run.t0; ok && tile < run.t1; ++tile, ++z) {
            if (!(ok = wait(B_ZFREE + (z & 1), ((z >> 1) & 1) ^ 1))) break;
            for (int i = 0; i < R::kSteps; ++i, ++g) {
              const int c = kKind == 2 ? i >> 1 : i;   // block scales: two chunks per query chunk
              const uint32_t st = g % R::kTiles;
              if (!(ok = wait(B_FULL + st, (g / R::kTiles) & 1))) break;
              ptx::tc_fence_after();
              const uint32_t x = base + kOffRing + st * kStage, q = base + c * kQChunk;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ptx::mma_bf16_ss(tmem + 128 * (z & 1), ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                                 ptx::smem_desc(q + 32 * k, 16, 1024, ptx::kSwizzle128), idesc,
                                 (i || k) ? 1u : 0u);
              ptx::mma_commit(bar(B_EMPTY + st));
            }
            if (!ok) break;
            ptx::mma_commit(bar(B_ZFULL + (z & 1)));
            if (tile == run.t1 - 1) ptx::mma_commit(bar(B_QEMPTY));
          }
        }
      }
      if (*abort) {
        ptx::mma_commit(bar(B_TEAR));
        drain_wait(bar(B_TEAR), 0);
        if (q_iter) drain_wait(bar(B_QFULL), (q_iter - 1) & 1);
        drain_wait(bar(B_QFULL), q_iter & 1);
      }
    }
  } else if (warp < 6) {
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16);
    float* lse_s = reinterpret_cast<float*>(basep + kOffLse);
    uint32_t z = 0, meets = 0;
    bool ok = true;
    // tensor-memory accesses are warp-wide: a warp goes on, or leaves, as one
    auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
    auto meet = [&]() {                          // the four warps (bounded, unlike a named barrier)
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_MEET));
      return wait_w(B_MEET, meets++ & 1);
    };
    while (ok && run.next()) {
      const int S = p.seq_lens[run.rb];
      const int32_t* bt = p.block_table + (long long)run.rb * p.max_pages;
      float* w = p.weights + (long long)run.rb * p.max_pages * p.P;
      for (int t = 0; ok && t < p.q_len; ++t) {
        const float* lse = p.lse + ((long long)run.rb * p.q_len + t) * p.H;
        if (!(ok = meet())) break;
        if (row < p.H) lse_s[row] = lse[row] * kLog2e;
        if (!(ok = meet())) break;
        for (int tile = run.t0; tile < run.t1; ++tile, ++z) {
          if (!(ok = wait_w(B_ZFULL + (z & 1), (z >> 1) & 1))) break;
          ptx::tc_fence_after();
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          for (int h0 = 0; h0 < p.H; h0 += 16) {
            uint32_t v[16];
            ptx::tmem_ld16(t_row + 128 * (z & 1) + h0, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 off = *reinterpret_cast<const float4*>(lse_s + h0 + j);
              sum[0] += ptx::ex2(fmaf(__uint_as_float(v[j]), p.scale_log2, -off.x));
              sum[1] += ptx::ex2(fmaf(__uint_as_float(v[j + 1]), p.scale_log2, -off.y));
              sum[2] += ptx::ex2(fmaf(__uint_as_float(v[j + 2]), p.scale_log2, -off.z));
              sum[3] += ptx::ex2(fmaf(__uint_as_float(v[j + 3]), p.scale_log2, -off.w));
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(B_ZFREE + (z & 1)));
          const int j = tile * kTile + row;
          if (j < S) {
            const int page = bt[j / p.P];
            if (page >= 0 && page < p.num_pages) {
              const bool sees = j <= S - p.q_len + t;
              const float mass = sees ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
              if (t == 0) w[j] = (p.decay != 0.f && j < S - p.q_len) ? fmaf(p.decay, w[j], mass) : mass;
              else if (sees) w[j] += mass;
            }
          }
        }
      }
    }
  } else if (kKind != 0) {
    // converters: two threads per token row of the chunk, 32 dims each
    const int row = (threadIdx.x - 192) & 127, half = (threadIdx.x - 192) >> 7;
    uint32_t gr = 0, g = 0;
    bool ok = true;
    auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
    auto done = [&](uint32_t slot) {
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_FULL + slot));
    };
    while (ok && run.next()) {
      const int32_t* bt = p.block_table + (long long)run.rb * p.max_pages;
      const int S = p.seq_lens[run.rb];
      float4 sc = make_float4(0.f, 0.f, 0.f, 0.f), sc_next = sc;
      uint4 pe[4], pe_next[4];
      // block scales: a token's four scales and its half of the bf16 rotary key, from memory
      auto fetch = [&](int tile) {
        const int j = tile * kTile + row;
        int page = j < S ? bt[j / 64] : -1;
        if (page >= p.num_pages) page = -1;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.cache) +
                             ((long long)(page < 0 ? 0 : page) * 64 + (row & 63)) * p.row_bytes + 512;
        if (page >= 0) {
          sc_next = *reinterpret_cast<const float4*>(src);
#pragma unroll
          for (int i = 0; i < 4; ++i) pe_next[i] = *reinterpret_cast<const uint4*>(src + 16 + 64 * half + 16 * i);
        }
      };
      for (int t = 0; ok && t < p.q_len; ++t) {
        if (kKind == 2) fetch(run.t0);
        for (int tile = run.t0; ok && tile < run.t1; ++tile) {
          if (kKind == 2) {
            sc = sc_next;
#pragma unroll
            for (int i = 0; i < 4; ++i) pe[i] = pe_next[i];
            if (tile + 1 < run.t1) fetch(tile + 1);
          }
          for (int c = 0; c < R::kLoads; ++c, ++gr) {
            const uint32_t rs = gr % R::kRaw, st = g % R::kTiles, st2 = (g + 1) % R::kTiles;
            if (!(ok = wait_w(B_RAWFULL + rs, (gr / R::kRaw) & 1))) break;
            if (!(ok = wait_w(B_EMPTY + st, ((g / R::kTiles) & 1) ^ 1))) break;
            uint4 codes[2];
            load_codes_half_row(basep + R::kOffRaw + rs * (kStage / 2), row, half, codes);
            if (kKind == 1) {
              expand_codes_half_row<false, false>(codes, basep + kOffRing + st * kStage, nullptr, row, half, 1.f);
              done(st);
              ++g;
            } else {
              if (!(ok = wait_w(B_EMPTY + st2, (((g + 1) / R::kTiles) & 1) ^ 1))) break;
              const float s = (c >> 1) == 0 ? sc.x : ((c >> 1) == 1 ? sc.y : ((c >> 1) == 2 ? sc.z : sc.w));
              expand_codes_half_row<true, true>(codes, basep + kOffRing + st * kStage,
                                                basep + kOffRing + st2 * kStage, row, half, s);
              done(st);
              if (lane == 0) ptx::mbar_arrive(bar(B_FULL + st2));
              g += 2;
            }
            if (lane == 0) ptx::mbar_arrive(bar(B_RAWEMPTY + rs));
          }
          if (kKind == 2 && ok) {                      // the rotary chunk
            const uint32_t st = g % R::kTiles;
            if (!(ok = wait_w(B_EMPTY + st, ((g / R::kTiles) & 1) ^ 1))) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(basep + kOffRing + st * kStage + row * 128 +
                                        (((4 * half + i) ^ (row & 7)) << 4)) = pe[i];
            done(st);
            ++g;
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

namespace weigh {
template <int kKind>
static cudaError_t run(const CUtensorMap& x, const CUtensorMap& q, const KeyWeightParams& p, int ctas,
                       cudaStream_t s) {
  auto kern = key_weights_tc_kernel<kKind>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kern<<<ctas, Ring<kKind>::kThreads, kSmem, s>>>(x, q, p);
  note_launch();
  return cudaGetLastError();
}
}  // namespace weigh

cudaError_t launch_key_weights_tc(mla_dtype cache, const KeyWeightParams& p, cudaStream_t s) {
  using namespace weigh;
  CUtensorMap x, q;
  const uint64_t rows = (uint64_t)p.num_pages * 64;
  const bool bf = cache == MLA_BF16;
  if (!tensor_map_3d(&x, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     bf ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, p.cache,
                     cache == MLA_FP8_E4M3_B128 ? 512 : kD, rows, 1, (uint64_t)p.row_bytes, rows * p.row_bytes,
                     64, 64) ||
      !tensor_map_bf16(&q, p.q_lat, kD, (uint64_t)p.H, (uint64_t)p.batch * p.q_len, kD * 2,
                       (uint64_t)p.H * kD * 2, 64, (uint32_t)p.H))
    return cudaErrorInvalidValue;
  // no more CTAs than tiles that the tables can hold
  const long long most = (long long)p.batch * ((p.max_pages + 1) / 2);
  const int ctas = (int)(most < device_sms() ? most : device_sms());
  if (bf) return run<0>(x, q, p, ctas, s);
  return cache == MLA_FP8_E4M3 ? run<1>(x, q, p, ctas, s) : run<2>(x, q, p, ctas, s);
}

}  // namespace mla
