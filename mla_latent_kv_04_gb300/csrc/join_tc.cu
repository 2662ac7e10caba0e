// The output projection over a request's own tokens and a shared prefix, on the tensor cores:
//
//   u[r][h] = a (o_lat[r][h] W_UV[:, h]) + b u_prefix[r][h]     (a, b: softmax weights of the two
//   out[r]  = sum_h u[r][h] W_O[h]                               key sets, from their LSEs)
//
// join_kernel computes u: one CTA per (head, 128 rows), rows in the MMA's M, so that a thread of
// the epilogue has one row, one pair of weights (a, b) and contiguous values to join and store.
// (The weights-in-M form of the unfolded projection's lift, with an element-wise epilogue, took
// 430 us for 512 rows: every element looked its LSEs up and stored two bytes.) It is bound by memory:
// o_lat, W_UV, u_prefix and u once each.
//
// For more than 128 rows the product with W_O runs as tiles of 256 columns and 256 or 512 rows
// on CTA pairs (cta_group::2, M = 256, N = 256): with 512 rows a weight chunk is multiplied with two
// row tiles, whose accumulators fill the tensor memory, so that the weights are read once and
// shared memory takes 48 + 64 bytes a cycle instead of 64 + 64. The (tile, 64-deep chunk) units are
// cut into one contiguous range per pair; pieces of a tile go to the workspace in fp32 and
// gemm_merge_kernel adds them in order. Short products (few heads) take whole tiles instead. Fewer rows are bound by W_O's bytes and take the cluster
// split-K GEMM (gemm_tc.cu). In a graph of such calls 512 rows take 89 us (join 25, product 54, merge 12,
// each by itself) and 32 rows 34; a call by itself 92 and 37. u is rounded to bf16 between the two
// products, as in mla_output_proj_unfolded: W_O's MMAs take it as an operand.
#include "fp8_tiles.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace join {

// ======================================================================== u
constexpr int kBox = 128 * 64 * 2;                     // 64 dims of 128 rows; of W_UV's 128 columns
constexpr int kStage = 2 * kBox;
constexpr int kStages = 3;                             // two CTAs fit on an SM
constexpr int kOffBar = kStages * kStage;
constexpr int kSmem = kOffBar + 128 + 1024;
constexpr int kThreads = 192;
enum { B_FULL = 0, B_EMPTY = kStages, B_DONE = 2 * kStages, B_COUNT };

struct Params {
  const bf16* u_prefix;                                // [rows][H][128]
  const float* lse;                                    // [rows][H]
  const float* lse_prefix;
  bf16* u;
  int rows, H, chunks;                                 // chunks = d_c / 64
  int32_t* status;
};

__global__ void __launch_bounds__(kThreads)
    join_kernel(const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_w, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + kOffBar + 112);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + kOffBar + 116);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int h = blockIdx.x % p.H, r0 = blockIdx.x / p.H * 128;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) ptx::mbar_init(bar(i), 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_o);
    ptx::prefetch_tensormap(&tm_w);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 128);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = ptx::l2_policy_evict_first();
      int c = 0;
      for (; c < p.chunks; ++c) {
        const int st = c % kStages;
        if (!wait(B_EMPTY + st, ((c / kStages) & 1) ^ 1)) break;
        const uint32_t dst = base + st * kStage, full = bar(B_FULL + st);
        ptx::mbar_arrive_expect_tx(full, kStage);
        ptx::tma_load_3d_hint(dst, &tm_o, 64 * c, r0, h, full, pol);
        ptx::tma_load_3d(dst + kBox, &tm_w, h * 128, 64 * c, 0, full);
        ptx::tma_load_3d(dst + kBox + kBox / 2, &tm_w, h * 128 + 64, 64 * c, 0, full);
      }
      if (*abort)
        for (int i = c > kStages ? c - kStages : 0; i < c; ++i) drain_wait(bar(B_FULL + i % kStages), (i / kStages) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(128, 128, false, true);
    bool ok = true;
    for (int c = 0; c < p.chunks; ++c) {
      const int st = c % kStages;
      if (!(ok = __all_sync(0xffffffffu, wait(B_FULL + st, (c / kStages) & 1)) != 0)) break;
      ptx::tc_fence_after();
      const uint32_t x = base + st * kStage;
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_bf16_ss(tmem, ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                           ptx::smem_desc(x + kBox + 2048 * k, kBox / 2, 1024, ptx::kSwizzle128), kIdesc,
                           (c || k) ? 1u : 0u);
        ptx::mma_commit(bar(B_EMPTY + st));
        if (c == p.chunks - 1) ptx::mma_commit(bar(B_DONE));
      }
      __syncwarp();
    }
    if (!ok) {
      if (ptx::elect_one()) ptx::mma_commit(bar(B_DONE));
      __syncwarp();
      drain_wait(bar(B_DONE), 0);
    }
  } else {
    const int quad = warp & 3, r = r0 + 32 * quad + lane;
    const bool live = r < p.rows;
    const long long at = ((long long)r * p.H + h) * 128;
    float a = 0.f, b = 0.f;
    uint4 up[16];                                      // the prefix's row, fetched under the MMAs
    if (live) {
      merge_weights(p.lse[(long long)r * p.H + h], p.lse_prefix[(long long)r * p.H + h], &a, &b);
#pragma unroll
      for (int i = 0; i < 16; ++i) up[i] = reinterpret_cast<const uint4*>(p.u_prefix + at)[i];
    }
    const bool ok = __all_sync(0xffffffffu, wait(B_DONE, 0) && !*abort) != 0;   // (a warp reads, or gives up, as one)
    ptx::tc_fence_after();
    if (ok) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t v[32];
        __syncwarp();                                  // the load is warp-wide
        ptx::tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + 32 * q, v);
        ptx::tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 y = up[4 * q + i];
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = pack_bf16(
                  merge_parts(a, __uint_as_float(v[8 * i + 2 * j]), b, __uint_as_float(w[j] << 16)),
                  merge_parts(a, __uint_as_float(v[8 * i + 2 * j + 1]), b, __uint_as_float(w[j] & 0xFFFF0000u)));
            reinterpret_cast<uint4*>(p.u + at)[4 * q + i] = make_uint4(o[0], o[1], o[2], o[3]);
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
    ptx::tmem_dealloc(tmem, 128);
  }
}

// ======================================================================== u W_O
namespace gemm2 {

template <int kTiles> struct Cfg {                     // row tiles of 256 that share a weight chunk
  static constexpr int kStage = (kTiles + 1) * kBox;   // this CTA's rows and half of the columns
  static constexpr int kNS = kTiles == 1 ? 6 : 4;
  static constexpr int kOffBar = kNS * kStage;
  static constexpr int kSmem = kOffBar + 256 + 1024;
};
static_assert(Cfg<1>::kSmem <= 232448 && Cfg<2>::kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kThreads2 = 384;
// FULL and DFREE in the even CTA (its MMA warp waits for both), EMPTY and DFULL in each
enum { G_FULL = 0, G_EMPTY = 6, G_DFULL = 12, G_DFREE = 14, G_TEAR = 16, G_COUNT };

struct Work {
  int rows, K, N;
  int row_tiles, n_tiles, chunks, pairs;               // tile = n tile * row_tiles + row tile
  int k_tiles;                                         // row tiles of 256 that share a weight chunk
  int whole;                                           // 1: cuts between tiles only, no pieces
  bf16* out;
  float* part;                                         // [2 pairs][2 CTAs][kTiles][64][128][4]: columns
                                                       // by 4, rows, column
  int32_t* status;
  __host__ __device__ long long units() const { return (long long)row_tiles * n_tiles * chunks; }
  __host__ __device__ long long begin(int w) const {
    return whole ? (long long)row_tiles * n_tiles * w / pairs * chunks : units() * w / pairs;
  }
};

struct Segment {
  long long u, end;
  int chunks, tile, k0, k1;
  __device__ Segment(const Work& w, int pair) : u(w.begin(pair)), end(w.begin(pair + 1)), chunks(w.chunks) {}
  __device__ bool next() {
    if (u >= end) return false;
    tile = (int)(u / chunks);
    k0 = (int)(u - (long long)tile * chunks);
    const long long left = end - u;
    k1 = left < chunks - k0 ? k0 + (int)left : chunks;
    u += k1 - k0;
    return true;
  }
};

template <int kTiles>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads2, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Work w) {
  using C = Cfg<kTiles>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + C::kOffBar + 240);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + C::kOffBar + 244);
  auto bar = [&](int i) { return base + C::kOffBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank(), pair = blockIdx.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G_COUNT; ++i) ptx::mbar_init(bar(i), i == G_DFREE || i == G_DFREE + 1 ? 16 : 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_x);
    ptx::prefetch_tensormap(&tm_w);
  }
  __syncthreads();
  ptx::cluster_sync();
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
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, w.status); };
  auto lead = [&](int i) { return ptx::map_to_rank(bar(i), 0u); };
  constexpr int kBufs = kTiles == 1 ? 2 : 1;           // accumulators of 256 kTiles columns
  Segment seg(w, pair);

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = ptx::l2_policy_evict_first();
      uint32_t st = 0, wrap = 0, g = 0;
      bool ok = true;
      while (ok && seg.next()) {
        const int n0 = seg.tile / w.row_tiles * 256 + 128 * rank;
        const int r0 = seg.tile % w.row_tiles * 256 * kTiles + 128 * rank;
        for (int k = seg.k0; k < seg.k1; ++k, ++g) {
          if (!(ok = wait(G_EMPTY + st, (wrap & 1) ^ 1))) break;
          const uint32_t dst = base + st * C::kStage, full = lead(G_FULL + st);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar(G_FULL + st), 2 * C::kStage);
          ptx::tma_load_3d_pair_hint(dst, &tm_w, n0, 64 * k, 0, full, pol);
          ptx::tma_load_3d_pair_hint(dst + kBox / 2, &tm_w, n0 + 64, 64 * k, 0, full, pol);
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
            ptx::tma_load_3d_pair(dst + (1 + i) * kBox, &tm_x, 64 * k, r0 + 256 * i, 0, full);
          if (++st == C::kNS) {
            st = 0;
            ++wrap;
          }
        }
      }
      if (*abort && rank == 0)
        for (uint32_t i = g > C::kNS ? g - C::kNS : 0; i < g; ++i)
          drain_wait(bar(G_FULL + i % C::kNS), (i / C::kNS) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(256, 256, false, true);
      uint32_t st = 0, wrap = 0, s = 0;
      bool ok = true;
      auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
      while (ok && seg.next()) {
        const uint32_t b = s % kBufs, turn = s / kBufs;
        if (!(ok = __all_sync(0xffffffffu, bounded_wait<true>(bar(G_DFREE + b), (turn & 1) ^ 1, abort, w.status)) != 0))
          break;
        const uint32_t d = tmem + 256 * b;
        for (int k = seg.k0; k < seg.k1; ++k) {
          if (!(ok = wait_w(G_FULL + st, wrap & 1))) break;
          ptx::tc_fence_after();
          const uint32_t x = base + st * C::kStage;
          if (ptx::elect_one()) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                ptx::mma_bf16_ss_pair(d + 256 * i, ptx::smem_desc(x + (1 + i) * kBox + 32 * j, 16, 1024, ptx::kSwizzle128),
                                      ptx::smem_desc(x + 2048 * j, kBox / 2, 1024, ptx::kSwizzle128), kIdesc,
                                      (k > seg.k0 || j) ? 1u : 0u);
            ptx::mma_commit_pair(bar(G_EMPTY + st));
            if (k == seg.k1 - 1) ptx::mma_commit_pair(bar(G_DFULL + b));
          }
          __syncwarp();
          if (++st == C::kNS) {
            st = 0;
            ++wrap;
          }
        }
        ++s;
      }
      if (*abort) {
        if (ptx::elect_one()) ptx::mma_commit_pair(bar(G_TEAR));
        __syncwarp();
        drain_wait(bar(G_TEAR), 0);
      }
    }
  } else if (warp >= 4) {
    const int quad = warp & 3, part = warp >= 8 ? 1 : 0, row = 32 * quad + lane;   // columns 128 part ..
    const uint32_t free0 = lead(G_DFREE);
    uint32_t s = 0;
    while (seg.next()) {
      const uint32_t b = s % kBufs;
      if (!__all_sync(0xffffffffu, wait(G_DFULL + b, (s / kBufs) & 1))) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(32 * quad) << 16) + 256 * b;
      const bool full = seg.k0 == 0 && seg.k1 == w.chunks;
      const long long slot = 2LL * pair + (seg.k0 == 0 ? 1 : 0);
      const int n0 = seg.tile / w.row_tiles * 256 + 128 * part;
#pragma unroll 1
      for (int i = 0; i < kTiles; ++i) {
        const int r = (seg.tile % w.row_tiles * kTiles + i) * 256 + 128 * rank + row;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32];
          __syncwarp();                                // the load is warp-wide (rows behind the last left early)
          ptx::tmem_ld32(d + 256 * i + 128 * part + 32 * q, v);
          ptx::tmem_wait_ld();
          if (i == kTiles - 1 && q == 3) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_remote_relaxed(free0 + 8 * b, 0u);
          }
          if (r >= w.rows) continue;
          if (!full) {
            float4* dst = reinterpret_cast<float4*>(w.part) +
                          (((slot * 2 + rank) * kTiles + i) * 64 + 32 * part + 8 * q) * 128 + row;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[j * 128] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                         __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          } else {
            const int n = n0 + 32 * q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {              // N is a multiple of 8
              if (n + 8 * j >= w.N) break;
              uint32_t o[4];
#pragma unroll
              for (int t = 0; t < 4; ++t)
                o[t] = pack_bf16(__uint_as_float(v[8 * j + 2 * t]), __uint_as_float(v[8 * j + 2 * t + 1]));
              *reinterpret_cast<uint4*>(w.out + (long long)r * w.N + n + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
      }
      ++s;
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Adds a cut tile's pieces, in order. Block (tile, 16 columns, row tile), thread per row.
template <int kTiles>
__global__ void __launch_bounds__(256) gemm_merge_kernel(const Work w) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tile = blockIdx.x, i = blockIdx.z, tr = threadIdx.x;
  const int n = tile / w.row_tiles * 256 + 16 * blockIdx.y;
  const int r = (tile % w.row_tiles * kTiles + i) * 256 + tr;
  if (r >= w.rows || n >= w.N) return;
  const long long t0 = (long long)tile * w.chunks, U = w.units();
  auto owner = [&](long long u) {
    int c = (int)(u * w.pairs / U);
    while (w.begin(c + 1) <= u) ++c;
    while (w.begin(c) > u) --c;
    return c;
  };
  const int c0 = owner(t0), c1 = owner(t0 + w.chunks - 1);
  if (c0 == c1) return;                                // written whole
  const int rank = tr >> 7, row = tr & 127;
  float acc[16] = {};
  for (int c = c0; c <= c1; ++c) {
    const long long slot = 2LL * c + (c == c0 ? 1 : 0);
    const float4* src = reinterpret_cast<const float4*>(w.part) +
                        (((slot * 2 + rank) * kTiles + i) * 64 + 4 * blockIdx.y) * 128 + row;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 y = src[j * 128];
      acc[4 * j] += y.x;
      acc[4 * j + 1] += y.y;
      acc[4 * j + 2] += y.z;
      acc[4 * j + 3] += y.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (n + 8 * j >= w.N) break;
    uint32_t o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = pack_bf16(acc[8 * j + 2 * t], acc[8 * j + 2 * t + 1]);
    *reinterpret_cast<uint4*>(w.out + (long long)r * w.N + n + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Whole tiles of 256 rows, or even cuts of tiles of 256 (more than 256 rows: 512), whose pieces cost a
// way through the workspace and the merge, as long as some 30 chunks of a tile for every 256 rows: whichever
// is shorter. 512 rows, the whole call: 16 heads 23 us whole and 36 cut, 32 heads 34.5 and 42; 64 and 128
// heads are cut (56 and 90 us).
constexpr int kMergeChunks = 30;
static Work plan(int rows, int K, int N) {
  Work w{};
  w.rows = rows;
  w.K = K;
  w.N = N;
  w.n_tiles = (N + 255) / 256;
  w.chunks = (K + 63) / 64;
  const int most = device_sms() > 1 ? device_sms() / 2 : 1, k_tiles = rows > 256 ? 2 : 1;
  auto tiles = [&](int k) { return (long long)((rows + 256 * k - 1) / (256 * k)) * w.n_tiles; };
  const long long whole = (tiles(1) + most - 1) / most * w.chunks;
  const long long cut = tiles(k_tiles) * w.chunks * k_tiles / most + kMergeChunks * k_tiles;
  w.whole = whole <= cut;
  w.k_tiles = w.whole ? 1 : k_tiles;
  w.row_tiles = (rows + 256 * w.k_tiles - 1) / (256 * w.k_tiles);
  const long long parts = w.whole ? tiles(1) : w.units();
  w.pairs = (int)(parts < most ? parts : most);
  return w;
}

template <int kTiles>
static cudaError_t run(const CUtensorMap& x, const CUtensorMap& wm, const Work& w, cudaStream_t s) {
  using C = Cfg<kTiles>;
  auto kern = gemm_pair_kernel<kTiles>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * w.pairs), 1, 1);
  cfg.blockDim = dim3(kThreads2, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, x, wm, w);
  if (e != cudaSuccess) return e;
  note_launch();
  if (w.whole) return cudaSuccess;
  cfg.gridDim = dim3((unsigned)(w.row_tiles * w.n_tiles), 16, kTiles);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, gemm_merge_kernel<kTiles>, w);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace gemm2
}  // namespace join

bool prefix_join_tc_supported(const mla_config* c) {
  return c->act_dtype == MLA_BF16 && c->d_v == 128 && c->d_latent % 64 == 0;
}

// More rows than this take the pair GEMM.
constexpr int kPairRows = 128;
static bool pair_gemm(int rows, int N) { return rows > kPairRows && N % 8 == 0; }

size_t prefix_join_tc_workspace(int rows, int H, int d_v, int N) {
  if (!pair_gemm(rows, N)) return 0;
  const join::gemm2::Work w = join::gemm2::plan(rows, H * d_v, N);
  return w.whole ? 0 : (size_t)2 * w.pairs * 2 * w.k_tiles * 256 * 128 * 4;
}

cudaError_t launch_prefix_join_tc(const void* o_lat, const void* W_UV, int rows, int H, int d_c, const PrefixJoin& j,
                                  void* u, int32_t* status, cudaStream_t s) {
  using namespace join;
  CUtensorMap o, wv;
  if (!tensor_map_bf16(&o, o_lat, (uint64_t)d_c, (uint64_t)rows, (uint64_t)H, (uint64_t)H * d_c * 2, (uint64_t)d_c * 2, 64, 128) ||
      !tensor_map_bf16(&wv, W_UV, (uint64_t)H * 128, (uint64_t)d_c, 1, (uint64_t)H * 256, (uint64_t)H * 256 * d_c, 64, 64))
    return cudaErrorInvalidValue;
  Params p;
  p.u_prefix = reinterpret_cast<const bf16*>(j.u_prefix);
  p.lse = j.lse;
  p.lse_prefix = j.lse_prefix;
  p.u = reinterpret_cast<bf16*>(u);
  p.rows = rows;
  p.H = H;
  p.chunks = d_c / 64;
  p.status = status;
  cudaError_t e = cudaFuncSetAttribute(join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(H * ((rows + 127) / 128)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, join_kernel, o, wv, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_prefix_project_tc(const void* u, const void* W_O, int rows, int K, int N, void* out, void* part,
                                     int32_t* status, cudaStream_t s) {
  using namespace join;
  if (!pair_gemm(rows, N)) return launch_output_proj_tc(u, W_O, rows, K, N, out, status, s);
  gemm2::Work w = gemm2::plan(rows, K, N);
  w.out = reinterpret_cast<bf16*>(out);
  w.part = reinterpret_cast<float*>(part);
  w.status = status;
  CUtensorMap x, wm;
  if (!tensor_map_bf16(&x, u, (uint64_t)K, (uint64_t)rows, 1, (uint64_t)K * 2, (uint64_t)K * rows * 2, 64, 128) ||
      !tensor_map_bf16(&wm, W_O, (uint64_t)N, (uint64_t)K, 1, (uint64_t)N * 2, (uint64_t)N * K * 2, 64, 64))
    return cudaErrorInvalidValue;
  return w.k_tiles == 2 ? gemm2::run<2>(x, wm, w, s) : gemm2::run<1>(x, wm, w, s);
}

}  // namespace mla
