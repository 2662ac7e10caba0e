// Product with 4-bit weights on the tensor cores (bf16 activations).
//
//   out^T = W^T x^T: M = 128 columns of W, N = columns made of the rows of x, the scales of both operands
// (a power of two per 32 elements of K) applied by the MMA itself. x is not rounded: a row is several
// columns whose fp32 sums are added in the epilogue. With E the exponent of a block's largest magnitude,
//   form 4 (kind::mxf4, up to 40 rows): e2m1 holds the integers -3 .. 4, digits enough for a base-8 number;
//     with s = 2^(E - 1)
//       |x| = s (d_0 + d_1 / 8 + ... + d_5 / 8^5),  d_0 in 0 .. 4, the others in -3 .. 4,
//     for |x| / s rounded to a multiple of 8^-5: off by at most 2^(E - 17) (E not below -111, where the last
//     digit's scale ends), and exact for elements down to
//     2^-9 of the largest (bf16 has 8 significant bits). Six columns a row, digit i under s / 8^i.
//   form 8 (kind::mxf8f6f4, more rows): an e4m3 value has 4 significant bits; with s = 2^(E - 7)
//       x = s (hi + lo / 16),  hi = e4m3(x / s), lo = e4m3(16 (x / s - hi)),
//     exactly for elements down to 2^-13 of the largest, off by at most 2^(E - 21). Two columns a row.
// The form of six columns reads the codes as they lie in memory. For an 8-bit MMA they are spread to 8
// bytes in 16 of shared memory, which the TMA does at 3.5 TB/s in all; with many rows the MMAs count, and
// six columns of 4 bits take 1.5 times two of 8. 65536 x 5120 weights with a cold L2, form 4 against form 8: 1
// row 44 against 56 us, 32 rows 50 against 61, 64 rows 74 against 67, 128 rows 124 against 83, 512 rows 519
// against 267 (the bf16 product with the same weights: 115 to 320).
//
// Bound: up to 40 rows HBM (32 rows: 182 MB in 41 us among calls, the product alone 35, 5.2 TB/s), with the
// split in front and the sum of pieces behind (6 and 4 us); many rows the MMAs, whose pipe is busy 56 percent of the
// cycles at 512 rows x 16384 x 5120 (65 of 79 us; columns of two terms double the products).
//
// Work is the sequence of (128 columns, row tile, 256 or 128 of K) steps, cut into one equal range per CTA; a
// CTA that does not have all of a tile's steps writes its fp32 sums to a piece, and a second kernel adds a
// tile's pieces in order: the same bits every time. The MMAs are issued by an elected lane from uniform
// registers, unrolled: issued from computed descriptors they took 250 cycles each (32 rows: 97 us).
#include "internal.h"
#include "mx4.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace mx4 {

constexpr int kA = 128 * 128;                  // a step's codes in shared memory
constexpr int kMaxStages = 10;
constexpr int kThreads = 192;
constexpr int kBarBytes = 256;
constexpr int kPrefetch = 16;                  // steps asked of L2 while the activations are split

template <bool kForm8> struct Form;
template <> struct Form<false> {
  static constexpr int kStepK = 256, kGroups = 2, kCols = 6, kMaxT = 40, kTx = kA;
};
template <> struct Form<true> {                // (an unpacking load counts the packed bytes)
  static constexpr int kStepK = 128, kGroups = 1, kCols = 2, kMaxT = 128, kTx = kA / 2;
};

// A tile of T rows, its columns and their scale atoms (an atom: 128 columns x 4 blocks, 512 bytes).
struct TileShape {
  int T, tiles, cols, atoms;
  int stage, stages, sf;                       // bytes and scale columns of a stage
};
template <bool kForm8>
inline TileShape tile_shape(int rows) {
  typedef Form<kForm8> F;
  TileShape t;
  t.tiles = (rows + F::kMaxT - 1) / F::kMaxT;
  t.T = ((rows + t.tiles - 1) / t.tiles + 7) / 8 * 8;
  t.tiles = (rows + t.T - 1) / t.T;
  t.cols = F::kCols * t.T;
  t.atoms = (t.cols + 127) / 128;
  t.stage = kA + t.cols * 128 + (F::kGroups * 512 * (1 + t.atoms) + 1023) / 1024 * 1024;
  t.stages = ((int)kSmemPerCta - 1024 - kBarBytes) / t.stage;
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  t.sf = F::kGroups * 4 * (1 + t.atoms);
  return t;
}

struct Work {
  long long units;                             // steps of all tiles
  int steps, tiles, row_tiles, grid;           // steps of a tile, tiles, row tiles of a column tile
  __host__ __device__ long long start(int c) const { return units * c / grid; }
  __host__ __device__ int owner(long long u) const { return (int)(((u + 1) * grid - 1) / units); }
};

// ======================================================================== activations
// x [rows][K] -> per row tile the columns' codes [columns][K / 2 or K bytes] (every row's first column, every
// row's second one, ..) and scale atoms [tile][K / 128][atom][512] (column % 32, then column / 32, then
// block). Four lanes a block of 32, eight elements each. Columns of rows behind the last one are not
// written (nor read from the product).
template <bool kForm8>
__device__ __forceinline__ void split_row(const bf16* __restrict__ x, int r, int k, int K, const TileShape& t,
                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  uint4 v4 = make_uint4(0u, 0u, 0u, 0u);
  if (k < K) v4 = *reinterpret_cast<const uint4*>(x + (long long)r * K + k);
  const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
  const unsigned lanes = 0xFFFFu << (threadIdx.x & 16);
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, v[i] & 0x7FFF7FFFu);
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  m = max(m, __shfl_xor_sync(lanes, m, 1));
  m = max(m, __shfl_xor_sync(lanes, m, 2));
  const int tile = r / t.T, rr = r - tile * t.T, groups = (K + 127) / 128;
  int e;                                       // s = 2^(e - 127), large enough for the last column's scale
  if constexpr (!kForm8) {
    e = max(15, (int)(m >> 7) - 1);
    const float inv = __uint_as_float((uint32_t)(254 + 15 - e) << 23);     // 8^5 / s
    // |x| / s in units of 8^-5, plus 3 of every digit: digit i is bits 15 - 3 i .. of it, less 3
    uint32_t u[8], sign = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = (uint32_t)__float2int_rn(__uint_as_float((v[i] & 0x7FFFu) << 16) * inv) + 112347u;
      u[2 * i + 1] = (uint32_t)__float2int_rn(__uint_as_float(v[i] & 0x7FFF0000u) * inv) + 112347u;
      sign |= ((v[i] >> 15 & 1u) << 3 | (v[i] >> 31) << 7) << (8 * i);
    }
    uint8_t* dst = codes + ((long long)tile * t.cols + rr) * (K / 2) + k / 2;
#pragma unroll
    for (int d = 0; d < 6; ++d) {
      const int sh = 15 - 3 * d;
      uint32_t even = 0, odd = 0;              // digits + 3 of four elements, as byte selectors
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        even |= (u[2 * i] >> sh & 7u) << (4 * i);
        odd |= (u[2 * i + 1] >> sh & 7u) << (4 * i);
      }
      // codes of -3 .. 4
      const uint32_t word = __byte_perm(0x000A0C0Du, 0x06050402u, even) | __byte_perm(0x000A0C0Du, 0x06050402u, odd) << 4;
      if (k < K) *reinterpret_cast<uint32_t*>(dst + (long long)d * t.T * (K / 2)) = word ^ sign;
    }
  } else {
    e = max(4, (int)(m >> 7) - 7);
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = make_float2(__uint_as_float(v[i] << 16) * inv, __uint_as_float(v[i] & 0xFFFF0000u) * inv);
      const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
      const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
      const float2 d = make_float2((y.x - b.x) * 16.f, (y.y - b.y) * 16.f);
      hi[i / 2] |= (uint32_t)h << (16 * (i & 1));
      lo[i / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(d, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
    }
    uint8_t* dst = codes + ((long long)tile * t.cols + rr) * K + k;
    *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(dst + (long long)t.T * K) = make_uint2(lo[0], lo[1]);
  }
  // the scale bytes of the group's four blocks (infinities and NaN: 255), column c of the row in lane c
  constexpr int kCols = Form<kForm8>::kCols, kLess = kForm8 ? 4 : 3;
  const int byte = m >= 0x7F80u ? 255 : e, c = threadIdx.x & 15;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = __shfl_sync(lanes, byte, 4 * i, 16);
    w |= (uint32_t)(b == 255 ? 255 : b - kLess * c) << (8 * i);
  }
  if (c < kCols) {
    const int at = c * t.T + rr;
    uint8_t* sc = scales + (((long long)tile * groups + k / 128) * t.atoms + at / 128) * 512;
    *reinterpret_cast<uint32_t*>(sc + (at % 32) * 16 + (at % 128) / 32 * 4) = w;
  }
}

template <bool kForm8>
__global__ void __launch_bounds__(256) split_kernel(const bf16* __restrict__ x, int rows, int K, TileShape t,
                                                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                    int32_t* status) {
  const int k = (blockIdx.x * 256 + threadIdx.x) * 8;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (k == 0 && blockIdx.y == 0) *status = 0;
  if (k >= (K + 127) / 128 * 128) return;      // (sixteen lanes together)
  for (int r = blockIdx.y; r < rows; r += gridDim.y)
    split_row<kForm8>(x, r, k, K, t, codes, scales);
}

// ======================================================================== product
// Block-scaled MMA, K = 64 (form 4) or 32 (form 8) a step: scales in tensor memory, two or one of the four
// bytes of a word chosen by the instruction descriptor.
template <bool kForm8>
__device__ __forceinline__ void mma_mx_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  if constexpr (kForm8)
    ptx::mma_mx8_ss(d, a, b, idesc, sfa, sfb, accumulate);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// Untiled copy of `bytes` (a multiple of 16) into shared memory, counted on a barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}

// Instruction descriptor of the block-scaled kinds: bits [4,6) first scale byte of B, [7,10) A format (mxf4: 1 =
// e2m1; mxf8f6f4: 5 = e2m1), [10,13) B format (mxf4: 1; mxf8f6f4: 0 = e4m3), [17,23) N >> 3, bit 23 scales as
// powers of two, [27,29) M >> 7, [29,31) first scale byte of A.
template <bool kForm8>
__device__ __forceinline__ uint32_t idesc_mx(int N) {
  return ((kForm8 ? 5u : 1u) << 7) | ((kForm8 ? 0u : 1u) << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27);
}
constexpr uint32_t kIdescByte = (1u << 4) | (1u << 29);    // one scale byte further, in both

struct ProjectParams {
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  Work work;
  TileShape shape;
  int rows, N, groups;
  bf16* out;
  float* pieces;               // [2 grid][T][128]
  int32_t* status;             // the call's, cleared by the split
  TestWaits test;
};

enum { B_FULL = 0, B_EMPTY = kMaxStages, B_DFULL = 2 * kMaxStages, B_DFREE, B_TEAR, B_COUNT };

template <bool kForm8, int kAtoms>
__global__ void __launch_bounds__(kThreads, 1)
    project_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const ProjectParams p) {
  typedef Form<kForm8> F;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t bars = base + p.shape.stages * p.shape.stage;
  uint8_t* barp = smem_raw + (bars - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(barp + 8 * B_COUNT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(barp + 8 * B_COUNT + 4);
  auto bar = [&](int i) { return bars + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int T = p.shape.T, steps = p.work.steps, stages = p.shape.stages;
  const long long u0 = p.work.start(blockIdx.x), u1 = p.work.start(blockIdx.x + 1);
  const uint32_t off_x = kA, off_sfw = off_x + p.shape.cols * 128, off_sfx = off_sfw + F::kGroups * 512;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) ptx::mbar_init(bar(i), i == B_DFREE ? 4 : 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_w);
    ptx::prefetch_tensormap(&tm_x);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  ptx::griddep_launch_dependents();
  const uint64_t limit = p.test.limit_ns;
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status, limit); };
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = ptx::l2_policy_evict_first();
      // the first codes into L2 while the kernel before ends
      const int tile0 = (int)(u0 / steps);
      int k = (int)(u0 % steps), rt = tile0 % p.work.row_tiles, mt = tile0 / p.work.row_tiles;
      constexpr int kX = kForm8 ? F::kStepK : F::kStepK / 2;   // a step's codes of a column, in the map's elements
      for (int i = k; i < steps && i < k + kPrefetch && i < k + u1 - u0; ++i)
        ptx::tma_prefetch_3d_hint(&tm_w, kX * i, 128 * mt, 0, pol);
      ptx::griddep_wait();
      uint32_t g = 0, st = 0, phase = 1;
      // (the testing hook: no step from a withheld one on, those before it are awaited by their products)
      const long long stop = p.test.withhold > 0 && blockIdx.x == 0 ? min(u1, u0 + p.test.withhold - 1) : u1;
      for (long long u = u0; u < stop; ++u, ++g) {
        const uint32_t dst = base + st * p.shape.stage, full = bar(B_FULL + st);
        if (!wait(B_EMPTY + st, phase)) break;
        const uint32_t n = (uint32_t)min(F::kGroups, p.groups - F::kGroups * k);   // groups of 128 of this step
        ptx::mbar_arrive_expect_tx(full, F::kTx + p.shape.cols * 128 + n * 512 * (1 + kAtoms));
        if (p.work.row_tiles == 1) ptx::tma_load_3d_hint(dst, &tm_w, kX * k, 128 * mt, 0, full, pol);
        else ptx::tma_load_3d(dst, &tm_w, kX * k, 128 * mt, 0, full);
        ptx::tma_load_3d(dst + off_x, &tm_x, 128 * k, 0, rt, full);
        bulk_load(dst + off_sfw, p.w_scales + ((long long)mt * p.groups + F::kGroups * k) * 512, n * 512, full);
        bulk_load(dst + off_sfx, p.x_scales + ((long long)rt * p.groups + F::kGroups * k) * (kAtoms * 512),
                  n * (kAtoms * 512), full);
        if (++st == (uint32_t)stages) {
          st = 0;
          phase ^= 1;
        }
        if (++k == steps) {
          k = 0;
          if (++rt == p.work.row_tiles) {
            rt = 0;
            ++mt;
          }
        }
      }
      if (*abort)
        for (uint32_t i = g > (uint32_t)stages ? g - stages : 0; i < g; ++i)
          drain_wait(bar(B_FULL + i % stages), (i / stages) & 1, limit);
    }
  } else if (warp == 1) {
    ptx::griddep_wait();                                       // (from here on the waits have an end)
    uint32_t st = 0, phase = 0, seg = 0;
    bool ok = true;
    // in units of 16 bytes, as descriptors count
    const uint32_t stage16 = p.shape.stage >> 4;
    const uint64_t desc = ptx::smem_desc(base, 16, 1024, ptx::kSwizzle128);
    const uint64_t scale_desc = ptx::smem_desc(base + off_sfw, 0, 128, ptx::kSwizzleNone);
    const uint32_t idesc = idesc_mx<kForm8>(p.shape.cols);
    int left = p.groups - F::kGroups * (int)(u0 % steps);      // groups of the tile from here on
    for (long long u = u0; ok && u < u1; ++seg) {
      const long long end = min(u1, (u / steps + 1) * steps);
      if (!(ok = wait_w(B_DFREE, (seg & 1) ^ 1))) break;
      const long long first = u;
      for (; u < end; ++u) {
        if (!(ok = wait_w(B_FULL + st, phase))) break;
        ptx::tc_fence_after();
        const uint32_t acc = u > first ? 1u : 0u;
        const uint64_t a = desc + st * stage16, x = a + (off_x >> 4), s = scale_desc + st * stage16;
        const uint32_t sf = tmem + 512 - p.shape.sf * (st + 1);
        const bool half = left < F::kGroups;                   // a last group of 128
        if (ptx::elect_one()) {
          // scale columns: 4 of W per group, then 4 an atom of x per group
#pragma unroll
          for (int i = 0; i < F::kGroups; ++i) {
            if (i == 1 && half) break;
            ptx::tmem_cp_scales(sf + 4 * i, s + 32 * i);
#pragma unroll
            for (int at = 0; at < kAtoms; ++at)
              ptx::tmem_cp_scales(sf + 4 * (F::kGroups + kAtoms * i + at), s + 32 * (F::kGroups + kAtoms * i + at));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i == 2 && half) break;
            const int group = kForm8 ? 0 : i >> 1;
            mma_mx_ss<kForm8>(tmem, a + 2 * i, x + 2 * i, idesc + (kForm8 ? i : 2 * (i & 1)) * kIdescByte, sf + 4 * group,
                              sf + 4 * (F::kGroups + kAtoms * group), i ? 1u : acc);
          }
          ptx::mma_commit(bar(B_EMPTY + st));
          if (u == end - 1) ptx::mma_commit(bar(B_DFULL));
        }
        __syncwarp();
        if (++st == (uint32_t)stages) {
          st = 0;
          phase ^= 1;
        }
        if ((left -= F::kGroups) <= 0) left = p.groups;
      }
    }
    if (*abort) {
      if (ptx::elect_one()) ptx::mma_commit(bar(B_TEAR));
      __syncwarp();
      drain_wait(bar(B_TEAR), 0, limit);
    }
  } else {
    const int quad = warp & 3, col = 32 * quad + lane;         // column of the tile
    const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16);
    ptx::griddep_wait();                                       // the pieces of the call before are read
    uint32_t seg = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1; ++seg) {
      const long long end = min(u1, (u / steps + 1) * steps);
      const int tile = (int)(u / steps), mt = tile / p.work.row_tiles, rt = tile % p.work.row_tiles;
      const bool whole = end - u == steps;
      const int n = 128 * mt + col, r_end = min(T, p.rows - rt * T);
      float* piece = p.pieces + (long long)(2 * blockIdx.x + (u > u0)) * T * 128 + col;
      bf16* out = p.out + (long long)rt * T * p.N + n;
      if (!(ok = wait_w(B_DFULL, seg & 1))) break;
      ptx::tc_fence_after();
      for (int r = 0; r < T; r += 8) {
        uint32_t d[F::kCols][8];
#pragma unroll
        for (int i = 0; i < F::kCols; ++i) ptx::tmem_ld8(t_row + i * T + r, d[i]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v = __uint_as_float(d[F::kCols - 1][i]);
#pragma unroll
          for (int j = F::kCols - 2; j >= 0; --j) v += __uint_as_float(d[j][i]);
          if (r + i >= r_end) break;
          if (!whole) piece[(long long)(r + i) * 128] = v;
          else if (n < p.N) out[(long long)(r + i) * p.N] = __float2bfloat16_rn(v);
        }
        __syncwarp();                                          // the next load is warp-wide
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_DFREE));
      u = end;
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Adds a tile's pieces in the order of its steps; nothing where a CTA gave up before it wrote its own. Block (tile, 8 rows): thread = column and four rows. Bound by
// L2: pieces of 152 CTAs, 4.7 us for 32 rows x 5120 columns, 9 for 512.
__global__ void __launch_bounds__(256) merge_kernel(const Work work, const float* __restrict__ pieces, int rows, int N,
                                                    int T, bf16* __restrict__ out, const int32_t* status) {
  const int tile = blockIdx.x, mt = tile / work.row_tiles, rt = tile % work.row_tiles;
  const int col = threadIdx.x % 128, n = 128 * mt + col;
  const long long s0 = (long long)tile * work.steps;
  const int c0 = work.owner(s0), c1 = work.owner(s0 + work.steps - 1);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (c0 == c1) return;                        // written by its only CTA
  const int32_t gave_up = *status;             // (looked at last: its load is in flight with the pieces')
  const int r0 = 8 * blockIdx.y + 4 * (threadIdx.x / 128), m = min(4, min(T, rows - rt * T) - r0);
  // a CTA that began before this tile (the first one, if any) has it as its second piece
  const float* src = pieces + ((long long)2 * c0 * T + r0) * 128 + col;
  const long long step = (long long)2 * T * 128, second = work.start(c0) < s0 ? (long long)T * 128 : 0;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float* piece = src + (c - c0) * step + (c == c0 ? second : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < m) v[i] += piece[i * 128];
  }
  if (n >= N || gave_up != 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < m) out[(long long)(rt * T + r0 + i) * N + n] = __float2bfloat16_rn(v[i]);
}

}  // namespace mx4

using namespace mx4;

namespace {

// At least two steps a CTA: the pieces of a tile have to be added.
template <bool kForm8>
Work make_work(int K, int N, const TileShape& t) {
  Work w;
  w.steps = (K + Form<kForm8>::kStepK - 1) / Form<kForm8>::kStepK;
  w.row_tiles = t.tiles;
  w.tiles = (N + 127) / 128 * t.tiles;
  w.units = (long long)w.tiles * w.steps;
  const long long most = w.steps > 1 ? (w.units + 1) / 2 : w.units;
  w.grid = (int)(most < device_sms() ? most : device_sms());
  return w;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct ProjectLayout {                         // (behind the status word)
  size_t codes, scales, pieces, total;
};
template <bool kForm8>
ProjectLayout project_layout(int K, const TileShape& t, int grid) {
  ProjectLayout l;
  l.codes = 256;
  l.scales = up256(l.codes + (size_t)t.tiles * t.cols * (kForm8 ? K : K / 2));
  l.pieces = up256(l.scales + (size_t)t.tiles * ((K + 127) / 128) * t.atoms * 512);
  l.total = up256(l.pieces + (size_t)2 * grid * t.T * 128 * 4);
  return l;
}

template <bool kForm8>
size_t project_workspace(int K, int N, int rows) {
  const TileShape t = tile_shape<kForm8>(rows);
  return project_layout<kForm8>(K, t, make_work<kForm8>(K, N, t).grid).total;
}

template <bool kForm8>
cudaError_t project(const void* x, const void* codes, const void* scales, int K, int N, int rows, void* out,
                    void* workspace, const TestWaits& test, cudaStream_t s) {
  const TileShape t = tile_shape<kForm8>(rows);
  ProjectParams p;
  p.work = make_work<kForm8>(K, N, t);
  const ProjectLayout l = project_layout<kForm8>(K, t, p.work.grid);
  uint8_t* ws = (uint8_t*)workspace;
  p.shape = t;
  p.w_scales = (const uint8_t*)scales;
  p.x_scales = ws + l.scales;
  p.rows = rows;
  p.N = N;
  p.groups = (K + 127) / 128;
  p.out = (bf16*)out;
  p.pieces = (float*)(ws + l.pieces);
  p.status = (int32_t*)workspace;
  p.test = test;
  CUtensorMap tw, tx;
  const uint64_t row = (uint64_t)K / 2, x_row = kForm8 ? K : K / 2;
  if (!tensor_map_3d(&tw, kForm8 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     CU_TENSOR_MAP_SWIZZLE_128B, codes, kForm8 ? (uint64_t)K : row, (uint64_t)N, 1, row, (uint64_t)N * row,
                     128, 128) ||
      !tensor_map_3d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, ws + l.codes, x_row,
                     (uint64_t)t.cols, (uint64_t)t.tiles, x_row, t.cols * x_row, 128, (uint32_t)t.cols))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)t.stages * t.stage + kBarBytes;
  auto kern = t.atoms == 2 ? project_tc_kernel<kForm8, 2> : project_tc_kernel<kForm8, 1>;
  cudaError_t e = allow_smem(kern, smem);
  if (e == cudaSuccess)
    e = launch_pdl(split_kernel<kForm8>, dim3((unsigned)((K + 2047) / 2048), (unsigned)(rows < 32768 ? rows : 32768), 1), 256, 0, s, (const bf16*)x,
                   rows, K, t, ws + l.codes, ws + l.scales, p.status);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3((unsigned)p.work.grid, 1, 1), kThreads, smem, s, tw, tx, p);
  if (e == cudaSuccess)
    e = launch_pdl(merge_kernel, dim3((unsigned)p.work.tiles, (unsigned)((t.T + 7) / 8), 1), 256, 0, s, p.work,
                   (const float*)p.pieces, rows, N, t.T, (bf16*)out, (const int32_t*)p.status);
  return e;
}

// Form 8 for more rows than one tile of form 4 takes (measured above); its unpacking load wants rows of a
// multiple of 64 bytes.
bool form8_fits(int K, int rows) { return rows > Form<false>::kMaxT && K % 128 == 0; }

}  // namespace

bool mx4_project_tc_supported(mla_dtype act) { return act == MLA_BF16; }

size_t mx4_project_tc_workspace(int K, int N, int rows) {
  const size_t four = project_workspace<false>(K, N, rows);
  if (!form8_fits(K, rows)) return four;
  const size_t eight = project_workspace<true>(K, N, rows);
  return eight > four ? eight : four;          // (which one runs depends on the codes' address too)
}

cudaError_t launch_mx4_project_tc(const void* x, const void* codes, const void* scales, int K, int N, int rows,
                                  void* out, void* workspace, const TestWaits& test, cudaStream_t s) {
  if (form8_fits(K, rows) && ((uintptr_t)codes & 31) == 0)
    return project<true>(x, codes, scales, K, N, rows, out, workspace, test, s);
  return project<false>(x, codes, scales, K, N, rows, out, workspace, test, s);
}

}  // namespace mla
