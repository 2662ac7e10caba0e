// Decode over chosen pages on the tensor cores (bf16 activations, every bf16 and fp8 cache, 64-token pages,
// d_c 512, d_r 64, a multiple of 16 heads).
//
// A CTA has a block of up to 64 heads and walks its work items (ranges of one query token's list) two pages,
// 128 tokens, at a time, with tokens in the rows of the first product and latent dims in those of
// the second:
//   S^T = X q_lat^T         (M = 128 tokens, N = heads, K = 576)
//   P   = 2^(c S - r_h)     (c = softmax scale * log2 e, r_h a running reference of the head)
//   O^T += C^T P^T          (M = 4 x 128 latent dims, N = heads, K = 128 tokens)
// 64 heads by 512 dims of fp32 sums are half of tensor memory, and 64 heads of the query a third of shared
// memory: scores are whole fp32 sums of exact products, with nothing to exchange between CTAs (the decode
// over all pages splits the latent dims of 128 heads over two CTAs and exchanges partial scores in fp16,
// which costs the LSE its last bits). The reference r_h moves only when a score exceeds it by 8 (log2
// units); P is formed under the old one meanwhile, and the barrier that hands P over tells all warps
// whether it holds. If not, references, O and sums are rescaled and P is formed again.
//
// bf16 cache: the staged rows are both products' operands (K-major rows of S^T, dims-major columns of O^T);
// P is rounded to bf16 (the type of the rows, which both operands of an MMA share; the sums count the unrounded
// weights) and takes the place of the tile's rotary keys, which S^T has used up.
// fp8 caches: the codes themselves are the operands (kind::f8f6f4). The query is the sum of two e4m3 terms
// under a power of two per head (two columns of S^T, split4). So is P, under a power of two per head and 32
// tokens (kind::mxf8f6f4, which applies it): y = hi + lo / 16, the largest y of the 32 between 2^7 and 2^8.5, so a
// weight is off by 2^-9 of itself or 2^-21 of the largest of the 32, whatever came before it. Under one power of two for the
// whole list, what lay 2^-14 below the largest weight was lost: a heavy first token in front of 6000 others had them
// as 0. Such a P has no reference to try either: the sums' and scales' own moves when one exceeds it by 2^64.
// Block-scaled rows: each block of 128 dims has a product of its own in S^T, added under the token's scale in
// registers, and a P of its own, times that scale, in O^T; the 32 tokens' power of two covers the largest weight and
// the largest scale.
//
// Bound: the load, product, softmax, product chain of a tile, whose rows fill shared memory (bf16: 2.6 us a
// tile); e4m3: the MMAs (64 columns as long as 128 would) and, as long again, the way from scores to P. 32
// queries of 64 pages, 128 heads, a cold L2: bf16 71 us (151 MB), e4m3 61, block scales 102. 64 x 2 queries of 96
// pages, e4m3: 192. (Under one power of two for the list, without the maxima of every 32 tokens: 59, 93 and 181.)
#include <math.h>

#include "fp8_tiles.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace pdec {

enum { kBf16 = 0, kE4m3 = 1, kB128 = 2 };
constexpr int kTok = 128;
constexpr int kChunk = kTok * 128;             // 128 bytes of 128 rows
constexpr int kThreads = 576;                  // producer, MMA issuer, 16 softmax warps
constexpr float kGrow = 8.75f;                 // how far scores may exceed the reference (log2)
constexpr float kGrow8 = 64.f;                 // fp8: and scales of P, which fp32 sums hold by themselves

template <int kFmt> struct Fmt;
template <> struct Fmt<kBf16> {                // latent chunks of a tile, chunk buffers, bytes of the regions, score buffers
  static constexpr int kChunks = 8, kBufs = 8, kQ = 9 * 8192, kRope = kChunk, kP = 0, kAtoms = 0, kSBufs = 2;
};
template <> struct Fmt<kE4m3> {
  static constexpr int kChunks = 4, kBufs = 8, kQ = 4 * kChunk + 8192, kRope = 8192, kP = kChunk, kAtoms = 1, kSBufs = 1;
};
template <> struct Fmt<kB128> {
  static constexpr int kChunks = 4, kBufs = 4, kQ = 4 * kChunk + 8192, kRope = kChunk, kP = 4 * kChunk, kAtoms = 6, kSBufs = 2;
};

template <int kFmt> struct Layout {
  typedef Fmt<kFmt> F;
  static constexpr int kRing = F::kQ;
  static constexpr int kRope = kRing + F::kBufs * kChunk;
  static constexpr int kP = kFmt == kBf16 ? kRope : kRope + F::kRope;      // (bf16: over the rotary keys)
  static constexpr int kAlpha = kRope + F::kRope + F::kP;                  // [64] rescaling factors
  static constexpr int kHead = kAlpha + 256;                               // [64] factors of the fp8 query
  static constexpr int kWarp = kHead + 256;                                // [4][64] of the four token quarters
  static constexpr int kRef = kWarp + 1024;                                // [64] references
  static constexpr int kBar = kRef + 256;
  static constexpr int kSf = kBar + 256;                                   // scale atoms of P (fp8), then constant ones
  static constexpr int kUsed = kSf + F::kAtoms * 512;
  // what rounding the base up to 1024 may take; e4m3 has no room for it (a base off that is refused)
  static constexpr int kSmem = kUsed + 1024 <= 232448 ? kUsed + 1024 : 232448;
  static_assert(kUsed <= kSmem, "dynamic shared memory per CTA");
};

enum { B_CFULL = 0, B_CFREE = 8, B_RFULL = 16, B_RFREE, B_QFULL, B_QFREE, B_SFULL, B_SFREE = B_SFULL + 2,
       B_PFULL = B_SFREE + 2, B_PAGAIN, B_OFREE, B_MEET, B_PDONE, B_TEAR, B_COUNT };
static_assert(B_COUNT * 8 <= 240, "barrier area");

struct Maps {
  CUtensorMap c, rope, q;
};

// kind::f8f6f4, e4m3 A and B with their majors
constexpr uint32_t idesc_e4m3(int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// kind::mxf8f6f4, e4m3 A and B in the order of their MN dimensions, scales as powers of two; the scale byte of
// a step of 32 tokens is its own (kIdescByte further).
constexpr uint32_t idesc_mx_e4m3(int N) {
  return (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27);
}
constexpr uint32_t kIdescByte = (1u << 4) | (1u << 29);

// 2^x of a whole x, 0 below 2^-126.
__device__ __forceinline__ float pow2(float x) {
  return __uint_as_float((uint32_t)((int)fminf(fmaxf(x, -127.f), 127.f) + 127) << 23);
}
// The byte of a scale 2^x, at the ends of its range the end.
__device__ __forceinline__ uint8_t scale_byte(float x) { return (uint8_t)((int)fminf(fmaxf(x, -127.f), 127.f) + 127); }

// Sums over the warp's lanes of 16 columns: lanes j and j + 16 are left with column j.
__device__ __forceinline__ float column_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float give = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}
// The largest value of the warp's lanes (NaN only if all are).
__device__ __forceinline__ float warp_most(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1)
    decode_pages_kernel(const __grid_constant__ Maps maps, const DecodeParams p, int blocks) {
  typedef Fmt<kFmt> F;
  typedef Layout<kFmt> L;
  constexpr bool kFp8 = kFmt != kBf16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw + L::kUsed > L::kSmem) {
    ptx::griddep_wait();
    if (threadIdx.x == 0) flag_status(p.status, MLA_ERR_CUDA);
    return;
  }
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + L::kBar + 240);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + L::kBar + 244);
  volatile int* grown = reinterpret_cast<volatile int*>(basep + L::kBar + 248);      // [2]
  auto bar = [&](int i) { return base + L::kBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int worker = blockIdx.x / blocks, h0 = 64 * (blockIdx.x % blocks), N = min(64, p.H - h0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      ptx::mbar_init(bar(i), (i >= B_SFREE && i <= B_MEET) || (kFp8 && i == B_QFULL) ? 16 : 1);
    *abort = 0;
    grown[0] = grown[1] = -1;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&maps.c);
    ptx::prefetch_tensormap(&maps.rope);
    ptx::prefetch_tensormap(&maps.q);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if constexpr (kFmt == kB128) {               // scales of 1 and of 1 / 16
    if (threadIdx.x < 256)
      reinterpret_cast<uint32_t*>(basep + L::kSf + 4 * 512)[threadIdx.x] = threadIdx.x < 128 ? 0x7F7F7F7Fu : 0x7B7B7B7Bu;
    ptx::fence_proxy_async_smem();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // O: 4 x 64 columns; S: 2 x 128. P's scales (of A, for the terms' 1 and 1 / 16, then of B): e4m3, which has one S
  // buffer, behind it; block scales in an S buffer, between a tile's scores and the next tile's
  const uint32_t t_o = tmem, t_s = tmem + 256, t_sf = tmem + 384;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();                         // the plan and the lists' pages
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  const int it0 = p.worker_off[worker], it1 = p.worker_off[worker + 1];

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = ptx::l2_policy_evict_first();
      const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.cache);
      const uint32_t page_bytes = (uint32_t)(64 * p.row_bytes);
      uint32_t c_seq = 0, tile = 0, q_seq = 0;
      bool ok = true;
      for (int it = it0; ok && it < it1; ++it, ++q_seq) {
        const WorkItem item = p.items[it];
        const int32_t* bt = p.block_table + (long long)item.group * p.max_pages;
        const int pg0 = 2 * item.page_begin, pg1 = min(2 * item.page_end, (item.kv + 63) / 64);
        auto page_of = [&](int pg) {
          if (pg >= pg1) return -1;
          const int page = bt[pg];
          if (page >= 0 && page < p.num_pages) return page;
          flag_status(p.status, MLA_ERR_DEVICE_GUARD);
          return 0;
        };
        if constexpr (!kFp8) {
          if (!(ok = wait(B_QFREE, (q_seq & 1) ^ 1))) break;
          const int rows = min(64, p.H);       // (rows behind the last head read as zero)
          ptx::mbar_arrive_expect_tx(bar(B_QFULL), 9 * rows * 128);
          for (int c = 0; c < 9; ++c) ptx::tma_load_3d(base + 8192 * c, &maps.q, 64 * c, h0, item.group, bar(B_QFULL));
        }
        if (it + 1 < it1)                      // the next item's query into L2
          ptx::bulk_prefetch_l2(reinterpret_cast<const bf16*>(p.q_lat) + ((long long)p.items[it + 1].group * p.H + h0) * 576,
                                (uint32_t)(N * 1152));
        int a = page_of(pg0), b = page_of(pg0 + 1);
        for (int pg = pg0; ok && pg < pg1; pg += 2, ++tile) {
          const int na = page_of(pg + 2), nb = page_of(pg + 3);
          if (h0 == 0) {                       // the next tile's pages into L2
            if (na >= 0) ptx::bulk_prefetch_l2_hint(cache + (long long)na * page_bytes, page_bytes, pol);
            if (nb >= 0) ptx::bulk_prefetch_l2_hint(cache + (long long)nb * page_bytes, page_bytes, pol);
          }
          auto load = [&](uint32_t dst, const CUtensorMap* map, int x, uint32_t half, uint32_t full) {
            ptx::mbar_arrive_expect_tx(full, b >= 0 ? 2 * half : half);
            ptx::tma_load_3d(dst, map, x, a * 64, 0, full);
            if (b >= 0) ptx::tma_load_3d(dst + half, map, x, b * 64, 0, full);
          };
          for (int c = 0; c < F::kChunks; ++c, ++c_seq) {
            const uint32_t st = c_seq % F::kBufs;
            if (!(ok = wait(B_CFREE + st, ((c_seq / F::kBufs) & 1) ^ 1))) break;
            load(base + L::kRing + st * kChunk, &maps.c, (kFp8 ? 128 : 64) * c, kChunk / 2, bar(B_CFULL + st));
          }
          if (!ok || !(ok = wait(B_RFREE, (tile & 1) ^ 1))) break;
          load(base + L::kRope, &maps.rope, kFmt == kB128 ? 528 : 512, kFmt == kE4m3 ? 4096 : kChunk / 2, bar(B_RFULL));
          a = na;
          b = nb;
        }
      }
      if (*abort) {                            // the last copies into each buffer have landed
        for (uint32_t i = c_seq > (uint32_t)F::kBufs ? c_seq - F::kBufs : 0; i < c_seq; ++i)
          drain_wait(bar(B_CFULL + i % F::kBufs), (i / F::kBufs) & 1);
        if (tile) drain_wait(bar(B_RFULL), (tile - 1) & 1);
        if (!kFp8 && q_seq) drain_wait(bar(B_QFULL), (q_seq - 1) & 1);
        if (!kFp8) drain_wait(bar(B_QFULL), q_seq & 1);
      }
    }
  } else if (warp == 1) {
    // In one place tiles follow each other as S(0), [S(i + 1),] O(i), .. where the ring holds two tiles, and
    // S(i), O(i) where it holds one.
    constexpr bool kAhead = F::kBufs >= 2 * F::kChunks;
    constexpr uint32_t kQStep = kFp8 ? kChunk : 8192;      // bytes of a chunk's query rows
    const uint32_t id_s = kFp8 ? idesc_e4m3(2 * N, false, false) : ptx::idesc_bf16_f32(128, N, false, false);
    const uint32_t id_r = kFmt == kB128 ? ptx::idesc_bf16_f32(128, N, false, false) : id_s;
    const uint32_t id_o = kFp8 ? idesc_mx_e4m3(N) : ptx::idesc_bf16_f32(128, N, true, true);
    const uint64_t sf_d = ptx::smem_desc(base + L::kSf, 0, 128, ptx::kSwizzleNone);
    const uint64_t q_d = ptx::smem_desc(base, 16, 1024, ptx::kSwizzle128);
    const uint64_t x_d = ptx::smem_desc(base + L::kRing, 16, 1024, ptx::kSwizzle128);
    constexpr uint32_t kRopeSw = kFmt == kE4m3 ? (uint32_t)ptx::kSwizzle64 : (uint32_t)ptx::kSwizzle128;
    constexpr uint32_t kRopeSbo = kFmt == kE4m3 ? 512 : 1024;
    const uint64_t qr_d = ptx::smem_desc(base + (kFp8 ? 4 * kChunk : 8 * 8192), 16, kRopeSbo, kRopeSw);
    const uint64_t xr_d = ptx::smem_desc(base + L::kRope, 16, kRopeSbo, kRopeSw);
    // dims-major: two chunks of 64 dims (bf16) or one of 128; P by heads
    const uint64_t c_d = ptx::smem_desc(base + L::kRing, kChunk, 1024, ptx::kSwizzle128);
    const uint64_t p_d = kFp8 ? ptx::smem_desc(base + L::kP, 16, 512, ptx::kSwizzle64)
                              : ptx::smem_desc(base + L::kP, 16, 1024, ptx::kSwizzle128);
    uint32_t c_seq = 0, o_seq = 0, s_tile = 0, s_seq = 0, o_tile = 0, q_seq = 0, again = 0;
    bool ok = true;
    auto product_s = [&](bool last) {
      for (int c = 0; ok && c < F::kChunks; ++c, ++c_seq) {
        const uint32_t st = c_seq % F::kBufs, sb = s_seq % F::kSBufs;
        if (c == 0 || kFmt == kB128) ok = wait_w(B_SFREE + sb, ((s_seq / F::kSBufs) & 1) ^ 1);
        // (the buffer that held the scales of the tile before)
        if (ok && kFmt == kB128 && c == 1 && o_tile > 0) ok = wait_w(B_PDONE, (o_tile - 1) & 1);
        if (!ok || !(ok = wait_w(B_CFULL + st, (c_seq / F::kBufs) & 1))) return;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t a = x_d + (st * (kChunk >> 4) + 2 * k), b = q_d + (c * (kQStep >> 4) + 2 * k);
            const uint32_t acc = k || (c && kFmt != kB128) ? 1u : 0u;
            if (kFp8) ptx::mma_e4m3_ss(t_s + 128 * sb, a, b, id_s, acc);
            else ptx::mma_bf16_ss(t_s + 128 * sb, a, b, id_s, acc);
          }
          if (kFmt == kB128) ptx::mma_commit(bar(B_SFULL + sb));
        }
        __syncwarp();
        if (kFmt == kB128) ++s_seq;
      }
      const uint32_t sb = s_seq % F::kSBufs;
      if (kFmt == kB128) ok = wait_w(B_SFREE + sb, ((s_seq / F::kSBufs) & 1) ^ 1);
      if (!ok || !(ok = wait_w(B_RFULL, s_tile & 1))) return;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < (kFmt == kE4m3 ? 2 : 4); ++k) {
          const uint32_t acc = k || kFmt != kB128 ? 1u : 0u;
          if (kFmt == kE4m3) ptx::mma_e4m3_ss(t_s + 128 * sb, xr_d + 2 * k, qr_d + 2 * k, id_r, acc);
          else ptx::mma_bf16_ss(t_s + 128 * sb, xr_d + 2 * k, qr_d + 2 * k, id_r, acc);
        }
        ptx::mma_commit(bar(B_SFULL + sb));
        if (kFp8) ptx::mma_commit(bar(B_RFREE));
        if (!kFp8 && last) ptx::mma_commit(bar(B_QFREE));
      }
      __syncwarp();
      ++s_seq;
      ++s_tile;
    };
    for (int it = it0; ok && it < it1; ++it, ++q_seq) {
      const WorkItem item = p.items[it];
      const int tiles = item.page_end - item.page_begin;
      if (!(ok = wait_w(B_QFULL, q_seq & 1))) break;
      if (kAhead) product_s(tiles == 1);
      for (int i = 0; ok && i < tiles; ++i, ++o_tile) {
        if (!kAhead) product_s(i == tiles - 1);
        else if (i + 1 < tiles) product_s(i + 2 == tiles);
        if (!ok || !(ok = wait_w(B_PFULL, o_tile & 1))) break;
        if (i > 0 && grown[o_tile & 1] == (int)o_tile && !(ok = wait_w(B_PAGAIN, again++ & 1))) break;
        if (i == 0 && !(ok = wait_w(B_OFREE, (q_seq & 1) ^ 1))) break;
        ptx::tc_fence_after();
        const uint32_t sf = kFmt == kB128 ? t_s + 128 * ((s_seq + 1) & 1) : t_sf;
        if (ptx::elect_one()) {
          const uint32_t acc0 = i ? 1u : 0u;
          if constexpr (kFmt == kE4m3) {
            ptx::tmem_cp_scales(sf + 8, sf_d);
          } else if constexpr (kFmt == kB128) {
#pragma unroll
            for (int k = 0; k < 2; ++k) ptx::tmem_cp_scales(sf + 4 * k, sf_d + 32 * (4 + k));
#pragma unroll
            for (int m = 0; m < 4; ++m) ptx::tmem_cp_scales(sf + 8 + 4 * m, sf_d + 32 * m);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t st = o_seq % F::kBufs;
            const uint64_t a = c_d + st * (kChunk >> 4);
            if (!kFp8) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                ptx::mma_bf16_ss(t_o + 64 * m, a + 128 * k, p_d + 128 * k, id_o, k ? 1u : acc0);
              ptx::mma_commit(bar(B_CFREE + st));
              ptx::mma_commit(bar(B_CFREE + st + 1));
              o_seq += 2;
            } else {
              const uint64_t pm = p_d + (kFmt == kB128 ? m * (kChunk >> 4) : 0);
              const uint32_t sfb = sf + 8 + (kFmt == kB128 ? 4 * m : 0);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                ptx::mma_mx8_ss(t_o + 64 * m, a + 256 * k, pm + 128 * k, id_o + k * kIdescByte, sf, sfb, k ? 1u : acc0);
                ptx::mma_mx8_ss(t_o + 64 * m, a + 256 * k, pm + (8192 >> 4) + 128 * k, id_o + k * kIdescByte, sf + 4, sfb, 1u);
              }
              ptx::mma_commit(bar(B_CFREE + st));
              o_seq += 1;
            }
          }
          if (!kFp8) ptx::mma_commit(bar(B_RFREE));
          ptx::mma_commit(bar(B_PDONE));
        }
        o_seq = __shfl_sync(0xffffffffu, (uint32_t)((o_tile + 1) * F::kChunks), 0);
      }
    }
    if (*abort) {
      if (ptx::elect_one()) ptx::mma_commit(bar(B_TEAR));
      __syncwarp();
      drain_wait(bar(B_TEAR), 0);
    }
  } else {
    // four threads a token: heads 16 part .. of the block (parts behind the last head have none, but their
    // share of O, the dims tile 128 part)
    const int quad = warp & 3, part = (warp - 2) >> 2, tok = 32 * quad + lane, hp = 16 * part;
    const bool heads = hp < N;
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    float* alpha = reinterpret_cast<float*>(basep + L::kAlpha);
    float* head = reinterpret_cast<float*>(basep + L::kHead);
    float* quarter = reinterpret_cast<float*>(basep + L::kWarp);         // [4][64]
    float* ref = reinterpret_cast<float*>(basep + L::kRef);              // [64] (from registers, which spilled, bf16 took 75 us, not 71)
    uint32_t s_seq = 0, tile = 0, meets = 0, c_seq = 0;
    bool ok = true;
    uint8_t* scale = basep + L::kSf + ((hp + lane) & 31) * 16 + ((hp + lane) >> 5) * 4 + quad;   // (lanes 0 .. 15)
    if constexpr (kFmt == kE4m3) {             // P's terms count 1 and 1 / 16 (four words of each; the rest is not read)
      if (part == 0) {
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = k < 4 ? 0x7F7F7F7Fu : 0x7B7B7B7Bu;
        ptx::tmem_st16(t_sf + lane_off, v);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
      }
    }
    auto meet = [&]() {                        // the sixteen warps (bounded, unlike a named barrier)
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_MEET));
      return wait_w(B_MEET, meets++ & 1);
    };
    for (int it = it0; ok && it < it1; ++it) {
      const WorkItem item = p.items[it];
      const long long g = item.group;
      if constexpr (kFp8) {
        // the query of these heads as two e4m3 terms (the scores of the item before have all been read, so
        // its products are done): a warp takes heads in turn, 16 latent elements and 2 rotary ones a lane
        for (int h = warp - 2; h < N; h += 16) {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(p.q_lat) + (g * p.H + h0 + h) * 576);
          const uint4 x = src[2 * lane], y = src[2 * lane + 1];
          const uint32_t pe = reinterpret_cast<const uint32_t*>(src + 64)[lane];
          const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          uint32_t m2 = kFmt == kB128 ? 0u : pe & 0x7FFF7FFFu;
#pragma unroll
          for (int k = 0; k < 8; ++k) m2 = __vmaxu2(m2, v[k] & 0x7FFF7FFFu);
          const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16)) << 16);
          // 2^e m in [128, 256) (exponents clamped: an all-zero or tiny head stays finite)
          const int ex = max(-110, min(120, (int)((__float_as_uint(m) >> 23) & 255) - 127));
          const float s = __uint_as_float((uint32_t)(-1 - ex + 127) << 23);
          const float inv = __uint_as_float((uint32_t)(ex - 7 + 127) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split4(v[2 * k], v[2 * k + 1], s, &hi[k], &lo[k]);
          uint8_t* q = basep + (lane >> 3) * kChunk;
          const int unit = lane & 7, r1 = h + N;
          *reinterpret_cast<uint4*>(q + h * 128 + ((unit ^ (h & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(q + r1 * 128 + ((unit ^ (r1 & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          uint8_t* qp = basep + 4 * kChunk;
          if (kFmt == kB128) {
            *reinterpret_cast<uint32_t*>(qp + h * 128 + (((lane >> 2) ^ (h & 7)) << 4) + 4 * (lane & 3)) = pe;
          } else {
            uint32_t pe_hi, pe_lo;
            split4(pe, 0u, s, &pe_hi, &pe_lo);
            *reinterpret_cast<uint16_t*>(qp + h * 64 + (((lane >> 3) ^ ((h >> 1) & 3)) << 4) + 2 * (lane & 7)) = (uint16_t)pe_hi;
            *reinterpret_cast<uint16_t*>(qp + r1 * 64 + (((lane >> 3) ^ ((r1 >> 1) & 3)) << 4) + 2 * (lane & 7)) = (uint16_t)pe_lo;
          }
          // infinities and NaN in the query make its scores NaN
          if (lane == 0) head[h] = (kFmt == kE4m3 ? inv * p.scale_log2 : inv) + (m < INFINITY ? 0.f : m - m);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(B_QFULL));
      }
      if (kFp8 && !(ok = wait_w(B_QFULL, (uint32_t)(it - it0) & 1))) break;
      float sum[16];                           // of this thread's heads
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[j] = 0.f;
      for (int pg = 2 * item.page_begin; ok && pg < 2 * item.page_end; pg += 2, ++tile, c_seq += F::kChunks) {
        const int left = min(kTok, item.kv - pg * 64);                   // tokens of this tile
        const bool first = pg == 2 * item.page_begin;
        const bool live = tok < left;
        float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
        int fe[4] = {0, 0, 0, 0};
        if constexpr (kFmt == kB128) {
          if (live) {
            int page = p.block_table[g * p.max_pages + pg + (tok >> 6)];
            if (page < 0 || page >= p.num_pages) page = 0;               // (flagged by the producer)
            sc = *reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(p.cache) +
                                                  ((long long)page * 64 + (tok & 63)) * p.row_bytes + 512);
          }
          // powers of two above the 32 tokens' scales of each 128 dims (while the first scores are formed)
          const float f[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
          for (int m = 0; m < 4; ++m)
            fe[m] = min(126, (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(f[m]) & 0x7FFFFFFFu) >> 23) - 126);
        }
        // scores of this thread's heads, in log2 units
        float s[16];
#pragma unroll
        for (int c = 0; c < (kFmt == kB128 ? 5 : 1); ++c) {
          const uint32_t sb = s_seq % F::kSBufs, at = t_s + lane_off + 128 * sb + hp;
          if (ok) ok = wait_w(B_SFULL + sb, (s_seq / F::kSBufs) & 1);
          if (ok) {
            ptx::tc_fence_after();
            uint32_t hi[16], lo[16];
            if (heads) {
              ptx::tmem_ld16(at, hi);
              if (kFp8 && c < 4) ptx::tmem_ld16(at + N, lo);
              ptx::tmem_wait_ld();
            }
            const float f = c == 0 ? sc.x : (c == 1 ? sc.y : (c == 2 ? sc.z : sc.w));
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              float4 fac4 = make_float4(0.f, 0.f, 0.f, 0.f);
              if (kFmt == kE4m3 || c == 4) fac4 = *reinterpret_cast<const float4*>(head + hp + k);
              const float fac[4] = {fac4.x, fac4.y, fac4.z, fac4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x = heads ? __uint_as_float(hi[k + i]) : 0.f;
                if (kFmt == kBf16) {
                  s[k + i] = x * p.scale_log2;
                } else if (c == 4) {
                  s[k + i] = fmaf(s[k + i], fac[i], x) * p.scale_log2;
                } else {
                  const float v = fmaf(heads ? __uint_as_float(lo[k + i]) : 0.f, 0.0625f, x);
                  if (kFmt == kE4m3) s[k + i] = v * fac[i];
                  else s[k + i] = c ? fmaf(f, v, s[k + i]) : f * v;
                }
              }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_SFREE + sb));
            ++s_seq;
          }
        }
        if (!ok) break;
        if (!live) {                           // rows that may hold anything: their P is 0, 0 times NaN is not
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (int c = part; c < F::kChunks; c += 4) {
            uint4* row = reinterpret_cast<uint4*>(basep + L::kRing + (c_seq + c) % F::kBufs * kChunk + tok * 128);
#pragma unroll
            for (int k = 0; k < 8; ++k) row[k] = zero;
          }
        }
        auto hand_over = [&](int b) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(b));
        };
        // O of the tiles before, times the heads' alpha
        auto rescale = [&]() {
          ptx::tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < N; h += 16) {                // this warp's dims tile
            uint32_t v[16];
            const uint32_t at = t_o + lane_off + 64 * part + h;
            ptx::tmem_ld16(at, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha[h + k]);
            ptx::tmem_st16(at, v);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
        };
        uint8_t* prow = basep + L::kP;
        if constexpr (kFp8) {
          // A head's weights of the warp's 32 tokens, which are the K of one MMA, have a power of two of their own: the
          // largest is 2^7 to 2^8.5 of it (block scales: with the largest scale of each 128 dims in it as well).
          // Lane j keeps head j's.
          float k8 = 0.f, far = 0.f;
          {
            float m[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              m[j] = warp_most(live ? s[j] : -INFINITY);
              far = fmaxf(far, fabsf(m[j]));
            }
            if (far < 4194304.f) {             // to the nearest whole number
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float k = (m[j] + 12582912.f) - 12582920.f;
                s[j] -= k;
                if (lane == j) k8 = k;
              }
            } else {                           // no token, or scores that have no fractions
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float k = ceilf(fmaxf(m[j], -3.0e38f)) - 8.f;
                s[j] -= k;
                if (lane == j) k8 = k;
              }
            }
          }
          if constexpr (kFmt == kB128) {
            float* f[4] = {&sc.x, &sc.y, &sc.z, &sc.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) *f[m] *= __uint_as_float((uint32_t)(127 - fe[m]) << 23);
          }
          const float top = k8 + (float)max(max(fe[0], fe[1]), max(fe[2], fe[3]));
          if (first) {                         // the item's reference: the largest of the four warps
            if (heads && lane < 16) quarter[64 * quad + hp + lane] = top;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_MEET));
          }
          // (the products with the tile before's P have to be done; e4m3: once the terms are formed)
          if (kFmt == kB128 && tile > 0 && !(ok = wait_w(B_PDONE, (tile - 1) & 1))) break;
          uint32_t terms[2][4];                // e4m3: both terms of P
          if (heads) {
#pragma unroll
            for (int j = 0; j < 16; j += 8) {
#pragma unroll
              for (int k = 0; k < 8; ++k) s[j + k] = live ? ptx::ex2(s[j + k]) : 0.f;
              const int hb = hp + j;           // first head of the eight
              const uint32_t at = tok * 64 + (((hb >> 4) ^ ((tok >> 1) & 3)) << 4) + (hb & 8);
#pragma unroll
              for (int m = 0; m < (kFmt == kB128 ? 4 : 1); ++m) {
                const float f = kFmt == kE4m3 ? 1.f : (m == 0 ? sc.x : (m == 1 ? sc.y : (m == 2 ? sc.z : sc.w)));
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 y = make_float2(f * s[j + 2 * k], f * s[j + 2 * k + 1]);
                  const uint32_t c = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                  const float2 b = e4m3x2_to_f32(c);
                  const uint32_t d = __nv_cvt_float2_to_fp8x2(make_float2((y.x - b.x) * 16.f, (y.y - b.y) * 16.f),
                                                              __NV_SATFINITE, __NV_E4M3);
                  hi[k >> 1] |= c << (16 * (k & 1));
                  lo[k >> 1] |= d << (16 * (k & 1));
                }
                if (kFmt == kB128) {
                  *reinterpret_cast<uint2*>(prow + m * kChunk + at) = make_uint2(hi[0], hi[1]);
                  *reinterpret_cast<uint2*>(prow + m * kChunk + 8192 + at) = make_uint2(lo[0], lo[1]);
                } else {
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    terms[0][j / 4 + k] = hi[k];
                    terms[1][j / 4 + k] = lo[k];
                  }
                }
              }
            }
          }
          if constexpr (kFmt == kE4m3) {
            if (tile > 0 && !(ok = wait_w(B_PDONE, (tile - 1) & 1))) break;
            if (heads) {
              uint8_t* at = prow + tok * 64 + (((hp >> 4) ^ ((tok >> 1) & 3)) << 4);
              *reinterpret_cast<uint4*>(at) = make_uint4(terms[0][0], terms[0][1], terms[0][2], terms[0][3]);
              *reinterpret_cast<uint4*>(at + 8192) = make_uint4(terms[1][0], terms[1][1], terms[1][2], terms[1][3]);
            }
          }
          if (first && !(ok = wait_w(B_MEET, meets++ & 1))) break;
          // The scales and sums count from the head's reference, which moves only when one exceeds it by 2^64.
          auto four = [&]() {
            const float* x = quarter + hp + lane;
            return fmaxf(fmaxf(x[0], x[64]), fmaxf(x[128], x[192]));
          };
          auto put = [&](float r) {
#pragma unroll
            for (int m = 0; m < (kFmt == kB128 ? 4 : 1); ++m) scale[512 * m] = scale_byte(k8 - r + (float)fe[m]);
          };
          float r = 0.f, w = 0.f;
          bool over = false;
          if (heads && lane < 16) {
            if (first) ref[hp + lane] = r = four();        // (the four warps of these heads write the same)
            else over = top - (r = ref[hp + lane]) > kGrow8;
            put(r);
            w = over ? 0.f : pow2(k8 - r);
          }
          over = __any_sync(0xffffffffu, over);
          if (over && lane == 0) grown[tile & 1] = (int)tile;
          hand_over(B_PFULL);
          if (heads) {
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[j] = fmaf(s[j], __shfl_sync(0xffffffffu, w, j), sum[j]);
          }
          if (!first) {
            if (!(ok = wait_w(B_PFULL, tile & 1))) break;
            if (grown[tile & 1] == (int)tile) {
              if (heads && lane < 16) quarter[64 * quad + hp + lane] = top;
              if (!(ok = meet())) break;
              float next = 0.f, a = 0.f;
              w = 0.f;
              if (heads && lane < 16) {
                next = fmaxf(r, four());
                a = pow2(r - next);
                if (top - r > kGrow8) w = pow2(k8 - next);               // (was left out of the sum)
                if (quad == 0) alpha[hp + lane] = a;
                put(next);
              }
              if (heads) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  sum[j] = fmaf(s[j], __shfl_sync(0xffffffffu, w, j), sum[j] * __shfl_sync(0xffffffffu, a, j));
              }
              if (!(ok = meet())) break;       // (all have read the old references)
              if (heads && lane < 16) ref[hp + lane] = next;
              __syncwarp();
              rescale();
              hand_over(B_PAGAIN);
            }
          }
        } else {
          // P: rows of tokens, heads contiguous, over the rotary keys (their product is done), and whether a score
          // exceeds its reference by too much
          float now[16];                       // the sums with this tile
          auto weights = [&]() {
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < 16; j += 8) {
              float e[8];
              const float4 r0 = *reinterpret_cast<const float4*>(ref + hp + j);
              const float4 r1 = *reinterpret_cast<const float4*>(ref + hp + j + 4);
              const float r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float d = s[j + k] - r[k];
                most = fmaxf(most, d);
                e[k] = live ? ptx::ex2(d) : 0.f;
                now[j + k] = sum[j + k] + e[k];
              }
              const int hb = hp + j;           // first head of the eight
              if (!heads) break;
              uint4 o;
              o.x = pack_bf16(e[0], e[1]);
              o.y = pack_bf16(e[2], e[3]);
              o.z = pack_bf16(e[4], e[5]);
              o.w = pack_bf16(e[6], e[7]);
              *reinterpret_cast<uint4*>(prow + tok * 128 + (((hb >> 3) ^ (tok & 7)) << 4)) = o;
            }
            return heads && live && most > kGrow;
          };
          auto renew = [&]() {
            // new references: the largest score so far (finite, so that scores of -infinity weigh 0)
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              float m[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) m[k] = fmaxf(warp_most(live ? s[j + k] : -INFINITY), -3.0e38f);
              if (heads && lane == 0)
                *reinterpret_cast<float4*>(quarter + 64 * quad + hp + j) = make_float4(m[0], m[1], m[2], m[3]);
            }
            if (!(ok = meet())) return;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 x = *reinterpret_cast<const float4*>(quarter + hp + j);
              const float4 y = *reinterpret_cast<const float4*>(quarter + 64 + hp + j);
              const float4 z = *reinterpret_cast<const float4*>(quarter + 128 + hp + j);
              const float4 w = *reinterpret_cast<const float4*>(quarter + 192 + hp + j);
              float4 next = make_float4(fmaxf(fmaxf(x.x, y.x), fmaxf(z.x, w.x)), fmaxf(fmaxf(x.y, y.y), fmaxf(z.y, w.y)),
                                        fmaxf(fmaxf(x.z, y.z), fmaxf(z.z, w.z)), fmaxf(fmaxf(x.w, y.w), fmaxf(z.w, w.w)));
              if (!first) {
                const float4 r = *reinterpret_cast<const float4*>(ref + hp + j);
                next = make_float4(fmaxf(r.x, next.x), fmaxf(r.y, next.y), fmaxf(r.z, next.z), fmaxf(r.w, next.w));
                const float a[4] = {ptx::ex2(r.x - next.x), ptx::ex2(r.y - next.y), ptx::ex2(r.z - next.z),
                                    ptx::ex2(r.w - next.w)};
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[j + k] *= a[k];
                if (heads && lane == 0 && quad == 0)
                  *reinterpret_cast<float4*>(alpha + hp + j) = make_float4(a[0], a[1], a[2], a[3]);
              } else if (heads && lane == 0) { // (the four warps of these heads write the same)
                *reinterpret_cast<float4*>(ref + hp + j) = next;
              }
            }
            __syncwarp();
            if (!first) {
              if (!(ok = meet())) return;
              if (heads && lane < 16) {        // (all have read the old ones; the same from each of the four warps)
                const float* x = quarter + hp + lane;
                ref[hp + lane] = fmaxf(ref[hp + lane], fmaxf(fmaxf(x[0], x[64]), fmaxf(x[128], x[192])));
              }
              __syncwarp();
              if (!(ok = wait_w(B_PDONE, (tile - 1) & 1))) return;
              rescale();
            }
          };
          // An item's first tile has no reference to try. (The code of both passes twice: 71 us at 32 queries of 64
          // pages, from one place 73.)
          if (!first) {
            if (__any_sync(0xffffffffu, weights()) && lane == 0) grown[tile & 1] = (int)tile;
            hand_over(B_PFULL);
            if (!(ok = wait_w(B_PFULL, tile & 1))) break;
          }
          if (first || grown[tile & 1] == (int)tile) {
            renew();
            if (!ok) break;
            weights();
            hand_over(first ? B_PFULL : B_PAGAIN);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[j] = now[j];
        }
      }
      if (!ok) break;
      // the item's sums, LSE and output
      const float mine = column_sums(sum, lane);
      if (!(ok = meet())) break;               // (the maxima of a first tile have been read)
      if (heads && lane < 16) quarter[64 * quad + hp + lane] = mine;
      if (!(ok = meet() && wait_w(B_PDONE, (tile - 1) & 1))) break;
      ptx::tc_fence_after();
      if (heads && lane < 16 && quad == 0) {
        const float* q = quarter + hp + lane;
        const float total = (q[0] + q[64]) + (q[128] + q[192]);
        alpha[hp + lane] = total == 0.f ? 0.f : p.out_scale / total;       // (every score -infinity)
        const float lse = (ref[hp + lane] + log2f(total)) * kLn2;
        const int h = h0 + hp + lane;
        if (item.single) p.lse[g * p.H + h] = lse;
        else p.part_lse[(long long)it * p.H + h] = lse;
      }
      if (!(ok = meet())) break;
#pragma unroll 1
      for (int h = 0; h < N; h += 16) {
        uint32_t v[16];
        ptx::tmem_ld16(t_o + lane_off + 64 * part + h, v);
        ptx::tmem_wait_ld();
        const long long at = (long long)(h0 + h) * 512 + 128 * part + 32 * quad + lane;
        if (item.single) {
          bf16* o = reinterpret_cast<bf16*>(p.out_latent) + g * p.H * 512 + at;
#pragma unroll
          for (int k = 0; k < 16; ++k) o[512 * k] = __float2bfloat16_rn(__uint_as_float(v[k]) * alpha[h + k]);
        } else {
          float* o = p.part_o + (long long)it * p.H * 512 + at;
#pragma unroll
          for (int k = 0; k < 16; ++k) o[512 * k] = __uint_as_float(v[k]) * alpha[h + k];
        }
        __syncwarp();                          // the next load is warp-wide
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_OFREE));
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

// A query's pieces under the weights of their LSEs: block (query, 4 heads), 64 threads a head, eight dims each.
// Pieces of one item are final and stay; a query without tokens (or with scores of -inf alone) gets 0 and -inf. Bound by L2, 10.5 us alone (32
// queries of 64 pages), most of its start-up hidden under the attention's end.
__global__ void __launch_bounds__(256) merge_pages_kernel(const DecodeParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int g = blockIdx.x, h = 4 * blockIdx.y + threadIdx.x / 64, d = 4 * (threadIdx.x % 64);
  const int first = p.group_first[g], last = p.group_last[g];
  const int n = first >= 0 && last >= first ? last - first + 1 : 0;
  if (blockIdx.y == 0 && threadIdx.x == 0 && p.bad_lists[g]) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  if (n == 1) return;
  const float* lse = p.part_lse + (long long)first * p.H + h;
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, lse[(long long)i * p.H]);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  float total = 0.f;
  const float* src = p.part_o + ((long long)first * p.H + h) * 512 + d;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(src + (long long)i * p.H * 512);
    const float4 y = *reinterpret_cast<const float4*>(src + (long long)i * p.H * 512 + 256);
    const float l = lse[(long long)i * p.H], w = l == -INFINITY ? 0.f : expf(l - m);
    total += w;
    a = make_float4(fmaf(w, x.x, a.x), fmaf(w, x.y, a.y), fmaf(w, x.z, a.z), fmaf(w, x.w, a.w));
    b = make_float4(fmaf(w, y.x, b.x), fmaf(w, y.y, b.y), fmaf(w, y.z, b.z), fmaf(w, y.w, b.w));
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  bf16* out = reinterpret_cast<bf16*>(p.out_latent) + ((long long)g * p.H + h) * 512 + d;
  if ((reinterpret_cast<uintptr_t>(p.out_latent) & 7) == 0) {
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    *reinterpret_cast<uint2*>(out + 256) = make_uint2(pack_bf16(b.x * inv, b.y * inv), pack_bf16(b.z * inv, b.w * inv));
  } else {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) out[(i >> 2) * 256 + (i & 3)] = __float2bfloat16_rn(v[i] * inv);
  }
  if (threadIdx.x % 64 == 0) p.lse[(long long)g * p.H + h] = total == 0.f ? -INFINITY : m + logf(total);
}

template <int kFmt>
static cudaError_t run(const Maps& maps, const DecodeParams& p, int blocks, cudaStream_t s) {
  auto kern = decode_pages_kernel<kFmt>;
  constexpr int smem = Layout<kFmt>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)(p.workers * blocks), 1, 1), kThreads, smem, s, maps, p, blocks);
  if (e == cudaSuccess)
    e = launch_pdl(merge_pages_kernel, dim3((unsigned)p.batch, (unsigned)(p.H / 4), 1), 256, 0, s, p);
  return e;
}

}  // namespace pdec

using namespace pdec;

bool decode_pages_tc_supported(const mla_config* c, long long num_pages) {
  return c->act_dtype == MLA_BF16 && c->page_size == 64 && c->d_latent == 512 && c->d_rope == 64 &&
         c->num_heads % 16 == 0 && c->num_heads <= 1024 && num_pages * 64 <= 0x7FFFFF00LL;
}

// Tiles that an item's first loads, first reference and epilogue are worth (measured, 1 to 6 tried: bf16 73 us
// at 1, 77 at 4; e4m3 205 at 1, 198 at 4; block-scaled 99 at 1 and 2, 108 at 4).
int decode_pages_item_cost(mla_dtype cache) { return cache == MLA_BF16 ? 1 : (cache == MLA_FP8_E4M3 ? 4 : 2); }

int decode_pages_tc_workers(int H) {
  const int blocks = (H + 63) / 64, n = device_sms() / blocks;
  return n > 0 ? n : 1;
}

cudaError_t launch_decode_pages_tc(mla_dtype cache, const DecodeParams& p, cudaStream_t s) {
  const int blocks = (p.H + 63) / 64;
  const uint64_t rows = (uint64_t)p.num_pages * 64, rb = (uint64_t)p.row_bytes;
  Maps m;
  if (!tensor_map_bf16(&m.q, p.q_lat, 576, (uint64_t)p.H, (uint64_t)p.batch, 1152, (uint64_t)p.H * 1152, 64,
                       (uint32_t)(p.H < 64 ? p.H : 64)))
    return cudaErrorInvalidValue;
  if (cache == MLA_BF16) {
    if (!tensor_map_bf16(&m.c, p.cache, 576, rows, 1, rb, rows * rb, 64, 64)) return cudaErrorInvalidValue;
    m.rope = m.c;
    return run<kBf16>(m, p, blocks, s);
  }
  const bool b128 = cache == MLA_FP8_E4M3_B128;
  if (!tensor_map_3d(&m.c, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, p.cache, 512, rows, 1, rb,
                     rows * rb, 128, 64) ||
      !tensor_map_3d(&m.rope, CU_TENSOR_MAP_DATA_TYPE_UINT8, b128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     p.cache, rb, rows, 1, rb, rows * rb, b128 ? 128 : 64, 64))
    return cudaErrorInvalidValue;
  return b128 ? run<kB128>(m, p, blocks, s) : run<kE4m3>(m, p, blocks, s);
}

}  // namespace mla
