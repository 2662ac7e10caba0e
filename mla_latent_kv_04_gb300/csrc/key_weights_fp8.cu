// Accumulated attention weight of every cached token of an fp8 cache, on the tensor cores: the
// cache's e4m3 codes are themselves the A operand (kind::f8f6f4), tokens in the rows as in
// key_weights_tc.cu, and nothing is expanded.
//
// The other operand has to be fp8 too. A bf16 query value has 8 significant bits, an e4m3 code 4:
// with a power of two 2^e_h per head that puts the head's largest element into [128, 256),
//   hi = e4m3(2^e q),   lo = e4m3(16 (2^e q - hi)),   2^e q = hi + lo / 16
// is exact down to elements of 2^-13 of the largest, and below that off by at most 2^-19 of the
// largest: an fp32 result. hi and lo are rows of one operand (N = 2 H), their products with a code
// are exact, and the epilogue adds the two columns of a head.
//
// Block-scaled cache: the four blocks of 128 codes are products of their own, each read from tensor
// memory and added, times the token's scale, to the head's score in registers (token = lane: the
// scale is one number per thread); the bf16 rotary part is a bf16 product.
//
// Against expanding the codes to bf16 in shared memory (converter warps), 64 requests of 1000 to
// 8192 tokens take 44 us instead of 70. Bound: the cache's bytes, 74 KB (84 KB) a tile, then the
// conversion of a run's query (H x 576 values), about 6 us of integer arithmetic; the MMAs take
// 2304 cycles a tile.
#include <math.h>

#include "fp8_tiles.cuh"
#include "internal.h"
#include "key_runs.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace weigh8 {

using weigh::kTile;
using weigh::Runs;

constexpr int kStage = kTile * 128;                    // 128 codes of a tile's tokens: 16 KB
constexpr int kStages = 5;
constexpr int kQChunk = 256 * 128;                     // 128 codes of the query's hi and lo rows
constexpr int kOffQPe = 4 * kQChunk;                   // e4m3: 64 codes of 256 rows; bf16: 64 of 128
constexpr int kOffRing = kOffQPe + 16384;
constexpr int kOffHead = kOffRing + kStages * kStage;  // per head: factor and offset of the exponent
constexpr int kOffSum = kOffHead + 1024;               // the second half-heads' sums, by token
constexpr int kOffBar = kOffSum + 512;
constexpr int kSmem = kOffBar + 256 + 1024;
static_assert(kSmem <= 232448 - 144, "dynamic shared memory per CTA");   // (first_run has 144 bytes)
constexpr int kEpiWarps = 8, kQWarps = 14;             // warps 4-11; all but the first two
constexpr int kQAtOnce = 5;                            // heads whose query a warp has in flight
constexpr int kThreads = 32 * 16;
enum { B_FULL = 0, B_EMPTY = kStages, B_QFULL = 2 * kStages, B_QEMPTY, B_ZFULL, B_ZFREE = B_ZFULL + 2,
       B_GIVEN = B_ZFREE + 2, B_TAKEN = B_GIVEN + 4, B_TEAR = B_TAKEN + 4, B_COUNT };
static_assert(B_COUNT * 8 <= 240, "barrier area");

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major.
constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Four bf16 values of the query (two pairs) times s -> four hi codes and four lo codes, by
// integer arithmetic (with conversion instructions a query took as long or longer). The values are formed as y = 2^-8 2^e q in f16 (s = 2^(e - 8)): then e4m3's exponent
// field is f16's (bias 7 against 15) and a code is bits 13 to 7 of y, rounded to nearest even at bit
// 7, its sign bit 15; subnormals alike.
__device__ __forceinline__ void split4(uint32_t q01, uint32_t q23, float s, uint32_t* hi, uint32_t* lo) {
  auto scaled = [&](uint32_t q) {
    const __half2 h = __floats2half2_rn(__uint_as_float(q << 16) * s, __uint_as_float(q & 0xFFFF0000u) * s);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  auto rounded = [](uint32_t y) { return y + 0x003F003Fu + ((y >> 7) & 0x00010001u); };
  auto codes = [](uint32_t t0, uint32_t t1) {
    const uint32_t mag = __byte_perm(t0 << 1, t1 << 1, 0x7531), sign = __byte_perm(t0, t1, 0x7531);
    return (mag & 0x7F7F7F7Fu) | (sign & 0x80808080u);
  };
  auto rest = [](uint32_t y, uint32_t t) {             // 16 (y - hi), exactly: at most 4 bits left, cut off
    t &= 0xFF80FF80u;
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&t)),
                              __floats2half2_rn(16.f, 16.f));
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  const uint32_t y0 = scaled(q01), y1 = scaled(q23), t0 = rounded(y0), t1 = rounded(y1);
  *hi = codes(t0, t1);
  *lo = codes(rest(y0, t0), rest(y1, t1));             // (nothing to round but subnormals)
}

// kB128: block-scaled rows
template <bool kB128>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_fp8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_pe,
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
    for (int i = 0; i < B_COUNT; ++i) {
      int n = 1;
      if (i == B_QFULL) n = kQWarps;
      if (i >= B_ZFREE && i < B_GIVEN) n = kEpiWarps;
      ptx::mbar_init(bar(i), n);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_x);
    ptx::prefetch_tensormap(&tm_pe);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  // a query's conversion counts as 5 tiles (64 requests of 1000 to 8192 tokens: 44.4 us; as 3 or 7
  // 45.5, as none 50.5)
  Runs run = weigh::first_run(p, reinterpret_cast<int*>(basep), 5, 16);
  ptx::tc_fence_before();
  ptx::fence_proxy_async_smem();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  const int N = 2 * p.cols;

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
            for (int c = 0; c < 5; ++c, ++g) {         // four latent chunks, the rotary part
              const uint32_t st = g % kStages;
              if (!(ok = wait(B_EMPTY + st, ((g / kStages) & 1) ^ 1))) break;
              const uint32_t dst = base + kOffRing + st * kStage, full = bar(B_FULL + st);
              const uint32_t half = c < 4 || kB128 ? 8192 : 4096;
              const CUtensorMap* tm = c < 4 ? &tm_x : &tm_pe;
              const int x = c < 4 ? 128 * c : (kB128 ? 528 : 512);
              ptx::mbar_arrive_expect_tx(full, two ? 2 * half : half);
              if (p.passes > 1) {
                ptx::tma_load_3d(dst, tm, x, y0, 0, full);
                if (two) ptx::tma_load_3d(dst + half, tm, x, y1, 0, full);
              } else {
                ptx::tma_load_3d_hint(dst, tm, x, y0, 0, full, pol);
                if (two) ptx::tma_load_3d_hint(dst + half, tm, x, y1, 0, full, pol);
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
    const uint32_t idesc = idesc_e4m3(128, N), idesc_pe = ptx::idesc_bf16_f32(128, p.cols, false, false);
    uint32_t g = 0, q_iter = 0, z = 0;
    bool ok = true;
    while (ok && run.next()) {
      for (int t = 0; ok && t < p.passes; ++t, ++q_iter) {
        if (!(ok = wait_w(B_QFULL, q_iter & 1))) break;
        for (int tile = run.t0; ok && tile < run.t1; ++tile) {
          for (int c = 0; c < 5; ++c, ++g) {
            const uint32_t st = g % kStages;
            // a new accumulator: per tile, or (block scales) per chunk
            if ((c == 0 || kB128) && !(ok = wait_w(B_ZFREE + (z & 1), ((z >> 1) & 1) ^ 1))) break;
            if (!(ok = wait_w(B_FULL + st, (g / kStages) & 1))) break;
            ptx::tc_fence_after();
            const uint32_t x = base + kOffRing + st * kStage, d = tmem + 256 * (z & 1);
            if (ptx::elect_one()) {
              if (c < 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_e4m3_ss(d, ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                                   ptx::smem_desc(base + c * kQChunk + 32 * k, 16, 1024, ptx::kSwizzle128), idesc,
                                   ((!kB128 && c) || k) ? 1u : 0u);
              } else if (kB128) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_bf16_ss(d, ptx::smem_desc(x + 32 * k, 16, 1024, ptx::kSwizzle128),
                                   ptx::smem_desc(base + kOffQPe + 32 * k, 16, 1024, ptx::kSwizzle128), idesc_pe,
                                   k ? 1u : 0u);
              } else {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  ptx::mma_e4m3_ss(d, ptx::smem_desc(x + 32 * k, 16, 512, ptx::kSwizzle64),
                                   ptx::smem_desc(base + kOffQPe + 32 * k, 16, 512, ptx::kSwizzle64), idesc, 1u);
              }
              ptx::mma_commit(bar(B_EMPTY + st));
              if (c == 4 || kB128) ptx::mma_commit(bar(B_ZFULL + (z & 1)));
              if (c == 4 && tile == run.t1 - 1) ptx::mma_commit(bar(B_QEMPTY));
            }
            __syncwarp();
            if (c == 4 || kB128) ++z;
          }
        }
      }
    }
    if (*abort) {
      if (ptx::elect_one()) ptx::mma_commit(bar(B_TEAR));
      __syncwarp();
      drain_wait(bar(B_TEAR), 0);
    }
  } else {
    float2* head = reinterpret_cast<float2*>(basep + kOffHead);
    // A run's query: the warps take heads in turn, 16 latent elements and 2 rotary ones a lane. The
    // query before is done with when its MMAs are (B_QEMPTY), the heads' factors when the last
    // scores were read (accumulator z - 1).
    auto convert = [&](const Runs& r, int t, uint32_t q_iter, uint32_t z) {
      const int qw = warp - 2;
      const long long g = (long long)r.rb * p.passes + t;
      bool good = wait_w(B_QEMPTY, (q_iter & 1) ^ 1);
      if (good && z > 0) good = wait_w(B_ZFREE + ((z - 1) & 1), ((z - 1) >> 1) & 1);
      if (!good) return false;
      for (int hb = qw; hb < p.cols; hb += kQAtOnce * kQWarps) {
        uint4 a[kQAtOnce], b[kQAtOnce];
        uint32_t e[kQAtOnce];
        float off[kQAtOnce];
#pragma unroll
        for (int i = 0; i < kQAtOnce; ++i) {
          const int h = min(hb + i * kQWarps, p.cols - 1);
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(p.q_lat) + (g * p.cols + h) * 576);
          a[i] = src[2 * lane];
          b[i] = src[2 * lane + 1];
          e[i] = reinterpret_cast<const uint32_t*>(src + 64)[lane];
          off[i] = p.lse[g * p.cols + h] * kLog2e;
        }
#pragma unroll
        for (int i = 0; i < kQAtOnce; ++i) {
          const int h = hb + i * kQWarps;
          if (h >= p.cols) break;
          const uint32_t pe = e[i];
          const uint32_t v[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
          // the largest magnitude, two at a time; the warp's by its bits (NaN above all: kept)
          const uint32_t z2 = kB128 ? 0u : pe & 0x7FFF7FFFu;
          uint32_t m2 = z2;
#pragma unroll
          for (int k = 0; k < 8; ++k) m2 = __vmaxu2(m2, v[k] & 0x7FFF7FFFu);
          const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16)) << 16);
          // 2^e with 2^e m in [128, 256) (exponents clamped: an all-zero or tiny head stays finite)
          const int ex = max(-110, min(120, (int)((__float_as_uint(m) >> 23) & 255) - 127));
          const float s = __uint_as_float((uint32_t)(-1 - ex + 127) << 23);
          const float inv = __uint_as_float((uint32_t)(ex - 7 + 127) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split4(v[2 * k], v[2 * k + 1], s, &hi[k], &lo[k]);
          uint8_t* q = basep + (lane >> 3) * kQChunk;
          const int unit = lane & 7, r1 = h + p.cols;
          *reinterpret_cast<uint4*>(q + h * 128 + ((unit ^ (h & 7)) << 4)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(q + r1 * 128 + ((unit ^ (r1 & 7)) << 4)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
          uint8_t* qp = basep + kOffQPe;
          if (kB128) {
            *reinterpret_cast<uint32_t*>(qp + h * 128 + (((lane >> 2) ^ (h & 7)) << 4) + 4 * (lane & 3)) = pe;
          } else {
            uint32_t pe_hi, pe_lo;
            split4(pe, 0u, s, &pe_hi, &pe_lo);
            *reinterpret_cast<uint16_t*>(qp + h * 64 + (((lane >> 3) ^ ((h >> 1) & 3)) << 4) + 2 * (lane & 7)) = (uint16_t)pe_hi;
            *reinterpret_cast<uint16_t*>(qp + r1 * 64 + (((lane >> 3) ^ ((r1 >> 1) & 3)) << 4) + 2 * (lane & 7)) = (uint16_t)pe_lo;
          }
          // infinities and NaN in the query make its weights NaN
          const float nan = m < INFINITY ? 0.f : m - m;
          if (lane == 0) head[h] = make_float2((kB128 ? inv : inv * p.scale_log2) + nan, off[i]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_QFULL));
      return true;
    };
    // the query after this one into L2
    auto prefetch = [&](Runs r, int t) {
      if (++t == p.passes) {
        if (!r.next()) return;
        t = 0;
      }
      ptx::bulk_prefetch_l2(reinterpret_cast<const bf16*>(p.q_lat) + ((long long)r.rb * p.passes + t) * p.cols * 576,
                            (uint32_t)(p.cols * 576 * 2));
    };
    constexpr uint32_t kZ = kB128 ? 5 : 1;             // accumulators of a tile
    if (warp < 4 || warp >= 12) {
      uint32_t q_iter = 0, z = 0;
      bool ok = true;
      while (ok && run.next()) {
        for (int t = 0; ok && t < p.passes; ++t, ++q_iter) {
          if (!(ok = convert(run, t, q_iter, z))) break;
          z += kZ * (uint32_t)(run.t1 - run.t0);
          if (warp == 2 && lane == 0) prefetch(run, t);
          __syncwarp();
        }
      }
    } else {
      // two threads per token: heads H/2 part .. of it
      const int quad = warp & 3, part = warp >= 8 ? 1 : 0, row = 32 * quad + lane;
      const uint32_t t_row = tmem + ((uint32_t)(32 * quad) << 16);
      const int hh = p.cols / 2, h0 = part * hh;         // columns of this thread (a multiple of 8)
      float* half_sum = reinterpret_cast<float*>(basep + kOffSum);
      uint32_t z = 0, x = 0, q_iter = 0;
      bool ok = true;
      while (ok && run.next()) {
        const int32_t* bt = p.block_table + (long long)run.rb * p.max_pages;
        const int S = run.S;
        float* w = p.weights + (long long)run.rb * p.max_pages * p.P;
        for (int t = 0; ok && t < p.passes; ++t, ++q_iter) {
          if (!(ok = convert(run, t, q_iter, z) && wait_w(B_QFULL, q_iter & 1))) break;
          for (int tile = run.t0; ok && tile < run.t1; ++tile) {
            const int j = tile * kTile + row, from = weigh::first_column(p, S, j, t);
            int page = j < S ? bt[j / 64] : -1;
            if (page >= p.num_pages) page = -1;
            float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kB128 && page >= 0)
              sc = *reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(p.cache) +
                                                    ((long long)page * 64 + (j & 63)) * p.row_bytes + 512);
            float sum = 0.f;
            if constexpr (!kB128) {
              if (!(ok = wait_w(B_ZFULL + (z & 1), (z >> 1) & 1))) break;
              ptx::tc_fence_after();
              const uint32_t d = t_row + 256 * (z & 1);
              float s4[4] = {0.f, 0.f, 0.f, 0.f};
              for (int h = h0; h < h0 + hh; h += 8) {
                uint32_t hi[8], lo[8];
                ptx::tmem_ld8(d + h, hi);
                ptx::tmem_ld8(d + p.cols + h, lo);
                ptx::tmem_wait_ld();
                const bool sees = h >= from;           // (a query token's columns are a multiple of 16)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float2 f = head[h + i];
                  const float v = fmaf(__uint_as_float(lo[i]), 0.0625f, __uint_as_float(hi[i]));
                  const float e = ptx::ex2(fmaf(v, f.x, -f.y));
                  s4[i & 3] += sees ? e : 0.f;
                }
                __syncwarp();                          // the next load is warp-wide
              }
              sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar(B_ZFREE + (z & 1)));
              ++z;
            } else {
              float acc[64];
#pragma unroll
              for (int i = 0; i < 64; ++i) acc[i] = 0.f;
#pragma unroll
              for (int c = 0; c < 5; ++c) {
                if (ok) ok = wait_w(B_ZFULL + (z & 1), (z >> 1) & 1);
                if (ok) {
                  ptx::tc_fence_after();
                  const uint32_t d = t_row + 256 * (z & 1);
                  const float s = c == 0 ? sc.x : (c == 1 ? sc.y : (c == 2 ? sc.z : sc.w));
#pragma unroll
                  for (int i = 0; i < 64; i += 8) {
                    if (i >= hh) break;
                    uint32_t hi[8], lo[8];
                    ptx::tmem_ld8(d + h0 + i, hi);
                    if (c < 4) ptx::tmem_ld8(d + p.cols + h0 + i, lo);
                    ptx::tmem_wait_ld();
                    // (the last chunk: a query token's columns are a multiple of 16)
                    if (c < 4) {
#pragma unroll
                      for (int k = 0; k < 8; ++k)
                        acc[i + k] = fmaf(s, fmaf(__uint_as_float(lo[k]), 0.0625f, __uint_as_float(hi[k])), acc[i + k]);
                    } else if (h0 + i >= from) {
#pragma unroll
                      for (int k = 0; k < 8; ++k) {
                        const float2 f = head[h0 + i + k];           // factor 2^-e, offset
                        sum += ptx::ex2(fmaf(fmaf(acc[i + k], f.x, __uint_as_float(hi[k])), p.scale_log2, -f.y));
                      }
                    }
                    if (c == 4) __syncwarp();                        // the next load is warp-wide
                  }
                  ptx::tc_fence_before();
                  __syncwarp();
                  if (lane == 0) ptx::mbar_arrive(bar(B_ZFREE + (z & 1)));
                  ++z;
                }
              }
              if (!ok) break;
            }
            // the other half's heads: the second half's thread hands its sum over
            if (part == 1) {
              if (!(ok = wait_w(B_TAKEN + quad, (x & 1) ^ 1))) break;
              half_sum[row] = sum;
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar(B_GIVEN + quad));
              ++x;
              continue;
            }
            if (!(ok = wait_w(B_GIVEN + quad, x & 1))) break;
            const float other = half_sum[row];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_TAKEN + quad));
            ++x;
            if (page >= 0) {
              const float mass = sum + other;
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
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <bool kB128>
static cudaError_t run(const CUtensorMap& x, const CUtensorMap& pe, const KeyWeightParams& p, cudaStream_t s) {
  auto kern = key_weights_fp8_kernel<kB128>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)weigh::grid_size(p), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, x, pe, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace weigh8

cudaError_t launch_key_weights_fp8(mla_dtype cache, const KeyWeightParams& p, cudaStream_t s) {
  using namespace weigh8;
  CUtensorMap x, pe;
  const uint64_t rows = (uint64_t)p.num_pages * 64, rb = (uint64_t)p.row_bytes;
  const bool b128 = cache == MLA_FP8_E4M3_B128;
  if (!tensor_map_3d(&x, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, p.cache, 512, rows, 1, rb,
                     rows * rb, 128, 64) ||
      !tensor_map_3d(&pe, CU_TENSOR_MAP_DATA_TYPE_UINT8, b128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     p.cache, rb, rows, 1, rb, rows * rb, b128 ? 128 : 64, 64))
    return cudaErrorInvalidValue;
  return b128 ? run<true>(x, pe, p, s) : run<false>(x, pe, p, s);
}

}  // namespace mla
