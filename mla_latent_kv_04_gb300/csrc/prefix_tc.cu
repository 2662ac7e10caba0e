// Attention of a whole batch to an expanded prefix, on the tensor cores (bf16, DeepSeek-V2 head
// shape: d_n 128, d_r 64, d_v 128).
//
// Every request's query tokens are the rows of one matrix per head, so the prefix's keys and
// values are read once for 128 rows. Per head, row tile (128 rows) and block of 128 keys:
//   S = [q_nope ; q_hi ; q_lo] [K ; k_pe ; k_pe]^T   (K = 128 + 64 + 64 of the MMA)
//   P = exp2(c S - c m),  O += P V,  l += sum P      (c = softmax scale * log2 e)
// The rotated query is the sum of two bf16 terms (residual 2^-16), so that the scores, and the
// LSE, are fp32 results: q_nope and the keys are exact. The low term costs a fifth of the MMA
// time; bf16 alone would put up to 2^-8 of the rotary score's terms into the LSE.
//
// Two key blocks are in flight: even blocks belong to softmax warpgroup 0, odd ones to
// warpgroup 1, each with its own scores, running maximum, sum and output in tensor memory (S
// 128 + O 128 columns each: all 512). The MMA warp issues S(n), then O(n - 1): the softmax of a
// block runs while the tensor cores work on the other warpgroup's. P (bf16) takes the place
// of its own S. A maximum moves only when it grows by more than 2^8 (O is then rescaled in
// tensor memory). At a segment's end the two halves are merged.
//
// Work: the (head, row tile, key block) triples in this order are cut into one contiguous range
// per CTA; a range may start and end inside a tile, whose pieces then go to the workspace
// (fp32) and are merged by attend_merge_kernel. If whole tiles spread evenly enough over the
// CTAs, the cuts are put between tiles.
//
// Bound: at up to about 200 rows the keys' and values' bytes (64 KB per head and block), then
// the MMAs.
#include <math.h>

#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace attend {

constexpr int kBM = 128, kBN = 128;
constexpr int kBox = 128 * 64 * 2;                 // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kOffQ = 0;                           // nope 0, nope 1, rotary high, rotary low
constexpr int kOffK = 4 * kBox;                    // 2 stages of nope 0, nope 1, rotary
constexpr int kOffV = kOffK + 2 * 3 * kBox;        // 2 stages of two 64-dim boxes
constexpr int kOffX = kOffV + 2 * 2 * kBox;        // merge exchange: 128 x 2 floats
constexpr int kOffBar = kOffX + 1024;
constexpr int kSmem = kOffBar + 256 + 1024;        // + slack to align the base to 1 KB
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kThreads = 384;
constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescO = ptx::idesc_bf16_f32(128, 128, false, true);
constexpr float kRescale = 8.f;                    // log2 units

enum { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8, B_QEMPTY, B_SFULL, B_PREADY = 12,
       B_ODONE = 14, B_XCH = 16, B_TEAR, B_COUNT };

struct Work {
  int tiles, row_tiles, blocks;                    // tiles = H * row_tiles; blocks per tile
  int ctas;
  int whole;                                       // 1: cuts between tiles only
  float* part_o;                                   // [2 ctas][128][128]
  float* part_lse;                                 // [2 ctas][128], log2 units
  __host__ __device__ long long begin(int c) const {
    return whole ? (long long)c * tiles / ctas * blocks : (long long)c * tiles * blocks / ctas;
  }
};

struct Segments {                                  // the pieces of a CTA's range, in order
  const Work* w;
  long long u, end;
  int tile, k0, k1;
  __device__ Segments(const Work& work, int cta) : w(&work), u(work.begin(cta)), end(work.begin(cta + 1)) {}
  __device__ bool next() {
    if (u >= end) return false;
    tile = (int)(u / w->blocks);
    k0 = (int)(u - (long long)tile * w->blocks);
    const long long left = end - u;
    k1 = left < w->blocks - k0 ? k0 + (int)left : w->blocks;
    u += k1 - k0;
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_pe, const __grid_constant__ CUtensorMap tm_v,
                     const PrefixAttendParams p, const Work work) {
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
      const bool p_ready = i == B_PREADY || i == B_PREADY + 1;
      ptx::mbar_init(bar(i), p_ready ? 4 : (i == B_QFULL ? 9 : (i == B_XCH ? 8 : 1)));
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_q);
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_pe);
    ptx::prefetch_tensormap(&tm_v);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  // a warp goes on, or gives up, as one
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  Segments seg(work, blockIdx.x);

  // registers: the softmax warps hold a row of scores (launched with 168 x 384; 88 x 128 + 200 x
  // 256 = 62464 of the 64512 after the split)
  if (warp < 4) {
    ptx::setmaxnreg_dec<88>();
    if (warp == 0) {
      if (lane == 0) {                               // keys
        const uint64_t pol = ptx::l2_policy_evict_first();
        const bool once = work.row_tiles == 1;       // each key is read by one tile
        uint32_t g = 0;
        while (seg.next()) {
          const int h = seg.tile / work.row_tiles;
          bool ok = true;
          for (int kb = seg.k0; kb < seg.k1 && (ok = wait(B_KEMPTY + (g & 1), ((g >> 1) & 1) ^ 1)); ++kb, ++g) {
            const uint32_t st = base + kOffK + (g & 1) * 3 * kBox, full = bar(B_KFULL + (g & 1));
            ptx::mbar_arrive_expect_tx(full, 3 * kBox);
            if (once) {
              ptx::tma_load_3d_hint(st, &tm_k, 0, kb * kBN, h, full, pol);
              ptx::tma_load_3d_hint(st + kBox, &tm_k, 64, kb * kBN, h, full, pol);
            } else {
              ptx::tma_load_3d(st, &tm_k, 0, kb * kBN, h, full);
              ptx::tma_load_3d(st + kBox, &tm_k, 64, kb * kBN, h, full);
            }
            ptx::tma_load_3d(st + 2 * kBox, &tm_pe, 0, kb * kBN, 0, full);
          }
          if (!ok) break;
        }
        if (*abort)
          for (uint32_t i = g > 2 ? g - 2 : 0; i < g; ++i) drain_wait(bar(B_KFULL + (i & 1)), (i >> 1) & 1);
      }
    } else if (warp == 3) {
      if (lane == 0) {                               // values
        const uint64_t pol = ptx::l2_policy_evict_first();
        const bool once = work.row_tiles == 1;
        uint32_t g = 0;
        while (seg.next()) {
          const int h = seg.tile / work.row_tiles;
          bool ok = true;
          for (int kb = seg.k0; kb < seg.k1 && (ok = wait(B_VEMPTY + (g & 1), ((g >> 1) & 1) ^ 1)); ++kb, ++g) {
            const uint32_t st = base + kOffV + (g & 1) * 2 * kBox, full = bar(B_VFULL + (g & 1));
            ptx::mbar_arrive_expect_tx(full, 2 * kBox);
            if (once) {
              ptx::tma_load_3d_hint(st, &tm_v, 0, kb * kBN, h, full, pol);
              ptx::tma_load_3d_hint(st + kBox, &tm_v, 64, kb * kBN, h, full, pol);
            } else {
              ptx::tma_load_3d(st, &tm_v, 0, kb * kBN, h, full);
              ptx::tma_load_3d(st + kBox, &tm_v, 64, kb * kBN, h, full);
            }
          }
          if (!ok) break;
        }
        if (*abort)
          for (uint32_t i = g > 2 ? g - 2 : 0; i < g; ++i) drain_wait(bar(B_VFULL + (i & 1)), (i >> 1) & 1);
      }
    } else if (warp == 2) {
      if (lane == 0) {                               // the content part of the queries
        uint32_t s = 0;
        while (seg.next() && wait(B_QEMPTY, (s & 1) ^ 1)) {
          const int h = seg.tile / work.row_tiles, r0 = seg.tile % work.row_tiles * kBM;
          ptx::mbar_arrive_expect_tx(bar(B_QFULL), 2 * kBox);
          ptx::tma_load_3d(base + kOffQ, &tm_q, 0, r0, h, bar(B_QFULL));
          ptx::tma_load_3d(base + kOffQ + kBox, &tm_q, 64, r0, h, bar(B_QFULL));
          ++s;
        }
        // after an abort the rotary part may never arrive: this wait may run its full second
        if (*abort && s) drain_wait(bar(B_QFULL), (s - 1) & 1);
      }
    } else if (warp == 1) {
      // MMAs: S(n), then O(n - 1)
      uint32_t gk = 0, gv = 0, s = 0, cnt[2] = {0, 0};
      bool ok = true;
      auto out = [&](int n) {                        // O(n) += P(n) V(n); n: block of the segment
        const int w = n & 1;
        if (!wait_w(B_PREADY + w, ((w ? cnt[1] : cnt[0]) - 1) & 1) || !wait_w(B_VFULL + (gv & 1), (gv >> 1) & 1))
          return false;
        ptx::tc_fence_after();
        const uint32_t v = base + kOffV + (gv & 1) * 2 * kBox;
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            ptx::mma_bf16_ts(tmem + 256 + 128 * w, tmem + 128 * w + 8 * k,
                             ptx::smem_desc(v + 2048 * k, kBox, 1024, ptx::kSwizzle128), kIdescO,
                             (n >= 2 || k) ? 1u : 0u);
          ptx::mma_commit(bar(B_VEMPTY + (gv & 1)));
          ptx::mma_commit(bar(B_ODONE + w));
        }
        __syncwarp();
        ++gv;
        return true;
      };
      while (ok && seg.next()) {
        ok = wait_w(B_QFULL, s & 1);
        const int nb = seg.k1 - seg.k0;
        for (int n = 0; ok && n < nb; ++n) {
          if (!(ok = wait_w(B_KFULL + (gk & 1), (gk >> 1) & 1))) break;
          ptx::tc_fence_after();
          // S(n) overwrites S and P of block n - 2, whose product was issued before
          const uint32_t q = base + kOffQ, k0 = base + kOffK + (gk & 1) * 3 * kBox;
          if (ptx::elect_one()) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t kbox = j < 12 ? j >> 2 : 2;     // the low rotary term meets k_pe again
              ptx::mma_bf16_ss(tmem + 128 * (n & 1),
                               ptx::smem_desc(q + (j >> 2) * kBox + 32 * (j & 3), 16, 1024, ptx::kSwizzle128),
                               ptx::smem_desc(k0 + kbox * kBox + 32 * (j & 3), 16, 1024, ptx::kSwizzle128),
                               kIdescS, j ? 1u : 0u);
            }
            ptx::mma_commit(bar(B_KEMPTY + (gk & 1)));
            ptx::mma_commit(bar(B_SFULL + (n & 1)));
            if (n == nb - 1) ptx::mma_commit(bar(B_QEMPTY));
          }
          __syncwarp();
          if (n & 1) ++cnt[1];
          else ++cnt[0];
          ++gk;
          // P(n - 1): the count of its warpgroup has not moved since S(n - 1)
          if (n > 0) ok = out(n - 1);
        }
        if (ok) ok = out(nb - 1);
        ++s;
      }
      if (*abort) {
        if (ptx::elect_one()) ptx::mma_commit(bar(B_TEAR));
        __syncwarp();
        drain_wait(bar(B_TEAR), 0);
      }
    }
  } else {
    ptx::setmaxnreg_inc<200>();
    // softmax warpgroup w: thread = row of the tile = lane of tensor memory
    const int w = warp >= 8 ? 1 : 0, quad = warp & 3, row = 32 * quad + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t t_s = t_lane + 128 * w, t_o = t_lane + 256 + 128 * w;
    const float c = p.scale_log2;
    float2* xch = reinterpret_cast<float2*>(basep + kOffX);
    uint32_t cnt = 0, cnt_other = 0, s = 0, meets = 0;
    bool ok = true;
    // both warpgroups meet (bounded, unlike a named barrier)
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_XCH));
      return wait_w(B_XCH, meets++ & 1);
    };
    while (seg.next()) {
      const int h = seg.tile / work.row_tiles, r = seg.tile % work.row_tiles * kBM + row;
      const int nb = seg.k1 - seg.k0;
      // the row's rotated query: pairs 16 w .. 16 w + 15, high and low term
      int S = 0;
      if (r < p.rows) S = p.seq_lens[r / p.q_len];
      const bool live = r < p.rows && S >= p.q_len;
      if (r < p.rows && S != 0 && S < p.q_len && h == 0 && seg.k0 == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
      if (!(ok = wait_w(B_QEMPTY, (s & 1) ^ 1))) break;
      {
        const long long pos = (long long)p.L + S - p.q_len + r % p.q_len;
        uint4 x[4];
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(p.q_pe) +
                                                          ((long long)r * p.H + h) * 64 + 32 * w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float sn, cs;
            turn_sincos<false>(p.tt, 16 * w + 4 * i + j, pos, &sn, &cs);
            const float a = __uint_as_float(in[j] << 16), b = __uint_as_float(in[j] & 0xFFFF0000u);
            const float y0 = a * cs - b * sn, y1 = a * sn + b * cs;
            const __nv_bfloat162 t = __floats2bfloat162_rn(y0, y1);
            const float2 f = __bfloat1622float2(t);
            const __nv_bfloat162 u = __floats2bfloat162_rn(y0 - f.x, y1 - f.y);
            hi[j] = *reinterpret_cast<const uint32_t*>(&t);
            lo[j] = *reinterpret_cast<const uint32_t*>(&u);
          }
          const int at = row * 128 + (((4 * w + i) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(basep + kOffQ + 2 * kBox + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(basep + kOffQ + 3 * kBox + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_QFULL));
      ++s;
      float m = -INFINITY, l = 0.f;
      for (int n = w; n < nb; n += 2) {
        if (!(ok = wait_w(B_SFULL + w, cnt & 1))) break;
        ptx::tc_fence_after();
        const int valid = min(kBN, p.L - (seg.k0 + n) * kBN);
        // the whole row at once: one wait for tensor memory instead of one per 32 columns
        uint32_t v[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::tmem_ld32(t_s + 32 * q, v[q]);
        ptx::tmem_wait_ld();
        if (valid < kBN) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * q + j >= valid) v[q][j] = 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; j += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(v[q][j]), __uint_as_float(v[q][j + 1])));
        const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (n == w) {
          m = mb;
        } else {
          const bool grow = (mb - m) * c > kRescale;
          // a warp rescales its rows together
          if (__any_sync(0xffffffffu, grow)) {
            if (!(ok = wait_w(B_ODONE + w, (cnt - 1) & 1))) break;
            ptx::tc_fence_after();
            const float a = grow ? (m == -INFINITY ? 0.f : ptx::ex2((m - mb) * c)) : 1.f;
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
              uint32_t o[16];
              ptx::tmem_ld16(t_o + 16 * q, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
              ptx::tmem_st16(t_o + 16 * q, o);
            }
            ptx::tmem_wait_st();
            l *= a;
            if (grow) m = mb;
          }
        }
        const float off = m == -INFINITY ? 0.f : m * c;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            // columns behind the prefix hold -infinity: exp2 gives 0
            const float e0 = ptx::ex2(fmaf(__uint_as_float(v[q][j]), c, -off));
            const float e1 = ptx::ex2(fmaf(__uint_as_float(v[q][j + 1]), c, -off));
            sum[j & 2] += e0;
            sum[(j & 2) + 1] += e1;
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
            pk[j >> 1] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          ptx::tmem_st16(t_s + 16 * q, pk);
        }
        ptx::tmem_wait_st();
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(B_PREADY + w));
        ++cnt;
      }
      if (!ok) break;
      // the other warpgroup's blocks of this segment
      cnt_other += w == 0 ? nb / 2 : (nb + 1) / 2;
      // (a warpgroup without a block here waits for its previous one, long done)
      if (!(ok = wait_w(B_ODONE + w, (cnt - 1) & 1) && wait_w(B_ODONE + (w ^ 1), (cnt_other - 1) & 1))) break;
      ptx::tc_fence_after();
      // both warpgroups' maximum and sum -> the factors of their outputs
      if (w == 1) xch[row] = make_float2(m, l);
      if (!(ok = meet())) break;
      float a0, a1;
      float mt = 0.f, L = 0.f;
      if (w == 0) {
        const float2 o = xch[row];
        mt = fmaxf(m, o.x);
        a0 = m == -INFINITY ? 0.f : ptx::ex2((m - mt) * c);
        a1 = o.x == -INFINITY ? 0.f : ptx::ex2((o.x - mt) * c);
        L = a0 * l + a1 * o.y;
        const float inv = L > 0.f ? 1.f / L : 0.f;
        a0 *= inv;
        a1 *= inv;
        xch[row] = make_float2(a0, a1);
      }
      if (!(ok = meet())) break;
      if (w == 1) {
        a0 = xch[row].x;
        a1 = xch[row].y;
      }
      const bool full = seg.k0 == 0 && seg.k1 == work.blocks;
      const int slot = 2 * blockIdx.x + (seg.k0 == 0 ? 1 : 0);
      if (w == 0) {
        const float lse2 = L > 0.f ? mt * c + log2f(L) : -INFINITY;
        if (!full) work.part_lse[slot * kBM + row] = lse2;
        else if (r < p.rows) p.lse[(long long)r * p.H + h] = live ? lse2 * kLn2 : -INFINITY;
      }
      // output columns 64 w .. 64 w + 63
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t v0[32], v1[32];
        const uint32_t col = 64 * w + 32 * q;
        ptx::tmem_ld32(t_lane + 256 + col, v0);
        if (nb > 1) ptx::tmem_ld32(t_lane + 384 + col, v1);
        ptx::tmem_wait_ld();
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          o[j] = a0 * __uint_as_float(v0[j]);
          if (nb > 1) o[j] = fmaf(a1, __uint_as_float(v1[j]), o[j]);
        }
        if (!full) {
          float4* dst = reinterpret_cast<float4*>(work.part_o + ((long long)slot * kBM + row) * 128 + col);
          if (r < p.rows) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        } else if (r < p.rows) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(p.u) + ((long long)r * p.H + h) * 128 + col);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(live ? o[8 * j + 2 * i] : 0.f,
                                                              live ? o[8 * j + 2 * i + 1] : 0.f);
              k[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dst[j] = make_uint4(k[0], k[1], k[2], k[3]);
          }
        }
      }
      // the next segment's products overwrite both outputs: not before both halves were read
      ptx::tc_fence_before();
      if (!(ok = meet())) break;
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

// Joins the pieces of a tile that was cut: out = sum_s w_s o_s, w_s = 2^(lse_s - L). Warp per row.
__global__ void __launch_bounds__(256) attend_merge_kernel(const PrefixAttendParams p, const Work work) {
  const int tile = blockIdx.x, row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int h = tile / work.row_tiles, r = tile % work.row_tiles * kBM + row;
  if (r >= p.rows) return;
  const long long t0 = (long long)tile * work.blocks, t1 = t0 + work.blocks;
  // the CTAs whose ranges hold the tile's first and last block
  const long long U = (long long)work.tiles * work.blocks;
  auto owner = [&](long long u) {
    int c = (int)(u * work.ctas / U);
    while (work.begin(c + 1) <= u) ++c;
    while (work.begin(c) > u) --c;
    return c;
  };
  const int c0 = owner(t0), c1 = owner(t1 - 1);
  if (c0 == c1) return;                            // written whole
  auto slot = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };
  const int S = p.seq_lens[r / p.q_len];
  float m = -INFINITY;
  for (int c = c0; c <= c1; ++c) m = fmaxf(m, work.part_lse[slot(c) * kBM + row]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  const bool live = S >= p.q_len && m > -INFINITY;
  if (live) {
    for (int c = c0; c <= c1; ++c) {
      const float w = ptx::ex2(work.part_lse[slot(c) * kBM + row] - m);
      const float4 o = *reinterpret_cast<const float4*>(work.part_o + ((long long)slot(c) * kBM + row) * 128 + 4 * lane);
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
      sum += w;
    }
  }
  const float inv = live ? 1.f / sum : 0.f;
  const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(p.u) + ((long long)r * p.H + h) * 128 + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (lane == 0) p.lse[(long long)r * p.H + h] = live ? (m + log2f(sum)) * kLn2 : -INFINITY;
}

// Cuts between tiles unless that leaves a CTA this many blocks more than an even share: a cut
// tile costs its pieces' way through the workspace and the merge.
constexpr int kCutGain = 4;

static Work plan(int rows, int H, int L) {
  Work w{};
  w.row_tiles = (rows + kBM - 1) / kBM;
  w.tiles = H * w.row_tiles;
  w.blocks = (L + kBN - 1) / kBN;
  const int sms = device_sms();
  const long long units = (long long)w.tiles * w.blocks;
  const long long even = (units + sms - 1) / sms;
  const long long uncut = (long long)((w.tiles + sms - 1) / sms) * w.blocks;
  w.whole = uncut <= even + kCutGain;
  w.ctas = w.whole ? (w.tiles < sms ? w.tiles : sms) : (int)(units < sms ? units : sms);
  return w;
}

}  // namespace attend

bool prefix_attend_tc_supported(const mla_config* c) {
  return c->act_dtype == MLA_BF16 && c->d_nope == 128 && c->d_rope == 64 && c->d_v == 128;
}

size_t prefix_attend_tc_workspace(int rows, int H, int L) {
  if (rows <= 0 || L <= 0) return 0;
  const attend::Work w = attend::plan(rows, H, L);
  return w.whole ? 0 : (size_t)2 * w.ctas * attend::kBM * (128 + 1) * 4;
}

cudaError_t launch_prefix_attend_tc(const PrefixAttendParams& p, void* workspace, cudaStream_t s) {
  using namespace attend;
  Work w = plan(p.rows, p.H, p.L);
  w.part_o = (float*)workspace;
  w.part_lse = w.whole ? nullptr : w.part_o + (size_t)2 * w.ctas * kBM * 128;
  CUtensorMap q, k, pe, v;
  const uint64_t H = (uint64_t)p.H, L = (uint64_t)p.L;
  if (!tensor_map_bf16(&q, p.q_nope, 128, (uint64_t)p.rows, H, H * 256, 256, 64, kBM) ||
      !tensor_map_bf16(&k, p.keys, 128, L, H, 256, L * 256, 64, kBN) ||
      !tensor_map_bf16(&pe, p.k_pe, 64, L, 1, 128, L * 128, 64, kBN) ||
      !tensor_map_bf16(&v, p.values, 128, L, H, 256, L * 256, 64, kBN))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  attend_tc_kernel<<<w.ctas, kThreads, kSmem, s>>>(q, k, pe, v, p, w);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess || w.whole) return e;
  const int groups = (min(p.rows, kBM) + 7) / 8;
  attend_merge_kernel<<<dim3(w.tiles, groups), 256, 0, s>>>(p, w);
  note_launch();
  return cudaGetLastError();
}

}  // namespace mla
