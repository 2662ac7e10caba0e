// Attention of a whole batch to an expanded prefix, on the tensor cores (bf16, DeepSeek-V2 head
// shape: d_n 128, d_r 64, d_v 128).
//
// Every request's query tokens are the rows of one matrix per head, so the prefix's keys and
// values are read once for all of a tile's rows. Per head, row tile and block of 128 keys:
//   S = [q_nope ; q_hi ; q_lo] [K ; k_pe ; k_pe]^T   (K = 128 + 64 + 64 of the MMA)
//   P = exp2(c S - c m),  O += P V,  l += sum P      (c = softmax scale * log2 e)
// The rotated query is the sum of two bf16 terms (off by at most 2^-17 of an element; q_nope and the
// keys are exact), since the LSE is joined with another one: the low term costs a fifth of the MMA
// time; bf16 alone would put up to 2^-8 of the rotary score's terms into the LSE. P is rounded to
// bf16 as the operand of O (its sum l is not): at most 2^-8 of a weight, about what the rounding of u
// to bf16 does; a second term would double O's MMAs, and P and O have no tensor memory to spare.
//
// A tile is 128 rows on one CTA, or, with more than 128 rows in the batch, 256 rows on a CTA pair
// whose MMAs run over both (cta_group::2, M = 256): each CTA holds half the keys of a block
// (the N of S) and half the values' dims (the N of O), so a pair reads the prefix once for 256
// rows and each CTA's operand reads and fills are halved.
//
// Tensor memory (512 columns): Q 128 (the A operand of S; from shared memory it would take half
// of that memory's read rate), S two buffers of 128, O 128. P (bf16) takes the place of its S.
// The MMA warp issues S(n + 1), then O(n): the softmax of a block runs under the next block's
// scores. Two threads per row, 64 columns each, in two warpgroups, share the row maximum through
// shared memory; the reference m moves only when the maximum grows by more than 2^8 (O is then
// rescaled in tensor memory). P is handed to the MMAs in two parts, since the time from S to P is
// what the pipeline waits for.
//
// Work: the (head, row tile, key block) triples in this order are cut into one contiguous range
// per CTA (or pair); a range may start and end inside a tile, whose pieces then go to the
// workspace (fp32) and are merged by attend_merge_kernel. If whole tiles spread evenly enough,
// the cuts are put between tiles.
//
// Times are those of a call in a graph of the same calls (a call by itself takes 7 us more).
// Bound: at up to about 200 rows the keys' and values' bytes (64 KB per head and block): 128 rows x
// 8192 keys take 90 us, 6.1 TB/s. Above, the MMAs would be (54 us for 256 rows x 4096 keys with the
// low term); it takes 80, since a block's softmax, about as long as its MMAs, overlaps them in part only
// and 128 heads are two rounds of 76 pairs.
#include <math.h>

#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"
#include "tc_wait.cuh"

namespace mla {
namespace attend {

constexpr int kBN = 128;                           // keys of a block
template <bool kPair> struct Cfg {
  static constexpr int kCtas = kPair ? 2 : 1;      // CTAs of a tile
  static constexpr int kKeys = kBN / kCtas;        // keys of a block in this CTA
  static constexpr int kKBox = kKeys * 128;        // 64 bf16 of each of them, 128-byte swizzle
  static constexpr int kKStage = 3 * kKBox;        // content 0-63, 64-127, rotary
  static constexpr int kVBox = kBN * 128;          // 64 dims of every value of the block
  static constexpr int kVStage = kVBox * (kPair ? 1 : 2);
  static constexpr int kNK = kPair ? 5 : 3, kNV = kPair ? 4 : 2;
  static constexpr int kOffV = kNK * kKStage;
  static constexpr int kOffRed = kOffV + kNV * kVStage;   // row maxima [block parity][half][128]
  static constexpr int kOffBar = kOffRed + 2048;
  static constexpr int kSmem = kOffBar + 512 + 1024;      // + slack to align the base to 1 KB
  static constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128 * kCtas, 128, false, false);
  static constexpr uint32_t kIdescO = ptx::idesc_bf16_f32(128 * kCtas, 128, false, true);
};
static_assert(Cfg<false>::kSmem <= 232448 && Cfg<true>::kSmem <= 232448, "dynamic shared memory per CTA");
constexpr int kThreads = 384;
constexpr uint32_t kColQ = 0, kColS = 128, kColO = 384;
constexpr float kRescale = 8.f;                    // log2 units

// In a pair, KFULL, VFULL, QFULL and PREADY are those of the even CTA, whose MMA warp waits for
// both; the MMAs' commits (KEMPTY, VEMPTY, QEMPTY, SFULL, ODONE) go to both. SFULL, PREADY and ODONE
// are per S buffer: a wait is never two phases behind, since S(n) is complete only after O(n - 2).
enum { B_KFULL = 0, B_KEMPTY = 5, B_VFULL = 10, B_VEMPTY = 14, B_QFULL = 18, B_QEMPTY, B_SFULL, B_PREADY = 22,
       B_ODONE = 26, B_OFREE = 28, B_RED, B_TEAR = B_RED + 8, B_COUNT };
static_assert(B_COUNT * 8 <= 480, "barrier area");

struct Work {
  int tiles, row_tiles, blocks;                    // tiles = H * row_tiles; blocks per tile
  int workers;                                     // CTAs or pairs
  int pair;
  int whole;                                       // 1: cuts between tiles only
  float* part_o;                                   // [2 CTAs][32][128][4]: columns by 4, rows, column
  float* part_lse;                                 // [2 CTAs][128], log2 units
  __host__ __device__ long long begin(int c) const {
    return whole ? (long long)c * tiles / workers * blocks : (long long)c * tiles * blocks / workers;
  }
};

struct Segments {                                  // the pieces of a worker's range, in order
  const Work* w;
  long long u, end;
  int tile, k0, k1;
  __device__ Segments(const Work& work, int c) : w(&work), u(work.begin(c)), end(work.begin(c + 1)) {}
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

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_pe,
                     const __grid_constant__ CUtensorMap tm_v, const PrefixAttendParams p, const Work work) {
  using C = Cfg<kPair>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  volatile int* abort = reinterpret_cast<volatile int*>(basep + C::kOffBar + 496);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(basep + C::kOffBar + 500);
  auto bar = [&](int i) { return base + C::kOffBar + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kPair ? (int)ptx::cluster_ctarank() : 0;
  const int worker = kPair ? blockIdx.x >> 1 : blockIdx.x;
  // the barriers that the MMA warp waits on, as an address that both CTAs can signal
  auto lead = [&](int i) { return kPair ? ptx::map_to_rank(bar(i), 0u) : bar(i); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      int n = 1;
      if (i == B_QFULL || i == B_OFREE || (i >= B_PREADY && i < B_ODONE)) n = 8 * C::kCtas;   // softmax warps
      if (i >= B_RED && i < B_TEAR) n = 2;                                    // the halves' warps
      ptx::mbar_init(bar(i), n);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_pe);
    ptx::prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  if (kPair) ptx::cluster_sync();                  // both CTAs run, with their barriers set up
  if (warp == 1) {
    if (kPair) {
      ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (kPair) ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  auto wait = [&](int i, uint32_t parity) { return bounded_wait(bar(i), parity, abort, p.status); };
  // a warp goes on, or gives up, as one
  auto wait_w = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  auto wait_lead = [&](int i, uint32_t parity) {   // for what the other CTA's threads arrived on
    return __all_sync(0xffffffffu, bounded_wait<kPair>(bar(i), parity, abort, p.status)) != 0;
  };
  Segments seg(work, worker);

  // registers: the softmax warps hold half a row of scores twice (launched with 168 x 384; 88 x 128
  // + 200 x 256 = 62464 of the 64512 after the split)
  if (warp < 4) {
    ptx::setmaxnreg_dec<88>();
    if (warp == 0) {
      if (lane == 0) {                             // keys
        const uint64_t pol = ptx::l2_policy_evict_first();
        const bool once = work.row_tiles == 1;     // each key is read by one tile
        uint32_t g = 0;
        bool ok = true;
        while (ok && seg.next()) {
          const int h = seg.tile / work.row_tiles;
          for (int kb = seg.k0; kb < seg.k1; ++kb, ++g) {
            const uint32_t st = g % C::kNK;
            if (!(ok = wait(B_KEMPTY + st, ((g / C::kNK) & 1) ^ 1))) break;
            const uint32_t dst = base + st * C::kKStage, full = lead(B_KFULL + st);
            const int y = kb * kBN + C::kKeys * rank;
            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_KFULL + st), C::kCtas * C::kKStage);
            if (kPair) {
              if (once) {
                ptx::tma_load_3d_pair_hint(dst, &tm_k, 0, y, h, full, pol);
                ptx::tma_load_3d_pair_hint(dst + C::kKBox, &tm_k, 64, y, h, full, pol);
              } else {
                ptx::tma_load_3d_pair(dst, &tm_k, 0, y, h, full);
                ptx::tma_load_3d_pair(dst + C::kKBox, &tm_k, 64, y, h, full);
              }
              ptx::tma_load_3d_pair(dst + 2 * C::kKBox, &tm_pe, 0, y, 0, full);
            } else {
              ptx::tma_load_3d_hint(dst, &tm_k, 0, y, h, full, pol);
              ptx::tma_load_3d_hint(dst + C::kKBox, &tm_k, 64, y, h, full, pol);
              ptx::tma_load_3d(dst + 2 * C::kKBox, &tm_pe, 0, y, 0, full);
            }
          }
        }
        if (*abort && rank == 0)
          for (uint32_t i = g > C::kNK ? g - C::kNK : 0; i < g; ++i)
            drain_wait(bar(B_KFULL + i % C::kNK), (i / C::kNK) & 1);
      }
    } else if (warp == 3) {
      if (lane == 0) {                             // values
        const uint64_t pol = ptx::l2_policy_evict_first();
        const bool once = work.row_tiles == 1;
        uint32_t g = 0;
        bool ok = true;
        while (ok && seg.next()) {
          const int h = seg.tile / work.row_tiles;
          for (int kb = seg.k0; kb < seg.k1; ++kb, ++g) {
            const uint32_t st = g % C::kNV;
            if (!(ok = wait(B_VEMPTY + st, ((g / C::kNV) & 1) ^ 1))) break;
            const uint32_t dst = base + C::kOffV + st * C::kVStage, full = lead(B_VFULL + st);
            if (rank == 0) ptx::mbar_arrive_expect_tx(bar(B_VFULL + st), C::kCtas * C::kVStage);
            if (kPair) {
              if (once) ptx::tma_load_3d_pair_hint(dst, &tm_v, 64 * rank, kb * kBN, h, full, pol);
              else ptx::tma_load_3d_pair(dst, &tm_v, 64 * rank, kb * kBN, h, full);
            } else {
              ptx::tma_load_3d_hint(dst, &tm_v, 0, kb * kBN, h, full, pol);
              ptx::tma_load_3d_hint(dst + C::kVBox, &tm_v, 64, kb * kBN, h, full, pol);
            }
          }
        }
        if (*abort && rank == 0)
          for (uint32_t i = g > C::kNV ? g - C::kNV : 0; i < g; ++i)
            drain_wait(bar(B_VFULL + i % C::kNV), (i / C::kNV) & 1);
      }
    } else if (warp == 1 && rank == 0) {
      // MMAs: S(n + 1), then O(n); n counts the blocks of all segments
      auto commit = [&](int i) {
        if (kPair) ptx::mma_commit_pair(bar(i));
        else ptx::mma_commit(bar(i));
      };
      uint32_t ns = 0, no = 0, s = 0;              // scores and outputs issued, segments
      bool ok = true;
      auto out = [&](bool first) {
        const uint32_t b = no & 1, st = no % C::kNV;
        if (!wait_lead(B_VFULL + st, (no / C::kNV) & 1)) return false;
        // a segment's first product overwrites O: its owners have read the one before
        if (first && !wait_lead(B_OFREE, (s & 1) ^ 1)) return false;
        const uint32_t v = base + C::kOffV + st * C::kVStage;
#pragma unroll
        for (int part = 0; part < 2; ++part) {     // keys 0-31 and 64-95 of the block, then the rest
          if (!wait_lead(B_PREADY + 2 * part + b, (no >> 1) & 1)) return false;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 2 * part + (i & 1) + 4 * (i >> 1);       // keys 16 k ..
              const uint32_t a = tmem + kColS + 128 * b + (k < 4 ? 8 * k : 64 + 8 * (k - 4));
              const uint64_t bd = ptx::smem_desc(v + 2048 * k, C::kVBox, 1024, ptx::kSwizzle128);
              if (kPair) ptx::mma_bf16_ts_pair(tmem + kColO, a, bd, C::kIdescO, (!first || k) ? 1u : 0u);
              else ptx::mma_bf16_ts(tmem + kColO, a, bd, C::kIdescO, (!first || k) ? 1u : 0u);
            }
            if (part == 1) {
              commit(B_VEMPTY + st);
              commit(B_ODONE + b);
            }
          }
          __syncwarp();
        }
        ++no;
        return true;
      };
      while (ok && seg.next()) {
        ok = wait_lead(B_QFULL, s & 1);
        const int nb = seg.k1 - seg.k0;
        for (int n = 0; ok && n < nb; ++n) {
          const uint32_t b = ns & 1, st = ns % C::kNK;
          if (!(ok = wait_lead(B_KFULL + st, (ns / C::kNK) & 1))) break;
          ptx::tc_fence_after();
          // S overwrites the S and P of two blocks ago, whose product was issued before
          const uint32_t k0 = base + st * C::kKStage;
          if (ptx::elect_one()) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t box = j < 12 ? j >> 2 : 2;      // the low rotary term meets k_pe again
              const uint64_t bd = ptx::smem_desc(k0 + box * C::kKBox + 32 * (j & 3), 16, 1024, ptx::kSwizzle128);
              if (kPair) ptx::mma_bf16_ts_pair(tmem + kColS + 128 * b, tmem + kColQ + 8 * j, bd, C::kIdescS, j ? 1u : 0u);
              else ptx::mma_bf16_ts(tmem + kColS + 128 * b, tmem + kColQ + 8 * j, bd, C::kIdescS, j ? 1u : 0u);
            }
            commit(B_KEMPTY + st);
            commit(B_SFULL + b);
            if (n == nb - 1) commit(B_QEMPTY);
          }
          __syncwarp();
          ++ns;
          if (n > 0) ok = out(n == 1);
        }
        if (ok) ok = out(nb == 1);
        ++s;
      }
      if (*abort) {
        if (ptx::elect_one()) commit(B_TEAR);
        __syncwarp();
        drain_wait(bar(B_TEAR), 0);
      }
    }
  } else {
    ptx::setmaxnreg_inc<200>();
    // softmax: thread = row of the CTA's tile = lane of tensor memory, columns 64 w .. 64 w + 63
    const int w = warp >= 8 ? 1 : 0, quad = warp & 3, row = 32 * quad + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t t_o = t_lane + kColO + 64 * w;
    const float c = p.scale_log2;
    float* red = reinterpret_cast<float*>(basep + C::kOffRed);
    const uint32_t qfull = lead(B_QFULL), pready = lead(B_PREADY), ofree = lead(B_OFREE);
    // What these arrivals announce lies in tensor memory (stores or loads already waited for), so
    // the pair's need no release: one at cluster scope waits out the thread's memory traffic
    // first (it cost 1.1 us of every block).
    auto arrive = [&](uint32_t b) {
      if (kPair) ptx::mbar_arrive_remote_relaxed(b);
      else ptx::mbar_arrive(b);
    };
    uint32_t g = 0, x = 0, s = 0;                  // blocks, exchanges and segments so far
    bool ok = true;
    // what the other half's thread of this row wrote (each exchange has its parity's slots)
    auto swap = [&](float mine, float* other) {
      const uint32_t b = x & 1;
      red[b * 256 + w * 128 + row] = mine;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(B_RED + 2 * quad + b));
      const bool good = wait_w(B_RED + 2 * quad + b, (x >> 1) & 1);
      *other = red[b * 256 + (w ^ 1) * 128 + row];
      ++x;
      return good;
    };
    // The row's query, raw: dims 64 w .. of the content part, pairs 16 w .. of the rotary part. It is
    // asked for before the segment before it is written out.
    uint4 qn[8], qr[4];
    int S = 0;                                     // own length of the row's request
    bool live = false;
    auto fetch = [&](const Segments& sg) {
      const int h = sg.tile / work.row_tiles;
      const int r = (sg.tile % work.row_tiles * C::kCtas + rank) * 128 + row;
      const uint4* n = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(p.q_nope) +
                                                      ((long long)r * p.H + h) * 128 + 64 * w);
      const uint4* e = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(p.q_pe) +
                                                      ((long long)r * p.H + h) * 64 + 32 * w);
#pragma unroll
      for (int i = 0; i < 8; ++i) qn[i] = r < p.rows ? n[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < 4; ++i) qr[i] = r < p.rows ? e[i] : make_uint4(0u, 0u, 0u, 0u);
      S = r < p.rows ? p.seq_lens[r / p.q_len] : 0;
      live = r < p.rows && S >= p.q_len;
      if (r < p.rows && S != 0 && S < p.q_len && h == 0 && sg.k0 == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    };
    bool more = seg.next();
    if (more) fetch(seg);
    while (ok && more) {
      const int h = seg.tile / work.row_tiles;
      const int r = (seg.tile % work.row_tiles * C::kCtas + rank) * 128 + row;
      const int nb = seg.k1 - seg.k0;
      const bool full = seg.k0 == 0 && seg.k1 == work.blocks;
      const int k_first = seg.k0;
      const bool row_live = live;
      {
        uint32_t hi[16], lo[16], raw_n[32];
        const long long pos = (long long)p.L + S - p.q_len + r % p.q_len;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          raw_n[4 * i] = qn[i].x;
          raw_n[4 * i + 1] = qn[i].y;
          raw_n[4 * i + 2] = qn[i].z;
          raw_n[4 * i + 3] = qn[i].w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t y = (i & 3) == 0 ? qr[i >> 2].x : ((i & 3) == 1 ? qr[i >> 2].y : ((i & 3) == 2 ? qr[i >> 2].z : qr[i >> 2].w));
          float sn, cs;
          turn_sincos<false>(p.tt, 16 * w + i, pos, &sn, &cs);
          const float a = __uint_as_float(y << 16), b = __uint_as_float(y & 0xFFFF0000u);
          const float y0 = a * cs - b * sn, y1 = a * sn + b * cs;
          const __nv_bfloat162 t = __floats2bfloat162_rn(y0, y1);
          const float2 f = __bfloat1622float2(t);
          const __nv_bfloat162 u = __floats2bfloat162_rn(y0 - f.x, y1 - f.y);
          hi[i] = *reinterpret_cast<const uint32_t*>(&t);
          lo[i] = *reinterpret_cast<const uint32_t*>(&u);
        }
        if (!(ok = wait_w(B_QEMPTY, (s & 1) ^ 1))) break;
        ptx::tc_fence_after();
        ptx::tmem_st32(t_lane + kColQ + 32 * w, raw_n);
        ptx::tmem_st16(t_lane + kColQ + 64 + 16 * w, hi);
        ptx::tmem_st16(t_lane + kColQ + 96 + 16 * w, lo);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(qfull);
      }
      float m = -INFINITY, l = 0.f;
      for (int n = 0; n < nb; ++n, ++g) {
        const uint32_t t_s = t_lane + kColS + 128 * (g & 1) + 64 * w;
        if (!(ok = wait_w(B_SFULL + (g & 1), (g >> 1) & 1))) break;
        ptx::tc_fence_after();
        uint32_t v[2][32];
        ptx::tmem_ld32(t_s, v[0]);
        ptx::tmem_ld32(t_s + 32, v[1]);
        ptx::tmem_wait_ld();
        const int valid = p.L - (k_first + n) * kBN - 64 * w;
        if (valid < 64) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * q + j >= valid) v[q][j] = 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; j += 4)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(v[q >> 1][j + 2 * (q & 1)]),
                                       __uint_as_float(v[q >> 1][j + 2 * (q & 1) + 1])));
        float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const uint32_t b = x & 1;
        red[b * 256 + w * 128 + row] = mb;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(B_RED + 2 * quad + b));
        if (!(ok = wait_w(B_RED + 2 * quad + b, (x >> 1) & 1))) break;
        mb = fmaxf(mb, red[b * 256 + (w ^ 1) * 128 + row]);
        ++x;
        if (n == 0) {
          m = mb;
        } else {
          const bool grow = (mb - m) * c > kRescale;
          // tensor-memory accesses are warp-wide: a warp's rows are rescaled together
          if (__any_sync(0xffffffffu, grow)) {
            if (!(ok = wait_w(B_ODONE + ((g - 1) & 1), ((g - 1) >> 1) & 1))) break;
            ptx::tc_fence_after();
            // (no branch: the warp stays together for the accesses below; m = -infinity gives 0)
            const float shrink = ptx::ex2((m - mb) * c), a = grow ? shrink : 1.f;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t o[16];
              ptx::tmem_ld16(t_o + 16 * q, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
              ptx::tmem_st16(t_o + 16 * q, o);
            }
            l *= a;
            if (grow) m = mb;
          }
        }
        // P against the reference m (columns behind the prefix hold -infinity: 0), handed over in
        // two parts: the product with the first 32 columns' keys runs while the rest are formed
        const float off = m == -INFINITY ? 0.f : m * c;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float e0 = ptx::ex2(fmaf(__uint_as_float(v[q][j]), c, -off));
            const float e1 = ptx::ex2(fmaf(__uint_as_float(v[q][j + 1]), c, -off));
            part[j & 2] += e0;
            part[(j & 2) + 1] += e1;
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
            pk[j >> 1] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          ptx::tmem_st16(t_s + 16 * q, pk);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(pready + 8 * (2 * q + (g & 1)));
        }
        l += (part[0] + part[1]) + (part[2] + part[3]);
      }
      if (!ok) break;
      more = seg.next();
      if (more) fetch(seg);                        // (the tile's own h, r and row_live are kept above)
      float l_other = 0.f;
      if (!(ok = swap(l, &l_other))) break;
      const float L = w ? l_other + l : l + l_other;
      const float inv = L == 0.f ? 0.f : 1.f / L;      // (a NaN in the scores stays one)
      if (!(ok = wait_w(B_ODONE + ((g - 1) & 1), ((g - 1) >> 1) & 1))) break;
      ptx::tc_fence_after();
      const long long slot = 2LL * blockIdx.x + (k_first == 0 ? 1 : 0);
      if (w == 0) {
        const float lse2 = L == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * c) + log2f(L);
        if (!full) work.part_lse[slot * 128 + row] = lse2;
        else if (r < p.rows) p.lse[(long long)r * p.H + h] = row_live ? lse2 * kLn2 : -INFINITY;
      }
      uint32_t o[2][32];                           // output columns 64 w .. 64 w + 63
      __syncwarp();                                // the loads are warp-wide
      ptx::tmem_ld32(t_o, o[0]);
      ptx::tmem_ld32(t_o + 32, o[1]);
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(ofree);
      if (r < p.rows) {
        if (!full) {
          // [slot][column / 4][row] float4: a warp's rows side by side
          float4* dst = reinterpret_cast<float4*>(work.part_o) + (slot * 32 + 16 * w) * 128 + row;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t* y = &o[j >> 3][4 * (j & 7)];
            dst[j * 128] = make_float4(__uint_as_float(y[0]) * inv, __uint_as_float(y[1]) * inv,
                                       __uint_as_float(y[2]) * inv, __uint_as_float(y[3]) * inv);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(p.u) + ((long long)r * p.H + h) * 128 + 64 * w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* y = &o[j >> 2][8 * (j & 3) + 2 * i];
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(row_live ? __uint_as_float(y[0]) * inv : 0.f,
                                                              row_live ? __uint_as_float(y[1]) * inv : 0.f);
              k[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dst[j] = make_uint4(k[0], k[1], k[2], k[3]);
          }
        }
      }
      ++s;
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (kPair) ptx::cluster_sync();                  // no copy, arrival or MMA of the pair is on its way
  if (warp == 1) {
    ptx::tc_fence_after();
    if (kPair) ptx::tmem_dealloc_pair(tmem, 512);
    else ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of a tile that was cut: out = sum_s w_s o_s, w_s = 2^(lse_s - L). Block (tile, 16
// columns), thread per row.
__global__ void __launch_bounds__(256) attend_merge_kernel(const PrefixAttendParams p, const Work work) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tile = blockIdx.x, rows = work.pair ? 256 : 128, tr = threadIdx.x;
  const int h = tile / work.row_tiles, r = tile % work.row_tiles * rows + tr;
  if (r >= p.rows) return;
  const long long t0 = (long long)tile * work.blocks, t1 = t0 + work.blocks;
  // the workers whose ranges hold the tile's first and last block
  const long long U = (long long)work.tiles * work.blocks;
  auto owner = [&](long long u) {
    int c = (int)(u * work.workers / U);
    while (work.begin(c + 1) <= u) ++c;
    while (work.begin(c) > u) --c;
    return c;
  };
  const int c0 = owner(t0), c1 = owner(t1 - 1);
  if (c0 == c1) return;                            // written whole
  const int rank = tr >> 7, row = tr & 127;
  auto slot = [&](int c) {
    const int cta = work.pair ? 2 * c + rank : c;
    return 2LL * cta + (c == c0 ? 1 : 0);
  };
  const int S = p.seq_lens[r / p.q_len];
  float m = -INFINITY;
  bool nan = false;
  for (int c = c0; c <= c1; ++c) {
    const float lse = work.part_lse[slot(c) * 128 + row];
    nan |= lse != lse;
    m = fmaxf(m, lse);
  }
  float acc[16] = {};
  float sum = 0.f;
  const bool live = S >= p.q_len && (nan || m > -INFINITY);
  if (live) {
    for (int c = c0; c <= c1; ++c) {
      const float w = ptx::ex2(work.part_lse[slot(c) * 128 + row] - m);
      const float4* o = reinterpret_cast<const float4*>(work.part_o) + (slot(c) * 32 + 4 * blockIdx.y) * 128 + row;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 y = o[i * 128];
        acc[4 * i] = fmaf(w, y.x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(w, y.y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(w, y.z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(w, y.w, acc[4 * i + 3]);
      }
      sum += w;
    }
  }
  const float inv = live ? 1.f / sum : 0.f;
  uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(p.u) + ((long long)r * p.H + h) * 128 + 16 * blockIdx.y);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[8 * j + 2 * i] * inv, acc[8 * j + 2 * i + 1] * inv);
      k[i] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    dst[j] = make_uint4(k[0], k[1], k[2], k[3]);
  }
  if (blockIdx.y == 0) p.lse[(long long)r * p.H + h] = live ? (m + log2f(sum)) * kLn2 : -INFINITY;
}

// Cuts between tiles unless that leaves a worker this many blocks (of about a microsecond) more
// than an even share: a cut tile costs a second epilogue and query load, its pieces' way through
// the workspace and the merge, 10 us in all. Measured where whole tiles leave 64 blocks instead of
// 54: 90.1 us uncut and 96.8 cut at 128 rows x 8192 keys, 79.9 and 82.6 at 256 rows x 4096 keys.
constexpr int kCutGain = 12;

static Work plan(int rows, int H, int L) {
  Work w{};
  w.pair = rows > 128 ? 1 : 0;
  const int tile_rows = w.pair ? 256 : 128;
  w.row_tiles = (rows + tile_rows - 1) / tile_rows;
  w.tiles = H * w.row_tiles;
  w.blocks = (L + kBN - 1) / kBN;
  const int sms = device_sms();
  const int most = w.pair ? (sms > 1 ? sms / 2 : 1) : sms;
  const long long units = (long long)w.tiles * w.blocks;
  const long long even = (units + most - 1) / most;
  const long long uncut = (long long)((w.tiles + most - 1) / most) * w.blocks;
  w.whole = uncut <= even + kCutGain;
  w.workers = w.whole ? (w.tiles < most ? w.tiles : most) : (int)(units < most ? units : most);
  return w;
}

template <bool kPair>
static cudaError_t run(const CUtensorMap& k, const CUtensorMap& pe, const CUtensorMap& v,
                       const PrefixAttendParams& p, const Work& w, cudaStream_t s) {
  using C = Cfg<kPair>;
  auto kern = attend_tc_kernel<kPair>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(w.workers * C::kCtas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, k, pe, v, p, w);
  if (e != cudaSuccess) return e;
  note_launch();
  if (w.whole) return cudaSuccess;
  cfg.gridDim = dim3((unsigned)w.tiles, 8, 1);
  cfg.blockDim = dim3(128 * C::kCtas, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attend_merge_kernel, p, w);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace attend

bool prefix_attend_tc_supported(const mla_config* c) {
  return c->act_dtype == MLA_BF16 && c->d_nope == 128 && c->d_rope == 64 && c->d_v == 128;
}

size_t prefix_attend_tc_workspace(int rows, int H, int L) {
  if (rows <= 0 || L <= 0) return 0;
  const attend::Work w = attend::plan(rows, H, L);
  return w.whole ? 0 : (size_t)2 * w.workers * (w.pair ? 2 : 1) * 128 * (128 + 1) * 4;
}

cudaError_t launch_prefix_attend_tc(const PrefixAttendParams& p, void* workspace, cudaStream_t s) {
  using namespace attend;
  Work w = plan(p.rows, p.H, p.L);
  w.part_o = (float*)workspace;
  w.part_lse = w.whole ? nullptr : w.part_o + (size_t)2 * w.workers * (w.pair ? 2 : 1) * 128 * 128;
  CUtensorMap k, pe, v;
  const uint64_t H = (uint64_t)p.H, L = (uint64_t)p.L;
  const uint32_t keys = w.pair ? kBN / 2 : kBN;
  if (!tensor_map_bf16(&k, p.keys, 128, L, H, 256, L * 256, 64, keys) ||
      !tensor_map_bf16(&pe, p.k_pe, 64, L, 1, 128, L * 128, 64, keys) ||
      !tensor_map_bf16(&v, p.values, 128, L, H, 256, L * 256, 64, kBN))
    return cudaErrorInvalidValue;
  return w.pair ? run<true>(k, pe, v, p, w, s) : run<false>(k, pe, v, p, w, s);
}

}  // namespace mla
