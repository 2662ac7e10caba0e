// Cache eviction: keep a request's first tokens (sinks), its latest ones and, of the rest,
// those with the largest accumulated attention weight; close the gaps in the paged cache.
//
// Two kernels. evict_select_kernel finds what is kept, per request: the k-th largest weight by
// a radix selection (three passes of 11, 11 and 10 bits over the weights' order-preserving
// integer form, held in shared memory), then one ordered pass that writes the kept indices
// in ascending order, equal weights going to the lowest index. It reads each weight once:
// what bounds it is the latency of its passes, not bytes (32 requests of 4096 tokens 11 us). A long request is spread over the
// CTAs of a cluster, which add up their digit counts through distributed shared memory.
// evict_move_kernel then copies row kept[i] to row i and turns its rotary key by
// (i - kept[i]) theta_k, so that a row again carries the rotation of its own index, the one
// that mla_decode and mla_append_cache assume. It is bound by memory: every moved row is
// read and written once (32 requests, 2048 rows each, in place: 44.5 us with the selection, of which
// the move's look-ups take 4 and the rows 23; 256 ragged requests into new pages 178 us, 4.8 TB/s).
#include <cuda_fp16.h>
#include <math.h>

#include "internal.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace mla {
namespace {

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSegMax = (int)(kEvictMaxKeys / kMaxCluster);   // weights one CTA holds in shared memory

// Order-preserving integer form: larger weight, larger key; -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the block's threads; *total gets the sum.
template <int kSelThreads>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_tot, uint32_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_tot[wid] = x;
  __syncthreads();
  if (wid == 0) {
    uint32_t w = lane < kSelThreads / 32 ? warp_tot[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_tot[lane] = w;
  }
  __syncthreads();
  *total = warp_tot[31];
  return x - v + (wid ? warp_tot[wid - 1] : 0u);
}

constexpr int kSelStatic = 18 * 1024;          // of the selection's static shared memory, at most
struct SelShared {
  uint32_t hist[2][kBins];
  uint32_t warp_tot[32];
  uint32_t counts[2];                          // this CTA's weights above / at the threshold
  uint32_t digit, left, whole;                 // the chosen digit, how many of it are kept, and whether all
};
static_assert(sizeof(SelShared) <= kSelStatic && kSegMax * 4 + kSelStatic <= (int)kSmemPerCta, "shared memory per CTA");

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Cluster of C CTAs per request (blockIdx.x / C); CTA r holds the r-th contiguous segment of
// the tokens that are neither sinks nor recent.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(EvictParams p, int C) {
  constexpr int kBinsPer = kBins / kSelThreads;
  extern __shared__ float w_s[];
  __shared__ SelShared sh;
  const int b = blockIdx.x / C, rank = blockIdx.x % C, tid = threadIdx.x;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int S = p.seq_lens[b];
  int32_t* kept = p.kept + (long long)b * p.budget;
  const float* w = p.weights + (long long)b * p.max_pages * p.P;
  float* nw = p.new_weights ? p.new_weights + (long long)b * p.new_max_pages * p.P : nullptr;
  const long long cap = (long long)p.max_pages * p.P, new_cap = (long long)p.new_max_pages * p.P;
  const bool bad = S < 0 || S > cap || min(S, p.budget) > new_cap;
  // every CTA of the cluster has read the length before one of them may replace it (the new
  // lengths may be the same array)
  if (C > 1) ptx::cluster_sync();
  else __syncthreads();
  if (bad || S <= p.budget) {                  // uniform over the cluster
    if (bad && rank == 0 && tid == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    const int n = bad ? 0 : S;
    for (int i = rank * kSelThreads + tid; i < p.budget; i += C * kSelThreads) {
      kept[i] = i < n ? i : -1;
      if (i < n && nw && nw != w) nw[i] = w[i];
    }
    if (rank == 0 && tid == 0) p.new_seq_lens[b] = S;
    return;
  }
  const int n_mid = S - p.sinks - p.recent;
  const int seg = (n_mid + C - 1) / C;
  const int s0 = min(n_mid, rank * seg), len = min(n_mid, s0 + seg) - s0;
  const float* mine = w + p.sinks + s0;
  for (int i = tid; i < len; i += kSelThreads) w_s[i] = mine[i];
  uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent);
  uint32_t prefix = 0, mask = 0;
  // the radix passes (none if nothing of the middle is kept: the threshold stays above all)
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t bins = pass == 2 ? 1024u : 2048u;
      uint32_t* hist = sh.hist[pass & 1];
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0u;
      __syncthreads();
      const int steps = (len + kSelThreads - 1) / kSelThreads;
      for (int k = 0; k < steps; ++k) {
        const int i = k * kSelThreads + tid;
        const uint32_t key = i < len ? weight_key(w_s[i]) : 0u;
        const bool in = i < len && (key & mask) == prefix;
        const uint32_t d = in ? (key >> shift) & (bins - 1) : kBins;
        int same;
        __match_all_sync(0xffffffffu, d, &same);     // equal weights (zeros above all): one add
        if (same) {
          if (in && (tid & 31) == 0) atomicAdd(&hist[d], 32u);
        } else if (in) {
          atomicAdd(&hist[d], 1u);
        }
      }
      if (C > 1) ptx::cluster_sync();
      else __syncthreads();
      // bins from the top: thread t has (descending) the kBinsPer ones from its first
      const uint32_t d0 = kBins - 1 - kBinsPer * tid;
      uint32_t c[kBinsPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        c[i] = 0;
        if (C == 1) {
          c[i] = hist[d0 - i];
        } else {
          const uint32_t a = ptx::smem_u32(&hist[d0 - i]);
          for (int r = 0; r < C; ++r) c[i] += ld_dsmem_u32(ptx::map_to_rank(a, (uint32_t)r));
        }
        sum += c[i];
      }
      uint32_t total;
      uint32_t above = block_scan<kSelThreads>(sum, sh.warp_tot, &total);
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        if (above < want && want <= above + c[i]) {
          sh.digit = d0 - i;
          sh.left = want - above;
          sh.whole = want == above + c[i];
        }
        above += c[i];
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      mask |= (bins - 1) << shift;
      want = sh.left;
      const bool whole = sh.whole && prefix > 0;
      __syncthreads();
      if (whole) {                             // all weights of these digits are kept: no need of the rest
        prefix -= 1;                           // (those above this one)
        want = 0;
        break;
      }
    }
  } else {
    __syncthreads();
  }
  const bool any = mask != 0;                  // `want` weights equal to the threshold are kept
  // ordered pass: thread t has a contiguous run of the segment (odd length: no bank conflicts)
  const int per = ((len + kSelThreads - 1) / kSelThreads) | 1;
  const int i0 = min(len, tid * per), i1 = min(len, i0 + per);
  uint32_t gt = 0, eq = 0;
  if (any) {
    for (int i = i0; i < i1; ++i) {
      const uint32_t key = weight_key(w_s[i]);
      gt += key > prefix;
      eq += key == prefix;
    }
  }
  uint32_t total;
  // both counts of a CTA stay below 2^16: one scan for the two
  const uint32_t before = block_scan<kSelThreads>(gt | (eq << 16), sh.warp_tot, &total);
  uint32_t gt_before = before & 0xFFFFu, eq_before = before >> 16, out0 = 0;
  if (C > 1) {
    if (tid == 0) {
      sh.counts[0] = total & 0xFFFFu;
      sh.counts[1] = total >> 16;
    }
    ptx::cluster_sync();
    uint32_t eq_ranks = 0;
    for (int r = 0; r < rank; ++r) {
      out0 += ld_dsmem_u32(ptx::map_to_rank(ptx::smem_u32(&sh.counts[0]), (uint32_t)r));
      eq_ranks += ld_dsmem_u32(ptx::map_to_rank(ptx::smem_u32(&sh.counts[1]), (uint32_t)r));
    }
    out0 += min(eq_ranks, want);               // ties that the ranks before this one keep
    // the ranks before took min(eq_ranks, want) ties; this one may take the rest
    want -= min(eq_ranks, want);
    ptx::cluster_sync();                       // counts read: the CTAs may leave
  }
  if (any) {
    uint32_t at = (uint32_t)p.sinks + out0 + gt_before + min(eq_before, want);
    for (int i = i0; i < i1; ++i) {
      const uint32_t key = weight_key(w_s[i]);
      const bool take = key > prefix || (key == prefix && eq_before < want);
      eq_before += key == prefix;
      if (take) {
        kept[at] = p.sinks + s0 + i;
        if (nw) nw[at] = w_s[i];
        ++at;
      }
    }
  }
  // sinks by the first CTA; the recent tokens by the last, in chunks read before written (in
  // place their new places may overlap their old ones, always to the left; the middle's new
  // places end before the first recent token)
  if (rank == 0) {
    for (int i = tid; i < p.sinks; i += kSelThreads) {
      kept[i] = i;
      if (nw && nw != w) nw[i] = w[i];
    }
    if (tid == 0) p.new_seq_lens[b] = p.budget;
  }
  if (rank == C - 1) {
    const int to = p.budget - p.recent, from = S - p.recent;
    for (int i0r = 0; i0r < p.recent; i0r += kSelThreads) {
      const int i = i0r + tid;
      const float v = (nw && i < p.recent) ? w[from + i] : 0.f;
      __syncthreads();
      if (i < p.recent) {
        kept[to + i] = from + i;
        if (nw) nw[to + i] = v;
      }
    }
  }
}

// ======================================================================== the move
template <int VB> struct Vec;
template <> struct Vec<16> { typedef uint4 type; };
template <> struct Vec<4> { typedef uint32_t type; };

// Turns the pairs of one vector of VB bytes at byte `off` of the rotary part, by `delta` positions.
// Kind: 0 fp32, 1 bf16, 2 e4m3 (codes; the scale cancels), 3 block-scaled rows (rotary part in
// bf16).
template <int kKind, int VB>
__device__ __forceinline__ void turn_vector(typename Vec<VB>::type& vec, int off, const TurnTable& tt, int delta) {
  constexpr int kPairBytes = kKind == 0 ? 8 : (kKind == 2 ? 2 : 4);
  uint32_t* words = reinterpret_cast<uint32_t*>(&vec);
#pragma unroll
  for (int q = 0; q < VB / kPairBytes; ++q) {
    float sn, cs;
    turn_sincos<kKind == 0>(tt, off / kPairBytes + q, delta, &sn, &cs);
    if constexpr (kKind == 0) {
      const float x0 = __uint_as_float(words[2 * q]), x1 = __uint_as_float(words[2 * q + 1]);
      words[2 * q] = __float_as_uint(x0 * cs - x1 * sn);
      words[2 * q + 1] = __float_as_uint(x0 * sn + x1 * cs);
    } else if constexpr (kKind == 2) {
      const uint32_t sh = 16u * (q & 1), pair = (words[q >> 1] >> sh) & 0xFFFFu;
      const float x0 = fp8_to_f32((uint8_t)pair), x1 = fp8_to_f32((uint8_t)(pair >> 8));
      const uint32_t y = (uint32_t)f32_to_fp8(x0 * cs - x1 * sn) |
                         ((uint32_t)f32_to_fp8(x0 * sn + x1 * cs) << 8);
      words[q >> 1] = (words[q >> 1] & ~(0xFFFFu << sh)) | (y << sh);
    } else {
      const float x0 = __uint_as_float(words[q] << 16), x1 = __uint_as_float(words[q] & 0xFFFF0000u);
      const __nv_bfloat162 y = __floats2bfloat162_rn(x0 * cs - x1 * sn, x0 * sn + x1 * cs);
      words[q] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 2048;                // rows whose places are looked up at a time
constexpr int kMoveU = 4;                      // vectors in flight per thread and chunk

// CTA (column slice, row part, request): copies its slice of rows kept[i] -> i. Slices of W vectors
// of the latent part come first, then slices of Wk vectors of the rotary part (narrower: their
// sines and cosines would otherwise make a few CTAs last). The slices of a row never meet, so in
// place a CTA only has to order itself: new places are at or before old ones, a chunk's rows are
// all read (a barrier) before the chunk is written, and later chunks read only rows behind it.
// The next chunk's loads are issued before this chunk's stores.
template <int kKind, int VB>
__global__ void __launch_bounds__(kMoveThreads, 3) evict_move_kernel(EvictParams p, int W, int Wk, int parts,
                                                                  int in_place) {
  typedef typename Vec<VB>::type V;
  __shared__ int src_s[kMoveRows], dst_s[kMoveRows];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();                         // the selection's kept tokens
  constexpr int kElem = kKind == 0 ? 4 : (kKind == 2 ? 1 : 2);
  const int nvec = (int)(p.row_bytes / VB), kvec = p.d_r * kElem / VB, lvec = nvec - kvec;
  const int lslices = (lvec + W - 1) / W;
  const bool rope = (int)blockIdx.x >= lslices;
  const int w = rope ? Wk : W, v0 = rope ? lvec + ((int)blockIdx.x - lslices) * Wk : (int)blockIdx.x * W;
  const int b = blockIdx.z, tid = threadIdx.x;
  const int vec = v0 + tid % w, lane_row = tid / w, rows_u = kMoveThreads / w;
  const bool mine = vec < (rope ? nvec : lvec);
  const int chunk = rows_u * kMoveU;
  const bool turn = rope && p.rotate;
  const int32_t* kept = p.kept + (long long)b * p.budget;
  // rows of this request: the new length, unless the request was skipped (kept[0] = -1)
  const int n = min(p.new_seq_lens[b], p.budget);
  if (n <= 0 || kept[0] < 0) return;
  const int r0 = (int)((long long)n * blockIdx.y / parts), r1 = (int)((long long)n * (blockIdx.y + 1) / parts);
  const int32_t* bt = p.block_table + (long long)b * p.max_pages;
  const int32_t* nt = p.new_block_table + (long long)b * p.new_max_pages;
  V* cache = reinterpret_cast<V*>(p.cache);
  const int shift = (p.P & (p.P - 1)) == 0 ? 31 - __clz(p.P) : -1;   // (a division costs 20 instructions)
  for (int base = r0; base < r1; base += kMoveRows) {
    const int m = min(kMoveRows, r1 - base);
    int moved = 0;
    __syncthreads();
#pragma unroll 8
    for (int x = tid; x < m; x += kMoveThreads) {
      const int i = base + x, j = kept[i];
      const int jp = shift >= 0 ? j >> shift : j / p.P, ip = shift >= 0 ? i >> shift : i / p.P;
      const int ps = bt[jp], pd = nt[ip];
      int src = -1, dst = -1;
      if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) {
        if (blockIdx.x == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
      } else {
        src = ps * p.P + (j - jp * p.P);
        dst = pd * p.P + (i - ip * p.P);
        if (src == dst) src = -1;              // already in its place
      }
      src_s[x] = src;
      dst_s[x] = dst;
      moved |= src >= 0;
    }
    if (!__syncthreads_or(moved)) continue;
    V cur[kMoveU], nxt[kMoveU];
    int from[kMoveU], from_nxt[kMoveU];
    auto load = [&](V* v, int* f, int c) {
#pragma unroll
      for (int u = 0; u < kMoveU; ++u) {
        const int x = c + lane_row + u * rows_u;
        f[u] = mine && x < m ? src_s[x] : -1;
        if (f[u] >= 0) v[u] = cache[(long long)f[u] * nvec + vec];
      }
    };
    load(cur, from, 0);
    for (int c = 0; c < m; c += chunk) {
      if (c + chunk < m) load(nxt, from_nxt, c + chunk);
      if (turn) {
#pragma unroll
        for (int u = 0; u < kMoveU; ++u) {
          const int i = base + c + lane_row + u * rows_u;
          if (from[u] < 0) continue;
          const int delta = i - kept[i];
          if (delta != 0) turn_vector<kKind, VB>(cur[u], (vec - lvec) * VB, p.tt, delta);
        }
      }
      if (in_place) __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveU; ++u)
        if (from[u] >= 0) cache[(long long)dst_s[c + lane_row + u * rows_u] * nvec + vec] = cur[u];
#pragma unroll
      for (int u = 0; u < kMoveU; ++u) {
        cur[u] = nxt[u];
        from[u] = from_nxt[u];
      }
    }
  }
}

template <int kKind, int VB>
cudaError_t move(const EvictParams& p, cudaStream_t s) {
  constexpr int kElem = kKind == 0 ? 4 : (kKind == 2 ? 1 : 2);
  const int nvec = (int)(p.row_bytes / VB), kvec = p.d_r * kElem / VB, lvec = nvec - kvec, sms = device_sms();
  const int in_place = p.new_block_table == p.block_table;
  // a line of a row at a time in place (32 requests of 4096 tokens 44.5 us; with 64 bytes 51, with 256
  // 55), two lines into new pages (256 ragged requests 178 us; with 128 bytes 184, with 512 183)
  int W = (in_place ? 128 : 256) / VB, parts = 1;
  const int Wk = 32 / VB;
  auto slices = [&]() { return (lvec + W - 1) / W + (kvec + Wk - 1) / Wk; };
  if (in_place) {
    // narrower slices for few requests, until the CTAs cover the SMs, down to 32-byte sectors
    while (W > 32 / VB && (long long)p.batch * slices() < sms) W /= 2;
  } else {
    // the rows in parts, until there are 8 CTAs per SM, of at least 256 rows
    const long long ctas = (long long)p.batch * slices(), most = (p.budget + 255) / 256;
    const long long want = 8LL * sms / ctas;
    parts = (int)(want < 1 ? 1 : (want < most ? want : most));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)slices(), (unsigned)parts, (unsigned)p.batch);
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_move_kernel<kKind, VB>, p, W, Wk, parts, in_place);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int kSelThreads>
cudaError_t select(const EvictParams& p, int C, int seg, cudaStream_t s) {
  auto kern = evict_select_kernel<kSelThreads>;
  const size_t smem = (size_t)(seg > 1 ? seg : 1) * 4;
  cudaError_t e = allow_smem(kern, smem, kSelStatic);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * C), 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, p, C);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t launch_evict(mla_dtype cache, const EvictParams& p, cudaStream_t s) {
  const long long keys = (long long)p.max_pages * p.P;
  int C = 1;
  while (C < kMaxCluster && keys > 16384LL * C) C *= 2;
  const int seg = (int)((keys + C - 1) / C);
  if (seg > kSegMax) return cudaErrorInvalidValue;
  // 1024 threads where every CTA has an SM to itself; otherwise 512, two of which fit on one (256
  // requests of up to 8192 tokens: one wave instead of two, 178.3 us in all instead of 180.2)
  cudaError_t e = p.batch * C <= device_sms() ? select<1024>(p, C, seg, s) : select<512>(p, C, seg, s);
  if (e != cudaSuccess) return e;
  // 16 bytes at a time where the rows and both of their parts allow it
  const int kpe = p.d_r * (cache == MLA_FP8_E4M3 ? 1 : 2);
  const bool wide = p.row_bytes % 16 == 0 && kpe % 16 == 0 && ((uintptr_t)p.cache & 15) == 0;
  switch (cache) {
    case MLA_F32: return move<0, 16>(p, s);
    case MLA_BF16: return wide ? move<1, 16>(p, s) : move<1, 4>(p, s);
    case MLA_FP8_E4M3: return wide ? move<2, 16>(p, s) : move<2, 4>(p, s);
    default: return wide ? move<3, 16>(p, s) : move<3, 4>(p, s);
  }
}

}  // namespace mla
