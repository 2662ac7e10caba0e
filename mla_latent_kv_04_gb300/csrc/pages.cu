// Page-sparse decoding: summaries of the cache's pages, their estimated attention (SIMT form; the
// tensor-core form is page_scores_tc.cu), the choice of the pages that a query keeps, and the
// prologue of the decode over chosen pages.
#include <math.h>

#include "fp8_tiles.cuh"
#include "internal.h"
#include "prologue.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace mla {
namespace {

// ======================================================================== page keys
// key_p = mean of the cached rows of page p, in fp32, rounded once. A block takes one page: its
// threads are (row group, VB-byte column) pairs that sum every G-th row, then the groups' sums are
// added in order. Bound by memory, which reads each row once: 32 x 4096 tokens of bf16 (151 MB) in 29 us among
// calls, 5.3 TB/s; e4m3 21 us and block scales 29, where conversions and the groups' sums add to it.
// Kind: 0 fp32, 1 bf16, 2 e4m3, 3 block-scaled e4m3 (codes, fp32 scales, bf16 rotary part).
constexpr int kKeyThreads = 288;               // 4 groups of a bf16 row's 72 columns, 8 of e4m3's 36, 7 of 41
// rows in flight per thread (block scales hold a scale for each as well: 4 of them take 38 us, 8 take 40, 16 65;
// the others at 8 as fast as at 4 or 16)
template <int kKind> constexpr int key_loads() { return kKind == 3 ? 4 : 8; }

template <int VB> struct KeyVec;
template <> struct KeyVec<16> { typedef uint4 type; };
template <> struct KeyVec<4> { typedef uint32_t type; };

template <int kKind, int VB, typename AT>
__global__ void __launch_bounds__(kKeyThreads) page_keys_kernel(PageKeysParams p, int G, int stride) {
  typedef typename KeyVec<VB>::type V;
  constexpr int kWords = VB / 4, kPer = kKind == 0 ? 1 : (kKind == 1 ? 2 : 4);   // elements of a word
  constexpr int kElems = kWords * kPer, kKeyLoads = key_loads<kKind>();
  extern __shared__ __align__(16) float sums[];                               // [G][D], or [G][cols][stride]
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int b = blockIdx.y, S = p.seq_lens[b], D = p.d_c + p.d_r;
  if (S <= 0 || S > (long long)p.max_pages * p.P) {
    if (S != 0 && blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    return;
  }
  const int pg = (S > p.new_tokens ? (S - p.new_tokens) / p.P : 0) + (int)blockIdx.x;
  if ((long long)pg * p.P >= S) return;
  const int page = p.block_table[(long long)b * p.max_pages + pg];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    return;
  }
  const int n = min(p.P, S - pg * p.P);
  const int cols = (int)(p.row_bytes / VB), grp = threadIdx.x / cols;
  const uint8_t* rows = reinterpret_cast<const uint8_t*>(p.cache) + (long long)page * p.P * p.row_bytes;
  const int code_words = p.d_c / 4, scale_words = p.d_c / 128;
  // (rows wider than the block's threads: one group, several columns a thread)
  for (int c = threadIdx.x % cols; c < cols && grp < G; c += kKeyThreads) {
    const int w0 = c * kWords;
    const bool code = kKind == 2 || (kKind == 3 && w0 < code_words);
    float acc[kElems];
#pragma unroll
    for (int i = 0; i < kElems; ++i) acc[i] = 0.f;
    for (int r0 = grp; r0 < n; r0 += kKeyLoads * G) {
      V v[kKeyLoads];
      float sc[kKeyLoads];
#pragma unroll
      for (int u = 0; u < kKeyLoads; ++u) {
        const int r = r0 + u * G;
        if (r >= n) break;
        const uint8_t* row = rows + (long long)r * p.row_bytes;
        v[u] = reinterpret_cast<const V*>(row)[c];
        sc[u] = kKind == 3 && code ? reinterpret_cast<const float*>(row)[code_words + w0 / 32] : 1.f;
      }
#pragma unroll
      for (int u = 0; u < kKeyLoads; ++u) {
        if (r0 + u * G >= n) break;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(&v[u]);
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const uint32_t x = words[j];
          if constexpr (kKind == 0) {
            acc[j] += __uint_as_float(x);
          } else if constexpr (kKind == 1) {
            acc[2 * j] += __uint_as_float(x << 16);
            acc[2 * j + 1] += __uint_as_float(x & 0xFFFF0000u);
          } else if (code) {
            const float2 a = e4m3x2_to_f32(x & 0xFFFFu), b = e4m3x2_to_f32(x >> 16);
            acc[4 * j] = fmaf(a.x, sc[u], acc[4 * j]);
            acc[4 * j + 1] = fmaf(a.y, sc[u], acc[4 * j + 1]);
            acc[4 * j + 2] = fmaf(b.x, sc[u], acc[4 * j + 2]);
            acc[4 * j + 3] = fmaf(b.y, sc[u], acc[4 * j + 3]);
          } else {
            acc[4 * j] += __uint_as_float(x << 16);
            acc[4 * j + 1] += __uint_as_float(x & 0xFFFF0000u);
          }
        }
      }
    }
    const int w = w0 - code_words - scale_words;                              // (kind 3: a rotary column's first word)
    if (stride > 0) {
      float* mine = sums + ((long long)grp * cols + c) * stride;
      if constexpr (kElems >= 4) {
        if (kKind < 3 || code) {
#pragma unroll
          for (int i = 0; i < kElems; i += 4)
            *reinterpret_cast<float4*>(mine + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < kWords; ++j) *reinterpret_cast<float2*>(mine + 2 * j) = make_float2(acc[4 * j], acc[4 * j + 1]);
        }
      }
    } else if (kKind < 3 || code) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) sums[(long long)grp * D + w0 * kPer + i] = acc[i];
    } else if (w >= 0) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        float* mine = sums + (long long)grp * D + p.d_c + 2 * (w + j);
        mine[0] = acc[4 * j];
        mine[1] = acc[4 * j + 1];
      }
    }
  }
  __syncthreads();
  AT* out = reinterpret_cast<AT*>(p.page_keys) + (long long)page * D;
  for (int d = threadIdx.x; d < D; d += kKeyThreads) {
    int at = d, step = D;
    if (stride > 0) {
      const int half = kElems / 2 > 0 ? kElems / 2 : 1;
      if (kKind < 3 || d < p.d_c) at = d / kElems * stride + d % kElems;
      else at = ((code_words + scale_words) / kWords + (d - p.d_c) / half) * stride + (d - p.d_c) % half;
      step = cols * stride;
    }
    float s = 0.f;
    for (int g = 0; g < G; ++g) s += sums[g * step + at];
    out[d] = from_f32<AT>(s * p.cache_scale / (float)n);
  }
}

// ======================================================================== page scores (SIMT)
// fp32, other shapes and addresses. Two passes over the keys, whose products are formed twice: nothing of size
// [heads][pages] is stored. Bound by latency and L1 (32 requests of 64 pages, 16 heads, 80 dims: 13 us).
// Pages that query (b, t) sees, and the tokens of page pg among them.
__device__ __forceinline__ int tokens_seen(const PageScoreParams& p, int g) {
  const int b = g / p.q_len, t = g % p.q_len, S = p.seq_lens[b];
  if (S < p.q_len || S <= 0 || S > (long long)p.max_pages * p.P) return 0;
  return S - p.q_len + t + 1;
}

// softmax scale * log2 e * q . key of one head and page; every lane of the warp gets it.
template <typename AT>
__device__ __forceinline__ float page_z(const PageScoreParams& p, const AT* q, int page, int lane) {
  const AT* key = reinterpret_cast<const AT*>(p.page_keys) + (long long)page * p.D;
  float acc = 0.f;
  for (int d = lane; d < p.D; d += 32) acc = fmaf(to_f32(q[d]), to_f32(key[d]), acc);
  return warp_sum(acc) * p.scale_log2;
}

// lse2[g][h] = log2 sum_pg m_pg 2^z (+inf without a page); a block per head, its warps take the pages in turn.
template <typename AT>
__global__ void __launch_bounds__(256) page_lse_kernel(PageScoreParams p) {
  __shared__ float2 part[8];
  const int g = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int see = tokens_seen(p, g);
  if (see == 0) {
    if (threadIdx.x == 0 && h == 0 && g % p.q_len == 0 && p.seq_lens[g / p.q_len] != 0)
      flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    return;
  }
  const int32_t* bt = p.block_table + (long long)(g / p.q_len) * p.max_pages;
  const AT* q = reinterpret_cast<const AT*>(p.q_lat) + ((long long)g * p.H + h) * p.D;
  float m = -INFINITY, l = 0.f;
  for (int pg = warp; (long long)pg * p.P < see; pg += 8) {
    const int page = bt[pg];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
      continue;
    }
    const float z = page_z(p, q, page, lane), top = fmaxf(m, z);
    if (z == -INFINITY) continue;
    l = (l > 0.f ? l * exp2f(m - top) : l) + exp2f(z - top) * (float)min(p.P, see - pg * p.P);
    m = top;
  }
  if (lane == 0) part[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < 8; ++w) m = fmaxf(m, part[w].x);
    l = 0.f;
    for (int w = 0; w < 8; ++w)
      if (part[w].y != 0.f) l = fmaf(part[w].y, exp2f(part[w].x - m), l);
    p.lse2[(long long)g * p.H + h] = l == 0.f ? INFINITY : m + log2f(l);
  }
}

// scores[g][pg] = m_pg sum_h 2^(z - lse2); a warp per page, over all heads.
template <typename AT>
__global__ void __launch_bounds__(256) page_mass_kernel(PageScoreParams p) {
  const int g = blockIdx.y, pg = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int see = tokens_seen(p, g);
  if ((long long)pg * p.P >= see) return;
  const int page = p.block_table[(long long)(g / p.q_len) * p.max_pages + pg];
  float s = 0.f;
  if (page >= 0 && page < p.num_pages) {
    const AT* q = reinterpret_cast<const AT*>(p.q_lat) + (long long)g * p.H * p.D;
    for (int h = 0; h < p.H; ++h)
      s += exp2f(page_z(p, q + (long long)h * p.D, page, lane) - p.lse2[(long long)g * p.H + h]);
  }
  if (lane == 0) p.scores[(long long)g * p.max_pages + pg] = s * (float)min(p.P, see - pg * p.P);
}

// ======================================================================== page selection
constexpr int kSelThreads = 512;
constexpr int kSelBins = 2048;

// Exclusive prefix sum of v over the block's threads.
__device__ __forceinline__ uint32_t sel_scan(uint32_t v, uint32_t* warp_tot) {
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
  return x - v + (wid ? warp_tot[wid - 1] : 0u);
}

// A block per query: radix selection of the want-th largest score of the middle (11, 11 and 10 bits of
// the scores' order-preserving integers), then one ordered pass that writes the list. Bound by latency, a
// chain of three histograms and scans: 32 queries of 512 pages 6.3 us among calls, 256 of up to 2048 11.3
// (the digits of two bits counted in registers, 25).
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(SelectParams p) {
  extern __shared__ uint32_t key_s[];                  // [pages of the middle]
  __shared__ uint32_t hist[kSelBins], warp_tot[32], digit, left;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int g = blockIdx.x, tid = threadIdx.x, b = g / p.q_len, S = p.seq_lens[b];
  int32_t* out = p.pages + (long long)g * p.budget;
  const bool bad = S < 0 || (S > 0 && S < p.q_len) || S > (long long)p.max_pages * p.P;
  if (bad && g % p.q_len == 0 && tid == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  const int n = bad || S == 0 ? 0 : (S - p.q_len + g % p.q_len) / p.P + 1;
  if (n <= p.budget) {
    for (int i = tid; i < p.budget; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int len = n - p.sinks - p.recent;
  const float* mine = p.scores + (long long)g * p.max_pages + p.sinks;
  for (int i = tid; i < len; i += kSelThreads) key_s[i] = order_key(mine[i]);
  uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent), prefix = 0, mask = 0;
  const bool any = want > 0;
  if (any) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t bins = pass == 2 ? 1024u : 2048u;
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0u;
      __syncthreads();
      for (int i = tid; i < len; i += kSelThreads) {
        const uint32_t key = key_s[i];
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      constexpr int kPer = kSelBins / kSelThreads;
      const int d0 = kSelBins - 1 - kPer * tid;        // bins from the top
      uint32_t c[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += c[i] = hist[d0 - i];
      uint32_t above = sel_scan(sum, warp_tot);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (above < want && want <= above + c[i]) {
          digit = (uint32_t)(d0 - i);
          left = want - above;
        }
        above += c[i];
      }
      __syncthreads();
      prefix |= digit << shift;
      mask |= (bins - 1) << shift;
      want = left;
      __syncthreads();
    }
    // thread t has a contiguous run of the middle; `want` of those equal to the threshold are kept
    const int per = (len + kSelThreads - 1) / kSelThreads;
    const int i0 = min(len, tid * per), i1 = min(len, i0 + per);
    uint32_t gt = 0, eq = 0;
    for (int i = i0; i < i1; ++i) {
      gt += key_s[i] > prefix;
      eq += key_s[i] == prefix;
    }
    const uint32_t before = sel_scan(gt | (eq << 16), warp_tot);
    uint32_t eq_before = before >> 16, at = (uint32_t)p.sinks + (before & 0xFFFFu) + min(eq_before, want);
    for (int i = i0; i < i1; ++i) {
      const uint32_t key = key_s[i];
      if (key > prefix || (key == prefix && eq_before < want)) out[at++] = p.sinks + i;
      eq_before += key == prefix;
    }
  }
  for (int i = tid; i < p.sinks; i += kSelThreads) out[i] = i;
  for (int i = tid; i < p.recent; i += kSelThreads) out[p.budget - p.recent + i] = n - p.recent + i;
}

// ======================================================================== decode over chosen pages
// Block 0 plans; block 1 + g writes the physical pages of query g's list. An entry that is out of
// order, behind a -1, or a page that the query does not see, becomes -1 and sets bad[g], which the merge of the pieces
// flags (block 0 clears the status word meanwhile). 6 us, the plan's chain of dependent steps.
__global__ void __launch_bounds__(256) pages_prep_kernel(PlanParams pp, const int32_t* __restrict__ block_table,
                                                         int32_t* __restrict__ table, int32_t* __restrict__ bad) {
  extern __shared__ int sm[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (blockIdx.x == 0) {
    plan_body(pp, sm, true);
    return;
  }
  const int g = blockIdx.x - 1, b = g / pp.q_len, S = pp.seq_lens[b];
  const int seen = S < pp.q_len || S <= 0 || S > (long long)pp.max_pages * pp.page_size
                       ? 0 : (S - pp.q_len + g % pp.q_len) / pp.page_size + 1;
  const int32_t* list = pp.pages + (long long)g * pp.budget;
  int wrong = 0;
  for (int k = threadIdx.x; k < pp.budget; k += 256) {
    const int pg = list[k], before = k > 0 ? list[k - 1] : -1;
    const bool ok = pg > before && pg < seen && (k == 0 || before >= 0);
    table[(long long)g * pp.budget + k] = ok ? block_table[(long long)b * pp.max_pages + pg] : -1;
    wrong |= pg >= 0 && !ok;
  }
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) bad[g] = wrong && seen > 0;
}

}  // namespace

// ======================================================================== launchers
template <int kKind, int VB, typename AT>
static cudaError_t page_keys_t(const PageKeysParams& p, cudaStream_t s) {
  const long long cols = p.row_bytes / VB;
  const int G = cols < kKeyThreads ? (int)(kKeyThreads / cols) : 1;
  constexpr int kElems = kKind == 0 ? VB / 4 : (kKind == 1 ? VB / 2 : VB);
  // Columns of 8 or 16 sums lie 4 words apart, so that a warp's 16-byte stores meet no bank twice (32 x 4096
  // tokens with a cold L2, element by element instead: e4m3 40 us against 30, block scales 60 against 40)
  const int stride = G > 1 && kElems >= 4 ? kElems + (kElems > 4 ? 4 : 0) : 0;
  const size_t smem = (size_t)G * (stride > 0 ? (size_t)cols * stride : p.d_c + p.d_r) * sizeof(float);
  auto kern = page_keys_kernel<kKind, VB, AT>;
  cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const long long touched = ((long long)p.new_tokens - 1) / p.P + 2;
  const unsigned gx = (unsigned)(touched < p.max_pages ? touched : p.max_pages);
  return launch_pdl(kern, dim3(gx, (unsigned)p.batch, 1), kKeyThreads, smem, s, p, G, stride);
}

bool page_keys_fits(int d_c, int d_r) { return (size_t)(d_c + d_r) * 4 <= kSmemPerCta; }

cudaError_t launch_page_keys(mla_dtype act, mla_dtype cache, const PageKeysParams& p, cudaStream_t s) {
  const bool v16 = p.row_bytes % 16 == 0 && ((uintptr_t)p.cache & 15) == 0;
  if (act == MLA_F32) return v16 ? page_keys_t<0, 16, float>(p, s) : page_keys_t<0, 4, float>(p, s);
  if (cache == MLA_BF16) return v16 ? page_keys_t<1, 16, bf16>(p, s) : page_keys_t<1, 4, bf16>(p, s);
  if (cache == MLA_FP8_E4M3) return v16 ? page_keys_t<2, 16, bf16>(p, s) : page_keys_t<2, 4, bf16>(p, s);
  // (a 16-byte column holds codes, scales or rotary values alone if the scales fill whole ones)
  return v16 && p.d_c % 512 == 0 ? page_keys_t<3, 16, bf16>(p, s) : page_keys_t<3, 4, bf16>(p, s);
}

template <typename AT>
static cudaError_t page_scores_t(const PageScoreParams& p, cudaStream_t s) {
  page_lse_kernel<AT><<<dim3((unsigned)p.groups, (unsigned)p.H, 1), 256, 0, s>>>(p);
  page_mass_kernel<AT><<<dim3((unsigned)((p.max_pages + 7) / 8), (unsigned)p.groups, 1), 256, 0, s>>>(p);
  note_launch(2);
  return cudaGetLastError();
}
cudaError_t launch_page_scores_simt(mla_dtype act, const PageScoreParams& p, cudaStream_t s) {
  return act == MLA_F32 ? page_scores_t<float>(p, s) : page_scores_t<bf16>(p, s);
}

cudaError_t launch_select_pages(const SelectParams& p, int groups, cudaStream_t s) {
  const size_t smem = (size_t)p.max_pages * 4;
  cudaError_t e = allow_smem(select_pages_kernel, smem, 16 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(select_pages_kernel, dim3((unsigned)groups, 1, 1), kSelThreads, smem, s, p);
}

cudaError_t launch_pages_prep(const PlanParams& pp, const int32_t* block_table, int32_t* table, int32_t* bad,
                              cudaStream_t s) {
  const int groups = pp.batch * pp.q_len;
  const size_t smem = plan_smem_bytes(groups, pp.workers);
  cudaError_t e = allow_smem(pages_prep_kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_prep_kernel, dim3((unsigned)(1 + groups), 1, 1), 256, smem, s, pp, block_table, table, bad);
}

}  // namespace mla
