// SIMT kernels of the shared-prefix and key-weight calls: every activation and cache format
// and every head shape, fp32 sums. The tensor-core kernels (prefix_tc.cu, key_weights_tc.cu)
// take the DeepSeek-V2 head shape in bf16; these serve the rest and cross-check them.
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "page_elem.cuh"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace mla {
namespace {

// ======================================================================== prefix expansion
template <typename AT, typename CT>
__device__ __forceinline__ void expand_rope(const PrefixExpandParams& p, int l0) {
  const int n = min(64, p.L - l0) * p.d_r;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int l = l0 + i / p.d_r, k = i % p.d_r;
    const int page = p.table[l / p.P];
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && k == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    const uint32_t* row = reinterpret_cast<const uint32_t*>(
        reinterpret_cast<const uint8_t*>(p.cache) + ((long long)(ok ? page : 0) * p.P + l % p.P) * p.row_bytes);
    reinterpret_cast<AT*>(p.k_pe)[(long long)l * p.d_r + k] =
        from_f32<AT>(ok ? page_rope_elem<CT>(row, k, p.d_c) * p.cache_scale : 0.f);
  }
}

// keys[h][l] = c_l W_UK[:, h], values[h][l] = c_l W_UV[:, h] (huny.dev "DeepSeek MLA 해부"
// §2-1: k^C = c W^UK, v^C = c W^UV). 64 x 64 output tile per block; z = 0 keys, 1 values, 2 the
// rotated keys as cached, k_pe[l], of 64 tokens.
template <typename AT, typename CT>
__global__ void __launch_bounds__(256) expand_simt_kernel(PrefixExpandParams p) {
  __shared__ float As[16][64 + 4], Bs[16][64 + 4];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (blockIdx.z == 2) {
    if (blockIdx.y == 0) expand_rope<AT, CT>(p, blockIdx.x * 64);
    return;
  }
  const int dh = blockIdx.z ? p.d_v : p.d_n;
  const int N = p.H * dh;
  const int n0 = blockIdx.y * 64, l0 = blockIdx.x * 64;
  if (n0 >= N) return;
  const AT* W = reinterpret_cast<const AT*>(blockIdx.z ? p.W_UV : p.W_UK);
  AT* out = reinterpret_cast<AT*>(blockIdx.z ? p.values : p.keys);
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  // a thread loads dim k0 + tx of four tokens and column tid % 64 of four dims, a step ahead
  const uint32_t* row[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int l = l0 + ty + 16 * m, page = l < p.L ? p.table[l / p.P] : -1;
    row[m] = nullptr;
    if (page >= 0 && page < p.num_pages)
      row[m] = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p.cache) +
                                                 ((long long)page * p.P + l % p.P) * p.row_bytes);
    else if (tx == 0 && l < p.L && l % p.P == 0)
      flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  }
  float a[4], w[4];
  auto load = [&](int k0) {
    const int n = n0 + tid % 64;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int k = k0 + tid / 64 + 4 * m;
      a[m] = row[m] && k0 + tx < p.d_c ? PageElem<CT>::get(row[m], k0 + tx, p.d_c) : 0.f;
      w[m] = k < p.d_c && n < N ? to_f32(W[(long long)k * N + n]) : 0.f;
    }
  };
  float acc[4][4] = {};
  load(0);
  for (int k0 = 0; k0 < p.d_c; k0 += 16) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      As[tx][ty + 16 * m] = a[m];
      Bs[tid / 64 + 4 * m][tid % 64] = w[m];
    }
    __syncthreads();
    if (k0 + 16 < p.d_c) load(k0 + 16);
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[kk][ty * 4 + i], Bs[kk][tx * 4 + j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int l = l0 + ty * 4 + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (l < p.L && n < N)
        out[((long long)(n / dh) * p.L + l) * dh + n % dh] = from_f32<AT>(acc[i][j] * p.cache_scale);
    }
  }
}

// ======================================================================== prefix attention
// Four elements, read at once.
template <typename AT> struct Quads;
template <> struct Quads<float> {
  float4 v;
  __device__ __forceinline__ float4 get() const { return v; }
};
template <> struct Quads<bf16> {
  uint2 v;
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
  }
};

// Block per (kR query rows, head): 128 keys at a time, one per thread, with the running maximum and
// sum of the softmax; the output's dims over the threads, narrow values several times, each copy of
// the threads taking every so manyth key. Small calls are bound by the latency of their loads, which
// the unrolled loops keep in flight together; large ones by the loads of keys (a thread reads a row of
// its own), which several query rows share: 64 rows x 16 heads, tiny shape, 1000 keys 62 us with 4 rows
// a block and four elements a load, 201 with one row and one element. (85 us among calls issued one by
// one: the next call's blocks, started early, are spread unevenly over the SMs.)
template <typename AT, int kR>
__global__ void __launch_bounds__(128) attend_simt_kernel(PrefixAttendParams p) {
  extern __shared__ __align__(16) float sm[];
  const int dn4 = (p.d_n + 3) & ~3, dq = dn4 + p.d_r;
  float* q = sm;                               // [kR][dq]: content, zeros up to dn4, rotary
  float* o = q + kR * dq;                      // [kR][d_v]
  __shared__ float ps[kR][128], red[kR][4], acc_s[128];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int r0 = blockIdx.x * kR, nr = min(kR, p.rows - r0), h = blockIdx.y, tid = threadIdx.x;
  auto own = [&](int r) { return p.seq_lens[(r0 + r) / p.q_len]; };
  for (int r = 0; r < nr; ++r) {
    const int S = own(r);
    const AT* qn = reinterpret_cast<const AT*>(p.q_nope) + ((long long)(r0 + r) * p.H + h) * p.d_n;
    const AT* qr = reinterpret_cast<const AT*>(p.q_pe) + ((long long)(r0 + r) * p.H + h) * p.d_r;
    const long long pos = (long long)p.L + S - p.q_len + (r0 + r) % p.q_len;
    for (int i = tid; i < dn4; i += 128) q[r * dq + i] = i < p.d_n ? to_f32(qn[i]) : 0.f;
    for (int k = tid; k < p.d_r / 2; k += 128) {
      float sn, cs;
      turn_sincos<sizeof(AT) == 4>(p.tt, k, pos, &sn, &cs);
      const float x0 = to_f32(qr[2 * k]), x1 = to_f32(qr[2 * k + 1]);
      q[r * dq + dn4 + 2 * k] = x0 * cs - x1 * sn;
      q[r * dq + dn4 + 2 * k + 1] = x0 * sn + x1 * cs;
    }
    if (S != 0 && S < p.q_len && h == 0 && tid == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  }
  for (int i = nr * dq + tid; i < kR * dq; i += 128) q[i] = 0.f;
  for (int i = tid; i < kR * p.d_v; i += 128) o[i] = 0.f;
  __syncthreads();
  const AT* K = reinterpret_cast<const AT*>(p.keys) + (long long)h * p.L * p.d_n;
  const AT* V = reinterpret_cast<const AT*>(p.values) + (long long)h * p.L * p.d_v;
  const AT* kp = reinterpret_cast<const AT*>(p.k_pe);
  typedef Quads<AT> Quad;
  const bool vec = p.d_n % 4 == 0 && ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(kp)) % sizeof(Quad)) == 0;
  int width = 128;                             // threads that cover the output's dims once
  while (width > 1 && width / 2 >= p.d_v) width /= 2;
  const int copies = 128 / width;
  float m[kR], l[kR], a[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  for (int l0 = 0; l0 < p.L; l0 += 128) {
    const int j = l0 + tid;
    float s[kR] = {};
    if (j < p.L) {
      auto add = [&](float4 k, int at) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float4 y = *reinterpret_cast<const float4*>(q + r * dq + at);
          s[r] = fmaf(y.w, k.w, fmaf(y.z, k.z, fmaf(y.y, k.y, fmaf(y.x, k.x, s[r]))));
        }
      };
      if (vec) {                               // four elements a load
        const Quad* kq = reinterpret_cast<const Quad*>(K + (long long)j * p.d_n);
        const Quad* kr = reinterpret_cast<const Quad*>(kp + (long long)j * p.d_r);
#pragma unroll 8
        for (int i = 0; i < p.d_n / 4; ++i) add(kq[i].get(), 4 * i);
#pragma unroll 8
        for (int i = 0; i < p.d_r / 4; ++i) add(kr[i].get(), dn4 + 4 * i);
      } else {
#pragma unroll 4
        for (int i = 0; i < dn4; i += 4) {
          float k[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) k[t] = i + t < p.d_n ? to_f32(K[(long long)j * p.d_n + i + t]) : 0.f;
          add(make_float4(k[0], k[1], k[2], k[3]), i);
        }
        for (int i = 0; i < p.d_r; i += 4) {
          const AT* k = kp + (long long)j * p.d_r + i;
          add(make_float4(to_f32(k[0]), to_f32(k[1]), to_f32(k[2]), to_f32(k[3])), dn4 + i);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      s[r] = j < p.L ? s[r] * p.scale_log2 : -INFINITY;
      const float wm = warp_max(s[r]);
      if ((tid & 31) == 0) red[r][tid >> 5] = wm;
    }
    __syncthreads();
    float ws[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const float m_new = fmaxf(m[r], fmaxf(fmaxf(red[r][0], red[r][1]), fmaxf(red[r][2], red[r][3])));
      // no finite score so far (all -inf): keep the sums at zero
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      a[r] = exp2f(m[r] - ref);
      const float e = exp2f(s[r] - ref);
      ps[r][tid] = e;
      ws[r] = warp_sum(e);
      m[r] = m_new;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kR; ++r)
      if ((tid & 31) == 0) red[r][tid >> 5] = ws[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kR; ++r) l[r] = l[r] * a[r] + ((red[r][0] + red[r][1]) + (red[r][2] + red[r][3]));
    const int n = min(128, p.L - l0);
    for (int v0 = 0; v0 < p.d_v; v0 += 128) {
      const int v = v0 + tid % width;
      float acc[kR] = {};
      if (v < p.d_v) {
#pragma unroll 8
        for (int i = tid / width; i < n; i += copies) {
          const float y = to_f32(V[(long long)(l0 + i) * p.d_v + v]);
#pragma unroll
          for (int r = 0; r < kR; ++r) acc[r] = fmaf(ps[r][i], y, acc[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (copies > 1) {
          __syncthreads();
          acc_s[tid] = acc[r];
          __syncthreads();
          if (tid < width) {
            acc[r] = 0.f;
            for (int g = 0; g < copies; ++g) acc[r] += acc_s[g * width + tid];
          }
        }
        if (tid < width && v < p.d_v) o[r * p.d_v + v] = o[r * p.d_v + v] * a[r] + acc[r];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    if (r >= nr) break;
    // an empty request (or a bad length), or no prefix: no keys
    const bool live = own(r) >= p.q_len && p.L > 0;
    const long long g = (long long)(r0 + r) * p.H + h;
    AT* out = reinterpret_cast<AT*>(p.u) + g * p.d_v;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];      // (a NaN in the scores stays one)
    for (int v = tid; v < p.d_v; v += 128) out[v] = from_f32<AT>(live ? o[r * p.d_v + v] * inv : 0.f);
    if (tid == 0) p.lse[g] = !live || l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
  }
}

// The same for a prefix of up to kPrefixShort keys: warp per (query row, head), dims over the lanes,
// the scores in registers. For every format: the tensor-core kernel's query, two bf16 terms, is
// too coarse for an LSE of one key, which may be near 0 (relative error 1.4e-6 over normal inputs,
// 1e-6 with two keys and 6e-7 with three, against 1e-7 here). 128 rows x 128 heads x 1 key take 11.7
// us (a block per row and head: 69).
template <typename AT>
__global__ void __launch_bounds__(256) attend_short_kernel(PrefixAttendParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long g = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);   // row * H + head
  if (g >= (long long)p.rows * p.H) return;
  const int r = (int)(g / p.H), h = (int)(g - (long long)r * p.H), S = p.seq_lens[r / p.q_len];
  AT* out = reinterpret_cast<AT*>(p.u) + g * p.d_v;
  if (S < p.q_len) {
    if (S != 0 && h == 0 && lane == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    for (int v = lane; v < p.d_v; v += 32) out[v] = from_f32<AT>(0.f);
    if (lane == 0) p.lse[g] = -INFINITY;
    return;
  }
  const long long pos = (long long)p.L + S - p.q_len + r % p.q_len;
  const AT* qn = reinterpret_cast<const AT*>(p.q_nope) + g * p.d_n;
  const AT* qr = reinterpret_cast<const AT*>(p.q_pe) + g * p.d_r;
  const AT* K = reinterpret_cast<const AT*>(p.keys) + (long long)h * p.L * p.d_n;
  const AT* V = reinterpret_cast<const AT*>(p.values) + (long long)h * p.L * p.d_v;
  const AT* kp = reinterpret_cast<const AT*>(p.k_pe);
  float s[kPrefixShort] = {};
  for (int i = lane; i < p.d_n; i += 32) {
    const float x = to_f32(qn[i]);
#pragma unroll
    for (int j = 0; j < kPrefixShort; ++j)
      if (j < p.L) s[j] = fmaf(x, to_f32(K[j * p.d_n + i]), s[j]);
  }
  for (int k = lane; k < p.d_r / 2; k += 32) {
    float sn, cs;
    turn_sincos<sizeof(AT) == 4>(p.tt, k, pos, &sn, &cs);
    const float x0 = to_f32(qr[2 * k]), x1 = to_f32(qr[2 * k + 1]);
    const float y0 = x0 * cs - x1 * sn, y1 = x0 * sn + x1 * cs;
#pragma unroll
    for (int j = 0; j < kPrefixShort; ++j)
      if (j < p.L) s[j] = fmaf(y1, to_f32(kp[j * p.d_r + 2 * k + 1]), fmaf(y0, to_f32(kp[j * p.d_r + 2 * k]), s[j]));
  }
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < kPrefixShort; ++j) {
    s[j] = j < p.L ? warp_sum(s[j]) * p.scale_log2 : -INFINITY;
    m = fmaxf(m, s[j]);
  }
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int j = 0; j < kPrefixShort; ++j) l += s[j] = exp2f(s[j] - ref);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int v = lane; v < p.d_v; v += 32) {
    float o = 0.f;
#pragma unroll
    for (int j = 0; j < kPrefixShort; ++j)
      if (j < p.L) o = fmaf(s[j], to_f32(V[j * p.d_v + v]), o);
    out[v] = from_f32<AT>(o * inv);
  }
  if (lane == 0) p.lse[g] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
}

// ======================================================================== joined projection
// out[z] = x[z] W[z] in fp32 sums of one order (the split-K form of the other projections adds by
// atomics, in three launches). With lse, the lift of head z joined with the prefix's part (`join`).
// Block: 16 rows x 32 columns, up to 512 of K at a time, an eighth of them per warp and a column
// per lane; the warps' sums meet in warp order. Few rows are bound by the latency of the loads: fp32
// tiny shape (512 x 256), 32 rows: lift and product 12 us, by the split-K form 32.
struct SimtProduct {
  const void* x;
  const void* W;
  void* out;
  int rows, K, N, heads;
  long long ldx, ldw, ldo, zx, zw, zo;         // strides of rows and of z
  PrefixJoin join;                             // lse null: no join
};
constexpr int kProjRows = 16, kProjCols = 32, kProjK = 512;
template <typename AT>
__global__ void __launch_bounds__(256) product_simt_kernel(SimtProduct p) {
  __shared__ __align__(16) float us[kProjRows * kProjK];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, z = blockIdx.z;
  // blockIdx.x: the column block, then the row block (any number of rows: y has 65535 blocks at most)
  const int col_blocks = (p.N + kProjCols - 1) / kProjCols;
  const int n0 = blockIdx.x % col_blocks * kProjCols, r0 = blockIdx.x / col_blocks * kProjRows;
  const int n = n0 + lane;
  const AT* x = reinterpret_cast<const AT*>(p.x) + z * p.zx;
  const AT* W = reinterpret_cast<const AT*>(p.W) + z * p.zw;
  const int chunk = min(kProjK, (p.K + 31) & ~31), slice = chunk / 8;
  float acc[kProjRows] = {};
  for (int kc = 0; kc < p.K; kc += chunk) {
    __syncthreads();
#pragma unroll 8
    for (int i = threadIdx.x; i < kProjRows * chunk; i += 256) {
      const int r = i / chunk, k = kc + i - r * chunk;
      us[i] = r0 + r < p.rows && k < p.K ? to_f32(x[(r0 + r) * p.ldx + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = slice * warp; k < slice * (warp + 1); k += 4) {
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = kc + k + j < p.K && n < p.N ? to_f32(W[(kc + k + j) * p.ldw + n]) : 0.f;
#pragma unroll
      for (int r = 0; r < kProjRows; ++r) {
        const float4 y = *reinterpret_cast<const float4*>(us + r * chunk + k);
        acc[r] = fmaf(y.w, w[3], fmaf(y.z, w[2], fmaf(y.y, w[1], fmaf(y.x, w[0], acc[r]))));
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kProjRows; ++r) us[(warp * kProjRows + r) * kProjCols + lane] = acc[r];
  __syncthreads();
  for (int i = threadIdx.x; i < kProjRows * kProjCols; i += 256) {
    const int r = r0 + i / kProjCols, c = n0 + i % kProjCols;
    float sum = 0.f;
    for (int w = 0; w < 8; ++w) sum += us[w * kProjRows * kProjCols + i];
    if (r >= p.rows || c >= p.N) continue;
    const long long at = r * p.ldo + z * p.zo + c;
    if (p.join.lse) {
      float a, b;
      merge_weights(p.join.lse[(long long)r * p.heads + z], p.join.lse_prefix[(long long)r * p.heads + z], &a, &b);
      sum = merge_parts(a, sum, b, to_f32(reinterpret_cast<const AT*>(p.join.u_prefix)[at]));
    }
    reinterpret_cast<AT*>(p.out)[at] = from_f32<AT>(sum);
  }
}

// ======================================================================== key weights
// Elements e .. e + 3 of a row in shared memory (e a multiple of 4, as d_c and d_r are).
template <typename CT>
__device__ __forceinline__ float4 row_quad(const uint32_t* row, int e, int d_c) {
  if constexpr (sizeof(CT) == 4 || sizeof(CT) == 2) {
    return make_float4(PageElem<CT>::get(row, e, d_c), PageElem<CT>::get(row, e + 1, d_c),
                       PageElem<CT>::get(row, e + 2, d_c), PageElem<CT>::get(row, e + 3, d_c));
  } else if constexpr (std::is_same<CT, E4m3B128>::value) {
    if (e >= d_c)
      return make_float4(page_rope_elem<CT>(row, e - d_c, d_c), page_rope_elem<CT>(row, e - d_c + 1, d_c),
                         page_rope_elem<CT>(row, e - d_c + 2, d_c), page_rope_elem<CT>(row, e - d_c + 3, d_c));
    const float4 c = row_quad<uint8_t>(row, e, d_c);
    const float s = __uint_as_float(row[(d_c >> 2) + (e >> 7)]);
    return make_float4(c.x * s, c.y * s, c.z * s, c.w * s);
  } else {
    const uint32_t w = row[e >> 2];
    return make_float4(fp8_to_f32((uint8_t)w), fp8_to_f32((uint8_t)(w >> 8)), fp8_to_f32((uint8_t)(w >> 16)),
                       fp8_to_f32((uint8_t)(w >> 24)));
  }
}

// Bytes of shared memory: the page's rows (an odd number of words each), the warps' queries and sums.
size_t key_weights_simt_smem(int P, long long row_bytes, long long D, int warps, int at_once) {
  return (((size_t)P * ((row_bytes / 4) | 1) + 3) / 4 * 4 + (size_t)warps * ((size_t)at_once * D + P)) * 4;
}

// Block per (request, page): the page's rows in shared memory (odd word stride), kQ queries (query
// token, head) per warp at a time, two tokens per lane: a row's element is read once for kQ products;
// the warps' sums meet in warp order. Few pages are bound by the latency of a warp's queries in turn,
// many by shared memory's reads. fp32 tiny shape, 16 heads, 4 query tokens: 2 requests of 319 tokens
// 8.2 us, 64 of up to 1000 22.4 (one query at a time in 8 warps: 26.5 and 72).
template <typename AT, typename CT, int kQ>
__global__ void __launch_bounds__(1024) key_weights_simt_kernel(KeyWeightParams p) {
  extern __shared__ __align__(16) uint32_t smem_kw[];
  const int row_words = (int)(p.row_bytes / 4), stride = row_words | 1;
  uint32_t* page_s = smem_kw;                                     // [P][stride]
  const int warps = blockDim.x >> 5;
  float* q_s = reinterpret_cast<float*>(smem_kw + ((p.P * stride + 3) & ~3));   // [warps][kQ][D]
  float* red = q_s + warps * kQ * p.D;                            // [warps][P]
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int b = blockIdx.x / p.max_pages, pg = blockIdx.x % p.max_pages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.seq_lens[b];
  if (S == 0) return;
  if (S < p.q_len || S > (long long)p.max_pages * p.P) {
    if (pg == 0 && threadIdx.x == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    return;
  }
  if ((long long)pg * p.P >= S) return;
  const int page = p.block_table[(long long)b * p.max_pages + pg];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
    return;
  }
  const int ntok = min(p.P, S - pg * p.P);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p.cache) +
                                                          (long long)page * p.P * p.row_bytes);
  for (int i = threadIdx.x; i < ntok * row_words; i += blockDim.x)
    page_s[(i / row_words) * stride + i % row_words] = src[i];
  __syncthreads();
  float* q = q_s + warp * kQ * p.D;
  const uint32_t* row0 = page_s + min(lane, p.P - 1) * stride;
  const uint32_t* row1 = page_s + min(lane + 32, p.P - 1) * stride;
  const int queries = p.q_len * p.H;
  const AT* ql = reinterpret_cast<const AT*>(p.q_lat) + (long long)b * queries * p.D;
  const float* lse = p.lse + (long long)b * queries;
  float w0 = 0.f, w1 = 0.f;
  for (int x0 = warp * kQ; x0 < queries; x0 += warps * kQ) {
    const int nq = min(kQ, queries - x0);
    __syncwarp();
    for (int i = lane; i < kQ * p.D; i += 32) q[i] = i < nq * p.D ? to_f32(ql[(long long)x0 * p.D + i]) : 0.f;
    __syncwarp();
    float a0[kQ] = {}, a1[kQ] = {};
#pragma unroll 2
    for (int e = 0; e < p.D; e += 4) {
      const float4 r0 = row_quad<CT>(row0, e, p.d_c), r1 = row_quad<CT>(row1, e, p.d_c);
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(q + k * p.D + e);
        a0[k] = fmaf(y.w, r0.w, fmaf(y.z, r0.z, fmaf(y.y, r0.y, fmaf(y.x, r0.x, a0[k]))));
        a1[k] = fmaf(y.w, r1.w, fmaf(y.z, r1.z, fmaf(y.y, r1.y, fmaf(y.x, r1.x, a1[k]))));
      }
    }
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
      if (k >= nq) break;
      const int last = S - p.q_len + (x0 + k) / p.H - pg * p.P;   // its query token sees tokens 0..last
      const float off = lse[x0 + k] * kLog2e;
      if (lane < ntok && lane <= last) w0 += exp2f(a0[k] * p.scale_log2 - off);
      if (lane + 32 < ntok && lane + 32 <= last) w1 += exp2f(a1[k] * p.scale_log2 - off);
    }
  }
  if (lane < p.P) red[warp * p.P + lane] = w0;
  if (lane + 32 < p.P) red[warp * p.P + lane + 32] = w1;
  __syncthreads();
  for (int i = threadIdx.x; i < ntok; i += blockDim.x) {
    float mass = 0.f;
    for (int w = 0; w < warps; ++w) mass += red[w * p.P + i];
    const int j = pg * p.P + i;
    float* dst = p.weights + (long long)b * p.max_pages * p.P + j;
    // a token of this step has no earlier weight
    *dst = (p.decay != 0.f && j < S - p.q_len) ? fmaf(p.decay, *dst, mass) : mass;
  }
}

// A cache format's tag type, and the call f(tag of the activations, tag of the cache).
template <typename F>
cudaError_t by_format(mla_dtype act, mla_dtype cache, F f) {
  if (act == MLA_F32) return f(float{}, float{});
  if (cache == MLA_BF16) return f(bf16{}, bf16{});
  if (cache == MLA_FP8_E4M3) return f(bf16{}, uint8_t{});
  return f(bf16{}, E4m3B128{});
}

}  // namespace

cudaError_t launch_prefix_expand_simt(mla_dtype act, mla_dtype cache, const PrefixExpandParams& p,
                                      cudaStream_t s) {
  if (p.L <= 0) return cudaSuccess;
  return by_format(act, cache, [&](auto a, auto c) {
    using AT = decltype(a);
    using CT = decltype(c);
    const int cols = p.H * (p.d_n > p.d_v ? p.d_n : p.d_v);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.L + 63) / 64), (unsigned)((cols + 63) / 64), 3);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, expand_simt_kernel<AT, CT>, p);
    if (e == cudaSuccess) note_launch();
    return e;
  });
}

static_assert((kPrefixMaxWidth + 3) * 4 + 528 + 1024 <= kSmemPerCta, "a query row in shared memory");

cudaError_t launch_prefix_attend_simt(mla_dtype act, const PrefixAttendParams& p, cudaStream_t s) {
  const bool brief = p.L > 0 && p.L <= kPrefixShort;
  // rows of a block: as many as leave a block per SM and fit its shared memory (a block's static
  // arrays: 528 bytes a row and 512, here rounded up)
  int at_once = 8;
  auto dynamic = [&]() { return (size_t)at_once * (((p.d_n + 3) & ~3) + p.d_r + p.d_v) * 4; };
  auto fixed = [&]() { return (size_t)(528 * at_once + 1024); };
  while (at_once > 1 && ((long long)((p.rows + at_once - 1) / at_once) * p.H < device_sms() ||
                         dynamic() + fixed() > kSmemPerCta))
    at_once /= at_once == 8 ? 2 : 4;
  const size_t smem = brief ? 0 : dynamic();
  auto go = [&](auto a) {
    using AT = decltype(a);
    auto kern = brief ? attend_short_kernel<AT>
                      : (at_once == 8 ? attend_simt_kernel<AT, 8>
                                      : (at_once == 4 ? attend_simt_kernel<AT, 4> : attend_simt_kernel<AT, 1>));
    cudaError_t e = allow_smem(kern, smem, fixed());
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = brief ? dim3((unsigned)(((long long)p.rows * p.H + 7) / 8), 1, 1)
                        : dim3((unsigned)((p.rows + at_once - 1) / at_once), (unsigned)p.H, 1);
    cfg.blockDim = dim3(brief ? 256 : 128, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) note_launch();
    return e;
  };
  return act == MLA_F32 ? go(float{}) : go(bf16{});
}

static cudaError_t product_simt(mla_dtype act, const SimtProduct& p, int batch, cudaStream_t s) {
  auto go = [&](auto a) {
    using AT = decltype(a);
    cudaLaunchConfig_t cfg = {};
    const long long blocks = (long long)((p.N + kProjCols - 1) / kProjCols) * ((p.rows + kProjRows - 1LL) / kProjRows);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)blocks, 1, (unsigned)batch);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, product_simt_kernel<AT>, p);
    if (e == cudaSuccess) note_launch();
    return e;
  };
  return act == MLA_F32 ? go(float{}) : go(bf16{});
}

cudaError_t launch_prefix_project_simt(mla_dtype act, const void* o_lat, const void* W_UV, const void* W_O, int rows,
                                       int H, int d_c, int d_v, int N, const PrefixJoin& join, void* u, void* out,
                                       cudaStream_t s) {
  const SimtProduct lift{o_lat, W_UV, u, rows, d_c, d_v, H, (long long)H * d_c, (long long)H * d_v,
                         (long long)H * d_v, d_c, d_v, d_v, join};
  cudaError_t e = product_simt(act, lift, H, s);
  if (e != cudaSuccess) return e;
  const SimtProduct prod{u, W_O, out, rows, H * d_v, N, H, (long long)H * d_v, N, N, 0, 0, 0, {}};
  return product_simt(act, prod, 1, s);
}

bool key_weights_simt_fits(int P, long long row_bytes, long long D) {
  return key_weights_simt_smem(P, row_bytes, D, 1, 1) <= kSmemPerCta;
}

cudaError_t launch_key_weights_simt(mla_dtype act, mla_dtype cache, const KeyWeightParams& p,
                                    cudaStream_t s) {
  // up to 32 warps of 4 queries each, as many as there are queries and as fit beside the page; less
  // than 8 warps of one query only beside the widest rows
  int warps = 32, at_once = 4;
  auto bytes = [&]() { return key_weights_simt_smem(p.P, p.row_bytes, p.D, warps, at_once); };
  while (warps > 8 && (bytes() > 200 * 1024 || warps / 2 * at_once >= p.q_len * p.H)) warps /= 2;
  if (bytes() > 220 * 1024) at_once = 1;
  while (warps > 1 && bytes() > kSmemPerCta) warps /= 2;
  const size_t smem = bytes();
  return by_format(act, cache, [&](auto a, auto c) {
    using AT = decltype(a);
    using CT = decltype(c);
    auto kern = at_once == 4 ? key_weights_simt_kernel<AT, CT, 4> : key_weights_simt_kernel<AT, CT, 1>;
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.batch * p.max_pages), 1, 1);
    cfg.blockDim = dim3(32 * warps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) note_launch();
    return e;
  });
}

}  // namespace mla
