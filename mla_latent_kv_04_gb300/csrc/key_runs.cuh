// How the key-weight kernels share out their work. Tiles are 128 tokens (two pages); a CTA's tiles
// of one request, for which it prepares the request's query, are a run. Either the tiles of all
// requests in order are cut into one contiguous range per CTA, all of the same length, or every
// request gets CTAs of its own, as many as a common quota of tiles asks for: fuller CTAs by up to
// the rounding, but one run each instead of up to two and more. With several query tokens a run is
// limited in length and passed over once per query token.
#pragma once
#include "internal.h"
#include "prologue.cuh"
#include "tc_host.h"

namespace mla {
namespace weigh {

constexpr int kTile = 128;

__device__ __forceinline__ int request_tiles(const KeyWeightParams& p, int b) {
  const int S = p.seq_lens[b];
  if (S < p.q_len || S <= 0 || S > (long long)p.max_pages * p.P) return 0;
  return (S + kTile - 1) / kTile;
}

// A CTA's runs in order: tiles [t0, t1) of request rb, of length S.
struct Runs {
  const KeyWeightParams* p;
  int b, at, tiles;            // next tile of request b, and how many it has
  long long left;              // tiles of the CTA's range still to come
  int limit, t0, t1, rb, S;
  __device__ bool next() {
    if (left <= 0) return false;
    while (at >= tiles) {
      tiles = request_tiles(*p, ++b);
      at = 0;
    }
    rb = b;
    S = p->seq_lens[b];
    t0 = at;
    int n = min(tiles - at, limit);
    if (n > left) n = (int)left;
    t1 = at + n;
    at = t1;
    left -= n;
    return true;
  }
  // First cache row of the request's page pg; behind its last page, or for a bad id, any page's
  // (those tokens are not written).
  __device__ int row_of(int pg) const {
    int page = (long long)pg * p->P < S ? p->block_table[(long long)rb * p->max_pages + pg] : 0;
    if (page < 0 || page >= p->num_pages) {
      flag_status(p->status, MLA_ERR_DEVICE_GUARD);
      page = 0;
    }
    return page * p->P;
  }
};

// Sum of v over the block (tmp: 32 ints).
__device__ __forceinline__ int block_sum(int v, int* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  int sum = 0;
  for (int i = 0; i < (int)(blockDim.x + 31) / 32; ++i) sum += tmp[i];
  return sum;
}

// The CTA's range. scratch: batch + 1 ints of shared memory. run_cost: what preparing a query
// costs, in tiles (0: no quotas); run_limit: the longest run with several query tokens. Called by the whole CTA,
// which it synchronises; the caller synchronises again before the scratch is used for something
// else.
__device__ __forceinline__ Runs first_run(const KeyWeightParams& p, int* scratch, int run_cost, int run_limit) {
  __shared__ int tmp[32], start[2];
  int* cu = scratch;
  const int ctas = gridDim.x, nt = blockDim.x;
  int tiles = 0;
  for (int b = threadIdx.x; b < p.batch; b += nt) {
    const int S = p.seq_lens[b];
    cu[b + 1] = request_tiles(p, b);
    tiles += cu[b + 1];
    if (blockIdx.x == 0 && S != 0 && cu[b + 1] == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  }
  if (threadIdx.x == 0) cu[0] = 0;
  const int total = block_sum(tiles, tmp);
  // the smallest quota, up to run_cost tiles above an even share, with CTAs enough
  int quota = 0;
  const int even = (total + ctas - 1) / ctas;
  if (run_cost > 0 && p.batch <= ctas && total > 0) {
    int lo = even, hi = even + run_cost + 1;           // hi: none
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      int n = 0;
      for (int b = threadIdx.x; b < p.batch; b += nt) n += (cu[b + 1] + mid - 1) / mid;
      if (block_sum(n, tmp) <= ctas) hi = mid;
      else lo = mid + 1;
    }
    if (lo <= even + run_cost) quota = lo;
  }
  Runs run;
  run.p = &p;
  run.limit = p.q_len > 1 ? run_limit : 0x7FFFFFFF;
  if (quota > 0) {
    __syncthreads();
    for (int b = threadIdx.x; b < p.batch; b += nt) cu[b + 1] = (cu[b + 1] + quota - 1) / quota;
    __syncthreads();
  }
  block_inclusive_scan(cu + 1, p.batch, tmp);
  const int units = cu[p.batch];                       // CTAs in use (quota), or tiles
  const int u0 = quota ? (int)blockIdx.x : (int)((long long)total * blockIdx.x / ctas);
  const int u1 = quota ? min(u0 + 1, units) : (int)((long long)total * (blockIdx.x + 1) / ctas);
  if (threadIdx.x == 0 && u1 > u0) {
    const int b = last_at_most(cu, p.batch, u0);       // its last request with cu[b] <= u0: not empty
    start[0] = b;
    start[1] = u0 - cu[b];
  }
  __syncthreads();
  run.left = u1 > u0 ? u1 - u0 : 0;
  run.b = run.left > 0 ? start[0] : 0;
  run.at = run.left > 0 ? start[1] : 0;
  run.tiles = run.left > 0 ? request_tiles(p, run.b) : 0;
  if (quota && run.left > 0) {                         // part `at` of the request's n
    const int n = cu[run.b + 1] - cu[run.b], i = run.at;
    run.at = (int)((long long)run.tiles * i / n);
    run.left = (int)((long long)run.tiles * (i + 1) / n) - run.at;
  }
  return run;
}

// One CTA per SM, and no more than tiles that the tables can hold.
inline int grid_size(const KeyWeightParams& p) {
  const long long most = (long long)p.batch * ((p.max_pages + 1) / 2);
  return (int)(most < device_sms() ? most : device_sms());
}

}  // namespace weigh
}  // namespace mla
