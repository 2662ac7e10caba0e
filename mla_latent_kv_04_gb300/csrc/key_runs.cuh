// How the key-weight kernels share out their work: the tiles of 128 tokens (two pages) of all
// requests in order, cut into one contiguous range per CTA; a CTA's tiles of one request, for which
// it prepares the request's query, are a run. The cuts are at equal cost, where a request costs
// its tiles plus the preparation of a query, in tiles (every CTA pays one for its first run anyway;
// the requests' own charges are for the further runs of the CTAs that they begin in).
//
// Several query tokens are columns of one product as far as they fit (heads * tokens <= 128); with more,
// a run is limited in length and passed over several times.
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
  return (S - 1) / kTile + 1;
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

// The CTA's range. scratch: 2 (batch + 1) ints of shared memory, or batch + 1 if batch is above
// kCostBatch (run_cost then counts as 0: CTAs have several runs each, whichever way they are cut).
// run_limit: the longest run with several passes. Called by the whole CTA, which it
// synchronises; the caller synchronises again before the scratch is used for something else.
constexpr int kCostBatch = 8192;
__device__ __forceinline__ Runs first_run(const KeyWeightParams& p, int* scratch, int run_cost, int run_limit) {
  __shared__ int warp_tot[32], start[3];
  const bool costs = run_cost > 0 && p.batch <= kCostBatch;
  int* tiles = scratch;                                // [batch + 1] prefix sums of the tiles
  int* cost = costs ? tiles + p.batch + 1 : tiles;     // and of the cost
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const int S = p.seq_lens[b], n = request_tiles(p, b);
    tiles[b + 1] = n;
    if (costs) cost[b + 1] = n > 0 ? n + run_cost : 0;
    if (blockIdx.x == 0 && S != 0 && n == 0) flag_status(p.status, MLA_ERR_DEVICE_GUARD);
  }
  if (threadIdx.x == 0) tiles[0] = cost[0] = 0;
  __syncthreads();
  block_inclusive_scan(tiles + 1, p.batch, warp_tot);
  if (costs) block_inclusive_scan(cost + 1, p.batch, warp_tot);
  // the tile at cost floor(V k / CTAs) (a cut inside a request's charge falls on its first tile)
  const long long V = cost[p.batch];
  auto cut = [&](int k, int* b) {
    *b = p.batch;
    if (k == (int)gridDim.x || V == 0) return tiles[p.batch];
    const long long c = V * k / (int)gridDim.x;
    *b = last_at_most(cost, p.batch, c);               // its last request with cost[b] <= c: not empty
    const long long in = c - cost[*b] - (costs ? run_cost : 0);
    return tiles[*b] + (int)(in < 0 ? 0 : in);
  };
  if (threadIdx.x == 0) {
    int b0, b1;
    const int t0 = cut(blockIdx.x, &b0), t1 = cut(blockIdx.x + 1, &b1);
    start[0] = b0;
    start[1] = t1 > t0 ? t0 - tiles[b0] : 0;
    start[2] = t1 - t0;
  }
  __syncthreads();
  Runs run;
  run.p = &p;
  run.limit = p.passes > 1 ? run_limit : 0x7FFFFFFF;
  run.left = start[2];
  run.b = run.left > 0 ? start[0] : 0;
  run.at = run.left > 0 ? start[1] : 0;
  run.tiles = run.left > 0 ? request_tiles(p, run.b) : 0;
  return run;
}

// Query tokens of a pass: the largest divisor of q_len with which the columns stay within 128 (64 requests
// of 300 tokens, 16 heads, 4 query tokens: 10.5 us at once, 24 in four passes).
inline void set_passes(KeyWeightParams& p) {
  int m = 1;
  for (int k = 2; k <= p.q_len && (long long)k * p.H <= 128; ++k)
    if (p.q_len % k == 0) m = k;
  p.tokens = m;
  p.passes = p.q_len / m;
  p.cols = p.H * m;
}
// The first column of pass t that counts for token j (those before it, possibly all, belong to query
// tokens that do not see j).
__device__ __forceinline__ int first_column(const KeyWeightParams& p, int S, int j, int t) {
  const int past = j - (S - p.q_len) - t * p.tokens;
  return past > 0 ? past * p.H : 0;
}

// One CTA per SM, and no more than tiles that the tables can hold.
inline int grid_size(const KeyWeightParams& p) {
  const long long most = (long long)p.batch * ((p.max_pages + 1) / 2);
  return (int)(most < device_sms() ? most : device_sms());
}

}  // namespace weigh
}  // namespace mla
