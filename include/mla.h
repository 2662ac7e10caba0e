/*
 * mla.h - C ABI of libmla: weight-absorbed Multi-head Latent Attention (MLA)
 * decode on one GB300 (sm_103a).
 *
 * What the library computes (pages cited by title and section):
 *   - "DeepSeek Multi-Head Latent Attention(MLA) 해부" (blog.huny.dev), §2-1 (the
 *     latent c_t = h_t W^DKV), §2-3 (decoupled RoPE key k^R = RoPE(h_t W^KR), the
 *     concatenated query/key and the score split), §3-1 (W^UK absorbed into the
 *     query) and §3-2 (W^UV folded into W^O);
 *   - "KV Cache를 10분의 1로 줄인 MLA의 트릭" (donmain.dev), "위치 정보와 압축의 충돌":
 *     the cache stores c_t (512) and k^R_t (64) = 576 elements per token, the
 *     absorption is done once at model load;
 *   - "[vLLM] Multi-head Latent Attention" (blog.secrett2633.cloud), "FlashMLABackend"
 *     (64-token pages, bf16 or fp8_e4m3 cache), "MLA의 MQA 디코딩 경로" (decode runs
 *     as MQA: every query head over one shared latent "KV head"), "FlashMLAImpl"
 *     (query given as (q_nope, q_pe) and concatenated, LSE returned, several query
 *     tokens per request for speculative decoding).
 *
 * Conventions shared by every call
 *   - Every tensor argument is a DEVICE pointer to a contiguous row-major array
 *     owned by the caller; the library allocates no device memory and keeps no
 *     global state beyond a per-device cache of attributes and tensor-map
 *     encoders. Sizes are element counts unless stated.
 *   - `stream` is a cudaStream_t passed as void*; NULL is the legacy default
 *     stream. Every call only enqueues work on `stream` and returns; results are
 *     ready when the stream reaches that point.
 *   - Host-side validation runs before anything is enqueued: a null pointer, a
 *     bad dimension, an unsupported dtype combination or a too-small workspace
 *     returns MLA_ERR_INVALID / MLA_ERR_UNSUPPORTED / MLA_ERR_WORKSPACE and
 *     enqueues nothing. A CUDA launch failure returns MLA_ERR_CUDA.
 *   - Device-side guards: data that only the device sees (a block-table entry
 *     outside [0, num_pages), a request id outside [0, batch), a position past the
 *     request's block-table row, a seq_len below q_len or above
 *     max_pages*page_size) never causes an out-of-bounds access: the offending
 *     row or request is skipped and MLA_ERR_DEVICE_GUARD is OR-ed into a device
 *     status word, which mla_read_device_status returns.
 *
 * Dtypes: act_dtype (activations, weights, queries, outputs) is MLA_F32 or
 * MLA_BF16; cache_dtype is MLA_F32 (only with MLA_F32 activations), MLA_BF16,
 * MLA_FP8_E4M3 or MLA_FP8_E4M3_B128 (the last two only with MLA_BF16 activations).
 * bf16 and fp8 values are rounded to nearest-even; fp8 saturates to +-448.
 *   - MLA_FP8_E4M3: c_kv and k_pe as e4m3 codes, dequantised as code * cache_scale
 *     (one per-tensor scale).
 *   - MLA_FP8_E4M3_B128: the fp8 cache huny.dev §6 describes for DeepSeek-V3. c_kv is in
 *     e4m3 with one fp32 scale per 128 consecutive latent elements of each token, computed
 *     from the values when the token is written: scale = amax|x| / 448 and
 *     code = e4m3(x / scale), both divisions in IEEE fp32; a block of zeros has scale 0 and
 *     codes 0. The rotated k_pe stays in bf16. A cache row holds d_c code bytes, then d_c/128
 *     fp32 scales, then d_r bf16 values: d_c + d_c/32 + 2 d_r bytes (656 at DeepSeek-V2
 *     shapes; mla_cache_row_bytes). d_c must be a multiple of 128, and cache_scale is
 *     ignored.
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID = 1,      /* bad argument (null pointer, bad size or layout)        */
  MLA_ERR_UNSUPPORTED = 2,  /* valid but not implemented (dtype or shape combination)  */
  MLA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required              */
  MLA_ERR_CUDA = 4,         /* a CUDA runtime/driver call or a launch failed           */
  MLA_ERR_DEVICE_GUARD = 5, /* device data out of range; the bad rows were skipped     */
  MLA_ERR_TIMEOUT = 6       /* a bounded device-side wait gave up; the work was skipped */
} mla_status;

typedef enum { MLA_F32 = 0, MLA_BF16 = 1, MLA_FP8_E4M3 = 2, MLA_FP8_E4M3_B128 = 3 } mla_dtype;

/* Model dimensions and numeric options of one MLA layer.
 *   num_heads H, d_model d, d_latent d_c (c_kv width), d_rope d_r (k_pe width),
 *   d_nope d_n (per-head content query/key width), d_v (per-head value width),
 *   page_size P (tokens per cache page; 64 as in the FlashMLA backend).
 *   softmax_scale: multiplies q.k; <= 0 selects 1/sqrt(d_n + d_r).
 *   rope_theta: RoPE base; <= 0 selects 10000. Pairs (2k, 2k+1) are rotated by
 *     pos * theta^(-2k/d_r) (rope_interleaved = 1, the only supported layout).
 *   cache_scale: fp8 dequantisation scale (ignored for other cache dtypes). */
typedef struct {
  int num_heads, d_model, d_latent, d_rope, d_nope, d_v, page_size;
  float softmax_scale;
  float rope_theta;
  int rope_interleaved;
  mla_dtype act_dtype;
  mla_dtype cache_dtype;
  float cache_scale;
} mla_config;

/* Fold the up-projections into the serving weights, once at model load
 * (donmain.dev "위치 정보와 압축의 충돌"; huny.dev §3-1, §3-2).
 *   W_UK [d_c][H*d_n], W_UV [d_c][H*d_v], W_O [H*d_v][d]  (act dtype, inputs; head i
 *     owns columns i*d_n.. of W_UK, i*d_v.. of W_UV and rows i*d_v.. of W_O)
 *   W_UK_abs [H][d_n][d_c]   out: W_UK_abs[i] = (W_i^UK)^T
 *   W_comb   [H*d_c][d]      out: block i = W_i^UV W_i^O  (fp32 accumulation) */
mla_status mla_absorb_weights(const mla_config* cfg, const void* W_UK, const void* W_UV,
                              const void* W_O, void* W_UK_abs, void* W_comb, void* stream);

/* Append T new tokens from hidden states (huny.dev §2-1 and §2-3):
 *   [c | k_raw] = h W_DKV_KR,  k^R = RoPE(k_raw, position),
 * encoded in the cache dtype and written to
 *   cache[block_table[req][pos / P]][pos % P][0 : d_c + d_r] = [c | k^R].
 *   h [T][d], W_DKV_KR [d][d_c + d_r] = [W^DKV | W^KR]   (act dtype)
 *   req_ids [T], positions [T]          int32 (device)
 *   block_table [batch][max_pages]      int32 (device)
 *   cache [num_pages][P][d_c + d_r]     cache dtype, updated in place (MLA_FP8_E4M3_B128:
 *                                       bytes, [num_pages][P][mla_cache_row_bytes])
 *   dev_status                          optional int32 device word (may be NULL):
 *                                       MLA_ERR_DEVICE_GUARD is OR-ed in for skipped rows.
 *   workspace                           device buffer of mla_append_cache_workspace_size
 *                                       bytes (may be NULL when that is 0, as it is now for
 *                                       every configuration: the bf16 path sums its split-K
 *                                       partials on chip and encodes in the same kernel).
 * Rows must not share a (request, position); T == 0 is a no-op. */
mla_status mla_append_cache(const mla_config* cfg, const void* h, const void* W_DKV_KR, int T,
                            const int32_t* req_ids, const int32_t* positions,
                            const int32_t* block_table, int batch, int max_pages, void* cache,
                            int num_pages, int32_t* dev_status, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Bytes of one token's row in the paged cache: (d_c + d_r) * element size, or
 * d_c + d_c/32 + 2 d_r for MLA_FP8_E4M3_B128. A page is P rows. */
mla_status mla_cache_row_bytes(const mla_config* cfg, size_t* bytes);

/* Bytes of workspace mla_append_cache needs for T rows (currently 0). */
mla_status mla_append_cache_workspace_size(const mla_config* cfg, int T, size_t* bytes);

/* Append T tokens given their latent c_kv [T][d_c] and raw k_pe [T][d_r] (act dtype).
 * rotate != 0 applies RoPE at `positions` to k_pe before encoding; rotate == 0 stores
 * k_pe as given. Placement, encoding and guards as mla_append_cache. */
mla_status mla_append_cache_latent(const mla_config* cfg, const void* c_kv, const void* k_pe,
                                   int T, const int32_t* req_ids, const int32_t* positions,
                                   const int32_t* block_table, int batch, int max_pages,
                                   void* cache, int num_pages, int rotate, int32_t* dev_status,
                                   void* stream);

/* Decode tuning knobs (NULL = defaults). num_workers: how many independent workers
 * share the key pages (0 = one per SM pair on this GPU); kernel: 0 = best available,
 * 1 = the SIMT kernel, 2 = the tensor-core (tcgen05) kernel. attn_events: optional
 * pair of cudaEvent_t (as void*) recorded on `stream` right before and right after
 * the attention kernel, for timing it alone; NULL entries are ignored.
 * Testing hooks of the tensor-core kernel's failure path (zero-initialise them otherwise):
 * wait_limit_us: how long any of its barrier waits may last before the kernel gives up,
 * records MLA_ERR_TIMEOUT in the status word, releases its tensor memory and exits
 * (0 = the default, 2 s); withhold_page: when >= 1, the page of index withhold_page - 1 in
 * worker 0's sequence is never loaded, so that the wait for it runs out (0 = off). Both
 * leave every other worker's results intact; the call's status then reads
 * MLA_ERR_TIMEOUT and its outputs for worker 0's requests are undefined. */
typedef struct {
  int num_workers;
  int kernel;
  void* attn_events[2];
  int wait_limit_us;
  int withhold_page;
} mla_decode_opts;

/* Bytes of workspace mla_decode needs for this batch on the current device. */
mla_status mla_decode_workspace_size(const mla_config* cfg, int batch, int q_len,
                                     const mla_decode_opts* opts, size_t* bytes);

/* Weight-absorbed decode (huny.dev §3-1; secrett2633.cloud "MLA의 MQA 디코딩 경로",
 * "FlashMLAImpl"). For request b, query token t (0 <= t < q_len) sits at position
 * p = seq_lens[b] - q_len + t and attends to the cached keys 0..p of its request;
 * for every head i:
 *   q_lat = [ q_nope[b][t][i] W_UK_abs[i] ; RoPE(q_pe[b][t][i], p) ]      (d_c + d_r)
 *   s_j   = softmax_scale * q_lat . cache_row_j            (fp8: * cache_scale)
 *   out_latent[b][t][i] = sum_j softmax(s)_j c_j,  lse[b][t][i] = ln sum_j exp(s_j).
 *   q_nope [batch][q_len][H][d_n], q_pe [batch][q_len][H][d_r], W_UK_abs [H][d_n][d_c]
 *     (act dtype); cache, num_pages as in mla_append_cache;
 *   block_table [batch][max_pages], seq_lens [batch]  int32 (device); seq_lens count the
 *     cached tokens including this step's q_len tokens (appended before the call);
 *   out_latent [batch][q_len][H][d_c] (act dtype), lse [batch][q_len][H] (fp32)  outputs.
 * seq_lens[b] == 0 marks an empty request: out_latent = 0, lse = -inf.
 * The cache has to start at a multiple of 4 bytes (a block-scaled one in the append calls too);
 * the tensor-core kernel's out_latent at one of 16. d_latent above 512: MLA_ERR_UNSUPPORTED.
 * workspace: device buffer of at least mla_decode_workspace_size bytes, 256-byte
 * aligned, owned by the caller, any initial contents; its first int32 is the device
 * status word, cleared by each call and then set by that call's guards. Calls that
 * share one workspace must be ordered on the GPU. */
mla_status mla_decode(const mla_config* cfg, const void* q_nope, const void* q_pe,
                      const void* W_UK_abs, const void* cache, int num_pages,
                      const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                      int batch, int q_len, void* out_latent, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream);

/* mla_decode with explicit knobs (opts may be NULL). */
mla_status mla_decode_ex(const mla_config* cfg, const void* q_nope, const void* q_pe,
                         const void* W_UK_abs, const void* cache, int num_pages,
                         const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                         int batch, int q_len, void* out_latent, float* lse, void* workspace,
                         size_t workspace_bytes, const mla_decode_opts* opts, void* stream);

/* mla_decode without a caller workspace, for callers that cannot allocate device memory
 * when they decode (a plugin inside a runtime that owns all device allocations, a serving
 * loop with a frozen memory footprint, an environment that bans dynamic allocation). The
 * pages have no counterpart to this call: it is a deployment convenience of this library.
 * Its scratch is one 64 MiB array in device memory, statically part of the library and
 * held by every GPU that loads it until the process exits; a batch whose
 * mla_decode_workspace_size exceeds 64 MiB is rejected with MLA_ERR_WORKSPACE and an
 * explanation in mla_last_error(). The first call on a device looks the array up
 * (cudaGetSymbolAddress) with that device current: make it outside any stream capture.
 * All calls share the array, so calls whose GPU work overlaps (other streams, unordered
 * host threads) race; order them on one stream. Nothing in the array needs to start at
 * zero. Arguments and results are those of mla_decode; the call's device status (its
 * guards) is read with mla_decode_noalloc_status. */
mla_status mla_decode_noalloc(const mla_config* cfg, const void* q_nope, const void* q_pe,
                              const void* W_UK_abs, const void* cache, int num_pages,
                              const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                              int batch, int q_len, void* out_latent, float* lse, void* stream);

/* The device status of the last mla_decode_noalloc on the current device: waits for
 * `stream`, then reads the status word at the start of the library's scratch array into
 * *code (MLA_OK, or MLA_ERR_DEVICE_GUARD when that call's guards skipped a request) and
 * resets it to 0. The pages have no counterpart to this call. The array's address is looked
 * up once per device and kept: neither call may be used on a device after a
 * cudaDeviceReset of it in the same process. Errors: MLA_ERR_INVALID (code is NULL),
 * MLA_ERR_CUDA. */
mla_status mla_decode_noalloc_status(void* stream, int* code);

/* Bytes of workspace mla_output_proj needs for `rows` rows (may be 0). */
mla_status mla_output_proj_workspace_size(const mla_config* cfg, int rows, size_t* bytes);

/* Output projection through the folded weights (huny.dev §3-2):
 *   out[r] = sum_i out_latent[r][i] W_comb[i*d_c : (i+1)*d_c]
 *   out_latent [rows][H*d_c], W_comb [H*d_c][d], out [rows][d]  (act dtype),
 *   fp32 accumulation. workspace: 256-byte aligned device buffer of
 *   mla_output_proj_workspace_size bytes (an fp32 accumulator, used with fp32 activations,
 *   plus a status word). */
mla_status mla_output_proj(const mla_config* cfg, const void* out_latent, const void* W_comb,
                           int rows, void* out, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Bytes of workspace mla_output_proj_unfolded needs for `rows` rows (may be 0). */
mla_status mla_output_proj_unfolded_workspace_size(const mla_config* cfg, int rows,
                                                   size_t* bytes);

/* Output projection without the fold, the two sides of huny.dev §3-2 read before the
 * absorption (its first equation, then the per-head output projection):
 *   u[r][i] = out_latent[r][i] W_i^UV      (per head: d_c -> d_v, rounded to the act dtype)
 *   out[r]  = sum_i u[r][i] W_i^O
 *   out_latent [rows][H*d_c]; W_UV [d_c][H*d_v] and W_O [H*d_v][d] as given to
 *   mla_absorb_weights (head i owns columns i*d_v.. of W_UV, rows i*d_v.. of W_O);
 *   out [rows][d]  (act dtype), fp32 accumulation. It streams H*d_c*d_v + H*d_v*d weight
 *   elements instead of W_comb's H*d_c*d (185 MB instead of 671 MB at DeepSeek-V2 shapes);
 *   equal to mla_output_proj up to the rounding of u. workspace: 256-byte aligned device
 *   buffer of mla_output_proj_unfolded_workspace_size bytes (an fp32 accumulator, used with
 *   fp32 activations, a status word and u). Errors as mla_output_proj. */
mla_status mla_output_proj_unfolded(const mla_config* cfg, const void* out_latent, const void* W_UV,
                                    const void* W_O, int rows, void* out, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Bytes of workspace mla_query_from_hidden needs for T query rows and query rank d_q. */
mla_status mla_query_workspace_size(const mla_config* cfg, int d_q, int T, size_t* bytes);

/* The step's queries from the hidden states, by low-rank query compression (huny.dev
 * "DeepSeek MLA 해부" §2-2) and the per-head rotary query (§2-3):
 *   c_q[t]       = h[t] W_DQ                              (d -> d_q, rounded to the act dtype)
 *   q_nope[t][i] = c_q[t] W_UQ[:, i*d_n : (i+1)*d_n]
 *   q_pe[t][i]   = h[t] W_QR[:, i*d_r : (i+1)*d_r]       (not rotated: mla_decode rotates it
 *                                                          at the query position)
 *   h [T][d]; W_DQ [d][d_q]; W_UQ [d_q][H*d_n]; W_QR [d][H*d_r]; outputs q_nope [T][H][d_n]
 *   and q_pe [T][H][d_r], the layouts mla_decode reads (row b*q_len + t), all in the act
 *   dtype, fp32 accumulation. W_UQ stays separate from W_UK: merging them per head
 *   (W_i^UQ (W_i^UK)^T, d_q x d_c) would make the step read H*d_q*d_c weight elements (201 MB at
 *   DeepSeek-V2 shapes) instead of H*d_q*d_n + H*d_n*d_c (67 MB).
 *   workspace: 256-byte aligned device buffer of mla_query_workspace_size bytes (an fp32
 *   accumulator, used with fp32 activations, a status word and c_q). d_q > 0; T == 0 is a no-op. Errors: MLA_ERR_INVALID
 *   (null pointers, bad sizes), MLA_ERR_WORKSPACE, MLA_ERR_CUDA; nothing is launched on an
 *   error found on the host. */
mla_status mla_query_from_hidden(const mla_config* cfg, int d_q, const void* h, const void* W_DQ,
                                 const void* W_UQ, const void* W_QR, int T, void* q_nope,
                                 void* q_pe, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* ---- a prefix shared by a batch -------------------------------------------------------
 * Requests that open with the same tokens (a system prompt, few-shot examples) can attend to
 * them together: the prefix is expanded once from its cached latents into per-head keys and
 * values (huny.dev §2-1: k^C = c W^UK, v^C = c W^UV), each step attends to those for every
 * request of the batch at once, and the result is joined with mla_decode's over the request's
 * own tokens. Per key, head and query this multiplies d_n + d_r + d_v elements instead of
 * the absorbed form's 2 d_c + d_r, and a step reads the expanded prefix once, not once per
 * request. But the expanded prefix is large: H (d_n + d_v) + d_r elements a token, 65.7 KB in bf16
 * at DeepSeek-V2 shapes (57 times its cached row; 538 MB per layer for 8192 tokens), so that a
 * step costs the same for one request as for 128. With few query tokens (batch * q_len) a plain
 * mla_decode, with block tables that all name the prefix's pages in front of the request's own, is
 * faster: measured, the attention to the prefix alone, it leads up to about 10 query tokens at 2048
 * prefix tokens, 33 at 8192 and 40 at 32768, and nowhere at 512 (8192 tokens: 57 us against 93 for 16
 * query tokens, 157 against 95 for 64, 287 against 99 for 128). (That form numbers a request's own
 * tokens from prefix_len, which has to be a whole number of pages.) A step is
 *   mla_prefix_attend(..)        -> u_prefix, lse_prefix   (the shared tokens)
 *   mla_decode(..)               -> out_latent, lse        (each request's own tokens)
 *   mla_output_proj_prefix(..)   -> out
 * Positions: the prefix's tokens were appended at positions 0..prefix_len - 1. A request's
 * own tokens are appended to its own pages, numbered from 0 (append and decode rotate by
 * that number; scores depend on differences of positions alone, so the decode over own
 * tokens needs no offset), and mla_prefix_attend rotates the query of token t at
 * prefix_len + seq_lens[b] - q_len + t, where seq_lens counts own tokens only, as given to
 * mla_decode. Every prefix key is visible to every query token. Several prefixes in one
 * batch: one mla_prefix_attend per prefix, on the rows of its requests.
 *
 * For these calls and those of eviction below: the tensor-core kernels serve bf16 activations at
 * DeepSeek-V2's head shape (d_n 128, d_r 64, d_v 128, d_c 512, 64-token pages, any number of heads;
 * key weights 16 to 128 heads by 16) and tensors that start at multiples of 16 bytes; any other
 * shape, fp32, or a tensor that starts elsewhere takes SIMT kernels with the same results up to
 * rounding, many times slower at large sizes. (mla_absorb_query takes the decode's GEMM for every bf16
 * shape with d_n and d_c multiples of 8 and a q_nope and W_UK_abs that start at multiples of 16 bytes.) The cache has to start at a multiple of 4 bytes (eviction
 * from an fp32 cache: 16). batch * q_len is limited to 32768 as in mla_decode. A tensor-core
 * kernel's waits are bounded: should one run out (2 s), the call's work is left undone and
 * MLA_ERR_TIMEOUT is OR-ed into *dev_status (mla_output_proj_prefix and mla_absorb_query have no such
 * word: their outputs are then not written). Sums are
 * made in one order, so that every run gives the same bits. Inputs and outputs must not overlap
 * unless a call says so. */

/* Expand the prefix's cached rows, once per prefix (and weights):
 *   keys[i][l] = c_l W_UK[:, i*d_n : (i+1)*d_n],  values[i][l] = c_l W_UV[:, i*d_v : (i+1)*d_v],
 *   k_pe[l] = the rotated key of row l as cached (fp8: the values of the codes).
 *   W_UK, W_UV as given to mla_absorb_weights; cache, num_pages as in mla_append_cache;
 *   prefix_pages [ceil(prefix_len / P)] int32 (device): the prefix's pages;
 *   keys [H][prefix_len][d_n], values [H][prefix_len][d_v], k_pe [prefix_len][d_r]: outputs,
 *   act dtype, fp32 sums. From a block-scaled fp8 cache the tensor-core form rounds code *
 *   scale to bf16 before the product. prefix_len == 0 is a no-op; above 4194304 it is
 *   MLA_ERR_UNSUPPORTED. A page id out of range gives rows of zeros and MLA_ERR_DEVICE_GUARD
 *   in *dev_status (optional, may be NULL; OR-ed in, never cleared by the call). */
mla_status mla_prefix_expand(const mla_config* cfg, const void* W_UK, const void* W_UV,
                             const void* cache, int num_pages, const int32_t* prefix_pages,
                             int prefix_len, void* keys, void* values, void* k_pe,
                             int32_t* dev_status, void* stream);

/* Bytes of workspace mla_prefix_attend needs for this batch on the current device (may be 0). */
mla_status mla_prefix_attend_workspace_size(const mla_config* cfg, int batch, int q_len,
                                            int prefix_len, size_t* bytes);

/* Attention of every request's query tokens to an expanded prefix; for each head i
 *   s_l = softmax_scale * (q_nope[b][t][i] . keys[i][l] + RoPE(q_pe[b][t][i], p) . k_pe[l]),
 *   p = prefix_len + seq_lens[b] - q_len + t,
 *   u[b][t][i] = sum_l softmax(s)_l values[i][l],  lse[b][t][i] = ln sum_l exp(s_l).
 *   q_nope [batch][q_len][H][d_n], q_pe [batch][q_len][H][d_r] as given to mla_decode (not
 *   rotated); keys, values, k_pe from mla_prefix_expand; seq_lens [batch] int32 (device): each
 *   request's own cached tokens including this step's q_len; u [batch][q_len][H][d_v] (act
 *   dtype), lse [batch][q_len][H] (fp32) outputs. d_n + d_r + d_v above 57344:
 *   MLA_ERR_UNSUPPORTED.
 * The softmax's weights are rounded to the act dtype for the product with the values; scores,
 * maxima and sums are held in fp32, and so is the rotated query up to 3 keys; above, with bf16, it is
 * the sum of two bf16 terms, each element off by at most 2^-17 of itself (sine and cosine by 2^-21). A NaN score makes its row's u and lse NaN.
 * seq_lens[b] == 0 marks an empty request (u = 0, lse = -inf), as does prefix_len == 0 for
 * every request; 0 < seq_lens[b] < q_len is a guard error (same outputs). workspace: 256-byte
 * aligned device buffer of mla_prefix_attend_workspace_size bytes (NULL if that is 0), any
 * contents; calls that share one must be ordered on the GPU. dev_status as above. */
mla_status mla_prefix_attend(const mla_config* cfg, const void* q_nope, const void* q_pe,
                             const void* keys, const void* values, const void* k_pe, int prefix_len,
                             const int32_t* seq_lens, int batch, int q_len, void* u, float* lse,
                             void* workspace, size_t workspace_bytes, int32_t* dev_status,
                             void* stream);

/* Bytes of workspace mla_output_proj_prefix needs for `rows` rows: as many as
 * mla_output_proj_unfolded (whose accumulator's place this call leaves unused) and, with bf16
 * activations above 128 rows, fp32 pieces of the product where it is cut, up to 80 MB. */
mla_status mla_output_proj_prefix_workspace_size(const mla_config* cfg, int rows, size_t* bytes);

/* mla_output_proj_unfolded of the attention over both key sets, own tokens and prefix:
 *   a = exp(lse) / (exp(lse) + exp(lse_prefix)) per row and head (both -inf: no keys at all,
 *       u = 0),
 *   u[r][i] = a out_latent[r][i] W_i^UV + (1 - a) u_prefix[r][i]   (rounded to the act dtype)
 *   out[r]  = sum_i u[r][i] W_i^O
 *   out_latent [rows][H*d_c] and lse [rows][H] from mla_decode, u_prefix [rows][H*d_v] and
 *   lse_prefix [rows][H] from mla_prefix_attend; the rest as mla_output_proj_unfolded. A part
 *   whose weight is 0 is not read into the sum, whatever it holds. */
mla_status mla_output_proj_prefix(const mla_config* cfg, const void* out_latent, const float* lse,
                                  const void* u_prefix, const float* lse_prefix, const void* W_UV,
                                  const void* W_O, int rows, void* out, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* ---- eviction by accumulated attention weight ------------------------------------------
 * mla_key_weights adds up how much attention each cached token receives; mla_evict_cache keeps
 * the tokens that received most and closes the gaps, so that the request goes on with a
 * shorter cache: mla_append_cache and mla_decode then take the new lengths (and pages). */

/* The query as mla_decode forms it, for mla_key_weights:
 *   q_lat[b][t][i] = [ q_nope[b][t][i] W_UK_abs[i] ; RoPE(q_pe[b][t][i], p) ],
 *   p = seq_lens[b] - q_len + t; arguments as in mla_decode, q_lat [batch][q_len][H][d_c + d_r]
 *   (act dtype, fp32 sums). Rows of a request with seq_lens[b] < q_len are not defined. */
mla_status mla_absorb_query(const mla_config* cfg, const void* q_nope, const void* q_pe,
                            const void* W_UK_abs, const int32_t* seq_lens, int batch, int q_len,
                            void* q_lat, void* stream);

/* Accumulate the attention weight of every cached token over heads and query tokens:
 *   mass_j = sum over t, i of exp(softmax_scale * q_lat[b][t][i] . cache_row_j - lse[b][t][i])
 *     (fp8: cache_row_j as the values of its codes), over the t that see j, i.e. with
 *     j <= seq_lens[b] - q_len + t;
 *   weights[b][j] = decay * weights[b][j] + mass_j   for tokens cached before this step
 *   weights[b][j] = mass_j                           for its q_len new tokens, or decay == 0
 * for j < seq_lens[b]; entries behind are left as they are. With lse from mla_decode on the
 * same step, mass sums to H * q_len over a request's tokens; with the LSE of a larger key set (a
 * shared prefix joined in) it is the own tokens' share of it.
 *   q_lat [batch][q_len][H][d_c + d_r] (act dtype; mla_absorb_query), lse [batch][q_len][H]
 *   (fp32); cache, block_table, seq_lens, batch, q_len as in mla_decode; decay in [0, 1];
 *   weights [batch][max_pages * P] fp32 (device), updated in place. With decay > 0 the entries of
 *   tokens cached before this step are read, so each has to be written first: by the call of the
 *   step that cached the token, or by the caller (0, say) for tokens cached without one: a prompt,
 *   or what was appended after an eviction, behind whose new lengths the old entries remain. Entries
 *   of this step's tokens and behind the request, and all of them with decay == 0, may hold anything.
 * Sums are fp32, in a fixed order (the same bits every time). On fp8 caches the tensor-core form
 * takes each head's latent query (and rotary one, with a per-tensor scale) as the sum of two e4m3
 * terms: exact for elements down to 2^-13 of the head's largest, smaller ones off by up to 2^-19 of
 * it. seq_lens[b] == 0: nothing is written. Requests with a bad length and tokens on a bad page are left out, with
 * MLA_ERR_DEVICE_GUARD in *dev_status (optional, OR-ed in). MLA_ERR_UNSUPPORTED: batch * max_pages
 * or max_pages * P above 2^31 - 1; rows so wide that a page of them and a query in fp32 do not fit
 * 227 KB (64-token pages: d_c + d_r above 892 in fp32, 1756 in bf16, 3412 in e4m3, 3136 block-scaled). */
mla_status mla_key_weights(const mla_config* cfg, const void* q_lat, const float* lse,
                           const void* cache, int num_pages, const int32_t* block_table,
                           int max_pages, const int32_t* seq_lens, int batch, int q_len, float decay,
                           float* weights, int32_t* dev_status, void* stream);

/* Cut every request's cache down to at most `budget` tokens. A request with
 * seq_lens[b] <= budget keeps all; otherwise its first `sinks` tokens, its last `recent` ones
 * and, of those between, the budget - sinks - recent with the largest weights (equal weights:
 * the lowest index first; NaN below every number). In ascending order they become tokens
 * 0, 1, .. of the request: row kept[i] of the old pages is written as row i of the new
 * pages, in the cache's own encoding. rotate != 0 turns its rotary key by (i - kept[i])
 * theta_k (fp32, rounded to the cache's type; e4m3 saturates), so that row i carries the
 * rotation of position i that mla_append_cache writes and mla_decode assumes; rotate == 0
 * copies rows as they are. Rows with i == kept[i] are copied bit for bit.
 *   weights [batch][max_pages * P] fp32; seq_lens [batch]; block_table [batch][max_pages];
 *   new_block_table [batch][new_max_pages] int32: the same array as block_table (in place:
 *     nothing moves for requests within the budget; no page may belong to two requests), or
 *     an array whose pages are none that block_table names;
 *   new_weights [batch][new_max_pages * P] fp32, optional (NULL): the kept tokens' weights in
 *     their new order (entries behind are left as they are); may be `weights` itself if
 *     new_max_pages == max_pages, otherwise they must not overlap;
 *   kept [batch][budget] int32: the kept tokens' old indices, ascending, then -1;
 *   new_seq_lens [batch] int32: min(seq_lens[b], budget); may be seq_lens itself.
 * A request with seq_lens[b] outside [0, max_pages * P], or more kept tokens than
 * new_max_pages * P, is left alone (kept all -1, new length the old one), and a row whose old
 * or new page is out of range is not moved: MLA_ERR_DEVICE_GUARD in *dev_status (optional,
 * OR-ed in). MLA_ERR_UNSUPPORTED: max_pages * P above 393216 tokens,
 * num_pages * P above 2^31 - 1, budget above 2^30. budget > 0, batch at most 32768. No workspace. */
mla_status mla_evict_cache(const mla_config* cfg, const float* weights, const int32_t* seq_lens,
                           const int32_t* block_table, int max_pages, int batch, int budget,
                           int sinks, int recent, int rotate, void* cache, int num_pages,
                           const int32_t* new_block_table, int new_max_pages, float* new_weights,
                           int32_t* kept, int32_t* new_seq_lens, int32_t* dev_status, void* stream);

/* ---- page-sparse decoding -----------------------------------------------------------------
 * A long context's cache is read whole by every mla_decode. These calls let each query token read only
 * the pages that an estimate finds worth reading: a summary of each page (mla_page_keys), the attention
 * that the query would pay to each page by those summaries (mla_page_scores: 1/64 of the cache's bytes),
 * the pages kept (mla_select_pages) and the attention over their tokens (mla_decode_pages). A step is
 *   mla_append_cache(..), mla_page_keys(.., new_tokens = q_len, ..)
 *   mla_absorb_query(..)  -> q_lat
 *   mla_page_scores(..)   -> scores
 *   mla_select_pages(..)  -> pages
 *   mla_decode_pages(..)  -> out_latent, lse     (then an output projection as ever)
 * The cache, its block tables and lengths are those of mla_append_cache and mla_decode and are not
 * changed. A page is one of the cache's own, of P tokens: page p of a request holds its tokens
 * p P .. p P + P - 1. Query token t of request b sits at seq_lens[b] - q_len + t and sees the pages
 * 0 .. (seq_lens[b] - q_len + t) / P. Sums are made in one order: every run gives the same bits. Inputs
 * and outputs must not overlap. *dev_status (optional, may be NULL) has MLA_ERR_DEVICE_GUARD OR-ed in. */

/* The mean of a page's cached rows, latent and rotary part, as its key:
 *   page_keys[page] = (1 / n) sum over its n cached tokens of the row   (fp8: the values of the codes)
 * for every page that holds one of the request's last new_tokens tokens (all its pages if new_tokens >=
 * seq_lens[b]: a prompt, or after mla_evict_cache); other rows are left as they are. fp32 sums, rounded
 * once.
 *   cache, num_pages, block_table, max_pages, seq_lens, batch as in mla_decode (batch at most 32768);
 *   page_keys [num_pages][d_c + d_r] act dtype, indexed like the cache by physical page (a page that
 *   several requests share has one key; the requests have to agree on how many of its tokens are cached).
 * seq_lens[b] == 0: nothing is written; a length outside [0, max_pages * P] or a page id out of range is
 * left out, with the guard. The cache has to start at a multiple of 4 bytes. MLA_ERR_UNSUPPORTED:
 * d_c + d_r above 58112, max_pages * P above 2^31 - 1. No workspace. */
mla_status mla_page_keys(const mla_config* cfg, const void* cache, int num_pages, const int32_t* block_table,
                         int max_pages, const int32_t* seq_lens, int batch, int new_tokens, void* page_keys,
                         int32_t* dev_status, void* stream);

/* Bytes of workspace mla_page_scores needs for this batch on the current device: every head's sum for the SIMT
 * kernels, asked for whichever kernel a call's addresses will choose. */
mla_status mla_page_scores_workspace_size(const mla_config* cfg, int batch, int q_len, int max_pages,
                                          size_t* bytes);

/* The attention that each query token would pay to each page if every token's key were its page's:
 *   z_ip = softmax_scale * q_lat[b][t][i] . page_keys[page p],
 *   scores[b][t][p] = sum over heads i of m_p exp(z_ip) / sum_p' m_p' exp(z_ip'),
 * m_p the tokens of page p that the query sees (P, or fewer on its last page), over the pages it sees:
 * they share out H. Entries behind them are left as they are.
 *   q_lat [batch][q_len][H][d_c + d_r] (act dtype; mla_absorb_query); page_keys from mla_page_keys;
 *   block_table, seq_lens as in mla_decode; scores [batch][q_len][max_pages] fp32.
 * fp32 sums and softmax. The tensor-core kernel takes bf16 at d_c 512, d_r 64, 64-token pages, up to 128
 * heads and max_pages up to 8192, for q_lat and page_keys that start at multiples of 16 bytes; anything else
 * takes SIMT kernels, many times slower at large sizes. A page with an id out of range scores 0, a request with seq_lens[b] < q_len or
 * above max_pages * P is left out, both with the guard; seq_lens[b] == 0 is left out. Should a bounded wait of the
 * tensor-core kernel run out, MLA_ERR_TIMEOUT is OR-ed into *dev_status and that query's scores are not written.
 * workspace: 256-byte
 * aligned device buffer of mla_page_scores_workspace_size bytes, any contents; calls that share one must be
 * ordered on the GPU. */
mla_status mla_page_scores(const mla_config* cfg, const void* q_lat, const void* page_keys, int num_pages,
                           const int32_t* block_table, int max_pages, const int32_t* seq_lens, int batch,
                           int q_len, float* scores, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, void* stream);

/* The pages that each query token keeps: all it sees if they are at most `budget`, otherwise its first
 * `sinks`, its last `recent` and, of those between, the budget - sinks - recent with the largest scores
 * (equal scores: the lowest index first; NaN below every number).
 *   scores [batch][q_len][max_pages] fp32; seq_lens [batch]; pages [batch][q_len][budget] int32: page
 *   indices of the request, ascending, then -1.
 * seq_lens[b] == 0 gives an empty list (all -1), as does a length below q_len or above max_pages * P, with
 * the guard. MLA_ERR_UNSUPPORTED: max_pages above 49152. No workspace. Use recent >= 1 to keep the page of
 * the query itself. */
mla_status mla_select_pages(const mla_config* cfg, const float* scores, int max_pages, const int32_t* seq_lens,
                            int batch, int q_len, int budget, int sinks, int recent, int32_t* pages,
                            int32_t* dev_status, void* stream);

/* Bytes of workspace mla_decode_pages needs for this batch on the current device. */
mla_status mla_decode_pages_workspace_size(const mla_config* cfg, int batch, int q_len, int budget,
                                           size_t* bytes);

/* mla_decode over the tokens of chosen pages: query token t of request b attends to the tokens of the
 * pages on its list that it sees (j <= seq_lens[b] - q_len + t),
 *   s_j = softmax_scale * q_lat[b][t][i] . cache_row_j,  out_latent = sum_j softmax(s)_j c_j,
 *   lse = ln sum_j exp(s_j).
 *   q_lat [batch][q_len][H][d_c + d_r] as formed by mla_absorb_query (act dtype, rotated); pages
 *   [batch][q_len][budget] int32: page indices of the request, ascending, -1 behind the end (from
 *   mla_select_pages, or any other choice); the rest as in mla_decode. A list of all pages gives
 *   mla_decode's result up to rounding.
 * An empty list or seq_lens[b] == 0: out_latent = 0, lse = -inf. A length below q_len or above max_pages *
 * P is skipped like an empty request, with the guard; a list that is not ascending, has a page behind a -1 or names
 * one that the query does not see sets the guard and leaves that query's result undefined. workspace: as in
 * mla_decode (its first int32 is the call's status word, cleared by each call). MLA_ERR_UNSUPPORTED:
 * d_latent above 512, batch * q_len above 8192. The tensor-core kernel takes bf16 activations at d_c 512, d_r
 * 64, 64-token pages, any cache format and a multiple of 16 heads up to 1024, for a q_lat and cache that start
 * at multiples of 16 bytes; anything else takes the SIMT kernel, and a cache that does not start at a multiple
 * of 4 bytes is refused. Scores and LSE are fp32 results; the softmax's weights are rounded to bf16 for the
 * product with the latents. On the tensor cores an fp8 cache's are two e4m3 terms under a power of two per head and
 * 32 tokens of a page (block scales: the weights times the tokens' scales, per 128 dims): off by 2^-9 of
 * themselves, or by 2^-21 of the largest of the 32 (of the largest weight times the largest scale) where that is
 * more. */
mla_status mla_decode_pages(const mla_config* cfg, const void* q_lat, const void* cache, int num_pages,
                            const int32_t* block_table, int max_pages, const int32_t* seq_lens, int batch,
                            int q_len, const int32_t* pages, int budget, void* out_latent, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ---- 4-bit weights ------------------------------------------------------------------------
 * A weight W [K][N] (as every weight of this library: x W with x [rows][K]) as 4-bit floating point with
 * microscaling: 17/32 of a byte an element instead of 2. Each block of 32 elements along K of one column
 * has a scale 2^e and 32 codes of e2m1 (a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6); an element's value
 * is code * 2^e. e is the exponent of the block's largest magnitude, rounded to two significant bits,
 * less 2 (the largest magnitude then lies in [3.5, 7) scales; at most 125, at least -127), and codes
 * round to nearest even, +-6 at most. A block that holds an infinity or NaN has the scale NaN.
 *   codes [N][K / 2] bytes: column n contiguous, element 2 j in the low half of byte j, 2 j + 1 in the high;
 *   scales [ceil(N / 128)][ceil(K / 128)][32][4][4] bytes, e + 127 (255: NaN): block kb = k / 32 of column
 *   n at [n / 128][kb / 4][n % 32][(n % 128) / 32][kb % 4]; entries of columns behind N and blocks behind
 *   K hold 127.
 * K is a multiple of 32 (MLA_ERR_INVALID otherwise), K and N at most 8388608; codes and scales start at
 * multiples of 16 bytes. Of cfg these calls use the act dtype (and refuse an invalid one). */

/* Sizes of the two arrays. */
mla_status mla_mx4_bytes(const mla_config* cfg, int K, int N, size_t* codes_bytes, size_t* scales_bytes);

/* W [K][N] (act dtype) -> codes, scales; once at load, say for W_comb, W_O, W_DQ, W_UQ or W_QR. */
mla_status mla_mx4_quantize(const mla_config* cfg, const void* W, int K, int N, void* codes, void* scales,
                            void* stream);

/* codes, scales -> the values W [K][N] (act dtype; every value is exact in bf16). */
mla_status mla_mx4_dequantize(const mla_config* cfg, const void* codes, const void* scales, int K, int N, void* W,
                              void* stream);

/* Bytes of workspace mla_mx4_project needs for `rows` rows (may be 0). */
mla_status mla_mx4_project_workspace_size(const mla_config* cfg, int K, int N, int rows, size_t* bytes);

/* out = x W for a 4-bit W: x [rows][K], out [rows][N] (act dtype), fp32 sums. With W = W_comb and x =
 * out_latent this is mla_output_proj with a quarter of its bytes to read.
 *   workspace: 256-byte aligned device buffer of mla_mx4_project_workspace_size bytes (NULL if that is 0),
 *   any contents; calls that share one must be ordered on the GPU. Its first int32 is the call's status word,
 *   cleared by each call (mla_read_device_status). rows == 0 is a no-op.
 * bf16 activations run on the tensor cores (an x that does not start at a multiple of 16 bytes on the SIMT
 * kernel): x enters as exact sums of 4-bit or e4m3 values under a power of two per 32 elements, off by at most
 * 2^-17 of the largest of the 32 (or 2^-128 where that is more), and a row that holds an infinity or NaN gives NaN in all its outputs. A
 * column with a NaN scale gives NaN. Should a bounded wait of the kernel run out, the status word gets
 * MLA_ERR_TIMEOUT and outputs may be left as they were; none gets a partial sum. */
mla_status mla_mx4_project(const mla_config* cfg, const void* x, const void* codes, const void* scales, int K,
                           int N, int rows, void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Wait for `stream`, then read the device status word at `status_word` (a decode
 * workspace or an append dev_status) into *code (an mla_status value, MLA_OK if clean)
 * and reset it to 0. */
mla_status mla_read_device_status(const void* status_word, void* stream, int* code);

/* Static description of a status code. */
const char* mla_status_string(mla_status status);

/* Text of the last CUDA error seen by this thread's calls ("" if none). */
const char* mla_last_error(void);

/* Library ABI version (major * 100 + minor). 1.02: mla_append_cache needs no workspace
 * (its size is 0). 1.03: the shared-prefix and eviction calls. 1.04: page-sparse decoding and 4-bit
 * weights. 1.05: the workspace of mla_mx4_project starts with its status word. */
int mla_version(void);

/* Testing hook of the failure paths of the tensor-core kernels of mla_mx4_project and mla_page_scores, for this host
 * thread's calls until it is set again: wait_limit_us (0: the default, 2 s) is how long a barrier wait may last. With
 * withhold >= 1 the first CTA's copy of index withhold - 1 never arrives (mla_mx4_project: nor those behind it), so that
 * the wait for it runs out; 0: all do. */
void mla_testing_waits(int wait_limit_us, int withhold);

/* Number of CUDA kernels the library has launched in this process so far (all
 * threads, all devices); lets a caller count the kernels of a timed region. */
uint64_t mla_kernel_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
