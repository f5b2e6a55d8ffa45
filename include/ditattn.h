/*
 * ditattn — non-causal DiT self-attention on GB300 (sm_103a), C ABI.
 *
 * The library computes O = softmax(scale * Q K^T) V per (batch, head) over
 * long token sequences, either in one fused pass or as p KV chunks whose
 * partial outputs and log-sum-exps are merged exactly as one Ring-attention
 * hop merges them: by a separate merge of the p stacked partials, or hop by
 * hop into a running output inside each chunk pass.  On one GPU the p chunks
 * are virtual ranks: a "hop" is a pointer to the next chunk, with no
 * communication.
 *
 * Conventions shared by every entry point:
 *  - Tensors are plain device pointers, contiguous row-major [B, H, N, D]
 *    ("BHND"), except where a head stride is passed explicitly.  Q, K, V are
 *    bf16 (IEEE binary16-brain, 2 bytes).  LSE buffers are fp32 [B, H, N].
 *  - lse is the NATURAL log of sum_j exp(scale * q_i . k_j) over the keys the
 *    call covers (the kernels work in base 2 internally and convert).
 *  - The caller owns every buffer.  The library calls no device allocator.
 *    Besides a cache of host-side TMA-descriptor encoders it holds two
 *    fixed device arrays in its own module: one status word, and the 128 MiB
 *    scratch array of dit_attn_chunk_fwd_splitkv_noalloc.  The CUDA runtime
 *    reserves them on a device when it loads the library's device code there:
 *    on the first call that uses that device under the default lazy module
 *    loading, or when the library is loaded under CUDA_MODULE_LOADING=EAGER.
 *    On a device too full to take them, that first call fails with
 *    DIT_ERR_CUDA.  Device addresses are looked up once per device number and
 *    assume the runtime's primary context (no cudaDeviceReset in between).
 *  - Calls are asynchronous on `stream` (0 = legacy default stream).  Argument
 *    errors are returned before anything is launched.  A launch failure
 *    returns DIT_ERR_CUDA.  Device-side timeouts (a bounded wait that
 *    expired) are recorded in the status word and reported by
 *    dit_attn_check(), which synchronises the stream.
 *  - Validation (before launch): B, H, N, n_kv, p >= 1; D in {64, 128} (else
 *    DIT_ERR_UNSUPPORTED); pointers non-null; q, k, v, out, partials 16-byte
 *    aligned; lse buffers 4-byte aligned; scale finite and > 0; outputs must
 *    not overlap inputs; sizes must fit the kernels' 32-bit tile coordinates
 *    (N < 2^31, B*H < 2^31).
 */
#ifndef DITATTN_H
#define DITATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DIT_OK = 0,
  DIT_ERR_INVALID_ARG = 1,  /* bad pointer, size, alignment, aliasing or scale */
  DIT_ERR_UNSUPPORTED = 2,  /* valid request the kernels do not implement (e.g. D = 96) */
  DIT_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
  DIT_ERR_TIMEOUT = 4       /* a kernel's bounded wait expired (reported by dit_attn_check) */
} dit_status;

typedef enum { DIT_F32 = 0, DIT_BF16 = 1 } dit_dtype;

/* Opaque CUDA stream (cudaStream_t / CUstream). */
typedef void* dit_stream;

/* Element strides of a logical [B, H, N, D] view whose last dimension is
 * contiguous: with s = the strides, element (i_b, i_h, i_n, i_d) sits
 * i_b*s.b + i_h*s.h + i_n*s.n + i_d elements from the base.  Contiguous BHND
 * is {H*N*D, N*D, D}; the token-major BSND layout ([B, N, H, D] in memory) is
 * {N*H*D, D, H*D}. */
typedef struct {
  long long b, h, n;
} dit_strides;

/*
 * Fused attention over all N keys.
 * Defines: per head, s_ij = scale * q_i . k_j; o_i = sum_j softmax_j(s_ij) v_j;
 * every query sees every key (non-causal).  Pages: MindIE-SD parallelism docs,
 * "Ring Sequence Parallel" usage example (local attention = softmax of the
 * scaled scores times V); arganzheng.life multi-GPU diffusion parallelism,
 * section 4.1 Ulysses (full attention per head over all N tokens).
 *   q, k, v : device bf16 [B, H, N, D], contiguous, 16-byte aligned (read only)
 *   out     : device [B, H, N, D] of out_dtype (written)
 *   lse     : device fp32 [B, H, N] (written), or NULL when the caller needs only O:
 *             the pass then skips the LSE and its unrounded row sum (O is the same)
 *   scale   : score scale, usually 1/sqrt(D)
 */
dit_status dit_attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
                        int B, int H, int N, int D, float scale, dit_dtype out_dtype,
                        dit_stream stream);

/*
 * Attention of all N_q queries against ONE KV chunk: keys/values rows
 * [0, n_kv) starting at k, v (pass pointers already offset to the chunk's
 * first row).  This is one round of Ring attention: round i of rank r uses
 * the K/V block of rank (r + i) mod p, and after p rounds every query has
 * seen every key (arganzheng.life, section 4.2 Ring).
 *   q              : device bf16 [B, H, N_q, D], contiguous
 *   k, v           : device bf16; head (b*H + h) starts kv_head_stride
 *                    elements after the previous one, rows are D elements
 *                    apart.  N*D for a view into full [B,H,N,D] tensors,
 *                    n_kv*D for a packed chunk buffer as a ring hop would
 *                    receive it.  kv_head_stride must be >= n_kv*D and a
 *                    multiple of 8 (16-byte TMA stride).
 *   out_partial    : device [B, H, N_q, D] of partial_dtype: the softmax-
 *                    normalised output over this chunk's keys
 *   lse_partial    : device fp32 [B, H, N_q]: natural log-sum-exp over this chunk
 */
dit_status dit_attn_chunk_fwd(const void* q, const void* k, const void* v, void* out_partial,
                              float* lse_partial, int B, int H, int N_q, int n_kv, int D,
                              long long kv_head_stride, float scale, dit_dtype partial_dtype,
                              dit_stream stream);

/*
 * All virtual ranks of the ring decomposition in one launch: for each of p key
 * chunks c = [chunk_starts[c], chunk_starts[c+1]) of k / v, the partial output and
 * LSE of all N_q queries against that chunk alone, exactly as dit_attn_chunk_fwd
 * defines them (a Ring round's local attention on the block a rank holds;
 * arganzheng.life, section 4.2 Ring: one KV block per round, combined by online
 * softmax).  Bitwise equal to p dit_attn_chunk_fwd calls on the chunk views; one
 * persistent launch has no per-chunk launch gaps or tails.  dit_attn_lse_merge
 * then combines the partials.
 *   q, k, v, B, H, N_q, n_kv, D, kv_head_stride, scale : as dit_attn_chunk_fwd,
 *                  k / v holding all n_kv key rows
 *   partials     : device [p, B, H, N_q, D] of partial_dtype, contiguous, 16-byte
 *                  aligned (written)
 *   lses         : device fp32 [p, B, H, N_q], contiguous (written)
 *   p            : 1 .. 64
 *   chunk_starts : HOST array of p + 1 key-row offsets, 0 <= chunk_starts[0] <
 *                  chunk_starts[1] < ... < chunk_starts[p] <= n_kv (read before the
 *                  call returns; the chunks need not cover all keys)
 * partials and lses must not overlap each other or q, k, v (DIT_ERR_INVALID_ARG).
 */
dit_status dit_attn_chunks_fwd(const void* q, const void* k, const void* v, void* partials,
                               float* lses, int B, int H, int N_q, int n_kv, int D,
                               long long kv_head_stride, int p, const int* chunk_starts,
                               float scale, dit_dtype partial_dtype, dit_stream stream);

/*
 * General-layout form of dit_attn_fwd / dit_attn_chunk_fwd: attention of N_q
 * queries against n_kv keys, each of q, k, v and out an arbitrary strided
 * [B, H, N, D] view (last dimension contiguous).  This reads and writes the
 * token-major BSND layout in which the pages' sequence-parallel code keeps its
 * activations (the MindIE-SD parallelism docs run their attention kernel on
 * BSND tensors; valdrada.cn Wan2.2, CP section: tokens are split across ranks
 * and heads kept whole) directly, with no transpose.
 *   q, k, v     : device bf16 views; NULL strides = contiguous BHND
 *   out         : device view of out_dtype (written); NULL strides = contiguous
 *   lse         : device fp32 [B, H, N_q], contiguous (written), or NULL (no LSE,
 *                 as for dit_attn_fwd)
 * Strides must be positive multiples of 8 elements (16-byte TMA strides) below
 * 2^39; out must not map two elements to one address; out and lse must not
 * overlap the address range of q, k or v (DIT_ERR_INVALID_ARG otherwise).
 */
dit_status dit_attn_fwd_strided(const void* q, const dit_strides* q_strides, const void* k,
                                const dit_strides* k_strides, const void* v,
                                const dit_strides* v_strides, void* out,
                                const dit_strides* out_strides, float* lse, int B, int H, int N_q,
                                int n_kv, int D, float scale, dit_dtype out_dtype,
                                dit_stream stream);

/*
 * One Ring-attention hop with the merge fused into the chunk pass: the attention
 * of all N_q queries against ONE KV chunk, (O_c, lse_c) exactly as
 * dit_attn_chunk_fwd defines them, is merged in place into a running output:
 *   M = max(lse_run, lse_c);  lse' = M + ln(exp(lse_run - M) + exp(lse_c - M));
 *   O' = exp(lse_run - lse') O_run + exp(lse_c - lse') O_c
 * which is the online-softmax accumulation a Ring round performs on the block it
 * receives (arganzheng.life, section 4.2 Ring).  Applying it once per chunk of
 * the keys, in any order, gives the full attention.  No stacked partials and no
 * separate merge pass.
 *   q, k, v, B, H, N_q, n_kv, D, kv_head_stride, scale : as dit_attn_chunk_fwd
 *   o_run   : device fp32 [B, H, N_q, D], 16-byte aligned (read and written)
 *   lse_run : device fp32 [B, H, N_q], 4-byte aligned (read and written)
 * A row whose lse_run is -inf is empty: its o_run is never read (it may hold
 * anything, NaN included) and the row becomes this chunk's own attention.  So a
 * running state starts either as lse_run = -inf everywhere (o_run
 * uninitialised) or as the fp32 output of dit_attn_chunk_fwd for the first
 * chunk.  o_run and lse_run must not overlap each other or q, k, v
 * (DIT_ERR_INVALID_ARG).  Rows whose lse_run is +inf or NaN propagate NaN.
 */
dit_status dit_attn_chunk_fwd_accumulate(const void* q, const void* k, const void* v, float* o_run,
                                         float* lse_run, int B, int H, int N_q, int n_kv, int D,
                                         long long kv_head_stride, float scale, dit_stream stream);

/*
 * Split-KV form of dit_attn_chunk_fwd for problems with few queries (few
 * (head, Q pair) work items for the persistent grid, e.g. a stale-KV patch or a
 * short query block against long keys): every item is split over `splits`
 * contiguous ranges of the key tiles, computed in one launch into fp32 partials
 * in `workspace`, then merged exactly (the dit_attn_lse_merge combination) into
 * out / lse by a second launch.  Same result as dit_attn_chunk_fwd up to fp32
 * rounding of the merge.  The library allocates nothing: the caller passes the
 * workspace (device memory, 256-byte aligned, at least
 * dit_attn_splitkv_workspace_bytes(B, H, N_q, D, splits) bytes, overlapping no
 * other argument); it is scratch, overwritten by every call, so two calls in
 * flight at once must not share it.
 *   arguments as dit_attn_chunk_fwd (out contiguous, of out_dtype), plus
 *   splits : 1 (no split: workspace may be NULL) to min(64, ceil(n_kv / 128))
 */
dit_status dit_attn_chunk_fwd_splitkv(const void* q, const void* k, const void* v, void* out,
                                      float* lse, int B, int H, int N_q, int n_kv, int D,
                                      long long kv_head_stride, float scale, dit_dtype out_dtype,
                                      int splits, void* workspace, size_t workspace_bytes,
                                      dit_stream stream);

/*
 * dit_attn_chunk_fwd_splitkv without a caller workspace and without any device
 * allocation: the fp32 partials live in the library's own fixed device scratch
 * array of 128 MiB (set up once per device).  The pages have no counterpart; this
 * serves callers that must not allocate.  Requests whose partials need more than
 * 128 MiB (dit_attn_splitkv_workspace_bytes > 2^27) return DIT_ERR_UNSUPPORTED;
 * splits == 1 uses no scratch.  Nothing in the scratch needs clearing: the pass
 * writes every partial before the merge reads it.  There is one scratch array per
 * device: calls that overlap in time (other streams or host threads) race on it
 * and must be serialised by the caller.
 */
dit_status dit_attn_chunk_fwd_splitkv_noalloc(const void* q, const void* k, const void* v,
                                              void* out, float* lse, int B, int H, int N_q,
                                              int n_kv, int D, long long kv_head_stride,
                                              float scale, dit_dtype out_dtype, int splits,
                                              dit_stream stream);

/* Workspace bytes a split-KV call with these sizes needs (0 when splits <= 1 or a
 * size is not positive): splits * B*H*N_q * (D + 1) * 4, the LSE part 256-byte aligned. */
size_t dit_attn_splitkv_workspace_bytes(int B, int H, int N_q, int D, int splits);

/* A split count for an N_q x n_kv problem on the current device (1 to 16, at least two
 * key tiles per split): the one with the smallest estimated time, where the estimate is the
 * persistent grid's waves of (head, Q pair, key range) items times one item's KV tiles plus
 * a fixed per-item cost, plus (for splits > 1) the merge launch and its fp32 partial
 * traffic.  Never suggests a split the estimate puts behind no split.  Reads the device's SM
 * count; returns 1 if it cannot. */
int dit_attn_splitkv_suggest(int B, int H, int N_q, int n_kv);

/*
 * Exact merge of p chunk partials (O_c, lse_c) of the same queries:
 *   M = max_c lse_c;  lse = M + ln sum_c exp(lse_c - M);  O = sum_c exp(lse_c - lse) O_c
 * which is what the Ring section's online-softmax accumulation over the p
 * rounds computes (arganzheng.life, section 4.2 Ring).  A chunk whose lse is
 * -inf contributes nothing; a row whose lse_c are all -inf gets O = 0 and
 * lse = -inf.
 *   partials : device [p, B, H, N, D] of partial_dtype (chunk c at c*B*H*N*D)
 *   lses     : device fp32 [p, B, H, N]
 *   out      : device [B, H, N, D] of out_dtype;  lse: device fp32 [B, H, N]
 */
dit_status dit_attn_lse_merge(const void* partials, const float* lses, int p, void* out,
                              float* lse, int B, int H, int N, int D, dit_dtype partial_dtype,
                              dit_dtype out_dtype, dit_stream stream);

/*
 * Stale-KV attention of one patch, as displaced patch parallelism runs it
 * (PipeFusion / DistriFusion: arganzheng.life multi-GPU diffusion parallelism,
 * section 6 PipeFusion; xllm-io review of PipeFusion, method section; TACO-DiT,
 * hybrid SP KV buffer): a KV buffer holds K, V of all N tokens from the previous
 * diffusion step; the patch's freshly computed K, V rows [row0, row0 + m)
 * overwrite their stale rows in place, then the patch's m queries attend to the
 * whole buffer (their own rows fresh, every other row stale).  Launches on
 * `stream`: the row update (K and V together), then the attention, split over
 * `splits` key ranges plus a merge when splits > 1 (as dit_attn_chunk_fwd_splitkv:
 * a patch has few queries, so splitting its long key range fills the GPU).
 *   q            : device bf16 [B, H, m, D] (the patch's queries), contiguous
 *   k_new, v_new : device bf16 [B, H, m, D], contiguous (read)
 *   k_buf, v_buf : device bf16 [B, H, N, D], contiguous (rows [row0, row0+m)
 *                  overwritten, then read)
 *   out, lse     : as dit_attn_chunk_fwd for N_q = m queries over n_kv = N keys
 *   splits, workspace, workspace_bytes : as dit_attn_chunk_fwd_splitkv (1, NULL, 0: none)
 * 0 <= row0 <= N - m; the buffers must not overlap each other or q, k_new, v_new.
 */
dit_status dit_attn_stale_kv_fwd(const void* q, const void* k_new, const void* v_new, void* k_buf,
                                 void* v_buf, void* out, float* lse, int B, int H, int m, int N,
                                 int D, int row0, float scale, dit_dtype out_dtype, int splits,
                                 void* workspace, size_t workspace_bytes, dit_stream stream);

/*
 * Copies a logical [B, H, N, D] tensor of `dtype` elements from one strided
 * view to another (last dimension contiguous in both).  This is the local, on-GPU
 * half of Ulysses sequence parallelism's re-shard around attention, where an
 * all-to-all turns each rank's token shard of all heads into all tokens of its
 * head shard (arganzheng.life multi-GPU diffusion parallelism, section 4.1
 * Ulysses; valdrada.cn Wan2.2, CP section): the token-major (BSND) <-> head-major
 * (BHND) transpose and the packing of per-rank send buffers are such copies, and
 * so is writing fresh K/V rows into a KV buffer in place (a row-range view as dst).
 *   src, dst     : device pointers, 16-byte aligned; NULL strides = contiguous BHND
 *   D            : 64 or 128 (else DIT_ERR_UNSUPPORTED)
 * Strides follow dit_attn_fwd_strided's rules; dst must not map two elements to
 * one address and the two views' address ranges must not overlap
 * (DIT_ERR_INVALID_ARG).  Bit-exact: values are moved, never converted.
 */
dit_status dit_layout_copy(const void* src, const dit_strides* src_strides, void* dst,
                           const dit_strides* dst_strides, int B, int H, int N, int D,
                           dit_dtype dtype, dit_stream stream);

/*
 * Norms of queries and keys for each head and rotary positions, in one pass, before the attention or
 * before the cache (arganzheng.life multi-GPU diffusion parallelism, section 4.1 Ulysses: RoPE sliced with the
 * tokens).  The norm is of each head by itself; Wan's is over all heads of a token (valdrada.cn Wan2.2, TP section: its
 * sum of squares is reduced over the ranks that hold them) and is not computed here: such a model norms before this
 * call, which then turns alone (norm = 0).  For every head x of every token,
 *   z = w x / sqrt(mean_d x_d^2 + eps)                                            (norm; else z = x)
 * and pair i of the first 2 n channels, n the sum of axis_pairs, (2 i, 2 i + 1) where `interleaved`, else
 * (i, i + n), at the angle t = pos_a(i) * freqs[i],
 *   y_first = s (z_first cos t - z_second sin t),  y_second = s (z_first sin t + z_second cos t)
 * with s = rot_scale; the channels behind them are y = z.  In 32 bits, rounded to bf16 once; the angle
 * is taken modulo a turn exactly, whatever the position.  A sum of squares that overflows 32 bits makes its head 0 or NaN;
 * one of values all below 2^-62 loses digits or vanishes there, which an eps of 1e-30 or more hides.
 *   q, k          : device bf16 [B, H, N, D] views (read); NULL strides: contiguous.  A packed step's [T, H, D] is
 *                   B = 1, N = T.  k may be NULL (H_k = 0, no k_out, no k_weight): queries alone.
 *   q_out, k_out  : device bf16 views of the same shapes (written), of any layout (token-major in, head-major out):
 *                   each may be its input in place (the same view), and shares no element with anything else (views
 *                   may interleave, as slices of one allocation do: heads, halves of the tokens, a block for each b).
 *   norm          : 0 or 1; eps >= 0 (read with norm alone)
 *   q_weight, k_weight : device [D] of weight_dtype (read), or NULL (1); NULL without norm
 *   freqs         : device fp32 [n] (read): the angle of each pair per position, so that stretched and
 *                   scaled positions are a matter of the table; NULL (axes = 0): no rotation
 *   axis_pairs    : host int [axes]: pair i turns with the position axis a(i) in which it falls (a video's frame,
 *                   row and column); 1 axis: a token's index.  n a multiple of 8, 2 n <= D; axes <= 4
 *                   (more, or other n: DIT_ERR_UNSUPPORTED).
 *   positions     : device int32 (read): token (b, n) is at positions[b * pos_b + a * pos_axis + n] on axis a (pos_b = 0:
 *                   the same for every b); any value.  NULL: packed requests (B = 1, one axis),
 *   cu_new, start_lens, requests : device int32 [requests + 1], [requests] (read): token n of request r (dit_paged_plan's
 *                   cu_new) is at start_lens[r] + n - cu_new[r].  Tokens of no request are left as they are.
 *                   cu_new ascends (else its tokens' positions are unspecified).
 *   B * N         : at most 2^30;  requests : at most 2^20
 */
dit_status dit_qk_norm_rope(const void* q, const dit_strides* q_strides, void* q_out,
                            const dit_strides* q_out_strides, int H_q, const void* k,
                            const dit_strides* k_strides, void* k_out, const dit_strides* k_out_strides,
                            int H_k, int norm, float eps, const void* q_weight, const void* k_weight,
                            dit_dtype weight_dtype, const float* freqs, const int* axis_pairs, int axes,
                            int interleaved, float rot_scale, const int* positions, long long pos_b,
                            long long pos_axis, const int* cu_new, const int* start_lens, int requests, int B,
                            int N, int D, dit_stream stream);

/* ---------------------------------------------------------------------------
 * Paged key/value caches: requests of different and growing lengths in pages of
 * one pool, for generation with cached keys (text encoders and captioners of the pages'
 * pipelines, video generated block by block).  One step of a batch is
 *   dit_paged_plan         pages and slots for the step's new tokens, from lengths
 *   dit_qk_norm_rope       norms and positions of their queries and keys
 *   dit_paged_kv_write     their keys and values into the slots, page summaries
 *   dit_paged_prefill_fwd  any number of new tokens of each request against its pages, or
 *   dit_paged_select       (sparse attention only) the best pages for each query
 *   dit_paged_attn_fwd     one query token of each request against its pages
 *   dit_paged_page_mass    (caches with a budget) the weight that each page has drawn
 *   dit_paged_evict        ... and the pages that drew least back to the pool
 * All lengths, tables and slots live on the device, so that a step can be captured
 * into a graph once and replayed as the lengths grow.
 *
 *  - A cache is a pool of n_pages pages: a [n_pages, H_kv, page_size, D] bf16 view
 *    (dit_strides: b = page, h = head, n = row; NULL = contiguous).  page_size is a
 *    multiple of 16 from 16 to 1024.  A token's slot is page * page_size + row.
 *  - block_table: int32 [B, max_pages], rows table_stride >= max_pages entries apart;
 *    entry (b, i) is the page that holds tokens i * page_size .. of request b.
 *    max_pages * page_size < 2^31.  Entries past a request's length are never used.
 *    An entry outside [0, n_pages) is a page without keys: nothing is read for it.
 *  - seq_lens: int32 [B], the cached tokens of each request.  Values below 0 count as
 *    0 and values above max_pages * page_size as that.
 *  - Device contents cannot be refused; every value of the tables, lengths, slots and
 *    lists is safe (no access outside the buffers), and what an unusual one means is
 *    said at each call.
 *  - Workspaces are scratch: 256-byte aligned, need no clearing, overwritten by every
 *    call, and not to be shared by calls (or captured graphs) that can run at once.
 * ------------------------------------------------------------------------- */

/*
 * Block tables and slot maps of one step from the requests' lengths.  Request b holds
 * s_b = seq_lens[b] tokens in ceil(s_b / page_size) pages already in its table row and
 * appends n_b = max(0, new_lens[b]) tokens (0: an idle request).  The step's tokens are
 * packed in request order: request b's are rows cu_new[b] .. cu_new[b + 1] - 1 of the
 * step's batch.  Pages are granted in request order from the top of the free-page stack
 * (free_pages[n_free - 1] first) and written behind the request's pages in its table row;
 * no other table entry changes.  Pages come back by writing them at free_pages[n_free ..]
 * and raising n_free between steps.
 *   new_lens, seq_lens : device int32 [B] (read)
 *   block_table        : device int32 (read; granted entries written)
 *   free_pages, n_free : device int32 [pool_capacity] and [1] (read); n_free counts as
 *                        within [0, pool_capacity]
 *   seq_lens_out       : device int32 [B] (written): the lengths after the step; may be
 *                        seq_lens itself
 *   n_free_out         : device int32 [1] (written): pages left; may be n_free itself
 *   cu_new             : device int32 [B + 1] (written): prefix sums of n_b
 *   slots              : device int64 [max_tokens] (written): the slot of each token of
 *                        the batch, -1 for a token without one and behind the last token
 * A token has no slot where the stack has run out, where its request's table row is full,
 * or where its page's entry is outside [0, n_pages); tokens past max_tokens are dropped
 * (cu_new stops there).  seq_lens_out counts the tokens that fitted, so that
 * seq_lens_out[b] < s_b + n_b shows a request that ran out of pages.
 *   B : 1 .. 8192 (above: DIT_ERR_UNSUPPORTED);  max_tokens : 1 .. 2^30
 * Outputs must not overlap each other or the inputs, but for the two pairs named.
 */
dit_status dit_paged_plan(const int* new_lens, const int* seq_lens, int* block_table,
                          long long table_stride, const int* free_pages, const int* n_free,
                          int* seq_lens_out, int* n_free_out, int* cu_new, long long* slots, int B,
                          int max_pages, int page_size, int n_pages, int pool_capacity,
                          int max_tokens, dit_stream stream);

/*
 * Stores the keys and values of T tokens into their slots of the two caches, bit for bit.
 *   k_new, v_new  : device bf16 views [T, H, D] (read); token t, head h starts
 *                   t * s.n + h * s.h elements from the base (s.b is not used): slices of
 *                   a fused projection need no copy.  NULL strides: contiguous [T, H, D].
 *   slots         : device int64 [T]; a slot outside [0, n_pages * page_size) skips its
 *                   token, and rows without a token are left as they are
 *   k_cache, v_cache : paged caches (written); they may be interleaved in one allocation
 *                   ([n_pages, 2, H, page_size, D], [n_pages, page_size, 2, H, D] ..) where
 *                   their strides are equal and no element is shared
 *   summary       : device bf16 [n_pages, H, 2, D], contiguous, or NULL: for every page
 *                   and channel the minimum (index 0) and maximum (1) of its keys.  A page
 *                   whose row 0 is written starts anew from the rows of this call; any
 *                   other touched page is widened by them.  NaN keys make it NaN.
 *   T             : 1 .. 2^30
 * Slots are distinct, and with a summary the tokens of one page follow each other in
 * ascending slots, as dit_paged_plan lays them out.  (A slot that is repeated is
 * left with any mix of its tokens' 16-byte pieces, keys and values apart; it, and scattered rows of a page, leave
 * the page's summary unspecified.  Nothing else is touched.)
 */
dit_status dit_paged_kv_write(const void* k_new, const dit_strides* k_new_strides,
                              const void* v_new, const dit_strides* v_new_strides,
                              const long long* slots, void* k_cache,
                              const dit_strides* k_strides, void* v_cache,
                              const dit_strides* v_strides, void* summary, int T, int H, int D,
                              int page_size, int n_pages, dit_stream stream);

/*
 * Attention of one new token of each request over its cached keys: for query head h of
 * request b, with key/value head h / (H_q / H_kv),
 *   s_j = scale * q_bh . k_j;  out_bh = sum_j softmax_j(s_j) v_j;  lse_bh = ln sum_j exp(s_j)
 * over the seq_lens[b] first tokens (the new token's own key among them, once written).
 * A request without keys, or without one that scores above -inf, gets out = 0, lse = -inf.  A score
 * that is NaN or +inf in 32 bits makes its row NaN; a value that is not finite makes its channel of every
 * other row that sees it infinite or NaN (a weight of 0 does not hide it).  Sums of weights, up to 2^8 each,
 * times values are held in fp32 before the division: values past 2^120 / seq_lens[b] may overflow
 * there.  The keys' length is split over the GPU and the parts are joined exactly (the
 * dit_attn_lse_merge combination), in an order that the sizes and lengths alone fix: equal calls give
 * equal bits.
 *   q           : device bf16 [B, H_q, D] view (s.b, s.h; s.n is not used); NULL strides:
 *                 contiguous
 *   k_cache, v_cache, block_table, seq_lens : as above (read).  Rows past a request's
 *                 length may hold anything, NaN included.
 *   selected    : device int32 [B, H_kv, n_selected], contiguous, or NULL (all pages): only
 *                 the pages (table columns) listed for the key/value head take part, in
 *                 dit_paged_select's form: ceil(seq_lens[b] / page_size) entries are
 *                 looked at, at most n_selected.  An entry that is negative or past the
 *                 request's last page is skipped; one that is repeated counts repeatedly.
 *   out         : device [B, H_q, D] of out_dtype, contiguous, 16-byte aligned (written)
 *   lse         : device fp32 [B, H_q] (written), or NULL
 *   H_q         : a multiple of H_kv
 *   scale       : > 0, and finite times log2 e in 32 bits
 *   workspace   : at least dit_paged_attn_workspace_bytes(B, H_q, H_kv, D, page_size, pages) bytes,
 *                 pages = n_selected with `selected`, else max_pages; NULL where that is 0
 */
dit_status dit_paged_attn_fwd(const void* q, const dit_strides* q_strides, const void* k_cache,
                              const dit_strides* k_strides, const void* v_cache,
                              const dit_strides* v_strides, const int* block_table,
                              long long table_stride, const int* seq_lens, const int* selected,
                              int n_selected, void* out, float* lse, int B, int H_q, int H_kv,
                              int D, int page_size, int n_pages, int max_pages, float scale,
                              dit_dtype out_dtype, void* workspace, size_t workspace_bytes,
                              dit_stream stream);

/* Workspace bytes of a dit_paged_attn_fwd call with these sizes on the current device: 0 for
 * few requests with room for few keys (pages * page_size), which need none, and when a size is not positive. */
size_t dit_paged_attn_workspace_bytes(int B, int H_q, int H_kv, int D, int page_size, int pages);

/*
 * Attention of a step's new tokens over the cache: prompts, chunks of prompts, a block of video
 * tokens behind the blocks before it, a few candidate tokens of each request.  The step's tokens are
 * packed as dit_paged_plan packs them: request b's are the n_b rows cu_new[b] .. cu_new[b + 1] - 1 of q and
 * out, at the positions start_b, start_b + 1 ..., their own keys and values in the cache already.  For
 * query head h at position p, with key/value head h / (H_q / H_kv),
 *   s_j = scale * q . k_j;  out = sum_j softmax_j(s_j) v_j;  lse = ln sum_j exp(s_j)
 * over the cached keys j < seq_lens[b], with `causal` those j <= p.  A row that sees no key, or none that
 * scores above -inf, gets out = 0, lse = -inf.  A score that is NaN or +inf in 32 bits makes its row NaN; a
 * value that is not finite makes its channel of the rows that see it infinite or NaN (a weight of 0 does
 * not hide it), and of no other row.  Weights are rounded to bf16 (off by at most 2^-8 of each, and normalised
 * by the sum of the rounded ones), in fp32 output too; the lse is that of the unrounded ones.  Sums of weights,
 * up to 2^8 each, times values are held in fp32 before the division: values past 2^120 / seq_lens[b] may
 * overflow there.
 * Rows of q in front of cu_new[0] and from cu_new[B] on have no request: their rows of out and lse are left
 * as they are.  Work is split by the lengths on the device and joined in a fixed order: equal calls
 * give equal bits.
 *   q           : device bf16 view [T, H_q, D] (read); token t, head h starts t * s.n + h * s.h elements from
 *                 the base (s.b is not used).  NULL strides: contiguous.
 *   k_cache, v_cache, block_table, seq_lens : as above (read).  Rows past a request's length may hold
 *                 anything, NaN included.
 *   cu_new      : device int32 [B + 1], as dit_paged_plan writes it (read).  Entries count as within [0, T], and
 *                 a request whose entries descend has no tokens; rows that two requests claim are left with
 *                 either's values.
 *   start_lens  : device int32 [B] (read), or NULL: start_b = seq_lens[b] - n_b, the request's last tokens.
 *                 Give the lengths before the step where a request may have run out of pages: its tokens
 *                 without a slot then keep their positions and see the keys that were stored.
 *   out         : device [T, H_q, D] of out_dtype, contiguous, 16-byte aligned (written)
 *   lse         : device fp32 [T, H_q] (written), or NULL
 *   T           : 1 .. 2^30;  B : 1 .. 2^20;  H_q : a multiple of H_kv, at most 128 H_kv;
 *                 max_pages * page_size : at most 2^30 (above either of these two: DIT_ERR_UNSUPPORTED)
 *   causal      : 0 or 1
 *   scale       : > 0, and finite times log2 e in 32 bits
 *   workspace   : at least dit_paged_prefill_workspace_bytes(D, page_size, max_pages) bytes; NULL where that is 0
 */
dit_status dit_paged_prefill_fwd(const void* q, const dit_strides* q_strides, const void* k_cache,
                                 const dit_strides* k_strides, const void* v_cache,
                                 const dit_strides* v_strides, const int* block_table,
                                 long long table_stride, const int* seq_lens, const int* cu_new,
                                 const int* start_lens, void* out, float* lse, int T, int B, int H_q,
                                 int H_kv, int D, int page_size, int n_pages, int max_pages, int causal,
                                 float scale, dit_dtype out_dtype, void* workspace,
                                 size_t workspace_bytes, dit_stream stream);

/* Workspace bytes of a dit_paged_prefill_fwd call with these sizes on the current device: 0 for
 * requests with room for few keys (max_pages * page_size), which need none, and when a size is not positive. */
size_t dit_paged_prefill_workspace_bytes(int D, int page_size, int max_pages);

/*
 * The attention weight that each page has drawn, brought up to date by a step's queries: for every page of a
 * request with new tokens, and key/value head g,
 *   mass_out[page, g] = (0 where the page's first key is new, else mass[page, g])
 *                       + sum over the page's keys j, the observing tokens t that see them, the query heads h of g's
 *                         group: exp(scale * q_th . k_j - lse_th)
 * Observing are the last `window` new tokens of each request (0: all); they see keys as with `causal` in
 * dit_paged_prefill_fwd, whose lse this takes (dit_paged_attn_fwd's, of single tokens).  A row whose lse is -inf
 * adds nothing; a NaN lse, or score, makes the pages that the row sees NaN.  The lse is that of an attention over all of a
 * request's pages: behind one over selected pages the others' weights mean nothing.  Rows of no request are not
 * looked at.  Sums are in 32 bits, in an order that the sizes and lengths alone fix: equal calls give equal bits.
 *   q, k_cache, block_table, seq_lens, start_lens : as dit_paged_prefill_fwd (read)
 *   lse       : device fp32 [T, H_q] (read)
 *   cu_new    : device int32 [B + 1] (read), or NULL: one token of each request, its last (T = B; no start_lens)
 *   mass      : device fp32 [n_pages, H_kv], contiguous (read)
 *   mass_out  : device fp32 [n_pages, H_kv] (written: the pages of requests with new tokens alone); may be mass
 *               itself.  A page that is in the table more than once is left with any of its sums.  The weight that a
 *               page's former owner left is dropped by the call in the step in which the page's first key is new, and by
 *               nothing else: a program that does not call this in every step sets the weights of pages that were handed
 *               out in the others to 0 itself, or their requests inherit them.
 *   window    : >= 0;  T : 1 .. 2^30;  B : 1 .. 2^20;  H_q : a multiple of H_kv, at most 256 H_kv;
 *               max_pages * page_size : at most 2^30 (above either of these two: DIT_ERR_UNSUPPORTED)
 *   scale     : > 0, and finite times log2 e in 32 bits
 */
dit_status dit_paged_page_mass(const void* q, const dit_strides* q_strides, const float* lse, const void* k_cache,
                               const dit_strides* k_strides, const int* block_table, long long table_stride,
                               const int* seq_lens, const int* cu_new, const int* start_lens, const float* mass,
                               float* mass_out, int T, int B, int H_q, int H_kv, int D, int page_size,
                               int n_pages, int max_pages, int window, float scale, dit_stream stream);

/*
 * Eviction: a request of n > keep pages, n = ceil(seq_lens[b] / page_size), keeps its newest `recent` pages and,
 * of the others, the keep - recent that drew most weight over all heads (sum_g mass[page, g] in 64 bits; equal ones:
 * the lower index; NaN above every number, an entry outside the pool below).  The kept ones close up in order, so that
 * keys keep their order and the newest page stays the last; entries keep .. n - 1 of the table row become -1 and those
 * behind are as they were; the length falls by (n - keep) * page_size.  The freed pages go onto the stack of free pages by
 * request and column; what does not fit into it is dropped.  Other requests keep theirs.  Positions that keys were
 * turned by (dit_qk_norm_rope) stay: a program counts them apart from the lengths (its start_lens).
 * Every page is in one request's row, once: one that others hold too would go to the stack while they use it.
 *   mass        : device fp32 [n_pages, H_kv], contiguous (read)
 *   block_table : device int32 (read); table_out: device int32 [B, max_pages], rows table_out_stride apart
 *                 (written), may be block_table itself (the same stride)
 *   seq_lens, n_free, seq_lens_out, n_free_out : as dit_paged_plan
 *   free_pages  : device int32 [pool_capacity] (entries from n_free on are written)
 *   keep        : >= 1;  recent : 1 .. keep;  B : 1 .. 8192 (above: DIT_ERR_UNSUPPORTED)
 *   workspace   : at least dit_paged_evict_workspace_bytes(B, max_pages) bytes
 * Outputs must not overlap each other or the inputs, but for the three pairs named; rows of block_table and
 * table_out may lie in turn in one allocation.
 */
dit_status dit_paged_evict(const float* mass, const int* block_table, long long table_stride, int* table_out,
                           long long table_out_stride, const int* seq_lens, int* seq_lens_out, int* free_pages,
                           const int* n_free, int* n_free_out, int B, int H_kv, int page_size, int n_pages,
                           int max_pages, int pool_capacity, int keep, int recent, void* workspace,
                           size_t workspace_bytes, dit_stream stream);

/* Workspace bytes of a dit_paged_evict call with these sizes; 0 when a size is not positive. */
size_t dit_paged_evict_workspace_bytes(int B, int max_pages);

/*
 * The pages whose keys can score highest, for attention over those alone.  For request b
 * and key/value head g the score of page i is
 *   max over the query heads h of the group of  sum_d max(q_hd * lo_d, q_hd * hi_d)
 * with (lo, hi) the page's summary: no key of the page has a larger q . k.  Listed are the
 * request's newest page and the top_k - 1 others with the highest scores (all pages where
 * there are no more than top_k); equal scores go to the lower index, and a NaN score counts
 * as +inf.  The choice is that of the scores in 64 bits.
 *   q, block_table, seq_lens : as dit_paged_attn_fwd
 *   summary  : device bf16 [n_pages, H_kv, 2, D], contiguous, as dit_paged_kv_write keeps it.
 *              A page without keys (its entry outside [0, n_pages)) scores -inf.
 *   selected : device int32 [B, H_kv, top_k], contiguous (written): table columns in
 *              ascending order, then -1
 *   top_k    : 1 .. max_pages
 *   workspace: at least dit_paged_select_workspace_bytes(B, H_kv, max_pages) bytes; NULL where
 *              that is 0
 */
dit_status dit_paged_select(const void* q, const dit_strides* q_strides, const void* summary,
                            const int* block_table, long long table_stride, const int* seq_lens,
                            int* selected, int B, int H_q, int H_kv, int D, int page_size,
                            int n_pages, int max_pages, int top_k, void* workspace,
                            size_t workspace_bytes, dit_stream stream);

/* Workspace bytes of a dit_paged_select call with these sizes on the current device: 0 for few
 * requests with room for few pages, which need none, and when a size is not positive. */
size_t dit_paged_select_workspace_bytes(int B, int H_kv, int max_pages);

/*
 * Synchronises `stream`, then reads and clears the library's device status
 * word.  Returns DIT_ERR_TIMEOUT if any kernel since the last check gave up
 * on a bounded wait, DIT_ERR_CUDA if the synchronisation failed, else DIT_OK.
 */
dit_status dit_attn_check(dit_stream stream);

/*
 * TEST ONLY: failure injection for the timeout path.  While `enable` is
 * non-zero, attention launches from this process load Q but never issue the
 * K/V copies, so the MMA warp's bounded wait on the first K tile expires
 * after `wait_limit_cycles` SM clocks (<= 0 keeps the default of about two
 * seconds); the kernel then records DIT_ERR_TIMEOUT in the status word and
 * exits cleanly, and dit_attn_check() reports it.  Nothing faults or hangs.
 * dit_paged_attn_fwd, dit_paged_prefill_fwd and dit_paged_page_mass (of more than 16 rows) withhold their copies and
 * report in the same way.
 * Call with enable = 0 to restore normal operation.  Not thread-safe with
 * concurrent launches from other host threads.
 */
void dit_test_inject_stall(int enable, long long wait_limit_cycles);

/*
 * TEST ONLY: caps the number of CTAs of the persistent attention kernel
 * (normally one per SM; max_ctas <= 0 restores that).  With a small cap every
 * CTA walks many work items, which exercises the cross-item pipeline on small
 * inputs.  Affects later launches from this process; results do not change.
 * dit_paged_attn_fwd takes the cap too and, while one is set, deals its work
 * out over the capped grid at any size (its results change by the rounding of
 * the joins).
 */
void dit_test_set_grid_limit(int max_ctas);

/* Static, human-readable name of a status code. */
const char* dit_status_string(dit_status s);

/* Library version: major * 10000 + minor * 100 + patch. */
int dit_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DITATTN_H */
