/*
 * csa2.h - C ABI of the GB300 (sm_103a) CSA2 index + sparse-attention step.
 *
 * The step (one query per decode request, or many queries sharing one cache):
 *   1. csa2_quantize_append  - KV append: RoPE then FP4 (E2M1, one E4M3 scale
 *                              per 16 channels) for the main latent; FP4 for
 *                              indexer K/Q rows; FP8 E4M3 for window latents.
 *   2. csa2_index_full       - Full layer: score every visible entry, keep the
 *                              top pool blocks of 8 by block maximum, and pick
 *                              the top-k positions.
 *   3. csa2_index_reindex    - Reindex layer: re-score only the pool's
 *                              positions with this layer's own indexer query.
 *      (csa2_index_full_bf16 / csa2_index_reindex_bf16 take the indexer
 *      query as bf16 and quantize it themselves, saving its FP4 append.)
 *      (Reuse layers make no call: they pass the previous top-k buffer again.)
 *   4. csa2_sparse_attn      - 64-head attention over the selected FP4 latents
 *                              plus the FP8 sliding window, one merged softmax.
 *
 * Sources, four secondary web pages about DeepSeek-V4.1-Flash:
 *   [T1] "DeepSeek V4.1-Flash 为什么这么强？CED 与 CSA2 架构全拆解"
 *   [T2] the blog post "DeepSeek V4.1 Flash vs V4 Pro"
 *   [T3] "DeepSeek-V4.1-Flash：全局 KV 仅 890 B/token，百万上下文怎么做成的？"
 * The pages fix formats, shapes and modes but no formula; the score, the
 * rounding and every memory layout below are this library's definitions.
 *
 * Conventions for every call:
 *   - All data pointers are DEVICE pointers owned by the caller; the library
 *     allocates nothing.  Data pointers must be 16-byte aligned.
 *   - Calls are asynchronous and stream-ordered on `stream` (a cudaStream_t;
 *     NULL is the legacy default stream).
 *   - Argument errors are detected on the host and return before any launch
 *     (CSA2_ERR_INVALID_ARG / CSA2_ERR_UNSUPPORTED / CSA2_ERR_WORKSPACE).  A
 *     launch failure returns CSA2_ERR_CUDA.
 *   - Values only the device can see (rows, positions, indices held in device
 *     arrays) are checked by the kernels: an offending item is skipped and the
 *     first problem is recorded in the status word at the start of `ws`
 *     (read it with csa2_status_fetch).  No kernel traps or asserts.
 *   - `ws` is caller-provided scratch of csa2_workspace_bytes(...) bytes.  Its
 *     first 256 bytes hold the status word; zero them once with
 *     csa2_status_reset.  Calls sharing one `ws` must be stream-ordered.
 */
#ifndef CSA2_H
#define CSA2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int csa2_status;
enum {
    CSA2_OK = 0,
    CSA2_ERR_INVALID_ARG = 1,   /* null pointer, misalignment, bad size      */
    CSA2_ERR_UNSUPPORTED = 2,   /* a shape or format this library does not run */
    CSA2_ERR_CUDA = 3,          /* a CUDA launch or runtime error             */
    CSA2_ERR_TIMEOUT = 4,       /* device: a bounded wait gave up             */
    CSA2_ERR_DEVICE_BOUNDS = 5, /* device: a row/index outside its bounds was skipped */
    CSA2_ERR_WORKSPACE = 6      /* ws smaller than csa2_workspace_bytes()     */
};

/* Shapes fixed by the pages ([T1] §二, layout paragraph; [T1] 层级化稀疏索引器). */
#define CSA2_INDEX_HEADS 32   /* indexer query heads                        */
#define CSA2_INDEX_DIM 128    /* indexer head dim                           */
#define CSA2_ATTN_HEADS 64    /* main attention heads                       */
#define CSA2_LATENT_DIM 512   /* shared main latent (K = V)                 */
#define CSA2_BLOCK 8          /* positions per pool block                   */
#define CSA2_STATUS_BYTES 256 /* status area at the start of every ws       */
#define CSA2_TREE_NODES 1024  /* nodes of a request's tree                  */
#define CSA2_LOGPROBS_TOP 64  /* alternatives, and given tokens, of a row   */

/* Formats and layouts for csa2_quantize_append. */
enum { CSA2_FMT_FP4 = 0, CSA2_FMT_FP8 = 1 };
/*
 * CSA2_LAYOUT_ROWS: FP4 codes row-major, codes[row][dim/2] (two codes per
 *   byte, even channel in the low nibble), scales[row][dim/16] (E4M3 bytes).
 *   FP8: bytes[row][dim].  Used for the main latent and the window latents.
 * CSA2_LAYOUT_BLOCK8 (FP4, dim 128 only): rows in blocks of 8; the 64 code
 *   bytes of row r sit at byte (r/8)*512 + c*128 + (r%8)*16 + j for byte
 *   b = 16c + j of the row (c = 0..3).  Scales stay row-major [row][8].  Used
 *   for indexer K and indexer Q: a block of 8 rows is 512 contiguous bytes
 *   holding four 8-row x 16-byte tiles, the shape tensor cores read.
 * CSA2_LAYOUT_BLOCK8R (FP4, dim 128 only): BLOCK8 with each block's scales
 *   beside its codes: block b of 8 rows is a 576-byte record at byte 576*b,
 *   its 512 code bytes as in BLOCK8 followed by the 8 rows x 8 scale bytes
 *   (row r's scale byte g at 576*(r/8) + 512 + (r%8)*8 + g).  dst_scales
 *   must be NULL.  Used for indexer K: a block the index gathers is then one
 *   contiguous read instead of two.
 */
enum { CSA2_LAYOUT_ROWS = 0, CSA2_LAYOUT_BLOCK8 = 1, CSA2_LAYOUT_BLOCK8R = 2 };

/* Output element type of csa2_sparse_attn. */
enum { CSA2_OUT_BF16 = 0, CSA2_OUT_F32 = 1 };

/* Operation ids for csa2_workspace_bytes. */
enum { CSA2_OP_APPEND = 0, CSA2_OP_INDEX_FULL = 1, CSA2_OP_INDEX_REINDEX = 2, CSA2_OP_SPARSE_ATTN = 3 };

typedef void* csa2_stream_t; /* a cudaStream_t */

/* ABI version (increments on any signature change). */
int csa2_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* csa2_status_string(csa2_status status);

/*
 * Bytes of workspace an operation needs for n_q queries whose visible entry
 * counts are at most max_visible, with pool_blocks pool blocks and topk
 * selections.  Always >= CSA2_STATUS_BYTES.  Returns 0 for bad arguments.
 */
size_t csa2_workspace_bytes(int op, int64_t n_q, int32_t max_visible, int pool_blocks, int topk);

/* Zero the status word of `ws` (stream-ordered). */
csa2_status csa2_status_reset(void* ws, csa2_stream_t stream);

/*
 * Copy the status area to host out[4] = {status, detail0, detail1, detail2}
 * and synchronize `stream`.  out[0] is CSA2_OK or the first device-detected
 * problem (CSA2_ERR_DEVICE_BOUNDS: detail0 = which check, detail1 = the query
 * or row, detail2 = the offending value).
 */
csa2_status csa2_status_fetch(const void* ws, int32_t out[4], csa2_stream_t stream);

/*
 * RoPE tables.  [T1] §三 and [T3] 第三刀: the main latent is quantized after
 * RoPE.  Rotation of channel pair (2i, 2i+1) by p * theta^(-2i/dim), p the
 * 0-based position; the angle is split as p = hi*1024 + lo and the table
 * holds cos/sin of hi*1024*w_i and lo*w_i (computed in fp64, stored fp32),
 * combined on the device by angle addition.  The table covers positions
 * [0, max_pos).  csa2_rope_table_init fills a caller-allocated device buffer
 * of csa2_rope_table_bytes(dim, max_pos) bytes.
 */
size_t csa2_rope_table_bytes(int dim, int64_t max_pos);
csa2_status csa2_rope_table_init(float theta, int dim, int64_t max_pos, void* table,
                                 csa2_stream_t stream);

/*
 * KV append ([T1] §三; [T2] 黑科技之三; [T3] 第三刀).
 *   x_bf16     [n][dim] bf16 rows to append.
 *   fmt        CSA2_FMT_FP4: per group of 16 channels s = RNE_E4M3(amax/6)
 *              (saturating at 448), codes = nearest E2M1 of x/s, ties to the
 *              even code, saturating at 6, sign kept; s == 0 gives zero codes.
 *              CSA2_FMT_FP8: each element to E4M3 (nearest-even, saturating).
 *   layout     CSA2_LAYOUT_ROWS, or CSA2_LAYOUT_BLOCK8 / CSA2_LAYOUT_BLOCK8R
 *              (FP4, dim 128).
 *   dim        512 or 128 (FP4 and FP8 rows; BLOCK8 needs 128).
 *   pos        [n] int64 RoPE positions, or NULL for no RoPE.  Needs
 *              rope_table from csa2_rope_table_init for the same dim, covering
 *              rope_max_pos positions; a position outside [0, rope_max_pos)
 *              skips the row and records CSA2_ERR_DEVICE_BOUNDS.
 *   dst_row    [n] int64 destination rows, or NULL for rows 0..n-1.  A row
 *              outside [0, n_rows) is skipped and recorded.
 *   dst_codes  codes plane of n_rows rows (FP4), or the FP8 byte plane.
 *   dst_scales scales plane [n_rows][dim/16] (FP4), NULL for FP8 and for
 *              CSA2_LAYOUT_BLOCK8R (the scales sit in the records).
 *   n_rows     rows in the destination planes (BLOCK8: a multiple of 8).
 *   ws         at least CSA2_STATUS_BYTES bytes (status word).
 */
csa2_status csa2_quantize_append(const void* x_bf16, int64_t n, int dim, int fmt, int layout,
                                 const int64_t* pos, const void* rope_table, int64_t rope_max_pos,
                                 const int64_t* dst_row, int64_t n_rows,
                                 uint8_t* dst_codes, uint8_t* dst_scales,
                                 void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * Full-layer hierarchical index ([T1] §二 mode table and 层级化稀疏索引器;
 * [T3] 第二刀, Fig. 5).  For query t with n = n_visible[t] entries at cache
 * rows kv_start[t] .. kv_start[t]+n-1:
 *   I(t,s) = sum_h w[t][h] * max(0, q~[t][h] . k~[s])  for s < n,
 * q~, k~ the dequantized FP4 indexer query and key.  Block b covers positions
 * [8b, 8b+8) (a partial last block uses its visible positions).
 *   out_pool[t][pool_blocks]: the top-min(pool_blocks, ceil(n/8)) blocks by
 *     block maximum, ties to the lower block, ascending, padded with -1.
 *   out_topk[t][topk]: the top-min(topk, n) positions by I over ALL visible
 *     positions, ties to the lower position, ascending, padded with -1.
 *     (Computed exactly by re-scoring the top-max(pool_blocks, topk) blocks,
 *     which contain every top-k position.)
 *   q_codes/q_scales: indexer Q, BLOCK8 layout, n_q*32 rows of 128 channels
 *     (row t*32+h is head h of query t).  w: [n_q][32] fp32.
 *   k_codes/k_scales: indexer K plane, n_rows rows: BLOCK8 codes and
 *     row-major scales, or (k_scales NULL) BLOCK8R records in k_codes.
 *   kv_start [n_q] int64 (multiples of 8), n_visible [n_q] int32, device.
 *   max_visible: host upper bound of n_visible (sizes the launch).
 *   pool_blocks in [1, 4096], topk in [1, 2048].
 * Checked on the device: kv_start % 8 == 0, 0 <= n_visible <= max_visible
 * and kv_start + n_visible <= n_rows; a failing query gets empty (-1) outputs.
 */
csa2_status csa2_index_full(const uint8_t* q_codes, const uint8_t* q_scales, const float* w,
                            int64_t n_q, const uint8_t* k_codes, const uint8_t* k_scales,
                            int64_t n_rows, const int64_t* kv_start, const int32_t* n_visible,
                            int32_t max_visible, int pool_blocks, int topk,
                            int32_t* out_pool, int32_t* out_topk,
                            void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * Reindex layer ([T1] §二 mode table; [T2] 黑科技之二; [T3] 第二刀): the same
 * score with this layer's own q, w against the shared indexer K, over the
 * positions of `pool` (a Full layer's out_pool, [n_q][pool_blocks], -1 pads
 * ignored) only; out_topk[t][topk] = the top-min(topk, |pool positions|)
 * positions, ties to the lower position, ascending, padded with -1.
 * Other arguments as in csa2_index_full.  A pool entry outside
 * [0, ceil(n/8)) is skipped and recorded.
 */
csa2_status csa2_index_reindex(const uint8_t* q_codes, const uint8_t* q_scales, const float* w,
                               int64_t n_q, const uint8_t* k_codes, const uint8_t* k_scales,
                               int64_t n_rows, const int64_t* kv_start, const int32_t* n_visible,
                               int32_t max_visible, const int32_t* pool, int pool_blocks, int topk,
                               int32_t* out_topk, void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * csa2_index_full and csa2_index_reindex with the indexer query given as
 * bf16 rows, q_bf16 [n_q*32][128] (row t*32+h is head h of query t, 16-byte
 * aligned), instead of FP4 codes and scales.  The query is quantized to FP4
 * (E2M1, one E4M3 scale per 16 channels; [T1] 层级化稀疏索引器, [T3] 第二刀:
 * the indexer runs in FP4) inside the call, exactly as csa2_quantize_append
 * with CSA2_FMT_FP4 would, so the results are those of the FP4 calls on that
 * quantization.  Decode batches (fewer than 256 queries) and every Reindex
 * call quantize it in the scoring kernels' prologue, which saves the
 * separate quantization launch; a many-query Full call quantizes it into
 * its workspace first (the workspace size is the same as the FP4 call's).
 * Other arguments, results and errors as in the FP4 calls.
 */
csa2_status csa2_index_full_bf16(const void* q_bf16, const float* w, int64_t n_q, const uint8_t* k_codes,
                                 const uint8_t* k_scales, int64_t n_rows, const int64_t* kv_start,
                                 const int32_t* n_visible, int32_t max_visible, int pool_blocks, int topk,
                                 int32_t* out_pool, int32_t* out_topk, void* ws, size_t ws_bytes,
                                 csa2_stream_t stream);
csa2_status csa2_index_reindex_bf16(const void* q_bf16, const float* w, int64_t n_q, const uint8_t* k_codes,
                                    const uint8_t* k_scales, int64_t n_rows, const int64_t* kv_start,
                                    const int32_t* n_visible, int32_t max_visible, const int32_t* pool,
                                    int pool_blocks, int topk, int32_t* out_topk, void* ws, size_t ws_bytes,
                                    csa2_stream_t stream);

/*
 * csa2_index_reindex without a workspace, for callers that cannot allocate
 * device memory: runtimes without a device allocator, callers whose memory
 * is fixed before the model starts, or code running where cudaMalloc is not
 * permitted.  The pages describe nothing like it; it exists only for such
 * callers.  Arguments and results are those of csa2_index_reindex, except:
 *   - the per-position scores go to one library-owned device array of 2 MiB
 *     (held by every GPU that loads the library until the process exits):
 *     n_q * 8 * pool_blocks must be at most 524,288, else the call returns
 *     CSA2_ERR_UNSUPPORTED without launching (e.g. 32 queries at 2048 pool
 *     blocks);
 *   - status: a caller-owned device int32[4] that receives the first
 *     device-detected problem (as the status word of a workspace), or NULL.
 *     It is not cleared by the call.
 * The first call on a device looks up the array's device address (one
 * runtime query); make that first call before any stream capture.  Every
 * call shares the array, whose contents are fully rewritten by each call;
 * calls that overlap on the GPU (other streams, other threads) race on it.
 * The call allocates nothing.
 */
csa2_status csa2_index_reindex_noalloc(const uint8_t* q_codes, const uint8_t* q_scales,
                                       const float* w, int64_t n_q, const uint8_t* k_codes,
                                       const uint8_t* k_scales, int64_t n_rows,
                                       const int64_t* kv_start, const int32_t* n_visible,
                                       int32_t max_visible, const int32_t* pool, int pool_blocks,
                                       int topk, int32_t* out_topk, int32_t* status,
                                       csa2_stream_t stream);

/*
 * Sparse attention with one merged softmax ([T1] §二: 64 heads over a
 * 512-dim latent, every layer has its own Q and window KV; [T3] 第三刀: FP4
 * main KV dequantized before attention, window kept in FP8).  For query t,
 * head h, with E = {selected entries} U {window entries} (no dedup):
 *   l_j = sm_scale * q[t][h] . c_j,  p = softmax over E,  o[t][h] = sum p_j c_j
 * where selected entry j is main-KV row kv_start[t] + topk[t][j] (FP4,
 * dequantized; -1 pads skipped) and the window is the last min(window, n)
 * positions p of the query, read from swa[t][p mod window] (E4M3).
 *   q_bf16   [n_q][64][512] bf16.
 *   kv_codes [n_rows][256], kv_scales [n_rows][32]: main latent, ROWS layout.
 *   topk     [n_q][k] int32 positions (a Full/Reindex layer's out_topk).
 *   swa      [n_q][window][512] E4M3 ring (slot = position mod window).
 *   swa_new_bf16  [n_q][512] bf16 window latent of each query's current
 *            token (position n-1), or NULL.  When given, the kernel rounds it
 *            to E4M3 exactly as csa2_quantize_append (CSA2_FMT_FP8) would,
 *            stores it to ring slot (n-1) mod window and uses it: the
 *            window append fused into the attention call.
 *   window   0..128.
 *   out      [n_q][64][512], bf16 (out_dtype CSA2_OUT_BF16) or fp32
 *            (CSA2_OUT_F32); the result is rounded once, from fp32.  bf16's
 *            unit roundoff is 2^-8, so the fp32 form carries the kernels'
 *            own accuracy (about 1e-6 relative).
 *   out_lse  [n_q][64] fp32 natural-log log-sum-exp of the scaled logits,
 *            or NULL.
 * An empty E gives zeros and lse = -inf.  A topk entry outside [-1, n) is
 * skipped and recorded.
 */
csa2_status csa2_sparse_attn(const void* q_bf16, int64_t n_q,
                             const uint8_t* kv_codes, const uint8_t* kv_scales, int64_t n_rows,
                             const int64_t* kv_start, const int32_t* n_visible,
                             const int32_t* topk, int k, uint8_t* swa, const void* swa_new_bf16,
                             int window, float sm_scale, void* out, int out_dtype, float* out_lse,
                             void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * Prefill sparse attention over a shared sequence ([T1] §二 layout paragraph:
 * the encoder runs CSA2 at m = 2 in groups of one Full and five Reuse
 * layers, over a prefill chunk of many query tokens).  As csa2_sparse_attn,
 * except that each query's window is its own causal window over the
 * sequence the queries share: the last min(window, n) positions p < n of
 * query t, read from
 *   swa_rows [n_rows][512] E4M3, row kv_start[t] + p
 * (the same row numbering as the main latent; one array per layer, written
 * with csa2_quantize_append CSA2_FMT_FP8), instead of a ring per query.
 * There is no current-token append.  The workspace is that of
 * csa2_sparse_attn (CSA2_OP_SPARSE_ATTN).
 */
csa2_status csa2_sparse_attn_prefill(const void* q_bf16, int64_t n_q,
                                     const uint8_t* kv_codes, const uint8_t* kv_scales, int64_t n_rows,
                                     const int64_t* kv_start, const int32_t* n_visible,
                                     const int32_t* topk, int k, const uint8_t* swa_rows, int window,
                                     float sm_scale, void* out, int out_dtype, float* out_lse,
                                     void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * ---- A layer's step over a paged cache ----
 *
 * The next calls run a step in which every request brings a chunk of new
 * tokens (one for a decoding request) and keeps its latents in pages: page p
 * holds rows p*page_size .. p*page_size + page_size - 1 of a latent plane,
 * and position i of request r is row table[r][i / page_size] * page_size +
 * i % page_size.  In order:
 *   csa2_rmsnorm_fp8      residual, norm and E4M3 activations
 *   csa2_fp4_matvec       queries and latents of a few tokens, FP4 weights
 *   csa2_page_plan        pages, rows and positions of the new tokens
 *   csa2_quantize_append  with the plan's rows (dst_row) and positions (pos)
 *   csa2_paged_attn       the new tokens over everything their request holds
 * Tokens are packed: request r owns tokens q_start[r] .. q_start[r+1] - 1.
 */

/* Activations of csa2_fp4_matvec. */
enum { CSA2_X_BF16 = 0, CSA2_X_E4M3 = 1 };

/*
 * Block tables and slot maps of a step, from the requests' lengths.
 * Request r holds cached[r] entries in the first held = ceil(cached[r] /
 * page_size) pages of its table row and brings added[r] new ones.  It takes
 * need = ceil((cached[r] + added[r]) / page_size) - held pages off the end of
 * the free list, requests in order: with o the pages that earlier requests
 * take, table[r][held + j] = free_pages[n_free - 1 - (o + j)], j < need.
 *   cached, added [n_req] int32.
 *   page_size     a multiple of 8, 8..65536.
 *   table         [n_req][max_pages] int32, in place: only the new pages'
 *                 entries are written.
 *   free_pages    [n_pages] int32, the free pages' ids; n_free int32[1], how
 *                 many of them are.  n_pages: the cache's pages.
 *   n_free_out    int32[1]: n_free minus the pages taken (may be n_free).
 *   q_start       [n_req + 1] int32 out: exclusive sums of added.
 *   kv_len        [n_req] int32 out: cached + added (not cached itself).
 *   slots, pos    [max_new] int64 out: destination row and position of each
 *                 new token, request after request; -1 behind the last one.
 * A call that cannot be served takes nothing: where a length is negative, a
 * request does not fit its table row, the new tokens exceed max_new or the
 * pages n_free, the table stays as it is, n_free_out = n_free, q_start and
 * kv_len are 0, slots and pos are -1, and the first problem is recorded in
 * ws.  A page id outside [0, n_pages) gives slots of -1 and is recorded (a
 * new page's table entry is then -1).  ws: CSA2_STATUS_BYTES bytes, zeroed
 * once with csa2_status_reset.
 */
csa2_status csa2_page_plan(const int32_t* cached, const int32_t* added, int64_t n_req, int page_size,
                           int32_t* table, int64_t max_pages, const int32_t* free_pages, int64_t n_pages,
                           const int32_t* n_free, int32_t* n_free_out, int32_t* q_start, int32_t* kv_len,
                           int64_t* slots, int64_t* pos, int64_t max_new, void* ws, size_t ws_bytes,
                           csa2_stream_t stream);

/*
 * Causal attention of each request's new tokens over its paged latents (keys
 * and values are the same 512-wide latent, shared by the heads).  Token i of
 * request r sits at position t = kv_len[r] - (q_start[r+1] - q_start[r]) + i
 * and sees positions max(0, t + 1 - window) .. t (window 0: all up to t):
 *   l_p = sm_scale * q . c_p,  o = sum softmax(l)_p c_p.
 *   q_bf16   [n_tokens][n_heads][512] bf16; n_heads 1..128, n_tokens up to
 *            2^22, n_req up to 2^20.
 *   q_start  [n_req + 1] int32, kv_len [n_req] int32 (csa2_page_plan's).
 *   max_q, max_kv: host upper bounds of a request's tokens and entries
 *            (max_kv up to 2^30).
 *   fmt      CSA2_FMT_FP4: codes [n_rows][256] and scales [n_rows][32], as
 *            csa2_quantize_append writes them (CSA2_LAYOUT_ROWS);
 *            CSA2_FMT_FP8: codes are E4M3 rows [n_rows][512], scales NULL.
 *   table    [n_req][max_pages] int32; page_size a multiple of 8, 8..65536.
 *   out      [n_tokens][n_heads][512] bf16, rounded once from fp32 sums (the
 *            probabilities enter the product in f16); apart from q_bf16.
 *   out_lse  [n_tokens][n_heads] fp32, natural log-sum-exp of the scaled
 *            logits, or NULL.
 * A token that sees nothing gets zeros and lse = -inf.  Tokens from
 * q_start[n_req] on are left as they are.  A request whose kv_len lies
 * outside [0, min(max_kv, max_pages * page_size)] is recorded and sees
 * nothing; one whose tokens lie outside [0, n_tokens) or exceed max_q is
 * recorded and skipped; a table entry outside [0, n_rows / page_size) is
 * recorded and its page is not seen.  (Where n_tokens, n_req or max_q is 0
 * nothing is launched, and nothing recorded.)  Latents that no token sees may hold
 * anything, NaN included.
 * The same call gives the same bits every time; the keys are split by the
 * lengths of all requests, so an output's last bits can depend on the others.
 * ws: csa2_paged_attn_workspace_bytes (0 for bad sizes) for the same sizes.
 */
size_t csa2_paged_attn_workspace_bytes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q,
                                       int32_t max_kv, int window);
csa2_status csa2_paged_attn(const void* q_bf16, int64_t n_tokens, int n_heads, const int32_t* q_start,
                            const int32_t* kv_len, int64_t n_req, int32_t max_q, int32_t max_kv, int fmt,
                            const uint8_t* codes, const uint8_t* scales, int64_t n_rows, const int32_t* table,
                            int64_t max_pages, int page_size, int window, float sm_scale, void* out,
                            float* out_lse, void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * Residual addition, root-mean-square norm and E4M3 output:
 *   h = bf16(x + residual)  (h = x without a residual)
 *   y = h / sqrt(mean(h^2) + eps) * weight            (fp32)
 *   s = max|y| / 448 over the row (group 0) or each 128 channels (group 128)
 *   codes = nearest-even E4M3 of y / s (0 where s is 0), both unrounded
 *   x            [n] rows of dim bf16, x_stride elements apart (>= dim, a
 *                multiple of 8).
 *   residual     [n][dim] bf16 or NULL; residual_out [n][dim] takes h (may be
 *                residual itself; needed with a residual, else NULL).
 *   weight       [dim] bf16.  dim: a multiple of 8, 8..16384 (group 128: a
 *                multiple of 128).  eps >= 0, finite.
 *   codes        [n][dim] E4M3; scales [n] or [n][dim/128] fp32.
 *   y_bf16       [n][dim] bf16 of y, or NULL.
 * The mean is an fp32 sum: |h| up to 2^56 (where eps is 0, rows of 2^-60 and
 * more).  A NaN or infinite h makes the codes and the scale of the row's
 * groups what the formula gives (NaN).
 */
csa2_status csa2_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual, void* residual_out,
                             const void* weight, int64_t n, int dim, float eps, int group, uint8_t* codes,
                             float* scales, void* y_bf16, csa2_stream_t stream);

/*
 * Products of a few rows with FP4 weights: out[i][j] = alpha * sum_c x[i][c]
 * W[j][c].
 *   x            [n] rows of k elements, x_stride elements apart (>= k, a
 *                multiple of 16): bf16 (x_fmt CSA2_X_BF16, x_scales NULL), or
 *                E4M3 with one fp32 scale per row, x_scales [n] (CSA2_X_E4M3;
 *                csa2_rmsnorm_fp8 with group 0 gives both).
 *   codes, scales  W: n_out rows of k channels, [n_out][k/2] E2M1 codes and
 *                [n_out][k/16] E4M3 scales: csa2_quantize_append of the
 *                weights in CSA2_LAYOUT_ROWS, as n_out*k/128 rows of 128.
 *   k            a multiple of 128, up to 65536.  n rows: up to 65536; the
 *                weights are read once for each 16 rows.
 *   out          [n][n_out], bf16 (CSA2_OUT_BF16) or fp32 (CSA2_OUT_F32);
 *                apart from x.  Sums and alpha times them are fp32.
 * ws: csa2_fp4_matvec_workspace_bytes(n, k, n_out) bytes (0 for bad sizes).
 */
size_t csa2_fp4_matvec_workspace_bytes(int64_t n, int k, int64_t n_out);
csa2_status csa2_fp4_matvec(const void* x, int x_fmt, const float* x_scales, int64_t x_stride, int64_t n, int k,
                            const uint8_t* codes, const uint8_t* scales, int64_t n_out, float alpha, void* out,
                            int out_dtype, void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * Norms of every head's query and of the latents, turned by their positions
 * and stored, in one pass:
 *   y = x / sqrt(mean(x^2) + eps) * weight  (without a weight: y = x), then
 *   pairs (2i, 2i+1) turned by pos * theta^(-2i/512) where a table is given.
 *   q_bf16       [n] rows of n_heads x 512, q_stride elements apart (>=
 *                n_heads * 512, a multiple of 8); n_heads 1..128; n up to 2^22.
 *   q_weight     [512] bf16, of every head; NULL: no norm.
 *   q_out        [n][n_heads][512] bf16, rounded once from fp32; q_bf16 itself
 *                where its rows stand close together, or apart from it.
 *   latents      [n] rows of 512 bf16, lat_stride elements apart; lat_weight as
 *                q_weight.  They go to cache rows dst_row[i] (NULL: row i) of
 *                dst_codes / dst_scales in CSA2_LAYOUT_ROWS, in the form `fmt`
 *                (see csa2_quantize_append): nearest codes of y in 64-bit
 *                arithmetic.  A group of 16 with NaN or infinity gets a scale
 *                of NaN (FP4); E4M3 keeps NaN and takes infinities to 448.
 *   pos          [n] int64, or NULL without a table.  rope_table as in
 *                csa2_quantize_append (theta and positions are the table's), or
 *                NULL: nothing is turned.
 *   Queries or latents may be NULL (with their weight and outputs): only the
 *   other ones are done then.
 * A token of position -1 (behind a padded step's last one) is left out, its
 * q_out and cache row stay as they are; so does a latent of dst_row -1.  Other
 * positions outside [0, rope_max_pos) (below 0 without a table) and rows outside
 * [0, n_rows) are left out and recorded.  Sums of squares are fp32: |x| up to
 * 2^56, and where eps is 0 rows of 2^-60 and more (a row of zeros stays one).
 * What is written lies apart from what is read.  ws: CSA2_STATUS_BYTES bytes.
 */
csa2_status csa2_head_norm_rope(const void* q_bf16, int64_t q_stride, int n_heads, const void* q_weight, void* q_out,
                                const void* latents, int64_t lat_stride, const void* lat_weight, int64_t n, float eps,
                                const int64_t* pos, const void* rope_table, int64_t rope_max_pos, int fmt,
                                const int64_t* dst_row, int64_t n_rows, uint8_t* dst_codes, uint8_t* dst_scales, void* ws,
                                size_t ws_bytes, csa2_stream_t stream);

/*
 * ---- Steps whose new tokens are trees of drafted ones ----
 *
 * A request's tokens of the step are the nodes of a tree, in an order that puts
 * a parent before its children: parent[q_start[r] + i] is the place of node i's
 * parent among the request's nodes (below i), or -1 for one that continues the
 * cached entries.  (A chain, parent i - 1, is an ordinary chunk.)  Node i's
 * latent is entry kv_len - nodes + i of its request, csa2_page_plan's slot; its
 * position is that of the first node plus its depth:
 *   csa2_page_plan, csa2_tree_plan   slots; positions and masks
 *   csa2_head_norm_rope or csa2_quantize_append   by those positions
 *   csa2_tree_attn                   in every layer
 *   csa2_token_logprobs              the model's choice after every node
 *   csa2_tree_commit                 what was accepted stays
 * Requests bring up to 1024 nodes.
 *
 * csa2_tree_plan:
 *   parent       [n_tokens] int32; q_start, kv_len as csa2_page_plan gives them;
 *                max_q: host upper bound of a request's nodes (up to 1024).
 *   pos          [n_tokens] int64 out: kv_len - nodes + depth.
 *   mask         [n_tokens][mask_words] 32-bit words out, mask_words =
 *                ceil(max_q / 32): bit j of node i's row (word j / 32, bit j %
 *                32) is set where j is i or an ancestor of it and, with a window,
 *                lies fewer than `window` levels above it.
 * A node whose parent is none of the earlier ones is recorded; it and what
 * descends from it get pos = -1 and an empty mask, and see nothing.  A request
 * whose kv_len is below its nodes is recorded, and all its nodes get that; one
 * whose tokens lie outside [0, n_tokens) or exceed max_q is recorded and skipped.
 * Tokens behind q_start[n_req] are left as they are.  What is written lies apart
 * from what is read.  ws: CSA2_STATUS_BYTES.
 */
csa2_status csa2_tree_plan(const int32_t* parent, const int32_t* q_start, const int32_t* kv_len, int64_t n_req,
                           int64_t n_tokens, int32_t max_q, int window, int64_t* pos, uint32_t* mask, int mask_words,
                           void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * csa2_paged_attn for trees: node i of request r sees
 *   - the entries before the request's nodes, p < kv_len - nodes, with a window
 *     those of max(0, pos + 1 - window) <= p, and
 *   - the request's nodes whose bits its mask row has.
 * pos and mask are csa2_tree_plan's for the same window; a node of pos below 0
 * sees nothing.  (With other masks: bits at and behind the nodes' number, and
 * above the node's own, are to be 0.  A pos above kv_len - nodes + i counts as
 * that, one below kv_len - nodes as the first node's.)  What is written lies
 * apart from what is read and from each other.  Everything else, max_q up to 1024
 * apart, is as in csa2_paged_attn (the keys are split in other places than there).
 * ws: csa2_tree_attn_workspace_bytes (0 for bad sizes) for the same sizes.
 */
size_t csa2_tree_attn_workspace_bytes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q, int32_t max_kv,
                                      int window);
csa2_status csa2_tree_attn(const void* q_bf16, int64_t n_tokens, int n_heads, const int32_t* q_start,
                           const int32_t* kv_len, int64_t n_req, int32_t max_q, int32_t max_kv, const int64_t* pos,
                           const uint32_t* mask, int mask_words, int fmt, const uint8_t* codes, const uint8_t* scales,
                           int64_t n_rows, const int32_t* table, int64_t max_pages, int page_size, int window,
                           float sm_scale, void* out, float* out_lse, void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * Rows of logits x: with m = max x, y = (x - m) * scale and S = sum e^y,
 *   lse = m * scale + log S, entropy = log S - sum(e^y y) / S,
 *   log probability of token t: y_t - log S.
 *   logits       [n] rows of vocab elements, stride elements apart (>= vocab;
 *                rows, the first one too, may begin at any element), bf16 (dtype
 *                CSA2_OUT_BF16) or fp32 (CSA2_OUT_F32).  vocab 1..2^21, n up to
 *                2^24.
 *   scale        of the logits (one over a temperature), 2^-20..2^20.
 *   tokens       [n][given] int64 (8-byte aligned), given 0..64; logprobs
 *                [n][given] fp32 out.  A token of -1 is none: -inf.  Others
 *                outside [0, vocab) give -inf and are recorded.
 *   lse, entropy [n] fp32 out, or NULL.
 *   top          0..64 alternatives: ids [n][top] int32 and best [n][top] fp32 out,
 *                the tokens of the largest logits and their log probabilities,
 *                largest first, equal logits by the lower token.  A logit of -inf
 *                is no alternative: behind the last one ids are -1, best -inf.
 * A row of -inf alone: lse and log probabilities -inf, entropy 0.  A row with NaN
 * or +infinity: NaN, and ids -1.  Sums are fp32.  The outputs lie apart from the
 * logits.  ws: CSA2_STATUS_BYTES bytes.
 */
csa2_status csa2_token_logprobs(const void* logits, int dtype, int64_t stride, int64_t n, int64_t vocab, float scale,
                                const int64_t* tokens, int given, float* logprobs, float* lse, float* entropy, int top,
                                int32_t* ids, float* best, void* ws, size_t ws_bytes, csa2_stream_t stream);

/*
 * The commit of a step of trees.  From each request's node 0 (whose parent is to
 * be -1; it is the token that was sure before the step) the path goes on to the
 * child whose token is the choice at its parent, the lowest of several, as long
 * as there is one.
 *   token        [n_tokens] int64, the nodes' tokens; choice [n_tokens] int64, what
 *                the model goes on with after each node (its first alternative, or
 *                a sample).
 *   parent, q_start, kv_len, max_q: as in csa2_tree_plan.  (parent, token, choice
 *                and path may be NULL where n_tokens is 0: accepted and next are
 *                those of requests without nodes then.)
 *   codes, scales  the cache's planes (n_rows rows in the form fmt), or codes and
 *                scales NULL: no rows are moved.  The row of the path's j-th node
 *                goes to the request's entry kv_len - nodes + j.
 *   table        [n_req][max_pages] int32.  Pages that hold none of the kept
 *                entries go back to the end of free_pages [n_pages], in the order
 *                that undoes csa2_page_plan's taking; their table entries stay.
 *                n_free int32[1], n_free_out int32[1] (may be n_free).
 *   cached       [n_req] int32 out: kv_len - nodes + accepted; left as it is where
 *                a request has no nodes.
 *   path         [n_tokens] int32 out: at q_start[r] + j the place of the path's
 *                j-th node among the request's nodes, -1 behind the last one.
 *   accepted     [n_req] int32 out: nodes of the path (0 without nodes).
 *   next         [n_req] int64 out: the choice at the path's last node, the token
 *                that the next step begins with; -1 where there is none.
 * A request with bad bounds (as in csa2_tree_plan, or a kv_len beyond its table
 * row) is recorded and keeps nothing of the step: accepted 0, no rows moved, no
 * pages back, cached as it was.  A node with a bad parent is recorded and
 * accepted never; without a first node of parent -1 nothing is accepted.  A page
 * outside the cache is recorded, and its rows are not moved, or it does not go
 * back; where the free list has no room, that is recorded and nothing goes back.
 * The step is done once: again on the same planes it would move rows that have
 * moved.  Path entries behind q_start[n_req] are left as they are.  What is written
 * lies apart from what is read (n_free_out apart).  ws: CSA2_STATUS_BYTES bytes,
 * zeroed once with csa2_status_reset.
 */
csa2_status csa2_tree_commit(const int32_t* parent, const int64_t* token, const int64_t* choice, const int32_t* q_start,
                             const int32_t* kv_len, int64_t n_req, int64_t n_tokens, int32_t max_q, int fmt, uint8_t* codes,
                             uint8_t* scales, int64_t n_rows, const int32_t* table, int64_t max_pages, int page_size,
                             int32_t* free_pages, int64_t n_pages, const int32_t* n_free, int32_t* n_free_out,
                             int32_t* cached, int32_t* path, int32_t* accepted, int64_t* next, void* ws, size_t ws_bytes,
                             csa2_stream_t stream);

/*
 * Instrumentation (off by default; the compute path never depends on it).
 * csa2_launch_count: kernels launched through the library by this process.
 * csa2_timer_enable: bracket the next max_launches launches of kernel
 *   `kernel_id` (0 scan_blockmax, 1 select_blocks, 2 pool_score,
 *   3 select_topk, 4 attn_split (either attention kernel), 5 attn_merge, 6 quantize_fp4,
 *   7 quantize_fp8, 8 rope_table, 9 page_plan, 10 paged_attn, 11 paged_merge,
 *   12 rmsnorm_fp8, 13 fp4_matvec, 14 paged_decode, 15 head_norm_rope, 16 tree_plan,
 *   17 token_logprobs, 18 tree_commit) with CUDA events on their stream.  Not for
 *   use during stream capture.
 * csa2_timer_read: wait for those events, return the summed device time and
 *   the number of launches timed, and switch the timer off.
 */
int64_t csa2_launch_count(void);

/*
 * Test hook for the device give-up paths.  Every wait of a library kernel on
 * a barrier (copies arriving, MMAs completing) is bounded: after 2 s it
 * records CSA2_ERR_TIMEOUT in the status word, stops issuing work, waits for
 * the copies and MMAs it already started, and returns.  csa2_debug_wait_limit
 * sets that limit (in nanoseconds) for kernels launched afterwards, on every
 * device (it is a launch argument: a graph captured earlier keeps the limit
 * it was captured with); 0 restores 2 s.  A limit under 1 ms makes every
 * bounded wait give up at once, so a test can check the status, that the
 * copies and MMAs in flight were waited for, and that the next normal call
 * is correct.  Not for production use and not during stream capture.
 */
csa2_status csa2_debug_wait_limit(int64_t ns);
const char* csa2_kernel_name(int kernel_id);
csa2_status csa2_timer_enable(int kernel_id, int max_launches);
csa2_status csa2_timer_read(int kernel_id, double* total_ms, int32_t* launches);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_H */
