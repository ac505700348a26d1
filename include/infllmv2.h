/*
 * infllmv2.h -- C ABI of libinfllmv2.so: InfLLM v2 trainable block-sparse
 * attention (semantic-kernel pooling, block scoring, top-k block selection,
 * block-sparse flash attention) for NVIDIA GB300 (sm_103a).
 *
 * The method, as the pages describe it:
 *   [MiniCPM4-1.1]  "MiniCPM4: 如何在手机电脑上高效运行大语言模型"
 *                   (xugj520.cn), section 1.1 "InfLLM v2" -- context split into
 *                   blocks; overlapping semantic kernels of 32 tokens, stride
 *                   16; each query keeps its top-K most relevant blocks; the
 *                   opening tokens and the sliding window are always kept;
 *                   attention runs on the kept blocks only; kernel-level
 *                   relevance avoids token-level work; a uint64-packed mask
 *                   supports tree-speculative decoding.
 *   [MiniCPM4.0-sparse] "MiniCPM40极速狂飙端侧模型的比赛结束了"
 *                   (shadowrocket9.top), section "InfLLM v2：重新定义注意力
 *                   机制" -- 64-token blocks, top-64 blocks, dense attention
 *                   below 8192 tokens; its deployment guide sets
 *                   sparse_config = {topk, block_size, dense_len}.
 *   [CPM.cu]        "CPM.cu：端侧大模型推理的 CUDA 加速引擎" (pomoai.com),
 *                   section 4 -- static memory (preallocated KV cache),
 *                   CUDA graphs, chunked prefill.
 * The pages disagree on block size (64 vs 128) and top-k (64 vs 6), so every
 * method parameter is a runtime argument (infllmv2_params).
 *
 * Conventions for every entry point
 *   - Tensors are plain device pointers, row-major, densely packed, 16-byte
 *     aligned (infllmv2_decode_host also takes host buffers, as its comment
 *     says).  bf16 tensors are passed as void*.  Index/length arrays are
 *     device int32.  The caller owns every buffer and the stream; the library
 *     never allocates device memory (the static-memory design of [CPM.cu]).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     All work is enqueued on it; calls return before the GPU finishes.
 *   - Argument errors are found on the host and returned before anything is
 *     enqueued.  Errors only the device can see (a kv_len out of range, a
 *     selected block past the query's own block, a wait that ran out) set a
 *     device error word; infllmv2_sync_status() reports and clears it.
 *   - Supported: bf16 Q/K/V; head_dim d in {64, 128}; query heads per KV head
 *     G = Hq/Hkv in {1, 2, 4, 8, 16}; block_size in {64, 128}; kernel_size and
 *     kernel_stride positive with kernel_size <= block_size; n_local_blocks >= 1;
 *     at most 64 draft tokens (one uint64 mask word each).
 *
 * Layouts (B = batch, Tq = queries per sequence, Hq/Hkv = query/KV heads)
 *   q            [B, Tq, Hq, d]        bf16; heads g*G .. g*G+G-1 share KV head g
 *   k_cache      [B, Hkv, L_max, d]    bf16; token x of a sequence is row x
 *   v_cache      [B, Hkv, L_max, d]    bf16
 *   kernel_cache [B, Hkv, M_max, d]    bf16; kernel j = mean of tokens
 *                                      [j*stride, j*stride + kernel_size)
 *   kv_len       [B]                   int32; tokens in the cache, including
 *                                      the tokens of this call
 *   o            [B, Tq, Hq, d]        bf16
 *   lse          [B, Hq, Tq]           fp32, natural-log sum of exp(scale*q.k)
 *   idx          [B, Hkv, Tq, S_max]   int32 selected block ids, ascending,
 *                                      padded with -1
 *   counts       [B, Hkv, Tq]          int32 number of valid entries in idx
 */
#ifndef INFLLMV2_H_
#define INFLLMV2_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Method parameters ([MiniCPM4-1.1]; sparse_config of [MiniCPM4.0-sparse]). */
typedef struct infllmv2_params {
    int32_t block_size;      /* tokens per KV block: 64 or 128                        */
    int32_t kernel_size;     /* tokens per semantic kernel (the pages: 32)            */
    int32_t kernel_stride;   /* token stride between kernels (the pages: 16)          */
    int32_t topk;            /* blocks chosen by score, on top of the forced ones     */
    int32_t n_init_blocks;   /* leading blocks always kept ("opening tokens")         */
    int32_t n_local_blocks;  /* blocks ending at the query's own block, always kept   */
    int32_t dense_len;       /* sequences with kv_len < dense_len attend densely      */
    float softmax_scale;     /* 0 selects 1/sqrt(d)                                   */
} infllmv2_params;

typedef enum infllmv2_status {
    INFLLMV2_OK = 0,
    INFLLMV2_ERR_INVALID_ARG = -1,     /* null/misaligned pointer, bad size or range   */
    INFLLMV2_ERR_UNSUPPORTED = -2,     /* d, G, block size ... outside the set above   */
    INFLLMV2_ERR_WORKSPACE = -3,       /* workspace missing or smaller than required   */
    INFLLMV2_ERR_CUDA = -4,            /* a CUDA runtime call failed (launch, ...)     */
    INFLLMV2_ERR_DEVICE_TIMEOUT = -5,  /* a bounded device-side wait ran out           */
    INFLLMV2_ERR_DEVICE_INDEX = -6,    /* device saw kv_len or a block id out of range */
    INFLLMV2_ERR_NOT_IMPLEMENTED = -7
} infllmv2_status;

/* Entry ids for infllmv2_workspace_size. */
enum {
    INFLLMV2_ENTRY_BLOCK_SELECT = 1,
    INFLLMV2_ENTRY_SPARSE_ATTN_FWD = 2,
    INFLLMV2_ENTRY_DECODE = 3,
    INFLLMV2_ENTRY_SPARSE_ATTN_BWD = 4,
    INFLLMV2_ENTRY_NORM_ROPE_BWD = 5
};

/* Human-readable text of a status code (static storage, never NULL). */
const char* infllmv2_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int infllmv2_version(void);

/*
 * Synchronise `stream`, then report and clear the device error word of the
 * current device.  Returns INFLLMV2_OK, INFLLMV2_ERR_DEVICE_TIMEOUT,
 * INFLLMV2_ERR_DEVICE_INDEX or INFLLMV2_ERR_CUDA.
 */
int infllmv2_sync_status(void* stream);

/*
 * Most selected blocks any query can get for these parameters and an L_max-token
 * cache: topk + n_init + n_local, or every causal block while kv_len < dense_len
 * (whichever is larger, capped at ceil(L_max/block_size)).  idx buffers need at
 * least this many columns (S_max).  Returns -1 on invalid parameters.
 */
int infllmv2_selection_capacity(const infllmv2_params* params, int L_max);

/*
 * Bytes of device workspace an entry point needs (entry = INFLLMV2_ENTRY_*).
 * Tq is the number of queries per sequence (n_draft for decode).  Returns 0
 * for invalid arguments (and for entries that need none).  For
 * INFLLMV2_ENTRY_NORM_ROPE_BWD only d is read (params may be NULL).
 */
size_t infllmv2_workspace_size(int entry, int B, int Tq, int Hq, int Hkv, int d, int L_max,
                               const infllmv2_params* params);

/*
 * Step 1, semantic kernels ([MiniCPM4-1.1], semantic-kernel item):
 *   kernel_cache[b,g,j,:] = bf16_rne( (1/kernel_size) * sum of k_cache[b,g,x,:]
 *                           over x in [j*stride, j*stride + kernel_size) )
 * for every kernel j whose last token lies in [tok_begin, tok_end) -- that is,
 * the kernels that become complete once tokens [tok_begin, tok_end) are in the
 * cache.  Call it after appending tokens (a prefill chunk, or each decode token;
 * a new kernel completes every `stride` tokens).  Sums are exact -- integer
 * fixed-point sums of the bf16 inputs under a shared per-column exponent -- and
 * the mean is rounded to bf16 once, nearest-even.
 * (Terms more than 2^40 below a column's largest lose their bits below that.)  A
 * column with infinities of one sign has that infinity as its mean; with both, or
 * with a NaN, its mean is NaN.
 * Requires 0 <= tok_begin <= tok_end <= L_max and
 * M_max >= (tok_end - kernel_size)/kernel_stride + 1.  Other kernels are untouched.
 */
int infllmv2_kernel_pool(const void* k_cache, void* kernel_cache, int B, int Hkv, int L_max,
                         int M_max, int d, int tok_begin, int tok_end,
                         const infllmv2_params* params, void* stream);

/*
 * Variable-length batched prefill ([CPM.cu] section 4 chunked prefill, many
 * sequences with different chunk lengths in one launch).  Sequence b's chunk is
 * len_b = cu_q[b+1] - cu_q[b] queries: the last len_b tokens of its cache, so
 * query t sits at position kv_len[b] - len_b + t.  Packed layouts (total_q =
 * cu_q[B] query rows; cu_q is device int32 [B+1], ascending, cu_q[0] = 0):
 *   q, o     [total_q, Hq, d]       row cu_q[b] + t
 *   idx      [Hkv, total_q, S_max]  counts [Hkv, total_q]
 *   lse      [Hq, total_q]
 * Tq_max (host) bounds every len_b; total_q (host) is cu_q[B].  A len_b outside
 * [0, Tq_max] or a kv_len[b] < len_b sets the device error word and skips that
 * sequence.  Each varlen call computes exactly what its fixed-chunk counterpart
 * computes for every sequence on its own.
 *
 * infllmv2_kernel_pool_varlen: the kernels completed by each sequence's chunk
 * (step 1, as infllmv2_kernel_pool per sequence).
 */
int infllmv2_kernel_pool_varlen(const void* k_cache, void* kernel_cache, const int32_t* kv_len,
                                const int32_t* cu_q, int B, int Hkv, int L_max, int M_max, int d,
                                int Tq_max, const infllmv2_params* params, void* stream);

/* Steps 2-3 for packed chunks (as infllmv2_block_select per sequence).  Requires
 * ws_bytes >= infllmv2_workspace_size(INFLLMV2_ENTRY_BLOCK_SELECT, 1, total_q, ...). */
int infllmv2_block_select_varlen(const void* q, const void* kernel_cache, const int32_t* kv_len,
                                 const int32_t* cu_q, int B, int Tq_max, int total_q, int Hq,
                                 int Hkv, int d, int L_max, int M_max, int32_t* idx,
                                 int32_t* counts, int S_max, void* workspace, size_t ws_bytes,
                                 const infllmv2_params* params, void* stream);

/* Step 4 for packed chunks (as infllmv2_sparse_attn_fwd per sequence); idx NULL:
 * dense causal attention. */
int infllmv2_sparse_attn_fwd_varlen(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* idx, const int32_t* counts, int S_max,
                                    const int32_t* kv_len, const int32_t* cu_q, int B, int Tq_max,
                                    int total_q, int Hq, int Hkv, int d, int L_max, void* o,
                                    float* lse, const infllmv2_params* params, void* stream);

/*
 * Decode-step append (the per-token cache update of [CPM.cu] section 4, static
 * preallocated caches, together with step 1's pooling; one launch, so a CUDA
 * graph of infllmv2_append + infllmv2_decode is one whole decode step).
 * For every sequence b and KV head g, with p = kv_len[b] - 1 (kv_len counts the
 * new token):
 *   k_cache[b,g,p,:] = k_new[b,g,:];  v_cache[b,g,p,:] = v_new[b,g,:]
 * and, if the new token is the last token of semantic kernel
 *   j = (kv_len[b] - kernel_size) / kernel_stride   (kv_len[b] >= kernel_size and
 *   kv_len[b] - kernel_size divisible by kernel_stride),
 * kernel_cache[b,g,j,:] is computed exactly as infllmv2_kernel_pool does.
 *   k_new, v_new  [B, Hkv, d] bf16, read only.
 *   kv_len        [B] device int32, per sequence (read on the device).
 * kernel_cache may be NULL only when M_max == 0.  Device errors (kv_len[b] < 1 or
 * > L_max, a kernel index >= M_max) set the error word; that row is skipped.
 * Cache rows other than p and kernels other than j are untouched.
 */
int infllmv2_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                    void* kernel_cache, const int32_t* kv_len, int B, int Hkv, int d,
                    int L_max, int M_max, const infllmv2_params* params, void* stream);

/*
 * Steps 2-3, block scores and top-k selection for a causal chunk
 * ([MiniCPM4-1.1] dynamic block selection and local retention;
 * [MiniCPM4.0-sparse] dense switch).  Query t of sequence b sits at position
 * p = kv_len[b] - Tq + t (the chunk is the last Tq tokens of the cache; Tq = 1
 * is single-token decode).  With bt = p / block_size:
 *   S[t,g,blk] = max over heads h of group g and over kernels j that share a
 *                token with blk and end at or before p, of q[t,h] . kernel[j]
 *   forced     = blocks [0, n_init) and [bt - n_local + 1, bt], within [0, bt]
 *   selected   = forced + the topk other blocks <= bt by (S desc, id asc);
 *                every block <= bt when kv_len[b] < dense_len.
 * Writes idx [B,Hkv,Tq,S_max] (ascending, -1 padded) and counts [B,Hkv,Tq].
 * Needs S_max >= infllmv2_selection_capacity(params, L_max), kernels pooled up
 * to kv_len[b], kv_len[b] in [Tq, L_max], and
 * ws_bytes >= infllmv2_workspace_size(INFLLMV2_ENTRY_BLOCK_SELECT, ...).
 * Once the call's work is done, the workspace starts with the scores S as float
 * [B, Hkv, Tq, ceil(L_max / block_size)]: entries of blocks 0..bt of each query
 * of a sequence with kv_len[b] >= dense_len are written, the others are
 * unspecified; they stay there until the workspace is used again.
 */
int infllmv2_block_select(const void* q, const void* kernel_cache, const int32_t* kv_len, int B,
                          int Tq, int Hq, int Hkv, int d, int L_max, int M_max, int32_t* idx,
                          int32_t* counts, int S_max, void* workspace, size_t ws_bytes,
                          const infllmv2_params* params, void* stream);

/*
 * Step 4, block-sparse attention for a causal chunk ([MiniCPM4-1.1], attention
 * on the selected blocks only; chunked prefill of [CPM.cu]).  For query t of
 * sequence b at p = kv_len[b] - Tq + t and head h of group g:
 *   keys = tokens x <= p of the blocks idx[b,g,t,0..counts-1]
 *   o    = softmax_x(scale * q.k_x) v_x    (fp32 online softmax, bf16 output)
 * idx == NULL (and counts == NULL) means dense causal attention (every block).
 * lse may be NULL.  Selected ids must lie in [0, bt] (checked on the device).
 * Requires ws_bytes >= infllmv2_workspace_size(INFLLMV2_ENTRY_SPARSE_ATTN_FWD, ...).
 */
int infllmv2_sparse_attn_fwd(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* idx, const int32_t* counts, int S_max,
                             const int32_t* kv_len, int B, int Tq, int Hq, int Hkv, int d,
                             int L_max, void* o, float* lse, void* workspace, size_t ws_bytes,
                             const infllmv2_params* params, void* stream);

/*
 * Gradients of step 4 for a causal chunk with the selection held fixed (InfLLM
 * v2 is trainable sparse attention, [MiniCPM4-1.1]; the block choice is
 * discrete, so the gradient flows through the attention over the selected
 * keys).  Inputs as for infllmv2_sparse_attn_fwd, plus that call's output o
 * and lse (required here) and dout [B, Tq, Hq, d] bf16.  With P the weights of
 * a row and D = dout . o:
 *   dS = P o (dout v^T - D);  dq = scale dS k;  dk = scale dS^T q;  dv = P^T dout
 * dq [B, Tq, Hq, d] and dk, dv [B, Hkv, L_max, d] are fp32 and overwritten (dk,
 * dv are summed over the heads of a group and over the chunk's rows; cache rows
 * no row attends to get 0).  idx == NULL: dense causal, as in the forward.
 * Requires ws_bytes >= infllmv2_workspace_size(INFLLMV2_ENTRY_SPARSE_ATTN_BWD, ...).
 */
int infllmv2_sparse_attn_bwd(const void* q, const void* k_cache, const void* v_cache, const void* o,
                             const float* lse, const void* dout, const int32_t* idx,
                             const int32_t* counts, int S_max, const int32_t* kv_len, int B, int Tq,
                             int Hq, int Hkv, int d, int L_max, float* dq, float* dk, float* dv,
                             void* workspace, size_t ws_bytes, const infllmv2_params* params,
                             void* stream);

/*
 * Steps 2-4 for decoding: selection from the cached kernels, split-KV
 * attention over the selected blocks, and the merge of the splits.
 *   tree_mask == NULL: single-token decode (n_draft must be 1); the query is
 *     the newest cached token, p = kv_len[b] - 1.
 *   tree_mask != NULL: tree-speculative verification ([MiniCPM4-1.1] uint64
 *     mask; [CPM.cu] tree verification inside flash attention).  n_draft <= 64
 *     draft tokens come after kv_len[b] committed tokens; bit j of
 *     tree_mask[b,i] says draft i attends to draft j (the mask holds the
 *     draft's own bit and its ancestors').  Each draft selects its own blocks
 *     from all cached kernels (bt = the last cached block) and attends to
 *     every cached token of them plus the masked drafts, whose keys and values
 *     come from draft_k/draft_v [B, Hkv, n_draft, d] (not pooled, not cached).
 * q [B, n_draft, Hq, d]; o [B, n_draft, Hq, d]; lse [B, Hq, n_draft] or NULL;
 * idx_out [B, Hkv, n_draft, S_max] / counts_out [B, Hkv, n_draft] receive the
 * selection when not NULL (S_max is ignored when idx_out is NULL).
 * Requires ws_bytes >= infllmv2_workspace_size(INFLLMV2_ENTRY_DECODE, ...).
 * Single-token decode runs as one kernel (one thread-block cluster per
 * (sequence, KV head) row, every intermediate on chip) when the shape allows
 * (G <= 16, d in {64, 128}, block 64/128, at most 4096 blocks); trees and
 * other shapes run separate scoring, top-k, split and merge kernels that use
 * the workspace.  Results are the same either way.
 */
int infllmv2_decode(const void* q, const void* k_cache, const void* v_cache,
                    const void* kernel_cache, const int32_t* kv_len, const void* draft_k,
                    const void* draft_v, const uint64_t* tree_mask, int B, int n_draft, int Hq,
                    int Hkv, int d, int L_max, int M_max, void* o, float* lse, int32_t* idx_out,
                    int32_t* counts_out, int S_max, void* workspace, size_t ws_bytes,
                    const infllmv2_params* params, void* stream);

/*
 * infllmv2_decode of one single-token step whose query, cache lengths and
 * output live in host memory: q_host [B, Hq, d] bf16 and kv_len_host [B] in,
 * o_host [B, Hq, d] bf16 (and lse_host [B, Hq] fp32, when not NULL) out; on
 * return the host output is complete.  Two ways, chosen per call:
 *   - zero-copy: when every host buffer is 16-byte aligned and usable by the
 *     device -- any host memory on a device that reads pageable memory through
 *     the host's page tables (cudaDevAttrPageableMemoryAccess and
 *     ...UsesHostPageTables, as a GPU attached to a Grace CPU), else memory
 *     page-locked and mapped into the device's address space (cudaHostAlloc /
 *     cudaMallocHost, or registered with mapping) -- and the single-kernel
 *     decode covers the shape, that kernel reads q and the lengths and writes
 *     o and lse straight through host memory (on a Grace host, over
 *     NVLink-C2C); the buffers must then be valid host memory of the stated
 *     sizes (the device reads and writes them as they are); device errors go
 *     to a page-locked error word of the calling host thread (allocated on its
 *     first such call, kept until the process exits); one launch and one wait.
 *     The staging buffers are not touched.
 *   - staged: otherwise q and kv_len are copied to the caller's device staging
 *     buffers q_dev, kv_len_dev on `stream` (cudaMemcpyAsync, one per buffer),
 *     infllmv2_decode runs on them into o_dev (and lse_dev), o and lse are
 *     copied back, the device error word is read in the same round trip and
 *     the stream is waited for.
 * q_dev, kv_len_dev, o_dev, lse_dev are the caller's device staging buffers
 * (16-byte aligned; lse_dev is required when lse_host is given; the library
 * allocates no device memory); the other arguments are those of
 * infllmv2_decode (n_draft = 1, no selection output).  Arguments are checked
 * before anything is enqueued.  Returns the first of: an argument error,
 * infllmv2_decode's status, INFLLMV2_ERR_CUDA for a failed copy or wait, and
 * the call's device error (INFLLMV2_ERR_DEVICE_INDEX or _TIMEOUT; the staged
 * way reads and clears the device error word as infllmv2_sync_status does).
 */
int infllmv2_decode_host(const void* q_host, const int32_t* kv_len_host, void* o_host, float* lse_host,
                         void* q_dev, int32_t* kv_len_dev, void* o_dev, float* lse_dev,
                         const void* k_cache, const void* v_cache, const void* kernel_cache, int B,
                         int Hq, int Hkv, int d, int L_max, int M_max, void* workspace,
                         size_t ws_bytes, const infllmv2_params* params, void* stream);

/*
 * Whether infllmv2_decode_host's zero-copy way takes pageable host buffers on
 * the current device: *direct = 1 when the device reads and writes pageable
 * memory coherently through the host's page tables (a GPU attached to a Grace
 * CPU over NVLink-C2C), else 0 (then only page-locked, mapped buffers avoid the
 * staged copies; also 0 when no device can be queried).  Returns INFLLMV2_OK,
 * or INFLLMV2_ERR_INVALID_ARG when direct is NULL.
 */
int infllmv2_host_memory_direct(int* direct);

/*
 * One whole single-token decode step: infllmv2_append (the new token's K and V
 * into row kv_len[b]-1 of the caches, and the semantic kernel it completes),
 * then infllmv2_decode of q over the updated caches ([CPM.cu] section 4: the
 * per-token cache update and attention of a CUDA-graph decode step).  kv_len
 * counts the new token.  Arguments as for those two calls (k_new, v_new
 * [B, Hkv, d] bf16; caches writable; M_max >= 1).  When the kernel the new
 * token completes can only overlap the query's forced local blocks
 * (n_local_blocks >= ceil((kernel_size-1)/block_size) + 1) and the
 * single-kernel decode covers the shape, both happen in that one launch: this
 * step's scores never use the new kernel, so it is pooled alongside.  Otherwise
 * the append kernel runs first.  Results are the same either way.
 */
int infllmv2_decode_step(const void* q, const void* k_new, const void* v_new, void* k_cache,
                         void* v_cache, void* kernel_cache, const int32_t* kv_len, int B, int Hq,
                         int Hkv, int d, int L_max, int M_max, void* o, float* lse,
                         int32_t* idx_out, int32_t* counts_out, int S_max, void* workspace,
                         size_t ws_bytes, const infllmv2_params* params, void* stream);

/*
 * Rotary positions.  The method's q and K carry their positions when they reach
 * the scores and the caches; these entry points put them on.  Pair i of a head
 * (i < rotary_dim / 2) is elements i and rotary_dim/2 + i, or, interleaved, 2i
 * and 2i + 1.  In the row at position x it turns by x * theta_i:
 *   y_a = attn_scale (a cos - b sin),  y_b = attn_scale (a sin + b cos)
 * in fp32 (cos and sin, attn_scale in them, to 2^-23 of attn_scale), rounded once;
 * elements from rotary_dim on are copied bit for bit.
 */
typedef struct infllmv2_rope_params {
    int32_t rotary_dim;   /* leading elements of a head that turn: even, 2 .. d      */
    int32_t interleaved;  /* 0: pairs (i, rotary_dim/2 + i); 1: pairs (2i, 2i + 1)    */
    float attn_scale;     /* factor on the rotated elements; 0 selects 1             */
} infllmv2_rope_params;

/* Scalings for contexts longer than the trained one (infllmv2_rope_freqs). */
enum {
    INFLLMV2_ROPE_PLAIN = 0,   /* theta_i = base^(-2i / rotary_dim)                        */
    INFLLMV2_ROPE_LINEAR = 1,  /* theta_i / factor (positions squeezed)                   */
    INFLLMV2_ROPE_NTK = 2,     /* plain with base * factor^(rotary_dim / (rotary_dim-2))  */
    INFLLMV2_ROPE_YARN = 3,    /* by wavelength: theta_i where a pair turns more than
                                  beta_fast times within orig_len tokens, theta_i / factor
                                  where less than beta_slow times, a ramp over i between;
                                  attn_scale = 0.1 ln(factor) + 1 (1 for factor <= 1)     */
    INFLLMV2_ROPE_DIVISORS = 4 /* theta_i / divisors[i] (searched per-pair factors);
                                  attn_scale = sqrt(1 + ln(factor) / ln(orig_len)), 1 for
                                  factor <= 1                                             */
};

/* Types of the tensors that take a dtype argument. */
enum { INFLLMV2_BF16 = 0, INFLLMV2_FP32 = 1 };

/*
 * Host helper: the table of frequencies that the entry points below read from
 * device memory.  freqs_host[i] = floor(frac(theta_i / 2 pi) * 2^64), the turns
 * per position in units of 2^-64, computed in fp64: position times it, modulo
 * 2^64, is the fraction of a turn, with no rounding of its own for any int32
 * position.
 * Writes rotary_dim / 2 entries and, when attn_scale is not NULL, the scaling's
 * factor.  base > 1; factor > 0 is read by every scaling but PLAIN; orig_len > 1
 * by YARN and DIVISORS; beta_fast > beta_slow > 0 by YARN; divisors
 * [rotary_dim / 2], each > 0, by DIVISORS.  NTK needs rotary_dim > 2.
 */
int infllmv2_rope_freqs(int scaling, int rotary_dim, double base, double factor, int orig_len, double beta_fast,
                        double beta_slow, const float* divisors, uint64_t* freqs_host, float* attn_scale);

/*
 * Rotary positions of q and K rows at explicit positions.  Row r of q is Hq
 * heads of d elements at q + r*ld_q (likewise the others; ld in elements, at
 * least heads * d, so slices of a fused projection are taken as they are).
 *   pos     [rows] device int32, any value
 *   freqs   [rotary_dim / 2] device uint64 (infllmv2_rope_freqs)
 *   dtype   of q, k and the outputs: INFLLMV2_BF16 or INFLLMV2_FP32
 *   transposed != 0: the transpose (opposite angles, the same factor): the
 *           gradient of the inputs from the gradient of the outputs.
 * k may be NULL with k_out NULL and Hk 0.  An output may be its input (the same
 * pointer and ld); any other overlap is refused (here and below: of row tensors
 * with each other; caches and draft buffers overlap nothing else).  d 64 or 128;
 * at most 2^30 rows and 2^14 heads.
 */
int infllmv2_rope(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const int32_t* pos, const uint64_t* freqs,
                  int rows, int Hq, int Hk, int d, int dtype, int transposed, void* q_out, int64_t ld_qo, void* k_out,
                  int64_t ld_ko, const infllmv2_rope_params* rope, void* stream);

/*
 * A chunk into the caches: q rotated to q_out, K rotated into k_cache and V
 * copied into v_cache, each token at its position.  The chunk is the last tokens
 * of each sequence, as for the attention calls:
 *   cu_q == NULL: Tq tokens per sequence, rows b*Tq + t at positions
 *                 kv_len[b] - Tq + t (total_q is B*Tq);
 *   cu_q != NULL: packed, rows cu_q[b] + t at kv_len[b] - len_b + t, len_b at
 *                 most Tq; rows from cu_q[B] to total_q are left as they are.
 * q [total_q rows of ld_q], k_new, v_new [rows of ld_k, ld_v] bf16; q_out
 * [total_q, Hq, d] packed, q itself when ld_q = Hq*d; caches [B, Hkv, L_max, d].
 * Kernels that the chunk completes are pooled by infllmv2_kernel_pool(_varlen).
 * Device errors (kv_len[b] below the chunk's length or past L_max, a length
 * outside [0, Tq], cu_q[0] not 0, cu_q[B] past total_q) set the error word.  A
 * sequence is taken whole or skipped: those of such a length or kv_len, those
 * that reach outside [0, total_q), and, of sequences that share rows (descending
 * offsets), all or all but one.  Calls without work (B, Tq or total_q 0) read no offsets.
 */
int infllmv2_rope_append(const void* q, int64_t ld_q, const void* k_new, int64_t ld_k, const void* v_new, int64_t ld_v,
                         void* q_out, void* k_cache, void* v_cache, const int32_t* kv_len, const int32_t* cu_q,
                         const uint64_t* freqs, int B, int Tq, int total_q, int Hq, int Hkv, int d, int L_max,
                         const infllmv2_rope_params* rope, void* stream);

/*
 * The gradient of infllmv2_rope_append: from the fp32 gradients that
 * infllmv2_sparse_attn_bwd gives -- dq [total_q, Hq, d] of the rotated q, dk and
 * dv [B, Hkv, L_max, d] of the caches -- those of the chunk's q, K and V rows
 * before rotation, dq_out, dk_out, dv_out (row strides ld_*, as above; dtype
 * INFLLMV2_BF16 or INFLLMV2_FP32).  dq_out may be dq (fp32, ld_dq = Hq*d).
 * Rows of skipped sequences and behind the last sequence are left as they are.
 */
int infllmv2_rope_append_bwd(const float* dq, const float* dk, const float* dv, void* dq_out, int64_t ld_dq, void* dk_out,
                             int64_t ld_dk, void* dv_out, int64_t ld_dv, const int32_t* kv_len, const int32_t* cu_q,
                             const uint64_t* freqs, int B, int Tq, int total_q, int Hq, int Hkv, int d, int L_max,
                             int dtype, const infllmv2_rope_params* rope, void* stream);

/*
 * A draft tree's q, K and V as infllmv2_decode takes them.  Draft i of sequence
 * b sits depth - 1 positions after the committed tokens, depth = the bits of
 * tree_mask[b, i] (its ancestors and itself; an empty mask counts as 1):
 * position kv_len[b] + depth - 1.  q, k_new, v_new are rows b*n_draft + i of
 * ld_q, ld_k, ld_v elements; q_out [B, n_draft, Hq, d] (q itself when
 * ld_q = Hq*d), draft_k and draft_v [B, Hkv, n_draft, d].  A kv_len outside
 * [0, 2^28] sets the error word; that sequence is skipped.
 */
int infllmv2_rope_drafts(const void* q, int64_t ld_q, const void* k_new, int64_t ld_k, const void* v_new, int64_t ld_v,
                         void* q_out, void* draft_k, void* draft_v, const int32_t* kv_len, const uint64_t* tree_mask,
                         const uint64_t* freqs, int B, int n_draft, int Hq, int Hkv, int d,
                         const infllmv2_rope_params* rope, void* stream);

/*
 * Norms of q and K for each head in front of the rotation, in the same pass: every
 * head x of q and K becomes
 *   R(x r (w + weight_offset)),  r = 1 / sqrt(mean(x^2) + eps)
 * with the mean over its d elements, w the [d] weight of q's or of K's heads
 * (NULL: the factor is 1) and R the rotation of the calls above; elements from
 * rotary_dim on are normed too, V is copied.  fp32 arithmetic, rounded once.  A
 * head whose squares pass fp32's range is normed like any other; in one with an
 * infinite element that element and what it turns with become NaN, the others 0.
 *
 * infllmv2_norm_rope, _append and _drafts take, read and write what infllmv2_rope
 * (not transposed), infllmv2_rope_append and infllmv2_rope_drafts do.
 */
typedef struct infllmv2_norm_params {
    float eps;             /* in (0, 1]                                                */
    float weight_offset;   /* added to the weights: 1 for those stored as w - 1        */
    int32_t weight_dtype;  /* of q_weight and k_weight: INFLLMV2_BF16 or INFLLMV2_FP32 */
} infllmv2_norm_params;

int infllmv2_norm_rope(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const int32_t* pos, const uint64_t* freqs,
                       int rows, int Hq, int Hk, int d, int dtype, void* q_out, int64_t ld_qo, void* k_out, int64_t ld_ko,
                       const void* q_weight, const void* k_weight, const infllmv2_norm_params* norm,
                       const infllmv2_rope_params* rope, void* stream);

int infllmv2_norm_rope_append(const void* q, int64_t ld_q, const void* k_new, int64_t ld_k, const void* v_new, int64_t ld_v,
                              void* q_out, void* k_cache, void* v_cache, const int32_t* kv_len, const int32_t* cu_q,
                              const uint64_t* freqs, int B, int Tq, int total_q, int Hq, int Hkv, int d, int L_max,
                              const void* q_weight, const void* k_weight, const infllmv2_norm_params* norm,
                              const infllmv2_rope_params* rope, void* stream);

int infllmv2_norm_rope_drafts(const void* q, int64_t ld_q, const void* k_new, int64_t ld_k, const void* v_new, int64_t ld_v,
                              void* q_out, void* draft_k, void* draft_v, const int32_t* kv_len, const uint64_t* tree_mask,
                              const uint64_t* freqs, int B, int n_draft, int Hq, int Hkv, int d, const void* q_weight,
                              const void* k_weight, const infllmv2_norm_params* norm, const infllmv2_rope_params* rope,
                              void* stream);

/*
 * Gradients of infllmv2_norm_rope: from dq and dk of its outputs (dk NULL with
 * Hk 0) and its inputs q and k, those of the inputs, dq_out and dk_out, and of
 * the weights.  With g the gradient turned back and w' = w + weight_offset:
 *   dx = r (g w' - x r mean(g w' x r)),  d_weight = sum over rows and heads of g x r
 * dtype is the type of all rows.  dq_weight and dk_weight [d] fp32 are overwritten
 * (zeros for calls without rows); either may be NULL.  Unless both are, workspace
 * needs infllmv2_workspace_size(INFLLMV2_ENTRY_NORM_ROPE_BWD, ...) bytes.  dq_out
 * may be dq, dk_out dk (the same pointer and ld); no other tensors overlap.  The
 * same call on the same inputs gives the same bits.  The workspace holds nothing
 * between calls; calls that may overlap on the GPU need one each.
 */
int infllmv2_norm_rope_bwd(const void* dq, int64_t ld_dq, const void* dk, int64_t ld_dk, const void* q, int64_t ld_q,
                           const void* k, int64_t ld_k, const int32_t* pos, const uint64_t* freqs, int rows, int Hq, int Hk,
                           int d, int dtype, void* dq_out, int64_t ld_dqo, void* dk_out, int64_t ld_dko, const void* q_weight,
                           const void* k_weight, float* dq_weight, float* dk_weight, void* workspace, size_t ws_bytes,
                           const infllmv2_norm_params* norm, const infllmv2_rope_params* rope, void* stream);

/*
 * Gradients of infllmv2_norm_rope_append: dq, dk, dv (fp32), the outputs dq_out,
 * dk_out, dv_out and their dtype, kv_len and cu_q as for infllmv2_rope_append_bwd;
 * q [total_q rows of ld_q] and k_new [rows of ld_k] bf16 are the chunk's rows that
 * went into the forward call; weights, their gradients and the workspace as above.
 * Skipped sequences and rows behind the last sequence add nothing to the weights'
 * gradients and are left as they are.
 */
int infllmv2_norm_rope_append_bwd(const float* dq, const float* dk, const float* dv, const void* q, int64_t ld_q,
                                  const void* k_new, int64_t ld_k, void* dq_out, int64_t ld_dq, void* dk_out, int64_t ld_dk,
                                  void* dv_out, int64_t ld_dv, const int32_t* kv_len, const int32_t* cu_q,
                                  const uint64_t* freqs, int B, int Tq, int total_q, int Hq, int Hkv, int d, int L_max,
                                  int dtype, const void* q_weight, const void* k_weight, float* dq_weight, float* dk_weight,
                                  void* workspace, size_t ws_bytes, const infllmv2_norm_params* norm,
                                  const infllmv2_rope_params* rope, void* stream);

/*
 * Penalties for repeated tokens, biases and grammar masks on the logits of a draft
 * tree's nodes (n_draft 1: of plain decoding), and the distributions they leave,
 * as infllmv2_verify takes them.  Row i of sequence b is the logits after node i.
 * With c(t) how often token t was generated -- in the history and among the drafts
 * on node i's way, the root (whose token is in the history) not counted -- and
 * seen(t) whether c(t) > 0 or t is in the prompt, every logit l of token t becomes
 *   l1 = seen(t) ? (l > 0 ? l / repetition : l * repetition) : l
 *   l2 = l1 - frequency * c(t) - presence * [c(t) > 0]
 *   l3 = l2 + bias(t);  -inf where the row's mask has no bit for t, and for NaN
 * in fp32: the quotient as the product with the rounded 1 / repetition, frequency's
 * and presence's parts summed before they are taken off, with one rounding for l2.
 * probs == 0: the row becomes l3.
 * probs != 0: softmax(l3 / temperature) -- infinite logits share the whole, logits
 * that differ by more than fp32's range count as infinitely far apart -- and at
 * temperature 0 a one at the first of its largest elements.  A row of which
 * nothing is left (-inf everywhere) becomes zeros, which infllmv2_verify reports
 * where it needs the row.
 *   logits, out   rows b*n_draft + i of ld, ld_out elements, dtype and out_dtype
 *                 INFLLMV2_BF16 or INFLLMV2_FP32; out may be logits (the same
 *                 pointer, ld and type) and overlaps nothing else.  Like every
 *                 tensor they start on 16 bytes: the last row of a [T, V] tensor
 *                 with an odd V may not, and is copied first
 *   tokens        [B, n_draft] int32, the drafts (a root's is not read); NULL: no
 *                 drafts are counted
 *   tree_mask     [B, n_draft] as for infllmv2_decode, given with tokens alone;
 *                 NULL: a chain
 *   n_nodes       [B] int32 in [0, n_draft], nodes in use; rows behind them are
 *                 left as they are; NULL: n_draft everywhere
 *   history       [B] rows of ld_history 16-bit counts of the V tokens: bit 15 in
 *                 the prompt, bits 0..14 generated count (infllmv2_count_tokens);
 *                 NULL: nothing was seen
 *   allowed       [B * n_draft] rows of ld_allowed words: token t is allowed iff
 *                 bit t % 32 of word t / 32 is set; NULL: all are
 *   bias          [B] rows of ld_bias fp32 (ld_bias 0: one row for all); NULL: 0
 *   controls      [B, 4] fp32: repetition (> 0), frequency, presence, temperature
 *                 (>= 0), all finite; NULL: 1, 0, 0, 1
 * Device errors (controls out of range, n_nodes out of range, a token of a draft on
 * a row's way outside [0, V), bits of a row's mask from n_draft on, the root's too)
 * set the error word; those rows become zeros (probs == 0: -inf).
 * V <= 2^24; at most 2^18 rows.
 */
int infllmv2_constrain(const void* logits, int64_t ld, const int32_t* tokens, const uint64_t* tree_mask,
                       const int32_t* n_nodes, const uint16_t* history, int64_t ld_history, const uint32_t* allowed,
                       int64_t ld_allowed, const float* bias, int64_t ld_bias, const float* controls, int B, int n_draft,
                       int V, int dtype, int probs, void* out, int64_t ld_out, int out_dtype, void* stream);

/*
 * The token counts that infllmv2_constrain reads.  Sequence b's tokens are added
 * to row b of history: with prompt != 0 their bit 15 is set, else their count goes
 * up by their occurrences (and stays at 32767 where it would pass it).
 *   cu == NULL: tokens [B, T] int32, of each sequence the first n_tokens[b] (NULL:
 *               T), so infllmv2_verify's out_tokens and n_path are taken as they are;
 *   cu != NULL: packed, sequence b's are tokens cu[b] .. cu[b+1] - 1 of total.
 * reset != 0: the rows of all B sequences are cleared before (a slot that another
 * sequence takes).  history rows are ld_history elements apart; what lies behind
 * their V counts is left as it is.  (With ld_history a multiple of 8 every row starts
 * on 16 bytes, and a call can be given one slot's row alone.)
 * Device errors (a token outside [0, V), n_tokens outside [0, T], offsets that do
 * not ascend from 0 to at most total) set the error word; those tokens and the
 * tokens of such a length are left out, and of packed sequences each is taken
 * whole or left out.  V <= 2^24, B <= 65535.
 */
int infllmv2_count_tokens(const int32_t* tokens, const int32_t* n_tokens, const int32_t* cu, int B, int T, int total, int V,
                          int prompt, int reset, uint16_t* history, int64_t ld_history, void* stream);

/*
 * Verification of a draft tree ([MiniCPM4-1.1] tree-speculative decoding) by
 * recursive rejection sampling, from given random numbers.  Node 0 is the tree's
 * root, the token sampled last: it always stands.  Node i's parent is the
 * ancestor whose mask is tree_mask[b, i] without bit i; ancestors come before
 * their descendants.  Rows of probabilities:
 *   target [B, n_draft, V]: row i is the target's distribution after node i
 *   draft  [B, n_draft, V]: row i is the distribution node i's children were
 *          drawn from; only rows of nodes with children are read.  NULL: the
 *          drafts were chosen, not drawn (a child's own probability is then 1).
 * From the root down, the children x of a node (by index) are tried in turn with
 * w = p, Z = 1, R = 1 (p, q the node's target and draft rows):
 *   x stands iff u[x] Z q(x) < w(x) R.  Otherwise w(y) becomes
 *   max(w(y) - (Z/R) q(y), 0) for every token y, Z the sum of w, and, without
 *   replacement (replace == 0), R loses q(x); with R <= 0 nothing changes.
 *   draft == NULL: x stands iff u[x] Z < w(x); otherwise Z loses w(x), w(x) = 0.
 * The first child that stands is the next node; where none does, the last token
 * is the first one whose running sum of w passes u[0] * (sum of w), or of p when
 * w has nothing left.  Weights are held in units of 2^-62 (what of a probability
 * lies below that is dropped); their sums and the comparisons are exact.  So is w
 * after one rejection at a node; from the second on the factor of q in w, a sum of
 * the quotients Z/R, is rounded up by less than 2^-57 of itself, and its product
 * with q down to whole units.
 *   tokens    [B, n_draft] int32; a root's is not read
 *   tree_mask [B, n_draft], NULL: a chain (node i's parent is i - 1)
 *   n_nodes   [B] int32 in [0, n_draft], nodes in use (0: the sequence is idle);
 *             NULL: n_draft everywhere
 *   u         [B, n_draft] fp32 in [0, 1): u[b, i] tries node i, u[b, 0] draws
 *   dtype     of target and draft: INFLLMV2_FP32 or INFLLMV2_BF16
 * Out: path [B, n_draft], the nodes that stand, from the root, then -1; n_path
 * [B] their number; out_tokens [B, n_draft], the n_path[b] new tokens (the
 * path's behind the root, then the one drawn), then -1; and, with kv_len given,
 * kv_len_out[b] = kv_len[b] + n_path[b] (the lengths with the path committed;
 * kv_len_out may be kv_len; both NULL or neither).
 * Probabilities: NaN and values below 0 are read as 0, values above 1 as 1.
 * Device errors (masks that are no tree, a token outside [0, V), n_nodes out of
 * range, a target row that had to be summed -- the last node's, or one with
 * children left after a rejection -- with a sum above 2, or the last node's with
 * a sum of 0) set the error word; that sequence's outputs are those of an idle
 * one: n_path 0, -1 elsewhere, kv_len unchanged.  (After a wait that ran out,
 * INFLLMV2_ERR_DEVICE_TIMEOUT, a sequence's outputs are undefined.)
 * Needs no workspace.  n_draft <= 64, V <= 2^24.
 */
int infllmv2_verify(const int32_t* tokens, const uint64_t* tree_mask, const int32_t* n_nodes, const void* target,
                    const void* draft, const float* u, const int32_t* kv_len, int B, int n_draft, int V, int dtype,
                    int replace, int32_t* path, int32_t* n_path, int32_t* out_tokens, int32_t* kv_len_out,
                    void* stream);

/*
 * Commit of a verified path: the accepted drafts' K and V become the last
 * n_path[b] tokens of each sequence, and the semantic kernels that they complete
 * are pooled exactly as infllmv2_kernel_pool does (one launch).  kv_len counts
 * the committed tokens (infllmv2_verify's kv_len_out):
 *   cache row kv_len[b] - n_path[b] + t = draft row path[b, t],  t < n_path[b]
 *   draft_k, draft_v [B, Hkv, n_draft, d] bf16, as for infllmv2_decode, and not
 *   overlapping the caches; path [B, n_draft], n_path [B] device int32.
 * kernel_cache may be NULL only when M_max == 0.  Device errors (n_path outside
 * [0, n_draft], kv_len below it or past L_max, a path entry that is no draft, a
 * completed kernel past M_max) set the error word; that sequence is skipped.
 * Other cache rows and kernels are untouched.
 */
int infllmv2_commit(const void* draft_k, const void* draft_v, const int32_t* path, const int32_t* n_path, void* k_cache,
                    void* v_cache, void* kernel_cache, const int32_t* kv_len, int B, int n_draft, int Hkv, int d,
                    int L_max, int M_max, const infllmv2_params* params, void* stream);

/*
 * Allocation-free decode.  The paper has no counterpart: this entry point is
 * for callers of this library that cannot provide a workspace -- a process whose
 * device memory is reserved up front by its own pool, a plugin that receives
 * only input and output pointers, or a loop that must not allocate after
 * start-up.  It behaves exactly like infllmv2_decode (same arguments without
 * workspace/ws_bytes, same results) but takes its scratch from one fixed array
 * of INFLLMV2_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that
 * loads the library holds until the process exits.
 *   - Problems whose decode workspace (infllmv2_workspace_size with
 *     INFLLMV2_ENTRY_DECODE) exceeds that size are rejected with
 *     INFLLMV2_ERR_WORKSPACE before anything is enqueued.
 *   - The first call on each device looks up the array's device address with
 *     cudaGetSymbolAddress (the device must be current); make that first call
 *     before any stream capture.
 *   - All calls share the array and it keeps the last call's contents (nothing
 *     in it needs to start at zero).  Calls that overlap on the GPU -- other
 *     streams, other host threads -- race on it; serialise them.
 *   - It never calls cudaMalloc, cudaFree or any allocating routine.
 */
#define INFLLMV2_NOALLOC_SCRATCH_BYTES (16u << 20)
int infllmv2_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                            const void* kernel_cache, const int32_t* kv_len, const void* draft_k,
                            const void* draft_v, const uint64_t* tree_mask, int B, int n_draft,
                            int Hq, int Hkv, int d, int L_max, int M_max, void* o, float* lse,
                            int32_t* idx_out, int32_t* counts_out, int S_max,
                            const infllmv2_params* params, void* stream);

/*
 * Stage timing (the pages' CPM.cu lists a performance-analysis module next to
 * the inference entry; this is the library's counterpart).  While enabled,
 * every entry point records a CUDA event on its stream before its first kernel
 * and after each kernel it launches; infllmv2_profile_read then waits for
 * those events and writes the elapsed milliseconds of each stage of the most
 * recent call into ms[0 .. *n_stages-1] (at most max_stages), and
 * infllmv2_profile_stage_name(i) names stage i ("pool", "score", "topk",
 * "attend", "combine", "rope", "norm_rope", "constrain",
 * "count", "verify", "commit").  Events live in the library, per device, created on
 * first use; enabling costs one event record per kernel.  Not thread-safe.
 * Returns INFLLMV2_OK or INFLLMV2_ERR_CUDA.
 */
int infllmv2_profile_enable(int on);
int infllmv2_profile_read(float* ms, int max_stages, int* n_stages);
const char* infllmv2_profile_stage_name(int i);

#ifdef __cplusplus
}
#endif

#endif /* INFLLMV2_H_ */
