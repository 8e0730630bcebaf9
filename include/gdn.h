/*
 * gdn.h -- C ABI of the Gated DeltaNet (GDN) speculative-decoding hot path on GB300 (sm_103a).
 *
 * The operation is the GDN linear-attention core that hybrid Qwen3-Next-style layers run when a
 * speculative (draft + verify) step and ordinary decode/prefill rows share one batch:
 *   (1) a width-W causal depthwise conv1d + SiLU over the packed q|k|v channels, with each
 *       sequence's conv history kept as a rolled ring in a pool slot;
 *   (2) the sigmoid-gated delta rule over an fp32 d_v x d_k state per v-head, with one state
 *       slot per speculative position;
 *   (3) the split of a mixed batch into speculative and non-speculative rows, each read from
 *       and written back to interleaved global token positions through its own token index.
 *
 * Sources (page title, section):
 *   "[GDN] Spec-decoding-aware attention kernel" (vllm-xpu-kernels PR 336) -- Problem: the conv
 *       ring is a rolled history at column 0 of cache_indices, read at offset num_accepted-1;
 *       Changes: the two-pass conv (stage, then a roll pass that is the slot's only writer),
 *       the state load from spec_state_indices[n, num_accepted[n]-1], the per-token store to
 *       spec_state_indices[n, t], slot <= 0 meaning "no prior state", and the rule that
 *       spec_state_indices and num_accepted_tokens come as a pair.
 *   "[XE2] Support MTP of QWEN model" (vllm-xpu-kernels PR 368) -- Copilot overview: the
 *       spec/non-spec split, num_spec_decodes, token_indx remapping of reads and writes, the
 *       chunked prefill path; review notes: every optional tensor is checked before use;
 *       commit message: no rectangular assumption on spec rows, only the conservation check
 *       non_spec_tokens + spec_tokens == num_actual_tokens.
 *   "[Bugfix] Align Qwen GDN gates with speculative tokens" (vllm PR 51812) -- Purpose: the
 *       a/b gates are gathered with the same index as q|k|v.
 *
 * Conventions shared by every entry point.
 *   Pointers are DEVICE pointers unless stated, borrowed for the duration of the stream work;
 *   the caller owns all memory.  Calls only enqueue work on `stream` (a cudaStream_t passed as
 *   void*, NULL = legacy default stream); they never synchronise, never read device memory on
 *   the host, and allocate nothing.
 *   Dense row-major layouts, no strides.  C = 2*Hk*dk + Hv*dv channels, packed as
 *   q (Hk*dk) | k (Hk*dk) | v (Hv*dv), head-major (x may instead arrive per k-head, see
 *   gdn_qkv_layout).  v-head h uses k-head h / (Hv/Hk).
 *   Activations (x, a, b, out, conv pool, conv weight/bias) use gdn_layer_desc.act_dtype.
 *   The SSM pool is fp32 [num_slots, Hv, dv, dk] (dk fastest).  Conv pool [num_slots,
 *   conv_state_len, C].  Slot values <= 0 are NULL: zero prior on load, no write.
 *   Integer metadata is int32.  All activation, pool and weight pointers must be 16-byte
 *   aligned.
 *   Host-detectable problems return a negative gdn_error before anything is enqueued.
 *   Problems only visible in device data (an index out of range, num_accepted outside
 *   [1, spec_cols], a non-monotone query_start_loc, a spec row longer than spec_cols) never
 *   trap: the kernel ORs a GDN_STATUS_* bit into *d_status (if d_status is not NULL), treats
 *   the bad load as zero and skips the bad write (or the whole row, for row-level problems).
 *   Rows of one call must use distinct slots; overlapping slots give undefined results.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDN_OK = 0,
  GDN_ERR_NULL_ARG = -1,     /* a required pointer is NULL                                   */
  GDN_ERR_SPEC_PAIR = -2,    /* spec_state_indices without num_accepted_tokens, or vice versa */
  GDN_ERR_SHAPE = -3,        /* head/conv sizes, spec_cols, row counts or limits unsupported  */
  GDN_ERR_CONSERVATION = -4, /* non-spec tokens + spec tokens != num_actual_tokens            */
  GDN_ERR_WORKSPACE = -5,    /* workspace NULL or smaller than gdn_workspace_bytes()         */
  GDN_ERR_DTYPE = -6,        /* unknown gdn_dtype                                             */
  GDN_ERR_CUDA = -7,         /* a kernel launch failed (cudaGetLastError after the launch)    */
  GDN_ERR_ALIGN = -8         /* a pointer is not 16-byte aligned                              */
} gdn_error;

/* Bits ORed into *d_status by the kernels. */
#define GDN_STATUS_SLOT_RANGE 0x1u   /* a slot index >= num_slots (load read as zero, store skipped) */
#define GDN_STATUS_NUM_ACCEPTED 0x2u /* num_accepted_tokens[n] outside [1, spec_cols] (row skipped)  */
#define GDN_STATUS_TOKEN_RANGE 0x4u  /* token_indx outside [0, num_global_tokens) (read zero, write skipped) */
#define GDN_STATUS_ROW_RANGE 0x8u    /* query_start_loc not monotone / past num_tokens, or a spec row
                                        longer than spec_cols (row skipped)                            */
#define GDN_STATUS_WAIT_TIMEOUT 0x10u /* a bounded wait inside a tensor-core kernel gave up; that
                                         block's results are missing (never expected in practice)  */
#define GDN_STATUS_PAGE_RANGE 0x20u  /* a page id >= num_pages, a table row or a page range outside the table, or a
                                        page released more often than it was held (that entry is skipped)  */
#define GDN_STATUS_PAGE_SHARED 0x40u /* an append met a page that several rows hold (that token is skipped)  */
#define GDN_STATUS_NO_PAGES 0x80u    /* reserve/fork: the free pages did not cover a row (that row is skipped)  */

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

/* Channel order of the pre-conv activation x ("[GDN] Spec-decoding-aware attention kernel",
 * Test Plan: reorder_input).  Packed: q (Hk*dk) | k (Hk*dk) | v (Hv*dv), head-major
 * (reorder_input=True).  Per k-head: for each k-head g, q_g (dk) | k_g (dk) | v of its
 * G = Hv/Hk v-heads (G*dv) -- the projection order of production Qwen3-Next traffic
 * (reorder_input=False).  Conv weights, bias, the conv pool and every post-conv tensor use the
 * packed order in both cases. */
typedef enum { GDN_QKV_PACKED = 0, GDN_QKV_PER_KHEAD = 1 } gdn_qkv_layout;

/* How a speculative row keeps its conv history.  Rolled: one rolled history in column 0 of the
 * row's slots, read at offset num_accepted-1 ("[GDN] Spec-decoding-aware attention kernel",
 * Problem; needs conv_state_len >= W-2+spec_cols).  Per slot: after spec token t the last W-1
 * inputs are written to columns 0..W-2 of spec_state_indices[n, t] and the next step reads
 * spec_state_indices[n, num_accepted-1] ("[XE2] Support MTP of QWEN model", review thread).
 * Non-speculative rows behave the same in both. */
typedef enum { GDN_CONV_ROLLED = 0, GDN_CONV_PER_SLOT = 1 } gdn_conv_layout;

typedef struct {
  int32_t num_k_heads;    /* Hk >= 1                                                   */
  int32_t num_v_heads;    /* Hv, a multiple of Hk                                      */
  int32_t head_k_dim;     /* dk in {16, 32, 64, 128}                                    */
  int32_t head_v_dim;     /* dv, a multiple of 16, <= 256                               */
  int32_t conv_width;     /* W in {2, 3, 4}                                             */
  int32_t conv_state_len; /* columns per conv slot, >= W-1 (rolled spec rows: >= W-2+spec_cols) */
  gdn_dtype act_dtype;    /* GDN_BF16 or GDN_F32                                        */
  float scale;            /* multiplies the normalised q; <= 0 selects 1/sqrt(dk)       */
  int32_t qkv_layout;     /* gdn_qkv_layout of x                                        */
  int32_t conv_layout;    /* gdn_conv_layout of speculative rows                        */
} gdn_layer_desc;

typedef struct {
  const void* conv_weight; /* [C, W] act dtype; w[c][W-1] multiplies the current token */
  const void* conv_bias;   /* [C] act dtype, or NULL for no bias                         */
  const float* A_log;      /* [Hv]: g = -exp(A_log[h]) * softplus(a + dt_bias[h])       */
  const float* dt_bias;    /* [Hv]                                                       */
} gdn_layer_params;

typedef struct {
  void* conv_pool;   /* [num_slots, conv_state_len, C] act dtype (read and written) */
  float* ssm_pool;   /* [num_slots, Hv, dv, dk] fp32 (read and written)             */
  int64_t num_slots; /* slot 0 is conventionally reserved as NULL                   */
} gdn_pools;

/*
 * One subset of rows.  spec_state_indices and num_accepted_tokens come as a pair (both, or
 * GDN_ERR_SPEC_PAIR).  A subset is speculative when it has the pair and no state_indices.
 * A non-speculative subset (state_indices given) may also carry the pair: its rows are then
 * acceptance-aware, i.e. each continues from what its previous verify step accepted -- a
 * verify row cut to a prefix by the batch token budget and scheduled as a plain row ("[Bugfix]
 * Align Qwen GDN gates with speculative tokens", the second mechanism in the reachability
 * comment).  Such a row reads its conv history at column offset num_accepted-1 of
 * state_indices[n] (rolled layout) or from spec_state_indices[n, num_accepted-1] (per-slot
 * layout), loads its SSM state from spec_state_indices[n, num_accepted-1], and writes like any
 * non-spec row.  A row that accepted one token with spec_state_indices[n, 0] == state_indices[n]
 * is an ordinary non-spec row.
 * Local tokens are numbered 0..num_tokens-1 in row order; row n owns local tokens
 * [query_start_loc[n], query_start_loc[n+1]).
 */
typedef struct {
  int32_t num_seqs;                   /* N_sub rows (may be 0)                                   */
  int32_t num_tokens;                 /* T_sub local tokens; query_start_loc[N_sub] must equal it */
  const int32_t* query_start_loc;     /* [N_sub+1], query_start_loc[0] == 0                       */
  const int32_t* token_indx;          /* [T_sub] global token of each local token; NULL = identity */
  const int32_t* state_indices;       /* non-spec: [N_sub] conv+SSM slot of each row              */
  const int32_t* has_initial_state;   /* non-spec: [N_sub], 0 = start from zeros; NULL = all 1    */
  const int32_t* spec_state_indices;  /* spec: [N_sub, spec_cols]; column 0 is also the conv slot;
                                         non-spec: the previous verify step's slots, or NULL     */
  const int32_t* num_accepted_tokens; /* spec (and acceptance-aware non-spec): [N_sub], in
                                         [1, spec_cols]                                          */
  int32_t spec_cols;                  /* spec: columns of spec_state_indices, 1..64                */
} gdn_rows;

/*
 * Bytes of device workspace gdn_mixed_batch needs for a batch without prefill rows (non_spec
 * and spec as they will be passed; either may be NULL): the fp32 post-conv q|k|v of every token,
 * spec subset first, each part rounded up to 256 bytes.  The pages stage the conv output of a
 * step in a buffer between the conv and the recurrence ("[GDN] Spec-decoding-aware attention
 * kernel", Changes: causal_conv1d pass 1 writes its outputs for the gated-delta-rule kernel);
 * keeping it in fp32 rather than the activation dtype is this library's reading (a bf16 rounding
 * of the post-conv values moves the state by more than the 1e-4 the path is held to).
 * Depends only on the host-side counts in the descriptors.  Returns 0 for invalid descriptors.
 */
size_t gdn_workspace_bytes(const gdn_layer_desc* layer, const gdn_rows* non_spec, const gdn_rows* spec);

/*
 * Extra workspace the chunked prefill needs when `rows` (a non-spec subset) holds num_prefills
 * prefill rows: one record of 123904 bytes per (64-token chunk, v-head), the chunk count bounded
 * from rows->num_tokens and num_prefills (ceil(num_tokens / 64) + num_prefills).  The pages run
 * prefill rows through a chunked kernel ("[XE2] Support MTP of QWEN model", Copilot overview:
 * chunk gated delta rule); the record holds that chunk form's state-independent terms, which
 * one kernel computes for all chunks at once and the chunk-by-chunk scan reads.  gdn_mixed_batch needs gdn_workspace_bytes() + gdn_prefill_workspace_bytes(
 * layer, non_spec, num_prefills); gdn_chunk_prefill needs gdn_prefill_workspace_bytes(layer,
 * rows, rows->num_seqs).  0 when the layer does not take the tensor-core path (see
 * gdn_chunk_prefill) or num_prefills is 0.
 */
size_t gdn_prefill_workspace_bytes(const gdn_layer_desc* layer, const gdn_rows* rows, int32_t num_prefills);

/*
 * Conv update of one subset (step (1); "[GDN] Spec-decoding-aware attention kernel",
 * Changes, causal_conv1d.hpp bullets; the review thread of "[XE2] Support MTP of QWEN model").
 * For row n with L tokens, history h = conv_pool[slot][a : a+W-1] where
 *   spec:     slot = spec_state_indices[n, 0], a = num_accepted_tokens[n] - 1 (rolled layout;
 *             per-slot layout: slot = spec_state_indices[n, num_accepted-1], a = 0);
 *   non-spec: slot = state_indices[n], a = 0 (acceptance-aware rows: a = num_accepted-1, or
 *             with the per-slot layout the history slot spec_state_indices[n, num_accepted-1]);
 * h is zero when the history slot is <= 0 or has_initial_state[n] == 0.  With H = h ++ x[token_indx[row]]:
 *   y[t][c] = SiLU(bias[c] + sum_i conv_weight[c][i] * H[t+i][c])     (fp32 arithmetic)
 * and, after every read of the slot, the slot's columns are rewritten as bit copies:
 *   spec:     columns 0 .. W-3+L  <- H[1 .. W-2+L]   (column W-2+t holds token t)
 *   non-spec: columns 0 .. W-2    <- H[L .. L+W-2]   (the last W-1 inputs)
 *   per-slot spec: columns 0 .. W-2 of spec_state_indices[n, t] <- H[t+1 .. t+W-1], t < L
 * other columns and slots are untouched; slot <= 0 is not written; L = 0 rows do nothing.
 *   x [num_global_tokens, C] act dtype (global order, gathered through token_indx);
 *   y [rows->num_tokens, C] in y_dtype (local order).
 * Size limit: one launch covers at most 65535 work units (a spec row is one unit; a non-spec
 * subset counts ceil(num_tokens / 16) + num_seqs), else GDN_ERR_SHAPE; gdn_mixed_batch counts
 * both subsets together.
 */
int gdn_conv_update(const gdn_layer_desc* layer, const gdn_layer_params* params, const gdn_pools* pools,
                    const void* x, int32_t num_global_tokens, const gdn_rows* rows, void* y,
                    gdn_dtype y_dtype, uint32_t* d_status, void* stream);

/*
 * Gated delta rule over one subset, token by token (step (2); "[GDN] Spec-decoding-aware
 * attention kernel", Changes, gated_delta_rule.hpp bullet).  For v-head h of row n:
 *   load S (dv x dk) from spec_state_indices[n, num_accepted[n]-1] (spec, and acceptance-aware
 *   non-spec rows) or state_indices[n] (other non-spec rows); zeros for a non-spec row with
 *   has_initial_state[n] == 0 and whenever the slot is <= 0;
 *   per token: g = -exp(A_log[h]) softplus(a + dt_bias[h]) (softplus(x) = x for x > 20),
 *   beta = sigmoid(b), q^ = q / sqrt(|q|^2 + 1e-6) * scale, k^ = k / sqrt(|k|^2 + 1e-6),
 *   S <- e^g S (I - beta k^ k^T) + beta v k^T,  out[token_indx[i]][h] = S q^;
 *   spec rows store S after token t to spec_state_indices[n, t]; non-spec rows store S after
 *   their last token to state_indices[n]; slots <= 0 are not written.
 *   qkv [rows->num_tokens, C] post-conv activation in qkv_dtype (local order);
 *   a, b [num_global_tokens, Hv] act dtype, read at token_indx (the same index as qkv);
 *   out [num_global_tokens, Hv, dv] act dtype, written at token_indx.
 */
int gdn_recurrent_step(const gdn_layer_desc* layer, const gdn_layer_params* params, const gdn_pools* pools,
                       const void* qkv, gdn_dtype qkv_dtype, const void* a, const void* b,
                       int32_t num_global_tokens, const gdn_rows* rows, void* out, uint32_t* d_status,
                       void* stream);

/*
 * The same result as gdn_recurrent_step for non-speculative rows of any length, computed
 * chunk by chunk (chunk_size tokens; 64 is the supported size) in the WY/UT form of the gated
 * delta rule on tcgen05 tensor cores ("[XE2] Support MTP of QWEN model", Copilot overview: XE2
 * chunk gated delta rule with remapped output writes).  Only the final state of each row is
 * stored.  The tensor-core path covers dk = dv = 128 with bf16 activations; other layers run the
 * token recurrence of gdn_recurrent_step (and need no workspace).
 *   rows must be non-speculative (GDN_ERR_SPEC_PAIR otherwise);
 *   workspace: at least gdn_prefill_workspace_bytes(layer, rows, rows->num_seqs) bytes,
 *   256-byte aligned (may be NULL when that is 0).
 */
int gdn_chunk_prefill(const gdn_layer_desc* layer, const gdn_layer_params* params, const gdn_pools* pools,
                      const void* qkv, gdn_dtype qkv_dtype, const void* a, const void* b,
                      int32_t num_global_tokens, const gdn_rows* rows, int32_t chunk_size, void* out,
                      void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/*
 * The whole path over a mixed batch (step (3); "[XE2] Support MTP of QWEN model", Copilot
 * overview and commit message; "[Bugfix] Align Qwen GDN gates with speculative tokens").
 * x [num_actual_tokens, C], a, b [num_actual_tokens, Hv] and out [num_actual_tokens, Hv, dv]
 * are in global token order.  The non-spec subset lists num_decodes rows first, then
 * num_prefills rows; the spec subset follows its own order.  Each subset gathers x, a and b
 * through its own token_indx and scatters out through it; when both subsets are non-empty
 * both token_indx must be given.  Requires
 *   non_spec->num_tokens + spec->num_tokens == num_actual_tokens (GDN_ERR_CONSERVATION) and
 *   num_decodes + num_prefills == non_spec->num_seqs (GDN_ERR_SHAPE).
 * Results equal gdn_conv_update (y in fp32) followed by gdn_recurrent_step on the spec rows and
 * the decode rows, and gdn_chunk_prefill on the prefill rows.
 * workspace: at least gdn_workspace_bytes(layer, non_spec, spec) +
 * gdn_prefill_workspace_bytes(layer, non_spec, num_prefills) bytes, 256-byte aligned.
 */
int gdn_mixed_batch(const gdn_layer_desc* layer, const gdn_layer_params* params, const gdn_pools* pools,
                    const void* x, const void* a, const void* b, int32_t num_actual_tokens,
                    const gdn_rows* non_spec, int32_t num_decodes, int32_t num_prefills, const gdn_rows* spec,
                    void* out, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/*
 * gdn_mixed_batch without a workspace argument, for callers that cannot allocate device
 * memory: a plain C host or a plugin whose framework owns every device allocation and offers
 * no hook for scratch, or a serving loop that must not call cudaMalloc/cudaFree because they
 * can synchronise the device and stall other streams.  The scratch is a fixed device array of
 * GDN_STATIC_WORKSPACE_BYTES (16 MiB) inside the library:
 *   - a batch fits when gdn_workspace_bytes(layer, non_spec, spec) +
 *     gdn_prefill_workspace_bytes(layer, non_spec, num_prefills) is at most 16 MiB.  Without
 *     chunked prefill rows that is 512 tokens of an 8192-channel layer; a prefill row on the
 *     tensor-core path also needs one 123904-byte record per (64-token chunk, v-head), about
 *     3.8 MiB per chunk at 32 v-heads, so on that layer a batch holds prefill rows of a few
 *     chunks at most (one 130-token row is already refused);
 *   - it is reserved on every GPU that loads it and stays reserved until the process exits;
 *   - every call on a device shares it, so calls that may overlap on the GPU race on it;
 *   - it keeps the previous call's contents and is never cleared: no scratch element needs to
 *     start at zero, every element a call reads is written earlier by the same call;
 *   - the first call in each CUDA context (the device's primary context, normally) looks up the
 *     array's device address with that device current (cudaGetSymbolAddress); make that first
 *     call before any stream capture, and do not use this entry point across cudaDeviceReset.
 * The caller still passes inputs and outputs exactly as for gdn_mixed_batch.  Returns
 * GDN_ERR_WORKSPACE when the batch does not fit (nothing is enqueued), GDN_ERR_CUDA when the
 * address lookup fails, and otherwise what gdn_mixed_batch returns for the same arguments.
 * The paper has no counterpart to this entry point.
 */
#define GDN_STATIC_WORKSPACE_BYTES (16u << 20)
int gdn_mixed_batch_static_workspace(const gdn_layer_desc* layer, const gdn_layer_params* params,
                                     const gdn_pools* pools, const void* x, const void* a, const void* b,
                                     int32_t num_actual_tokens, const gdn_rows* non_spec, int32_t num_decodes,
                                     int32_t num_prefills, const gdn_rows* spec, void* out, uint32_t* d_status,
                                     void* stream);

/* ------------------------------------------------------------------------------------------
 * The paged key-value cache of the full-attention layers.
 *
 * A hybrid model interleaves GDN layers with full-attention layers over the same batch of
 * decode, verify and prefill rows.  The attention layers keep their keys and values in pages:
 * fixed blocks of page_size tokens in one pool, listed per sequence in a block table.  Nothing
 * here reads device memory on the host, so a whole step -- reserving pages, appending,
 * attending -- can be captured in a CUDA graph.
 *
 * Page ids <= 0 are NULL: they hold no tokens (no attention sees them, nothing is written).
 * Page 0 is reserved as NULL.  refcount[p] counts the table entries that hold page p; a page is
 * free when it is 0.  Pages are handed out lowest id first, in the order of the rows of a call
 * and of the entries of a row, so the result of every call is determined by its inputs.
 */
typedef struct {
  void* k_pool;          /* [num_pages, num_kv_heads, page_size, head_dim] dtype                    */
  void* v_pool;          /* the same shape                                                          */
  int64_t page_stride;   /* elements from one page to the next in both pools; 0 = dense; else a multiple
                            of page_size * head_dim, below 2^38 (a larger stride lets K and V share
                            one allocation)                                                          */
  int32_t* block_table;  /* [num_table_rows, max_pages] page id of each page_size tokens of a row   */
  int32_t* refcount;     /* [num_pages]; NULL where a call says that it may be                      */
  int32_t num_pages;     /* 2..2^28 (page 0 is NULL)                                                */
  int32_t num_table_rows;
  int32_t max_pages;     /* entries of a table row; max_pages <= 2^20, max_pages * page_size < 2^31  */
  int32_t page_size;     /* tokens of a page: 16, 32, 64, 128 or 256                                */
  int32_t num_kv_heads;  /* Hkv, 1..1024                                                            */
  int32_t head_dim;      /* d, a multiple of 16, <= 256                                             */
  gdn_dtype dtype;       /* GDN_BF16 or GDN_F32: pools, q, k, v and out                             */
} gdn_kv_cache;

/*
 * The rows of one subset of the batch as an attention layer sees them.  query_start_loc and
 * token_indx are those of gdn_rows.  Row n owns table row table_rows[n]; its L =
 * query_start_loc[n+1] - query_start_loc[n] new tokens are the last L of its kv_lens[n] tokens,
 * i.e. token t is at position kv_lens[n] - L + t.  After a verify step that accepted fewer
 * tokens the next step's kv_lens simply counts from the accepted ones.
 * A row with L > max_query_len, kv_lens[n] < L or kv_lens[n] > max_pages * page_size, or a table
 * row out of range is skipped (GDN_STATUS_ROW_RANGE, GDN_STATUS_PAGE_RANGE).
 */
typedef struct {
  int32_t num_seqs;               /* may be 0                                                  */
  int32_t num_tokens;             /* query_start_loc[num_seqs]                                 */
  const int32_t* query_start_loc; /* [num_seqs+1]                                              */
  const int32_t* token_indx;      /* [num_tokens] global token of each local token; NULL = identity */
  const int32_t* table_rows;      /* [num_seqs]; NULL = identity                               */
  const int32_t* kv_lens;         /* [num_seqs]                                                */
  int32_t max_query_len;          /* no row is longer (1 for decode rows, drafts + 1 for verify) */
} gdn_kv_rows;

typedef struct {
  int32_t num_q_heads; /* Hq, a multiple of Hkv; q-head h reads kv-head h / (Hq/Hkv)          */
  float scale;         /* multiplies q.k; <= 0 selects 1/sqrt(d)                              */
  int32_t window;      /* > 0: a query at position p sees keys p-window+1 .. p; <= 0: all up to p */
  int32_t num_sinks;   /* with a window: positions below this stay visible (>= 0)             */
} gdn_attn_desc;

/*
 * Writes the new tokens' keys and values into the rows' pages: position p of row n goes to page
 * block_table[table_rows[n]][p / page_size], slot p % page_size, as bit copies.  Pages must have
 * been reserved; a NULL entry is not written.  With refcount given, a page that several rows
 * hold is not written either (GDN_STATUS_PAGE_SHARED): gdn_kv_fork leaves no row such a page at
 * the end of its tokens.
 *   k, v [num_global_tokens, Hkv, d] dtype, read at token_indx; k_stride, v_stride: elements from
 *   one token to the next (0 = dense), their bytes a multiple of 16 -- slices of one fused
 *   projection need no copy.
 */
int gdn_kv_append(const gdn_kv_cache* cache, const gdn_kv_rows* rows, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, int32_t num_global_tokens, uint32_t* d_status, void* stream);

/*
 * Causal attention of the rows' new tokens over the cache (whose pages already hold them).  The
 * query of q-head h at position p of row n sees the row's key j when j <= p, and (window <= 0 or
 * j > p - window or j < num_sinks), and the page of j is not NULL:
 *   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  s_j = scale q.k_j,  m = max_j s_j,
 * scores, maximum and sums in fp32, rounded once to dtype; a query that sees no key gives 0.  The weights
 * e^(s_j - m) <= 1 go into the second sum in fp32 (GDN_F32, and head dimensions other than 64, 128 and 256), as a
 * pair of bf16 that keeps 16 bits (bf16 rows of up to 64 queries per kv-head), or as one bf16, 2^-8 relative at most
 * (longer bf16 rows: the tensor core's operand): the same token may differ by that between a prompt and a verify row.
 * What a query does not see never reaches its result, whatever it holds (infinities and NaN included).
 *   q, out [num_global_tokens, Hq, d] dtype, read and written at token_indx; q_stride,
 *   out_stride: elements from one token to the next (0 = dense), their bytes a multiple of 16.
 * The cache's refcount is not used and may be NULL.
 * max_query_len and the sizes pick the kernel on the host: rows of few new tokens share the cache's length out to
 * all SMs, long ones take the tensor cores 128 queries at a time.  A bf16 call of 5 rows or more whose num_tokens are
 * less than half of num_seqs * max_query_len goes both ways, a row by its own length; decode rows beside prompts in
 * other calls go the prompts' way and are faster in one of their own (another gdn_kv_rows over the same tokens).
 * workspace: at least gdn_attention_workspace_bytes(attn, cache, rows) bytes, 256-byte aligned
 * (may be NULL when that is 0); it holds the partial results of rows whose cache is split.
 */
int gdn_paged_attention(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows, const void* q,
                        int64_t q_stride, int32_t num_global_tokens, void* out, int64_t out_stride, void* workspace,
                        size_t workspace_bytes, uint32_t* d_status, void* stream);

/* Depends only on the host-side values of the descriptors and on the device; 0 for invalid descriptors. */
size_t gdn_attention_workspace_bytes(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows);

/*
 * Groups of rows that share the beginning of their caches: group g is rows [group_start_loc[g], group_start_loc[g+1]) of
 * the call.  Its rows hold the same pages in the entries of its first prefix_lens[g] tokens, as gdn_kv_fork leaves them
 * (lens may be passed on as they are: of a partly filled last page every row has its own copy, and only whole pages
 * count).  Rows of no group share nothing.
 */
typedef struct {
  int32_t num_groups;             /* 0..65535                                                  */
  const int32_t* group_start_loc; /* [num_groups+1], ascending, within [0, num_seqs]           */
  int32_t* prefix_lens;           /* [num_groups] tokens; read, and by gdn_kv_common_prefix written */
} gdn_kv_groups;

/*
 * gdn_paged_attention over groups of rows, with every group's shared pages read once for all of its rows.  The result is
 * gdn_paged_attention's: the same keys are seen, in the same positions, by the same formula; (m, l, sum) over the
 * shared and over the row's own tokens meet as those of a split row do.
 * Shared are min(prefix_lens[g], kv_lens[n] - L of the rows with new tokens) tokens, down to whole pages, where at least
 * two rows of the group have new tokens; prefix_lens <= 0 shares nothing.  They are read by the table row of the
 * first such row: where the rows' entries differ after all, its pages count.  A row is in one group at most, a token in
 * one row: where the bounds of a group do not ascend or leave the rows, or those of a row do not ascend or leave the
 * tokens (GDN_STATUS_ROW_RANGE), nothing is shared, and rows that are well formed go over their own caches.
 * bf16 rows of more than 256 queries per kv-head (d = 64, 128; 128 at d = 256; max_query_len decides) go over their
 * whole caches as in gdn_paged_attention, whatever the groups are: they fill the tensor cores by themselves.  Weights go
 * into the second sum with the bits that gdn_paged_attention keeps of them: 16 of bf16 rows (d = 64, 128, 256) in calls
 * without a row of more than 64 queries per kv-head, and of all rows in calls that it would take both ways; else 8 of bf16
 * rows of these head dimensions, 24 of all others.
 * Sharing pays from a few thousand tokens on for groups of four rows or more, hardly for pairs, and not for rows that have as
 * many tokens of their own; then a call takes up to 2.3 times as long as in gdn_paged_attention, which finds the other rows'
 * pages in the L2.
 * workspace: at least gdn_shared_attention_workspace_bytes(attn, cache, rows, groups) bytes, 256-byte aligned; it holds
 * the plan (a copy for each CTA that makes its own), two states of (2 + d) fp32 per query and head, and partial results.
 */
int gdn_shared_attention(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows,
                         const gdn_kv_groups* groups, const void* q, int64_t q_stride, int32_t num_global_tokens, void* out,
                         int64_t out_stride, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/* Depends only on the host-side values of the descriptors and on the device; 0 for invalid descriptors. */
size_t gdn_shared_attention_workspace_bytes(const gdn_attn_desc* attn, const gdn_kv_cache* cache, const gdn_kv_rows* rows,
                                            const gdn_kv_groups* groups);

/*
 * Finds what groups share: prefix_lens[g] = page_size x the largest E for which the rows of group g that have new
 * tokens agree in their table entries [0, E) (NULL entries agree with one another) and E whole pages lie before the new
 * tokens of each.  0 for a group without such rows.  Rows that gdn_paged_attention would skip do not count.
 * The cache's pools are not read, its refcount is not used and may be NULL.
 */
int gdn_kv_common_prefix(const gdn_kv_cache* cache, const gdn_kv_rows* rows, const gdn_kv_groups* groups,
                         uint32_t* d_status, void* stream);

/* ------------------------------------------------------------------------------------------
 * Rotary positions.
 *
 * Pair i < rotary_dim / 2 of a head is (x[i], x[i + rotary_dim/2]) in the half layout and (x[2i], x[2i+1]) in the
 * interleaved one; at position p it becomes
 *   (x cos a - y sin a, y cos a + x sin a) * magnitude,   a = p * f_i,
 * in fp32, rounded once to the dtype; values from rotary_dim on are copied.  A negative position turns back, so the same
 * call at -p is the transposed map: the gradient of the inputs, and (magnitude 1) the inverse.
 * Frequencies are 64-bit binary fractions of a turn: the product of a position and a stored fraction is exact modulo a turn and
 * then rounded by 2^-33 of a turn.  The fractions of gdn_rope_turns are made in doubles, off by 2^-53 of a turn at most (of
 * frequencies up to 1 radian a position), which the position multiplies: 2^-33 of a turn at 2^20, 2^-22 at 2^31.
 */
typedef enum { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout;

typedef struct {
  const uint64_t* turns; /* device, [rotary_dim/2]: f_i / (2 pi) in units of 2^-64, modulo 1        */
  int32_t rotary_dim;    /* even, 2..head_dim                                                       */
  int32_t layout;        /* gdn_rope_layout                                                         */
  float magnitude;       /* multiplies cosine and sine; 0 selects 1                                 */
} gdn_rope_desc;

/*
 * How the frequencies f_i = base^(-2i/rotary_dim) are scaled for contexts longer than the one that was trained on:
 *   PLAIN   not at all;
 *   LINEAR  f_i / factor;
 *   NTK     base * factor^(r/(r-2)) in base's place, r = rotary_dim > 2: the slowest pair as LINEAR, the fastest as PLAIN;
 *   BANDS   pairs that turn `high` times or more over original_len are kept, those of `low` or fewer are divided by factor,
 *           and between them w f_i + (1-w) f_i / factor with w linear in the number of turns (0: low 1, high 4);
 *   RAMP    as BANDS, with w linear in the pair's number between the pair that turns `high` times (rounded down, at least
 *           0) and the one that turns `low` times (rounded up, at most r-1) (0: low 1, high 32); magnitude 0.1 ln factor + 1,
 *           for factors up to 1 it is 1.
 */
typedef enum {
  GDN_ROPE_PLAIN = 0,
  GDN_ROPE_LINEAR = 1,
  GDN_ROPE_NTK = 2,
  GDN_ROPE_BANDS = 3,
  GDN_ROPE_RAMP = 4
} gdn_rope_scaling;

typedef struct {
  int32_t rotary_dim;  /* even, 2..256                                 */
  int32_t scaling;     /* gdn_rope_scaling                             */
  double base;         /* > 1                                          */
  double factor;       /* > 0; not used by PLAIN                       */
  double original_len; /* BANDS, RAMP: > 0                             */
  double low, high;    /* BANDS, RAMP: 0 < low < high; 0 selects the default */
} gdn_rope_freq;

/* Host only: writes the rotary_dim/2 fractions for gdn_rope_desc to `turns` (host) and, where not NULL, the magnitude.
 * gdn_rope_turns_of takes `count` (1..128) frequencies in radians a position instead. */
int gdn_rope_turns(const gdn_rope_freq* freq, uint64_t* turns, float* magnitude);
int gdn_rope_turns_of(const double* radians, int32_t count, uint64_t* turns);

/*
 * Turns the heads of x [num_tokens, num_heads, head_dim] by positions[token] into out (the same shape).  Tokens behind
 * num_tokens are neither read nor written.  out may be x (with one stride), or other columns of the same wider
 * tensor; any other overlap is refused (GDN_ERR_SHAPE).
 *   num_heads 1..65535, head_dim a multiple of 16, <= 256; x_stride, out_stride: elements from one token to the next
 *   (0 = dense), their bytes a multiple of 16.
 */
int gdn_rope(const gdn_rope_desc* rope, int32_t num_heads, int32_t head_dim, gdn_dtype dtype, const int32_t* positions,
             int32_t num_tokens, const void* x, int64_t x_stride, void* out, int64_t out_stride, void* stream);

/*
 * gdn_kv_append with the rotation on the way, at the positions that the rows' kv_lens give: the new tokens' keys are
 * turned into their pages, their values copied, and the q heads of the same tokens turned from q to q_out (which may be q).
 * Everything that gdn_kv_append says holds; q_out is written for every token of a well-formed row, wherever its page
 * is.  num_q_heads = 0: keys and values only.
 *   q, q_out [num_global_tokens, num_q_heads, d], read and written at token_indx (which then names no token twice);
 *   q_out overlaps neither k nor v, and q only as in gdn_rope.
 */
int gdn_kv_append_rope(const gdn_kv_cache* cache, const gdn_kv_rows* rows, const gdn_rope_desc* rope, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, int32_t num_q_heads, const void* q,
                       int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_global_tokens, uint32_t* d_status,
                       void* stream);

/*
 * Makes room: for each of the `count` table rows listed, the entries of tokens
 * [from_lens[i], to_lens[i]) that begin a page -- entries ceil(from/page_size) ..
 * ceil(to/page_size)-1 -- and hold no page get a free one (refcount 1).  A row gets all of them
 * or none: when the needs of the rows up to and with it exceed the free pages it is left as it
 * was (GDN_STATUS_NO_PAGES).  table_rows must not repeat.  NULL table_rows = identity.
 * workspace (reserve, fork, compact): at least gdn_kv_workspace_bytes(cache, count) bytes,
 * 256-byte aligned.
 */
int gdn_kv_reserve(const gdn_kv_cache* cache, int32_t count, const int32_t* table_rows, const int32_t* from_lens,
                   const int32_t* to_lens, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/*
 * Gives pages back: entries [first_page[i], last_page[i]) of each listed table row become NULL
 * and their pages lose a holder.  NULL first_page = 0, NULL last_page = max_pages, so both NULL
 * frees whole rows; a finished window's old pages or a rolled-back tail are given back by range.
 * table_rows must not repeat.
 */
int gdn_kv_release(const gdn_kv_cache* cache, int32_t count, const int32_t* table_rows, const int32_t* first_page,
                   const int32_t* last_page, uint32_t* d_status, void* stream);

/*
 * Forks sequences: table row dst_rows[i] becomes a holder of the first lens[i] tokens of
 * src_rows[i].  Pages that these tokens fill are shared; the tokens of a partly filled last page
 * are copied into a free page, so both rows can append.  NULL entries stay NULL.  A dst row must
 * hold no page in the entries it gets (else it is skipped, GDN_STATUS_PAGE_RANGE); dst rows must
 * be distinct and not among the src rows.  When the free pages do not cover the needs of the
 * rows up to and with i, row i is skipped (GDN_STATUS_NO_PAGES).  A hybrid model's sequence also
 * has GDN state: gdn_copy_slots copies that.
 */
int gdn_kv_fork(const gdn_kv_cache* cache, int32_t count, const int32_t* src_rows, const int32_t* dst_rows,
                const int32_t* lens, void* workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/* Copies page src_pages[i] onto dst_pages[i] in both pools (pairs with a NULL side are skipped;
 * dst pages distinct and not among the src pages).  block_table and refcount are not used (may be NULL). */
int gdn_kv_copy_pages(const gdn_kv_cache* cache, int32_t count, const int32_t* src_pages, const int32_t* dst_pages,
                      uint32_t* d_status, void* stream);

/*
 * Moves the M live pages (refcount > 0) to ids 1..M, so that the pool's tail is free in one
 * piece: the live pages with ids above M, lowest first, go to the free ids up to M, lowest
 * first.  Every entry of the block table and refcount follow.  num_live (device, may be NULL)
 * receives M.  Pages must be moved while nothing else uses the cache (one stream orders that).
 */
int gdn_kv_compact(const gdn_kv_cache* cache, int32_t* num_live, void* workspace, size_t workspace_bytes,
                   uint32_t* d_status, void* stream);

/* Workspace of gdn_kv_reserve and gdn_kv_fork over `count` rows and of gdn_kv_compact (any count);
 * 0 for an invalid descriptor or a negative count. */
size_t gdn_kv_workspace_bytes(const gdn_kv_cache* cache, int32_t count);

/*
 * Copies GDN state: slot src_slots[i] of both pools (conv history and SSM state; conv_pool may be
 * NULL) onto dst_slots[i].  A NULL source reads as zeros, a NULL destination is not written, as
 * in every call of this library; dst slots distinct and not among the src slots.
 */
int gdn_copy_slots(const gdn_layer_desc* layer, const gdn_pools* pools, int32_t count, const int32_t* src_slots,
                   const int32_t* dst_slots, uint32_t* d_status, void* stream);

/* Static text for a gdn_error value. */
const char* gdn_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
