/*
 * dex.h -- C ABI of the GB300 (sm_103a) Depth Exploration Decoding library.
 *
 * Depth Exploration Decoding (DEX), "Depth Exploration for LLM Decoding"
 * (arXiv 2606.29223): each expand-commit-collapse cycle expands a depth-position
 * lattice of exploration tokens (section 3.2, Figure 2), decodes every node with
 * depth-coupled sampling (section 3.3, Appendix C.1 Algorithm 2), commits the
 * final-depth token y = u_{N-1}, keeps the shallowest anchor branch with u_k = y and
 * collapses the lattice onto it (Algorithm 1, expand / DECS / insert /
 * validate_and_commit / collapse / advance).
 *
 * On one GPU, a round batches every live lattice node of every sequence into one
 * pass: the decoder-layer slice (d_{k-1}, d_k] of each node's stage with
 * lattice-masked attention, the shared exit head (final RMSNorm + LM head) over all
 * nodes, DECS, and the host-side commit that decides the next round.
 *
 * Conventions
 *  - Every entry point returns DEX_OK (0) or a negative dex_status; dex_strerror()
 *    names it.  A failing call leaves the handle usable unless it returns DEX_ECUDA.
 *  - "device" pointers are CUDA global-memory addresses on the handle's device;
 *    "host" pointers are ordinary process memory.  Weights are bf16, row-major
 *    [out_features][in_features], and stay owned by the caller, who keeps them alive
 *    until dex_free().  The library owns its KV caches and workspaces, allocated in
 *    dex_init() and released by dex_free().
 *  - Arithmetic: bf16 weights on the tensor cores with fp32 accumulation; activations
 *    enter every GEMM as a pair of bf16 operands (x ~= hi + lo, about 17 significant
 *    bits), hidden states are fp32, and the K/V caches hold fp16 (11 significant bits,
 *    8x finer than bf16 at the same two bytes) read into fp32 attention arithmetic.
 *  - All work is issued on the stream given to dex_init().  Calls returning host data
 *    synchronise that stream.  A handle is not thread-safe.
 *  - Positions are absolute token indices starting at 0; the commit position p_c is
 *    the index of the next token to be committed.
 */
#ifndef DEX_H_
#define DEX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dex_status {
  DEX_OK = 0,
  DEX_EINVAL = -1,     /* a bad argument (null pointer, size out of range, unsupported shape) */
  DEX_ENOMEM = -2,     /* device or host allocation failed */
  DEX_ECUDA = -3,      /* a CUDA runtime or driver call failed; the handle should be freed */
  DEX_ECAPACITY = -4,  /* a sequence would exceed max_ctx or max_new */
  DEX_ETIMEOUT = -5,   /* a bounded device wait gave up (kernel reported a stalled pipeline) */
  DEX_ESTATE = -6,     /* call out of order (e.g. dex_step before dex_prefill) */
  DEX_ENODEV = -7,     /* no usable sm_103 device */
  DEX_ERANGE = -8      /* a linear layer's split-K partial sum was not finite or reached 2^30 in
                          magnitude (the range of the exact fixed-point segment sum); the
                          round's results are void, the handle stays usable */
} dex_status;

/* Model description (Llama-style pre-norm decoder, no biases, SwiGLU FFN, RoPE).
 * The residual-branch scale of the method's synthetic models is expected folded
 * into wo and wd.  layers points to a HOST array of n_layers * 9 DEVICE pointers,
 * per layer in the order: attn_norm[d], wq[H*hd][d], wk[KVH*hd][d], wv[KVH*hd][d],
 * wo[d][H*hd], ffn_norm[d], wg[d_ff][d], wu[d_ff][d], wd[d][d_ff].  The array is
 * copied by dex_init().  Constraints: d_model % 128 == 0 and <= 8192, head_dim in {64, 128},
 * n_heads % n_kv_heads == 0, n_heads*head_dim and n_kv_heads*head_dim multiples of 128,
 * d_ff a multiple of 8 (>= 64), every weight 16-byte aligned (DEX_EINVAL otherwise). */
typedef struct dex_model {
  int32_t n_layers, d_model, n_heads, n_kv_heads, head_dim, d_ff, vocab;
  float rms_eps, rope_theta;
  const void* embed;        /* device, [vocab][d_model] bf16 */
  const void* final_norm;   /* device, [d_model] bf16 */
  const void* lm_head;      /* device, [vocab][d_model] bf16 (== embed for a tied head) */
  const void* const* layers;/* host array of n_layers*9 device pointers (see above) */
  /* Inducing adapters (Appendix C.2), or NULL: a host array of (n_X - 1) * 5 device pointers,
   * one adapter per non-final depth X[k], k < n_X - 1, of the X given to dex_init, in the
   * order g[d] (RMSNorm gain), w1[2d][d], b1[2d], w2[d][2d], b2[d] (bf16), with
   * adapter_alpha a host array of the n_X - 1 scalar gates.  The node of a non-final stage
   * is decoded from h + alpha (w2 SiLU(w1 RMSNorm(h; g) + b1) + b2); the final depth never is. */
  const void* const* adapters;
  const float* adapter_alpha;
} dex_model;

/* Decode setup.  sample=0: greedy (ties -> lowest id); sample=1: Gumbel-max at
 * temperature tau with noise rows keyed by (seed, sequence, target position).
 * decs=1 enables DECS masking (Algorithm 2); decs=0 decodes every node
 * independently.  debug_logits=1 keeps the fp32 logits of the last round's nodes
 * for dex_debug_logits() (costs vocab*4 bytes per node of device memory). */
typedef struct dex_decode_cfg {
  int32_t batch;        /* independent sequences, 1..64 */
  int32_t max_ctx;      /* capacity in positions per sequence (prompt + new + N), <= 4096 */
  int32_t max_new;      /* tokens to commit per sequence */
  int32_t sample;
  float tau;
  uint64_t seed;
  int32_t decs;
  int32_t debug_logits;
  int32_t max_branch;   /* 0: the full lattice; k > 0: a sparse lattice whose nodes speculate at
                           most k tokens ahead of the commit (k position moves on their path;
                           the final-depth commit, hence the token stream, is unchanged) */
} dex_decode_cfg;

typedef struct dex_handle dex_handle;

/* Create a handle for exploration set X = {d_0 < ... < d_{N-1} = n_layers}
 * (Definition 4), 1 <= N <= 10.  stream: a cudaStream_t (NULL = legacy default).
 * Allocates every device buffer the decode needs.  Errors: DEX_EINVAL for a bad
 * model/X/cfg, DEX_ENODEV, DEX_ENOMEM, DEX_ECUDA. */
int dex_init(const dex_model* model, const int32_t* X, int32_t n_X, const dex_decode_cfg* cfg,
             void* stream, dex_handle** out);

/* init(x, {E_k}) of Algorithm 1 for sequence seq: writes the committed KV cache of
 * prompt positions 0..n_tokens-2 and makes the last prompt token the root input
 * (state q = 0, empty explore buffer).  tokens: HOST int32 [n_tokens], n_tokens >= 1,
 * ids in [0, vocab).  Resets the sequence's decode state. */
int dex_prefill(dex_handle* h, int32_t seq, const int32_t* tokens, int32_t n_tokens);

/* One DEX round over every prefilled, unfinished sequence: expand the level-q nodes,
 * exit head + DECS, insert, and -- for sequences whose anchor reached the final
 * depth -- validate_and_commit and collapse.  out_tokens / n_committed: HOST int32
 * [batch]; n_committed[b] is 1 when sequence b committed out_tokens[b] this round,
 * else 0.  Returns DEX_ESTATE when no sequence is active. */
int dex_step(dex_handle* h, int32_t* out_tokens, int32_t* n_committed);

/* Run dex_step until every prefilled sequence has committed max_new tokens.
 * out: HOST int32 [batch][max_new]; rows of sequences never prefilled are left as is. */
int dex_generate(dex_handle* h, int32_t* out);

/* Plain autoregressive round on the same kernels (one node per sequence through all
 * layers, exit at the final depth): the lossless reference DEX must equal.  Same
 * outputs as dex_step.  Must not be mixed with dex_step on a sequence between two
 * dex_prefill calls (DEX_ESTATE). */
int dex_ar_step(dex_handle* h, int32_t* out_tokens, int32_t* n_committed);

/* Run dex_ar_step until every prefilled sequence has max_new tokens; out as dex_generate. */
int dex_ar_generate(dex_handle* h, int32_t* out);

/* Counters since dex_init / the last dex_reset_stats. */
typedef struct dex_stats {
  int64_t rounds;           /* rounds executed (DEX or AR) */
  int64_t commits;          /* committed tokens over all sequences */
  int64_t nodes;            /* lattice nodes evaluated */
  int64_t max_round_nodes;  /* largest single-round node batch */
  int64_t layer_passes;     /* sum over rounds of d of the deepest live stage */
  int64_t node_layers;      /* sum over nodes of the layer count of their stage */
  int64_t depth_charge;     /* sum over committed tokens of d_{k*} (Eq. 12's W) */
  int64_t kstar_hist[16];   /* committed tokens by accepted branch k* */
  int64_t weight_bytes;     /* algorithmic weight bytes streamed (each live layer once per round) */
  int64_t kv_bytes;         /* algorithmic committed + branch KV bytes read */
  int64_t h2d_bytes, d2h_bytes;
  int64_t kernel_launches;
  int64_t gemm_launches;    /* linear-layer GEMM launches (the dominant kernel) */
  int64_t gemm_bytes;       /* their algorithmic bytes (weights + activations in/out) */
  double ms_gemm;           /* summed CUDA-event duration of those launches (timing >= 2) */
  double ms_expand, ms_exit, ms_collapse, ms_host;  /* phase split (timing >= 1) */
  int64_t attn_launches;    /* lattice-attention launches */
  double ms_attn;           /* summed CUDA-event duration of those launches (timing >= 2) */
} dex_stats;

int dex_get_stats(const dex_handle* h, dex_stats* out);
int dex_reset_stats(dex_handle* h);

/* timing: 0 off; 1 = CUDA events around the expansion / exit+DECS / collapse phases of
 * each round; 2 = also around every linear-layer GEMM and attention launch (adds events,
 * which also stop programmatic-dependent-launch overlap across them); 3 = level 1
 * plus per-CTA clock records of the GEMM launches that follow (diagnostics: only when the
 * environment variable DEX_TIMELINE names a file, which dex_free() writes; the first
 * DEX_TIMELINE_LAUNCHES launches, default 512, are kept). */
int dex_set_timing(dex_handle* h, int32_t level);

/* Lattice nodes of the most recent round, in evaluation order: HOST int32
 * [max_rows][8] = {seq, heap index, stage, plen, target position, token, prior
 * count, input position}.  *rows_out receives the number of nodes. */
int dex_last_round_nodes(const dex_handle* h, int32_t* host_out, int32_t max_rows, int32_t* rows_out);

/* fp32 logits of the most recent round's nodes (same order as dex_last_round_nodes),
 * before masking and noise.  Needs cfg.debug_logits = 1.  host_out: HOST float
 * [max_rows][vocab]. */
int dex_debug_logits(dex_handle* h, float* host_out, int32_t max_rows, int32_t* rows_out);

const char* dex_strerror(int code);
void dex_free(dex_handle* h);

/* Failure-path self-test (diagnostics; the paper has no counterpart).  Runs the bounded
 * mbarrier wait that every pipeline of the library uses against a barrier that nothing
 * completes, with a limit of limit_us microseconds (1..1000000), on the handle's stream,
 * and reads the device error flag back exactly as a decode round does.  Returns
 * DEX_ETIMEOUT when the wait gave up as designed (the flag is then cleared and the handle
 * stays usable), DEX_OK if it did not, DEX_EINVAL for a bad argument.  Synchronises the
 * stream.  Allocation failures of dex_init can likewise be injected on the host: with the
 * environment variable DEX_FAIL_ALLOC_AT=k set, the k-th device or pinned-host allocation
 * of dex_init reports failure, and dex_init returns DEX_ENOMEM after releasing everything
 * it had allocated. */
int dex_selftest_stall(dex_handle* h, int32_t limit_us);

/* ---- kernels in isolation ------------------------------------------------------ */

/* One node of an isolated exit-head + DECS call. */
typedef struct dex_exit_node {
  int32_t seq;          /* sequence id (Gumbel row key) */
  int32_t target_pos;   /* absolute position being predicted (Gumbel row key) */
  int32_t unmasked;     /* 1 for the final-depth reference: no DECS mask */
  int32_t prior_off;    /* first prior token in the priors array */
  int32_t n_prior;      /* number of prior tokens (shallower proposals of the slot chain) */
} dex_exit_node;

/* Exit head + DECS over n nodes (section 3.3, Appendix C.1 Algorithm 2, exit head of
 * Appendix C.2): token[i] = argmax_v score_i(v), with logits z = RMSNorm(h_i; g) W^T,
 * score = -inf for masked priors, else z (greedy) or z / tau + G(seed, seq, pos, v).
 * h: device bf16 [n][d]; final_norm: device bf16 [d]; lm_head: device bf16
 * [vocab][d]; nodes: device [n]; priors: device int32; tokens: device int32 [n];
 * logits: device fp32 [n][vocab] or NULL.  1 <= n <= 256, d % 128 == 0, d <= 8192.
 * Allocates its scratch with the stream-ordered allocator; stream-ordered, no sync, so
 * device-side failures cannot be returned: if a bounded wait inside the GEMM gives up
 * (the decoder would report DEX_ETIMEOUT), every token of the call is written as -1. */
int dex_exit_head_decs(const void* h, int32_t n, int32_t d, const void* final_norm, float rms_eps,
                       const void* lm_head, int32_t vocab, const dex_exit_node* nodes,
                       const int32_t* priors, int32_t sample, float tau, uint64_t seed,
                       int32_t* tokens, float* logits, void* stream);

/* Size of the fixed device scratch of dex_exit_head_decs_noalloc: 32 MiB per GPU. */
#define DEX_NOALLOC_SCRATCH_BYTES (32u << 20)

/* The exit head + DECS of dex_exit_head_decs, for callers that must not allocate device
 * memory during the call (for example code running under another component's stream
 * capture or allocator, or with a memory budget fixed at start-up).  The paper has no
 * counterpart: this is a deployment convenience of this library.
 * It runs the GEMM on one CTA per SM (a deeper weight ring; its split-K partials then fit
 * the fixed scratch) where dex_exit_head_decs uses two, so the k-segment split and hence
 * the last bits of the logits may differ between the two entry points; each is within the
 * same tolerance of the fp64 exit head, and tokens agree wherever the decision margin is
 * not within rounding of zero.  A stalled bounded wait writes every token as -1, as in
 * dex_exit_head_decs (the stall flag lives in the scratch and is cleared by the next call).
 * Scratch comes from one file-scope device array of DEX_NOALLOC_SCRATCH_BYTES that every
 * GPU loading the library keeps until the process exits; no cudaMalloc/cudaFree or other
 * allocating routine is called.  The array's device address is looked up on the first call
 * made on each device (with that device current), so make that first call before any
 * stream capture.  Calls share the array: calls that may overlap on the GPU (different
 * streams, or several host threads) race and must be serialised by the caller.  Returns
 * DEX_ECAPACITY, doing nothing, when the call's scratch (hidden tile, RMSNorm partials,
 * split-K partials) would exceed DEX_NOALLOC_SCRATCH_BYTES; other arguments and errors as
 * dex_exit_head_decs. */
int dex_exit_head_decs_noalloc(const void* h, int32_t n, int32_t d, const void* final_norm, float rms_eps,
                               const void* lm_head, int32_t vocab, const dex_exit_node* nodes,
                               const int32_t* priors, int32_t sample, float tau, uint64_t seed,
                               int32_t* tokens, float* logits, void* stream);

/* Geometry of the KV caches used by dex_kv_collapse.  committed: [batch][n_layers][2]
 * [n_kv_heads][max_ctx][head_dim] bf16; pool: [batch][n_slots][n_layers][2]
 * [n_kv_heads][head_dim] bf16 (one slot per sampling-slot chain). */
typedef struct dex_kv_geom {
  int32_t batch, n_layers, n_kv_heads, head_dim, max_ctx, n_slots;
} dex_kv_geom;

/* Copy the branch KV of a surviving slot chain into the committed cache at its
 * position (the collapse of section 3.2 for the new anchor path). */
typedef struct dex_copy_job {
  int32_t seq, slot, pos, n_layers;   /* layers 0..n_layers-1 of slot -> position pos */
} dex_copy_job;

/* Vectorised gather/scatter of n_jobs copy jobs (device array, 0 <= n_jobs <= 65535).
 * committed / pool: device, 16-byte aligned, with geom's layouts; head_dim a multiple of 8.
 * A job with seq outside [0, batch), slot outside [0, n_slots), pos outside [0, max_ctx) or
 * n_layers outside [1, n_layers] is skipped without any memory access.  rejected: device
 * int32 or NULL; when given, the call zeroes it (stream-ordered) and adds one per skipped
 * job.  Stream-ordered, no sync.  DEX_EINVAL for a bad geometry or pointer. */
int dex_kv_collapse(void* committed, const void* pool, const dex_kv_geom* geom,
                    const dex_copy_job* jobs, int32_t n_jobs, int32_t* rejected, void* stream);

/* ---- paged K/V cache: append and shared-prefix attention --------------------------- */

typedef enum dex_dtype { DEX_DT_BF16 = 0, DEX_DT_FP16 = 1, DEX_DT_FP32 = 2 } dex_dtype;

/* One layer of a paged K/V cache.  A page holds page_size consecutive positions of one
 * sequence, head-major like the committed cache: [2 (K, V)][n_kv_heads][page_size][head_dim].
 * Position p of sequence b is row p % page_size of page table[b * table_stride + p / page_size].
 * Pages lie page_stride elements apart, so the layers of a model can share one allocation
 * (page_stride = n_layers * 2 * n_kv_heads * page_size * head_dim, pages offset to the layer).
 * Several sequences may name the same page (a shared prefix).
 * Constraints (DEX_EINVAL otherwise): head_dim 64 or 128; page_size 16, 32, 64, 128 or 256;
 * dtype DEX_DT_BF16 or DEX_DT_FP16; pages 16-byte aligned, n_pages >= 1; page_stride a multiple of 8
 * and at least one page; n_kv_heads and batch 1 .. 1024; table_width >= 1, table_width * page_size <=
 * 2^31 - 512; table_stride >= table_width.  A call takes at most 2^23 tokens. */
typedef struct dex_paged_kv {
  void* pages;            /* device, bf16 or fp16 */
  const int32_t* table;   /* device, int32 [batch][table_stride] page ids */
  int64_t page_stride;    /* elements between pages */
  int32_t n_pages, page_size, n_kv_heads, head_dim;
  int32_t batch, table_width, table_stride, dtype;
} dex_paged_kv;

/* The tokens of one dex_paged_append call.  q (may be NULL, with q_out), k and v: device,
 * [n_tokens][heads][head_dim] in in_dtype (the cache's type or DEX_DT_FP32), rows of one token
 * contiguous, tokens *_stride elements apart (slices of a fused projection are fine).  q_out:
 * device, in the cache's type; it may be q itself when in_dtype is the cache's type and the
 * strides agree.  Every pointer 16-byte aligned, every stride a multiple of 16 bytes. */
typedef struct dex_append_args {
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int32_t* seq;       /* device [n_tokens]: sequence, -1 for a padding token */
  const int32_t* pos;       /* device [n_tokens]: cache position */
  const int32_t* rope_pos;  /* device [n_tokens]: rotation position, or NULL for pos */
  int32_t n_tokens, n_heads, in_dtype;
  float rope_theta;         /* >= 1, or 0 to store k and q unrotated */
} dex_append_args;

/* Append n_tokens keys and values to a paged cache, rotating k (and q into q_out) on the way:
 * the pair (x_j, x_{j + head_dim/2}) turns by rope_pos * theta^(-2j / head_dim), in fp32 with the
 * angle reduced exactly, rounded once to the cache's type.  A token with seq -1 is skipped; one
 * whose sequence, position or page id is out of range is skipped without any access to the cache
 * and counted in rejected.  A skipped token's row of q_out is left as it was.  Two tokens of
 * one call must not name the same cache row.  rejected: device int32 or NULL; when given, the
 * call zeroes it (stream-ordered) and adds one per rejected token.  Runs on the current
 * device; stream-ordered, no allocation, no sync, capturable.  n_tokens 0 is a no-op. */
int dex_paged_append(const dex_paged_kv* kv, const dex_append_args* a, int32_t* rejected, void* stream);

/* One dex_prefix_attention call.  The queries of sequence b are tokens q_start[b] ..
 * q_start[b+1]-1 and stand at its last positions: query i of n at p = seq_len[b] - n + i
 * (seq_len counts the prefix and the queries' own positions, already appended).  It sees the
 * positions 0..p, or with tree_mask every position before seq_len[b] - n and, of the last n,
 * position seq_len[b] - n + j where bit j of its word is set (n <= 64).  A query that sees
 * nothing gets zeros and lse -inf.  Query head h reads K/V head h / (n_heads / n_kv_heads).
 * prefix_len is a promise: the positions below it hold the same keys and values for every
 * sequence with queries, and every such sequence's table names them (usually the same pages).
 * Where it pays they are read once for the whole batch, through prefix_table (NULL: row 0 of the
 * cache's table, which has to name them then even if sequence 0 has no queries).  A query at a position
 * below prefix_len still sees no position beyond its own. */
typedef struct dex_attention_args {
  const void* q;               /* device, cache's type, [n_tokens][n_heads][head_dim] */
  void* out;                   /* device, cache's type, [n_tokens][n_heads][head_dim] */
  float* lse;                  /* device [n_tokens][n_heads] or NULL: log of the softmax denominator */
  int64_t q_stride, out_stride;/* elements between tokens (a multiple of 8) */
  const int32_t* q_start;      /* device [batch + 1], non-decreasing, within 0..n_tokens */
  const int32_t* seq_len;      /* device [batch] */
  const int32_t* prefix_table; /* device [ceil(prefix_len / page_size)] page ids or NULL */
  const uint64_t* tree_mask;   /* device [n_tokens] or NULL */
  int32_t n_tokens, n_heads;
  int32_t max_q;               /* no sequence has more queries than this (<= 64 with tree_mask) */
  int32_t prefix_len;          /* >= 0 */
  float scale;                 /* of the scores, usually 1 / sqrt(head_dim); below 2^127 in size */
} dex_attention_args;

/* Bits a call ORs into *status (device int32, cleared by the caller). */
#define DEX_ATTN_BAD_PAGE 1    /* a page id in use is outside [0, n_pages) */
#define DEX_ATTN_BAD_RANGE 2   /* a sequence's q_start or seq_len is out of range */
#define DEX_ATTN_TIMEOUT 4     /* a bounded device wait gave up */

/* Device scratch that dex_prefix_attention needs for these sizes (host call, no GPU work; reads the
 * integer fields only).  Depends on n_tokens, n_heads, max_q, prefix_len and the cache's
 * geometry, not on the lengths. */
int dex_prefix_attention_workspace(const dex_paged_kv* kv, const dex_attention_args* a, size_t* bytes);

/* Attention of a ragged batch of queries over a paged cache whose sequences share their first
 * prefix_len positions.  Scores, softmax statistics and sums are fp32; the probabilities enter the
 * second product in the cache's type.  Rows of out and lse that belong to no sequence are
 * left as they were; out must not overlap q.  Keys and values at positions below seq_len, and with
 * prefix_len > 0 below that, must be finite, seen by a query or not; what pages hold beyond is never
 * used.  The lengths must not change while the call runs.  A page id that is out of range is never followed: the rows that see
 * a position on such a page, in the table it is read through, become NaN, all others are unaffected, and status gets
 * DEX_ATTN_BAD_PAGE.  A sequence whose seq_len is negative or beyond the
 * table gets NaN rows, one whose queries exceed max_q or n_tokens is skipped, both with DEX_ATTN_BAD_RANGE.
 * workspace: device, 256-byte aligned, at least the bytes dex_prefix_attention_workspace gives
 * (DEX_ECAPACITY otherwise); calls that may overlap on the GPU need workspaces of their own.
 * Constraints: the cache's, n_heads a multiple of n_kv_heads with at most 128 query heads per
 * K/V head, q and out 16-byte aligned, prefix_len within the table, and (n_tokens * (n_heads /
 * n_kv_heads) / 256 + batch + 2) * n_kv_heads * (table_width * page_size / 64 + 6) < 2^31.  Runs on the current device;
 * stream-ordered, no allocation, no sync, capturable: lengths, tables and masks are read
 * on the device, so a captured call can be replayed on new ones. */
int dex_prefix_attention(const dex_paged_kv* kv, const dex_attention_args* a, void* workspace, size_t workspace_bytes,
                         int32_t* status, void* stream);

/* One dex_attention_mass call.  Queries as in dex_attention_args, causal; of a sequence with n of them the last
 * min(n, window) count.  lse is what dex_prefix_attention wrote for the same queries, cache and scale (rows of
 * queries that do not count are not read). */
typedef struct dex_mass_args {
  const void* q;               /* device, cache's type, [n_tokens][n_heads][head_dim] */
  const float* lse;            /* device [n_tokens][n_heads] */
  float* mass;                 /* device, position j of K/V head g of sequence b at (b * n_kv_heads + g) * mass_stride + j */
  int64_t q_stride;            /* elements between tokens (a multiple of 8) */
  int64_t mass_stride;         /* at least table_width * page_size */
  const int32_t* q_start;      /* device [batch + 1], non-decreasing, within 0..n_tokens */
  const int32_t* seq_len;      /* device [batch] */
  int32_t n_tokens, n_heads;
  int32_t window;              /* >= 1 */
  int32_t first;               /* >= 0: positions below it are not looked at */
  int32_t accumulate;          /* 0: mass is set, 1: added to */
  float scale;                 /* of the scores, as given to dex_prefix_attention */
} dex_mass_args;

/* The attention weight that cached positions receive:
 *   mass[b][g][j] (+)= sum_i sum_h exp(scale q_ih . k_jg - lse_ih),   first <= j < seq_len[b],
 * over the queries i of sequence b that count and see position j and the query heads h of K/V head g.  Scores and
 * sums are fp32, in an order that depends on sizes and lengths alone.  A query whose lse is -inf adds nothing; a NaN (in
 * lse, or in q or k at a position that it sees) makes the masses that it enters NaN.  Positions at or beyond seq_len, sequences
 * without queries and those named by DEX_ATTN_BAD_RANGE are left as they were: a seq_len that is negative or beyond the
 * table, a q_start that decreases or leaves 0..n_tokens.  Masses of positions on a page whose id is out of range are NaN,
 * with DEX_ATTN_BAD_PAGE.  What pages hold at or beyond seq_len, and below first, is never used.  DEX_ATTN_TIMEOUT: a bounded
 * device wait gave up, masses are void.  Constraints: the cache's, n_heads a multiple of n_kv_heads with at most 128 query heads
 * per K/V head, q 16-byte aligned, q_stride at least n_heads * head_dim and below 2^38 (with several tokens), and
 * (table_width * page_size / 256 + 1) * batch * n_kv_heads < 2^30.  Runs on the current device;
 * stream-ordered, no allocation, no workspace, no sync, capturable (lengths and tables are read on the device). */
int dex_attention_mass(const dex_paged_kv* kv, const dex_mass_args* a, int32_t* status, void* stream);

/* One dex_paged_evict call.  Sequence b with more than keep positions keeps, for each K/V head by itself, positions [0, first),
 * the last recent ones and, of those in between, the keep - first - recent with the largest mass (equal ones:
 * the lowest positions; -0 equals 0; NaN comes last), in their order.  A sequence of at most keep keeps all. */
typedef struct dex_evict_args {
  const float* mass;           /* device, as dex_attention_mass writes it */
  float* mass_out;             /* device, or NULL; may be mass itself (then with the same stride), else must not overlap it */
  int64_t mass_stride;         /* at least table_width * page_size */
  int64_t mass_out_stride;     /* the same */
  const int32_t* seq_len;      /* device [batch] */
  int32_t* new_len;            /* device [batch]: min(seq_len, keep); must not overlap seq_len */
  int32_t* kept;               /* device [batch][n_kv_heads][keep]: the positions kept, then -1 */
  const int32_t* out_table;    /* device [batch][out_table_stride], or NULL: in place */
  int32_t out_table_width, out_table_stride;   /* with out_table */
  int32_t keep, recent, first; /* recent, first >= 0, first + recent <= keep, keep >= 1 */
} dex_evict_args;

/* Evict the positions of a paged cache that received the least attention: the rows of kept position i >= first
 * (K and V of a head) become position i of the sequence, in the pages of its own table or of out_table's (which
 * must not be pages that the call reads).  Rows and masses below first stay where they are and are not copied, so a shared prefix of first
 * positions stays shared; pages that hold positions from first on must be the sequence's own.  mass_out gets the
 * masses of the positions kept, and zeros from new_len to seq_len.  Keys keep the rotation of their old
 * positions: new tokens go on being rotated by their positions in the text (dex_append_args.rope_pos).  A seq_len that is
 * negative or beyond the table leaves the sequence as it was, with new_len = seq_len, kept -1 and DEX_ATTN_BAD_RANGE.  A page id
 * out of range is never followed: rows that would come from such a page become NaN, rows that would go to one are
 * dropped, with DEX_ATTN_BAD_PAGE.  DEX_ATTN_TIMEOUT: a bounded device wait gave up, rows are missing.  The same position of all K/V heads need not come from the same position: order is kept for
 * each head.  Runs on the current device; stream-ordered, no allocation, no workspace, no sync, capturable. */
int dex_paged_evict(const dex_paged_kv* kv, const dex_evict_args* a, int32_t* status, void* stream);

/* ---- sampling ------------------------------------------------------------------------ */

/* One dex_sample call over n_rows rows of logits.  Settings come per row from device arrays, or where the
 * pointer is NULL from the value beside it. */
typedef struct dex_sample_args {
  const void* logits;          /* device, [n_rows][vocab] in dtype */
  int64_t logits_stride;       /* elements between rows */
  const float* u;              /* device [n_rows]: random numbers in [0, 1) */
  const float* temperature;    /* device [n_rows] or NULL */
  const int32_t* top_k;        /* device [n_rows] or NULL */
  const float* top_p;          /* device [n_rows] or NULL */
  const float* min_p;          /* device [n_rows] or NULL */
  float temperature_all;       /* >= 0; 0: the largest logit */
  int32_t top_k_all;           /* >= 0; 0: no limit */
  float top_p_all;             /* (0, 1]; 1: no limit */
  float min_p_all;             /* [0, 1]; 0: no limit */
  const int32_t* exclude;      /* device [n_rows][exclude_stride] token ids, or NULL; ids outside [0, vocab) name nothing */
  int64_t exclude_stride;      /* elements between rows, >= n_exclude */
  int32_t n_exclude;           /* per row, 0 .. 1024 */
  int32_t n_rows;              /* 0 .. 2^20 */
  int32_t vocab;               /* 1 .. 2^18 */
  int32_t dtype;               /* dex_dtype */
  int32_t* tokens;             /* device [n_rows] */
  float* logprob;              /* device [n_rows] or NULL */
} dex_sample_args;

/* Sample a token from each row of logits x.  Tokens named in exclude (the shallower proposals of a lattice node) and tokens
 * of logit -inf have no chance.  With w_v = exp((x_v - max x) / temperature):
 *   top_k   leaves the top_k largest x (equal ones: the lowest ids),
 *   top_p   of these, in descending order of (x, then ascending id), those before which less than top_p of
 *           the mass of what top_k left lies (the first one always),
 *   min_p   of these the ones with w_v >= min_p,
 * and the token is the lowest id up to which more than u of the mass that is left lies.  So rows that share u and
 * settings are coupled.  logprob: the log of the token's share of that mass, good to 2^-19 and 2^-22 of its
 * size.  Temperature 0: the largest logit (lowest
 * id), log-probability 0; one so small that log2(e) / temperature is no float (below 4.3e-39): only tokens of the largest logit have a
 * chance.  Weights are integers in units of 2^-43 of the largest, each good to two, and their sums exact, so the result does not
 * depend on any order; the border between two tokens is off by at most 2 vocab units.  A token below 2^-44 of the largest counts for nothing: it
 * has no chance, at u = 0 either, and adds nothing to the mass that top_p is a part of.  In the arrays top_k <= 0 or >= vocab, top_p >= 1
 * and min_p <= 0 limit nothing, top_p <= 0 leaves the largest, min_p > 1 counts as 1, u is clamped to [0, 1).
 * A row that has no token to choose (NaN or +inf among its logits that are not excluded, all -inf or excluded, a setting or u that is NaN, a
 * negative or infinite temperature) gets token -1 and logprob NaN.  Runs on the current device; stream-ordered, no allocation, no workspace,
 * no sync, capturable.  n_rows 0 is a no-op. */
int dex_sample(const dex_sample_args* a, void* stream);

/* ---- host-only lattice scheduler (no GPU needed) ---------------------------------- */

/* One planned lattice node (HOST struct). */
typedef struct dex_plan_node {
  int32_t seq, heap, stage, plen;
  int32_t pos;          /* position of the node's input token: p_c - 1 + plen */
  int32_t c_end;        /* keys at positions < c_end come from the committed cache */
  int32_t slot;         /* pool slot of the node's slot chain */
  int32_t kv_commit;    /* 1 for the anchor path: K/V written to the committed cache */
  int32_t token;        /* input token for stage-0 nodes, -1 for depth children */
  int32_t target_pos;   /* p_c + plen */
  int32_t unmasked;     /* 1 for the final-depth reference node */
  int32_t n_prior, n_tail;
  int32_t prior[16];    /* DECS priors: tokens of shallower nodes in the slot chain */
  int32_t tail[16];     /* pool slots holding the KV of positions c_end .. pos */
} dex_plan_node;

typedef struct dex_lattice dex_lattice;

int dex_lattice_new(const int32_t* X, int32_t n_X, int32_t batch, int32_t decs, int32_t max_branch,
                    dex_lattice** out);
/* Start sequence seq with p_c committed tokens, last_token at position p_c - 1. */
int dex_lattice_start(dex_lattice* lat, int32_t seq, int32_t p_c, int32_t last_token);
/* Nodes of the next round (level q of each active sequence), grouped by stage. */
int dex_lattice_plan(dex_lattice* lat, dex_plan_node* out, int32_t max_nodes, int32_t* n_nodes);
/* Insert the planned nodes' tokens; commit and collapse where the anchor reached the
 * final depth.  committed: HOST int32 [batch] (-1 = none); kstar: HOST int32 [batch]
 * (-1 = none); jobs: copy jobs the collapse needs (n_jobs <= max_jobs). */
int dex_lattice_update(dex_lattice* lat, const int32_t* tokens, int32_t* committed, int32_t* kstar,
                       dex_copy_job* jobs, int32_t max_jobs, int32_t* n_jobs);
/* State of sequence seq: {q, p_c, slots in use}. */
int dex_lattice_state(const dex_lattice* lat, int32_t seq, int32_t* q, int32_t* p_c, int32_t* slots_used);
void dex_lattice_free(dex_lattice* lat);

#ifdef __cplusplus
}
#endif
#endif /* DEX_H_ */
