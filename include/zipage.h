/*
 * zipage.h — C ABI of the Compressed-PagedAttention compression pass (sm_103a).
 *
 * The operation is the compression step of Zipage ("Zipage: Maintain High Request Concurrency
 * for LLM Reasoning through Compressed PagedAttention", summaries on gist.science; zh page §2.1,
 * de page §2 "Methodik", es page §2 "Metodología", fr page §2.A–§2.E).  A request that holds
 * N_max blocks of b tokens and has filled its last block is compressed: every cached token of
 * every layer and KV head is scored, the top k = (N_max-1)*b per KV head are kept in their
 * original order and rewritten compactly into the first N_max-1 blocks (or into newly
 * allocated target blocks where the leading blocks are shared prefix blocks), and the last
 * block is released.
 *
 * Conventions
 *   - Every device buffer is allocated and owned by the caller; the library never frees
 *     caller memory.  "device" below means a pointer into GPU global memory, "host" a pointer
 *     into CPU memory.
 *   - Calls that launch work are asynchronous on the given stream and return as soon as the
 *     launch is queued.  Host-side argument errors are returned immediately and nothing is
 *     launched.  Errors that only the GPU can see (a block id outside the pool, a seq_len or
 *     query slot out of range, a wait that gave up) are written to the error word at the
 *     start of the caller's workspace; the unit concerned is skipped, never half-written.
 *     Read it with zp_read_error().
 *   - bf16 is passed as raw 16-bit storage (`uint16_t`): the library does not depend on any
 *     C++ bf16 type.
 *   - KV pool layout (bf16): [num_layers][num_blocks][2][num_kv_heads][block_size][head_dim],
 *     index 0 of the third dimension = K, 1 = V.  Each (layer, block, K|V, head) tile of
 *     block_size*head_dim values is contiguous.
 */
#ifndef ZIPAGE_H
#define ZIPAGE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t zp_status;
enum {
  ZP_OK = 0,
  ZP_ERR_INVALID_ARG = 1,  /* a host-side argument is out of range or inconsistent */
  ZP_ERR_NO_BLOCKS = 2,    /* the allocator cannot satisfy the request; nothing changed */
  ZP_ERR_BAD_TABLE = 3,    /* (device) a block id, seq_len or query slot is out of range */
  ZP_ERR_TIMEOUT = 4,      /* (device) a bounded wait inside a kernel gave up */
  ZP_ERR_CUDA = 5,         /* a CUDA runtime/driver call failed */
  ZP_ERR_UNSUPPORTED = 6,  /* valid arguments outside what the library implements */
  ZP_ERR_TOO_LARGE = 7     /* the call needs more scratch than zp_paged_decode_attn_static holds */
};

/* Opaque stream handle: a cudaStream_t (CUstream) passed through as a pointer, NULL = legacy
 * default stream. */
typedef void* zp_stream;

/* Method parameters.  The pages fix N_max, b and w; alpha, beta, decay and scale are readings
 * (the pages name the three scores but print no weights). */
typedef struct zp_params {
  int32_t num_layers;     /* layers in the pool */
  int32_t num_q_heads;    /* H_q */
  int32_t num_kv_heads;   /* H_kv; H_q % H_kv == 0, G_q = H_q / H_kv query heads per KV head */
  int32_t head_dim;       /* d: 64 or 128 */
  int32_t block_size;     /* b: 16 or 32 tokens per block */
  int32_t n_max;          /* N_max: block cap per request, >= 2 */
  int32_t window;         /* w: observation-window length, 1 <= w <= (n_max-1)*b */
  float alpha;            /* weight of the carried global score */
  float beta;             /* weight of the redundancy score (subtracted) */
  float decay;            /* global-score decay: G' = decay*G + attn */
  float scale;            /* logit scale, normally 1/sqrt(d) */
  int32_t protect_window; /* 1: the last w tokens are always kept */
  int32_t causal;         /* 1: window row i sees keys t <= L-w+i */
} zp_params;

typedef struct zp_kv_pool {
  void* base;             /* device, bf16, layout above; 16-byte aligned */
  int64_t num_blocks;     /* blocks per layer */
} zp_kv_pool;

typedef struct zp_seq_meta {
  int32_t num_requests;       /* R: requests compressed by this call */
  int32_t max_blocks;         /* row stride of the block tables (>= ceil(L_max / b)) */
  const int32_t* seq_len;     /* device [R]: cached tokens L of each request, k < L <= L_max
                                 (L = n_max*b at the decode trigger; a request that left a long
                                 prefill may hold more, zh §2.1) */
  const int32_t* qslot;       /* device [R]: query slot of each request, 0 <= qslot < num_qslots */
  const int32_t* dst_tables;  /* device [R][max_blocks]: where survivors go; equals the source
                                 table except at target blocks (zp_plan_compress) */
  int32_t max_seq_len;        /* L_max: the longest seq_len of the call (<= 16384), or 0 for
                                 n_max*b.  It is also the row length of global_scores and of
                                 the zp_debug arrays. */
  const int32_t* n_max_per_req; /* device [R] or NULL: per-request block budgets
                                   2 <= N_max_r <= params.n_max (the pages' per-request dynamic
                                   budgets, de §5); request r keeps k_r = (N_max_r-1)*b tokens per
                                   head.  NULL: every request uses params.n_max. */
  int32_t layer_begin;        /* the call compresses layers [layer_begin, layer_begin +
                                 layer_count) of every request; layer_count 0 means all layers
                                 (then layer_begin must be 0).  Layer indices into the pool,
                                 obs_q, global_scores and the zp_debug arrays stay absolute, so a
                                 caller can compress a model layer by layer (for instance while
                                 the next layer's blocks are still being copied in). */
  int32_t layer_count;
} zp_seq_meta;

/* Optional per-token outputs, each device [R][num_layers][num_kv_heads][L_max] (row-major),
 * any field may be NULL.  attn = window attention score, redund = Lightning redundancy,
 * score = combined score S (+inf on protected tokens), keep = 1 if kept else 0. */
typedef struct zp_debug {
  float* attn;
  float* redund;
  float* score;
  int32_t* keep;
} zp_debug;

/* ---------------------------------------------------------------------------------------
 * Compression pass (zh §2.1 core mechanism; zh §2.3 cross-layer parallel compression).
 *
 * One launch covers every (request, layer, kv head) unit.  For unit (r, l, h) with
 * L = seq_len[r] cached tokens read through block_tables[r]:
 *   attn[t]  = mean over the w*G_q window rows (i, g) of softmax_t(scale*<q_{i,g}, k_t>),
 *              row i being the query of position L-w+i (causal if params.causal);
 *   R[t]     = mean cosine similarity of k_t to the other keys of its block (Lightning);
 *   S[t]     = attn[t] + alpha*G[t] - beta*R[t]  (+inf for the last w if protect_window);
 *   keep the k = (n_max-1)*b tokens first in (S desc, t asc); survivor j (ascending t) is
 *   copied bit for bit to logical slot j of dst_tables[r]; G'[j] = decay*G[src_j] + attn[src_j]
 *   for j < k and 0 for k <= j < L.
 * Arguments
 *   pool          device KV pool, read through block_tables and written through dst_tables.
 *   block_tables  device [R][max_blocks] int32, physical block of each logical block.
 *   meta          host struct with device pointers (see zp_seq_meta).
 *   obs_q         device bf16 [num_qslots][num_layers][w][H_q][d]: the window queries;
 *                 16-byte aligned.
 *   num_qslots    M, number of query slots in obs_q and global_scores.
 *   global_scores device fp32 [num_qslots][num_layers][H_kv][L_max], updated in place.
 *   params        host.
 *   dbg           host struct or NULL.
 *   workspace     device, >= zp_compress_workspace_size() bytes, 256-byte aligned; holds the
 *                 error word (cleared by the call before any kernel runs), the unit counters,
 *                 and the request order grouped by length that the call builds when the
 *                 requests' lengths may need clusters of different sizes (max_seq_len above
 *                 n_max*b, or per-request budgets): each group then runs in a launch of its
 *                 own cluster size.  One workspace serves one call in flight at a time.
 *   stream        stream to launch on.
 * Source and destination blocks of different requests must not overlap (shared prefix
 * blocks are only read).  Returns ZP_OK once queued.
 * A unit with bad metadata (ZP_ERR_BAD_TABLE) is skipped whole and every other unit is
 * compressed.  ZP_ERR_TIMEOUT (a wait inside the kernel gave up after 2 s, which only a broken
 * device or driver state produces) means the call failed: the pool and the global scores of
 * the units the stalled cluster went on to process are undefined.
 * --------------------------------------------------------------------------------------- */
zp_status zp_compress(const zp_kv_pool* pool, const int32_t* block_tables, const zp_seq_meta* meta,
                      const uint16_t* obs_q, int32_t num_qslots, float* global_scores,
                      const zp_params* params, const zp_debug* dbg, void* workspace,
                      size_t workspace_bytes, zp_stream stream);

/* Bytes of workspace zp_compress needs.  max_seq_len 0 means n_max*b.  Up to 4096 tokens: a
 * 512-byte header (error word, unit counters, length groups) and 4 bytes per request (the
 * grouped request order), rounded up to 256.  Above 4096: 256 bytes and the scratch of the
 * multi-pass form (per unit: 1 KB per 256-token chunk and 16 bytes per token). */
size_t zp_compress_workspace_size(const zp_params* params, int32_t num_requests, int32_t max_seq_len);

/* Kernel launches one zp_compress call makes for this max_seq_len (0 means n_max*b) and
 * budget form (per_request_budgets != 0 when meta->n_max_per_req is given): 1 when every
 * request fits one cluster size, 1 + G when the call groups the requests by length into G
 * cluster sizes (the grouping kernel and one launch per size, empty groups included), 4 for
 * the multi-pass form (max_seq_len above 4096).  0 for arguments zp_compress rejects on its
 * sizes.  Host only; launches nothing. */
int32_t zp_compress_kernel_launches(const zp_params* params, int32_t max_seq_len, int32_t per_request_budgets);

/* ---------------------------------------------------------------------------------------
 * Original (all-pairs) redundancy score — the ablation of the Lightning Redundancy Score
 * (zh §2.1 and es §2: the original compares every pair of the N*b cached tokens, O(N^2 b^2),
 * where Lightning compares the b^2 pairs of each block, O(N b^2); de §2: the original needs
 * the full similarity matrix).  Not used by zp_compress: it exists to measure what Lightning
 * saves.
 *   redund[r][l][h][t] = (1/(L-1)) * sum over j < L, j != t of cos(k_t, k_j),
 * cosine with norms clamped at 1e-12, for t < L = seq_len[r]; 0 for t >= L and when L < 2.
 * Arguments
 *   pool          device KV pool, read through block_tables (only K is read).
 *   block_tables  device [R][max_blocks] int32.
 *   meta          host struct: num_requests, max_blocks, seq_len (device [R]) and
 *                 max_seq_len (the row length L_max of redund; n_max*b when 0).  The other
 *                 fields are ignored.  L_max <= 4096.
 *   params        host; num_layers, num_kv_heads, head_dim (64 or 128), block_size (16 or
 *                 32) and n_max are used.
 *   redund        device fp32 [R][num_layers][H_kv][L_max], written.
 *   workspace     device, >= zp_redundancy_workspace_size(params, R, max_seq_len) bytes,
 *                 256-byte aligned: the error word (a block id outside the pool or a seq_len
 *                 above L_max: ZP_ERR_BAD_TABLE; a wait that gave up: ZP_ERR_TIMEOUT), then
 *                 the squared key norms that a pre-pass computes.
 * Returns ZP_OK once queued.
 * --------------------------------------------------------------------------------------- */
zp_status zp_redundancy_all_pairs(const zp_kv_pool* pool, const int32_t* block_tables, const zp_seq_meta* meta,
                                  const zp_params* params, float* redund, void* workspace,
                                  size_t workspace_bytes, zp_stream stream);

/* Bytes of workspace zp_redundancy_all_pairs needs: the error word and one fp32 squared key
 * norm per (request, layer, kv head, token < L_max). */
size_t zp_redundancy_workspace_size(const zp_params* params, int32_t num_requests, int32_t max_seq_len);

/* ---------------------------------------------------------------------------------------
 * Paged decode attention over the (compacted) cache — the consumer that runs on the main
 * stream while compression runs on a side stream (zh §2.1 asynchronous compression and
 * decoding; fr §2.D).
 *   out[r][qh] = softmax_t(scale*<q[r][qh], k_t>) . v_t over t < seq_lens[r], with keys and
 *   values of kv head qh / G_q of `layer`, read through block_tables[r].
 * q, out: device bf16 [B][H_q][d]; block_tables device [B][max_blocks]; seq_lens device [B]
 * (1 <= seq_len <= max_blocks*b).  workspace >= zp_paged_decode_workspace_size() bytes,
 * 256-byte aligned (split-KV partials + error word).
 * --------------------------------------------------------------------------------------- */
zp_status zp_paged_decode_attn(const zp_kv_pool* pool, int32_t layer, const uint16_t* q,
                               const int32_t* block_tables, const int32_t* seq_lens, int32_t B,
                               int32_t max_blocks, uint16_t* out, const zp_params* params,
                               void* workspace, size_t workspace_bytes, zp_stream stream);

size_t zp_paged_decode_workspace_size(const zp_params* params, int32_t B, int32_t max_blocks);

/* Kernel launches one zp_paged_decode_attn call with these sizes makes on the current device:
 * 1 when every request fits one split (the split size is chosen per call from B, H_kv,
 * max_blocks and the device's SM count), 2 with the kernel that merges the splits.  0 for
 * invalid arguments.  Host only; launches nothing. */
int32_t zp_paged_decode_kernel_launches(const zp_params* params, int32_t B, int32_t max_blocks);

/* ---------------------------------------------------------------------------------------
 * zp_paged_decode_attn without any device allocation by anyone.  The paper has no
 * counterpart: this is a convenience of this library.
 *
 * For callers that cannot allocate device memory: a host runtime that owns every device
 * buffer through its own pool and hands this library no allocator, a serving loop that must
 * not call cudaMalloc (which can synchronise the whole device) in its hot path, or a process
 * that must know its complete device footprint when the library is loaded.
 *
 * Same operation and arguments as zp_paged_decode_attn, except that the split-KV partials
 * live in a fixed 16 MiB array inside the library (held by every GPU that loads it until the
 * process exits), so no workspace is passed.  A call needs
 * B * H_q * ceil(max_blocks / 32) * (head_dim + 2) * 4 bytes of it, at most 16 MiB - 256 B;
 * larger calls return ZP_ERR_TOO_LARGE and launch nothing.
 *   dev_status  device int32 written with the call's device-side status (0, or
 *               ZP_ERR_BAD_TABLE for a block id outside the pool or a bad seq_len); it is
 *               cleared on the stream before the kernel runs.  May be NULL, in which case
 *               device-side errors are not reported.
 * The first call on a device looks up the array's device address for that device (with the
 * device current); make that first call before any stream capture.  The address is kept for
 * the life of the process: after cudaDeviceReset, or anything else that destroys the device's
 * primary context, do not call this entry point on that device again in the same process (the
 * library would be reloaded at an address it does not know).  Every call shares the
 * one array: calls whose kernels may overlap on the GPU (different streams without an
 * ordering between them) race on it and must be serialised by the caller.  The call
 * allocates and frees nothing.
 * --------------------------------------------------------------------------------------- */
zp_status zp_paged_decode_attn_static(const zp_kv_pool* pool, int32_t layer, const uint16_t* q,
                                      const int32_t* block_tables, const int32_t* seq_lens, int32_t B,
                                      int32_t max_blocks, uint16_t* out, const zp_params* params,
                                      int32_t* dev_status, zp_stream stream);

/* Test hook of the device-side failure detection (bounded waits).  Not for production use.
 * Same operation, arguments and workspace as zp_paged_decode_attn, plus stall_limit_ns
 * (1 .. 10^9).  Before its first chunk of K/V, every warp of the decode kernel first waits, for
 * at most stall_limit_ns, on a shared-memory barrier that nothing ever completes.  That wait
 * runs out, and the kernel then takes the path of any wait that gives up: it waits (bounded,
 * 2 s) for the copies it has already issued, writes its outputs from the keys it has folded in
 * (none: zeros) and records ZP_ERR_TIMEOUT in the workspace's error word, which
 * zp_read_error() returns.  Nothing faults or hangs, and the context stays usable.  Returns
 * ZP_OK once queued. */
zp_status zp_test_decode_stalled(const zp_kv_pool* pool, int32_t layer, const uint16_t* q,
                                 const int32_t* block_tables, const int32_t* seq_lens, int32_t B,
                                 int32_t max_blocks, uint16_t* out, const zp_params* params,
                                 void* workspace, size_t workspace_bytes, int64_t stall_limit_ns,
                                 zp_stream stream);

/* Test hook of the same kind for the compression pass.  Not for production use.  Same
 * operation, arguments and workspace as zp_compress (no debug outputs), plus stall_limit_ns
 * (1 .. 10^9); meta->max_seq_len must exceed 4096, so that the call takes the multi-pass form,
 * whose CTAs exchange nothing with one another (ZP_ERR_INVALID_ARG otherwise).  Before its first
 * chunk, thread 0 of every CTA of the statistics launch first waits, for at most stall_limit_ns,
 * on a shared-memory barrier that nothing ever completes.  That wait runs out, and the CTA then
 * takes the path of any wait that gives up: its chunks get empty row statistics, it waits
 * (bounded, 2 s) for the copy it has in flight and records ZP_ERR_TIMEOUT in the error word.
 * The later launches of the call run as usual, so, as for any ZP_ERR_TIMEOUT, the pool rows and
 * global scores of the call's units are undefined afterwards; nothing is written outside the
 * call's buffers.  Nothing faults or hangs, and the context stays usable.  Returns ZP_OK once
 * queued. */
zp_status zp_test_compress_stalled(const zp_kv_pool* pool, const int32_t* block_tables, const zp_seq_meta* meta,
                                   const uint16_t* obs_q, int32_t num_qslots, float* global_scores,
                                   const zp_params* params, void* workspace, size_t workspace_bytes,
                                   int64_t stall_limit_ns, zp_stream stream);

/* ---------------------------------------------------------------------------------------
 * Operators around the cache: rotary positions, a step's slots and cache writes, an 8-bit form of
 * the pool, and attention with a sliding window.
 *
 * They share these conventions, on top of the ones at the top of this file:
 *   - A workspace belongs to one call in flight at a time; calls of any of these operators may
 *     follow one another on a stream with the same one, and captured graphs may share one if they
 *     are replayed one after the other.
 *   - The error word at the start of the workspace is sticky: zero it once (the Python binding's
 *     new_workspace does).  A call writes it only when it finds an error, and it keeps the first one
 *     until zp_read_error() reads and clears it, so one read can cover all layers of a step.
 *     Nothing else in a workspace has to hold any value.
 *   - Attention splits few requests, or few new tokens, among more CTAs, and then asks for a larger
 *     workspace than for a larger batch.  A call also takes a smaller one whose size is a multiple of 256
 *     bytes, as the sizes of all these operators are, and then splits its work less: one workspace can serve
 *     a batch that grows and shrinks, at full speed if it is the largest that any of its sizes asks for.
 *     The splits decide how sums are grouped, so a row's last bit may depend on the workspace's size.
 *   - params.scale is finite and above 0 where a call uses it.
 *   - Kernels are launched with programmatic stream serialization: they come in while the one ahead of
 *     them on the stream still runs, and wait for it on the device.  The stream's order is kept.
 *   - A zp_rows describes bf16 rows [tokens][heads][head_dim] whose last dimension is
 *     contiguous; strides are in elements.  Any strides are accepted (0 for broadcast rows that are only
 *     read), but rows that a call writes must not overlap: a stride below head_dim between several of them
 *     is refused.  Rows whose base address and strides are multiples of 16 bytes are moved with wide
 *     loads and stores.
 * --------------------------------------------------------------------------------------- */
typedef struct zp_rows {
  void* data;             /* device, bf16; NULL only where the call says so */
  int64_t token_stride;
  int64_t head_stride;
} zp_rows;

/* How the angles of far positions are scaled.  f_i = theta^(-2i / rotary_dim), i < rotary_dim/2,
 * is the unscaled angle per position of pair i. */
enum {
  ZP_ROPE_NONE = 0,
  ZP_ROPE_LINEAR = 1,     /* f_i / factor */
  ZP_ROPE_BASE = 2,       /* theta * factor^(rotary_dim / (rotary_dim - 2)) in place of theta */
  ZP_ROPE_YARN = 3,       /* f_i for pairs that turn at least `high` times over original_len
                             positions, f_i / factor for those below `low` turns, a linear ramp
                             over the pair index between; cos and sin times 0.1 ln(factor) + 1 */
  ZP_ROPE_WAVELENGTH = 4  /* the same ends, blended between by (turns - low) / (high - low) */
};

typedef struct zp_rope_config {
  int32_t head_dim;       /* even, 2 .. 512 */
  int32_t rotary_dim;     /* the first rotary_dim values of a head are rotated: even,
                             2 .. min(head_dim, 256); the others pass through */
  int32_t interleaved;    /* 1: pair i is (x[2i], x[2i+1]); 0: (x[i], x[i + rotary_dim/2]) */
  int32_t scaling;        /* ZP_ROPE_* */
  double theta;           /* > 1 */
  double factor;          /* >= 1; ignored with ZP_ROPE_NONE */
  int32_t original_len;   /* > 0 for ZP_ROPE_YARN and ZP_ROPE_WAVELENGTH */
  double low, high;       /* 0 < low < high, for the same two */
  double mscale;          /* factor on cos and sin; 0: the scaling's own (1, or the one above) */
} zp_rope_config;

/* What zp_rope_apply needs, filled by zp_rope_init and passed with every call.  Angles are held
 * as turns per position in units of 2^-64, so that position * angle wraps exactly. */
typedef struct zp_rope {
  int32_t head_dim, rotary_dim, interleaved;
  float mscale;
  uint64_t turns[128];
} zp_rope;

/* Host only. */
zp_status zp_rope_init(const zp_rope_config* config, zp_rope* out);

/* Rotary positions of the queries and keys of T tokens in one launch:
 *   (y_a, y_b) = mscale * (x_a cos - x_b sin, x_b cos + x_a sin),  angle = positions[t] * f_i,
 * computed in fp32 and rounded to bf16 once.
 *   q, k            rows [T][num_q_heads] and [T][num_kv_heads]; either may be NULL (or have no
 *                   heads).
 *   q_out, k_out    where the results go: the same rows (in place) or others that do not overlap
 *                   them.  In place, values past rotary_dim are not touched.
 *   positions       device int32 [T], any value (negative angles turn backwards).
 * Returns ZP_OK once queued.  No workspace. */
zp_status zp_rope_apply(const zp_rope* rope, const zp_rows* q, const zp_rows* q_out, int32_t num_q_heads,
                        const zp_rows* k, const zp_rows* k_out, int32_t num_kv_heads, const int32_t* positions,
                        int32_t T, zp_stream stream);

/* Rotary positions with several axes: a token of an image or video frame has a time, a height and a
 * width (text has the same number on each), and every pair of a head is turned by one of them. */
#define ZP_ROPE_MAX_AXES 4
enum {
  ZP_AXES_SECTIONS = 0,   /* the first sections[0] pairs belong to axis 0, the next sections[1] to axis 1, ... */
  ZP_AXES_CYCLE = 1,      /* pair i belongs to axis i % num_axes while that axis has had fewer than its
                             section's pairs, and to axis 0 otherwise */
  ZP_AXES_RESTART = 2     /* as ZP_AXES_SECTIONS, and each section has the angles of a head whose rotary_dim
                             is twice the section: the f_i start again */
};

typedef struct zp_rope_axes_config {
  int32_t num_axes;       /* 1 .. ZP_ROPE_MAX_AXES */
  int32_t layout;         /* ZP_AXES_* */
  int32_t sections[ZP_ROPE_MAX_AXES]; /* pairs of each axis, >= 1, together rotary_dim / 2; a layout that
                             cannot give an axis its pairs is refused */
} zp_rope_axes_config;

/* What zp_rope_apply_axes needs, filled by zp_rope_axes_init. */
typedef struct zp_rope_axes {
  zp_rope rope;           /* its turns hold each pair's own */
  int32_t num_axes;
  uint8_t axis[128];      /* of each pair */
} zp_rope_axes;

/* Host only. */
zp_status zp_rope_axes_init(const zp_rope_config* config, const zp_rope_axes_config* axes, zp_rope_axes* out);

/* zp_rope_apply where pair i of token t is turned by positions[axis[i] * axis_stride + t] * f_i.
 *   positions       device int32 [num_axes][axis_stride], any values; axis_stride 0: all axes share one row.
 * Tokens with the same position on every axis get the bits that zp_rope_apply gives them (but for
 * ZP_AXES_RESTART, whose angles are others). */
zp_status zp_rope_apply_axes(const zp_rope_axes* axes, const zp_rows* q, const zp_rows* q_out, int32_t num_q_heads,
                             const zp_rows* k, const zp_rows* k_out, int32_t num_kv_heads, const int32_t* positions,
                             int64_t axis_stride, int32_t T, zp_stream stream);

/* The blocks, slots and positions of a step, made on the device in one launch from lengths that the
 * device alone may know (what the step before accepted of its drafts, say), so that steps follow one another
 * without the host, and can be captured and replayed.
 *   cached          device int32 [B], tokens in request r's cache before the step
 *   new_tokens      device int32 [B], tokens that the step adds (0: none, as for a padded request)
 *   first_pos       device int32 [B] or NULL: the position of request r's first new token, where it is not
 *                   cached[r] (a compression pass drops tokens, and positions go on).  NULL: cached[r].
 *   free_ids        device int32 [num_free], ids of free blocks (zp_alloc_blocks gives the host some to hand out)
 *   free_at         device int32 [1] or NULL: how many of free_ids are taken.  The call takes the next ones,
 *                   in the order of requests and tokens, and advances it.  NULL: none are taken before the call.
 *   num_blocks      blocks of the pool (num_blocks * block_size <= 2^31 - 1)
 *   block_tables    device int32 [B][max_blocks].  The call writes the entries of blocks whose first token is
 *                   new, and reads those of part-full blocks that get tokens; no others.
 *                   Where tokens were taken back since (rejected drafts), a block that they had begun counts as
 *                   new: it gets another id, and the old one is the caller's to hand out again
 *                   (zp_step_slots_held uses it).
 *   token_start     device int32 [B + 1], written: request r owns rows token_start[r] .. token_start[r + 1] - 1.
 *   seq_lens        device int32 [B], written: cached + new.  May be `cached` itself; no other arrays overlap.
 *   positions       device int32 [T] or NULL, written.  Rows behind the last request's: 0.
 *   slots           device int32 [T], written: block * block_size + place in the block, as zp_kv_append takes
 *                   it.  Rows behind the last request's: -1.
 *   T               rows of the step's buffers, at least the tokens of all requests.
 *   params          block_size (16 or 32) is used.
 *   workspace       device, >= 256 bytes, 256-byte aligned.
 * A request whose cached or new_tokens is out of range (or that would pass max_blocks) takes part without
 * tokens (seq_lens: its cached tokens, 0 if those are out of range), ZP_ERR_BAD_TABLE; so do tokens of a block
 * with an id outside the pool (slot -1).  If the requests' tokens do not fit T (ZP_ERR_BAD_TABLE) or their blocks do not fit
 * free_ids (ZP_ERR_NO_BLOCKS; a free_at outside 0 .. num_free: ZP_ERR_BAD_TABLE), the step is one without tokens:
 * token_start is all 0, seq_lens what was cached, slots all -1, and tables and free_at stay.  B up to 65535. */
zp_status zp_step_slots(const int32_t* cached, const int32_t* new_tokens, const int32_t* first_pos, int32_t B,
                        const int32_t* free_ids, int32_t num_free, int32_t* free_at, int64_t num_blocks,
                        int32_t* block_tables, int32_t max_blocks, int32_t* token_start, int32_t* seq_lens,
                        int32_t* positions, int32_t* slots, int32_t T, const zp_params* params, void* workspace,
                        size_t workspace_bytes, zp_stream stream);

/* The same where tokens are taken back between steps (rejected drafts, cached[r] lowered): blocks that they had begun stay
 * the request's, and its next tokens go there.
 *   held_blocks     device int32 [B] or NULL (as zp_step_slots): how many entries of request r's table hold blocks, at least
 *                   those of its cached tokens.  The call reads entries of those blocks that get tokens, takes free ids
 *                   for the blocks behind them alone, and advances held_blocks[r] by those.  Blocks that are given back lower it.
 * A request whose held_blocks is below its cached tokens' blocks or above max_blocks takes part without tokens,
 * ZP_ERR_BAD_TABLE.  A step that does not fit leaves held_blocks as they are. */
zp_status zp_step_slots_held(const int32_t* cached, const int32_t* new_tokens, const int32_t* first_pos, int32_t* held_blocks,
                             int32_t B, const int32_t* free_ids, int32_t num_free, int32_t* free_at, int64_t num_blocks,
                             int32_t* block_tables, int32_t max_blocks, int32_t* token_start, int32_t* seq_lens,
                             int32_t* positions, int32_t* slots, int32_t T, const zp_params* params, void* workspace,
                             size_t workspace_bytes, zp_stream stream);

/* New keys and values of one layer into the bf16 pool, bit for bit.
 *   k, v            rows [T][num_kv_heads][head_dim]
 *   slots           device int32 [T]: row t becomes token slots[t] % block_size of block slots[t] / block_size.
 *                   Below 0: the row goes nowhere.  Other slots are distinct.
 *   workspace       device, >= 256 bytes, 256-byte aligned.
 * A slot outside the pool: that row is not written, ZP_ERR_BAD_TABLE.  head_dim 64 or 128, block_size 16 or 32,
 * num_blocks * block_size <= 2^31 - 1. */
zp_status zp_kv_append(const zp_kv_pool* pool, int32_t layer, const zp_rows* k, const zp_rows* v, const int32_t* slots,
                       int32_t T, const zp_params* params, void* workspace, size_t workspace_bytes, zp_stream stream);

/* The 8-bit pool: E4M3 codes in the bf16 pool's layout, [num_layers][num_blocks][2]
 * [num_kv_heads][block_size][head_dim], and one fp32 scale per (layer, block, K|V, head); a value
 * is code * scale.  zp_kv8_append and zp_kv8_pack_blocks write scales that are powers of two: the
 * smallest 2^e >= amax / 448, e >= -126, over the finite values of the block's tokens (0 for a
 * block of zeros).  With such a scale dividing by it is exact, so a code is off by E4M3's own
 * rounding only, reading back to bf16 is exact, and a scale that grows later keeps every code
 * that stays in E4M3's normal range.  Values that are not finite are stored as E4M3's NaN.
 * zp_kv8_unpack_blocks and zp_kv8_decode_attn take any finite scales, zp_kv8_window_attn those that it names. */
typedef struct zp_kv8_pool {
  void* codes;            /* device, 16-byte aligned */
  float* scales;          /* device [num_layers][num_blocks][2][num_kv_heads] */
  int64_t num_blocks;
} zp_kv8_pool;

/* Quantises new keys and values of one layer as they enter the cache.
 *   k, v            rows [T][num_kv_heads][head_dim] of the new tokens of all requests, request
 *                   after request.
 *   token_start     device int32 [B + 1], 0 = token_start[0] <= ... <= token_start[B] <= T: request r
 *                   owns rows token_start[r] .. token_start[r + 1] - 1 (none is fine).  Rows behind
 *                   the last request's are not read.
 *   cached          device int32 [B], tokens in request r's cache before the call: its new tokens
 *                   take positions cached[r], cached[r] + 1, ...
 *   block_tables    device int32 [B][max_blocks]; only the entries of blocks that receive tokens
 *                   are read.  A block that receives tokens belongs to one request and stands once
 *                   in its table (shared prefix blocks are full, and never appended to).
 * A block whose first token is new starts with a scale of its own.  In a part-full block the
 * scale is the larger of the old one and the one the new tokens need; if that is larger, the
 * codes already there are brought to it (rounded once more).  Rows behind the last token are not
 * written.
 *   workspace       device, >= 256 bytes, 256-byte aligned.
 * A request whose entries of token_start or cached are out of range, or that would pass
 * max_blocks, is skipped; so is a block with an id outside the pool: ZP_ERR_BAD_TABLE.  If
 * token_start decreases anywhere, which requests are written is undefined (nothing outside their
 * blocks is).  Tokens without a request (B = 0 with T > 0) are refused.  head_dim 64 or 128, block_size 16 or 32. */
zp_status zp_kv8_append(const zp_kv8_pool* pool, int32_t layer, const zp_rows* k, const zp_rows* v, int32_t T,
                        const int32_t* token_start, const int32_t* cached, int32_t B, const int32_t* block_tables,
                        int32_t max_blocks, const zp_params* params, void* workspace, size_t workspace_bytes,
                        zp_stream stream);

/* Whole blocks between the bf16 pool that the compression pass works on and the 8-bit pool, for
 * layers [layer_begin, layer_begin + layer_count) (count 0: all, then begin must be 0):
 *   pack    block src_ids[i] of `pool`  -> block dst_ids[i] of `kv8`;
 *   unpack  block src_ids[i] of `kv8` -> block dst_ids[i] of `pool`, bf16(code * scale).
 *   src_ids, dst_ids  device int32 [n]; dst_ids are distinct.
 *   fill        pack only: device int32 [n] or NULL, tokens in each block (0 .. block_size; NULL:
 *               all are full).  Rows past them are neither read nor written.
 *   workspace   device, >= 256 bytes, 256-byte aligned.
 * An id outside its pool, or a bad fill: that block is skipped, ZP_ERR_BAD_TABLE. */
zp_status zp_kv8_pack_blocks(const zp_kv_pool* pool, const int32_t* src_ids, const int32_t* fill,
                             const zp_kv8_pool* kv8, const int32_t* dst_ids, int32_t n, int32_t layer_begin,
                             int32_t layer_count, const zp_params* params, void* workspace, size_t workspace_bytes,
                             zp_stream stream);
zp_status zp_kv8_unpack_blocks(const zp_kv8_pool* kv8, const int32_t* src_ids, const zp_kv_pool* pool,
                               const int32_t* dst_ids, int32_t n, int32_t layer_begin, int32_t layer_count,
                               const zp_params* params, void* workspace, size_t workspace_bytes, zp_stream stream);

/* Paged decode attention over the 8-bit pool: zp_paged_decode_attn's operation on code * scale,
 * optionally with a window.  Request r's one query is at position L - 1, L = seq_lens[r]:
 *   out[r][qh] = softmax_t(params.scale * <q[r][qh], k_t>) . v_t over t < L with
 *   t >= L - window or t < sinks   (window 0: every t < L).
 *   q, out        rows [B][H_q][head_dim]; out does not overlap q.
 *   seq_lens      device int32 [B], 0 <= L <= max_blocks * b.  0 (a padded row): zeros are written.
 *   workspace     >= zp_kv8_decode_workspace_size() bytes, 256-byte aligned.
 * A bad seq_len or block id: that row (request and kv head) is not written, ZP_ERR_BAD_TABLE.
 * ZP_ERR_TIMEOUT (a wait inside the kernel gave up) as for zp_compress: the output is undefined.
 * Table entries of blocks that are not visible may hold anything.  A query's largest value times params.scale and a visible K
 * scale stays below 2^127 (logits of 0 beside it would be NaN).  head_dim 64 or 128, block_size
 * 16 or 32, up to 16 query heads per kv head. */
zp_status zp_kv8_decode_attn(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q, const int32_t* block_tables,
                             const int32_t* seq_lens, int32_t B, int32_t max_blocks, int32_t window, int32_t sinks,
                             const zp_rows* out, const zp_params* params, void* workspace, size_t workspace_bytes,
                             zp_stream stream);

size_t zp_kv8_decode_workspace_size(const zp_params* params, int32_t B, int32_t max_blocks);

/* Attention with a sliding window and a few first tokens that stay visible, over the bf16 pool,
 * for one to many new tokens per request (decode, verification of drafts, chunked prefill).  The
 * new tokens' keys and values are already in the pool.  Query i of request r's n is at position
 * p = seq_lens[r] - n + i and sees
 *   t <= p with t > p - window or t < sinks   (window 0: every t <= p).
 *   q, out        rows [T][H_q][head_dim], request after request; out does not overlap q.
 *   q_start       device int32 [B + 1], as token_start of zp_kv8_append.  Rows of out
 *                 outside q_start's range are not written; those of q have to be memory that can be
 *                 read (tiles of queries are loaded whole), but have no effect, whatever they hold
 *                 and even if they are written meanwhile.
 *   max_q         the most new tokens of a request of this call (an upper bound is fine; a request
 *                 above it is skipped: ZP_ERR_BAD_TABLE).
 *   seq_lens      device int32 [B], tokens in the cache, the new ones included: n <= L <=
 *                 max_blocks * b.
 *   workspace     >= zp_paged_window_workspace_size() bytes, 256-byte aligned.
 * A bad length, q_start or block id: the rows concerned are not written, ZP_ERR_BAD_TABLE.
 * ZP_ERR_TIMEOUT (a wait inside the kernel gave up) as for zp_compress: the output is undefined.
 * Weights are held to 16 bits where head groups times max_q is 16 or less, and rounded to bf16 above
 * (off by at most 2^-8 of themselves, as the tensor cores take them); sums and maxima are fp32.
 * Keys and values that a row does not see do not reach it, whatever they hold.  head_dim 64 or
 * 128, block_size 16 or 32, up to 16 query heads per kv head. */
zp_status zp_paged_window_attn(const zp_kv_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start,
                               int32_t T, int32_t max_q, const int32_t* block_tables, const int32_t* seq_lens,
                               int32_t B, int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                               const zp_params* params, void* workspace, size_t workspace_bytes, zp_stream stream);

size_t zp_paged_window_workspace_size(const zp_params* params, int32_t T, int32_t B, int32_t max_q,
                                      int32_t max_blocks, int32_t window, int32_t sinks);

/* Attention of whole prompts over their own keys and values, which are rows of memory: before they enter a
 * cache, or where none is kept, and before they are rounded to 8 bits.  Prompts are packed: prompt r owns rows
 * token_start[r] .. token_start[r + 1] - 1 of q, k, v and out, and its i-th token sees the tokens of its own prompt with
 *   t <= i and t > i - window or t < sinks   (window 0: every t <= i).
 *   q, out        rows [T][H_q][head_dim];  k, v  rows [T][H_kv][head_dim].  out overlaps none of the others.
 *   token_start   device int32 [B + 1], as for zp_kv8_append.  Rows of out outside its range are not written;
 *                 those of q, k and v have to be memory that can be read (tiles are loaded whole), but have no
 *                 effect, whatever they hold.
 *   max_len       the most tokens of a prompt (an upper bound is fine; a prompt above it is skipped:
 *                 ZP_ERR_BAD_TABLE).  At most 2^30.
 *   params        num_q_heads, num_kv_heads, head_dim and scale are used.
 *   workspace     >= zp_prompt_workspace_size() bytes, 256-byte aligned.
 * A bad token_start: that prompt is not written, ZP_ERR_BAD_TABLE; ZP_ERR_TIMEOUT, weights and what a row does not
 * see as for zp_paged_window_attn's form for many rows.  Which kernel takes a call follows from its sizes, so a row's last bit
 * may depend on the batch.  Rows of k and v at other than 16-byte boundaries or
 * strides are loaded value by value, at a tenth of the speed.  head_dim 64 or 128, up to 16 query heads per kv head. */
zp_status zp_prompt_attn(const zp_rows* q, const zp_rows* k, const zp_rows* v, const int32_t* token_start, int32_t T,
                         int32_t B, int32_t max_len, int32_t window, int32_t sinks, const zp_rows* out,
                         const zp_params* params, void* workspace, size_t workspace_bytes, zp_stream stream);

size_t zp_prompt_workspace_size(const zp_params* params, int32_t T, int32_t B, int32_t max_len, int32_t window, int32_t sinks);

/* zp_paged_window_attn over the 8-bit pool: attention of a chunk of new tokens (drafts, chunked prefill, a question
 * about a document in the cache), whose codes are already in the pool.  Arguments, masks and errors are
 * zp_paged_window_attn's.
 * Scales are finite, and V scales other than 0 of the blocks that a request's new tokens see are within 2^100 of one another.
 * Where head groups times max_q is 16 or less, everything is held as by zp_kv8_decode_attn (weights to 11 bits down to 2^-18 of the
 * row's largest, whatever their V scales).  Above:
 *   - keys are taken as they are; values are exact where their scale is a power of two, not below 2^-15 of the
 *     largest of the 128 tokens that are walked together, and otherwise within 2^-10 of themselves and 2^-25 of the largest
 *     value at that scale (448 times it);
 *   - a weight times the largest V scale of those 128 tokens (as a power of two) keeps 11 bits down to 2^-18 of the row's
 *     largest such product, and 2^-29 of it is the last that counts: a row whose largest weight stands beside V scales 2^15 times
 *     its own has 15 powers of two less for the others.  Sums of weights are fp32;
 *   - V scales below 2^-104 count as that (values of 0, with scales of 0, in the sum of weights alone), and above 2^104 values may
 *     overflow. */
zp_status zp_kv8_window_attn(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start,
                             int32_t T, int32_t max_q, const int32_t* block_tables, const int32_t* seq_lens,
                             int32_t B, int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                             const zp_params* params, void* workspace, size_t workspace_bytes, zp_stream stream);

size_t zp_kv8_window_workspace_size(const zp_params* params, int32_t T, int32_t B, int32_t max_q, int32_t max_blocks,
                                    int32_t window, int32_t sinks);

/* Test hooks of the bounded waits inside the attention operators: same operation, arguments and
 * workspace, plus stall_limit_ns (1 .. 1e9).  With the first copies (and products) in flight a warp of
 * each CTA waits, for at most stall_limit_ns, on a barrier that nothing completes.  That wait
 * runs out, the kernel drains what is in flight, records ZP_ERR_TIMEOUT and returns; the output rows are
 * undefined, nothing else is written, and the next call is an ordinary one. */
zp_status zp_test_kv8_decode_stalled(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q, const int32_t* block_tables,
                                     const int32_t* seq_lens, int32_t B, int32_t max_blocks, int32_t window, int32_t sinks,
                                     const zp_rows* out, const zp_params* params, void* workspace, size_t workspace_bytes,
                                     int64_t stall_limit_ns, zp_stream stream);
zp_status zp_test_paged_window_stalled(const zp_kv_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start,
                                       int32_t T, int32_t max_q, const int32_t* block_tables, const int32_t* seq_lens,
                                       int32_t B, int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                                       const zp_params* params, void* workspace, size_t workspace_bytes,
                                       int64_t stall_limit_ns, zp_stream stream);
zp_status zp_test_prompt_stalled(const zp_rows* q, const zp_rows* k, const zp_rows* v, const int32_t* token_start, int32_t T,
                                 int32_t B, int32_t max_len, int32_t window, int32_t sinks, const zp_rows* out,
                                 const zp_params* params, void* workspace, size_t workspace_bytes, int64_t stall_limit_ns,
                                 zp_stream stream);
zp_status zp_test_kv8_window_stalled(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start,
                                     int32_t T, int32_t max_q, const int32_t* block_tables, const int32_t* seq_lens,
                                     int32_t B, int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                                     const zp_params* params, void* workspace, size_t workspace_bytes,
                                     int64_t stall_limit_ns, zp_stream stream);

/* Synchronises `stream`, copies the error word at the start of `workspace` to *out_status and
 * clears it.  Returns ZP_ERR_CUDA if the copy fails. */
zp_status zp_read_error(void* workspace, zp_stream stream, zp_status* out_status);

/* ---------------------------------------------------------------------------------------
 * Block allocator with reference counts (the PagedAttention block manager with prefix
 * sharing: zh §2.2, de §2 "Prefix Caching", fr §2.C).  Host only.  Free ids are handed out
 * lowest first so that plans are deterministic.  Every call is all-or-nothing.
 * --------------------------------------------------------------------------------------- */
typedef struct zp_alloc zp_alloc;

zp_status zp_alloc_create(int64_t num_blocks, zp_alloc** out);
void zp_alloc_destroy(zp_alloc* a);
/* n fresh blocks (refcount 1) into ids[n]; ZP_ERR_NO_BLOCKS if fewer than n are free. */
zp_status zp_alloc_blocks(zp_alloc* a, int32_t n, int32_t* ids);
/* Marks the given free ids as allocated (refcount 1), e.g. to restore a saved state;
 * ZP_ERR_INVALID_ARG if any is out of range, repeated or not free. */
zp_status zp_alloc_reserve(zp_alloc* a, const int32_t* ids, int32_t n);
zp_status zp_incref(zp_alloc* a, const int32_t* ids, int32_t n);
/* A block whose refcount reaches 0 becomes free.  ZP_ERR_INVALID_ARG on a free id. */
zp_status zp_decref(zp_alloc* a, const int32_t* ids, int32_t n);
/* Deferred decref: applied once all work queued on `stream` before this call has finished
 * (the library records its own event).  stream may be NULL only if no CUDA work reads the
 * blocks; then the decref is applied at once. */
zp_status zp_decref_after(zp_alloc* a, const int32_t* ids, int32_t n, zp_stream stream);
/* Applies the deferred decrefs whose work has finished (non-blocking). */
zp_status zp_alloc_poll(zp_alloc* a);
/* Waits for all deferred decrefs and applies them. */
zp_status zp_alloc_drain(zp_alloc* a);
/* Test hook (host-side fault injection): the nth_call-th allocating call from now returns
 * ZP_ERR_NO_BLOCKS without changing anything; 0 disables. */
zp_status zp_alloc_inject_failure(zp_alloc* a, int64_t nth_call);
int32_t zp_refcount(const zp_alloc* a, int32_t id);   /* -1 if id out of range */
int64_t zp_num_free(const zp_alloc* a);
int64_t zp_num_pending(const zp_alloc* a);           /* blocks waiting in deferred decrefs */

/* Plan of one compression (zh §2.2 / fr §2.C target blocks).  host_tables, host_dst_tables:
 * host [R][max_blocks].  For each request and each logical block i < n_max-1 the destination
 * is the same physical block unless its refcount is > 1 (shared prefix block), in which case
 * it is a freshly allocated target block.  Entries i >= n_max-1 are copied unchanged.
 * Transactional: ZP_ERR_NO_BLOCKS leaves the allocator unchanged. */
zp_status zp_plan_compress(zp_alloc* a, const int32_t* host_tables, int32_t R, int32_t max_blocks,
                           int32_t n_max, int32_t* host_dst_tables);
/* As zp_plan_compress with a per-request budget host_n_max[R] (2 <= N_max_r <= max_blocks). */
zp_status zp_plan_compress_budgets(zp_alloc* a, const int32_t* host_tables, int32_t R, int32_t max_blocks,
                                   const int32_t* host_n_max, int32_t* host_dst_tables);

/* After the compression launched on `stream`: for each request, decref every replaced shared
 * block (old != new for i < n_max-1) and every old block past the first n_max-1
 * (old[n_max-1 .. ceil(seq_len/b)) — the last block at the decode trigger, more after a
 * prefill), deferred until the work queued on `stream` has finished (the kernel still reads
 * those blocks).  host_seq_len: host [R], or NULL when every request holds n_max blocks. */
zp_status zp_commit_compress(zp_alloc* a, const int32_t* old_tables, const int32_t* new_tables,
                             int32_t R, int32_t max_blocks, int32_t n_max, int32_t block_size,
                             const int32_t* host_seq_len, zp_stream stream);
/* As zp_commit_compress with a per-request budget host_n_max[R] (NULL: n_max for all). */
zp_status zp_commit_compress_budgets(zp_alloc* a, const int32_t* old_tables, const int32_t* new_tables,
                                     int32_t R, int32_t max_blocks, const int32_t* host_n_max, int32_t n_max,
                                     int32_t block_size, const int32_t* host_seq_len, zp_stream stream);

/* ---------------------------------------------------------------------------------------
 * Hybrid scheduler (zh §2.2, de §2 "Hybrid Scheduling", es §2, fr §2.B).  Host only.
 *
 * Plans engine steps around the compression pass: only the first num_slots running requests
 * (admission order) hold a query slot; requests below n_max blocks, or whose last block still
 * has room, decode without one; a request at n_max blocks with a full last block (or longer,
 * after a prefill) compresses if it holds a slot and waits otherwise; when a block cannot be
 * allocated the most recently admitted request without a slot is preempted (it returns to the
 * front of the queue and recomputes); with none left the step runs in restricted mode (only
 * slot holders grow).  Blocks come from the given allocator; compressions keep the first
 * n_max-1 blocks and release the rest when the next step applies them.
 * --------------------------------------------------------------------------------------- */
typedef struct zp_sched zp_sched;

typedef struct zp_sched_config {
  int32_t n_max;        /* block cap per request */
  int32_t block_size;   /* b */
  int32_t num_slots;    /* M query slots */
  int32_t max_running;  /* cap on running requests, 0 = none */
} zp_sched_config;

/* The plan of one step; the arrays belong to the scheduler and stay valid until the next
 * zp_sched_step or zp_sched_destroy. */
typedef struct zp_sched_plan {
  int32_t num_decode;           /* requests that decode one token */
  const int32_t* decode_ids;
  int32_t num_compress;         /* requests whose compression runs this step (async) */
  const int32_t* compress_ids;
  int32_t num_prefill;          /* requests admitted this step */
  const int32_t* prefill_ids;
  int32_t num_preempted;        /* requests preempted this step */
  const int32_t* preempted_ids;
  int32_t restricted;           /* 1: this step ran in restricted mode */
} zp_sched_plan;

typedef struct zp_sched_request_info {
  int32_t state;                /* 0 waiting, 1 running, 2 finished */
  int32_t seq_len;              /* cached tokens */
  int32_t generated;            /* tokens decoded so far */
  int32_t num_blocks;
  const int32_t* table;         /* host [num_blocks], valid until the next step */
  int32_t has_slot;
  int32_t preemptions;
} zp_sched_request_info;

typedef struct zp_sched_stats {
  int64_t steps, submitted, admitted, finished, decoded_tokens, compressions, preemptions, slot_waits,
      restricted_steps, blocks_in_use;
  int32_t running;
} zp_sched_stats;

zp_status zp_sched_create(zp_alloc* alloc, const zp_sched_config* cfg, zp_sched** out);
void zp_sched_destroy(zp_sched* s);
/* Queues a request of prompt_len tokens that will decode gen_len tokens; *req_id = its id. */
zp_status zp_sched_submit(zp_sched* s, int32_t prompt_len, int32_t gen_len, int32_t* req_id);
/* Applies the previous step's plan (decoded tokens, compressions, finished requests) and
 * plans the next one. */
zp_status zp_sched_step(zp_sched* s, zp_sched_plan* plan);
zp_status zp_sched_request(const zp_sched* s, int32_t req_id, zp_sched_request_info* info);
zp_status zp_sched_get_stats(const zp_sched* s, zp_sched_stats* out);

/* Library version, for the binding's sanity check. */
int32_t zp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZIPAGE_H */
