/*
 * llama_layer.h -- C ABI of the GB300 (sm_103a) forward pass of one
 * Llama-style decoder layer.
 *
 * The operator chain follows the page "Which ops-transformer operators one
 * Llama2-7B layer calls" (seekfood.cn/news/1207529), section "single-layer
 * operator call chain": x -> RMSNorm -> merged Q/K/V Linear -> RotaryEmbedding
 * -> Self-Attention (GQA) -> Attention Output Linear -> residual -> RMSNorm ->
 * merged Gate/Up Linear -> SiLU * up -> Down Linear -> residual.  Prefill and
 * decode take different attention kernels (same page, section "KV Cache and
 * the operators").  The KV cache is paged as on the page "ATB KV-cache paging,
 * quantisation, speculative decoding and communication overlap"
 * (hwcomputing.csdn.net), section "KV Cache memory wall": fixed-size blocks,
 * a block_table from logical to physical blocks, contextLens per request, and
 * ReshapeAndCache writing each step's K/V into its slot.
 *
 * Conventions shared by every call
 *  - All tensor pointers are DEVICE pointers, caller-owned, row-major, and
 *    16-byte aligned.  BF16 is IEEE bfloat16 (2 bytes); gains are float32.
 *  - Every call is asynchronous on `stream` (a cudaStream_t, NULL = legacy
 *    default stream).  No call allocates device memory, synchronises, or
 *    keeps a pointer after it returns, except ll_pack_weights (see there).
 *  - The return value reports what the host can check before launching
 *    (LL_OK or an LL_ERR_* code; nothing is launched on error).  Problems
 *    only the device can see (a block_table entry or slot out of range, a
 *    position beyond the RoPE table) are OR-ed as LL_DEV_* bits into
 *    `*status`, a caller-owned device int32 that the caller zeroes and reads
 *    after synchronising.  The offending row is skipped; kernels never trap.
 *  - Every bounded wait inside a kernel gives up after about two seconds,
 *    sets LL_DEV_TIMEOUT and lets the kernel finish.
 *  - The KV pool is two tensors, K and V, each BF16
 *    [num_blocks, n_kv_heads, block_size, head_dim] ("BNSD" inside a block, as
 *    the 910B layout on the paging page).  Slot s = block * block_size + offset.
 *  - block_table is int32 [batch, max_blocks]; entry j is the physical block
 *    holding positions j*block_size .. (j+1)*block_size-1 of that sequence.
 */
#ifndef LLAMA_LAYER_H
#define LLAMA_LAYER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* host-detectable errors (return values) */
#define LL_OK 0
#define LL_ERR_INVALID_ARG 1   /* null pointer, non-positive or inconsistent size */
#define LL_ERR_UNSUPPORTED 2   /* shape outside what the kernels implement */
#define LL_ERR_WORKSPACE 3     /* workspace missing or smaller than required */
#define LL_ERR_CUDA 4          /* a CUDA runtime/driver call failed */

/* device-detected problems (bits OR-ed into *status) */
#define LL_DEV_BAD_BLOCK 1     /* block_table entry < 0 or >= num_blocks where a block was needed */
#define LL_DEV_BAD_SLOT 2      /* slot_mapping entry >= num_blocks * block_size */
#define LL_DEV_BAD_POSITION 4  /* position < 0 or >= max_position, or context_len out of range */
#define LL_DEV_TIMEOUT 8       /* a bounded in-kernel wait gave up */

/* Layer shape.  head_dim must be 64 or 128; n_heads % n_kv_heads == 0;
 * n_heads / n_kv_heads <= 16; hidden and intermediate multiples of 16;
 * block_size a power of two in [16, 256]; max_position = rows of the RoPE
 * table (largest position + 1).
 * RoPE uses half-split pairs and angle pos * rope_theta^(-2i/head_dim). */
typedef struct {
    int32_t hidden;
    int32_t n_heads;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t intermediate;
    int32_t block_size;
    int32_t max_position;
    float rms_eps;
    float rope_theta;
} ll_config;

/* Canonical weights as a model stores them, all BF16 [out, in] row-major:
 * w_qkv [(n_heads + 2 n_kv_heads) head_dim, hidden], rows = Q heads, then K
 * heads, then V heads (the merged QKV MatMul of the chain page);
 * w_o [hidden, n_heads head_dim]; w_gate and w_up [intermediate, hidden];
 * w_down [hidden, intermediate]; g_attn and g_ffn float32 [hidden]. */
typedef struct {
    const void* w_qkv;
    const void* w_o;
    const void* w_gate;
    const void* w_up;
    const void* w_down;
    const float* g_attn;
    const float* g_ffn;
} ll_weights;

typedef struct {
    void* k;              /* BF16 [num_blocks, n_kv_heads, block_size, head_dim] */
    void* v;              /* same shape */
    int32_t num_blocks;
} ll_kv_pool;

/* An INT8 KV pool (paging page, section "KV Cache quantisation": per-token
 * granularity, each token's K and V with their own float32 scale).  Codes in the
 * layout of ll_kv_pool; one scale per token and KV head.  A cached row reads back
 * as code * scale. */
typedef struct {
    void* k;              /* int8 [num_blocks, n_kv_heads, block_size, head_dim] */
    void* v;              /* same shape */
    float* k_scale;       /* float32 [num_blocks, n_kv_heads, block_size] */
    float* v_scale;       /* same shape */
    int32_t num_blocks;
} ll_kv_pool_q8;

/* Human-readable name of an LL_ERR_* code (static string). */
const char* ll_strerror(int code);

/* Description of the last failure behind an LL_ERR_* return on the calling
 * thread (the failing step and CUDA's message), or "" if none.  Valid until
 * the thread's next library call. */
const char* ll_last_error(void);

/* Bytes of the packed-weight buffer for `cfg` (0 if cfg is invalid). */
size_t ll_packed_weights_size(const ll_config* cfg);

/* Lays out the weights the way the kernels read them, into the caller-owned
 * device buffer `packed` (ll_packed_weights_size bytes): Q/K head rows
 * reordered so that each RoPE pair is adjacent, gate and up rows interleaved
 * (the MergedMatMul(GateUp) of the chain page), the other weights copied, and
 * a float32 cos/sin table for max_position positions computed in float64.
 * The canonical weights may be freed once the stream has passed this call.
 * Setup-time call: it synchronises `stream` before returning. */
int ll_pack_weights(const ll_config* cfg, const ll_weights* w, void* packed, size_t packed_bytes,
                    void* stream);

/* Workspace bytes for layer calls of up to max_tokens tokens (prefill: batch *
 * seq_len; decode: batch) and block tables up to max_blocks wide. */
size_t ll_workspace_size(const ll_config* cfg, int32_t max_tokens, int32_t max_blocks);

/* Checkpoints of the fused layer (page "ATB fused-operator matrix and KV-cache
 * management", section on the engineering limits of fusion granularity: besides
 * the step-by-step and fully fused execution modes it names a fused mode with
 * verification checkpoints at key nodes, so that a wrong result can be traced to
 * one step).  A layer call leaves the output of every kernel of its chain in the
 * workspace; these are their byte offsets from the workspace start, for a
 * workspace sized by ll_workspace_size(cfg, max_tokens, max_blocks).  After a call
 * over T tokens (and until the next call on the same workspace), row t < T of:
 *   x_hat  BF16    [T][hidden]           RMSNorm(x) * g_attn
 *   q      BF16    [T][n_heads*head_dim] q after RoPE, heads in order, element i of a
 *                                        head at i (RoPE pairs i, i + head_dim/2)
 *   o      BF16    [T][n_heads*head_dim] attention output
 *   h      float32 [T][hidden]           x + o W_o^T
 *   h_hat  BF16    [T][hidden]           RMSNorm(h) * g_ffn
 *   a      BF16    [T][intermediate]     SiLU(x_hat2 W_gate^T) * (x_hat2 W_up^T)
 * The new tokens' K and V are in the KV pool at their slots.  Host-only; no GPU
 * work.  Returns LL_ERR_INVALID_ARG for an invalid cfg or sizes. */
typedef struct {
    size_t x_hat, q, o, h, h_hat, a;
} ll_checkpoints;

int ll_workspace_checkpoints(const ll_config* cfg, int32_t max_tokens, int32_t max_blocks,
                             ll_checkpoints* out);

/* Execution modes of a layer call (page "ATB fused-operator matrix and KV-cache
 * management", section on the engineering limits of fusion granularity, which
 * names a step-by-step mode, a fused mode and a fused mode with verification
 * checkpoints).  LL_MODE_FUSED is the fused chain of ll_layer_prefill and
 * ll_layer_decode_step, whose kernel outputs stay readable through
 * ll_workspace_checkpoints (the checkpointed mode needs nothing more).
 * LL_MODE_STEP_BY_STEP runs every operator of the chain as its own kernel and
 * keeps every intermediate: RMSNorm, the merged QKV Linear (float32 output),
 * RotaryEmbedding, the slot mapping, ReshapeAndCache, attention, the O Linear,
 * the residual add, RMSNorm, the merged gate/up Linear, SiLU * up, the down
 * Linear and the residual add.  Its element-wise arithmetic is the fused
 * epilogues', so the two modes compute the same values; it exists to locate a
 * wrong result by comparing one operator at a time.  It takes BF16 pools. */
#define LL_MODE_FUSED 0
#define LL_MODE_STEP_BY_STEP 1

/* Workspace bytes for calls in `mode` (LL_MODE_FUSED: ll_workspace_size). */
size_t ll_workspace_size_mode(const ll_config* cfg, int32_t max_tokens, int32_t max_blocks, int32_t mode);

/* The step-by-step mode's extra intermediates, as byte offsets from the start of a
 * workspace sized by ll_workspace_size_mode(cfg, max_tokens, max_blocks,
 * LL_MODE_STEP_BY_STEP); the offsets of ll_workspace_checkpoints hold in that
 * workspace too.  After a step-by-step call over T tokens, row t < T of:
 *   qkv      float32 [T][(n_heads + 2 n_kv_heads) head_dim]  x_hat W_qkv^T before RoPE, in the
 *            packed column order: within each Q and K head column 2i holds element i and
 *            2i + 1 element i + head_dim/2; V heads in element order
 *   k, v     BF16    [T][n_kv_heads head_dim]   K after RoPE and V, element order
 *   slots    int32   [T]                        cache slot of each token (-1 if invalid)
 *   o_proj   float32 [T][hidden]                o W_o^T
 *   gate_up  float32 [T][2 intermediate]        h_hat W_gate^T and h_hat W_up^T, interleaved
 *                                               (column 2j gate j, 2j + 1 up j)
 *   down     float32 [T][hidden]                a W_down^T
 * Host-only; no GPU work. */
typedef struct {
    size_t qkv, k, v, slots, o_proj, gate_up, down;
} ll_step_checkpoints;

int ll_workspace_step_checkpoints(const ll_config* cfg, int32_t max_tokens, int32_t max_blocks,
                                  ll_step_checkpoints* out);

/* Prefill: x BF16 [batch*seq_len, hidden], token-major; token t belongs to
 * sequence t / seq_len and sits at positions[t] (int32 [batch*seq_len]).
 * Writes every token's K and V (after RoPE on K) into the pool at
 * block_table[seq][pos / block_size], offset pos % block_size; then every
 * query at position p attends (causally, GQA) over cache positions 0..p of
 * its sequence, which therefore must already be cached below this call's
 * first position (chunked prefill).  Writes y BF16 [batch*seq_len, hidden];
 * y must not alias x.  The chain page's prefill path. */
int ll_layer_prefill(const ll_config* cfg, const void* packed, const void* x,
                     const int32_t* positions, int32_t batch, int32_t seq_len,
                     const ll_kv_pool* pool, const int32_t* block_table, int32_t max_blocks,
                     void* y, void* workspace, size_t workspace_bytes, int32_t* status,
                     void* stream);

/* Decode step: x BF16 [batch, hidden], one new token per sequence.
 * context_lens (int32 [batch]) counts each sequence's cache INCLUDING the new
 * token, which is written at position context_lens[b] - 1; its query attends
 * over positions 0..context_lens[b]-1.  y BF16 [batch, hidden].  The chain
 * page's decode path (one-row query against the cached K/V). */
int ll_layer_decode_step(const ll_config* cfg, const void* packed, const void* x,
                         const ll_kv_pool* pool, const int32_t* block_table, int32_t max_blocks,
                         const int32_t* context_lens, int32_t batch, void* y, void* workspace,
                         size_t workspace_bytes, int32_t* status, void* stream);

/* ll_layer_prefill and ll_layer_decode_step with an execution mode (LL_MODE_FUSED or
 * LL_MODE_STEP_BY_STEP; anything else is LL_ERR_INVALID_ARG).  Arguments as there; the
 * workspace comes from ll_workspace_size_mode for the same mode. */
int ll_layer_prefill_mode(const ll_config* cfg, const void* packed, const void* x, const int32_t* positions,
                          int32_t batch, int32_t seq_len, const ll_kv_pool* pool, const int32_t* block_table,
                          int32_t max_blocks, void* y, void* workspace, size_t workspace_bytes, int32_t* status,
                          int32_t mode, void* stream);
int ll_layer_decode_step_mode(const ll_config* cfg, const void* packed, const void* x, const ll_kv_pool* pool,
                              const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                              int32_t batch, void* y, void* workspace, size_t workspace_bytes, int32_t* status,
                              int32_t mode, void* stream);

/* ll_layer_decode_step over an INT8 pool: the new tokens' K and V (after RoPE,
 * BF16) are quantised into the pool as ll_reshape_and_cache_q8 does, and the
 * attention reads code * scale (ll_paged_attention_decode_q8).  head_dim 128;
 * workspace from ll_workspace_size; other arguments as ll_layer_decode_step.
 * (Prefill into an INT8 pool is not provided.) */
int ll_layer_decode_step_q8(const ll_config* cfg, const void* packed, const void* x, const ll_kv_pool_q8* pool,
                            const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                            int32_t batch, void* y, void* workspace, size_t workspace_bytes, int32_t* status,
                            void* stream);

/* ReshapeAndCache (paging page, section "KV Cache memory wall",
 * ReshapeAndCacheOperation): k, v BF16 [tokens, n_kv_heads, head_dim];
 * slot_mapping int32 [tokens]; token t's rows go to
 * pool[slot / block_size, :, slot % block_size, :].  slot -1 skips the token;
 * slot >= num_blocks*block_size sets LL_DEV_BAD_SLOT and skips it.  Bit-exact
 * copy.  head_dim a multiple of 8. */
int ll_reshape_and_cache(const void* k, const void* v, const int32_t* slot_mapping, int32_t tokens,
                         int32_t n_kv_heads, int32_t head_dim, int32_t block_size,
                         const ll_kv_pool* pool, int32_t* status, void* stream);


/* ReshapeAndCache into an INT8 pool, quantising online: for token t and KV head h,
 * scale = max_i |row_i| / 127 and code_i = round-half-even(row_i / scale) in
 * float32 (IEEE division), clipped to [-127, 127]; a row of zeros gets scale 0
 * and codes 0.  Arguments and slot rules as ll_reshape_and_cache; head_dim a
 * multiple of 32, at most 256.  Codes and scales are bit-exact. */
int ll_reshape_and_cache_q8(const void* k, const void* v, const int32_t* slot_mapping, int32_t tokens,
                            int32_t n_kv_heads, int32_t head_dim, int32_t block_size,
                            const ll_kv_pool_q8* pool, int32_t* status, void* stream);

/* Workspace bytes for ll_paged_attention_decode. */
size_t ll_attention_workspace_size(int32_t batch, int32_t n_heads, int32_t head_dim,
                                   int32_t max_blocks, int32_t block_size);

/* Decode attention over the paged cache (chain page, section "KV Cache and
 * the operators", flash_attention_decode; paging page PagedAttentionOperation):
 * q BF16 [batch, n_heads, head_dim]; sequence b's query head h attends over
 * positions 0..context_lens[b]-1 of KV head h / (n_heads / n_kv_heads) with
 * softmax(q k^T * scale).  out BF16 [batch, n_heads, head_dim]; a sequence
 * with context length 0 gets zero rows.  head_dim 64 or 128, n_heads /
 * n_kv_heads <= 16, block_size a power of two in [16, 256]. */
int ll_paged_attention_decode(const void* q, const ll_kv_pool* pool, const int32_t* block_table,
                              int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                              int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                              int32_t block_size, float scale, void* out, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream);

/* ll_paged_attention_decode over an INT8 pool: the cached rows are code * scale
 * (paging page, section "KV Cache quantisation": dequantised as the cache block
 * is loaded).  head_dim 128; workspace sized by ll_attention_workspace_size; the
 * other arguments and limits as ll_paged_attention_decode. */
int ll_paged_attention_decode_q8(const void* q, const ll_kv_pool_q8* pool, const int32_t* block_table,
                                 int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                                 int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                 int32_t block_size, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* status, void* stream);

/* ll_paged_attention_decode for callers that cannot allocate device memory.
 * The pages have no counterpart of this call.  Some callers only own the
 * buffers they pass in: a plugin that receives input and output tensors from
 * a host framework with no hook for extra workspace, or code running where a
 * device allocation would synchronise the device or bypass the allocator that
 * owns the memory.  This variant takes the same arguments minus the workspace
 * and keeps the per-split partial results in a fixed device array inside the
 * library (32 MiB; every GPU that loads the library holds it until the
 * process exits).  It allocates nothing and calls no allocator.
 *  - Limit: with rows = batch * n_heads * ceil(max_blocks * block_size / 1024)
 *    (one per 1024-key split of every query head), the call needs
 *    rows * ((head_dim + 2) * 4 + 16) + 16 bytes of the array (per row the
 *    float32 partial output, its running max and sum, and a 16-byte entry of
 *    the splits' dispatch order; then a 16-byte pad);
 *    ll_attention_workspace_size gives the same figure rounded up to a
 *    multiple of 256.  Beyond 32 MiB it returns LL_ERR_UNSUPPORTED
 *    (ll_last_error gives the sizes) and launches nothing.
 *  - The first call on a device resolves the array's device address (this may
 *    load the library's device code); make that first call before any stream
 *    capture on the device.
 *  - All calls share the one array and each overwrites what it uses (nothing
 *    in it needs to start at zero): calls that may overlap on the GPU (other
 *    streams, other host threads) race on it and must be serialised.
 * Results equal ll_paged_attention_decode's for the same inputs. */
int ll_paged_attention_decode_noalloc(const void* q, const ll_kv_pool* pool,
                                      const int32_t* block_table, int32_t max_blocks,
                                      const int32_t* context_lens, int32_t batch, int32_t n_heads,
                                      int32_t n_kv_heads, int32_t head_dim, int32_t block_size,
                                      float scale, void* out, int32_t* status, void* stream);

/* Workspace bytes for ll_linear. */
size_t ll_linear_workspace_size(int32_t m, int32_t n, int32_t k);

/* Plain Linear y = x w^T (the chain page's Q/K/V, Output, Gate/Up and Down
 * Linear without their fused epilogues): x BF16 [m, k], w BF16 [n, k],
 * y BF16 [m, n], float32 accumulation.  n and k multiples of 16.  Runs the
 * same tensor-core GEMM the layer uses (m <= 256 takes the decode form). */
int ll_linear(const void* x, const void* w, void* y, int32_t m, int32_t n, int32_t k,
              void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* ---- Operators around the cache that the layer does not fuse.  The pages name
 * the steps (RotaryEmbedding, the paged cache and its quantisation); the forms
 * below (frequency scaling, scales per block, block copies) are this library's. */

#define LL_BF16 0
#define LL_F32 1

#define LL_ROPE_HALF 0         /* pair i is elements (i, i + rotary_dim / 2) */
#define LL_ROPE_INTERLEAVED 1  /* pair i is elements (2 i, 2 i + 1) */

#define LL_ROPE_FORWARD 0
#define LL_ROPE_BACKWARD 1     /* the gradient: the transposed rotation */

/* Inverse frequencies w_i = theta^(-2 i / rotary_dim), i < rotary_dim / 2, and
 * how a table scales them for contexts beyond the trained one: */
#define LL_ROPE_PLAIN 0        /* w */
#define LL_ROPE_LINEAR 1       /* w / factor */
#define LL_ROPE_NTK 2          /* w with theta * factor^(rotary_dim / (rotary_dim - 2)) */
#define LL_ROPE_BANDED 3       /* pairs that turn >= high_turns times over original_max_position keep w, those
                                * that turn <= low_turns times get w / factor, linear in the turns between */
#define LL_ROPE_YARN 4         /* the same two ends, linear in the pair index between the pairs (rounded
                                * outwards) that turn high_turns and low_turns times; cos and sin times
                                * attention_factor (0: 0.1 ln(factor) + 1) */

/* rotary_dim even, 2 .. 1024; theta > 1; factor >= 1 unless plain.  The fields
 * from original_max_position on are read for BANDED and YARN only
 * (attention_factor for YARN only): 0 < low_turns < high_turns. */
typedef struct {
    int32_t rotary_dim;
    int32_t scaling;
    float theta;
    float factor;
    int32_t original_max_position;
    float low_turns, high_turns;
    float attention_factor;
} ll_rope_config;

/* Bytes of a cos/sin table of max_position positions (0 if cfg is invalid). */
size_t ll_rope_table_size(const ll_rope_config* cfg, int32_t max_position);

/* Fills `table` (device, 16-byte aligned): float32 [max_position][rotary_dim / 2]
 * pairs (cos, sin) of position * frequency, computed in float64.  Setup-time
 * call, asynchronous on `stream`. */
int ll_rope_table(const ll_rope_config* cfg, int32_t max_position, void* table, size_t table_bytes, void* stream);

/* The same table into packed weights (ll_pack_weights of `cfg`), in place of the
 * plain one: every layer call with `packed` then rotates by the scaled
 * frequencies.  rope->rotary_dim must be cfg->head_dim (the layer rotates whole
 * heads, half-split).  Must not run while a layer call reads `packed`. */
int ll_pack_rope(const ll_config* cfg, const ll_rope_config* rope, void* packed, size_t packed_bytes, void* stream);

/* Rotary positions: q [tokens, n_heads, head_dim] and k [tokens, n_kv_heads,
 * head_dim] of `dtype` (LL_BF16 or LL_F32), rows of tokens q_stride and k_stride
 * elements apart (views of a merged QKV output).  Pair i of every head turns by
 * the angle of table[positions[t]][i]: (a, b) -> (a c - b s, b c + a s), float32
 * arithmetic, rounded once; LL_ROPE_BACKWARD is the transpose (s -> -s), the
 * gradient of the forward call.  Elements from rotary_dim on are copied.  Either
 * of q and k may be left out (its head count 0).  An output may be its input
 * (same pointer and stride); otherwise it must share no byte with the inputs or the
 * other output (columns of one buffer at the same stride do not).  A token whose position is outside 0 .. max_position - 1 sets
 * LL_DEV_BAD_POSITION and its rows are not written.  head_dim <= 1024. */
int ll_rope(const void* q, const void* k, int32_t dtype, const int32_t* positions, int32_t tokens, int32_t n_heads,
            int32_t n_kv_heads, int32_t head_dim, int32_t rotary_dim, int32_t layout, int32_t direction, int64_t q_stride,
            int64_t k_stride, const void* table, int32_t max_position, void* q_out, void* k_out, int64_t q_out_stride,
            int64_t k_out_stride, int32_t* status, void* stream);

/* Q or K heads of `tokens` tokens: [tokens][n_heads][head_dim], rows of tokens
 * `stride` elements apart (views of a merged QKV output).  n_heads 0: none. */
typedef struct {
    void* data;
    int64_t stride;
    int32_t n_heads;
} ll_head_rows;

/* Norms of the Q and K heads and their rotary positions in one pass: every head row x
 * of q and k becomes R(p) (x / sqrt(mean(x^2) + eps) * gain), R the rotation of ll_rope
 * at the token's position (elements from rotary_dim on are normed only), float32
 * arithmetic, rounded once to `dtype` (squares are summed in float32: heads with
 * elements beyond 2^58 are not supported).  gains float32 [head_dim], one for all Q heads
 * and one for all K heads; eps > 0.  Positions, table, layout and limits as ll_rope; an
 * output may be its input (same pointer and stride), otherwise it must share no byte with
 * the inputs or the other output.  Rows of bad positions are not written. */
int ll_norm_rope(const ll_head_rows* q, const ll_head_rows* k, int32_t dtype, const float* q_gain, const float* k_gain,
                 float eps, const int32_t* positions, int32_t tokens, int32_t head_dim, int32_t rotary_dim, int32_t layout,
                 const void* table, int32_t max_position, const ll_head_rows* q_out, const ll_head_rows* k_out,
                 int32_t* status, void* stream);

/* Workspace bytes for ll_norm_rope_backward (0 if head_dim is not supported). */
size_t ll_norm_rope_backward_workspace_size(int32_t head_dim);

/* The gradient of ll_norm_rope: q and k are its inputs, dq and dk the gradients of its
 * outputs.  Writes the gradients of the inputs (q_grad, k_grad, of `dtype`; each may be dq or
 * dk itself, same pointer and stride, and otherwise shares no byte with any other tensor)
 * and of the gains (float32 [head_dim], sums over all tokens and heads in float32 in a fixed
 * order: the same bits every time; zeros for no tokens).  A token of a bad position is left
 * out: its rows are not written and its gain terms not counted.  The workspace needs no initial
 * contents; calls that may overlap on the GPU need one each. */
int ll_norm_rope_backward(const ll_head_rows* dq, const ll_head_rows* dk, const ll_head_rows* q, const ll_head_rows* k,
                          int32_t dtype, const float* q_gain, const float* k_gain, float eps, const int32_t* positions,
                          int32_t tokens, int32_t head_dim, int32_t rotary_dim, int32_t layout, const void* table,
                          int32_t max_position, const ll_head_rows* q_grad, const ll_head_rows* k_grad, float* q_gain_grad,
                          float* k_gain_grad, void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* A KV pool of 8-bit floating-point codes (e4m3, largest 448) with one float32
 * scale per block of tokens and KV head.  A cached row reads back as code *
 * scale.  ll_append_to_cache_f8 writes powers of two as scales; the attention
 * takes any finite scales >= 0 (0: the block's rows are zeros).  A cached row counts
 * in a query's answer down to about 2^-27 of the largest probability times V scale
 * that the query itself sums; blocks that it does not see take no bits from the rest. */
typedef struct {
    void* k;              /* e4m3 [num_blocks, n_kv_heads, block_size, head_dim] */
    void* v;              /* same shape */
    float* k_scale;       /* float32 [num_blocks, n_kv_heads] */
    float* v_scale;       /* same shape */
    int32_t num_blocks;
} ll_kv_pool_f8;

/* Appends new tokens' K and V (after RoPE) to an e4m3 cache.  k, v BF16 [tokens,
 * n_kv_heads, head_dim], rows of tokens k_stride and v_stride elements apart
 * (multiples of 8).  Sequence b's new tokens are rows cu_new[b] .. cu_new[b+1]-1
 * (int32 [batch + 1], device; none where equal, at most max_new) and take
 * positions context_lens[b] - n .. context_lens[b] - 1 of its block table row
 * (context_lens counts them).  cu_new NULL: one new token per sequence (tokens =
 * batch, max_new = 1).
 * Per block and KV head the scale is the smallest power of two s >= 2^-117 with
 * |x| <= 448 s for every finite value in the block so far (0 while all are zeros):
 * a call that writes a block's first token starts the block afresh, a later one
 * keeps s' = max(s, scale of its rows) and, where that is larger, rounds the
 * block's earlier rows again to e4m3(code * s / s').  New codes are e4m3(x / s'),
 * nearest even; infinities saturate (to 448 s', so to 0 beside zeros alone), NaN
 * stays NaN.  Bit-exact.  Rows behind the
 * last new token, and blocks that get no token, keep their bytes.
 * Two sequences of a call must not append to the same physical block (fork it
 * with ll_copy_blocks first): its contents would be unspecified.
 * Counts that do not fit together (n < 0, n > max_new, n > context_lens[b], rows
 * beyond `tokens`, a context beyond the table) set LL_DEV_BAD_POSITION and skip
 * the sequence; a bad block sets LL_DEV_BAD_BLOCK and is skipped.  Limits as
 * ll_paged_attention_decode_f8, and n_kv_heads times the blocks that max_new tokens
 * can touch below 2^30. */
int ll_append_to_cache_f8(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* cu_new,
                          int32_t tokens, const int32_t* context_lens, int32_t batch, int32_t max_new, int32_t n_kv_heads,
                          int32_t head_dim, int32_t block_size, const ll_kv_pool_f8* pool, const int32_t* block_table,
                          int32_t max_blocks, int32_t* status, void* stream);

/* Workspace bytes for ll_paged_attention_decode_f8 (independent of the context
 * lengths and of the table's width). */
size_t ll_attention_decode_f8_workspace_size(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);

/* ll_paged_attention_decode over an e4m3 cache: q BF16 [batch, n_heads, head_dim],
 * one query per sequence over positions 0 .. context_lens[b] - 1, softmax(q k^T *
 * scale) v; zero rows where there is no key (context length 0, or no valid block), or
 * where every score is -infinity (an infinity in q).
 * Whatever lies in the cache behind a context, NaN too, is not read into the
 * result.  head_dim 64 or 128, n_heads / n_kv_heads <= 16, block_size a power of
 * two in [16, 256], batch <= 65535, max_blocks * block_size <= 2^30, scale finite
 * and >= 0.  The workspace needs no initial contents; calls that may overlap on
 * the GPU (other streams, graphs replayed at once) need one each. */
int ll_paged_attention_decode_f8(const void* q, const ll_kv_pool_f8* pool, const int32_t* block_table, int32_t max_blocks,
                                 const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim, int32_t block_size, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* status, void* stream);

/* Workspace bytes for ll_paged_attention_prefill_f8. */
size_t ll_attention_prefill_f8_workspace_size(int32_t batch, int32_t tokens, int32_t max_new, int32_t n_heads,
                                              int32_t n_kv_heads, int32_t head_dim);

/* Causal attention of a ragged batch of new tokens over an e4m3 cache that already
 * holds them (ll_append_to_cache_f8 with the same cu_new and context_lens): q and
 * out BF16 [tokens, n_heads, head_dim]; row cu_new[b] + i sits at position p =
 * context_lens[b] - n + i and attends over positions 0 .. p of its sequence.
 * Covers prompts, chunks behind a cached prefix and a few tokens per sequence.
 * Rows of `out` that belong to no sequence, or to one whose counts do not fit
 * together (LL_DEV_BAD_POSITION, as ll_append_to_cache_f8), are not written.
 * What lies in the cache behind a sequence's context is not read into the result;
 * a NaN among the new tokens' V may reach earlier rows of the call.  Limits and
 * workspace rule as ll_paged_attention_decode_f8, and batch * n_kv_heads times the
 * pairs of query tiles of max_new tokens (floor(128 n_kv_heads / n_heads) tokens a
 * tile) at most 2^30. */
int ll_paged_attention_prefill_f8(const void* q, const int32_t* cu_new, int32_t tokens, const ll_kv_pool_f8* pool,
                                  const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                  int32_t batch, int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                  int32_t block_size, float scale, void* out, void* workspace, size_t workspace_bytes,
                                  int32_t* status, void* stream);

/* Workspace bytes for layer calls over an e4m3 pool (max_tokens and max_blocks as
 * for ll_workspace_size; the checkpoints of ll_workspace_checkpoints hold in it). */
size_t ll_workspace_size_f8(const ll_config* cfg, int32_t max_tokens, int32_t max_blocks);

/* ll_layer_prefill over an e4m3 pool: every sequence's seq_len new tokens take its
 * last positions, context_lens[b] - seq_len .. context_lens[b] - 1 (a prompt, a
 * chunk behind a cached prefix, or a few tokens).  Their K and V go into the pool
 * as ll_append_to_cache_f8 does, the attention is ll_paged_attention_prefill_f8's.
 * x and y as ll_layer_prefill. */
int ll_layer_prefill_f8(const ll_config* cfg, const void* packed, const void* x, const int32_t* context_lens, int32_t batch,
                        int32_t seq_len, const ll_kv_pool_f8* pool, const int32_t* block_table, int32_t max_blocks, void* y,
                        void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* ll_layer_decode_step over an e4m3 pool (ll_append_to_cache_f8 and
 * ll_paged_attention_decode_f8); the other arguments as there, workspace from
 * ll_workspace_size_f8. */
int ll_layer_decode_step_f8(const ll_config* cfg, const void* packed, const void* x, const ll_kv_pool_f8* pool,
                            const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                            void* y, void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* ---- Attention weights, and evictions by them.  `weights` is float32 [batch,
 * n_kv_heads, weights_width], the caller's: for each sequence, KV head and cached
 * position the sum of the softmax probabilities that queries have given it, over the
 * query heads of the KV head and over all calls since the caller zeroed it.  Calls that
 * add to the same weights must not overlap on the GPU. */

/* Workspace bytes for ll_paged_attention_decode_weights(_q8) (0 for sizes that these
 * refuse).  Beside the partials it holds a float32 score for each query head and
 * position of the table. */
size_t ll_attention_decode_weights_workspace_size(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                  int32_t max_blocks, int32_t block_size);

/* ll_paged_attention_decode (same output) that also adds each position's attention
 * weight: weights[b][hk][p] += sum over the query heads h of hk of softmax(q_h k^T *
 * scale)[p], for p < context_lens[b].  A position without a valid block, and a query
 * without any score above -infinity, add nothing; positions from weights_width on set
 * LL_DEV_BAD_POSITION and are not added.  What lies behind a context keeps its value.
 * The sums are float32 and the same bits every time.  head_dim 64 or 128, n_heads /
 * n_kv_heads <= 16, block_size a power of two in [16, 256], batch <= 65535, max_blocks *
 * block_size <= 2^30, num_blocks * n_kv_heads * block_size < 2^31, scale finite and >= 0.
 * The workspace needs no initial contents; calls that may overlap on the GPU need one each. */
int ll_paged_attention_decode_weights(const void* q, const ll_kv_pool* pool, const int32_t* block_table, int32_t max_blocks,
                                      const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                      int32_t head_dim, int32_t block_size, float scale, float* weights, int32_t weights_width,
                                      void* out, void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* The same over an INT8 pool (output as ll_paged_attention_decode_q8; head_dim 128).  Queries
 * enter the scores, and so the weights, as FP16 there: exact between 2^-14 and 65504 in
 * size, in steps of 2^-24 below; an element beyond is infinite. */
int ll_paged_attention_decode_weights_q8(const void* q, const ll_kv_pool_q8* pool, const int32_t* block_table, int32_t max_blocks,
                                         const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                         int32_t head_dim, int32_t block_size, float scale, float* weights, int32_t weights_width,
                                         void* out, void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* Workspace bytes for ll_paged_attention_weights (0 for sizes that it refuses), on the
 * current device.  Enough for calls of fewer sequences, tokens, rows of a sequence
 * (max_new) or blocks too: the size does not depend on batch and max_new. */
size_t ll_attention_weights_workspace_size(int32_t batch, int32_t tokens, int32_t max_new, int32_t n_heads, int32_t n_kv_heads,
                                           int32_t head_dim, int32_t max_blocks, int32_t block_size);

/* The weights alone, of a ragged batch of query rows (a whole prompt, a chunk, or the last
 * rows of each context): q BF16 [tokens, n_heads, head_dim] after RoPE, sequence b's rows
 * cu_new[b] .. cu_new[b+1]-1 (int32 [batch + 1], device; at most max_new), row i of n at
 * position context_lens[b] - n + i, seeing positions 0 .. that one of the K pool (BF16), which
 * already holds them.  Adds to weights as ll_paged_attention_decode_weights, summed over the
 * rows too (the same bits every time); a row of NaN scores gives NaN to what it sees.
 * Sequences whose counts do not fit together (n < 0, n > max_new, n > context_lens[b], rows
 * beyond `tokens`, a context beyond the table) set LL_DEV_BAD_POSITION and add nothing.
 * Limits and workspace rule as ll_paged_attention_decode_weights, and batch * n_kv_heads
 * times the CTAs that max_new rows ask for below 2^31 (LL_ERR_UNSUPPORTED). */
int ll_paged_attention_weights(const void* q, const int32_t* cu_new, int32_t tokens, const void* k_pool, int32_t num_blocks,
                               const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                               int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t block_size,
                               float scale, float* weights, int32_t weights_width, void* workspace, size_t workspace_bytes,
                               int32_t* status, void* stream);

/* Workspace bytes for ll_layer_decode_step_weights(_q8) (sizes as for ll_workspace_size;
 * the checkpoints of ll_workspace_checkpoints hold in it). */
size_t ll_workspace_size_weights(const ll_config* cfg, int32_t max_tokens, int32_t max_blocks);

/* ll_layer_decode_step (and _q8) that adds its attention weights as
 * ll_paged_attention_decode_weights does, and can rotate by positions of the uncut sequence:
 * positions int32 [batch] are the new tokens' rotary positions (NULL: context_lens[b] - 1),
 * context_lens[b] - 1 stays the place in the cache.  A position beyond the table sets
 * LL_DEV_BAD_POSITION: that token's K and V are not written, and its sequence's y and what is
 * added to its weights are unspecified.  y as that call's for the same positions.  Limits of
 * both calls. */
int ll_layer_decode_step_weights(const ll_config* cfg, const void* packed, const void* x, const ll_kv_pool* pool,
                                 const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                 const int32_t* positions, int32_t batch, float* weights, int32_t weights_width, void* y,
                                 void* workspace, size_t workspace_bytes, int32_t* status, void* stream);
int ll_layer_decode_step_weights_q8(const ll_config* cfg, const void* packed, const void* x, const ll_kv_pool_q8* pool,
                                    const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                    const int32_t* positions, int32_t batch, float* weights, int32_t weights_width, void* y,
                                    void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* One tensor of a paged pool, by the bytes of a cached row (K or V rows, codes, scales). */
typedef struct {
    void* data;           /* device, [num_blocks][n_kv_heads][block_size][row_bytes], 4-byte aligned (16: faster) */
    int64_t row_bytes;    /* a multiple of 4, at most 4096 */
} ll_row_tensor;

/* Evicts cached rows by their weights, in place and for every KV head by itself.  With n =
 * context_lens[b] and m = min(n, keep[b]) (keep NULL: max_keep for all), each KV head of
 * sequence b keeps m rows: the last min(recent, m), the first min(sinks, m - those), and of
 * the rows between the ones of the largest weight (ties: the lowest position; NaN counts
 * below every number).  The kept rows move, in order, to positions 0 .. m - 1 of the
 * sequence's blocks in all tensors (a HOST array of 1 .. 8, read before the call returns).
 * Writes
 *   kept [batch, n_kv_heads, max_keep]  the position that row j had, -1 from m on (int32)
 *   new_lens [batch]                    m (int32)
 *   weights_out                         as weights: its rows [0, m) the kept ones', [m, n) zeros,
 *                                       the rest as it was; weights itself or memory apart from it
 * Blocks behind the last one that m rows need are free for the caller to reuse; a block that
 * a moved row is written to must not be part of another sequence (fork it with ll_copy_blocks first)
 * or stand twice in the table.  Tensors and outputs that share memory with each other or with
 * weights, context_lens or keep are refused (LL_ERR_INVALID_ARG).
 * Cached keys keep the rotary positions they were written with: go on with positions of the
 * uncut sequence, not with the cut length.
 * Sizes that do not fit (n < 0 or beyond the table or weights_width, keep[b] < 0, m >
 * max_keep) set LL_DEV_BAD_POSITION, a bad block among the n rows of a sequence that loses any sets
 * LL_DEV_BAD_BLOCK: that sequence's kept are -1, its new_lens n, and nothing else of it is touched.
 * The same rows every time.  max_keep >= 1, sinks, recent >= 0; block_size a power of two in [16,
 * 256], batch <= 65535, n_kv_heads <= 32767, max_blocks * block_size <= 2^30, num_blocks *
 * n_kv_heads * block_size < 2^31. */
int ll_evict_rows(const ll_row_tensor* tensors, int32_t n_tensors, int32_t num_blocks, int32_t n_kv_heads, int32_t block_size,
                  const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                  const float* weights, int32_t weights_width, const int32_t* keep, int32_t max_keep, int32_t sinks,
                  int32_t recent, float* weights_out, int32_t* kept, int32_t* new_lens, int32_t* status, void* stream);

/* One tensor of a pool whose first dimension is the physical block: K or V codes,
 * or their scales, of one layer. */
typedef struct {
    void* data;           /* device, [num_blocks][block_bytes], 4-byte aligned (16: faster) */
    int64_t block_bytes;  /* a multiple of 4, at most 2^30 */
} ll_block_tensor;

/* Copies blocks in all tensors at once (the pools of every layer share their block
 * ids): block pairs[i][0] to block pairs[i][1] (int32 [max_pairs][2], device, 8-byte
 * aligned), for i below *n_pairs (device int32; NULL: max_pairs; at most max_pairs
 * are done).  `tensors` is a HOST array, read before the call returns.  A pair (-1,
 * -1) is skipped; any other id outside 0 .. num_blocks - 1 sets LL_DEV_BAD_BLOCK and
 * skips the pair.  No block may be the destination of two pairs, or the destination
 * of one and the source of another: its contents would be unspecified. */
int ll_copy_blocks(const ll_block_tensor* tensors, int32_t n_tensors, int32_t num_blocks, const int32_t* pairs,
                   int32_t max_pairs, const int32_t* n_pairs, int32_t* status, void* stream);

/* The plan that packs the blocks in use to the front of a pool.  In use are the
 * ids >= 0 in block_table [rows, max_blocks]; a block that several rows share
 * counts once.  With U of them, every block in use at or behind place U moves, in
 * ascending order, to the free places before U: the fewest moves, and no source is
 * a destination.  Writes, all int32 on the device:
 *   new_table [rows, max_blocks]  the table after the moves (may be block_table);
 *                                 negative entries stay as they are
 *   pairs [num_blocks / 2][2]     the moves (from, to), then (-1, -1)
 *   counts [2]                    U and the number of moves
 *   block_map [num_blocks]        each block's new id, -1 where not in use
 * An id >= num_blocks sets LL_DEV_BAD_BLOCK and stays as it is.  Then
 * ll_copy_blocks(tensors, ..., pairs, num_blocks / 2, counts + 1, ...) moves the
 * contents.  num_blocks <= 524288. */
int ll_compact_blocks(const int32_t* block_table, int32_t rows, int32_t max_blocks, int32_t num_blocks, int32_t* new_table,
                      int32_t* pairs, int32_t* counts, int32_t* block_map, int32_t* status, void* stream);

/* Launch tracing, for measurement (off by default).  ll_trace_begin creates
 * 2 * capacity CUDA events on the current device; until ll_trace_end, each
 * kernel launch the library makes is bracketed by two of them, recorded on
 * the launch's stream, and its kernel name kept.  ll_trace_end returns the
 * number of launches recorded (at most capacity; later ones are not traced).
 * Once the stream has been synchronised, ll_trace_elapsed_ms(i) is launch i's
 * duration in milliseconds (-1 on error) and ll_trace_name(i) its kernel.
 * Process-wide state, not thread-safe.  This is a measuring aid the pages do
 * not describe (their profiler is the graph timeline of the ATB debugging
 * section). */
int ll_trace_begin(int32_t capacity);
int32_t ll_trace_end(void);
float ll_trace_elapsed_ms(int32_t i);
const char* ll_trace_name(int32_t i);

/* Self-test of the in-kernel failure detection (not a layer operation): one
 * block of 64 threads waits on an mbarrier that nothing completes, with a
 * limit of limit_us microseconds (1 .. 2,000,000).  Each wait gives up, sets
 * LL_DEV_TIMEOUT in *status and adds 1 to *out (device int32, caller-zeroed),
 * and the kernel finishes normally: the context stays usable. */
int ll_selftest_bounded_wait(int32_t limit_us, int32_t* status, int32_t* out, void* stream);

/* Number of streaming multiprocessors the library sizes its grids for
 * (queried once per device), or -1 without a device. */
int ll_device_sm_count(void);

/* Upper bound on the CTAs of the prefill attention, which is persistent: each
 * CTA (one per SM by default) runs a fixed list of (sequence, query head,
 * 128-query tile) items back to back.  n <= 0 restores one per SM.  A smaller
 * bound leaves SMs to other work on the device, and lets small problems run
 * several items per CTA.  Applies to launches made after the call, from any
 * thread.  Always returns LL_OK. */
int ll_set_prefill_attention_ctas(int32_t n);

#ifdef __cplusplus
}
#endif

#endif /* LLAMA_LAYER_H */
