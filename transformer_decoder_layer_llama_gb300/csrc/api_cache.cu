// C ABI of the operators around the paged cache (declared in include/llama_layer.h): rotary positions,
// the e4m3 cache with block scales, block copies and compaction.  Checks arguments and enqueues launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../include/llama_layer.h"
#include "api_util.h"
#include "kernels.h"

using ll::aligned16;
using ll::align_up;
using ll::cuda_rc;

namespace {

constexpr int64_t kMaxPositions = 1LL << 30;   // block_table width times block_size

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

// `tokens` rows of `width` elements, `stride` elements apart.
struct Rows {
    const void* p;
    int64_t stride, width;
};
// Whether two such tensors may share a byte.  Rows of one buffer at the same stride (the heads of a merged QKV
// output) do not where their columns lie apart; other strides that meet count as sharing.
bool rows_overlap(const Rows& a, const Rows& b, int64_t tokens, int64_t esz) {
    const auto bytes = [&](const Rows& r) { return (size_t)(((tokens - 1) * r.stride + r.width) * esz); };
    if (!overlap(a.p, bytes(a), b.p, bytes(b))) return false;
    if (a.stride != b.stride || tokens == 1) return true;
    const int64_t step = a.stride * esz;
    const int64_t apart = (static_cast<const char*>(b.p) - static_cast<const char*>(a.p)) % step;
    const int64_t at = apart < 0 ? apart + step : apart;        // b's column in a's rows
    return at < a.width * esz || at + b.width * esz > step;
}

int rope_config_ok(const ll_rope_config* c) {
    if (!c || c->rotary_dim < 2 || c->rotary_dim % 2 != 0 || !(c->theta > 1.f) || !std::isfinite(c->theta))
        return LL_ERR_INVALID_ARG;
    if (c->rotary_dim > 1024) return LL_ERR_UNSUPPORTED;
    if (c->scaling < LL_ROPE_PLAIN || c->scaling > LL_ROPE_YARN) return LL_ERR_INVALID_ARG;
    if (c->scaling == LL_ROPE_PLAIN) return LL_OK;
    if (!(c->factor >= 1.f) || !std::isfinite(c->factor)) return LL_ERR_INVALID_ARG;
    if (c->scaling == LL_ROPE_NTK && c->rotary_dim == 2) return LL_ERR_INVALID_ARG;
    if (c->scaling == LL_ROPE_BANDED || c->scaling == LL_ROPE_YARN) {
        if (c->original_max_position <= 0 || !(c->low_turns > 0.f) || !(c->high_turns > c->low_turns) ||
            !std::isfinite(c->high_turns))
            return LL_ERR_INVALID_ARG;
    }
    if (c->scaling == LL_ROPE_YARN && (!(c->attention_factor >= 0.f) || !std::isfinite(c->attention_factor)))
        return LL_ERR_INVALID_ARG;
    return LL_OK;
}

ll::RopeTableArgs rope_table_args(const ll_rope_config* c) {
    ll::RopeTableArgs f{};
    const double two_pi = 6.283185307179586476925286766559, r = c->rotary_dim;
    f.rotary_dim = c->rotary_dim;
    f.scaling = c->scaling;
    f.theta = c->theta;
    f.factor = c->scaling == LL_ROPE_PLAIN ? 1.0 : (double)c->factor;
    f.magnitude = 1.0;
    if (c->scaling == LL_ROPE_NTK) {
        f.theta *= std::pow(f.factor, r / (r - 2.0));
        f.factor = 1.0;
    }
    if (c->scaling == LL_ROPE_BANDED || c->scaling == LL_ROPE_YARN) {
        f.original = c->original_max_position;
        f.low = c->low_turns;
        f.high = c->high_turns;
    }
    if (c->scaling == LL_ROPE_YARN) {
        // the (fractional) pair that turns t times over the original context
        const auto pair_of = [&](double t) { return r * std::log(f.original / (t * two_pi)) / (2.0 * std::log(f.theta)); };
        const double lo = std::max(std::floor(pair_of(f.high)), 0.0);
        const double hi = std::min(std::ceil(pair_of(f.low)), r - 1.0);
        f.ramp_lo = lo;
        f.ramp_width = std::max(hi - lo, 0.001);
        f.magnitude = c->attention_factor > 0.f ? (double)c->attention_factor : 0.1 * std::log(f.factor) + 1.0;
    }
    return f;
}

// The shape limits that every call over an e4m3 cache shares.
int f8_shape(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_blocks,
             const ll_kv_pool_f8* pool) {
    if (batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || max_blocks <= 0 || block_size <= 0) return LL_ERR_INVALID_ARG;
    if (!pool || !pool->k || !pool->v || !pool->k_scale || !pool->v_scale || pool->num_blocks <= 0) return LL_ERR_INVALID_ARG;
    if (!aligned16(pool->k) || !aligned16(pool->v)) return LL_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(pool->k_scale) | reinterpret_cast<uintptr_t>(pool->v_scale)) & 3u) != 0)
        return LL_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return LL_ERR_UNSUPPORTED;
    if (!ll::block_size_ok(block_size)) return LL_ERR_UNSUPPORTED;
    if (n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 16) return LL_ERR_UNSUPPORTED;
    if (batch > 65535 || n_kv_heads > 32767) return LL_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks * block_size > kMaxPositions) return LL_ERR_UNSUPPORTED;
    // rows of the pool are TMA coordinates
    if ((int64_t)pool->num_blocks * n_kv_heads * block_size > (1LL << 31) - 1) return LL_ERR_UNSUPPORTED;
    return LL_OK;
}

ll::AttnF8Args f8_args(const void* q, const ll_kv_pool_f8* pool, const int32_t* block_table, int32_t max_blocks,
                       const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                       int32_t block_size, float scale, void* out, int32_t* status) {
    ll::AttnF8Args a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k_pool = static_cast<const uint8_t*>(pool->k);
    a.v_pool = static_cast<const uint8_t*>(pool->v);
    a.k_scale = pool->k_scale;
    a.v_scale = pool->v_scale;
    a.context_lens = context_lens;
    a.block_table = block_table;
    a.batch = batch;
    a.max_blocks = max_blocks;
    a.num_blocks = pool->num_blocks;
    a.block_size = block_size;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.scale = scale;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.status = status;
    return a;
}

}  // namespace

extern "C" {

size_t ll_rope_table_size(const ll_rope_config* cfg, int32_t max_position) {
    if (rope_config_ok(cfg) != LL_OK || max_position <= 0) return 0;
    return (size_t)max_position * (cfg->rotary_dim / 2) * sizeof(float2);
}

int ll_rope_table(const ll_rope_config* cfg, int32_t max_position, void* table, size_t table_bytes, void* stream) {
    ll::clear_last_error();
    const int rc = rope_config_ok(cfg);
    if (rc != LL_OK) return rc;
    if (!table || max_position <= 0 || !aligned16(table) || table_bytes < ll_rope_table_size(cfg, max_position))
        return LL_ERR_INVALID_ARG;
    return cuda_rc(ll::launch_rope_scaled_table(static_cast<float2*>(table), max_position, rope_table_args(cfg),
                                                static_cast<cudaStream_t>(stream)));
}

int ll_rope(const void* q, const void* k, int32_t dtype, const int32_t* positions, int32_t tokens, int32_t n_heads,
            int32_t n_kv_heads, int32_t head_dim, int32_t rotary_dim, int32_t layout, int32_t direction, int64_t q_stride,
            int64_t k_stride, const void* table, int32_t max_position, void* q_out, void* k_out, int64_t q_out_stride,
            int64_t k_out_stride, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (dtype != LL_BF16 && dtype != LL_F32) return LL_ERR_INVALID_ARG;
    if (layout != LL_ROPE_HALF && layout != LL_ROPE_INTERLEAVED) return LL_ERR_INVALID_ARG;
    if (direction != LL_ROPE_FORWARD && direction != LL_ROPE_BACKWARD) return LL_ERR_INVALID_ARG;
    if (tokens < 0 || n_heads < 0 || n_kv_heads < 0 || n_heads + (int64_t)n_kv_heads <= 0 || head_dim <= 0 ||
        max_position <= 0 || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > head_dim)
        return LL_ERR_INVALID_ARG;
    if (head_dim > 1024 || n_heads > 4096 || n_kv_heads > 4096 || tokens > (1 << 24)) return LL_ERR_UNSUPPORTED;
    if (!table || !status || !aligned16(table)) return LL_ERR_INVALID_ARG;
    if (tokens == 0) return LL_OK;
    if (!positions) return LL_ERR_INVALID_ARG;
    const size_t esz = dtype == LL_F32 ? 4 : 2;
    const int64_t qw = (int64_t)n_heads * head_dim, kw = (int64_t)n_kv_heads * head_dim;
    if (n_heads > 0 && (!q || !q_out || q_stride < qw || q_out_stride < qw)) return LL_ERR_INVALID_ARG;
    if (n_kv_heads > 0 && (!k || !k_out || k_stride < kw || k_out_stride < kw)) return LL_ERR_INVALID_ARG;
    const int64_t big = 1LL << 34;                    // (2^24 rows of 4-byte elements: byte offsets stay in 64 bits)
    if (q_stride > big || k_stride > big || q_out_stride > big || k_out_stride > big) return LL_ERR_UNSUPPORTED;
    const void* ptrs[4] = {n_heads ? q : nullptr, n_kv_heads ? k : nullptr, n_heads ? q_out : nullptr,
                           n_kv_heads ? k_out : nullptr};
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % esz != 0) return LL_ERR_INVALID_ARG;
    // an output is its input itself (same rows), or shares no byte with either input or the other output
    const Rows in[2] = {{q, q_stride, qw}, {k, k_stride, kw}}, out[2] = {{q_out, q_out_stride, qw}, {k_out, k_out_stride, kw}};
    const bool q_in = n_heads > 0 && q == q_out && q_stride == q_out_stride;
    const bool k_in = n_kv_heads > 0 && k == k_out && k_stride == k_out_stride;
    const bool here[2] = {n_heads > 0, n_kv_heads > 0}, own[2] = {q_in, k_in};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (here[i] && here[j] &&
                ((!(i == j && own[i]) && rows_overlap(out[i], in[j], tokens, esz)) || (i < j && rows_overlap(out[i], out[j], tokens, esz))))
                return LL_ERR_INVALID_ARG;
    ll::RopeArgs a{};
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    a.positions = positions;
    a.table = static_cast<const float2*>(table);
    a.tokens = tokens;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.max_position = max_position;
    a.interleaved = layout == LL_ROPE_INTERLEAVED;
    a.backward = direction == LL_ROPE_BACKWARD;
    a.copy_tail = rotary_dim < head_dim && ((n_heads > 0 && !q_in) || (n_kv_heads > 0 && !k_in));
    a.status = status;
    return cuda_rc(ll::launch_rope(a, dtype == LL_F32, static_cast<cudaStream_t>(stream)));
}

int ll_append_to_cache_f8(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* cu_new,
                          int32_t tokens, const int32_t* context_lens, int32_t batch, int32_t max_new, int32_t n_kv_heads,
                          int32_t head_dim, int32_t block_size, const ll_kv_pool_f8* pool, const int32_t* block_table,
                          int32_t max_blocks, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!context_lens || !block_table || !status || tokens < 0 || max_new <= 0) return LL_ERR_INVALID_ARG;
    const int rc = f8_shape(batch, n_kv_heads, n_kv_heads, head_dim, block_size, max_blocks, pool);
    if (rc != LL_OK) return rc;
    if (!cu_new && (max_new != 1 || tokens != batch)) return LL_ERR_INVALID_ARG;
    if (tokens == 0) return LL_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        k_stride < (int64_t)n_kv_heads * head_dim || v_stride < (int64_t)n_kv_heads * head_dim)
        return LL_ERR_INVALID_ARG;
    if (!ll::append_f8_fits(std::min(max_new, tokens), n_kv_heads, block_size, max_blocks)) return LL_ERR_UNSUPPORTED;
    ll::AppendArgs a{};
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.cu_new = cu_new;
    a.context_lens = context_lens;
    a.block_table = block_table;
    a.k_pool = static_cast<uint8_t*>(pool->k);
    a.v_pool = static_cast<uint8_t*>(pool->v);
    a.k_scale = pool->k_scale;
    a.v_scale = pool->v_scale;
    a.tokens = tokens;
    a.batch = batch;
    a.max_new = std::min(max_new, tokens);
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.num_blocks = pool->num_blocks;
    a.max_blocks = max_blocks;
    a.max_context = max_blocks * block_size;
    a.status = status;
    return cuda_rc(ll::launch_append_f8(a, static_cast<cudaStream_t>(stream)));
}

size_t ll_attention_decode_f8_workspace_size(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    if (batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 16 ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return align_up(ll::attn_decode_f8_scratch_bytes(batch, n_heads, n_kv_heads, head_dim));
}

int ll_paged_attention_decode_f8(const void* q, const ll_kv_pool_f8* pool, const int32_t* block_table, int32_t max_blocks,
                                 const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim, int32_t block_size, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!q || !block_table || !context_lens || !out || !status || !(scale >= 0.f) || !std::isfinite(scale))
        return LL_ERR_INVALID_ARG;
    const int rc = f8_shape(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks, pool);
    if (rc != LL_OK) return rc;
    if (!aligned16(q) || !aligned16(out)) return LL_ERR_INVALID_ARG;
    const size_t need = ll_attention_decode_f8_workspace_size(batch, n_heads, n_kv_heads, head_dim);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return LL_ERR_WORKSPACE;
    ll::AttnF8Args a = f8_args(q, pool, block_table, max_blocks, context_lens, batch, n_heads, n_kv_heads, head_dim,
                               block_size, scale, out, status);
    a.tokens = batch;
    a.max_new = 1;
    return cuda_rc(ll::launch_attn_decode_f8(a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t ll_attention_prefill_f8_workspace_size(int32_t batch, int32_t tokens, int32_t max_new, int32_t n_heads,
                                              int32_t n_kv_heads, int32_t head_dim) {
    if (batch <= 0 || tokens < 0 || max_new <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 ||
        n_heads / n_kv_heads > 16 || (head_dim != 64 && head_dim != 128))
        return 0;
    return align_up(ll::attn_prefill_f8_scratch_bytes(head_dim));
}

int ll_paged_attention_prefill_f8(const void* q, const int32_t* cu_new, int32_t tokens, const ll_kv_pool_f8* pool,
                                  const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                  int32_t batch, int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                  int32_t block_size, float scale, void* out, void* workspace, size_t workspace_bytes,
                                  int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!cu_new || !block_table || !context_lens || !status || !(scale >= 0.f) || !std::isfinite(scale) || tokens < 0 ||
        max_new <= 0)
        return LL_ERR_INVALID_ARG;
    const int rc = f8_shape(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks, pool);
    if (rc != LL_OK) return rc;
    if (tokens > 0 && (!q || !out || !aligned16(q) || !aligned16(out))) return LL_ERR_INVALID_ARG;
    if (!ll::attn_prefill_f8_fits(batch, std::min(max_new, tokens), n_heads, n_kv_heads)) return LL_ERR_UNSUPPORTED;
    const size_t need = ll_attention_prefill_f8_workspace_size(batch, tokens, max_new, n_heads, n_kv_heads, head_dim);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return LL_ERR_WORKSPACE;
    ll::AttnF8Args a = f8_args(q, pool, block_table, max_blocks, context_lens, batch, n_heads, n_kv_heads, head_dim,
                               block_size, scale, out, status);
    a.cu_new = cu_new;
    a.tokens = tokens;
    a.max_new = std::min(max_new, tokens);
    return cuda_rc(ll::launch_attn_prefill_f8(a, workspace, static_cast<cudaStream_t>(stream)));
}

int ll_copy_blocks(const ll_block_tensor* tensors, int32_t n_tensors, int32_t num_blocks, const int32_t* pairs,
                   int32_t max_pairs, const int32_t* n_pairs, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!tensors || n_tensors <= 0 || num_blocks <= 0 || max_pairs < 0 || !status || (max_pairs > 0 && !pairs))
        return LL_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(pairs) & 7u) != 0) return LL_ERR_INVALID_ARG;
    const int64_t piece = ll::copy_blocks_piece_bytes();
    for (int32_t i = 0; i < n_tensors; ++i) {
        const ll_block_tensor& t = tensors[i];
        if (!t.data || t.block_bytes <= 0 || t.block_bytes % 4 != 0 || (reinterpret_cast<uintptr_t>(t.data) & 3u) != 0)
            return LL_ERR_INVALID_ARG;
        if (t.block_bytes > (1LL << 30)) return LL_ERR_UNSUPPORTED;
    }
    for (int32_t i0 = 0; i0 < n_tensors; i0 += ll::kCopyMaxTensors) {
        ll::CopyBlocksArgs a{};
        a.n_tensors = std::min(n_tensors - i0, ll::kCopyMaxTensors);
        a.num_blocks = num_blocks;
        a.max_pairs = max_pairs;
        a.pairs = pairs;
        a.n_pairs = n_pairs;
        a.status = status;
        for (int i = 0; i < a.n_tensors; ++i) {
            a.data[i] = tensors[i0 + i].data;
            a.bytes[i] = tensors[i0 + i].block_bytes;
            a.pieces[i + 1] = a.pieces[i] + (int)((a.bytes[i] + piece - 1) / piece);
        }
        if (ll::launch_copy_blocks(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) return LL_ERR_CUDA;
    }
    return LL_OK;
}

int ll_compact_blocks(const int32_t* block_table, int32_t rows, int32_t max_blocks, int32_t num_blocks, int32_t* new_table,
                      int32_t* pairs, int32_t* counts, int32_t* block_map, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (rows < 0 || max_blocks < 0 || num_blocks <= 0 || !counts || !block_map || !status) return LL_ERR_INVALID_ARG;
    const int64_t entries = (int64_t)rows * max_blocks;
    if (entries > 0 && (!block_table || !new_table)) return LL_ERR_INVALID_ARG;
    if (num_blocks > 1 && (!pairs || (reinterpret_cast<uintptr_t>(pairs) & 7u) != 0)) return LL_ERR_INVALID_ARG;
    if (num_blocks > ll::kCompactMaxBlocks) return LL_ERR_UNSUPPORTED;
    if (entries > 0 && block_table != new_table && overlap(block_table, entries * 4, new_table, entries * 4))
        return LL_ERR_INVALID_ARG;
    ll::CompactArgs a{};
    a.table = block_table;
    a.entries = entries;
    a.num_blocks = num_blocks;
    a.pair_rows = num_blocks / 2;
    a.new_table = new_table;
    a.pairs = pairs;
    a.counts = counts;
    a.block_map = block_map;
    a.status = status;
    return cuda_rc(ll::launch_compact_plan(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
