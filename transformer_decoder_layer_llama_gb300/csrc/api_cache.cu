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

// What ll_norm_rope and its gradient check of their sizes.
int norm_shape(const ll_head_rows* q, const ll_head_rows* k, int32_t dtype, float eps, int32_t tokens, int32_t head_dim,
               int32_t rotary_dim, int32_t layout, const void* table, int32_t max_position, const int32_t* status) {
    if (!q || !k || (dtype != LL_BF16 && dtype != LL_F32)) return LL_ERR_INVALID_ARG;
    if (layout != LL_ROPE_HALF && layout != LL_ROPE_INTERLEAVED) return LL_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !std::isfinite(eps) || tokens < 0 || q->n_heads < 0 || k->n_heads < 0 ||
        q->n_heads + (int64_t)k->n_heads <= 0 || head_dim <= 0 || max_position <= 0 || rotary_dim < 2 || rotary_dim % 2 != 0 ||
        rotary_dim > head_dim)
        return LL_ERR_INVALID_ARG;
    if (head_dim > 1024 || q->n_heads > 4096 || k->n_heads > 4096 || tokens > (1 << 24)) return LL_ERR_UNSUPPORTED;
    if (!table || !status || !aligned16(table)) return LL_ERR_INVALID_ARG;
    return LL_OK;
}

bool gain_ok(const float* g) { return g && (reinterpret_cast<uintptr_t>(g) & 3u) == 0; }

int heads_ok(const ll_head_rows* t, int32_t head_dim, int64_t esz) {
    if (t->n_heads == 0) return LL_OK;
    if (!t->data || reinterpret_cast<uintptr_t>(t->data) % esz != 0 || t->stride < (int64_t)t->n_heads * head_dim) return LL_ERR_INVALID_ARG;
    return t->stride > (1LL << 34) ? LL_ERR_UNSUPPORTED : LL_OK;
}

bool same_heads(const ll_head_rows* a, const ll_head_rows* b) { return a->data == b->data && a->stride == b->stride; }

bool heads_overlap(const ll_head_rows* a, const ll_head_rows* b, int64_t tokens, int64_t head_dim, int64_t esz) {
    if (a->n_heads == 0 || b->n_heads == 0) return false;
    return rows_overlap({a->data, a->stride, a->n_heads * head_dim}, {b->data, b->stride, b->n_heads * head_dim}, tokens, esz);
}

// The shape limits of the calls around attention weights.
int paged_shape(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_blocks) {
    if (batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || max_blocks <= 0 || block_size <= 0) return LL_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return LL_ERR_UNSUPPORTED;
    if (!ll::block_size_ok(block_size)) return LL_ERR_UNSUPPORTED;
    if (n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 16) return LL_ERR_UNSUPPORTED;
    if (batch > 65535 || n_kv_heads > 32767 || (int64_t)max_blocks * block_size > kMaxPositions) return LL_ERR_UNSUPPORTED;
    return LL_OK;
}

int decode_weights_args(ll::AttnDecodeArgs& a, const void* q, int32_t num_blocks, const int32_t* block_table, int32_t max_blocks,
                        const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                        int32_t block_size, float scale, float* weights, int32_t weights_width, void* out, void* workspace,
                        size_t workspace_bytes, int32_t* status) {
    if (!q || !block_table || !context_lens || !weights || weights_width <= 0 || !out || !status || !(scale >= 0.f) ||
        !std::isfinite(scale))
        return LL_ERR_INVALID_ARG;
    const int rc = paged_shape(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks);
    if (rc != LL_OK) return rc;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(weights) & 3u) != 0) return LL_ERR_INVALID_ARG;
    // rows of the pool are TMA coordinates
    if ((int64_t)num_blocks * n_kv_heads * block_size > (1LL << 31) - 1) return LL_ERR_UNSUPPORTED;
    const size_t need = ll_attention_decode_weights_workspace_size(batch, n_heads, n_kv_heads, head_dim, max_blocks, block_size);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return LL_ERR_WORKSPACE;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.context_lens = context_lens;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.scale = scale;
    a.out = static_cast<__nv_bfloat16*>(out);
    const size_t rows = (size_t)batch * n_heads * ll::attn_decode_max_splits(max_blocks, block_size);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = a.part_o + rows * head_dim;
    a.weights = weights;
    a.weights_width = weights_width;
    a.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        align_up(ll::attn_decode_scratch_bytes(batch, n_heads, head_dim, max_blocks, block_size)));
    a.score_stride = (long long)max_blocks * block_size;
    a.status = status;
    return LL_OK;
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

int ll_norm_rope(const ll_head_rows* q, const ll_head_rows* k, int32_t dtype, const float* q_gain, const float* k_gain,
                 float eps, const int32_t* positions, int32_t tokens, int32_t head_dim, int32_t rotary_dim, int32_t layout,
                 const void* table, int32_t max_position, const ll_head_rows* q_out, const ll_head_rows* k_out,
                 int32_t* status, void* stream) {
    ll::clear_last_error();
    const int rc = norm_shape(q, k, dtype, eps, tokens, head_dim, rotary_dim, layout, table, max_position, status);
    if (rc != LL_OK) return rc;
    if (!q_out || !k_out || q_out->n_heads != q->n_heads || k_out->n_heads != k->n_heads) return LL_ERR_INVALID_ARG;
    if (tokens == 0) return LL_OK;
    if (!positions || (q->n_heads > 0 && !gain_ok(q_gain)) || (k->n_heads > 0 && !gain_ok(k_gain))) return LL_ERR_INVALID_ARG;
    const int64_t esz = dtype == LL_F32 ? 4 : 2;
    const ll_head_rows* in[2] = {q, k};
    const ll_head_rows* out[2] = {q_out, k_out};
    for (int i = 0; i < 2; ++i) {
        int bad = heads_ok(in[i], head_dim, esz);
        if (bad == LL_OK) bad = heads_ok(out[i], head_dim, esz);
        if (bad != LL_OK) return bad;
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if ((!(i == j && same_heads(out[i], in[j])) && heads_overlap(out[i], in[j], tokens, head_dim, esz)) ||
                (i < j && heads_overlap(out[i], out[j], tokens, head_dim, esz)))
                return LL_ERR_INVALID_ARG;
    ll::NormRopeArgs a{};
    a.q = q->data;
    a.k = k->data;
    a.q_out = q_out->data;
    a.k_out = k_out->data;
    a.q_stride = q->stride;
    a.k_stride = k->stride;
    a.q_out_stride = q_out->stride;
    a.k_out_stride = k_out->stride;
    a.q_gain = q->n_heads > 0 ? q_gain : k_gain;          // (no null pointer for heads that are not there)
    a.k_gain = k->n_heads > 0 ? k_gain : q_gain;
    a.positions = positions;
    a.table = static_cast<const float2*>(table);
    a.tokens = tokens;
    a.n_heads = q->n_heads;
    a.n_kv_heads = k->n_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.max_position = max_position;
    a.eps = eps;
    a.interleaved = layout == LL_ROPE_INTERLEAVED;
    a.status = status;
    return cuda_rc(ll::launch_norm_rope(a, dtype == LL_F32, static_cast<cudaStream_t>(stream)));
}

size_t ll_norm_rope_backward_workspace_size(int32_t head_dim) {
    if (head_dim <= 0 || head_dim > 1024) return 0;
    return align_up(ll::norm_rope_grad_scratch_bytes(head_dim));
}

int ll_norm_rope_backward(const ll_head_rows* dq, const ll_head_rows* dk, const ll_head_rows* q, const ll_head_rows* k,
                          int32_t dtype, const float* q_gain, const float* k_gain, float eps, const int32_t* positions,
                          int32_t tokens, int32_t head_dim, int32_t rotary_dim, int32_t layout, const void* table,
                          int32_t max_position, const ll_head_rows* q_grad, const ll_head_rows* k_grad, float* q_gain_grad,
                          float* k_gain_grad, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    ll::clear_last_error();
    const int rc = norm_shape(q, k, dtype, eps, tokens, head_dim, rotary_dim, layout, table, max_position, status);
    if (rc != LL_OK) return rc;
    const ll_head_rows* x[2] = {q, k};
    const ll_head_rows* dy[2] = {dq, dk};
    const ll_head_rows* dx[2] = {q_grad, k_grad};
    const float* gain[2] = {q_gain, k_gain};
    float* dgain[2] = {q_gain_grad, k_gain_grad};
    const int64_t esz = dtype == LL_F32 ? 4 : 2;
    for (int i = 0; i < 2; ++i) {
        if (!dy[i] || !dx[i] || dy[i]->n_heads != x[i]->n_heads || dx[i]->n_heads != x[i]->n_heads) return LL_ERR_INVALID_ARG;
        if (x[i]->n_heads == 0) continue;
        if (!gain_ok(gain[i]) || !gain_ok(dgain[i])) return LL_ERR_INVALID_ARG;
        if (tokens == 0) continue;
        for (const ll_head_rows* t : {x[i], dy[i], dx[i]}) {
            const int bad = heads_ok(t, head_dim, esz);
            if (bad != LL_OK) return bad;
        }
    }
    // the gains' gradients are written last: apart from everything that is read or written
    const size_t gain_bytes = (size_t)head_dim * 4;
    if (q->n_heads > 0 && k->n_heads > 0 && overlap(q_gain_grad, gain_bytes, k_gain_grad, gain_bytes)) return LL_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (x[i]->n_heads > 0 && x[j]->n_heads > 0 && overlap(dgain[i], gain_bytes, gain[j], gain_bytes)) return LL_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!positions) return LL_ERR_INVALID_ARG;
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2; ++j)
                if (heads_overlap(dx[i], x[j], tokens, head_dim, esz) ||
                    (!(i == j && same_heads(dx[i], dy[j])) && heads_overlap(dx[i], dy[j], tokens, head_dim, esz)) ||
                    (i < j && heads_overlap(dx[i], dx[j], tokens, head_dim, esz)))
                    return LL_ERR_INVALID_ARG;
    }
    if (!workspace || workspace_bytes < ll_norm_rope_backward_workspace_size(head_dim) || !aligned16(workspace))
        return LL_ERR_WORKSPACE;
    ll::NormRopeGradArgs a{};
    a.q = q->data;
    a.k = k->data;
    a.dq = dq->data;
    a.dk = dk->data;
    a.q_grad = q_grad->data;
    a.k_grad = k_grad->data;
    a.q_stride = q->stride;
    a.k_stride = k->stride;
    a.dq_stride = dq->stride;
    a.dk_stride = dk->stride;
    a.q_grad_stride = q_grad->stride;
    a.k_grad_stride = k_grad->stride;
    a.q_gain = q_gain;
    a.k_gain = k_gain;
    a.q_gain_grad = q_gain_grad;
    a.k_gain_grad = k_gain_grad;
    a.positions = positions;
    a.table = static_cast<const float2*>(table);
    a.tokens = tokens;
    a.n_heads = q->n_heads;
    a.n_kv_heads = k->n_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.max_position = max_position;
    a.eps = eps;
    a.interleaved = layout == LL_ROPE_INTERLEAVED;
    a.partials = static_cast<float*>(workspace);
    a.status = status;
    return cuda_rc(ll::launch_norm_rope_grad(a, dtype == LL_F32, static_cast<cudaStream_t>(stream)));
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

size_t ll_attention_decode_weights_workspace_size(int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                  int32_t max_blocks, int32_t block_size) {
    if (paged_shape(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks) != LL_OK) return 0;
    return align_up(ll::attn_decode_scratch_bytes(batch, n_heads, head_dim, max_blocks, block_size)) +
           align_up((size_t)batch * n_heads * max_blocks * block_size * sizeof(float));
}

int ll_paged_attention_decode_weights(const void* q, const ll_kv_pool* pool, const int32_t* block_table, int32_t max_blocks,
                                      const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                      int32_t head_dim, int32_t block_size, float scale, float* weights, int32_t weights_width,
                                      void* out, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!pool || !pool->k || !pool->v || pool->num_blocks <= 0 || !aligned16(pool->k) || !aligned16(pool->v)) return LL_ERR_INVALID_ARG;
    ll::AttnDecodeArgs a{};
    const int rc = decode_weights_args(a, q, pool->num_blocks, block_table, max_blocks, context_lens, batch, n_heads, n_kv_heads,
                                       head_dim, block_size, scale, weights, weights_width, out, workspace, workspace_bytes, status);
    if (rc != LL_OK) return rc;
    a.k_pool = static_cast<const __nv_bfloat16*>(pool->k);
    a.v_pool = static_cast<const __nv_bfloat16*>(pool->v);
    return cuda_rc(ll::launch_attn_decode(a, static_cast<cudaStream_t>(stream)));
}

int ll_paged_attention_decode_weights_q8(const void* q, const ll_kv_pool_q8* pool, const int32_t* block_table, int32_t max_blocks,
                                         const int32_t* context_lens, int32_t batch, int32_t n_heads, int32_t n_kv_heads,
                                         int32_t head_dim, int32_t block_size, float scale, float* weights, int32_t weights_width,
                                         void* out, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!pool || !pool->k || !pool->v || !pool->k_scale || !pool->v_scale || pool->num_blocks <= 0) return LL_ERR_INVALID_ARG;
    if (!aligned16(pool->k) || !aligned16(pool->v) || !aligned16(pool->k_scale) || !aligned16(pool->v_scale)) return LL_ERR_INVALID_ARG;
    if (head_dim != 128) return LL_ERR_UNSUPPORTED;
    ll::AttnDecodeArgs a{};
    const int rc = decode_weights_args(a, q, pool->num_blocks, block_table, max_blocks, context_lens, batch, n_heads, n_kv_heads,
                                       head_dim, block_size, scale, weights, weights_width, out, workspace, workspace_bytes, status);
    if (rc != LL_OK) return rc;
    a.k_q8 = static_cast<const int8_t*>(pool->k);
    a.v_q8 = static_cast<const int8_t*>(pool->v);
    a.k_scale = pool->k_scale;
    a.v_scale = pool->v_scale;
    return cuda_rc(ll::launch_attn_decode_q8(a, static_cast<cudaStream_t>(stream)));
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

size_t ll_attention_weights_workspace_size(int32_t batch, int32_t tokens, int32_t max_new, int32_t n_heads, int32_t n_kv_heads,
                                           int32_t head_dim, int32_t max_blocks, int32_t block_size) {
    if (tokens < 0 || max_new <= 0 || paged_shape(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks) != LL_OK) return 0;
    return align_up(std::max<size_t>(1, ll::observe_workspace_bytes(tokens, n_heads, n_kv_heads, max_blocks, block_size)));
}

int ll_paged_attention_weights(const void* q, const int32_t* cu_new, int32_t tokens, const void* k_pool, int32_t num_blocks,
                               const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                               int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t block_size,
                               float scale, float* weights, int32_t weights_width, void* workspace, size_t workspace_bytes,
                               int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!cu_new || !k_pool || num_blocks <= 0 || !block_table || !context_lens || !weights || weights_width <= 0 || !status ||
        !(scale >= 0.f) || !std::isfinite(scale) || tokens < 0 || max_new <= 0)
        return LL_ERR_INVALID_ARG;
    const int rc = paged_shape(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks);
    if (rc != LL_OK) return rc;
    if (!aligned16(k_pool) || (reinterpret_cast<uintptr_t>(weights) & 3u) != 0) return LL_ERR_INVALID_ARG;
    if (tokens > 0 && (!q || !aligned16(q))) return LL_ERR_INVALID_ARG;
    // rows of the pool are TMA coordinates
    if ((int64_t)num_blocks * n_kv_heads * block_size > (1LL << 31) - 1) return LL_ERR_UNSUPPORTED;
    if (!ll::observe_fits(batch, std::min(max_new, tokens), n_heads, n_kv_heads, max_blocks, block_size)) return LL_ERR_UNSUPPORTED;
    const size_t need = std::max<size_t>(1, ll::observe_scratch_bytes(batch, tokens, std::min(max_new, tokens), n_heads, n_kv_heads,
                                                                      max_blocks, block_size));
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return LL_ERR_WORKSPACE;
    ll::ObserveArgs a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
    a.cu_new = cu_new;
    a.context_lens = context_lens;
    a.block_table = block_table;
    a.tokens = tokens;
    a.batch = batch;
    a.max_new = std::min(max_new, tokens);
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.scale = scale;
    a.weights = weights;
    a.weights_width = weights_width;
    a.status = status;
    return cuda_rc(ll::launch_observe(a, workspace, static_cast<cudaStream_t>(stream)));
}

int ll_evict_rows(const ll_row_tensor* tensors, int32_t n_tensors, int32_t num_blocks, int32_t n_kv_heads, int32_t block_size,
                  const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens, int32_t batch,
                  const float* weights, int32_t weights_width, const int32_t* keep, int32_t max_keep, int32_t sinks,
                  int32_t recent, float* weights_out, int32_t* kept, int32_t* new_lens, int32_t* status, void* stream) {
    ll::clear_last_error();
    if (!tensors || n_tensors <= 0 || num_blocks <= 0 || n_kv_heads <= 0 || block_size <= 0 || max_blocks <= 0 || batch <= 0 ||
        weights_width <= 0 || max_keep <= 0 || sinks < 0 || recent < 0)
        return LL_ERR_INVALID_ARG;
    if (!block_table || !context_lens || !weights || !weights_out || !kept || !new_lens || !status) return LL_ERR_INVALID_ARG;
    for (const void* p : {(const void*)weights, (const void*)weights_out, (const void*)kept, (const void*)new_lens})
        if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return LL_ERR_INVALID_ARG;
    if (n_tensors > ll::kEvictMaxTensors || !ll::block_size_ok(block_size) || batch > 65535 || n_kv_heads > 32767 ||
        (int64_t)max_blocks * block_size > kMaxPositions || (int64_t)num_blocks * n_kv_heads * block_size > (1LL << 31) - 1)
        return LL_ERR_UNSUPPORTED;
    ll::EvictArgs a{};
    for (int32_t t = 0; t < n_tensors; ++t) {
        const ll_row_tensor& x = tensors[t];
        if (!x.data || x.row_bytes <= 0 || x.row_bytes % 4 != 0 || (reinterpret_cast<uintptr_t>(x.data) & 3u) != 0) return LL_ERR_INVALID_ARG;
        if (x.row_bytes > 4096) return LL_ERR_UNSUPPORTED;
        a.data[t] = x.data;
        a.row_bytes[t] = (int)x.row_bytes;
        a.wide[t] = x.row_bytes % 16 == 0 && aligned16(x.data);
    }
    // what is written: the tensors, weights_out (weights itself, or apart), kept, new_lens; apart from each other and what is read
    const size_t rows = (size_t)batch * n_kv_heads, pool_rows = (size_t)num_blocks * n_kv_heads * block_size;
    struct { const void* p; size_t bytes; } use[ll::kEvictMaxTensors + 6];
    int written = 0;
    for (; written < n_tensors; ++written) use[written] = {tensors[written].data, pool_rows * tensors[written].row_bytes};
    use[written++] = {kept, rows * max_keep * 4};
    use[written++] = {new_lens, (size_t)batch * 4};
    use[written++] = {weights_out, rows * weights_width * 4};
    int used = written;
    if (weights != weights_out) use[used++] = {weights, rows * weights_width * 4};
    use[used++] = {context_lens, (size_t)batch * 4};
    if (keep) use[used++] = {keep, (size_t)batch * 4};
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < used; ++j)
            if (overlap(use[i].p, use[i].bytes, use[j].p, use[j].bytes)) return LL_ERR_INVALID_ARG;
    a.n_tensors = n_tensors;
    a.num_blocks = num_blocks;
    a.n_kv_heads = n_kv_heads;
    a.block_size = block_size;
    a.max_blocks = max_blocks;
    a.batch = batch;
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.weights = weights;
    a.weights_out = weights_out;
    a.weights_width = weights_width;
    a.keep = keep;
    a.max_keep = max_keep;
    a.sinks = sinks;
    a.recent = recent;
    a.kept = kept;
    a.new_lens = new_lens;
    a.status = status;
    return cuda_rc(ll::launch_evict(a, static_cast<cudaStream_t>(stream)));
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
