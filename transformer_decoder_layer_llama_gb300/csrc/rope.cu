// Rotary positions as an operator of its own (the layer's QKV epilogue fuses the plain
// half-split form).  Pair i of a head, i < rotary_dim / 2, at position p turns by the angle
// p w_i:  (a, b) -> (a c - b s, b c + a s), c = m cos(p w_i), s = m sin(p w_i); the gradient is
// the transpose, s -> -s.  Elements from rotary_dim on pass through.  The pairs are elements
// (i, i + rotary_dim / 2) ("half") or (2i, 2i + 1) ("interleaved").
//
// c and s come from a float32 table computed once in float64 (positions reach 2^17 and more,
// where a float32 angle has lost its fraction of a turn).  The operator is bound by memory: a
// token's heads are read and written once, and its table row (8 bytes per pair) is read once
// per CTA and then served by L1 to the other heads.  16384 tokens of 64 + 8 heads of 128, BF16:
// 93 us, 6.6 TB/s (97% of the copy bandwidth); 5003 tokens of 32 + 4 heads, 64 of 128 elements,
// float32, backward: 31 us, 6.0 TB/s.  64 tokens take 6 us on the GPU, less than the call on the host.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "vec16.cuh"

namespace ll {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeHeads = 4;               // of a thread

// The position of token t, or -1 (flagged by the caller's chosen thread) where it is outside the table.
LL_DEVINL int rope_position(const RopeArgs& a, int t, bool flag) {
    const int p = a.positions[t];
    if (p < 0 || p >= a.max_position) {
        if (flag) flag_status(a.status, LL_DEV_BAD_POSITION);
        return -1;
    }
    return p;
}

// One thread rotates the same 16-byte column of U heads of one token (half: the two columns a
// pair spans), so that its table entries are loaded once.
template <typename T, bool HALF, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const RopeArgs a, int lanes_rot, int lanes, int rows) {
    using V = Vec<T>;
    constexpr int N = V::N, PAIRS = HALF ? N : N / 2;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const int lane = threadIdx.x % lanes, row = threadIdx.x / lanes;
    const int pos = rope_position(a, t, threadIdx.x == 0 && blockIdx.y == 0);
    if (pos < 0 || row >= rows) return;
    const int H = a.n_heads + a.n_kv_heads;
    const int h0 = blockIdx.y * rows * U + row;
    const T* src[U];
    T* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * rows;
        const bool isq = h < a.n_heads;
        const int hh = isq ? h : h - a.n_heads;
        src[u] = static_cast<const T*>(isq ? a.q : a.k) + (size_t)t * (isq ? a.q_stride : a.k_stride) +
                 (size_t)hh * a.head_dim;
        dst[u] = static_cast<T*>(isq ? a.q_out : a.k_out) + (size_t)t * (isq ? a.q_out_stride : a.k_out_stride) +
                 (size_t)hh * a.head_dim;
    }
    if (lane >= lanes_rot) {                              // behind the rotated part: copied
        const int e = a.rotary_dim + (lane - lanes_rot) * N;
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h0 + u * rows < H) w[u] = *reinterpret_cast<const uint4*>(src[u] + e);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h0 + u * rows < H) *reinterpret_cast<uint4*>(dst[u] + e) = w[u];
        return;
    }
    const int half = a.rotary_dim >> 1;
    const int e0 = lane * N;                              // first element; half: its partners at e0 + half
    uint4 w0[U], w1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u * rows < H) {
            w0[u] = *reinterpret_cast<const uint4*>(src[u] + e0);
            if (HALF) w1[u] = *reinterpret_cast<const uint4*>(src[u] + e0 + half);
        }
    }
    float c[PAIRS], s[PAIRS];
    const float4* cs = reinterpret_cast<const float4*>(a.table + (size_t)pos * half + (HALF ? e0 : e0 / 2));
#pragma unroll
    for (int i = 0; i < PAIRS / 2; ++i) {
        const float4 x = __ldg(cs + i);
        c[2 * i] = x.x;
        s[2 * i] = a.backward ? -x.y : x.y;
        c[2 * i + 1] = x.z;
        s[2 * i + 1] = a.backward ? -x.w : x.w;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u * rows >= H) break;
        float x[N], y[N];
        V::unpack(w0[u], x);
        if (HALF) {
            V::unpack(w1[u], y);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 r = rope_rotate(x[i], y[i], c[i % PAIRS], s[i % PAIRS]);
                x[i] = r.x;
                y[i] = r.y;
            }
            *reinterpret_cast<uint4*>(dst[u] + e0 + half) = V::pack(y);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 r = rope_rotate(x[2 * i], x[2 * i + 1], c[i], s[i]);
                x[2 * i] = r.x;
                x[2 * i + 1] = r.y;
            }
        }
        *reinterpret_cast<uint4*>(dst[u] + e0) = V::pack(x);
    }
}

// Any even rotary_dim, any element-aligned pointers and strides: one pair (or one element behind
// the rotated part) per thread and step.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const RopeArgs a) {
    using V = Vec<T>;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const int pos = rope_position(a, t, threadIdx.x == 0 && blockIdx.y == 0);
    if (pos < 0) return;
    const int half = a.rotary_dim >> 1, units = half + (a.copy_tail ? a.head_dim - a.rotary_dim : 0);
    const int H = a.n_heads + a.n_kv_heads;
    const long long total = (long long)H * units;
    for (long long i = (long long)blockIdx.y * blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.y * blockDim.x) {
        const int h = (int)(i / units), e = (int)(i - (long long)h * units);
        const bool isq = h < a.n_heads;
        const int hh = isq ? h : h - a.n_heads;
        const T* src = static_cast<const T*>(isq ? a.q : a.k) + (size_t)t * (isq ? a.q_stride : a.k_stride) +
                       (size_t)hh * a.head_dim;
        T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + (size_t)t * (isq ? a.q_out_stride : a.k_out_stride) +
                 (size_t)hh * a.head_dim;
        if (e >= half) {
            dst[e + half] = src[e + half];
            continue;
        }
        const int i0 = a.interleaved ? 2 * e : e, i1 = a.interleaved ? 2 * e + 1 : e + half;
        const float2 cs = a.table[(size_t)pos * half + e];
        const float2 r = rope_rotate(V::get(src + i0), V::get(src + i1), cs.x, a.backward ? -cs.y : cs.y);
        V::put(dst + i0, r.x);
        V::put(dst + i1, r.y);
    }
}

// (cos, sin) of every position and pair in float64.  Inverse frequencies w_i = theta^(-2i / r):
//  linear   w / factor (positions interpolated)
//  ntk      theta grows by factor^(r / (r - 2)): the slowest pair slows by the factor, the fastest stays
//  banded   pairs that turn at least `high` times over the original context keep w, those that turn at
//           most `low` times get w / factor, linear in the turns between
//  yarn     the same two ends, linear in the pair index between the pairs (rounded outwards) that turn
//           `high` and `low` times; cos and sin times the attention factor
__global__ void rope_scaled_table_kernel(float2* cs, int max_position, const RopeTableArgs f) {
    const int half = f.rotary_dim >> 1;
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= (long long)max_position * half) return;
    const int pos = (int)(idx / half), i = (int)(idx - (long long)pos * half);
    constexpr double two_pi = 6.283185307179586476925286766559;
    const double w = pow(f.theta, -(2.0 * i) / (double)f.rotary_dim);
    double t = 1.0;                                       // weight of the unscaled frequency
    if (f.scaling == LL_ROPE_LINEAR) t = 0.0;
    if (f.scaling == LL_ROPE_BANDED) t = fmin(fmax((f.original * w / two_pi - f.low) / (f.high - f.low), 0.0), 1.0);
    if (f.scaling == LL_ROPE_YARN) t = 1.0 - fmin(fmax((i - f.ramp_lo) / f.ramp_width, 0.0), 1.0);
    const double ang = (double)pos * (t * w + (1.0 - t) * w / f.factor);
    double s, c;
    sincos(ang, &s, &c);
    cs[idx] = make_float2((float)(c * f.magnitude), (float)(s * f.magnitude));
}

template <typename T>
cudaError_t rope_for(const RopeArgs& a, cudaStream_t stream) {
    constexpr int N = Vec<T>::N;
    const int H = a.n_heads + a.n_kv_heads;
    const auto ok = [](const void* p, long long stride) {
        return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * (long long)sizeof(T) % 16 == 0;
    };
    // 16-byte columns: every row of every tensor starts on 16 bytes and the rotated part splits
    // into whole columns (half: each of its halves)
    const bool vec = a.head_dim % N == 0 && a.rotary_dim % (a.interleaved ? N : 2 * N) == 0 &&
                     (a.rotary_dim / 2) % 2 == 0 && (a.n_heads == 0 || (ok(a.q, a.q_stride) && ok(a.q_out, a.q_out_stride))) &&
                     (a.n_kv_heads == 0 || (ok(a.k, a.k_stride) && ok(a.k_out, a.k_out_stride)));
    trace_before("rope", stream);
    cudaError_t e;
    if (vec) {
        const int lanes_rot = a.interleaved ? a.rotary_dim / N : a.rotary_dim / (2 * N);
        const int lanes = lanes_rot + (a.copy_tail ? (a.head_dim - a.rotary_dim) / N : 0);
        // Four heads per thread keep their loads in flight together and read a table row once (16384 tokens of 40
        // heads: 57 us, with one head per thread 61; up to 2048 tokens there is no difference).  Head rows of a CTA:
        // as even a split of the heads as the CTA's threads allow.
        const int most = std::max(1, kRopeThreads / lanes);
        const int parts = (H + kRopeHeads * most - 1) / (kRopeHeads * most);
        const int rows = (H + kRopeHeads * parts - 1) / (kRopeHeads * parts);
        const int threads = (rows * lanes + 31) / 32 * 32;
        const dim3 grid((unsigned)a.tokens, (unsigned)parts);
        e = a.interleaved ? launch_pdl(rope_vec_kernel<T, false, kRopeHeads>, grid, dim3(threads), 0, stream, 1, a, lanes_rot, lanes, rows)
                          : launch_pdl(rope_vec_kernel<T, true, kRopeHeads>, grid, dim3(threads), 0, stream, 1, a, lanes_rot, lanes, rows);
    } else {
        const long long units = (long long)H * (a.rotary_dim / 2 + (a.copy_tail ? a.head_dim - a.rotary_dim : 0));
        const unsigned y = (unsigned)std::min<long long>(16, (units + kRopeThreads - 1) / kRopeThreads);
        e = launch_pdl(rope_any_kernel<T>, dim3((unsigned)a.tokens, y), dim3(kRopeThreads), 0, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "rope launch");
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool f32, cudaStream_t stream) {
    if (a.tokens <= 0 || a.n_heads + a.n_kv_heads <= 0) return cudaSuccess;
    return f32 ? rope_for<float>(a, stream) : rope_for<__nv_bfloat16>(a, stream);
}

cudaError_t launch_rope_scaled_table(float2* cs, int max_position, const RopeTableArgs& f, cudaStream_t stream) {
    const long long n = (long long)max_position * (f.rotary_dim / 2);
    rope_scaled_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(cs, max_position, f);
    return record(cudaGetLastError(), "rope_scaled_table launch");
}

}  // namespace ll
