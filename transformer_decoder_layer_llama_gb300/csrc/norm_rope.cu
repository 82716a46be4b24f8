// RMS norm of every Q and K head with its gain, and the rotary positions, in one pass, and its gradient.
// Head row x of d elements:  r = 1 / sqrt(mean x^2 + eps),  n = x r g,  y = R(p) n, R the rotation of rope.cu.
// With dy given:  dn = R^T dy,  dx = r (g dn - x r^2 mean(g dn x)),  dg = sum over tokens and heads of dn x r.
//
// Bound by memory: forward reads and writes a head once, the gradient reads x and dy and writes dx.  The group of
// threads that holds a head sums its squares by shuffles, so nothing is read twice and nothing goes through shared
// memory; a token's (cos, sin) row and the gains stay in registers for a thread's heads.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "vec16.cuh"

namespace ll {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormHeads = 4;          // of a thread, forward
constexpr int kNormGradHeads = 2;      // of a thread, gradient (x and dy of each)
constexpr int kNormGradCtasPerSm = 2;
constexpr int kNormAnyWarps = 4;       // of the gradient's CTA for other shapes

// How the threads of a vector kernel share a token's heads: a head is `lanes` threads of a group of `width` (a power
// of two), each with two 16-byte columns; a token is `rows` groups, each with up to U heads at a time, in `parts`
// turns; a CTA has `slots` tokens at a time.
struct HeadSplit {
    int lanes, width, rows, parts, slots, threads;
};

HeadSplit head_split(int head_dim, int n, int heads, int per_thread) {
    HeadSplit s;
    s.lanes = head_dim / (2 * n);
    s.width = 1;
    while (s.width < s.lanes) s.width *= 2;
    const int most = kNormThreads / s.width;
    s.parts = (heads + per_thread * most - 1) / (per_thread * most);
    s.rows = (heads + per_thread * s.parts - 1) / (per_thread * s.parts);
    s.slots = std::max(1, most / s.rows);
    s.threads = (s.slots * s.rows * s.width + 31) / 32 * 32;
    return s;
}

// A thread's two columns: rotated half-split, they hold the two ends of its pairs; interleaved or behind the rotated
// part, neighbouring elements.
template <int N, bool HALF>
struct Columns {
    int e0, e1;
    bool turn;
    LL_DEVINL Columns(int lane, int rotary_dim) {
        const int first = lane * 2 * N;
        turn = first < rotary_dim;
        e0 = HALF && turn ? lane * N : first;
        e1 = HALF && turn ? e0 + (rotary_dim >> 1) : first + N;
    }
};

template <int N>
LL_DEVINL void load_angles(const float2* table, int pos, int half, int first_pair, float (&c)[N], float (&s)[N]) {
    const float4* cs = reinterpret_cast<const float4*>(table + (size_t)pos * half + first_pair);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float4 x = __ldg(cs + i);
        c[2 * i] = x.x;
        s[2 * i] = x.y;
        c[2 * i + 1] = x.z;
        s[2 * i + 1] = x.w;
    }
}

template <int N>
LL_DEVINL void load_gains(const float* g, int e0, int e1, float (&a)[N], float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(g + e0) + i), y = __ldg(reinterpret_cast<const float4*>(g + e1) + i);
        a[4 * i] = x.x; a[4 * i + 1] = x.y; a[4 * i + 2] = x.z; a[4 * i + 3] = x.w;
        b[4 * i] = y.x; b[4 * i + 1] = y.y; b[4 * i + 2] = y.z; b[4 * i + 3] = y.w;
    }
}

// The N pairs that the columns a and b hold, turned by (c, s).
template <int N, bool HALF>
LL_DEVINL void turn_pairs(float (&a)[N], float (&b)[N], const float (&c)[N], const float (&s)[N], float sign) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (HALF) {
            const float2 r = rope_rotate(a[i], b[i], c[i], sign * s[i]);
            a[i] = r.x;
            b[i] = r.y;
        } else {
            float* v = i < N / 2 ? a + 2 * i : b + 2 * i - N;
            const float2 r = rope_rotate(v[0], v[1], c[i], sign * s[i]);
            v[0] = r.x;
            v[1] = r.y;
        }
    }
}

LL_DEVINL float group_sum(float x, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

LL_DEVINL int norm_position(const int32_t* positions, int t, int max_position, int32_t* status, bool flag) {
    const int p = positions[t];
    if (p >= 0 && p < max_position) return p;
    if (flag) flag_status(status, LL_DEV_BAD_POSITION);
    return -1;
}

template <typename T, bool HALF>
__global__ void __launch_bounds__(kNormThreads) norm_rope_vec_kernel(const NormRopeArgs a, const HeadSplit hs) {
    using V = Vec<T>;
    constexpr int N = V::N, U = kNormHeads;
    pdl_wait();
    pdl_trigger();
    const int group = threadIdx.x / hs.width, lane = threadIdx.x % hs.width;
    const int slot = group / hs.rows, row = group - slot * hs.rows;
    const int t = blockIdx.x * hs.slots + slot;
    const bool here = slot < hs.slots && t < a.tokens;
    const int pos = here ? norm_position(a.positions, t, a.max_position, a.status, lane == 0 && row == 0 && blockIdx.y == 0) : -1;
    const bool live = pos >= 0 && lane < hs.lanes;      // (every thread takes part in the shuffles)
    const Columns<N, HALF> col(lane, a.rotary_dim);
    const int H = a.n_heads + a.n_kv_heads;
    const int h0 = blockIdx.y * hs.rows * U + row;
    uint4 w0[U], w1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * hs.rows;
        w0[u] = w1[u] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < H) {
            const bool isq = h < a.n_heads;
            const T* src = static_cast<const T*>(isq ? a.q : a.k) + (size_t)t * (isq ? a.q_stride : a.k_stride) +
                           (size_t)(isq ? h : h - a.n_heads) * a.head_dim;
            w0[u] = *reinterpret_cast<const uint4*>(src + col.e0);
            w1[u] = *reinterpret_cast<const uint4*>(src + col.e1);
        }
    }
    float c[N], s[N], g0[N], g1[N];
    bool gain_q = h0 < a.n_heads;
    if (live) {
        if (col.turn) load_angles<N>(a.table, pos, a.rotary_dim >> 1, HALF ? col.e0 : col.e0 / 2, c, s);
        load_gains<N>(gain_q ? a.q_gain : a.k_gain, col.e0, col.e1, g0, g1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * hs.rows;
        float x[N], y[N], sum = 0.f;
        V::unpack(w0[u], x);
        V::unpack(w1[u], y);
#pragma unroll
        for (int i = 0; i < N; ++i) sum += x[i] * x[i] + y[i] * y[i];
        sum = group_sum(sum, hs.width);
        if (!live || h >= H) continue;
        const bool isq = h < a.n_heads;
        if (isq != gain_q) {
            gain_q = isq;
            load_gains<N>(a.k_gain, col.e0, col.e1, g0, g1);
        }
        const float r = rsqrtf(sum / (float)a.head_dim + a.eps);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = x[i] * r * g0[i];
            y[i] = y[i] * r * g1[i];
        }
        if (col.turn) turn_pairs<N, HALF>(x, y, c, s, 1.f);
        T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + (size_t)t * (isq ? a.q_out_stride : a.k_out_stride) +
                 (size_t)(isq ? h : h - a.n_heads) * a.head_dim;
        *reinterpret_cast<uint4*>(dst + col.e0) = V::pack(x);
        *reinterpret_cast<uint4*>(dst + col.e1) = V::pack(y);
    }
}

// The elements of unit u of a head: a rotated pair, or (i1 < 0) one element behind the rotated part.
LL_DEVINL void unit_elements(int u, int rotary_dim, bool interleaved, int& i0, int& i1) {
    const int half = rotary_dim >> 1;
    if (u >= half) {
        i0 = u + half;
        i1 = -1;
    } else {
        i0 = interleaved ? 2 * u : u;
        i1 = interleaved ? 2 * u + 1 : u + half;
    }
}

// Any even rotary_dim, any element-aligned pointers and strides: a warp per head.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rope_any_kernel(const NormRopeArgs a) {
    using V = Vec<T>;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int pos = norm_position(a.positions, t, a.max_position, a.status, threadIdx.x == 0 && blockIdx.y == 0);
    if (pos < 0) return;
    const int half = a.rotary_dim >> 1, units = a.head_dim - half, H = a.n_heads + a.n_kv_heads;
    for (int h = blockIdx.y * warps + (threadIdx.x >> 5); h < H; h += gridDim.y * warps) {
        const bool isq = h < a.n_heads;
        const int hh = isq ? h : h - a.n_heads;
        const T* src = static_cast<const T*>(isq ? a.q : a.k) + (size_t)t * (isq ? a.q_stride : a.k_stride) + (size_t)hh * a.head_dim;
        T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + (size_t)t * (isq ? a.q_out_stride : a.k_out_stride) + (size_t)hh * a.head_dim;
        const float* g = isq ? a.q_gain : a.k_gain;
        float sum = 0.f;
        for (int i = lane; i < a.head_dim; i += 32) {
            const float x = V::get(src + i);
            sum += x * x;
        }
        const float r = rsqrtf(group_sum(sum, 32) / (float)a.head_dim + a.eps);
        for (int u = lane; u < units; u += 32) {          // (a lane's elements are its own: in place is safe, the sum is done)
            int i0, i1;
            unit_elements(u, a.rotary_dim, a.interleaved, i0, i1);
            const float x = V::get(src + i0) * r * g[i0];
            if (i1 < 0) {
                V::put(dst + i0, x);
                continue;
            }
            const float2 cs = a.table[(size_t)pos * half + u];
            const float2 y = rope_rotate(x, V::get(src + i1) * r * g[i1], cs.x, cs.y);
            V::put(dst + i0, y.x);
            V::put(dst + i1, y.y);
        }
    }
}

// ---------------------------------------------------------------- gradient

// Tokens go round the CTAs; a thread keeps the gain gradients of its columns over all of them.  The sums of a CTA's
// groups meet in shared memory in a fixed order, those of the CTAs in a second kernel: the same bits every time.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kNormThreads, kNormGradCtasPerSm)
    norm_rope_grad_vec_kernel(const NormRopeGradArgs a, const HeadSplit hs) {
    using V = Vec<T>;
    constexpr int N = V::N, U = kNormGradHeads;
    extern __shared__ float s_dg[];                       // [groups][head_dim]
    pdl_wait();
    pdl_trigger();
    const int group = threadIdx.x / hs.width, lane = threadIdx.x % hs.width;
    const int slot = group / hs.rows, row = group - slot * hs.rows;
    const Columns<N, HALF> col(lane, a.rotary_dim);
    const int H = a.n_heads + a.n_kv_heads;
    const bool worker = slot < hs.slots && lane < hs.lanes;
    float dg0[2][N], dg1[2][N];                           // [q, k]
#pragma unroll
    for (int i = 0; i < N; ++i) dg0[0][i] = dg0[1][i] = dg1[0][i] = dg1[1][i] = 0.f;
    const float inv_d = 1.f / (float)a.head_dim;

    for (int t0 = blockIdx.x * hs.slots; t0 < a.tokens; t0 += gridDim.x * hs.slots) {
        const int t = t0 + slot;
        const bool here = slot < hs.slots && t < a.tokens;
        const int pos = here ? norm_position(a.positions, t, a.max_position, a.status, lane == 0 && row == 0) : -1;
        const bool live = pos >= 0 && worker;
        float c[N], s[N];
        if (live && col.turn) load_angles<N>(a.table, pos, a.rotary_dim >> 1, HALF ? col.e0 : col.e0 / 2, c, s);
        for (int part = 0; part < hs.parts; ++part) {
            const int h0 = part * hs.rows * U + row;
            uint4 wx0[U], wx1[U], wy0[U], wy1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * hs.rows;
                wx0[u] = wx1[u] = wy0[u] = wy1[u] = make_uint4(0u, 0u, 0u, 0u);
                if (live && h < H) {
                    const bool isq = h < a.n_heads;
                    const size_t at = (size_t)(isq ? h : h - a.n_heads) * a.head_dim;
                    const T* x = static_cast<const T*>(isq ? a.q : a.k) + (size_t)t * (isq ? a.q_stride : a.k_stride) + at;
                    const T* dy = static_cast<const T*>(isq ? a.dq : a.dk) + (size_t)t * (isq ? a.dq_stride : a.dk_stride) + at;
                    wx0[u] = *reinterpret_cast<const uint4*>(x + col.e0);
                    wx1[u] = *reinterpret_cast<const uint4*>(x + col.e1);
                    wy0[u] = *reinterpret_cast<const uint4*>(dy + col.e0);
                    wy1[u] = *reinterpret_cast<const uint4*>(dy + col.e1);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * hs.rows;
                const bool isq = h < a.n_heads, on = live && h < H;
                float x0[N], x1[N], y0[N], y1[N], g0[N], g1[N];
                V::unpack(wx0[u], x0);
                V::unpack(wx1[u], x1);
                V::unpack(wy0[u], y0);
                V::unpack(wy1[u], y1);
                float sq = 0.f, dot = 0.f;
                if (on) {
                    load_gains<N>(isq ? a.q_gain : a.k_gain, col.e0, col.e1, g0, g1);
                    if (col.turn) turn_pairs<N, HALF>(y0, y1, c, s, -1.f);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        sq += x0[i] * x0[i] + x1[i] * x1[i];
                        dot += y0[i] * g0[i] * x0[i] + y1[i] * g1[i] * x1[i];
                    }
                }
                sq = group_sum(sq, hs.width);
                dot = group_sum(dot, hs.width);
                if (!on) continue;
                const float r = rsqrtf(sq * inv_d + a.eps), f = dot * inv_d * r * r;
                if (isq) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dg0[0][i] += y0[i] * (x0[i] * r);
                        dg1[0][i] += y1[i] * (x1[i] * r);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dg0[1][i] += y0[i] * (x0[i] * r);
                        dg1[1][i] += y1[i] * (x1[i] * r);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x0[i] = r * (y0[i] * g0[i] - x0[i] * f);
                    x1[i] = r * (y1[i] * g1[i] - x1[i] * f);
                }
                T* dst = static_cast<T*>(isq ? a.q_grad : a.k_grad) + (size_t)t * (isq ? a.q_grad_stride : a.k_grad_stride) +
                         (size_t)(isq ? h : h - a.n_heads) * a.head_dim;
                *reinterpret_cast<uint4*>(dst + col.e0) = V::pack(x0);
                *reinterpret_cast<uint4*>(dst + col.e1) = V::pack(x1);
            }
        }
    }
    const int groups = hs.slots * hs.rows;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (worker) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s_dg[group * a.head_dim + col.e0 + i] = dg0[which][i];
                s_dg[group * a.head_dim + col.e1 + i] = dg1[which][i];
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.head_dim; e += blockDim.x) {
            float sum = 0.f;
            for (int i = 0; i < groups; ++i) sum += s_dg[i * a.head_dim + e];
            a.partials[((size_t)blockIdx.x * 2 + which) * a.head_dim + e] = sum;
        }
        __syncthreads();
    }
}

// Any shape: a warp per head, the gain gradients of a warp in shared memory (a lane adds to its own elements only).
template <typename T>
__global__ void __launch_bounds__(kNormAnyWarps * 32) norm_rope_grad_any_kernel(const NormRopeGradArgs a) {
    using V = Vec<T>;
    extern __shared__ float s_dg[];                       // [warps][2][head_dim]
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = a.head_dim;
    const int half = a.rotary_dim >> 1, units = d - half, H = a.n_heads + a.n_kv_heads;
    for (int i = threadIdx.x; i < kNormAnyWarps * 2 * d; i += blockDim.x) s_dg[i] = 0.f;
    __syncthreads();
    const long long rows = (long long)a.tokens * H;
    for (long long i = (long long)blockIdx.x * kNormAnyWarps + warp; i < rows; i += (long long)gridDim.x * kNormAnyWarps) {
        const int t = (int)(i / H), h = (int)(i - (long long)t * H);
        const int pos = norm_position(a.positions, t, a.max_position, a.status, lane == 0 && h == 0);
        if (pos < 0) continue;
        const bool isq = h < a.n_heads;
        const size_t at = (size_t)(isq ? h : h - a.n_heads) * d;
        const T* x = static_cast<const T*>(isq ? a.q : a.k) + (size_t)t * (isq ? a.q_stride : a.k_stride) + at;
        const T* dy = static_cast<const T*>(isq ? a.dq : a.dk) + (size_t)t * (isq ? a.dq_stride : a.dk_stride) + at;
        T* dst = static_cast<T*>(isq ? a.q_grad : a.k_grad) + (size_t)t * (isq ? a.q_grad_stride : a.k_grad_stride) + at;
        const float* g = isq ? a.q_gain : a.k_gain;
        float* dg = s_dg + (warp * 2 + (isq ? 0 : 1)) * d;
        float r = 0.f, f = 0.f;
        for (int turn = 0; turn < 2; ++turn) {            // the sums, then the gradients
            float sq = 0.f, dot = 0.f;
            for (int u = lane; u < units; u += 32) {
                int i0, i1;
                unit_elements(u, a.rotary_dim, a.interleaved, i0, i1);
                const float x0 = V::get(x + i0), x1 = i1 < 0 ? 0.f : V::get(x + i1);
                float2 y = make_float2(V::get(dy + i0), 0.f);
                if (i1 >= 0) {
                    const float2 cs = a.table[(size_t)pos * half + u];
                    y = rope_rotate(y.x, V::get(dy + i1), cs.x, -cs.y);
                }
                const float g0 = g[i0], g1 = i1 < 0 ? 0.f : g[i1];
                if (turn == 0) {
                    sq += x0 * x0 + x1 * x1;
                    dot += y.x * g0 * x0 + y.y * g1 * x1;
                    continue;
                }
                dg[i0] += y.x * (x0 * r);
                V::put(dst + i0, r * (y.x * g0 - x0 * f));
                if (i1 >= 0) {
                    dg[i1] += y.y * (x1 * r);
                    V::put(dst + i1, r * (y.y * g1 - x1 * f));
                }
            }
            if (turn == 0) {
                r = rsqrtf(group_sum(sq, 32) / (float)d + a.eps);
                f = group_sum(dot, 32) / (float)d * r * r;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) {
        float sum = 0.f;
        for (int w = 0; w < kNormAnyWarps; ++w) sum += s_dg[w * 2 * d + i];
        a.partials[(size_t)blockIdx.x * 2 * d + i] = sum;
    }
}

// Gain gradients: the sum of the CTAs' partials [ctas][2][head_dim], eight of them at a time per column.
__global__ void __launch_bounds__(256) norm_rope_gains_kernel(const float* partials, int ctas, int head_dim, float* q_gain_grad,
                                                              float* k_gain_grad) {
    __shared__ float s_sum[8][32];
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float sum = 0.f;
    if (i < 2 * head_dim)
        for (int c = w; c < ctas; c += 8) sum += partials[(size_t)c * 2 * head_dim + i];
    s_sum[w][threadIdx.x & 31] = sum;
    __syncthreads();
    if (w != 0 || i >= 2 * head_dim) return;
    for (int j = 1; j < 8; ++j) sum += s_sum[j][threadIdx.x];
    float* out = i < head_dim ? q_gain_grad : k_gain_grad;
    if (out) out[i < head_dim ? i : i - head_dim] = sum;
}

bool rows16(const void* p, long long stride, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * esz % 16 == 0;
}

// 16-byte columns, two to a thread, a head within a warp: every row and the gains start on 16 bytes.
bool vec_shape(int head_dim, int rotary_dim, int n) {
    return head_dim % (2 * n) == 0 && rotary_dim % (2 * n) == 0 && head_dim / (2 * n) <= 32;
}

template <typename T>
cudaError_t norm_rope_for(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int N = Vec<T>::N, E = (int)sizeof(T);
    const int H = a.n_heads + a.n_kv_heads;
    const bool vec = vec_shape(a.head_dim, a.rotary_dim, N) &&
                     (a.n_heads == 0 || (rows16(a.q, a.q_stride, E) && rows16(a.q_out, a.q_out_stride, E) && rows16(a.q_gain, 0, 4))) &&
                     (a.n_kv_heads == 0 || (rows16(a.k, a.k_stride, E) && rows16(a.k_out, a.k_out_stride, E) && rows16(a.k_gain, 0, 4)));
    trace_before("norm_rope", stream);
    cudaError_t e;
    if (vec) {
        const HeadSplit hs = head_split(a.head_dim, N, H, kNormHeads);
        const dim3 grid((unsigned)((a.tokens + hs.slots - 1) / hs.slots), (unsigned)hs.parts);
        e = a.interleaved ? launch_pdl(norm_rope_vec_kernel<T, false>, grid, dim3(hs.threads), 0, stream, 1, a, hs)
                          : launch_pdl(norm_rope_vec_kernel<T, true>, grid, dim3(hs.threads), 0, stream, 1, a, hs);
    } else {
        const unsigned y = (unsigned)std::min(16, (H + kNormThreads / 32 - 1) / (kNormThreads / 32));
        e = launch_pdl(norm_rope_any_kernel<T>, dim3((unsigned)a.tokens, y), dim3(kNormThreads), 0, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "norm_rope launch");
}

template <typename T>
cudaError_t norm_rope_grad_for(const NormRopeGradArgs& a, cudaStream_t stream) {
    constexpr int N = Vec<T>::N, E = (int)sizeof(T);
    const int H = a.n_heads + a.n_kv_heads;
    const int most = std::min(kNormGradMaxCtas, std::max(1, device_sm_count()) * kNormGradCtasPerSm);
    const bool vec = vec_shape(a.head_dim, a.rotary_dim, N) &&
                     (a.n_heads == 0 || (rows16(a.q, a.q_stride, E) && rows16(a.dq, a.dq_stride, E) && rows16(a.q_grad, a.q_grad_stride, E) && rows16(a.q_gain, 0, 4))) &&
                     (a.n_kv_heads == 0 || (rows16(a.k, a.k_stride, E) && rows16(a.dk, a.dk_stride, E) && rows16(a.k_grad, a.k_grad_stride, E) && rows16(a.k_gain, 0, 4)));
    int ctas;
    cudaError_t e = cudaSuccess;
    trace_before("norm_rope_grad", stream);
    if (a.tokens == 0) {                                  // the gains' gradients are zeros
        ctas = 0;
    } else if (vec) {
        const HeadSplit hs = head_split(a.head_dim, N, H, kNormGradHeads);
        ctas = std::min(most, (a.tokens + hs.slots - 1) / hs.slots);
        const size_t smem = (size_t)hs.slots * hs.rows * a.head_dim * sizeof(float);   // at most 256 threads of 2 N columns: 16 KB
        e = a.interleaved ? launch_pdl(norm_rope_grad_vec_kernel<T, false>, dim3(ctas), dim3(hs.threads), smem, stream, 1, a, hs)
                          : launch_pdl(norm_rope_grad_vec_kernel<T, true>, dim3(ctas), dim3(hs.threads), smem, stream, 1, a, hs);
    } else {
        const long long rows = (long long)a.tokens * H;
        ctas = (int)std::min<long long>(most, (rows + kNormAnyWarps - 1) / kNormAnyWarps);
        const size_t smem = (size_t)kNormAnyWarps * 2 * a.head_dim * sizeof(float);    // 32 KB at head_dim 1024
        e = launch_pdl(norm_rope_grad_any_kernel<T>, dim3(ctas), dim3(kNormAnyWarps * 32), smem, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "norm_rope_grad launch");
    trace_before("norm_rope_gains", stream);
    e = launch_pdl(norm_rope_gains_kernel, dim3((2 * a.head_dim + 31) / 32), dim3(256), 0, stream, 1, (const float*)a.partials, ctas,
                   a.head_dim, a.n_heads ? a.q_gain_grad : nullptr, a.n_kv_heads ? a.k_gain_grad : nullptr);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "norm_rope_gains launch");
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool f32, cudaStream_t stream) {
    return f32 ? norm_rope_for<float>(a, stream) : norm_rope_for<__nv_bfloat16>(a, stream);
}

size_t norm_rope_grad_scratch_bytes(int head_dim) { return (size_t)kNormGradMaxCtas * 2 * head_dim * sizeof(float); }

cudaError_t launch_norm_rope_grad(const NormRopeGradArgs& a, bool f32, cudaStream_t stream) {
    return f32 ? norm_rope_grad_for<float>(a, stream) : norm_rope_grad_for<__nv_bfloat16>(a, stream);
}

}  // namespace ll
