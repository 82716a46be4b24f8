// RMS norm of every Q and K head with its gain, and the rotary positions, in one pass, and its gradient.
// Head row x of d elements:  r = 1 / sqrt(mean x^2 + eps),  n = x r g,  y = R(p) n, R the rotation of rope.cu.
// With dy given:  dn = R^T dy,  dx = r (g dn - x r^2 mean(g dn x)),  dg = sum over tokens and heads of dn x r.
//
// Bound by memory: forward reads and writes a head once, the gradient reads x and dy and writes dx.  The group of
// threads that holds a head sums its squares by shuffles, so nothing is read twice and nothing goes through shared
// memory; a token's (cos, sin) row and the gains stay in registers for a thread's heads.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "head_split.h"
#include "kernels.h"
#include "vec16.cuh"

namespace ll {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormGradThreads = 128;
constexpr int kNormGradCtasPerSm = 4;
// Heads of a thread: 48 bytes a column on their way (16384 tokens of 64 + 8 BF16 heads: 105 us with six, 113 with three;
// of 32 + 8 float32 heads: 103 with three, 109 with six); in the gradient, with x and dy, 32 (4096 tokens of 32 + 8: BF16
// 37.5 us with four, 41.6 with one; float32 48 with two, 54 with four).
// Element by element or in pairs a column takes more registers: 98 of 128 rotated, BF16, 385 us with six, 236 with three.
template <typename T, int VEC = 2>
constexpr int kNormHeads = VEC < 2 || sizeof(T) == 4 ? 3 : 6;
template <typename T, int VEC = 2>
constexpr int kNormGradHeads = VEC < 2 || sizeof(T) == 4 ? 2 : 4;
constexpr int kNormAnyWarps = 4;       // of the gradient's CTA for heads that no group holds

int head_lanes(int head_dim, int rotary_dim, int n, bool interleaved) {
    const int turned = interleaved ? (rotary_dim + 2 * n - 1) / (2 * n) : (rotary_dim / 2 + n - 1) / n;
    return turned + (head_dim - rotary_dim + 2 * n - 1) / (2 * n);
}

// A thread's two columns, at e0 and e1, of n0 and n1 elements (N each where a head divides into whole columns: VEC 2; VEC 1:
// an even number, which lie for loads of two; VEC 0: element by element):
// rotated half-split, they hold the two ends of its pairs; interleaved or behind the rotated part, neighbours.
template <int N, bool HALF, int VEC>
struct Columns {
    int e0, e1, n0, n1;
    bool turn;
    LL_DEVINL Columns(int lane, int head_dim, int rotary_dim) {
        const int half = rotary_dim >> 1, turned = HALF ? (half + N - 1) / N : (rotary_dim + 2 * N - 1) / (2 * N);
        turn = lane < turned;
        if (HALF && turn) {
            e0 = lane * N;
            e1 = half + e0;
            n0 = n1 = min(N, half - e0);
        } else {
            e0 = turn ? lane * 2 * N : rotary_dim + (lane - turned) * 2 * N;
            e1 = e0 + N;
            const int end = turn ? rotary_dim : head_dim;
            n0 = max(0, min(N, end - e0));
            n1 = max(0, min(N, end - e1));
        }
        if (VEC == 2) n0 = n1 = N;
    }
};

// N elements of T as they lie in memory.
template <typename T, int N, int VEC>
struct Column {
    static constexpr int WORDS = VEC > 0 ? N * (int)sizeof(T) / 4 : N;
    uint32_t w[WORDS];

    LL_DEVINL void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    LL_DEVINL void load(const T* p, int n) {
        if constexpr (VEC == 1) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if constexpr (sizeof(T) == 2) {
                    w[i] = 2 * i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
                } else {
                    const uint2 x = 2 * i < n ? reinterpret_cast<const uint2*>(p)[i] : make_uint2(0u, 0u);
                    w[2 * i] = x.x; w[2 * i + 1] = x.y;
                }
            }
        } else if constexpr (VEC == 2 && WORDS == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x; w[1] = x.y;
        } else if constexpr (VEC == 2) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 x = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if constexpr (sizeof(T) == 2) w[i] = i < n ? reinterpret_cast<const unsigned short*>(p)[i] : 0u;
                else w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
            }
        }
    }
    LL_DEVINL void unpack(float2 (&v)[N / 2]) const {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            else if constexpr (VEC > 0) v[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
            else v[i] = make_float2(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
        }
    }
    static LL_DEVINL void store(T* p, const float2 (&v)[N / 2], int n) {
        if constexpr (VEC == 1) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (2 * i >= n) continue;
                if constexpr (sizeof(T) == 2) reinterpret_cast<uint32_t*>(p)[i] = pack_bf16x2(v[i].x, v[i].y);
                else reinterpret_cast<float2*>(p)[i] = v[i];
            }
        } else if constexpr (VEC == 2) {
            uint32_t o[WORDS];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if constexpr (sizeof(T) == 2) {
                    o[i] = pack_bf16x2(v[i].x, v[i].y);
                } else {
                    o[2 * i] = __float_as_uint(v[i].x);
                    o[2 * i + 1] = __float_as_uint(v[i].y);
                }
            }
            if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
            else {
#pragma unroll
                for (int i = 0; i < WORDS / 4; ++i)
                    reinterpret_cast<uint4*>(p)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) Vec<T>::put(p + i, i & 1 ? v[i / 2].y : v[i / 2].x);
        }
    }
};

// Gains of a column (0 behind its elements).
template <int N, int VEC>
LL_DEVINL void load_gains(const float* p, int n, float2 (&v)[N / 2]) {
    if (VEC == 1) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) v[i] = 2 * i < n ? __ldg(reinterpret_cast<const float2*>(p) + i) : make_float2(0.f, 0.f);
    } else if (VEC == 2) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p) + i);
            v[2 * i] = make_float2(x.x, x.y);
            v[2 * i + 1] = make_float2(x.z, x.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) v[i] = make_float2(2 * i < n ? __ldg(p + 2 * i) : 0.f, 2 * i + 1 < n ? __ldg(p + 2 * i + 1) : 0.f);
    }
}

LL_DEVINL float2 swapped(float2 v) { return make_float2(v.y, v.x); }
LL_DEVINL float2 both(float x) { return make_float2(x, x); }

template <int W>
LL_DEVINL float group_sum(float x) {
#pragma unroll
    for (int o = W >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

LL_DEVINL int norm_position(const int32_t* positions, int t, int max_position, int32_t* status, bool flag) {
    const int p = positions[t];
    if (p >= 0 && p < max_position) return p;
    if (flag) flag_status(status, LL_DEV_BAD_POSITION);
    return -1;
}

// The (cos, sin) entries of a thread's two columns, as whole pairs of elements: half-split, c[i], s[i] belong to
// elements 2 i and 2 i + 1 of both columns; interleaved, to pair i of the thread's N, with s = (-sin, sin).
template <int N, bool HALF, int VEC>
struct Turn {
    static constexpr int M = HALF ? N / 2 : N;
    float2 c[M], s[M];
    LL_DEVINL void load(const float2* table, int pos, int half, const Columns<N, HALF, VEC>& col) {
        const float2* cs = table + (size_t)pos * half + (HALF ? col.e0 : col.e0 / 2);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {               // two pairs of the head at a time
            float4 x;
            if (VEC == 2) {
                x = __ldg(reinterpret_cast<const float4*>(cs) + i);
            } else if (VEC == 1 && HALF) {
                x = 2 * i < col.n0 ? __ldg(reinterpret_cast<const float4*>(cs) + i) : make_float4(1.f, 0.f, 1.f, 0.f);
            } else {
                // pairs 2 i, 2 i + 1 of the thread: of elements in the column (half), or in either column (interleaved)
                const int have = HALF ? col.n0 : (col.n0 + col.n1) / 2;
                const float2 a = 2 * i < have ? __ldg(cs + 2 * i) : make_float2(1.f, 0.f);
                const float2 b = 2 * i + 1 < have ? __ldg(cs + 2 * i + 1) : make_float2(1.f, 0.f);
                x = make_float4(a.x, a.y, b.x, b.y);
            }
            if (HALF) {
                c[i] = make_float2(x.x, x.z);
                s[i] = make_float2(x.y, x.w);
            } else {
                c[(2 * i) % M] = both(x.x);
                s[(2 * i) % M] = make_float2(-x.y, x.y);
                c[(2 * i + 1) % M] = both(x.z);
                s[(2 * i + 1) % M] = make_float2(-x.w, x.w);
            }
        }
    }
};

// Forward.  The gains are taken into the factors of the rotation once for a thread's U heads of a token: with a, b
// the columns of x,  a' = r (a fa + b ga),  b' = r (b fb + a gb)  (interleaved: a' = r (a fa + swapped(a) ga), b' likewise).
template <typename T, int N, bool HALF, int W, int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const NormRopeArgs a, const HeadSplit hs, float inv_d) {
    using Col = Column<T, N, VEC>;
    constexpr int P = N / 2, U = kNormHeads<T, VEC>;
    pdl_wait();
    pdl_trigger();
    const int group = threadIdx.x / W, lane = threadIdx.x % W;
    const int slot = group / hs.rows, row = group - slot * hs.rows;
    const int t = blockIdx.x * hs.slots + slot;
    const bool here = slot < hs.slots && t < a.tokens, mine = here && lane < hs.lanes;
    const Columns<N, HALF, VEC> col(lane, a.head_dim, a.rotary_dim);
    const int H = a.n_heads + a.n_kv_heads, gap = col.e1 - col.e0;
    const int h0 = first_head(hs, blockIdx.y, row, U);
    const int pos_read = here ? a.positions[t] : 0;
    const T* q = static_cast<const T*>(a.q) + (size_t)t * a.q_stride + col.e0;
    const T* k = static_cast<const T*>(a.k) + (size_t)t * a.k_stride + col.e0 - (long long)a.n_heads * a.head_dim;
    Col w0[U], w1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {                       // (on their way before the position is there)
        const int h = h0 + u * hs.rows;
        w0[u].zero();
        w1[u].zero();
        if (mine && h < H) {
            const T* src = (h < a.n_heads ? q : k) + (size_t)h * a.head_dim;
            w0[u].load(src, col.n0);
            w1[u].load(src + gap, col.n1);
        }
    }
    const bool known = pos_read >= 0 && pos_read < a.max_position;
    if (here && !known && lane == 0 && row == 0 && blockIdx.y == 0) flag_status(a.status, LL_DEV_BAD_POSITION);
    const bool live = known && mine;                    // (every thread takes part in the shuffles)
    float2 fa[P], ga[P], fb[P], gb[P];
    const auto factors = [&](const float* gain) {
        load_gains<N, VEC>(gain + col.e0, col.n0, fa);
        load_gains<N, VEC>(gain + col.e1, col.n1, fb);
        if (!col.turn) return;
        Turn<N, HALF, VEC> turn;
        turn.load(a.table, pos_read, a.rotary_dim >> 1, col);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (HALF) {
                ga[i] = mul2(fb[i], make_float2(-turn.s[i].x, -turn.s[i].y));
                gb[i] = mul2(fa[i], turn.s[i]);
                fa[i] = mul2(fa[i], turn.c[i]);
                fb[i] = mul2(fb[i], turn.c[i]);
            } else {
                constexpr int M = Turn<N, HALF, VEC>::M;
                ga[i] = mul2(swapped(fa[i]), turn.s[i]);
                gb[i] = mul2(swapped(fb[i]), turn.s[(P + i) % M]);
                fa[i] = mul2(fa[i], turn.c[i]);
                fb[i] = mul2(fb[i], turn.c[(P + i) % M]);
            }
        }
    };
    bool gain_q = h0 < a.n_heads;
    if (live && h0 < H) factors(gain_q ? a.q_gain : a.k_gain);      // (no head, no gain: Q alone has no k_gain)
    T* q_out = static_cast<T*>(a.q_out) + (size_t)t * a.q_out_stride + col.e0;
    T* k_out = static_cast<T*>(a.k_out) + (size_t)t * a.k_out_stride + col.e0 - (long long)a.n_heads * a.head_dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * hs.rows;
        float2 x[P], y[P], sum = make_float2(0.f, 0.f);
        w0[u].unpack(x);
        w1[u].unpack(y);
#pragma unroll
        for (int i = 0; i < P; ++i) sum = fma2(y[i], y[i], fma2(x[i], x[i], sum));
        const float total = group_sum<W>(sum.x + sum.y);
        if (!live || h >= H) continue;
        const bool isq = h < a.n_heads;
        if (isq != gain_q) {
            gain_q = isq;
            factors(a.k_gain);
        }
        const float2 r = both(rsqrtf(total * inv_d + a.eps));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (col.turn) {
                const float2 u0 = HALF ? y[i] : swapped(x[i]), u1 = HALF ? x[i] : swapped(y[i]);
                const float2 a0 = fma2(x[i], fa[i], mul2(u0, ga[i])), b0 = fma2(y[i], fb[i], mul2(u1, gb[i]));
                x[i] = mul2(a0, r);
                y[i] = mul2(b0, r);
            } else {
                x[i] = mul2(mul2(x[i], r), fa[i]);
                y[i] = mul2(mul2(y[i], r), fb[i]);
            }
        }
        T* dst = (isq ? q_out : k_out) + (size_t)h * a.head_dim;
        Col::store(dst, x, col.n0);
        Col::store(dst + gap, y, col.n1);
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

// Heads that no group of threads holds: a warp per head, two passes over it.
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
        const float r = rsqrtf(group_sum<32>(sum) / (float)a.head_dim + a.eps);
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

// Head rows of one tensor (q or k).
template <typename T>
struct HeadRows {
    const T *x, *dy;
    T* dx;
    long long x_stride, dy_stride, dx_stride;
    const float* gain;
    int heads;
};

// A head's columns x0, x1 and dy in y0, y1, the gains in g0, g1: turns y into dn, g into g dn, and adds to the sums.
template <int N, bool HALF, typename TURN>
LL_DEVINL void grad_sums(const float2 (&x0)[N / 2], const float2 (&x1)[N / 2], float2 (&y0)[N / 2], float2 (&y1)[N / 2],
                         float2 (&g0)[N / 2], float2 (&g1)[N / 2], bool turned, const TURN& turn, float2& sq, float2& dot) {
    constexpr int P = N / 2, M = TURN::M;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (turned) {                                     // dn = R^T dy
            if (HALF) {
                const float2 n0 = fma2(y0[i], turn.c[i], mul2(y1[i], turn.s[i]));
                y1[i] = fma2(y1[i], turn.c[i], mul2(y0[i], make_float2(-turn.s[i].x, -turn.s[i].y)));
                y0[i] = n0;
            } else {                                      // (s swapped is -s)
                y0[i] = fma2(y0[i], turn.c[i], mul2(swapped(y0[i]), swapped(turn.s[i])));
                y1[i] = fma2(y1[i], turn.c[(P + i) % M], mul2(swapped(y1[i]), swapped(turn.s[(P + i) % M])));
            }
        }
        g0[i] = mul2(y0[i], g0[i]);
        g1[i] = mul2(y1[i], g1[i]);
        sq = fma2(x1[i], x1[i], fma2(x0[i], x0[i], sq));
        dot = fma2(g1[i], x1[i], fma2(g0[i], x0[i], dot));
    }
}

// With the sums over the head: x0, x1 become dx, and dn x r goes to the gains' gradients.
template <int N>
LL_DEVINL void grad_values(float sum_sq, float sum_dot, float inv_d, float eps, float2 (&x0)[N / 2], float2 (&x1)[N / 2],
                           const float2 (&y0)[N / 2], const float2 (&y1)[N / 2], const float2 (&g0)[N / 2], const float2 (&g1)[N / 2],
                           float2 (&dg0)[N / 2], float2 (&dg1)[N / 2]) {
    const float r = rsqrtf(sum_sq * inv_d + eps), f = -(sum_dot * inv_d * r * r);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        dg0[i] = fma2(y0[i], mul2(x0[i], both(r)), dg0[i]);
        dg1[i] = fma2(y1[i], mul2(x1[i], both(r)), dg1[i]);
        x0[i] = mul2(fma2(x0[i], both(f), g0[i]), both(r));
        x1[i] = mul2(fma2(x1[i], both(f), g1[i]), both(r));
    }
}

// The tokens go round the CTAs of a tensor (q's, then k's); a group has U heads of a token at a time, its loads all on
// their way before the first is used, the token's position read a turn ahead.  A thread keeps the gain gradients of its
// columns over all its tokens.  The sums of a CTA's groups meet in shared memory in a fixed order, those of the CTAs in a
// second kernel: the same bits every time.
template <typename T, int N, bool HALF, int W, int VEC>
__global__ void __launch_bounds__(kNormGradThreads, N == 4 ? kNormGradCtasPerSm : 2)
    norm_rope_grad_kernel(const NormRopeGradArgs a, const HeadSplit q_split, const HeadSplit k_split, int q_ctas, float inv_d) {
    using Col = Column<T, N, VEC>;
    constexpr int P = N / 2, U = kNormGradHeads<T, VEC>;
    extern __shared__ float s_dg[];                       // [groups][head_dim]
    pdl_wait();
    pdl_trigger();
    const bool isq = (int)blockIdx.x < q_ctas;
    const int ctas = isq ? q_ctas : gridDim.x - q_ctas, cta = isq ? blockIdx.x : blockIdx.x - q_ctas;
    HeadRows<T> m;
    m.x = static_cast<const T*>(isq ? a.q : a.k);
    m.dy = static_cast<const T*>(isq ? a.dq : a.dk);
    m.dx = static_cast<T*>(isq ? a.q_grad : a.k_grad);
    m.x_stride = isq ? a.q_stride : a.k_stride;
    m.dy_stride = isq ? a.dq_stride : a.dk_stride;
    m.dx_stride = isq ? a.q_grad_stride : a.k_grad_stride;
    m.gain = isq ? a.q_gain : a.k_gain;
    m.heads = isq ? a.n_heads : a.n_kv_heads;
    const int rows = isq ? q_split.rows : k_split.rows, slots = isq ? q_split.slots : k_split.slots;
    const int parts = isq ? q_split.parts : k_split.parts;
    const int group = threadIdx.x / W, lane = threadIdx.x % W;
    const int slot = group / rows, row = group - slot * rows;
    const Columns<N, HALF, VEC> col(lane, a.head_dim, a.rotary_dim);
    const int gap = col.e1 - col.e0;
    const bool worker = slot < slots && lane < q_split.lanes;
    float2 dg0[P], dg1[P];
#pragma unroll
    for (int i = 0; i < P; ++i) dg0[i] = dg1[i] = make_float2(0.f, 0.f);

    const int t_step = ctas * slots;
    int t = cta * slots + slot;
    int pos_next = slot < slots && t < a.tokens ? a.positions[t] : 0;
    // (as many turns for every group of the CTA: the shuffles need whole warps)
    for (int t0 = cta * slots; t0 < a.tokens; t0 += t_step, t += t_step) {
        const int pos = pos_next;
        pos_next = slot < slots && t + t_step < a.tokens ? a.positions[t + t_step] : 0;
        const bool here = slot < slots && t < a.tokens, known = pos >= 0 && pos < a.max_position;
        if (here && !known && lane == 0 && row == 0) flag_status(a.status, LL_DEV_BAD_POSITION);
        const bool live = here && known && worker;
        for (int part = 0; part < parts; ++part) {
            const int h0 = part * rows * U + row;
            Col wx0[U], wx1[U], wy0[U], wy1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * rows;
                if (live && h < m.heads) {
                    const T* x = m.x + t * m.x_stride + h * a.head_dim + col.e0;
                    const T* dy = m.dy + t * m.dy_stride + h * a.head_dim + col.e0;
                    wx0[u].load(x, col.n0);
                    wx1[u].load(x + gap, col.n1);
                    wy0[u].load(dy, col.n0);
                    wy1[u].load(dy + gap, col.n1);
                }
            }
            Turn<N, HALF, VEC> turn;
            if (live && col.turn) turn.load(a.table, pos, a.rotary_dim >> 1, col);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * rows;
                const bool on = live && h < m.heads;
                float2 x0[P], x1[P], y0[P], y1[P], g0[P], g1[P], sq = make_float2(0.f, 0.f), dot = sq;
                if (on) {
                    wx0[u].unpack(x0);
                    wx1[u].unpack(x1);
                    wy0[u].unpack(y0);
                    wy1[u].unpack(y1);
                    load_gains<N, VEC>(m.gain + col.e0, col.n0, g0);
                    load_gains<N, VEC>(m.gain + col.e1, col.n1, g1);
                    grad_sums<N, HALF>(x0, x1, y0, y1, g0, g1, col.turn, turn, sq, dot);
                }
                const float sum_sq = group_sum<W>(sq.x + sq.y), sum_dot = group_sum<W>(dot.x + dot.y);
                if (!on) continue;
                grad_values<N>(sum_sq, sum_dot, inv_d, a.eps, x0, x1, y0, y1, g0, g1, dg0, dg1);
                T* dst = m.dx + t * m.dx_stride + h * a.head_dim + col.e0;
                Col::store(dst, x0, col.n0);
                Col::store(dst + gap, x1, col.n1);
            }
        }
    }
    if (worker) {
        float* s0 = s_dg + group * a.head_dim + col.e0;
        float* s1 = s_dg + group * a.head_dim + col.e1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i < col.n0) s0[i] = i & 1 ? dg0[i / 2].y : dg0[i / 2].x;
            if (i < col.n1) s1[i] = i & 1 ? dg1[i / 2].y : dg1[i / 2].x;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.head_dim; e += blockDim.x) {
        float sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < slots * rows; ++i) sum += s_dg[i * a.head_dim + e];
        a.partials[(size_t)blockIdx.x * a.head_dim + e] = sum;
    }
}

// The same for BF16 rows that start on 16 bytes: a turn's heads (a token's, or those of several tokens with few heads)
// come by bulk copies into shared memory while the turn before is worked on.  4096 tokens of 32 + 8 heads of 128: 31 us,
// with loads into registers 37.5; of 256: 50 and 62; three stages 33, five or six CTAs per SM 33 and 35.  (float32, with
// twice the bytes for the same work: no faster than loads into registers.)
constexpr int kGradStages = 2;
constexpr int kGradTurnBytes = kNormGradThreads * 8 * kNormGradHeads<__nv_bfloat16> * 2;       // of x, and of dy, at most

template <bool HALF, int W>
__global__ void __launch_bounds__(kNormGradThreads, kNormGradCtasPerSm)
    norm_rope_grad_bulk_kernel(const NormRopeGradArgs a, const HeadSplit q_split, const HeadSplit k_split, int q_ctas, float inv_d) {
    using T = __nv_bfloat16;
    using Col = Column<T, 4, 2>;
    constexpr int P = 2, U = kNormGradHeads<T>, BYTES = kGradTurnBytes;
    extern __shared__ __align__(128) uint8_t s_turn[];    // [kGradStages][x, dy]; then the groups' gain gradients
    __shared__ uint64_t full[kGradStages];
    __shared__ int abort_s;
    const bool isq = (int)blockIdx.x < q_ctas;
    const int ctas = isq ? q_ctas : gridDim.x - q_ctas, cta = isq ? blockIdx.x : blockIdx.x - q_ctas;
    HeadRows<T> m;
    m.x = static_cast<const T*>(isq ? a.q : a.k);
    m.dy = static_cast<const T*>(isq ? a.dq : a.dk);
    m.dx = static_cast<T*>(isq ? a.q_grad : a.k_grad);
    m.x_stride = isq ? a.q_stride : a.k_stride;
    m.dy_stride = isq ? a.dq_stride : a.dk_stride;
    m.dx_stride = isq ? a.q_grad_stride : a.k_grad_stride;
    m.gain = isq ? a.q_gain : a.k_gain;
    m.heads = isq ? a.n_heads : a.n_kv_heads;
    const int rows = isq ? q_split.rows : k_split.rows, slots = isq ? q_split.slots : k_split.slots;
    const int parts = isq ? q_split.parts : k_split.parts, d = a.head_dim;
    const int group = threadIdx.x / W, lane = threadIdx.x % W;
    const int slot = group / rows, row = group - slot * rows;
    const Columns<4, HALF, 2> col(lane, d, a.rotary_dim);
    const int gap = col.e1 - col.e0;
    const bool worker = slot < slots && lane < q_split.lanes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kGradStages; ++i) mbar_init(&full[i], 1);
        abort_s = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int t_step = ctas * slots;
    const int rounds = a.tokens > cta * slots ? (a.tokens - cta * slots + t_step - 1) / t_step : 0, turns = rounds * parts;
    // turn n: heads [part rows U, + rows U) of tokens t0 .. t0 + slots - 1; warp 0
    const auto issue = [&](int n) {
        const int t0 = cta * slots + n / parts * t_step, h0 = n % parts * rows * U, st = n % kGradStages;
        const int count = min(slots, a.tokens - t0);
        const uint32_t bytes = (uint32_t)(min(rows * U, m.heads - h0) * d * (int)sizeof(T));
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&full[st], 2 * count * bytes);
        __syncwarp();
        for (int i = threadIdx.x; i < 2 * count; i += 32) {
            const int s = i >> 1, t = t0 + s;
            const T* from = i & 1 ? m.dy + t * m.dy_stride : m.x + t * m.x_stride;
            bulk_load(s_turn + (st * 2 + (i & 1)) * BYTES + s * rows * U * d * (int)sizeof(T), from + h0 * d, bytes, &full[st]);
        }
    };
    int issued = 0;
    if (threadIdx.x < 32)
        for (; issued < min(kGradStages, turns); ++issued) issue(issued);
    float2 g0[P], g1[P], dg0[P], dg1[P];
#pragma unroll
    for (int i = 0; i < P; ++i) g0[i] = g1[i] = dg0[i] = dg1[i] = make_float2(0.f, 0.f);
    if (worker) {
        load_gains<4, 2>(m.gain + col.e0, 4, g0);
        load_gains<4, 2>(m.gain + col.e1, 4, g1);
    }
    int t = cta * slots + slot, n = 0;
    int pos_next = slot < slots && t < a.tokens ? a.positions[t] : 0;
    bool stop = false;
    for (int round = 0; round < rounds && !stop; ++round, t += t_step) {
        const int pos = pos_next;
        pos_next = slot < slots && t + t_step < a.tokens ? a.positions[t + t_step] : 0;
        const bool here = slot < slots && t < a.tokens, known = pos >= 0 && pos < a.max_position;
        if (here && !known && lane == 0 && row == 0) flag_status(a.status, LL_DEV_BAD_POSITION);
        const bool live = here && known && worker;
        Turn<4, HALF, 2> turn;
        if (live && col.turn) turn.load(a.table, pos, a.rotary_dim >> 1, col);
        for (int part = 0; part < parts; ++part, ++n) {
            const int st = n % kGradStages, h0 = part * rows * U + row;
            const T* sx = reinterpret_cast<const T*>(s_turn + st * 2 * BYTES) + (slot * rows * U + row) * d + col.e0;
            mbar_wait_bounded(&full[st], (uint32_t)(n / kGradStages) & 1u, &abort_s, a.status);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * rows;
                const bool on = live && h < m.heads;
                float2 x0[P], x1[P], y0[P], y1[P], z0[P], z1[P], sq = make_float2(0.f, 0.f), dot = sq;
                if (on) {
                    Col c;
                    const T* x = sx + u * rows * d;
                    const T* dy = x + BYTES / sizeof(T);
                    c.load(x, 4);
                    c.unpack(x0);
                    c.load(x + gap, 4);
                    c.unpack(x1);
                    c.load(dy, 4);
                    c.unpack(y0);
                    c.load(dy + gap, 4);
                    c.unpack(y1);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        z0[i] = g0[i];
                        z1[i] = g1[i];
                    }
                    grad_sums<4, HALF>(x0, x1, y0, y1, z0, z1, col.turn, turn, sq, dot);
                }
                const float sum_sq = group_sum<W>(sq.x + sq.y), sum_dot = group_sum<W>(dot.x + dot.y);
                if (!on) continue;
                grad_values<4>(sum_sq, sum_dot, inv_d, a.eps, x0, x1, y0, y1, z0, z1, dg0, dg1);
                T* dst = m.dx + t * m.dx_stride + h * d + col.e0;
                Col::store(dst, x0, 4);
                Col::store(dst + gap, x1, 4);
            }
            stop = __syncthreads_or(abort_s);             // everyone has read the turn
            if (stop) break;
            if (threadIdx.x < 32 && issued < turns) issue(issued++);
        }
    }
    if (stop && threadIdx.x == 0) {                       // wait (bounded) for the copies in flight before the CTA leaves
        volatile int never = 0;
        for (int i = max(0, issued - kGradStages); i < issued; ++i)
            mbar_wait_bounded(&full[i % kGradStages], (uint32_t)(i / kGradStages) & 1u, &never, nullptr);
    }
    __syncthreads();
    float* s_dg = reinterpret_cast<float*>(s_turn);       // [groups][head_dim], all turns have been read
    if (worker) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s_dg[group * d + col.e0 + i] = i & 1 ? dg0[i / 2].y : dg0[i / 2].x;
            s_dg[group * d + col.e1 + i] = i & 1 ? dg1[i / 2].y : dg1[i / 2].x;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < d; e += blockDim.x) {
        float sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < slots * rows; ++i) sum += s_dg[i * d + e];
        a.partials[(size_t)blockIdx.x * d + e] = sum;
    }
}

// Heads that no group holds: a warp per head, the gain gradients of a warp in shared memory (a lane adds to its own elements only).
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
                r = rsqrtf(group_sum<32>(sq) / (float)d + a.eps);
                f = group_sum<32>(dot) / (float)d * r * r;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) {
        float sum = 0.f;
        for (int w = 0; w < kNormAnyWarps; ++w) sum += s_dg[w * 2 * d + i];
        a.partials[((size_t)blockIdx.x + (i < d ? 0 : gridDim.x)) * d + (i < d ? i : i - d)] = sum;
    }
}

// Gain gradients: the sums of the partials [q_rows of q, k_rows of k][head_dim], 32 of them at a time per column.
__global__ void __launch_bounds__(1024) norm_rope_gains_kernel(const float* partials, int q_rows, int k_rows, int head_dim,
                                                               float* q_gain_grad, float* k_gain_grad) {
    __shared__ float s_sum[32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    const bool isq = blockIdx.y == 0;
    float* out = isq ? q_gain_grad : k_gain_grad;
    if (!out) return;
    if (!isq) partials += (size_t)q_rows * head_dim;
    const int rows = isq ? q_rows : k_rows;
    float sum = 0.f;
    if (i < head_dim) {
#pragma unroll 5
        for (int c = w; c < rows; c += 32) sum += partials[(size_t)c * head_dim + i];
    }
    s_sum[w][lane] = sum;
    __syncthreads();
    const float total = group_sum<32>(s_sum[lane][w]);    // warp w: column w
    const int e = blockIdx.x * 32 + w;
    if (lane == 0 && e < head_dim) out[e] = total;
}

// f(N, W, VEC) with the constants of a call: columns of four elements, of eight where a head then needs more than a warp
// (and no group for longer heads: a warp takes two passes over each).  Whole, aligned columns take vector loads, others loads
// of two elements where they lie for it (BF16, 32 + 8 heads of 128, 16384 tokens, and the gradient of 4096: all of a head
// rotated 62 and 37 us; 100 elements, in pairs, 159 and 70; 98 half-split, element by element, 236 and 75; a warp per head
// took 300 for the gradient).  16384 tokens: 64 us with columns of four, 76 with eight (twice the registers).
struct NormShape {
    int n, lanes, vec;
};

bool rows_on(const void* p, long long stride, int esz, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * esz % bytes == 0;
}

// n 0: a head does not fit a warp.
NormShape norm_shape(int head_dim, int rotary_dim, bool interleaved) {
    for (int n : {4, 8}) {
        const int lanes = head_lanes(head_dim, rotary_dim, n, interleaved);
        if (lanes <= 32)
            return {n, lanes, head_dim % (2 * n) == 0 && rotary_dim % (2 * n) == 0 ? 2 : head_dim % 2 == 0 && (interleaved || rotary_dim % 4 == 0) ? 1 : 0};
    }
    return {0, 0, 0};
}

// The widest loads that a shape allows and its tensors lie for: lies(bytes of a column's load, bytes of a gain's).
template <typename F>
int load_form(const NormShape& s, int esz, F&& lies) {
    const bool pairs = s.vec > 0 && lies(2 * esz, 8);
    return s.vec == 2 && lies(std::min(16, s.n * esz), 16) ? 2 : pairs ? 1 : 0;
}

template <typename F>
cudaError_t for_shape(const NormShape& s, F&& f) {
    const auto with = [&](auto n, auto w) {
        return s.vec == 2   ? f(n, w, std::integral_constant<int, 2>{})
               : s.vec == 1 ? f(n, w, std::integral_constant<int, 1>{})
                            : f(n, w, std::integral_constant<int, 0>{});
    };
    using Four = std::integral_constant<int, 4>;
    if (s.n == 8) return with(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{});
    if (s.lanes <= 4) return with(Four{}, std::integral_constant<int, 4>{});
    if (s.lanes <= 8) return with(Four{}, std::integral_constant<int, 8>{});
    if (s.lanes <= 16) return with(Four{}, std::integral_constant<int, 16>{});
    return with(Four{}, std::integral_constant<int, 32>{});
}

template <typename T>
cudaError_t norm_rope_for(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int E = (int)sizeof(T);
    const int H = a.n_heads + a.n_kv_heads;
    NormShape s = norm_shape(a.head_dim, a.rotary_dim, a.interleaved);
    // on `bytes` and gains on `gain`
    const auto lies = [&](int bytes, int gain) {
        return (a.n_heads == 0 || (rows_on(a.q, a.q_stride, E, bytes) && rows_on(a.q_out, a.q_out_stride, E, bytes) && rows_on(a.q_gain, 0, 4, gain))) &&
               (a.n_kv_heads == 0 || (rows_on(a.k, a.k_stride, E, bytes) && rows_on(a.k_out, a.k_out_stride, E, bytes) && rows_on(a.k_gain, 0, 4, gain)));
    };
    s.vec = load_form(s, E, lies);
    trace_before("norm_rope", stream);
    cudaError_t e;
    if (s.n) {
        HeadSplit hs = head_split(s.lanes, H, s.vec == 2 ? kNormHeads<T> : kNormHeads<T, 0>, kNormThreads);
        const dim3 grid((unsigned)((a.tokens + hs.slots - 1) / hs.slots), (unsigned)hs.parts);
        e = for_shape(s, [&](auto n, auto w, auto vec) {
            return launch_pdl(a.interleaved ? norm_rope_kernel<T, n.value, false, w.value, vec.value> : norm_rope_kernel<T, n.value, true, w.value, vec.value>,
                              grid, dim3(hs.threads), 0, stream, 1, a, hs, 1.f / (float)a.head_dim);
        });
    } else {
        const unsigned y = (unsigned)std::min(16, (H + kNormThreads / 32 - 1) / (kNormThreads / 32));
        e = launch_pdl(norm_rope_any_kernel<T>, dim3((unsigned)a.tokens, y), dim3(kNormThreads), 0, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "norm_rope launch");
}

// f(W) for a HeadSplit's width.
template <typename F>
cudaError_t for_width(int width, F&& f) {
    if (width == 4) return f(std::integral_constant<int, 4>{});
    if (width == 8) return f(std::integral_constant<int, 8>{});
    if (width == 16) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

template <typename K, typename... Args>
cudaError_t launch_staged(K kernel, dim3 grid, dim3 block, int bytes, cudaStream_t stream, const Args&... args) {
    const cudaError_t e = ensure_func_attr((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes,
                                           "cudaFuncSetAttribute(norm_rope_grad_bulk_kernel)");
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, block, bytes, stream, 1, args...);
}

template <typename T>
cudaError_t norm_rope_grad_for(const NormRopeGradArgs& a, cudaStream_t stream) {
    constexpr int E = (int)sizeof(T);
    const int most = std::min(kNormGradMaxCtas, std::max(1, device_sm_count()) * kNormGradCtasPerSm);
    NormShape s = norm_shape(a.head_dim, a.rotary_dim, a.interleaved);
    const auto lies = [&](int bytes, int gain) {
        return (a.n_heads == 0 || (rows_on(a.q, a.q_stride, E, bytes) && rows_on(a.dq, a.dq_stride, E, bytes) && rows_on(a.q_grad, a.q_grad_stride, E, bytes) && rows_on(a.q_gain, 0, 4, gain))) &&
               (a.n_kv_heads == 0 || (rows_on(a.k, a.k_stride, E, bytes) && rows_on(a.dk, a.dk_stride, E, bytes) && rows_on(a.k_grad, a.k_grad_stride, E, bytes) && rows_on(a.k_gain, 0, 4, gain)));
    };
    s.vec = load_form(s, E, lies);
    const bool bulk = E == 2 && s.vec == 2 && s.n == 4 &&
                      (a.n_heads == 0 || (rows_on(a.q, a.q_stride, E, 16) && rows_on(a.dq, a.dq_stride, E, 16))) &&
                      (a.n_kv_heads == 0 || (rows_on(a.k, a.k_stride, E, 16) && rows_on(a.dk, a.dk_stride, E, 16)));
    int q_rows = 0, k_rows = 0;                           // of partials
    cudaError_t e = cudaSuccess;
    trace_before("norm_rope_grad", stream);
    if (a.tokens == 0) {                                  // the gains' gradients are zeros
    } else if (s.n) {
        // CTAs for q and for k, as many as their tokens ask for, in proportion to their heads up to what runs at once
        const int per_thread = s.vec == 2 ? kNormGradHeads<T> : kNormGradHeads<T, 0>;
        const HeadSplit qs = head_split(s.lanes, std::max(a.n_heads, 1), per_thread, kNormGradThreads);
        const HeadSplit ks = head_split(s.lanes, std::max(a.n_kv_heads, 1), per_thread, kNormGradThreads);
        q_rows = a.n_heads ? (a.tokens + qs.slots - 1) / qs.slots : 0;
        k_rows = a.n_kv_heads ? (a.tokens + ks.slots - 1) / ks.slots : 0;
        if (q_rows + k_rows > most) {
            const int q_part = a.n_heads == 0 ? 0 : a.n_kv_heads == 0 ? most :
                std::min(most - 1, std::max(1, (int)((long long)most * a.n_heads / (a.n_heads + a.n_kv_heads))));
            q_rows = std::min(q_rows, q_part);
            k_rows = std::min(k_rows, most - q_rows);
        }
        const size_t smem = (size_t)std::max(qs.slots * qs.rows, ks.slots * ks.rows) * a.head_dim * sizeof(float);   // at most 8 KB
        if (bulk) {
            e = for_width(qs.width, [&](auto w) {
                const auto kernel = a.interleaved ? norm_rope_grad_bulk_kernel<false, w.value> : norm_rope_grad_bulk_kernel<true, w.value>;
                return launch_staged(kernel, dim3(q_rows + k_rows), dim3(kNormGradThreads), 2 * kGradStages * kGradTurnBytes, stream, a, qs, ks,
                                     q_rows, 1.f / (float)a.head_dim);
            });
        } else e = for_shape(s, [&](auto n, auto w, auto vec) {
            return launch_pdl(a.interleaved ? norm_rope_grad_kernel<T, n.value, false, w.value, vec.value> : norm_rope_grad_kernel<T, n.value, true, w.value, vec.value>,
                              dim3(q_rows + k_rows), dim3(kNormGradThreads), smem, stream, 1, a, qs, ks, q_rows, 1.f / (float)a.head_dim);
        });
    } else {
        const long long rows = (long long)a.tokens * (a.n_heads + a.n_kv_heads);
        q_rows = k_rows = (int)std::min<long long>(most / 2, (rows + kNormAnyWarps - 1) / kNormAnyWarps);
        const size_t smem = (size_t)kNormAnyWarps * 2 * a.head_dim * sizeof(float);    // 32 KB at head_dim 1024
        e = launch_pdl(norm_rope_grad_any_kernel<T>, dim3(q_rows), dim3(kNormAnyWarps * 32), smem, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "norm_rope_grad launch");
    trace_before("norm_rope_gains", stream);
    e = launch_pdl(norm_rope_gains_kernel, dim3((a.head_dim + 31) / 32, 2), dim3(1024), 0, stream, 1, (const float*)a.partials, q_rows,
                   k_rows, a.head_dim, a.n_heads ? a.q_gain_grad : nullptr, a.n_kv_heads ? a.k_gain_grad : nullptr);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "norm_rope_gains launch");
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool f32, cudaStream_t stream) {
    return f32 ? norm_rope_for<float>(a, stream) : norm_rope_for<__nv_bfloat16>(a, stream);
}

size_t norm_rope_grad_scratch_bytes(int head_dim) { return (size_t)kNormGradMaxCtas * head_dim * sizeof(float); }

cudaError_t launch_norm_rope_grad(const NormRopeGradArgs& a, bool f32, cudaStream_t stream) {
    return f32 ? norm_rope_grad_for<float>(a, stream) : norm_rope_grad_for<__nv_bfloat16>(a, stream);
}

}  // namespace ll
