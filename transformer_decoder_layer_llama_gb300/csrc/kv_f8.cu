// New tokens' K and V into a paged cache of e4m3 codes with one scale per block and KV head.
//
// A block's scale is the smallest power of two s with |x| <= 448 s for every row written so far (the
// values are finite ones; infinities saturate, NaN stays NaN).  The call that writes a block's first
// token starts it afresh; a later call keeps s' = max(s, scale of the new rows) and, where that grew,
// rounds the earlier codes again to e4m3(code * s / s').  With powers of two that is exact except for
// codes that become subnormal.  Rows behind the last new token keep their bytes.
//
// A sequence's new tokens lie at its last positions, so each (block, KV head, K or V) is owned by one
// group of threads, which needs no atomics: it finds the largest magnitude, then writes codes and scale.
// Bound by memory: two bytes read and one written per element, the rows kept in registers between the
// maximum and the codes.  Ragged 70B-shaped chunks (8 sequences, 777 to 4096 tokens each, 119 MB): 24 us, 4.9
// TB/s (72% of the copy bandwidth; the launch, and the CTAs of blocks that the shorter sequences do not have,
// are the rest).  One token of 64 sequences, 32 heads: 6 us on the GPU, 10 per call from the host.
#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kAppendThreads = 256;

// 8 BF16 of a 16-byte load, as float32
LL_DEVINL void unpack8(const uint4& w, float (&v)[8]) {
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

// Magnitudes of 16 bits in each half: the larger of each (a NaN loses to a number).
LL_DEVINL uint32_t max_abs2(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
    return r;
}
// Largest finite magnitude among the N loads, as BF16 bits.  The plain maximum, unless that is an infinity:
// then the infinities are left out one by one.
template <int N>
LL_DEVINL uint32_t amax(const uint4 (&w)[N]) {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, w[i].x), w[i].y), w[i].z), w[i].w);
    uint32_t m = max(m2 & 0xffffu, m2 >> 16);
    if (m >= 0x7f80u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t p[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = p[j] & 0x7fffu, b = (p[j] >> 16) & 0x7fffu;
                m = max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
            }
        }
    }
    return m;
}

// The codes of x / scale.  A power of two (every scale but one that somebody else wrote) is divided by
// exactly by a multiplication; IEEE divisions took the chunk kernel twice its time.
LL_DEVINL uint2 codes8(const uint4& w, float scale) {
    float v[8];
    unpack8(w, v);
    if (!(scale > 0.f)) {                               // no finite value but zeros so far: codes 0, NaN kept
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] != v[i] ? v[i] : 0.f;
        return make_uint2(f32x4_to_e4m3x4(v[0], v[1], v[2], v[3]), f32x4_to_e4m3x4(v[4], v[5], v[6], v[7]));
    }
    const uint32_t u = __float_as_uint(scale);
    if ((u & 0x7fffffu) == 0u && (u >> 23) < 254u) {       // 2^e: times 2^-e (both normal)
        const float inv = __uint_as_float((254u - (u >> 23)) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
    } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], scale);
    }
    return make_uint2(f32x4_to_e4m3x4(v[0], v[1], v[2], v[3]), f32x4_to_e4m3x4(v[4], v[5], v[6], v[7]));
}

// The new tokens of sequence b: rows [start, start + n) of k and v at positions ctx - n .. ctx - 1.
// False (n = 0) where there are none, or where the counts do not fit together (flagged).
struct AppendSpan {
    int start, n, p0;
};
LL_DEVINL bool append_span(const AppendArgs& a, int b, bool flag, AppendSpan& s) {
    const int ctx = a.context_lens[b];
    const int c0 = a.cu_new ? a.cu_new[b] : b, c1 = a.cu_new ? a.cu_new[b + 1] : b + 1;
    const long long n = (long long)c1 - c0;
    s.start = c0;
    s.n = 0;
    if (n == 0) return false;
    if (c0 < 0 || n < 0 || c1 > a.tokens || n > a.max_new || n > ctx || ctx > a.max_context) {
        if (flag) flag_status(a.status, LL_DEV_BAD_POSITION);
        return false;
    }
    s.n = (int)n;
    s.p0 = ctx - (int)n;
    return true;
}

// One new token per sequence at most (max_new = 1).  Half a warp per (sequence, KV head, K or V): D / 8
// lanes hold its row, 8 elements each.  The rare block whose scale grows is left to the whole CTA, since
// its earlier rows are up to 32 KB.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_step_kernel(const AppendArgs a) {
    struct Grow {
        uint8_t* codes;
        int bytes;
        float ratio;
    };
    __shared__ Grow grow[kAppendThreads / 16];
    __shared__ int n_grow;
    const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;     // groups of 16 lanes
    if (threadIdx.x == 0) n_grow = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const long long unit = (long long)blockIdx.x * (kAppendThreads / 16) + sub;
    const int which = (int)(unit & 1);
    const long long bh = unit >> 1;
    const int b = (int)(bh / a.n_kv_heads), h = (int)(bh - (long long)b * a.n_kv_heads);
    AppendSpan s;
    if (b < a.batch && append_span(a, b, h == 0 && which == 0 && l == 0, s)) {
        const __nv_bfloat16* x = (which ? a.v : a.k) + (size_t)s.start * (which ? a.v_stride : a.k_stride) + (size_t)h * D;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (l < D / 8) w = *reinterpret_cast<const uint4*>(x + l * 8);
        const int blk = a.block_table[(size_t)b * a.max_blocks + s.p0 / a.block_size];
        if (blk < 0 || blk >= a.num_blocks) {
            if (h == 0 && which == 0 && l == 0) flag_status(a.status, LL_DEV_BAD_BLOCK);
        } else {
            const int off = s.p0 % a.block_size;
            const size_t bhk = (size_t)blk * a.n_kv_heads + h;
            float* sp = (which ? a.v_scale : a.k_scale) + bhk;
            const float old = off ? *sp : 0.f;
            const uint4 one[1] = {w};
            uint32_t m = amax(one);
            const uint32_t mask = 0xffffu << (threadIdx.x & 16);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
            __syncwarp(mask);                           // every lane has read the old scale
            const float f = fmaxf(old, e4m3_scale(__uint_as_float(m << 16)));
            uint8_t* codes = (which ? a.v_pool : a.k_pool) + bhk * a.block_size * D;
            if (l < D / 8) *reinterpret_cast<uint2*>(codes + (size_t)off * D + l * 8) = codes8(w, f);
            if (l == 0) {
                if (f != old || off == 0) *sp = f;
                if (f > old && off) {
                    const int i = atomicAdd(&n_grow, 1);   // the order of the list changes nothing
                    grow[i].codes = codes;
                    grow[i].bytes = off * D;
                    grow[i].ratio = old / f;
                }
            }
        }
    }
    __syncthreads();
    const int n = n_grow;
    for (int i = 0; i < n; ++i) {
        const Grow g = grow[i];
        for (int o = threadIdx.x * 16; o < g.bytes; o += kAppendThreads * 16) {
            uint4 w = *reinterpret_cast<uint4*>(g.codes + o);
            w.x = e4m3x4_rescale(w.x, g.ratio);
            w.y = e4m3x4_rescale(w.y, g.ratio);
            w.z = e4m3x4_rescale(w.z, g.ratio);
            w.w = e4m3x4_rescale(w.w, g.ratio);
            *reinterpret_cast<uint4*>(g.codes + o) = w;
        }
    }
}

// Several new tokens per sequence: one CTA per (block, KV head, K or V), D / 8 lanes per row.  PASSES
// steps of 2048 / D rows cover a block; all rows' loads are in flight before the first is used.
template <int D, int PASSES>
__global__ void __launch_bounds__(kAppendThreads) append_chunk_kernel(const AppendArgs a) {
    constexpr int LANES = D / 8, ROWS = kAppendThreads / LANES;
    __shared__ uint32_t warp_max[kAppendThreads / 32];
    const int b = blockIdx.y, of = (int)(blockIdx.x / (2u * a.n_kv_heads)), wh = (int)(blockIdx.x - of * 2u * a.n_kv_heads);
    const int which = wh >= a.n_kv_heads, h = wh - (which ? a.n_kv_heads : 0);
    pdl_wait();
    pdl_trigger();
    AppendSpan s;
    if (!append_span(a, b, threadIdx.x == 0 && blockIdx.x == 0, s)) return;
    const int bs = a.block_size;
    const int j = s.p0 / bs + of;                           // logical block
    const int lo = max(s.p0 - j * bs, 0), hi = min(s.p0 + s.n - j * bs, bs);   // its new rows
    if (lo >= hi) return;
    const int blk = a.block_table[(size_t)b * a.max_blocks + j];
    const long long stride = which ? a.v_stride : a.k_stride;
    const int l = threadIdx.x % LANES, r0 = threadIdx.x / LANES;
    // row r of the block is token start + (j bs + r - p0)
    const __nv_bfloat16* x = (which ? a.v : a.k) + ((long long)s.start + (long long)j * bs - s.p0) * stride +
                             (size_t)h * D + l * 8;
    uint4 w[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = lo + r0 + i * ROWS;
        w[i] = r < hi ? *reinterpret_cast<const uint4*>(x + (long long)r * stride) : make_uint4(0, 0, 0, 0);
    }
    if (blk < 0 || blk >= a.num_blocks) {                   // (looked at behind the loads, which do not need it)
        if (threadIdx.x == 0 && wh == 0) flag_status(a.status, LL_DEV_BAD_BLOCK);
        return;
    }
    const size_t bhk = (size_t)blk * a.n_kv_heads + h;
    float* sp = (which ? a.v_scale : a.k_scale) + bhk;
    const float old = lo ? *sp : 0.f;
    uint32_t m = amax(w);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();                                        // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) m = max(m, warp_max[i]);
    const float f = fmaxf(old, e4m3_scale(__uint_as_float(m << 16)));
    uint8_t* codes = (which ? a.v_pool : a.k_pool) + bhk * bs * D;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = lo + r0 + i * ROWS;
        if (r < hi) *reinterpret_cast<uint2*>(codes + (size_t)r * D + l * 8) = codes8(w[i], f);
    }
    if (threadIdx.x == 0) *sp = f;
    if (lo && f > old) {
        const float ratio = old / f;
        for (int o = threadIdx.x * 16; o < lo * D; o += kAppendThreads * 16) {
            uint4 c = *reinterpret_cast<uint4*>(codes + o);
            c.x = e4m3x4_rescale(c.x, ratio);
            c.y = e4m3x4_rescale(c.y, ratio);
            c.z = e4m3x4_rescale(c.z, ratio);
            c.w = e4m3x4_rescale(c.w, ratio);
            *reinterpret_cast<uint4*>(codes + o) = c;
        }
    }
}

__global__ void f8_positions_kernel(const int32_t* context_lens, int batch, int seq_len, int32_t* positions, int32_t* cu_new) {
    pdl_wait();
    pdl_trigger();
    const int t = (int)(blockIdx.x * blockDim.x + threadIdx.x);
    if (t < batch * seq_len) {
        const int b = t / seq_len;
        positions[t] = context_lens[b] - seq_len + (t - b * seq_len);
    }
    if (t <= batch) cu_new[t] = t * seq_len;
}

// (block, KV head, K or V) of a sequence: blocks that max_new consecutive positions can touch.
long long append_pairs(int max_new, int n_kv_heads, int block_size, int max_blocks) {
    return 2LL * n_kv_heads * std::min(((long long)max_new + block_size - 2) / block_size + 1, (long long)max_blocks);
}

template <int D>
cudaError_t append_for(const AppendArgs& a, cudaStream_t stream) {
    // Heads fastest: the CTAs that run together read whole token rows (blocks fastest: 25.5 us for the 24.2 of ragged 70B-shaped chunks).
    const long long pairs = append_pairs(a.max_new, a.n_kv_heads, a.block_size, a.max_blocks);
    cudaError_t e;
    trace_before("append_f8", stream);
    if (a.max_new == 1) {
        const long long units = 2LL * a.batch * a.n_kv_heads;
        const unsigned ctas = (unsigned)((units + kAppendThreads / 16 - 1) / (kAppendThreads / 16));
        e = launch_pdl(append_step_kernel<D>, dim3(ctas), dim3(kAppendThreads), 0, stream, 1, a);
    } else {
        const int bs = a.block_size;
        const dim3 grid((unsigned)pairs, (unsigned)a.batch);
        const int passes = (bs * D + kAppendThreads * 8 - 1) / (kAppendThreads * 8);
        if (passes <= 1) e = launch_pdl(append_chunk_kernel<D, 1>, grid, dim3(kAppendThreads), 0, stream, 1, a);
        else if (passes <= 2) e = launch_pdl(append_chunk_kernel<D, 2>, grid, dim3(kAppendThreads), 0, stream, 1, a);
        else if (passes <= 4) e = launch_pdl(append_chunk_kernel<D, 4>, grid, dim3(kAppendThreads), 0, stream, 1, a);
        else if (D == 64 || passes <= 8) e = launch_pdl(append_chunk_kernel<D, 8>, grid, dim3(kAppendThreads), 0, stream, 1, a);
        else e = launch_pdl(append_chunk_kernel<128, 16>, grid, dim3(kAppendThreads), 0, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "append_f8 launch");
}

}  // namespace

cudaError_t launch_f8_positions(const int32_t* context_lens, int batch, int seq_len, int32_t* positions, int32_t* cu_new,
                                cudaStream_t stream) {
    const int n = std::max(batch * seq_len, batch + 1);
    trace_before("f8_positions", stream);
    cudaError_t e = launch_pdl(f8_positions_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, context_lens,
                               batch, seq_len, positions, cu_new);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "f8_positions_kernel launch");
}

bool append_f8_fits(int max_new, int n_kv_heads, int block_size, int max_blocks) {
    return append_pairs(max_new, n_kv_heads, block_size, max_blocks) <= 0x7fffffffLL;
}

cudaError_t launch_append_f8(const AppendArgs& a, cudaStream_t stream) {
    if (a.batch <= 0 || a.tokens <= 0) return cudaSuccess;
    return a.head_dim == 128 ? append_for<128>(a, stream) : append_for<64>(a, stream);
}

}  // namespace ll
