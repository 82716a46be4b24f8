// Eviction from a paged cache by accumulated attention weight.  Of a sequence's n cached rows each KV head keeps the
// last `recent`, the first `sinks`, and of those between the ones of largest weight (NaN below every number, -0 as 0, ties
// to the lowest position), m rows in all.  They move, in order, to positions 0 .. m - 1 of the same blocks.
//
// Two kernels.  The choice: a CTA (a cluster where there are few rows of weights) per sequence and KV head finds the
// weight of the last kept row digit by digit in histograms (11, 11 and 10 bits of an order-preserving integer), then
// every warp counts, and after one exchange of counts writes, its own stretch of positions: no sort, five passes over
// weights in shared memory, or in L2 where they are too long for it.  Short rows take a warp each, with the keys in registers.  The move: kept[j] >= j ascending, so a row's place is never the source of a later one.  A CTA
// goes through its rows in order and writes a run of them when all its threads have read theirs; heads, tensors
// and slices of a row's bytes do not meet, so they are what is spread over CTAs.  Bound by the bytes of the rows.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kSelectThreads = 1024;      // at most
constexpr int kWarpSelectThreads = 128;
constexpr int kBins = 2048;
constexpr int kSpan = 128;             // positions of a warp at a time, four a lane
constexpr size_t kSelectSmem = 200 * 1024;   // of weights
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;         // of a thread, between two barriers

// Larger weights have larger keys; NaN has 0, below -infinity.
LL_DEVINL uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);           // (-0 + 0 = +0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int NC>
LL_DEVINL void sync_all() {
    if (NC == 1) __syncthreads();
    else cluster_sync();
}

LL_DEVINL void dsmem_add(int* p, uint32_t rank, int v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(cluster_map(smem_u32(p), rank)), "r"(v) : "memory");
}

LL_DEVINL void dsmem_store(int* p, uint32_t rank, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_map(smem_u32(p), rank)), "r"(v) : "memory");
}

LL_DEVINL int dsmem_load(const int* p, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_map(smem_u32(p), rank)) : "memory");
    return v;
}

struct Budget {
    int ctx, left;                     // rows of the sequence, and how many stay
    bool skip;                         // sizes or blocks that do not fit: nothing is touched
};

LL_DEVINL Budget evict_budget(const EvictArgs& a, int b, bool flag) {
    Budget g;
    g.ctx = a.context_lens[b];
    const int keep = a.keep ? a.keep[b] : a.max_keep;
    g.left = min(g.ctx, keep);
    g.skip = g.ctx < 0 || (long long)g.ctx > (long long)a.max_blocks * a.block_size || g.ctx > a.weights_width || keep < 0 ||
             g.left > a.max_keep;
    if (g.skip && flag) flag_status(a.status, LL_DEV_BAD_POSITION);
    return g;
}

// n weights to shared memory, by cp.async; and zeros.  A CTA's threads, 16 bytes each where the row lies for it.
LL_DEVINL void copy_weights(float* dst, const float* src, int n) {
    const bool wide = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
    const int whole = wide ? n & ~3 : 0;
    for (int i = 4 * threadIdx.x; i < whole; i += 4 * blockDim.x)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + i)), "l"(src + i) : "memory");
    for (int i = whole + threadIdx.x; i < n; i += blockDim.x)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + i)), "l"(src + i) : "memory");
}

// w[j0 .. n) of a row, thread `at` of `all`.
LL_DEVINL void zero_weights(float* w, int j0, int n, int at, int all) {
    const int lead = min(n, j0 + (int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(w + j0) & 15u)) / 4u & 3u));      // up to 16 bytes' start
    const int whole = lead + ((n - lead) & ~3);
    if (at < lead - j0) w[j0 + at] = 0.f;
    for (int j = lead + 4 * at; j < whole; j += 4 * all) *reinterpret_cast<float4*>(w + j) = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at < n - whole) w[whole + at] = 0.f;
}

// The sum of v over the lanes before this one in the list s[0 .. n), n <= 32, that each warp reads by itself: the value for
// entry `at`, and the total.
LL_DEVINL int before_in(const int* s, int n, int at, int& total) {
    const int lane = threadIdx.x & 31;
    const int mine = lane < n ? s[lane] : 0;
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    total = __shfl_sync(0xffffffffu, run, 31);
    return __shfl_sync(0xffffffffu, run - mine, at);
}

// CACHED: the CTA's stretch of the weights lies in shared memory (a.cached of them at most), read once.
template <int NC, bool CACHED>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) float s_w[];
    __shared__ __align__(16) int s_hist[3][kBins], s_scan[32], s_gt[32], s_eq[32], s_total[2], s_pick[2];
    const int hk = blockIdx.x / NC, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int threads = blockDim.x, warps = threads >> 5;
    for (int i = 4 * tid; i < 3 * kBins; i += 4 * threads) *reinterpret_cast<int4*>(&s_hist[0][0] + i) = make_int4(0, 0, 0, 0);
    pdl_wait();
    pdl_trigger();
    const int rank = NC == 1 ? 0 : (int)cluster_rank();
    const bool first = hk == 0 && rank == 0;
    const Budget g = evict_budget(a, b, first && tid == 0);
    const size_t row = (size_t)b * a.n_kv_heads + hk;
    const float* w = a.weights + row * a.weights_width;
    float* w_out = a.weights_out + row * a.weights_width;
    int* kept = a.kept + row * a.max_keep;
    const int all = NC * threads, at = rank * threads + tid;      // this thread among the row's
    // a CTA has a stretch [c0, c1) of the positions, a warp [w0, w1) of that
    const int n = g.skip ? 0 : g.ctx;
    const int per_warp = ((n + NC * warps - 1) / (NC * warps) + kSpan - 1) / kSpan * kSpan;
    const int c0 = min(n, rank * warps * per_warp), c1 = min(n, c0 + warps * per_warp);
    const int w0 = min(n, c0 + warp * per_warp), w1 = min(n, w0 + per_warp);
    // the four weights from p on (a lane's, of a span of 128)
    const auto four = [&](int p, float (&v)[4]) {
        if (CACHED) {
            const float4 x = *reinterpret_cast<const float4*>(s_w + (p - c0));
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = p + e < w1 ? w[p + e] : 0.f;
        }
    };
    bool skip = g.skip;
    if (CACHED && !skip && g.left < n)
        copy_weights(s_w, w + c0, c1 - c0);                // all on their way at once
    if (!skip && g.left < n) {                             // rows will move: every block must be there
        bool bad = false;
        const int blocks = (n + a.block_size - 1) / a.block_size;
        for (int i = tid; i < blocks; i += threads) {
            const int blk = a.block_table[(size_t)b * a.max_blocks + i];
            bad = bad || blk < 0 || blk >= a.num_blocks;
        }
        if (CACHED) {
            cp_async_commit();
            cp_async_wait<0>();
        }
        skip = __syncthreads_or(bad);
        if (skip && first && tid == 0) flag_status(a.status, LL_DEV_BAD_BLOCK);
    }
    if (first && tid == 0) a.new_lens[b] = skip ? g.ctx : g.left;
    if (skip || g.left == n) {
        const int m = skip ? 0 : n;
        for (int j = at; j < a.max_keep; j += all) kept[j] = j < m ? j : -1;
        if (w_out != w)
            for (int j = at; j < m; j += all) w_out[j] = w[j];
        return;
    }
    if (NC > 1) cluster_sync();                            // the first CTA's histograms are there, and zeros
    const int last = min(a.recent, g.left), front = min(a.sinks, g.left - last);
    const int rest = g.left - last - front, lo = front, hi = n - last;    // `rest` of lo .. hi - 1, fewer than there are
    const int p_lo = max(lo, w0), p_hi = min(hi, w1);      // this warp's part of those
    // the key of the last row that stays, digit by digit: `prefix` in the bits above `shift`, `need` rows of that prefix
    uint32_t prefix = 0;
    int need = rest;
    // whether this warp's weights between the first and last rows are neither negative (-0 too) nor NaN, as sums of
    // probabilities are: their keys are their bits with the top one set (16 sequences of 4096 to 32768 rows: 31 us, 42 without)
    bool plain = rest > 0;
    constexpr uint32_t kInfinity = 0x7f800000u;
    if (rest > 0) {
        constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = kShift[pass];
            const uint32_t above = pass == 0 ? 0u : 0xffffffffu << kShift[pass - 1 < 0 ? 0 : pass - 1];
            const uint32_t mask = pass == 2 ? 1023u : 2047u;
            // a lane adds up runs of one bin before it adds them to the histogram, and zeros
            int run_bin = -1, run_len = 0, zeros = 0;
            const auto count = [&](int bin) {
                if (bin != run_bin) {
                    if (run_len) atomicAdd(&s_hist[pass][run_bin], run_len);
                    run_bin = bin;
                    run_len = 0;
                }
                ++run_len;
            };
            for (int p0 = w0 + 4 * lane; p0 < w1; p0 += kSpan) {
                float v[4];
                four(p0, v);
                if (p0 >= p_lo && p0 + 4 <= p_hi && (pass == 0 || plain)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = __float_as_uint(v[e]), key = u | 0x80000000u;
                        if (pass > 0) {
                            if ((key & above) == prefix) count((int)((key >> shift) & mask));
                        } else if (u == 0u) {
                            ++zeros;
                        } else if (u <= kInfinity) {
                            atomicAdd(&s_hist[0][key >> shift], 1);
                        } else {
                            plain = false;
                            count((int)(weight_key(v[e]) >> shift));
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t key = weight_key(v[e]);
                        if (p0 + e < p_lo || p0 + e >= p_hi || (key & above) != prefix) continue;
                        if (pass == 0 && __float_as_uint(v[e]) > kInfinity) plain = false;
                        count((int)((key >> shift) & mask));
                    }
                }
            }
            if (pass == 0) {
                zeros = __reduce_add_sync(0xffffffffu, zeros);
                if (lane == 0 && zeros) atomicAdd(&s_hist[0][1024], zeros);
                plain = __all_sync(0xffffffffu, plain);
            }
            if (run_len) atomicAdd(&s_hist[pass][run_bin], run_len);
            // (a cluster's histograms meet in its first CTA, bin by bin where there is something, and that one picks)
            const int per = kBins / threads;
            int* bins = &s_hist[pass][kBins - (tid + 1) * per];        // this thread's, the highest last
            __syncthreads();
            if (NC > 1) {
                if (rank > 0)
                    for (int i = 0; i < per; ++i)
                        if (bins[i]) dsmem_add(&bins[i], 0, bins[i]);
                cluster_sync();
            }
            if (NC == 1 || rank == 0) {
                // from the top bin down, the bin in which the count reaches `need`
                int c[kBins / 256], mine = 0;
#pragma unroll
                for (int i = 0; i < kBins / 256; ++i) {
                    c[i] = i < per ? bins[per - 1 - i] : 0;
                    mine += c[i];
                }
                int run = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += y;
                }
                if (lane == 31) s_scan[warp] = run;
                __syncthreads();
                int total;
                int before = run - mine + before_in(s_scan, warps, warp, total);
#pragma unroll
                for (int i = 0; i < kBins / 256; ++i) {
                    if (before < need && before + c[i] >= need) {
                        const int bin = kBins - 1 - (tid * per + i);
                        if (NC == 1) {
                            s_pick[0] = bin;
                            s_pick[1] = need - before;
                        } else {
#pragma unroll
                            for (int r = 0; r < NC; ++r) {
                                dsmem_store(&s_pick[0], r, bin);
                                dsmem_store(&s_pick[1], r, need - before);
                            }
                        }
                    }
                    before += c[i];
                }
            }
            sync_all<NC>();
            prefix |= (uint32_t)s_pick[0] << shift;
            need = s_pick[1];                              // (written again behind the next pass's barriers)
        }
    }
    // The first and last rows and those with a larger key stay, and the first `need` with this one.
    const auto stays = [&](int p, float v, bool& tie) {
        const uint32_t key = weight_key(v);
        const bool middle = rest > 0 && p >= lo && p < hi;
        tie = middle && p < w1 && key == prefix;
        return p < w1 && (p < lo || p >= hi || (middle && key > prefix));
    };
    int gt = 0, eq = 0;
    for (int p0 = w0 + 4 * lane; p0 < w1; p0 += kSpan) {
        float v[4];
        four(p0, v);
        if (plain && p0 >= p_lo && p0 + 4 <= p_hi) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t key = __float_as_uint(v[e]) | 0x80000000u;
                gt += key > prefix ? 1 : 0;
                eq += key == prefix ? 1 : 0;
            }
            continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bool tie;
            gt += stays(p0 + e, v[e], tie) ? 1 : 0;
            eq += tie ? 1 : 0;
        }
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    int gt_all, eq_all;
    int gt_before = before_in(s_gt, warps, warp, gt_all), eq_before = before_in(s_eq, warps, warp, eq_all);
    if (NC > 1) {
        if (tid == 0) {
            s_total[0] = gt_all;
            s_total[1] = eq_all;
        }
        cluster_sync();                                    // (every CTA has read its weights, too)
        for (int r = 0; r < rank; ++r) {
            gt_before += dsmem_load(&s_total[0], r);
            eq_before += dsmem_load(&s_total[1], r);
        }
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int q0 = w0; q0 < w1; q0 += kSpan) {
        const int p0 = q0 + 4 * lane;
        float v[4];
        bool in[4], tie[4];
        int g_rank = gt_before, e_rank = eq_before;        // before this lane's four
        if (p0 < w1) four(p0, v);
        if (plain && q0 >= p_lo && q0 + kSpan <= p_hi) {   // (the same for the warp)
            uint32_t gts[4], some = 0;
            bool same = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t key = __float_as_uint(v[e]) | 0x80000000u;
                in[e] = key > prefix;
                same = same || key == prefix;
                gts[e] = __ballot_sync(0xffffffffu, in[e]);
                some |= gts[e];
            }
            if (!__any_sync(0xffffffffu, same)) {          // no ties
                if (some == 0u) continue;
                int j = gt_before + min(eq_before, need);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    j += __popc(gts[e] & below);
                    gt_before += __popc(gts[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!in[e]) continue;
                    kept[j] = p0 + e;
                    if (CACHED) w_out[j] = v[e];           // (w_out may be w: all of it has been read)
                    ++j;
                }
                continue;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            in[e] = stays(p0 + e, p0 < w1 ? v[e] : 0.f, tie[e]);
            const uint32_t gts = __ballot_sync(0xffffffffu, in[e]), eqs = __ballot_sync(0xffffffffu, tie[e]);
            g_rank += __popc(gts & below);
            e_rank += __popc(eqs & below);
            gt_before += __popc(gts);
            eq_before += __popc(eqs);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (in[e] || (tie[e] && e_rank < need)) {
                const int j = g_rank + min(e_rank, need);
                kept[j] = p0 + e;
                if (CACHED) w_out[j] = v[e];               // (w_out may be w: all of it has been read)
            }
            g_rank += in[e] ? 1 : 0;
            e_rank += tie[e] ? 1 : 0;
        }
    }
    for (int j = g.left + at; j < a.max_keep; j += all) kept[j] = -1;
    if (CACHED) {
        zero_weights(w_out, g.left, n, at, all);
        sync_all<NC>();                                    // (counts of this CTA's may still be read)
        return;
    }
    // the weights move as the rows do: a run is written when all of it has been read
    constexpr int E = 4;
    sync_all<NC>();
    for (int j0 = 0; j0 < g.left; j0 += E * all) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = j0 + e * all + at;
            v[e] = j < g.left ? w[kept[j]] : 0.f;
        }
        sync_all<NC>();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = j0 + e * all + at;
            if (j < g.left) w_out[j] = v[e];
        }
    }
    for (int j = g.left + at; j < n; j += all) w_out[j] = 0.f;
}

// Short rows of weights, at most 32 V: a warp per sequence and KV head, the keys in registers.  The last kept row's key is
// found bit by bit (32 counts at most; it ends when a count is what is needed), without a barrier.  2048 rows of 1150
// weights: 29 us, in a CTA each 48.
template <int V>
__global__ void __launch_bounds__(kWarpSelectThreads) evict_select_warp_kernel(const EvictArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kWarpSelectThreads / 32) + (threadIdx.x >> 5);
    if (row >= (long long)a.batch * a.n_kv_heads) return;
    const int b = (int)(row / a.n_kv_heads);
    const bool first = row == (long long)b * a.n_kv_heads;
    const Budget g = evict_budget(a, b, first && lane == 0);
    const float* w = a.weights + row * a.weights_width;
    float* w_out = a.weights_out + row * a.weights_width;
    int* kept = a.kept + row * a.max_keep;
    const int n = g.skip ? 0 : g.ctx;
    const int last = min(a.recent, g.left), front = min(a.sinks, g.left - last);
    const int lo = front, hi = n - last;
    bool skip = g.skip;
    // the keys; kStays for the first and last rows, above every weight's, 0 (as NaN) behind the row
    constexpr uint32_t kStays = 0xffffffffu;
    uint32_t key[V], minus[V / 32 + 1];                    // minus: which of this lane's weights are -0
#pragma unroll
    for (int i = 0; i < V / 32 + 1; ++i) minus[i] = 0u;
    if (!skip && g.left < n) {
#pragma unroll
        for (int i = 0; i < V; ++i) {                      // all on their way at once
            const int p = i * 32 + lane;
            key[i] = p >= lo && p < hi ? __float_as_uint(w[p]) : 0u;
        }
        bool bad = false;
        for (int i = lane; i < (n + a.block_size - 1) >> a.block_shift; i += 32) {
            const int blk = a.block_table[(size_t)b * a.max_blocks + i];
            bad = bad || blk < 0 || blk >= a.num_blocks;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int p = i * 32 + lane;
            minus[i / 32] |= (key[i] == 0x80000000u ? 1u : 0u) << (i % 32);
            key[i] = p >= n ? 0u : p < lo || p >= hi ? kStays : weight_key(__uint_as_float(key[i]));
        }
        skip = __any_sync(0xffffffffu, bad);
        if (skip && first && lane == 0) flag_status(a.status, LL_DEV_BAD_BLOCK);
    }
    if (first && lane == 0) a.new_lens[b] = skip ? g.ctx : g.left;
    if (skip || g.left == n) {
        const int m = skip ? 0 : n;
        for (int j = lane; j < a.max_keep; j += 32) kept[j] = j < m ? j : -1;
        if (w_out != w)
            for (int j = lane; j < m; j += 32) w_out[j] = w[j];
        return;
    }
    const auto at_least = [&](uint32_t t) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) c += key[i] >= t ? 1 : 0;
        return (int)__reduce_add_sync(0xffffffffu, c);
    };
    // rows above `top` stay, and the first `need` at it
    uint32_t top = 0;
    int need = 0;
    bool done = false;
    for (int bit = 31; bit >= 0 && !done; --bit) {
        const uint32_t t = top | 1u << bit;
        const int c = at_least(t);
        if (c >= g.left) top = t;
        if (c == g.left) {                                 // exactly those
            top = t - 1;
            done = true;
        }
    }
    if (!done) need = g.left - at_least(top + 1);          // (top < kStays: that count is at most front + last, and they are in)
    int gt_before = 0, eq_before = 0;
    const uint32_t below = (1u << lane) - 1u;
    constexpr int AHEAD = 8;                               // rows of 32 whose weights are read again before they are due
    float again[AHEAD];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i * 32 >= n) break;
        if (i % AHEAD == 0) {
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const int p = (i + e) * 32 + lane;
                if (i + e < V && p < n && (key[i + e < V ? i + e : 0] == 0u || key[i + e < V ? i + e : 0] == kStays)) again[e] = w[p];
            }
            __syncwarp();
        }
        const int p = i * 32 + lane;
        const bool in = p < n && key[i] > top, tie = p < n && key[i] == top;
        const uint32_t gts = __ballot_sync(0xffffffffu, in), eqs = __ballot_sync(0xffffffffu, tie);
        const int g_rank = gt_before + __popc(gts & below), e_rank = eq_before + __popc(eqs & below);
        // a weight is what its key says, but for the first and last rows and NaN, which are read again (nothing behind row
        // i * 32 has been written: w_out may be w)
        float v = __uint_as_float(key[i] & 0x80000000u ? key[i] ^ 0x80000000u : ~key[i]);
        if ((minus[i / 32] >> (i % 32)) & 1u) v = -0.f;
        if (key[i] == 0u || key[i] == kStays) v = again[i % AHEAD];
        if (in || (tie && e_rank < need)) {
            const int j = g_rank + min(e_rank, need);
            kept[j] = p;
            w_out[j] = v;
        }
        gt_before += __popc(gts);
        eq_before += __popc(eqs);
        if (i % AHEAD == AHEAD - 1) __syncwarp();
    }
    __syncwarp();
    for (int j = g.left + lane; j < a.max_keep; j += 32) kept[j] = -1;
    for (int j = g.left + lane; j < n; j += 32) w_out[j] = 0.f;
}

// Moves the rows of one (tensor, slice of its rows' bytes, KV head, sequence).  T: the piece a thread moves at a time.
template <typename T, int ROWS, int THREADS>
LL_DEVINL void move_rows(const EvictArgs& a, char* data, int row_bytes, int slice0, int pieces, int hk, int b, int2* s_place) {
    constexpr int PER = ROWS / THREADS;
    const int* kept = a.kept + ((size_t)b * a.n_kv_heads + hk) * a.max_keep;
    const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
    const int run = THREADS * kMovePieces / pieces;          // rows between two barriers
    const int u = threadIdx.x % pieces, r0 = threadIdx.x / pieces, stride = THREADS / pieces;
    int src[PER], from[PER], to[PER];                             // rows of the next lookup, and the blocks they are in
    const auto look = [&](int base) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int j = base + e * THREADS + threadIdx.x;
            src[e] = j < a.max_keep ? kept[j] : -1;
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int j = base + e * THREADS + threadIdx.x;
            from[e] = src[e] > j ? table[src[e] >> a.block_shift] : 0;
            to[e] = src[e] > j ? table[j >> a.block_shift] : 0;
        }
    };
    look(0);
    for (int base = 0; base < a.max_keep; base += ROWS) {
        __syncthreads();                                          // (the places before have been used)
        bool any = false;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = e * THREADS + threadIdx.x, j = base + i;
            any = any || src[e] >= 0;
            s_place[i] = src[e] <= j ? make_int2(-1, -1)
                                     : make_int2(((from[e] * a.n_kv_heads + hk) << a.block_shift) + (src[e] & (a.block_size - 1)),
                                                 ((to[e] * a.n_kv_heads + hk) << a.block_shift) + (j & (a.block_size - 1)));
        }
        if (!__syncthreads_or(any)) return;                       // behind the last kept row
        if (base + ROWS < a.max_keep) look(base + ROWS);
        for (int i0 = 0; i0 < ROWS; i0 += run) {
            T v[kMovePieces];
#pragma unroll
            for (int e = 0; e < kMovePieces; ++e) {
                const int i = i0 + e * stride + r0;
                if (i < ROWS && s_place[i].x >= 0)
                    v[e] = *reinterpret_cast<const T*>(data + (size_t)s_place[i].x * row_bytes + slice0 + u * (int)sizeof(T));
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kMovePieces; ++e) {
                const int i = i0 + e * stride + r0;
                if (i < ROWS && s_place[i].x >= 0)
                    *reinterpret_cast<T*>(data + (size_t)s_place[i].y * row_bytes + slice0 + u * (int)sizeof(T)) = v[e];
            }
        }
    }
}

// ROWS: whose places a CTA looks up at a time, while the ones before them move.  Where there are many CTAs few (their
// registers are another CTA's: 64 sequences to 1024 rows of 32 heads 313 us with 512, 350 with 2048), where all run at once
// more, and with the SM to itself still more and twice the threads (8192 of 65536 rows of 128 bytes, 8 heads: 20 us with
// 4096, 24 with 2048 and 256 threads).
template <int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) evict_move_kernel(const EvictArgs a) {
    __shared__ int2 s_place[ROWS];
    pdl_wait();
    pdl_trigger();
    int t = 0, slice = blockIdx.x;
    while (slice >= a.slices[t]) slice -= a.slices[t++];
    const int bytes = a.row_bytes[t] / a.slices[t];
    char* data = static_cast<char*>(a.data[t]);
    if (a.wide[t]) move_rows<uint4, ROWS, THREADS>(a, data, a.row_bytes[t], slice * bytes, bytes / 16, blockIdx.y, blockIdx.z, s_place);
    else move_rows<uint32_t, ROWS, THREADS>(a, data, a.row_bytes[t], slice * bytes, bytes / 4, blockIdx.y, blockIdx.z, s_place);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& args, cudaStream_t stream) {
    EvictArgs a = args;
    a.block_shift = 0;
    while ((1 << a.block_shift) < a.block_size) ++a.block_shift;          // (a power of two)
    const long long rows = (long long)a.batch * a.n_kv_heads;
    const long long most = (long long)a.max_blocks * a.block_size;
    const int sms = std::max(1, device_sm_count());
    trace_before("evict_select", stream);
    // Few rows of weights are spread over clusters, as many CTAs as run at once, one on an SM (65536 positions of 8 heads: 21
    // us with eight CTAs each, 101 with one; of 32 heads 27 with four, 54 with eight in two turns; clusters of eight fill about
    // half of the SMs at once, 16 of them take 38).  Weights that fit lie in shared memory.
    const int nc = most < 4096 ? 1 : rows * 16 <= sms ? 8 : rows * 4 <= sms ? 4 : rows * 2 <= sms ? 2 : 1;
    const int threads = most >= 4096 && rows * nc <= sms ? 1024 : 512;
    const int warps = nc * threads / 32;
    const long long stretch = (most + warps - 1) / warps + kSpan - 1;    // of a warp, in whole spans
    const size_t smem = (size_t)(stretch / kSpan * kSpan) * (threads / 32) * sizeof(float);
    const bool cached = smem <= kSelectSmem;
    const auto select = [&](auto c, auto in_smem) {
        const auto kernel = evict_select_kernel<c.value, in_smem.value>;
        if (in_smem.value) {
            const cudaError_t e = ensure_func_attr((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem,
                                                   "cudaFuncSetAttribute(evict_select_kernel)");
            if (e != cudaSuccess) return e;
        }
        return launch_pdl(kernel, dim3(a.n_kv_heads * c.value, a.batch), dim3(threads), in_smem.value ? smem : 0, stream, c.value, a);
    };
    const auto for_cluster = [&](auto in_smem) {
        switch (nc) {
            case 8: return select(std::integral_constant<int, 8>{}, in_smem);
            case 4: return select(std::integral_constant<int, 4>{}, in_smem);
            case 2: return select(std::integral_constant<int, 2>{}, in_smem);
            default: return select(std::integral_constant<int, 1>{}, in_smem);
        }
    };
    const auto per_warp = [&](auto v) {
        constexpr int kRows = kWarpSelectThreads / 32;
        return launch_pdl(evict_select_warp_kernel<v.value>, dim3((unsigned)((rows + kRows - 1) / kRows)), dim3(kWarpSelectThreads), 0,
                          stream, 1, a);
    };
    cudaError_t e = most <= 1024   ? per_warp(std::integral_constant<int, 32>{})
                    : most <= 1536 ? per_warp(std::integral_constant<int, 48>{})
                    : most <= 2048 ? per_warp(std::integral_constant<int, 64>{})
                    : cached       ? for_cluster(std::true_type{})
                                   : for_cluster(std::false_type{});
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "evict_select launch");
    // Whole rows where that gives every SM a few CTAs, else slices of 64 bytes, and where those leave half of the SMs idle
    // smaller ones, down to a piece.  (8192 of 65536 rows of 128 bytes, K and V of 8 heads: 8 sequences 61 us with 64 bytes,
    // 115 with 16; one 27 and 20.)
    int slices = 0;
    for (int t = 0; t < a.n_tensors; ++t) {
        const int piece = a.wide[t] ? 16 : 4;
        a.slices[t] = 1;
        // pieces of a slice divide a CTA's threads: slices halve the row while that leaves whole pieces
        int n = a.row_bytes[t] / piece;
        const auto more = [&] {
            const long long ctas = rows * a.n_tensors * a.slices[t];
            return n % 2 == 0 && (n * piece >= 128 ? ctas < 4 * sms : 2 * ctas < sms);
        };
        while (n > kMoveThreads || kMoveThreads % n != 0 || more()) {
            int f = 2;
            while (n % f != 0) ++f;                        // the smallest factor
            n /= f;
            a.slices[t] *= f;
        }
        slices += a.slices[t];
    }
    trace_before("evict_move", stream);
    const dim3 grid(slices, a.n_kv_heads, a.batch);
    const long long ctas = rows * slices;
    e = ctas <= sms       ? launch_pdl(evict_move_kernel<4096, 2 * kMoveThreads>, grid, dim3(2 * kMoveThreads), 0, stream, 1, a)
        : ctas <= 2 * sms ? launch_pdl(evict_move_kernel<2048, kMoveThreads>, grid, dim3(kMoveThreads), 0, stream, 1, a)
                          : launch_pdl(evict_move_kernel<512, kMoveThreads>, grid, dim3(kMoveThreads), 0, stream, 1, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "evict_move launch");
}

}  // namespace ll
