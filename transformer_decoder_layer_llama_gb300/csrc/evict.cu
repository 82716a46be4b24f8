// Eviction from a paged cache by accumulated attention weight.  Of a sequence's n cached rows each KV head keeps the
// last `recent`, the first `sinks`, and of those between the ones of largest weight (NaN below every number, -0 as 0, ties
// to the lowest position), m rows in all.  They move, in order, to positions 0 .. m - 1 of the same blocks.
//
// Two kernels.  The choice: a CTA (a cluster where there are few rows of weights) per sequence and KV head finds the
// weight of the last kept row digit by digit in histograms (11, 11 and 10 bits of an order-preserving integer), then
// every warp counts, and after one exchange of counts writes, its own stretch of positions: no sort, five passes over
// weights that stay in L2.  The move: kept[j] >= j ascending, so a row's place is never the source of a later one.  A CTA
// goes through its rows in order and writes a run of them when all its threads have read theirs; heads, tensors
// and slices of a row's bytes do not meet, so they are what is spread over CTAs.  Bound by the bytes of the rows.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 1024;        // rows whose places a CTA looks up at a time
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

template <int NC>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
    __shared__ int s_hist[kBins], s_scan[32], s_gt[33], s_eq[33], s_total[2], s_pick[2];
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.x / NC, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int threads = blockDim.x, warps = threads >> 5;
    const int rank = NC == 1 ? 0 : (int)cluster_rank();
    const bool first = hk == 0 && rank == 0;
    const Budget g = evict_budget(a, b, first && tid == 0);
    const size_t row = (size_t)b * a.n_kv_heads + hk;
    const float* w = a.weights + row * a.weights_width;
    float* w_out = a.weights_out + row * a.weights_width;
    int* kept = a.kept + row * a.max_keep;
    bool skip = g.skip;
    if (!skip && g.left < g.ctx) {                         // rows will move: every block must be there
        bool bad = false;
        const int blocks = (g.ctx + a.block_size - 1) / a.block_size;
        for (int i = tid; i < blocks; i += threads) {
            const int blk = a.block_table[(size_t)b * a.max_blocks + i];
            bad = bad || blk < 0 || blk >= a.num_blocks;
        }
        skip = __syncthreads_or(bad);
        if (skip && first && tid == 0) flag_status(a.status, LL_DEV_BAD_BLOCK);
    }
    if (first && tid == 0) a.new_lens[b] = skip ? g.ctx : g.left;
    const int all = NC * threads, at = rank * threads + tid;      // this thread among the row's
    if (skip || g.left == g.ctx) {
        const int n = skip ? 0 : g.ctx;
        for (int j = at; j < a.max_keep; j += all) kept[j] = j < n ? j : -1;
        if (w_out != w)
            for (int j = at; j < n; j += all) w_out[j] = w[j];
        return;
    }
    const int n = g.ctx, last = min(a.recent, g.left), front = min(a.sinks, g.left - last);
    const int rest = g.left - last - front, lo = front, hi = n - last;    // `rest` of lo .. hi - 1, fewer than there are
    // the key of the last row that stays, digit by digit: `prefix` in the bits above `shift`, `need` rows of that prefix
    uint32_t prefix = 0;
    int need = rest;
    if (rest > 0) {
        constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = kShift[pass];
            const uint32_t above = pass == 0 ? 0u : 0xffffffffu << kShift[pass - 1 < 0 ? 0 : pass - 1];
            const uint32_t mask = pass == 2 ? 1023u : 2047u;
            for (int i = tid; i < kBins; i += threads) s_hist[i] = 0;
            __syncthreads();
            for (int p0 = lo + rank * threads + warp * 32; p0 < hi; p0 += all) {
                const int p = p0 + lane;
                const uint32_t key = p < hi ? weight_key(w[p]) : 0u;
                const bool in = p < hi && (key & above) == prefix;
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (who == 0) continue;
                const int bin = (int)((key >> shift) & mask);
                const int lead = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
                if (__all_sync(0xffffffffu, !in || bin == lead)) {        // one bin (zeros, say): one addition
                    if (lane == 0) atomicAdd(&s_hist[lead], __popc(who));
                } else if (in) {
                    atomicAdd(&s_hist[bin], 1);
                }
            }
            sync_all<NC>();
            // from the top bin down, the bin in which the count reaches `need`: a thread per kBins / threads bins
            const int per = kBins / threads;
            int mine = 0;
            for (int i = 0; i < per; ++i) {
                const int bin = kBins - 1 - (tid * per + i);
                int c = 0;
                if (NC == 1) c = s_hist[bin];
                else
                    for (int r = 0; r < NC; ++r) c += dsmem_load(&s_hist[bin], r);
                mine += c;
            }
            int run = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += y;
            }
            if (lane == 31) s_scan[warp] = run;
            __syncthreads();
            int before = run - mine;
            for (int i = 0; i < warp; ++i) before += s_scan[i];
            if (before < need && before + mine >= need) {
                for (int i = 0; i < per; ++i) {
                    const int bin = kBins - 1 - (tid * per + i);
                    int c = 0;
                    if (NC == 1) c = s_hist[bin];
                    else
                        for (int r = 0; r < NC; ++r) c += dsmem_load(&s_hist[bin], r);
                    if (before + c >= need) {
                        s_pick[0] = bin;
                        s_pick[1] = need - before;
                        break;
                    }
                    before += c;
                }
            }
            sync_all<NC>();                                // (the histograms have been read)
            prefix |= (uint32_t)s_pick[0] << shift;
            need = s_pick[1];
            __syncthreads();
        }
    }
    // rows with a larger key stay, and the first `need` with this one.  A warp has a stretch of positions.
    const int per_warp = ((hi - lo + NC * warps - 1) / (NC * warps) + 31) / 32 * 32;
    const int w0 = min(hi, lo + (rank * warps + warp) * per_warp), w1 = min(hi, w0 + per_warp);
    int gt = 0, eq = 0;
    if (rest > 0)
        for (int p0 = w0; p0 < w1; p0 += 32) {
            const int p = p0 + lane;
            const uint32_t key = p < w1 ? weight_key(w[p]) : 0u;
            gt += __popc(__ballot_sync(0xffffffffu, p < w1 && key > prefix));
            eq += __popc(__ballot_sync(0xffffffffu, p < w1 && key == prefix));
        }
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    if (NC > 1 && tid == 0) {
        s_total[0] = s_total[1] = 0;
        for (int i = 0; i < warps; ++i) {
            s_total[0] += s_gt[i];
            s_total[1] += s_eq[i];
        }
    }
    if (NC > 1) cluster_sync();
    int gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        gt_before += dsmem_load(&s_total[0], r);
        eq_before += dsmem_load(&s_total[1], r);
    }
    for (int i = 0; i < warp; ++i) {
        gt_before += s_gt[i];
        eq_before += s_eq[i];
    }
    for (int j = at; j < front; j += all) kept[j] = j;
    for (int j = at; j < last; j += all) kept[g.left - last + j] = n - last + j;
    for (int j = g.left + at; j < a.max_keep; j += all) kept[j] = -1;
    if (rest > 0)
        for (int p0 = w0; p0 < w1; p0 += 32) {
            const int p = p0 + lane;
            const uint32_t key = p < w1 ? weight_key(w[p]) : 0u;
            const bool is_gt = p < w1 && key > prefix, is_eq = p < w1 && key == prefix;
            const uint32_t gts = __ballot_sync(0xffffffffu, is_gt), eqs = __ballot_sync(0xffffffffu, is_eq);
            const uint32_t below = (1u << lane) - 1u;
            const int g_rank = gt_before + __popc(gts & below), e_rank = eq_before + __popc(eqs & below);
            if (is_gt || (is_eq && e_rank < need)) kept[front + g_rank + min(e_rank, need)] = p;
            gt_before += __popc(gts);
            eq_before += __popc(eqs);
        }
    // the weights move as the rows do (w_out may be w): a run is written when all of it has been read
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

// Moves the rows of one (tensor, slice of its rows' bytes, KV head, sequence).  T: the piece a thread moves at a time.
template <typename T>
LL_DEVINL void move_rows(const EvictArgs& a, char* data, int row_bytes, int slice0, int pieces, int hk, int b, int2* s_place) {
    const int* kept = a.kept + ((size_t)b * a.n_kv_heads + hk) * a.max_keep;
    const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
    const int run = kMoveThreads * kMovePieces / pieces;          // rows between two barriers
    const int u = threadIdx.x % pieces, r0 = threadIdx.x / pieces, stride = kMoveThreads / pieces;
    const bool worker = r0 < stride;                              // (pieces divides the threads: always)
    for (int base = 0; base < a.max_keep; base += kMoveRows) {
        __syncthreads();                                          // (the places before have been used)
        bool any = false;
        for (int i = threadIdx.x; i < kMoveRows; i += kMoveThreads) {
            const int j = base + i, src = j < a.max_keep ? kept[j] : -1;
            int2 place = make_int2(-1, -1);
            if (src > j) {
                place.x = (table[src / a.block_size] * a.n_kv_heads + hk) * a.block_size + src % a.block_size;
                place.y = (table[j / a.block_size] * a.n_kv_heads + hk) * a.block_size + j % a.block_size;
            }
            any = any || src >= 0;
            s_place[i] = place;
        }
        if (!__syncthreads_or(any)) return;                       // behind the last kept row
        for (int i0 = 0; i0 < kMoveRows; i0 += run) {
            T v[kMovePieces];
#pragma unroll
            for (int e = 0; e < kMovePieces; ++e) {
                const int i = i0 + e * stride + r0;
                if (worker && i < kMoveRows && s_place[i].x >= 0)
                    v[e] = *reinterpret_cast<const T*>(data + (size_t)s_place[i].x * row_bytes + slice0 + u * (int)sizeof(T));
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kMovePieces; ++e) {
                const int i = i0 + e * stride + r0;
                if (worker && i < kMoveRows && s_place[i].x >= 0)
                    *reinterpret_cast<T*>(data + (size_t)s_place[i].y * row_bytes + slice0 + u * (int)sizeof(T)) = v[e];
            }
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    __shared__ int2 s_place[kMoveRows];
    pdl_wait();
    pdl_trigger();
    int t = 0, slice = blockIdx.x;
    while (slice >= a.slices[t]) slice -= a.slices[t++];
    const int bytes = a.row_bytes[t] / a.slices[t];
    char* data = static_cast<char*>(a.data[t]);
    if (a.wide[t]) move_rows<uint4>(a, data, a.row_bytes[t], slice * bytes, bytes / 16, blockIdx.y, blockIdx.z, s_place);
    else move_rows<uint32_t>(a, data, a.row_bytes[t], slice * bytes, bytes / 4, blockIdx.y, blockIdx.z, s_place);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& args, cudaStream_t stream) {
    EvictArgs a = args;
    const long long rows = (long long)a.batch * a.n_kv_heads;
    const long long most = (long long)a.max_blocks * a.block_size;
    const int sms = std::max(1, device_sm_count());
    trace_before("evict_select", stream);
    // a cluster of eight CTAs per row of weights where they all fit at once and the rows can be long
    cudaError_t e;
    if (rows * 8 <= 2 * sms && most >= 8192) {
        e = launch_pdl(evict_select_kernel<8>, dim3(a.n_kv_heads * 8, a.batch), dim3(kSelectThreads), 0, stream, 8, a);
    } else {
        const int threads = most <= 2048 ? 256 : kSelectThreads;
        e = launch_pdl(evict_select_kernel<1>, dim3(a.n_kv_heads, a.batch), dim3(threads), 0, stream, 1, a);
    }
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "evict_select launch");
    // whole rows where that gives every SM a few CTAs, else slices of at least 16 bytes
    int slices = 0;
    for (int t = 0; t < a.n_tensors; ++t) {
        const int piece = a.wide[t] ? 16 : 4;
        a.slices[t] = 1;
        // pieces of a slice divide a CTA's threads: slices halve the row while that leaves whole pieces
        int n = a.row_bytes[t] / piece;
        while (n > kMoveThreads || kMoveThreads % n != 0 || (rows * a.n_tensors * a.slices[t] < 4 * sms && n % 2 == 0)) {
            int f = 2;
            while (n % f != 0) ++f;                        // the smallest factor
            n /= f;
            a.slices[t] *= f;
        }
        slices += a.slices[t];
    }
    trace_before("evict_move", stream);
    e = launch_pdl(evict_move_kernel, dim3(slices, a.n_kv_heads, a.batch), dim3(kMoveThreads), 0, stream, 1, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "evict_move launch");
}

}  // namespace ll
