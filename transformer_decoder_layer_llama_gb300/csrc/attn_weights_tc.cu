// Attention weights of a ragged batch of query rows over a paged BF16 cache, on the tensor cores (tcgen05, TMEM, TMA):
//   weights[b][hk][p] += sum over rows i of sequence b and heads h of hk of P_ih(p),  P_ih = softmax_p(scale q_ih k_p), p <= pos(i).
//
// A column sum of P needs every row's normaliser first, and the scores of all pairs are too many to keep (4 bytes a
// pair), so they are computed twice:
//   ROWS  128 query rows (tokens x heads of a KV head) in the lanes, keys in the columns: a thread has a row and runs over
//         its scores with a running maximum and sum.  Long rows are split into `pieces`, which a small kernel joins, or
//         COLS itself where a sequence has few rows.
//   COLS  128 keys in the lanes, query rows in the columns: a thread has a key, adds 2^(score - lse of the column) and at
//         the end adds its sum to the weight.  One thread per weight: no atomics, the same bits every time.
// Both are one persistent kernel.  Two tiles of 128 rows (A) stay in shared memory while tiles of 256 rows (B) stream past
// them; each meets both, which halves the traffic from L2 per score, and an MMA of M 128 N 256 takes 160 clocks where two of
// N 128 take 200 to 300 (operands in shared memory).  A tile's scores fill half of TMEM: while its four warps take their
// exponentials, the other tile's product runs.  A warp looks up the items ahead of the others, so that the
// next item's tiles load while the last one's scores are summed.  Every wait is bounded.
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "vec16.cuh"

namespace ll {

namespace {

constexpr int kTile = 128;               // rows of an A tile
constexpr int kWide = 256;               // rows of a B tile, and of a pair of A tiles
constexpr int kObsThreads = 352;         // TMA, MMA, four warps for each A tile's scores, items
constexpr int kObsItemWarp = 10;
constexpr float kLog2eObs = 1.4426950408889634f;
constexpr int kObsPieceTiles = 2;        // at least, of a piece of a row (the rows are fetched for each)
constexpr int kObsLoad = 64;             // columns of one load from TMEM (8192 rows of 64 heads over 8: rows 461 us, keys 538; 32: 584, 620)
constexpr int kObsItems = 4;             // looked up ahead
constexpr int kObsMostPieces = 16;       // of a row, where sequences have more rows than two A tiles

// FEW: no sequence has more rows than two A tiles.  They then stay: in ROWS beside the keys of a CTA's whole share, in COLS
// as the B tile that all of its keys meet.
template <int D, bool FEW>
struct ObsLayout {
    static constexpr uint32_t A_TILE = kTile * D * 2;        // [D / 64][128 rows][128 B], 128-byte swizzle
    static constexpr uint32_t B_TILE = kWide * D * 2;        // [D / 64][256 rows][128 B]
    static constexpr int A_BUFS = FEW ? 2 : 1;               // of two tiles
    static constexpr int STAGES = FEW ? 1 : 2;
    static constexpr uint32_t OFF_B = A_BUFS * 2 * A_TILE;
    static constexpr uint32_t TOTAL = OFF_B + STAGES * B_TILE;
};

// What a sequence brings: its first query row, their number, the context (0 rows: nothing to do).
struct ObsSeq {
    int row0, n, ctx;
};

LL_DEVINL ObsSeq obs_sequence(const ObserveArgs& a, int b, bool flag) {
    ObsSeq s;
    s.row0 = a.cu_new[b];
    const long long end = (long long)a.cu_new[b + 1];
    s.ctx = a.context_lens[b];
    s.n = (int)max(-1ll, min(end - s.row0, (long long)a.max_new + 1));
    if (s.row0 < 0 || s.n < 0 || s.n > a.max_new || end > a.tokens || s.ctx < s.n ||
        (long long)s.ctx > (long long)a.max_blocks * a.block_size) {
        if (flag) flag_status(a.status, LL_DEV_BAD_POSITION);
        s.n = 0;
    }
    return s;
}

// An item of a CTA: pairs of A tiles, and for each the B tiles first(pair) .. last - 1.
struct ObsItem {
    int row0, n, ctx, b, hk;
    int pair, pair_step, pairs;          // A tiles 2 pair and 2 pair + 1, pair += pair_step while below pairs
    int piece, j0, j1;                   // ROWS: key tiles of this piece
    int pieces;                          // FEW: of these rows
    int kind;                            // kObsEnd, kObsWork, or (not handed on) kObsNone, kObsEmpty
};
constexpr int kObsEnd = 0, kObsWork = 1, kObsNone = 2, kObsEmpty = 3;

template <bool ROWS>
struct ObsSteps {
    int first0, Tb, last_;               // COLS: positions before the call's first row, its tokens per B tile
    LL_DEVINL ObsSteps(const ObsItem& w, int G) {
        Tb = kWide / G;
        first0 = ROWS ? w.j0 : w.ctx - w.n;
        last_ = ROWS ? w.j1 : (w.n + Tb - 1) / Tb;
    }
    LL_DEVINL int first(int pair) const {
        if (ROWS) return first0;
        const int behind = kWide * pair - first0;            // tokens of the call before the pair's first key
        return behind <= 0 ? 0 : behind / Tb;
    }
    LL_DEVINL int last() const { return last_; }
};

template <bool ROWS>
LL_DEVINL ObsItem obs_item(const ObserveArgs& a, long long idx, int G) {
    ObsItem w;
    w.kind = kObsNone;
    w.hk = (int)(idx % a.n_kv_heads);
    idx /= a.n_kv_heads;
    w.b = (int)(idx % a.batch);
    const int sub = (int)(idx / a.batch);
    const ObsSeq s = obs_sequence(a, w.b, ROWS && w.hk == 0 && sub == 0);
    w.row0 = s.row0;
    w.n = s.n;
    w.ctx = s.ctx;
    w.piece = w.j0 = w.j1 = 0;
    if (s.n <= 0) return w;
    if (ROWS) {
        const int Tq = kTile / G;
        w.piece = sub % a.pieces;
        const int most = (a.max_new + 2 * Tq - 1) / (2 * Tq);
        w.pair = most - 1 - sub / a.pieces;                  // the pairs with the most keys first
        w.pairs = w.pair + 1;
        w.pair_step = 1;
        if (w.pair * 2ll * Tq >= s.n) return w;
        const int end = (int)min((long long)s.n, (w.pair + 1) * 2ll * Tq);     // tokens of the pair end here
        const int tiles = (s.ctx - s.n + end - 1) / kWide + 1;
        const int len = max(kObsPieceTiles, (tiles + a.pieces - 1) / a.pieces);
        w.j0 = min(tiles, w.piece * len);
        w.j1 = min(tiles, w.j0 + len);
        w.kind = w.j0 < w.j1 ? kObsWork : kObsEmpty;
    } else {
        w.pair = sub;
        w.pair_step = a.key_ctas;
        w.pairs = (s.ctx + kWide - 1) / kWide;
        w.kind = w.pair < w.pairs ? kObsWork : kObsNone;
    }
    return w;
}

// FEW: the key tiles of all sequences and heads, and how many of them each CTA has (so many that no head's are in more than
// a.pieces parts).  A warp.
struct ObsShare {
    long long total, each;
};

LL_DEVINL ObsShare obs_share(const ObserveArgs& a, bool flag) {
    long long sum = 0;
    int most = 0;
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) {
        const ObsSeq s = obs_sequence(a, b, flag);
        const int tiles = s.n > 0 ? (s.ctx + kWide - 1) / kWide : 0;
        sum += tiles;
        most = max(most, tiles);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = __reduce_max_sync(0xffffffffu, most);
    ObsShare sh;
    sh.total = sum * a.n_kv_heads;
    sh.each = max(max(1ll, (sh.total + gridDim.x - 1) / gridDim.x), (long long)((most + a.pieces - 2) / (a.pieces - 1)));
    return sh;
}

// The sum of x over the lanes before this one; adds that of all to `total`.
LL_DEVINL long long scan_before(long long x, long long& total) {
    const int lane = threadIdx.x & 31;
    long long run = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    total += __shfl_sync(0xffffffffu, run, 31);
    return run - x;
}

// Barrier of the four warps of an A tile, with an OR of `pred` for all its threads.
LL_DEVINL bool group_bar_any(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n"
        " barrier.cta.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)pred)
        : "memory");
    return r != 0;
}

LL_DEVINL void tma_load_3d(void* smem_dst, const void* tmap, int32_t c0, int32_t c1, int32_t c2, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

LL_DEVINL float max3(float a, float b, float c) {          // NaN if there is one
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

LL_DEVINL void add_exp2(float2 x, float2& sum) { sum = add2(sum, make_float2(ex2_approx(x.x), ex2_approx(x.y))); }

// tmQ: boxes of 128 / G tokens (ROWS: A tiles) or 256 / G (COLS: B tiles).
template <int D, bool ROWS, bool FEW>
__global__ void __launch_bounds__(kObsThreads, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const ObserveArgs a,
                        long long items) {
    using L = ObsLayout<D, FEW && !ROWS>;
    constexpr int STAGES = L::STAGES, ABUFS = L::A_BUFS, LOAD = kObsLoad;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t a_full[2], a_empty[2], b_full[2], b_empty[2], s_full[2], s_empty[2], i_full[kObsItems], i_empty[kObsItems], drain;
    __shared__ __align__(16) float s_lse[2][2][kWide];       // COLS: [tile][step parity][column]
    __shared__ ObsItem s_item[kObsItems];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.n_heads / a.n_kv_heads, Tq = (ROWS ? kTile : kWide) / G;      // query tokens per tile
    int32_t* status = a.status;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&a_full[i], 1);
            mbar_init(&a_empty[i], 1);
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 128);
        }
        for (int i = 0; i < kObsItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 10);                      // TMA, MMA, eight warps
        }
        mbar_init(&drain, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (!ROWS) {                                             // columns behind a tile's last row: zeros, for finite scores
        const int used = Tq * G, rows = kWide - used;
        for (int i = threadIdx.x; i < STAGES * (D / 64) * rows * 8; i += kObsThreads) {
            const int c = i & 7, r = used + (i >> 3) % rows, half = (i >> 3) / rows;     // half: of a stage
            *reinterpret_cast<uint4*>(smem + L::OFF_B + half * (kWide * 128) + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_s, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    pdl_wait();
    pdl_trigger();

    // The k-th item of this CTA for a role's warp or thread, and its return.
    const auto take = [&](int k, ObsItem& w) {
        if (!mbar_wait_bounded(&i_full[k % kObsItems], (uint32_t)(k / kObsItems) & 1u, &abort_s, status)) return false;
        w = s_item[k % kObsItems];
        return w.kind == kObsWork;
    };

    if (warp == kObsItemWarp) {
        // ---------------------------------------------------- items
        int k = 0;
        bool ok = true;
        // hands an item on, from lane l
        const auto hand_on = [&](const ObsItem& w, int l) {
            const int slot = k % kObsItems;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&i_empty[slot], ((uint32_t)(k / kObsItems) & 1u) ^ 1u, &abort_s, status));
            if (ok && lane == l) {
                s_item[slot] = w;
                mbar_arrive(&i_full[slot]);                  // (releases the item)
            }
            __syncwarp();
            ++k;
        };
        if constexpr (FEW) {
            // every CTA has an equal share of all sequences' and heads' key tiles, one after another (32 rows of 8 contexts to
            // 16384: 52 + 53 us; 56 + 63 with items of equal parts of a context, whose rows come anew for each; one row of
            // 16 contexts to 32768: 128 + 121, 185 + 145)
            const ObsShare sh = obs_share(a, ROWS && blockIdx.x == 0);
            const long long g0 = sh.each * blockIdx.x, g1 = min(sh.total, g0 + sh.each);
            long long before = 0;                            // tiles of the sequences before
            for (int b0 = 0; ok && b0 < a.batch && before < g1; b0 += 32) {
                const ObsSeq s = b0 + lane < a.batch ? obs_sequence(a, b0 + lane, false) : ObsSeq{0, 0, 0};
                const int tiles = s.n > 0 ? (s.ctx + kWide - 1) / kWide : 0;
                const long long all = (long long)tiles * a.n_kv_heads, first = before, start = first + scan_before(all, before);
                uint32_t todo = __ballot_sync(0xffffffffu, all > 0 && start < g1 && start + all > g0);
                while (todo && ok) {
                    const int l = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const long long from = __shfl_sync(0xffffffffu, start, l);
                    const int t = __shfl_sync(0xffffffffu, tiles, l);
                    for (int hk = (int)(max(0ll, g0 - from) / t); ok && hk < a.n_kv_heads && from + (long long)hk * t < g1; ++hk) {
                        const long long own = from + (long long)hk * t;          // this head's first tile
                        ObsItem w;
                        w.row0 = s.row0;
                        w.n = s.n;
                        w.ctx = s.ctx;
                        w.b = b0 + l;
                        w.hk = hk;
                        w.j0 = (int)(max(g0, own) - own);
                        w.j1 = (int)(min(g1, own + t) - own);
                        w.pair = ROWS ? 0 : w.j0;
                        w.pairs = ROWS ? 1 : w.j1;
                        w.pair_step = 1;
                        w.piece = (int)(blockIdx.x - own / sh.each);
                        w.pieces = (int)((own + t - 1) / sh.each - own / sh.each) + 1;
                        w.kind = kObsWork;
                        hand_on(w, l);
                    }
                }
            }
            ObsItem end;
            end.kind = kObsEnd;
            if (ok) hand_on(end, 0);
        } else {
            // 32 at a time are looked up, those with work handed on
            for (long long round = 0; ok; round += 32) {
                // every other round reversed: a CTA with one of the longest items has one of the shortest next
                const long long turn = round + lane, idx = turn * gridDim.x + (turn & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                ObsItem w;
                w.kind = turn * gridDim.x < items ? kObsNone : kObsEnd;
                if (idx < items) w = obs_item<ROWS>(a, idx, G);
                uint32_t todo = __ballot_sync(0xffffffffu, w.kind != kObsNone);
                if (todo == 0) continue;
                while (todo && ok) {
                    const int l = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const int kind = __shfl_sync(0xffffffffu, w.kind, l);
                    if (ROWS && kind == kObsEmpty) {             // nothing is left for this piece of the rows
                        const int pair = __shfl_sync(0xffffffffu, w.pair, l), n = __shfl_sync(0xffffffffu, w.n, l);
                        const int hk = __shfl_sync(0xffffffffu, w.hk, l), row0 = __shfl_sync(0xffffffffu, w.row0, l);
                        const int piece = __shfl_sync(0xffffffffu, w.piece, l);
                        const int64_t lse0 = ((int64_t)hk * a.tokens + row0) * G;
                        for (int r = lane; r < 2 * Tq * G; r += 32) {
                            const int64_t i = (int64_t)2 * pair * Tq * G + r;
                            if (i < (int64_t)n * G) a.part[(lse0 + i) * a.pieces + piece] = make_float2(-INFINITY, 0.f);
                        }
                        continue;
                    }
                    hand_on(w, l);
                    if (kind == kObsEnd) ok = false;
                }
            }
        }
    } else if (warp == 0) {
        // ---------------------------------------------------- TMA: the whole warp, a lane for each box of keys
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
        }
        const int br = min(a.block_size, kTile), boxes = kWide / br;
        uint32_t a_issued[2] = {0, 0}, b_issued[2] = {0, 0};
        int g = 0, step = 0;
        bool ok = true;
        ObsItem w;
        for (int k = 0; ok; ++k) {
            if (!__all_sync(0xffffffffu, take(k, w))) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&i_empty[k % kObsItems]);
            const int32_t* table = a.block_table + (size_t)w.b * a.max_blocks;
            const ObsSteps<ROWS> steps(w, G);
            // the block of this lane's box of the 256 keys from key0 on, -1: none to load
            const auto block = [&](int key0) {
                const int p = key0 + lane * br;
                return lane < boxes && p < w.ctx ? table[p / a.block_size] : -1;
            };
            // 256 keys from key0 on: rows 0 .. 255 of a B tile, or of two A tiles
            const auto load_keys = [&](uint8_t* dst, int key0, int blk, bool split, uint64_t* bar) {
                const int p = key0 + lane * br, r = lane * br;
                const bool there = blk >= 0 && blk < a.num_blocks;
                if (lane < boxes && p < w.ctx && !there) flag_status(status, LL_DEV_BAD_BLOCK);
                const uint32_t n = __popc(__ballot_sync(0xffffffffu, there));
                if (lane == 0) mbar_arrive_expect_tx(bar, n * (uint32_t)(D / 64) * br * 128u);
                __syncwarp();
                if (there) {
                    const int row = (blk * a.n_kv_heads + w.hk) * a.block_size + p % a.block_size;
                    uint8_t* to = split ? dst + (r / kTile) * L::A_TILE + (r % kTile) * 128 : dst + r * 128;
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh)
                        tma_load_2d(to + hh * (split ? kTile : kWide) * 128, &tmK, hh * 64, row, bar);
                }
            };
            int ahead = ROWS ? block(w.j0 * kWide) : block(w.pair * kWide);
            for (int pair = w.pair; pair < w.pairs && ok; pair += w.pair_step, ++g) {
                const int buf = g % ABUFS;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&a_empty[buf], ((uint32_t)(g / ABUFS) & 1u) ^ 1u, &abort_s, status));
                if (!ok) break;
                uint8_t* dst = smem + buf * 2 * L::A_TILE;
                if (ROWS) {
                    const bool second = (2 * pair + 1) * Tq < w.n;
                    if (lane == 0) {
                        const uint32_t bytes = (uint32_t)(Tq * G) * D * 2;
                        mbar_arrive_expect_tx(&a_full[buf], second ? 2 * bytes : bytes);
                        for (int h = 0; h < (second ? 2 : 1); ++h)
#pragma unroll
                            for (int hh = 0; hh < D / 64; ++hh)
                                tma_load_3d(dst + h * L::A_TILE + hh * (kTile * 128), &tmQ, hh * 64, w.hk * G, w.row0 + (2 * pair + h) * Tq,
                                            &a_full[buf]);
                    }
                } else {
                    const int blk = ahead;
                    if (pair + w.pair_step < w.pairs) ahead = block((pair + w.pair_step) * kWide);
                    load_keys(dst, pair * kWide, blk, true, &a_full[buf]);
                }
                ++a_issued[buf];
                if (FEW && !ROWS && pair != w.pair) continue;   // (the rows are there)
                for (int j = steps.first(pair); j < steps.last(); ++j, ++step) {
                    const int st = step % STAGES;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&b_empty[st], ((uint32_t)(step / STAGES) & 1u) ^ 1u, &abort_s, status));
                    if (!ok) break;
                    uint8_t* to = smem + L::OFF_B + st * L::B_TILE;
                    if (ROWS) {
                        const int blk = ahead;
                        if (j + 1 < steps.last()) ahead = block((j + 1) * kWide);
                        load_keys(to, j * kWide, blk, false, &b_full[st]);
                    } else if (lane == 0) {
                        mbar_arrive_expect_tx(&b_full[st], (uint32_t)(Tq * G) * D * 2);
#pragma unroll
                        for (int hh = 0; hh < D / 64; ++hh)
                            tma_load_3d(to + hh * (kWide * 128), &tmQ, hh * 64, w.hk * G, w.row0 + j * Tq, &b_full[st]);
                    }
                    ++b_issued[st];
                }
            }
        }
        if (abort_s && lane == 0) {                          // wait (bounded) for the copies in flight before the CTA leaves
            volatile int never = 0;
            for (int i = 0; i < 2; ++i) {
                if (a_issued[i]) mbar_wait_bounded(&a_full[i], (a_issued[i] - 1) & 1u, &never, nullptr);
                if (b_issued[i]) mbar_wait_bounded(&b_full[i], (b_issued[i] - 1) & 1u, &never, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMA: S[group] = A[group] B^T for every step
            const uint32_t idesc = umma_idesc_bf16(kTile, kWide);
            int g = 0, bstep = 0, step = 0;
            bool ok = true;
            ObsItem w;
            for (int k = 0; ok && take(k, w); ++k) {
                mbar_arrive(&i_empty[k % kObsItems]);
                const ObsSteps<ROWS> steps(w, G);
                for (int pair = w.pair; pair < w.pairs && ok; pair += w.pair_step, ++g) {
                    const int buf = g % ABUFS;
                    if (!mbar_wait_bounded(&a_full[buf], (uint32_t)(g / ABUFS) & 1u, &abort_s, status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem_u32(smem + buf * 2 * L::A_TILE);
                    for (int j = steps.first(pair); j < steps.last() && ok; ++j, ++step) {
                        const int st = bstep % STAGES;
                        if (!mbar_wait_bounded(&b_full[st], (uint32_t)(bstep / STAGES) & 1u, &abort_s, status)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sb = smem_u32(smem + L::OFF_B + st * L::B_TILE);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!mbar_wait_bounded(&s_empty[h], ((uint32_t)step & 1u) ^ 1u, &abort_s, status)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t in = (uint32_t)(kk & 3) * 32;
                                tc_mma_bf16(tmem + h * kWide, umma_desc_sw128(sa + h * L::A_TILE + (kk >> 2) * (kTile * 128) + in),
                                            umma_desc_sw128(sb + (kk >> 2) * (kWide * 128) + in), idesc, kk > 0 ? 1u : 0u);
                            }
                            tc_commit(&s_full[h]);
                        }
                        if (!FEW || ROWS || pair + w.pair_step >= w.pairs) {
                            tc_commit(&b_empty[st]);
                            ++bstep;
                        }
                    }
                    tc_commit(&a_empty[buf]);
                }
            }
            tc_commit(&drain);
            volatile int never = 0;
            mbar_wait_bounded(&drain, 0, &never, status);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- the scores of A tile `h` of every pair
        const int h = (warp - 2) >> 2, r = (warp & 3) * 32 + lane;       // r: TMEM lane = row of the A tile
        const uint32_t scores = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)h * kWide;
        // (a scale of 0 as the smallest number: masked scores stay -infinity, others are 0 in effect)
        const float sl2 = a.scale > 0.f ? a.scale * kLog2eObs : __uint_as_float(1u);
        int step = 0;
        ObsItem w, nw;
        bool more = __all_sync(0xffffffffu, take(0, w));
        if constexpr (ROWS) {
            // which 16-key runs of a key tile have a block, a tile ahead
            constexpr uint32_t kRuns = (1u << (LOAD / 16)) - 1u;
            const auto runs = [&](const ObsItem& w, int j) {
                const int p = j * kWide + (lane & 15) * 16;
                const int blk = p < w.ctx ? a.block_table[(size_t)w.b * a.max_blocks + p / a.block_size] : -1;
                return blk >= 0 && blk < a.num_blocks;
            };
            bool run_ok = more && runs(w, w.j0);
            for (int k = 0; more; ++k) {
                const int tok = (2 * w.pair + h) * Tq + r / G, before = w.ctx - w.n;
                const bool valid = r < Tq * G && tok < w.n;
                const int pos = valid ? before + tok : -1;
                // the lowest and highest position of the tile's rows
                const int tile_lo = before + (2 * w.pair + h) * Tq, tile_hi = before + min(w.n, (2 * w.pair + h + 1) * Tq) - 1;
                const bool any = (2 * w.pair + h) * Tq < w.n;
                float m = -INFINITY, l = 0.f;
                bool next_more = false;
                for (int j = w.j0; j < w.j1; ++j, ++step) {
                    const uint32_t ok16 = __ballot_sync(0xffffffffu, run_ok) & 0xffffu;
                    if (j + 1 < w.j1) {
                        run_ok = runs(w, j + 1);
                    } else {                                 // the next item, and what its first tile needs
                        next_more = __all_sync(0xffffffffu, take(k + 1, nw));
                        run_ok = next_more && runs(nw, nw.j0);
                    }
                    const int key0 = j * kWide;
                    if (!mbar_wait_bounded(&s_full[h], (uint32_t)step & 1u, &abort_s, status)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kWide; c += LOAD) {
                        const int k0 = key0 + c;
                        // (the same for the whole tile: nothing to see, or everything)
                        const bool none = !any || k0 > tile_hi, plain = ((ok16 >> (c / 16)) & kRuns) == kRuns && k0 + LOAD - 1 <= tile_lo;
                        float v[LOAD];
                        if (!none) tmem_ld64(scores + c, v);
                        if (c + LOAD == kWide) {
                            tc_fence_before();
                            mbar_arrive(&s_empty[h]);
                        }
                        if (none) continue;
                        if (!plain) {
#pragma unroll
                            for (int i = 0; i < LOAD; ++i)
                                if (!((ok16 >> (c / 16 + i / 16)) & 1u) || k0 + i > pos) v[i] = -INFINITY;
                        }
                        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                        for (int i = 4; i < LOAD - 4; i += 2) mx[i / 2 & 3] = max3(mx[i / 2 & 3], v[i], v[i + 1]);
                        const float top = max3(max3(mx[0], mx[1], v[LOAD - 4]), max3(mx[2], mx[3], v[LOAD - 3]), max3(v[LOAD - 2], v[LOAD - 1], v[LOAD - 1])) * sl2;
                        if (!(top <= m)) {                   // (NaN too: it stays)
                            l *= ex2_approx(m - top);        // (0 from -infinity)
                            m = top;
                        }
                        const float base = m == -INFINITY ? 0.f : m;
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        const float2 f = make_float2(sl2, sl2), n = make_float2(-base, -base);
#pragma unroll
                        for (int i = 0; i < LOAD; i += 2) {
                            const float2 e = fma2(make_float2(v[i], v[i + 1]), f, n);
                            add_exp2(e, sum[i / 2 & 1]);
                        }
                        l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    }
                }
                if (valid && !abort_s) {
                    const int64_t i = ((int64_t)w.hk * a.tokens + w.row0) * G + (int64_t)(2 * w.pair + h) * Tq * G + r;
                    if (!FEW && a.pieces == 1) a.lse[i] = m == -INFINITY ? INFINITY : m + log2f(l);
                    else a.part[i * a.pieces + w.piece] = make_float2(m, l);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&i_empty[k % kObsItems]);
                w = nw;
                more = next_more;
            }
        } else {
            // the normaliser of column c of query tile j (+infinity: adds nothing).  FEW: from its pieces, once per item.  (More
            // rows have theirs read a tile ahead, which joining on the way would hold up: 8192 rows 671 us for 538.)
            const auto column = [&](const ObsItem& w, int j, int c) {
                const int tok = j * Tq + c / G;
                if (c >= Tq * G || tok >= w.n) return INFINITY;
                const int64_t i = ((int64_t)w.hk * a.tokens + w.row0) * G + (int64_t)j * Tq * G + c;
                if (!FEW) return __ldg(a.lse + i);
                const float2* part = a.part + i * a.pieces;
                float2 x = __ldg(part);
                for (int p = 1; p < w.pieces; ++p) {
                    const float2 y = __ldg(part + p);
                    const float m = max3(x.x, y.x, y.x), base = m == -INFINITY ? 0.f : m;
                    x = make_float2(m, ex2_approx(x.x - base) * x.y + ex2_approx(y.x - base) * y.y);
                }
                return x.x == -INFINITY ? INFINITY : x.x + log2f(x.y);
            };
            float next[2];                                   // of the columns r and r + 128, which this thread brings
            const auto columns = [&](const ObsItem& w, int j) {
#pragma unroll
                for (int i = 0; i < 2; ++i) next[i] = column(w, j, r + i * 128);
            };
            if (more) columns(w, ObsSteps<ROWS>(w, G).first(w.pair));
            bool stop = false;
            for (int k = 0; more && !stop; ++k) {
                const ObsSteps<ROWS> steps(w, G);
                const int before = w.ctx - w.n;
                float* weights = a.weights + ((size_t)w.b * a.n_kv_heads + w.hk) * a.weights_width;
                bool next_more = false;
                for (int pair = w.pair; pair < w.pairs && !stop; pair += w.pair_step) {
                    const int tile0 = (2 * pair + h) * kTile, key = tile0 + r;
                    // the weight so far, and whether its key has a block, on their way beside the first scores
                    const bool in = key < w.ctx, wide = key < a.weights_width;
                    const int blk = in ? a.block_table[(size_t)w.b * a.max_blocks + key / a.block_size] : -1;
                    const float so_far = in && wide ? weights[key] : 0.f;
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    for (int j = steps.first(pair); j < steps.last(); ++j, ++step) {
                        float* lse = s_lse[h][step & 1];
                        lse[r] = -next[0];
                        lse[r + 128] = -next[1];
                        // (a thread whose wait has run out has set abort_s: all leave here)
                        stop = group_bar_any(2 + h, abort_s != 0);
                        if (stop) break;
                        const bool last_step = j + 1 == steps.last(), last_pair = pair + w.pair_step >= w.pairs;
                        if (last_step && last_pair) {        // the next item, and what its first step needs
                            next_more = __all_sync(0xffffffffu, take(k + 1, nw));
                            if (next_more) columns(nw, ObsSteps<ROWS>(nw, G).first(nw.pair));
                        } else if (!FEW) {                   // (FEW: the same rows for every pair)
                            columns(w, last_step ? steps.first(pair + w.pair_step) : j + 1);
                        }
                        const bool got = mbar_wait_bounded(&s_full[h], (uint32_t)step & 1u, &abort_s, status);
                        if (!__all_sync(0xffffffffu, got)) continue;
                        tc_fence_after();
                        const int tok0 = j * Tq, full_to = min(Tq, w.n - tok0) * G;      // columns with a row
                        // columns from `lo` on see this key; all of the tile's keys from `all` on, any from `some` on
                        const int lo = max(0, key - before - tok0) * G;
                        const int some = max(0, tile0 - before - tok0) * G, all = max(0, tile0 + kTile - 1 - before - tok0) * G;
#pragma unroll 1
                        for (int c = 0; c < kWide; c += LOAD) {
                            const bool none = c >= full_to || c + LOAD <= some || tile0 >= w.ctx;
                            const bool plain = c >= all && (c + LOAD <= full_to || full_to == Tq * G);
                            float v[LOAD];
                            if (!none) tmem_ld64(scores + c, v);
                            if (c + LOAD == kWide) {
                                tc_fence_before();
                                mbar_arrive(&s_empty[h]);
                            }
                            if (none) continue;
                            const float4* n4 = reinterpret_cast<const float4*>(lse + c);      // (negated)
                            const float2 f = make_float2(sl2, sl2);
                            if (plain) {
#pragma unroll
                                for (int i = 0; i < LOAD; i += 4) {
                                    const float4 n = n4[i / 4];
                                    add_exp2(fma2(make_float2(v[i], v[i + 1]), f, make_float2(n.x, n.y)), sum[0]);
                                    add_exp2(fma2(make_float2(v[i + 2], v[i + 3]), f, make_float2(n.z, n.w)), sum[1]);
                                }
                            } else {                         // (masked behind the product: the normaliser may be NaN)
#pragma unroll
                                for (int i = 0; i < LOAD; ++i) {
                                    const float e = fmaf(v[i], sl2, reinterpret_cast<const float*>(n4)[i]);
                                    sum[0].x += ex2_approx(c + i < lo || c + i >= full_to ? -INFINITY : e);
                                }
                            }
                        }
                    }
                    if (stop) break;
                    const float total = (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    if (in) {
                        if (!wide) flag_status(status, LL_DEV_BAD_POSITION);
                        else if (blk >= 0 && blk < a.num_blocks) weights[key] = so_far + total;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&i_empty[k % kObsItems]);
                w = nw;
                more = next_more;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// lse of every row from the (max, sum) of its pieces.
__global__ void __launch_bounds__(256) attn_weights_join_kernel(const float2* part, float* lse, long long rows, int pieces) {
    pdl_wait();
    pdl_trigger();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= rows) return;
    float M = -INFINITY, den = 0.f;
    for (int p = 0; p < pieces; ++p) M = max3(M, part[i * pieces + p].x, part[i * pieces + p].x);
    const float base = M == -INFINITY ? 0.f : M;
    for (int p = 0; p < pieces; ++p) {
        const float2 x = part[i * pieces + p];
        den += exp2f(x.x - base) * x.y;
    }
    lse[i] = M == -INFINITY ? INFINITY : base + log2f(den);
}

// Pieces of a row and parts of a KV head's keys: a few items per SM where the batch alone gives fewer.  Rows of whole prompts
// (no more than as many positions again in the table) are items of 1, 2, .. tiles, which fill the SMs without pieces once there
// are enough: 2048 rows of 32 heads 31 + 29 us, in three pieces 33 + 6 for the join + 29; behind longer contexts pieces even
// out what differs: 100 to 700 rows of two contexts to 8000, 8 heads, 60 + 6 us for the rows, 76 in one piece.
struct ObsSplit {
    long long row_items, key_items;
    int pieces, key_ctas;
    bool few;
};

ObsSplit obs_split(int batch, int max_new, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    const long long n = std::max(1, device_sm_count()), key_items = 6 * n;
    const long long row_items = 2LL * max_new >= (long long)max_blocks * block_size ? n : 4 * n;
    const long long Tq = kTile / (n_heads / n_kv_heads), bh = (long long)batch * n_kv_heads;
    const long long items = (max_new + 2 * Tq - 1) / (2 * Tq) * bh;
    const long long tiles = ((long long)max_blocks * block_size + kWide - 1) / kWide;
    ObsSplit s;
    s.pieces = (int)std::max<long long>(1, std::min<long long>({kObsMostPieces, (row_items + items - 1) / items, (tiles + kObsPieceTiles - 1) / kObsPieceTiles}));
    s.key_ctas = (int)std::max<long long>(1, std::min<long long>((key_items + bh - 1) / bh, tiles));
    s.row_items = items * s.pieces;
    s.key_items = bh * s.key_ctas;
    s.few = max_new <= 2 * Tq;
    if (s.few) {                                             // shares: a head's keys in at most so many parts
        s.pieces = (int)std::max<long long>(2, std::min({(n + n_kv_heads - 1) / n_kv_heads + 1, 4 * n / bh + 2, tiles}));
        s.row_items = s.key_items = bh * tiles;
    }
    return s;
}

template <int D, bool ROWS, bool FEW>
cudaError_t launch_pass(const ObserveArgs& a, const CUtensorMap& tmK, long long items, cudaStream_t stream) {
    const int G = a.n_heads / a.n_kv_heads;
    CUtensorMap tmQ;
    if (!make_tmap_heads_sw128(&tmQ, a.q, D, (uint64_t)a.n_heads, (uint64_t)a.tokens, (uint32_t)G, (uint32_t)((ROWS ? kTile : kWide) / G)))
        return cudaErrorInvalidValue;
    const auto kernel = attn_weights_kernel<D, ROWS, FEW>;
    const size_t smem = ObsLayout<D, FEW && !ROWS>::TOTAL + 1024;
    cudaError_t e = ensure_func_attr((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem,
                                     "cudaFuncSetAttribute(attn_weights_kernel)");
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::min<long long>(items, std::max(1, device_sm_count()));
    trace_before(ROWS ? "attn_weights_rows" : "attn_weights_cols", stream);
    e = launch_pdl(kernel, dim3(grid), dim3(kObsThreads), smem, stream, 1, tmQ, tmK, a, items);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "attn_weights_kernel launch");
}

template <int D>
cudaError_t observe_for(const ObserveArgs& a, const ObsSplit& s, cudaStream_t stream) {
    CUtensorMap tmK;
    const uint64_t rows = (uint64_t)a.num_blocks * a.n_kv_heads * a.block_size;
    if (!make_tmap_bf16_sw128(&tmK, a.k_pool, D, rows, (uint32_t)std::min(a.block_size, kTile))) return cudaErrorInvalidValue;
    if (s.few) {
        const cudaError_t e = launch_pass<D, true, true>(a, tmK, s.row_items, stream);
        return e != cudaSuccess ? e : launch_pass<D, false, true>(a, tmK, s.key_items, stream);
    }
    cudaError_t e = launch_pass<D, true, false>(a, tmK, s.row_items, stream);
    if (e != cudaSuccess) return e;
    if (a.pieces > 1) {
        const long long n = (long long)a.tokens * a.n_heads;
        trace_before("attn_weights_join", stream);
        e = launch_pdl(attn_weights_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, (const float2*)a.part, a.lse, n,
                       a.pieces);
        trace_after(stream);
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return record(e, "attn_weights_join launch");
    }
    return launch_pass<D, false, false>(a, tmK, s.key_items, stream);
}

}  // namespace

bool observe_fits(int batch, int max_new, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    const ObsSplit s = obs_split(batch, std::max(max_new, 1), n_heads, n_kv_heads, max_blocks, block_size);
    return s.few || (s.row_items < (1LL << 31) && s.key_items < (1LL << 31));
}

// The normalisers, and a (max, sum) for each piece of a row.
static size_t observe_bytes(int tokens, int n_heads, long long pieces) {
    const size_t rows = (size_t)tokens * n_heads;
    return (rows * sizeof(float) + 15) / 16 * 16 + rows * pieces * sizeof(float2);
}

size_t observe_scratch_bytes(int batch, int tokens, int max_new, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    return observe_bytes(tokens, n_heads, obs_split(batch, std::max(max_new, 1), n_heads, n_kv_heads, max_blocks, block_size).pieces);
}

size_t observe_workspace_bytes(int tokens, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    // (fewer rows and sequences are cut into more pieces: the most that obs_split gives any)
    const long long n = std::max(1, device_sm_count()), tiles = ((long long)max_blocks * block_size + kWide - 1) / kWide;
    const long long few = (n + n_kv_heads - 1) / n_kv_heads + 1;
    return observe_bytes(tokens, n_heads, std::max<long long>(2, std::min(tiles, std::max<long long>(few, kObsMostPieces))));
}

cudaError_t launch_observe(ObserveArgs a, void* workspace, cudaStream_t stream) {
    if (a.tokens <= 0) return cudaSuccess;
    const ObsSplit s = obs_split(a.batch, a.max_new, a.n_heads, a.n_kv_heads, a.max_blocks, a.block_size);
    a.pieces = s.pieces;
    a.key_ctas = s.key_ctas;
    a.lse = static_cast<float*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<char*>(workspace) + ((size_t)a.tokens * a.n_heads * 4 + 15) / 16 * 16);
    return a.head_dim == 128 ? observe_for<128>(a, s, stream) : observe_for<64>(a, s, stream);
}

}  // namespace ll
