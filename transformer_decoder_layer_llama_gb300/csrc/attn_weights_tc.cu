// Attention weights of a ragged batch of query rows over a paged BF16 cache, on the tensor cores (tcgen05, TMEM, TMA):
//   weights[b][hk][p] += sum over rows i of sequence b and heads h of hk of P_ih(p),  P_ih = softmax_p(scale q_ih k_p), p <= pos(i).
//
// A column sum of P needs every row's normaliser first, and the scores of all pairs are too many to keep (4 bytes a
// pair), so they are computed twice:
//   ROWS  128 query rows (tokens x heads of a KV head) in the lanes, keys in the columns: a thread has a row and runs over
//         its scores with a running maximum and sum.  Long rows are split into `pieces` and joined by a small kernel.
//   COLS  128 keys in the lanes, query rows in the columns: a thread has a key, adds 2^(score - lse of the column) and at
//         the end adds its sum to the weight.  One thread per weight: no atomics, the same bits every time.
// Both are one kernel: two tiles of 128 rows stay in shared memory (A), tiles of 128 rows stream past them (B), and each
// streamed tile meets both, which halves the traffic from L2 per score.  Warp 0 loads (TMA), warp 1 issues the MMAs, two
// groups of four warps take the scores of one A tile each from TMEM, two buffers a tile so that the next product runs
// beside the exponentials.  Every wait is bounded.
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kTile = 128;
constexpr int kObsThreads = 320;
constexpr float kLog2eObs = 1.4426950408889634f;
constexpr int kObsPieceTiles = 4;        // at least, of a piece of a row

template <int D, bool ROWS>
struct ObsLayout {
    static constexpr uint32_t TILE = kTile * D * 2;          // [D / 64][128 rows][128 B], 128-byte swizzle
    static constexpr int A_BUFS = ROWS ? 1 : 2;              // of two tiles
    static constexpr int STAGES = ROWS ? 4 : 2;
    static constexpr uint32_t OFF_B = A_BUFS * 2 * TILE;
    static constexpr uint32_t TOTAL = OFF_B + STAGES * TILE;
};

// What a sequence brings: its first query row, their number, the context (0 rows: nothing to do).
struct ObsSeq {
    int row0, n, ctx;
};

LL_DEVINL ObsSeq obs_sequence(const ObserveArgs& a, int b, bool flag) {
    ObsSeq s;
    s.row0 = a.cu_new[b];
    s.n = a.cu_new[b + 1] - s.row0;
    s.ctx = a.context_lens[b];
    const long long end = (long long)a.cu_new[b + 1];
    if (s.row0 < 0 || end < s.row0 || end > a.tokens || s.n > a.max_new || s.ctx < s.n ||
        (long long)s.ctx > (long long)a.max_blocks * a.block_size) {
        if (flag) flag_status(a.status, LL_DEV_BAD_POSITION);
        s.n = 0;
    }
    return s;
}

// The steps of a CTA: groups of two A tiles, and for each the B tiles first .. last - 1.
template <bool ROWS>
struct ObsWork {
    ObsSeq s;
    int b, hk, G, Tq;                    // heads per KV head, query tokens per tile
    int pair, pair_step, pairs;          // A tiles 2 pair and 2 pair + 1, pair += pair_step while below pairs
    int piece, j0, j1;                   // ROWS: key tiles of this piece
    int nq;                              // COLS: query tiles of the sequence

    LL_DEVINL int first(int p) const {
        if (ROWS) return j0;
        const int behind = 2 * kTile * p - (s.ctx - s.n);    // tokens of the call before the first key
        return behind <= 0 ? 0 : behind / Tq;
    }
    LL_DEVINL int last() const { return ROWS ? j1 : nq; }
};

template <bool ROWS>
LL_DEVINL bool obs_work(const ObserveArgs& a, ObsWork<ROWS>& w) {
    w.G = a.n_heads / a.n_kv_heads;
    w.Tq = kTile / w.G;
    int idx = blockIdx.x;
    w.hk = idx % a.n_kv_heads;
    idx /= a.n_kv_heads;
    w.b = idx % a.batch;
    idx /= a.batch;
    w.s = obs_sequence(a, w.b, ROWS && threadIdx.x == 0 && w.hk == 0 && idx == 0);
    if (w.s.n <= 0) return false;
    w.nq = (w.s.n + w.Tq - 1) / w.Tq;
    if (ROWS) {
        w.piece = idx % a.pieces;
        const int most = (a.max_new + 2 * w.Tq - 1) / (2 * w.Tq);
        w.pair = most - 1 - idx / a.pieces;                  // the pairs with the most keys first
        w.pairs = w.pair + 1;
        w.pair_step = 1;
        if (2 * w.pair >= w.nq) return false;
        const int end = min(w.s.n, (2 * w.pair + 2) * w.Tq);            // tokens of the pair end here
        const int tiles = (w.s.ctx - w.s.n + end - 1) / kTile + 1;
        const int len = max(kObsPieceTiles, (tiles + a.pieces - 1) / a.pieces);
        w.j0 = min(tiles, w.piece * len);
        w.j1 = min(tiles, w.j0 + len);
    } else {
        w.pair = idx;
        w.pair_step = a.key_ctas;
        w.pairs = (w.s.ctx + 2 * kTile - 1) / (2 * kTile);
        if (w.pair >= w.pairs) return false;
    }
    return true;
}

// Barrier of a group of four warps, with an OR of `pred` for all its threads.
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

template <int D, bool ROWS>
__global__ void __launch_bounds__(kObsThreads, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const ObserveArgs a) {
    using L = ObsLayout<D, ROWS>;
    constexpr int STAGES = L::STAGES, ABUFS = L::A_BUFS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t a_full[2], a_empty[2], b_full[STAGES], b_empty[STAGES], s_full[2][2], s_empty[2][2], drain;
    __shared__ __align__(16) float s_lse[2][2][kTile];                     // COLS: [group][step parity][column]
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* status = a.status;
    pdl_wait();
    pdl_trigger();
    ObsWork<ROWS> w;
    if (!obs_work<ROWS>(a, w)) return;
    const int32_t* table = a.block_table + (size_t)w.b * a.max_blocks;
    const int64_t lse0 = ((int64_t)w.hk * a.tokens + w.s.row0) * w.G;      // this sequence and KV head among the rows of normalisers

    if (ROWS && w.j0 >= w.j1) {                              // nothing left for this piece
        for (int r = threadIdx.x; r < 2 * w.Tq * w.G; r += kObsThreads) {
            const int64_t i = (int64_t)2 * w.pair * w.Tq * w.G + r;
            if (i < (int64_t)w.s.n * w.G) a.part[(lse0 + i) * a.pieces + w.piece] = make_float2(-INFINITY, 0.f);
        }
        return;
    }
    // COLS with few query tiles: they stay in their stages for all of the CTA's keys
    const bool resident = !ROWS && w.nq <= STAGES;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&a_full[i], 1);
            mbar_init(&a_empty[i], 1);
            for (int g = 0; g < 2; ++g) {
                mbar_init(&s_full[g][i], 1);
                mbar_init(&s_empty[g][i], 128);
            }
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        mbar_init(&drain, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (!ROWS) {                                             // columns behind the tile's last row: zeros, for finite scores
        const int used = w.Tq * w.G, rows = kTile - used;
        for (int i = threadIdx.x; i < STAGES * (D / 64) * rows * 8; i += kObsThreads) {
            const int c = i & 7, r = used + (i >> 3) % rows, half = (i >> 3) / rows;     // half: of a stage
            *reinterpret_cast<uint4*>(smem + L::OFF_B + half * (kTile * 128) + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
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

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            const int br = min(a.block_size, kTile);
            const auto load_queries = [&](uint8_t* dst, int tile, uint64_t* bar) {
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh)
                    tma_load_3d(dst + hh * (kTile * 128), &tmQ, hh * 64, w.hk * w.G, w.s.row0 + tile * w.Tq, bar);
            };
            const uint32_t query_bytes = (uint32_t)(w.Tq * w.G) * D * 2;
            const auto key_bytes = [&](int tile) {
                uint32_t bytes = 0;
                for (int p = tile * kTile; p < tile * kTile + kTile && p < w.s.ctx; p += br) {
                    const int blk = table[p / a.block_size];
                    if (blk >= 0 && blk < a.num_blocks) bytes += (uint32_t)(D / 64) * br * 128u;
                }
                return bytes;
            };
            const auto load_keys = [&](uint8_t* dst, int tile, uint64_t* bar) {
                for (int p = tile * kTile, sb = 0; p < tile * kTile + kTile && p < w.s.ctx; p += br, ++sb) {
                    const int blk = table[p / a.block_size];
                    if (blk < 0 || blk >= a.num_blocks) {
                        flag_status(status, LL_DEV_BAD_BLOCK);
                        continue;
                    }
                    const int row = (blk * a.n_kv_heads + w.hk) * a.block_size + p % a.block_size;
#pragma unroll
                    for (int hh = 0; hh < D / 64; ++hh)
                        tma_load_2d(dst + hh * (kTile * 128) + sb * br * 128, &tmK, hh * 64, row, bar);
                }
            };
            uint32_t a_issued[2] = {0, 0}, b_issued[STAGES];
            for (int i = 0; i < STAGES; ++i) b_issued[i] = 0;
            int g = 0, step = 0;
            bool ok = true;
            for (int pair = w.pair; pair < w.pairs && ok; pair += w.pair_step, ++g) {
                const int buf = g % ABUFS;
                if (!mbar_wait_bounded(&a_empty[buf], ((uint32_t)(g / ABUFS) & 1u) ^ 1u, &abort_s, status)) break;
                uint8_t* dst = smem + buf * 2 * L::TILE;
                if (ROWS) {
                    const bool second = 2 * pair + 1 < w.nq;
                    mbar_arrive_expect_tx(&a_full[buf], second ? 2 * query_bytes : query_bytes);
                    load_queries(dst, 2 * pair, &a_full[buf]);
                    if (second) load_queries(dst + L::TILE, 2 * pair + 1, &a_full[buf]);
                } else {
                    mbar_arrive_expect_tx(&a_full[buf], key_bytes(2 * pair) + key_bytes(2 * pair + 1));
                    load_keys(dst, 2 * pair, &a_full[buf]);
                    load_keys(dst + L::TILE, 2 * pair + 1, &a_full[buf]);
                }
                ++a_issued[buf];
                if (resident && g > 0) continue;
                for (int j = w.first(pair); j < w.last(); ++j, ++step) {
                    const int st = resident ? j : step % STAGES;
                    if (!resident && !mbar_wait_bounded(&b_empty[st], ((uint32_t)(step / STAGES) & 1u) ^ 1u, &abort_s, status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* to = smem + L::OFF_B + st * L::TILE;
                    if (ROWS) {
                        mbar_arrive_expect_tx(&b_full[st], key_bytes(j));
                        load_keys(to, j, &b_full[st]);
                    } else {
                        mbar_arrive_expect_tx(&b_full[st], query_bytes);
                        load_queries(to, j, &b_full[st]);
                    }
                    ++b_issued[st];
                }
            }
            if (abort_s) {                                   // wait (bounded) for the copies in flight before the CTA leaves
                volatile int never = 0;
                for (int i = 0; i < 2; ++i)
                    if (a_issued[i]) mbar_wait_bounded(&a_full[i], (a_issued[i] - 1) & 1u, &never, nullptr);
                for (int i = 0; i < STAGES; ++i)
                    if (b_issued[i]) mbar_wait_bounded(&b_full[i], (b_issued[i] - 1) & 1u, &never, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMA: S[group] = A[group] B^T for every step
            const uint32_t idesc = umma_idesc_bf16(kTile, kTile);
            int g = 0, step = 0;
            bool ok = true;
            for (int pair = w.pair; pair < w.pairs && ok; pair += w.pair_step, ++g) {
                const int buf = g % ABUFS;
                if (!mbar_wait_bounded(&a_full[buf], (uint32_t)(g / ABUFS) & 1u, &abort_s, status)) break;
                const uint32_t sa = smem_u32(smem + buf * 2 * L::TILE);
                for (int j = w.first(pair); j < w.last() && ok; ++j, ++step) {
                    const int st = resident ? j : step % STAGES;
                    if (!mbar_wait_bounded(&b_full[st], resident ? 0u : (uint32_t)(step / STAGES) & 1u, &abort_s, status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sb = smem_u32(smem + L::OFF_B + st * L::TILE);
                    const int par = step & 1;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!mbar_wait_bounded(&s_empty[h][par], ((uint32_t)(step >> 1) & 1u) ^ 1u, &abort_s, status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + (uint32_t)(h * 2 + par) * kTile;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (uint32_t)(kk >> 2) * (kTile * 128) + (uint32_t)(kk & 3) * 32;
                            tc_mma_bf16(d, umma_desc_sw128(sa + h * L::TILE + off), umma_desc_sw128(sb + off), idesc, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(&s_full[h][par]);
                    }
                    if (!resident) tc_commit(&b_empty[st]);
                }
                tc_commit(&a_empty[buf]);
            }
            tc_commit(&drain);
            volatile int never = 0;
            mbar_wait_bounded(&drain, 0, &never, status);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- the scores of A tile `h` of every group
        const int h = (warp - 2) >> 2, r = (warp & 3) * 32 + lane;       // r: TMEM lane = row of the A tile
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const float sl2 = a.scale * kLog2eObs;
        const int before = w.s.ctx - w.s.n;                  // positions before the call's first row
        int step = 0;
        if (ROWS) {
            const int tile = 2 * w.pair + h, tok = tile * w.Tq + r / w.G;
            const bool valid = r < w.Tq * w.G && tok < w.s.n;
            const int pos = valid ? before + tok : -1;
            const int tile_pos = before + tile * w.Tq;       // the lowest position of the tile's rows
            float m = -INFINITY, l = 0.f;
            // which 16-key runs of a key tile have a block, a tile ahead
            const auto runs = [&](int j) {
                const int p = j * kTile + (lane & 7) * 16;
                const int blk = p < w.s.ctx ? table[p / a.block_size] : -1;
                return blk >= 0 && blk < a.num_blocks;
            };
            bool run_ok = runs(w.j0);
            for (int j = w.j0; j < w.j1; ++j, ++step) {
                const uint32_t ok8 = __ballot_sync(0xffffffffu, run_ok) & 0xffu;
                if (j + 1 < w.j1) run_ok = runs(j + 1);
                const int par = step & 1, key0 = j * kTile;
                if (!mbar_wait_bounded(&s_full[h][par], (uint32_t)(step >> 1) & 1u, &abort_s, status)) break;
                tc_fence_after();
                const bool plain = ok8 == 0xffu && key0 + kTile - 1 <= tile_pos;       // the same for the whole group
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float v[64];
                    tmem_ld64(tmem + lane_base + (uint32_t)(h * 2 + par) * kTile + half * 64, v);
                    if (half == 1) {
                        tc_fence_before();
                        mbar_arrive(&s_empty[h][par]);
                    }
                    if (!plain) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((ok8 >> (half * 4 + c / 16)) & 1u) || key0 + half * 64 + c > pos) v[c] = -INFINITY;
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int c = 4; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], v[c]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                    if (top > m) {
                        l *= ex2_approx(m - top);            // (0 from -infinity)
                        m = top;
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 64; ++c) sum[c & 3] += ex2_approx(fmaf(v[c], sl2, -base));
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
            }
            if (valid && !abort_s) {
                const int64_t i = lse0 + (int64_t)tile * w.Tq * w.G + r;
                if (a.pieces == 1) a.lse[i] = l == 0.f ? INFINITY : m + log2f(l);
                else a.part[i * a.pieces + w.piece] = make_float2(m, l);
            }
        } else {
            // the normaliser of column r of query tile j (+infinity: adds nothing)
            const auto column = [&](int j) {
                const int tok = j * w.Tq + r / w.G;
                return r < w.Tq * w.G && tok < w.s.n ? __ldg(a.lse + lse0 + (int64_t)j * w.Tq * w.G + r) : INFINITY;
            };
            float* weights = a.weights + ((size_t)w.b * a.n_kv_heads + w.hk) * a.weights_width;
            float next = column(w.first(w.pair));
            bool stop = false;
            for (int pair = w.pair; pair < w.pairs && !stop; pair += w.pair_step) {
                const int tile0 = (2 * pair + h) * kTile, key = tile0 + r;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                for (int j = w.first(pair); j < w.last(); ++j, ++step) {
                    const int par = step & 1;
                    s_lse[h][par][r] = next;
                    stop = group_bar_any(2 + h, abort_s != 0);
                    if (stop) break;
                    if (j + 1 < w.last()) next = column(j + 1);
                    else if (pair + w.pair_step < w.pairs) next = column(w.first(pair + w.pair_step));
                    // (a thread whose wait runs out has set abort_s: all leave at the next barrier)
                    const bool got = mbar_wait_bounded(&s_full[h][par], (uint32_t)(step >> 1) & 1u, &abort_s, status);
                    if (!__all_sync(0xffffffffu, got)) continue;
                    tc_fence_after();
                    const int tok0 = j * w.Tq;
                    const bool plain = tok0 + w.Tq <= w.s.n && tile0 + kTile - 1 <= before + tok0;
                    // columns from `lo` on see this key, up to the sequence's last row
                    const int lo = max(0, key - before - tok0) * w.G, hi = min(w.Tq, w.s.n - tok0) * w.G;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float v[64];
                        tmem_ld64(tmem + lane_base + (uint32_t)(h * 2 + par) * kTile + half * 64, v);
                        if (half == 1) {
                            tc_fence_before();
                            mbar_arrive(&s_empty[h][par]);
                        }
                        const float4* lse = reinterpret_cast<const float4*>(&s_lse[h][par][half * 64]);
#pragma unroll
                        for (int c = 0; c < 64; c += 4) {
                            const float4 n = lse[c / 4];
                            float e[4] = {fmaf(v[c], sl2, -n.x), fmaf(v[c + 1], sl2, -n.y), fmaf(v[c + 2], sl2, -n.z), fmaf(v[c + 3], sl2, -n.w)};
                            if (!plain) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (half * 64 + c + i < lo || half * 64 + c + i >= hi) e[i] = -INFINITY;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[i] += ex2_approx(e[i]);
                        }
                    }
                }
                if (!stop && key < w.s.ctx) {
                    const int blk = table[key / a.block_size];
                    if (key >= a.weights_width) flag_status(status, LL_DEV_BAD_POSITION);
                    else if (blk >= 0 && blk < a.num_blocks) weights[key] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
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
    for (int p = 0; p < pieces; ++p) M = fmaxf(M, part[i * pieces + p].x);
    const float base = M == -INFINITY ? 0.f : M;
    for (int p = 0; p < pieces; ++p) {
        const float2 x = part[i * pieces + p];
        den += exp2f(x.x - base) * x.y;
    }
    lse[i] = den == 0.f ? INFINITY : base + log2f(den);
}

template <int D>
cudaError_t observe_for(const ObserveArgs& a, cudaStream_t stream) {
    CUtensorMap tmQ, tmK;
    const int G = a.n_heads / a.n_kv_heads, Tq = kTile / G;
    const uint64_t rows = (uint64_t)a.num_blocks * a.n_kv_heads * a.block_size;
    if (!make_tmap_bf16_sw128(&tmK, a.k_pool, D, rows, (uint32_t)std::min(a.block_size, kTile)) ||
        !make_tmap_heads_sw128(&tmQ, a.q, D, (uint64_t)a.n_heads, (uint64_t)a.tokens, (uint32_t)G, (uint32_t)Tq))
        return cudaErrorInvalidValue;
    const size_t smem_rows = ObsLayout<D, true>::TOTAL + 1024, smem_cols = ObsLayout<D, false>::TOTAL + 1024;
    cudaError_t e = ensure_func_attr((const void*)attn_weights_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem_rows, "cudaFuncSetAttribute(attn_weights_kernel)");
    if (e == cudaSuccess)
        e = ensure_func_attr((const void*)attn_weights_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_cols, "cudaFuncSetAttribute(attn_weights_kernel)");
    if (e != cudaSuccess) return e;
    const int pairs = (a.max_new + 2 * Tq - 1) / (2 * Tq);
    trace_before("attn_weights_rows", stream);
    e = launch_pdl(attn_weights_kernel<D, true>, dim3((unsigned)((long long)pairs * a.pieces * a.batch * a.n_kv_heads)), dim3(kObsThreads),
                   smem_rows, stream, 1, tmQ, tmK, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "attn_weights_kernel launch");
    if (a.pieces > 1) {
        const long long n = (long long)a.tokens * a.n_heads;
        trace_before("attn_weights_join", stream);
        e = launch_pdl(attn_weights_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, (const float2*)a.part, a.lse, n,
                       a.pieces);
        trace_after(stream);
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return record(e, "attn_weights_join launch");
    }
    trace_before("attn_weights_cols", stream);
    e = launch_pdl(attn_weights_kernel<D, false>, dim3((unsigned)((long long)a.key_ctas * a.batch * a.n_kv_heads)), dim3(kObsThreads),
                   smem_cols, stream, 1, tmQ, tmK, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "attn_weights_kernel launch");
}

// Pieces of a row and CTAs of a KV head's keys: about four CTAs per SM where the batch alone gives fewer.
struct ObsSplit {
    long long row_items, key_items;      // CTAs of the two passes
    int pieces, key_ctas;
};

ObsSplit obs_split(int batch, int max_new, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    constexpr int kCtas = 4 * 152;
    const long long Tq = kTile / (n_heads / n_kv_heads), bh = (long long)batch * n_kv_heads;
    const long long items = (max_new + 2 * Tq - 1) / (2 * Tq) * bh;
    const long long tiles = ((long long)max_blocks * block_size + kTile - 1) / kTile;
    ObsSplit s;
    s.pieces = (int)std::max<long long>(1, std::min<long long>({16, (kCtas + items - 1) / items, (tiles + kObsPieceTiles - 1) / kObsPieceTiles}));
    s.key_ctas = (int)std::max<long long>(1, std::min<long long>((kCtas + bh - 1) / bh, (tiles + 1) / 2));
    s.row_items = items * s.pieces;
    s.key_items = bh * s.key_ctas;
    return s;
}

}  // namespace

bool observe_fits(int batch, int max_new, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    const ObsSplit s = obs_split(batch, std::max(max_new, 1), n_heads, n_kv_heads, max_blocks, block_size);
    return s.row_items < (1LL << 31) && s.key_items < (1LL << 31);
}

size_t observe_scratch_bytes(int batch, int tokens, int max_new, int n_heads, int n_kv_heads, int max_blocks, int block_size) {
    // the normalisers, and room for the pieces of rows
    const size_t rows = (size_t)tokens * n_heads;
    const ObsSplit s = obs_split(batch, std::max(max_new, 1), n_heads, n_kv_heads, max_blocks, block_size);
    return (rows * 4 + 15) / 16 * 16 + (s.pieces > 1 ? rows * s.pieces * 8 : 0);
}

cudaError_t launch_observe(ObserveArgs a, void* workspace, cudaStream_t stream) {
    if (a.tokens <= 0) return cudaSuccess;
    const ObsSplit s = obs_split(a.batch, a.max_new, a.n_heads, a.n_kv_heads, a.max_blocks, a.block_size);
    a.pieces = s.pieces;
    a.key_ctas = s.key_ctas;
    a.lse = static_cast<float*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<char*>(workspace) + ((size_t)a.tokens * a.n_heads * 4 + 15) / 16 * 16);
    return a.head_dim == 128 ? observe_for<128>(a, stream) : observe_for<64>(a, stream);
}

}  // namespace ll
