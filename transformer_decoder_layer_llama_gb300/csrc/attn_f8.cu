// Decode attention over a paged cache of e4m3 codes with one scale per block and KV head:
// one query token per sequence, softmax(q k^T scale) v with k = code * k_scale[block][head] and
// v = code * v_scale[block][head].
//
// Bound by memory: every code of the contexts is read once, one byte per element.  The work is cut
// along the key axis into equal shares whatever the batch: all (sequence, KV head, 64-key tile)
// triples of the actual contexts form one list, and each CTA of a grid that fills the GPU once takes
// an equal run of it.  A CTA that holds all tiles of a (sequence, KV head) writes its output; one
// that shares them leaves a float32 partial (at most two per CTA), which the join kernel merges by
// the log-sum-exp.
//
// A CTA is four consumer warps and a producer warp.  The producer brings each tile's codes in by TMA
// (four stages) with the scales of its blocks, reading the block table and scales a batch of tiles
// ahead.  Each consumer warp owns 16 keys of a tile (they lie in one block, so its scales are scalars):
// S^T = K Q^T and O^T += V^T P^T by mma.sync with the keys, and the head dims, as the 16 rows of A
// and up to 8 (or 16) query heads of the KV head as columns, so a single query head wastes 7 of 8
// columns instead of 15 of 16 rows.  The tensor pipe has the room: per SM about 19 cache bytes a clock
// arrive, and a tile's MMAs take about a quarter of its load time.  7B shapes, 64 sequences of 512 to 4096 keys
// (1.2 GB): 205 us, 5.9 TB/s (87% of the copy bandwidth); 70B shapes, 16 of 4096 to 32768 (0.6 GB): 102 us,
// 5.9 TB/s.  The same sequences with head dim 64 take 134 and 71 us (66 and 62%: a tile's fixed work for half
// its bytes), with 16 query heads per KV head 138 (128) and 96 (64): twice the MMAs and exponentials a tile.
//
// Precision.  Codes become FP16 exactly.  A query row is scaled by a power of two so that its largest
// element lies in [2^14, 2^15) before it becomes FP16: BF16 has fewer bits, so only elements below
// 2^-28 of the row's largest are rounded.  Scores, the running maximum and sums are float32.  A
// probability enters P V as one FP16 (11 significant bits, relative error 2^-11, an eighth of the BF16
// output's half step) times its block's V scale, relative to the largest such term t that the warp has met
// for the query, times 2^6: below 2^15, and still exact to 2^-31 of the largest term.  So a block that hardly
// weighs takes no bits from the others, however large its V.  The sum of the probabilities has a base of its
// own (m); terms times one power of two per block are probabilities.
#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr float kLog2eF8 = 1.4426950408889634f;
constexpr int kF8Tile = 64;              // keys per tile
constexpr int kF8Stages = 4;
constexpr int kF8Threads = 160;
constexpr float kF8Shift = 6.f;          // probabilities times V scales enter P V times 2^6
constexpr float kF8Floor = 80.f;         // a V scale this far (in powers of two) below the largest term adds nothing
// Up to 8 query heads per KV head: three CTAs per SM of four stages each (192 KB of codes per SM at D = 128).
// 7B shapes 201 us, 70B shapes 102 when it was chosen; with three stages and four (7B) or three CTAs 201 and 110,
// with four CTAs throughout 217 and 108, for their 96 registers spill.  Head dim 64, calls one at a time: 145 us
// (7B heads) and 83 (70B); with two CTAs 188 and 96, with six stages 145 and 82.  Beyond 8 heads two CTAs, for the
// accumulators of a second column tile: 149 us (16 heads, dim 128) and 106 (64); with three 201, for spills, and 105.
constexpr int kF8MaxCtasPerSm = 3;

LL_DEVINL int f8_context(const AttnF8Args& a, int b, bool flag) {
    const int cap = a.max_blocks * a.block_size;
    const int ctx = a.context_lens[b];
    if (ctx < 0 || ctx > cap) {
        if (flag) flag_status(a.status, LL_DEV_BAD_POSITION);
        return min(max(ctx, 0), cap);
    }
    return ctx;
}
LL_DEVINL int f8_tiles(int ctx) { return (ctx + kF8Tile - 1) / kF8Tile; }

// Share c of P equal runs of n tiles: the first n % P shares are one tile longer.
LL_DEVINL long long share_begin(long long n, int P, int c) {
    const long long q = n / P, r = n - q * P;
    return q * c + min((long long)c, r);
}
LL_DEVINL int share_of(long long n, int P, long long t) {
    const long long q = n / P, r = n - q * P;
    return (int)(t < r * (q + 1) ? t / (q + 1) : r + (t - r * (q + 1)) / q);
}

// Byte offset of the 16-byte chunk that holds byte `at` of key row r in a tile of D-byte rows that TMA
// wrote as 128-byte lines with the 128-byte swizzle (two rows per line where D = 64).
template <int D>
LL_DEVINL uint32_t f8_chunk(int r, int at) {
    const int byte = r * D + at;
    const int line = byte >> 7, c = (byte >> 4) & 7;
    return (uint32_t)(line * 128 + ((c ^ (line & 7)) << 4));
}

// Where in the list of tiles a share begins: the sequence, and the tile's place in the sequence's part.
struct F8Start {
    long long total;     // tiles of all sequences and KV heads
    int b;
    long long at;        // tile within the Hkv * tiles(b) tiles of sequence b
};

// All threads of a CTA of nt threads (a multiple of 32, at most 160): sums the contexts, finds the place
// of tile share_begin(total, P, c).
LL_DEVINL void f8_find_start(const AttnF8Args& a, int P, int c, int nt, bool flag, long long* sums, F8Start* out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.batch + nt - 1) / nt;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += f8_tiles(f8_context(a, b, flag));
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
    for (int w = 0; w < nt / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    total *= a.n_kv_heads;
    before *= a.n_kv_heads;
    const long long t0 = share_begin(total, P, c);
    if (tid == 0) out->total = total;
    if (t0 < total && t0 >= before && t0 < before + mine * a.n_kv_heads) {
        int b = b0;
        for (;; ++b) {
            const long long n = (long long)f8_tiles(f8_context(a, b, false)) * a.n_kv_heads;
            if (t0 < before + n) break;
            before += n;
        }
        out->b = b;
        out->at = t0 - before;
    }
    __syncthreads();
}

// A run of tiles of one (sequence, KV head).
struct F8Segment {
    int b, hk, kt0, kt1, n_kt, ctx;
};

// Walks a share segment by segment.
struct F8Walk {
    int b;
    long long at;        // tile within sequence b
    long long left;      // tiles of the share still to do
    LL_DEVINL bool next(const AttnF8Args& a, F8Segment& s) {
        while (left > 0) {
            const int ctx = f8_context(a, b, false);
            const int n = f8_tiles(ctx);
            if (at >= (long long)n * a.n_kv_heads) {
                at = 0;
                ++b;
                continue;
            }
            s.b = b;
            s.ctx = ctx;
            s.n_kt = n;
            s.hk = (int)(at / n);
            s.kt0 = (int)(at - (long long)s.hk * n);
            s.kt1 = (int)min((long long)n, s.kt0 + left);
            at += s.kt1 - s.kt0;
            left -= s.kt1 - s.kt0;
            return true;
        }
        return false;
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(kF8Threads, NT == 1 ? kF8MaxCtasPerSm : 2)
    attn_decode_f8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const AttnF8Args a) {
    constexpr int BN = kF8Tile, STAGES = kF8Stages, NCONS = 128;
    constexpr int TILE = BN * D;
    constexpr int W = D / 16;                              // words of a key row per lane, MMA steps along D
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sk = sbase;                                   // [STAGES][TILE]
    uint8_t* sv = sk + STAGES * TILE;                      // [STAGES][TILE]
    float* s_acc = reinterpret_cast<float*>(sv + STAGES * TILE);   // [4 warps][G][32], for merging at a segment's end
    __shared__ uint64_t full_bar[STAGES], empty_bar[STAGES];
    __shared__ unsigned long long valid_s[STAGES];         // per stage: bit k = key k of the tile is cached
    __shared__ float2 scale_s[STAGES][4];                  // per stage and 16 keys: K scale, log2 of the V scale
    __shared__ float2 s_ml[4][16];                         // per warp and query head: max, sum
    __shared__ float s_t[4][16];                           // and largest term (below)
    __shared__ long long s_sums[kF8Threads / 32];
    __shared__ F8Start s_start;
    __shared__ int abort_s;

    const int G = a.n_heads / a.n_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = gridDim.x, cta = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(&full_bar[st], 1);
            mbar_init(&empty_bar[st], 4);
        }
        abort_s = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    f8_find_start(a, P, cta, kF8Threads, cta == 0, s_sums, &s_start);
    const long long total = s_start.total;
    const long long t_begin = share_begin(total, P, cta), t_end = share_begin(total, P, cta + 1);
    if (t_begin >= t_end) return;
    F8Walk walk{s_start.b, s_start.at, t_end - t_begin};
    F8Segment seg;

    if (warp == 4) {
        // ------------------------------------------------ producer
        // Lane i looks after 16-to-64-key box i % spt of tile i / spt of a batch of 32 / spt tiles: its
        // block and scales are loaded one batch ahead of its TMA loads.
        const int kt_rows = min(a.block_size, BN);
        const int spt = BN / kt_rows, tpb = 32 / spt;
        const int my_tile = lane / spt, sb = lane % spt;
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        uint32_t issued = 0, parity = 0;                   // per stage: a load was issued; parity of the loads
        int it = 0;                                        // tiles of the share so far
        bool ok = true;
        while (ok && walk.next(a, seg)) {
            const int32_t* table_row = a.block_table + (size_t)seg.b * a.max_blocks;
            int blk_n = -1;
            float ks_n = 0.f, vs_n = 0.f;
            auto fetch = [&](int kt) {                     // box of tile kt + my_tile: block and scales
                const int p = (kt + my_tile) * BN + sb * kt_rows;
                blk_n = -1;
                if (kt + my_tile < seg.kt1 && p < seg.ctx) {
                    const int v = table_row[p / a.block_size];
                    if (v >= 0 && v < a.num_blocks) {
                        blk_n = v;
                        ks_n = a.k_scale[(size_t)v * a.n_kv_heads + seg.hk];
                        vs_n = a.v_scale[(size_t)v * a.n_kv_heads + seg.hk];
                    } else {
                        flag_status(a.status, LL_DEV_BAD_BLOCK);
                    }
                }
            };
            fetch(seg.kt0);
            for (int kb = seg.kt0; kb < seg.kt1 && ok; kb += tpb) {
                const int blk = blk_n;
                const float ks = ks_n, lv = f8_log2_scale(vs_n);
                if (kb + tpb < seg.kt1) fetch(kb + tpb);
                const int nt = min(tpb, seg.kt1 - kb);
                for (int t = 0; t < nt; ++t, ++it) {
                    const int st = it % STAGES;
                    const uint32_t ph = (uint32_t)(it / STAGES) & 1u;
                    bool go = true;
                    if (lane == 0) go = mbar_wait_bounded(&empty_bar[st], ph ^ 1u, &abort_s, a.status);
                    ok = __shfl_sync(0xffffffffu, (int)go, 0) != 0;
                    if (!ok) break;
                    const bool mine = my_tile == t;
                    const uint32_t have = __ballot_sync(0xffffffffu, mine && blk >= 0);
                    const int p = (kb + t) * BN + sb * kt_rows;
                    unsigned long long valid = 0;
                    if (mine && blk >= 0) {
                        const int nk = min(kt_rows, seg.ctx - p);
                        valid = (nk == 64 ? ~0ull : ((1ull << nk) - 1ull)) << (sb * kt_rows);
                    }
                    const uint32_t vlo = __reduce_or_sync(0xffffffffu, (uint32_t)valid);
                    const uint32_t vhi = __reduce_or_sync(0xffffffffu, (uint32_t)(valid >> 32));
                    if (mine)
                        for (int i = 0; i < kt_rows / 16; ++i)
                            scale_s[st][sb * (kt_rows / 16) + i] = blk >= 0 ? make_float2(ks, lv) : make_float2(0.f, 0.f);
                    if (lane == 0) valid_s[st] = ((unsigned long long)vhi << 32) | vlo;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_expect_tx(&full_bar[st], (uint32_t)__popc(have) * 2u * (uint32_t)(kt_rows * D));
                    __syncwarp();
                    if (mine && blk >= 0) {
                        const long long row = ((long long)blk * a.n_kv_heads + seg.hk) * a.block_size + (p % a.block_size);
                        const int line = (int)(row * D / 128);
                        const uint32_t off = (uint32_t)(st * TILE + sb * kt_rows * D);
                        tma_load_2d(sk + off, &tmK, 0, line, &full_bar[st]);
                        tma_load_2d(sv + off, &tmV, 0, line, &full_bar[st]);
                    }
                    issued |= 1u << st;
                    parity ^= 1u << st;
                }
            }
        }
        __syncwarp();
        if (lane == 0 && abort_s) {
            // wait (bounded) for the copies in flight before the CTA leaves
            volatile int never = 0;
            for (int st = 0; st < STAGES; ++st)
                if ((issued >> st) & 1u) mbar_wait_bounded(&full_bar[st], ((parity >> st) & 1u) ^ 1u, &never, nullptr);
        }
        __syncwarp();
        return;
    }

    // ---------------------------------------------------- consumers (warps 0-3)
    const int g = lane >> 2, cq = lane & 3;
    const float sl2 = a.scale * kLog2eF8;
    int it = 0;
    bool dead = false;
    while (walk.next(a, seg)) {
        // B fragments of Q^T, column g of tile nt = query head 8 nt + g.  The head dims are permuted alike
        // in Q and K: MMA step s gives k indices 2 cq + e and 2 cq + 8 + e (e = 0, 1) the dims
        // (D / 4) cq + 4 s + e and + 2 + e, so that lane cq reads D / 4 consecutive code bytes of a key.
        uint2 qf[NT][W];
        float qs[NT][2];                                   // per own column 2 cq + e: sl2 times the row's power of two
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            uint2 w[W];
            uint32_t m = 0;
#pragma unroll
            for (int s = 0; s < W; ++s) {
                w[s] = make_uint2(0u, 0u);
                if (r < G)
                    w[s] = *reinterpret_cast<const uint2*>(a.q + ((size_t)seg.b * a.n_heads + seg.hk * G + r) * D +
                                                           (D / 4) * cq + 4 * s);
                m = max(m, max(max(w[s].x & 0x7fffu, (w[s].x >> 16) & 0x7fffu),
                               max(w[s].y & 0x7fffu, (w[s].y >> 16) & 0x7fffu)));
            }
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // exponent of the row's largest element; a row of zeros, or with an infinity or NaN, stays as it is.  Below 2^-112
            // it is scaled as if at 2^-112, so that the factor taken out of it keeps 20 bits.
            int ex = max((int)(m >> 7) - 127, -112);
            if (m == 0u || m >= 0x7f80u) ex = 14;
            // two powers of two, since their product may leave float32's range
            const int e0 = (14 - ex) / 2, e1 = 14 - ex - e0;
            const float up0 = __uint_as_float((uint32_t)(e0 + 127) << 23), up1 = __uint_as_float((uint32_t)(e1 + 127) << 23);
#pragma unroll
            for (int s = 0; s < W; ++s) {
                qf[nt][s].x = pack_f16x2(bf16_lo(w[s].x) * up0 * up1, bf16_hi(w[s].x) * up0 * up1);
                qf[nt][s].y = pack_f16x2(bf16_lo(w[s].y) * up0 * up1, bf16_hi(w[s].y) * up0 * up1);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int exc = __shfl_sync(0xffffffffu, ex, 4 * (2 * cq + e));   // of query row 8 nt + 2 cq + e
                qs[nt][e] = scalbnf(sl2, exc - 14);
            }
        }
        // O^T: row r of tile t is head dim (D / 8)(r & 7) + 2 t + (r >> 3), column n of tile nt query head
        // 8 nt + n; per query column the running max m of the scores and t of score + log2 of the V scale (the bases of
        // the probabilities and of the terms that P V sums), and the lane's part of the sum l of the probabilities.
        float acc[NT][W][4];
        float m[NT][2], t[NT][2], l[NT][2];
        // A term is 2^(score + nb), terms times to_p are probabilities, for V scales of 2^lv_at.
        float nb[NT][2], to_p[NT][2], lv_at = INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < W; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
            m[nt][0] = m[nt][1] = t[nt][0] = t[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }
        for (int kt = seg.kt0; kt < seg.kt1 && !dead; ++kt, ++it) {
            const int st = it % STAGES;
            const uint32_t ph = (uint32_t)(it / STAGES) & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full_bar[st], ph, &abort_s, a.status))) {
                dead = true;
                break;
            }
            const uint32_t okmask = (uint32_t)(valid_s[st] >> (warp * 16)) & 0xffffu;
            if (okmask) {
                const uint8_t* ktile = sk + st * TILE;
                const uint8_t* vtile = sv + st * TILE;
                const float2 kv = scale_s[st][warp];
                // S^T = K Q^T: A rows g and g + 8 are the warp's keys g and g + 8.  Keys that are not cached
                // hold whatever was there; their scores are masked below.
                uint32_t kw[2][W];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int R = warp * 16 + j * 8 + g;
#pragma unroll
                    for (int c = 0; c < W / 4; ++c) {
                        const uint4 w = *reinterpret_cast<const uint4*>(ktile + f8_chunk<D>(R, cq * (D / 4) + 16 * c));
                        kw[j][4 * c] = w.x; kw[j][4 * c + 1] = w.y; kw[j][4 * c + 2] = w.z; kw[j][4 * c + 3] = w.w;
                    }
                }
                float s[NT][4];
                {
                    float sp[NT][2][4];                    // two accumulators halve the MMA chain
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) sp[nt][h][0] = sp[nt][h][1] = sp[nt][h][2] = sp[nt][h][3] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < W; ++ks) {
                        uint32_t af[4];
                        e4m3x4_to_f16x4(kw[0][ks], af[0], af[2]);
                        e4m3x4_to_f16x4(kw[1][ks], af[1], af[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(sp[nt][ks & 1], af, qf[nt][ks].x, qf[nt][ks].y);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[nt][j] = sp[nt][0][j] + sp[nt][1][j];
                }
                // lane: keys g (s[.][0..1]) and g + 8 (s[.][2..3]) of query columns 2 cq and 2 cq + 1
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = qs[nt][e] * kv.x;
                        s[nt][e] *= f;
                        s[nt][2 + e] *= f;
                    }
                if (okmask != 0xffffu) {
                    const bool v0 = (okmask >> g) & 1u, v1 = (okmask >> (g + 8)) & 1u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            s[nt][e] = v0 ? s[nt][e] : -INFINITY;
                            s[nt][2 + e] = v1 ? s[nt][2 + e] : -INFINITY;
                        }
                }
                // The bases of a column move only when a score or a term exceeds its base by more than 2^8, so that
                // terms stay below 2^8.  So the column's maximum over the lanes is looked for only then.
                const float lv = kv.y;
                bool grow = false, anew = lv != lv_at;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        grow = grow || fmaxf(s[nt][e], s[nt][2 + e]) > fminf(m[nt][e], t[nt][e] - lv) + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    anew = true;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(s[nt][e], s[nt][2 + e]);
#pragma unroll
                            for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                            if (mx > m[nt][e] + 8.f) {
                                l[nt][e] *= ex2_approx(m[nt][e] - mx);
                                m[nt][e] = mx;
                            }
                            const float tn = mx + lv > t[nt][e] + 8.f ? mx + lv : t[nt][e];
                            const float al = tn == t[nt][e] ? 1.f : ex2_approx(t[nt][e] - tn);
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                acc[nt][i][e] *= al;
                                acc[nt][i][e + 2] *= al;
                            }
                            t[nt][e] = tn;
                        }
                }
                if (anew) {
                    lv_at = lv;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mb = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
                            const float tb = (t[nt][e] == -INFINITY ? 0.f : t[nt][e]) - kF8Shift;
                            nb[nt][e] = fmaxf(lv, tb - mb - kF8Floor) - tb;
                            to_p[nt][e] = ex2_approx(-mb - nb[nt][e]);
                        }
                }
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float p00 = ex2_approx(s[nt][0] + nb[nt][0]), p01 = ex2_approx(s[nt][1] + nb[nt][1]);
                    const float p10 = ex2_approx(s[nt][2] + nb[nt][0]), p11 = ex2_approx(s[nt][3] + nb[nt][1]);
                    l[nt][0] += (p00 + p10) * to_p[nt][0];
                    l[nt][1] += (p01 + p11) * to_p[nt][1];
                    pb[nt][0] = movmatrix_trans(pack_f16x2(p00, p01));     // keys 0-7
                    pb[nt][1] = movmatrix_trans(pack_f16x2(p10, p11));     // keys 8-15
                }
                // O^T += V^T P^T: lane g reads D / 8 consecutive code bytes (dims) of each of its key rows
                // 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9 and byte-interleaves the rows of a key pair: word i gives
                // tiles 2 i and 2 i + 1.  Rows without a cached key count as zeros: 0 * NaN is not 0.
                uint32_t vw[4][W / 2];
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const int key = 2 * cq + (q4 & 1) + (q4 >> 1) * 8;
                    const int R = warp * 16 + key;
                    if constexpr (D == 128) {
                        const uint4 w = *reinterpret_cast<const uint4*>(vtile + f8_chunk<D>(R, 16 * g));
                        vw[q4][0] = w.x; vw[q4][1] = w.y; vw[q4][2] = w.z; vw[q4][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(vtile + f8_chunk<D>(R, 8 * g) + (g & 1) * 8);
                        vw[q4][0] = w.x; vw[q4][1] = w.y;
                    }
                    if (okmask != 0xffffu && !((okmask >> key) & 1u)) {
#pragma unroll
                        for (int i = 0; i < W / 2; ++i) vw[q4][i] = 0u;
                    }
                }
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    uint32_t x01, y01, x23, y23;
                    asm("prmt.b32 %0, %1, %2, 0x5140;" : "=r"(x01) : "r"(vw[0][i]), "r"(vw[1][i]));
                    asm("prmt.b32 %0, %1, %2, 0x7362;" : "=r"(y01) : "r"(vw[0][i]), "r"(vw[1][i]));
                    asm("prmt.b32 %0, %1, %2, 0x5140;" : "=r"(x23) : "r"(vw[2][i]), "r"(vw[3][i]));
                    asm("prmt.b32 %0, %1, %2, 0x7362;" : "=r"(y23) : "r"(vw[2][i]), "r"(vw[3][i]));
                    uint32_t at0[4], at1[4];
                    e4m3x4_to_f16x4(x01, at0[0], at0[1]);
                    e4m3x4_to_f16x4(x23, at0[2], at0[3]);
                    e4m3x4_to_f16x4(y01, at1[0], at1[1]);
                    e4m3x4_to_f16x4(y23, at1[2], at1[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16_16816(acc[nt][2 * i], at0, pb[nt][0], pb[nt][1]);
                        mma_f16_16816(acc[nt][2 * i + 1], at1, pb[nt][0], pb[nt][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty_bar[st]);
        }
        // ------------------------------------------------ the segment's end: merge the four warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
        asm volatile("bar.sync 1, 128;" ::: "memory");         // the last segment's readers of s_ml are done
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s_ml[warp][8 * nt + 2 * cq + e] = make_float2(m[nt][e], l[nt][e]);
                    s_t[warp][8 * nt + 2 * cq + e] = t[nt][e];
                }
            }
        const bool whole = seg.kt0 == 0 && seg.kt1 == seg.n_kt;
        // slot 0: the segment holds the share's first tile; 1: it is the share's last one
        const int slot = 2 * cta + (it == (int)(t_end - t_begin) && it > seg.kt1 - seg.kt0 ? 1 : 0);
        // 32 head dims at a time, four of each lane group g, so that the buffer leaves room for four stages in three CTAs per SM
#pragma unroll
        for (int rd = 0; rd < W / 2; ++rd) {
            if (rd > 0) asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 8 * nt + 2 * cq + (j & 1);
                        if (r < G) s_acc[(warp * G + r) * 32 + 4 * g + 2 * i + (j >> 1)] = acc[nt][2 * rd + i][j];
                    }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            for (int i = threadIdx.x; i < G * 8; i += NCONS) {
                const int r = i >> 3, gg = i & 7, col = (D / 8) * gg + 4 * rd;
                float M = -INFINITY, T = -INFINITY;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    M = fmaxf(M, s_ml[w][r].x);
                    T = fmaxf(T, s_t[w][r]);
                }
                const float base = (M == -INFINITY) ? 0.f : M, top = (T == -INFINITY) ? 0.f : T;
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
                float den = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 ml = s_ml[w][r];
                    const float f = exp2f(s_t[w][r] - top);
                    const float4 x = *reinterpret_cast<const float4*>(&s_acc[(w * G + r) * 32 + 4 * gg]);
                    num.x += f * x.x;
                    num.y += f * x.y;
                    num.z += f * x.z;
                    num.w += f * x.w;
                    den += exp2f(ml.x - base) * ml.y;
                }
                // no valid key: zeros.  2^(T - M - 6) as two factors, exact where it is a power of two
                const float ex = top - kF8Shift - base, ex0 = rintf(0.5f * ex), u0 = exp2f(ex0), u1 = exp2f(ex - ex0);
                const float inv = den == 0.f ? 0.f : 1.f / den;
                const float4 o = make_float4(num.x * inv * u0 * u1, num.y * inv * u0 * u1, num.z * inv * u0 * u1, num.w * inv * u0 * u1);
                if (whole) {
                    *reinterpret_cast<uint2*>(a.out + ((size_t)seg.b * a.n_heads + (size_t)seg.hk * G + r) * D + col) =
                        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                } else {
                    *reinterpret_cast<float4*>(a.part_o + ((size_t)slot * G + r) * D + col) = o;
                    if (col == 0) a.part_ml[(size_t)slot * G + r] = make_float2(M, den);
                }
            }
        }
    }
}

// The partials of the CTAs c0 .. c1 that share the n tiles of (sequence b, KV head hk), joined by the log-sum-exp; zeros
// where n = 0.  A thread has four head dims of a query head, and takes the partials four at a time, so that their
// loads are in flight together.  What it keeps is their mean so far, which stays in float32's range where the sum
// of large values would not.
constexpr int kF8JoinThreads = 256;
LL_DEVINL void f8_join(const AttnF8Args& a, int b, int hk, int n, int c0, int c1, int slot0) {
    const int G = a.n_heads / a.n_kv_heads, D = a.head_dim;
    __nv_bfloat16* out = a.out + ((size_t)b * a.n_heads + (size_t)hk * G) * D;
    for (int i = threadIdx.x; i < G * D / 4; i += kF8JoinThreads) {
        const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
        float M = -INFINITY, den = 0.f;
        float4 mean = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1 && n > 0; c += 4) {
            float2 ml[4];
            float4 o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const size_t pr = (size_t)(c + k == c0 ? slot0 : 2 * min(c + k, c1)) * G + r;
                ml[k] = c + k <= c1 ? a.part_ml[pr] : make_float2(-INFINITY, 0.f);
                o[k] = *reinterpret_cast<const float4*>(a.part_o + pr * D + col);
            }
            const float mn = fmaxf(M, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
            const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(M - base);
            float w[4], sum = den * old;
            const float before = sum;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = exp2f(ml[k].x - base) * ml[k].y;
                sum += w[k];
            }
            const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum), keep = before * inv;   // (2^-22 off: the weights need no more)
            mean.x *= keep;
            mean.y *= keep;
            mean.z *= keep;
            mean.w *= keep;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c + k > c1) break;
                const float part = w[k] * inv;
                mean.x += part * o[k].x;
                mean.y += part * o[k].y;
                mean.z += part * o[k].z;
                mean.w += part * o[k].w;
            }
            M = mn;
            den = sum;
        }
        *reinterpret_cast<uint2*>(out + (size_t)r * D + col) = make_uint2(pack_bf16x2(mean.x, mean.y), pack_bf16x2(mean.z, mean.w));
    }
}

// Joins what several CTAs of the grid of P shared, and writes zeros for sequences without a key.  Grid (KV head,
// sequence).
__global__ void __launch_bounds__(kF8JoinThreads) attn_decode_f8_join_kernel(const AttnF8Args a, int P) {
    __shared__ long long s_all[kF8JoinThreads / 32], s_before[kF8JoinThreads / 32];
    // The context lengths are no output of the kernel before this one, which itself waited for their writers
    // before it let this one start: they are read beside its end.
    const int hk = blockIdx.x, b = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long all = 0, before = 0;
    for (int i = threadIdx.x; i < a.batch; i += kF8JoinThreads) {
        const int n = f8_tiles(f8_context(a, i, false));
        all += n;
        if (i < b) before += n;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (lane == 0) {
        s_all[warp] = all;
        s_before[warp] = before;
    }
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int w = 0; w < kF8JoinThreads / 32; ++w) {
        all += s_all[w];
        before += s_before[w];
    }
    const int n = f8_tiles(f8_context(a, b, false));
    const long long total = all * a.n_kv_heads;
    const long long u0 = before * a.n_kv_heads + (long long)hk * n, u1 = u0 + n;
    const int c0 = n ? share_of(total, P, u0) : 0, c1 = n ? share_of(total, P, u1 - 1) : 0;
    // partial of CTA c: its slot 0 where the tiles reach the share's first, else its slot 1 (only the first CTA)
    const int slot0 = n ? 2 * c0 + (share_begin(total, P, c0) >= u0 ? 0 : 1) : 0;
    pdl_wait();
    pdl_trigger();
    if (n > 0 && c0 == c1) return;                         // one CTA had them all
    f8_join(a, b, hk, n, c0, c1, slot0);
}

// The same for more than 1024 sequences: every CTA adds up all contexts, so it takes a run of the sequences (65535 of
// them: 3.4 ms -> 0.16; for the 7B and 70B shapes this form costs 2 us more).
constexpr int kF8JoinRuns = 1024;
__global__ void __launch_bounds__(kF8JoinThreads) attn_decode_f8_join_runs_kernel(const AttnF8Args a, int P) {
    __shared__ long long s_all[kF8JoinThreads / 32], s_before[kF8JoinThreads / 32];
    const int hk = blockIdx.x, per = (a.batch + (int)gridDim.y - 1) / (int)gridDim.y;
    const int b0 = (int)blockIdx.y * per, b1 = min(b0 + per, a.batch);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long all = 0, before = 0;
    for (int i = threadIdx.x; i < a.batch; i += kF8JoinThreads) {
        const int n = f8_tiles(f8_context(a, i, false));
        all += n;
        if (i < b0) before += n;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (lane == 0) {
        s_all[warp] = all;
        s_before[warp] = before;
    }
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int w = 0; w < kF8JoinThreads / 32; ++w) {
        all += s_all[w];
        before += s_before[w];
    }
    const long long total = all * a.n_kv_heads;
    pdl_wait();
    pdl_trigger();
    for (int b = b0; b < b1; ++b) {
        const int n = f8_tiles(f8_context(a, b, false));
        const long long u0 = before * a.n_kv_heads + (long long)hk * n, u1 = u0 + n;
        const int c0 = n ? share_of(total, P, u0) : 0, c1 = n ? share_of(total, P, u1 - 1) : 0;
        const int slot0 = n ? 2 * c0 + (share_begin(total, P, c0) >= u0 ? 0 : 1) : 0;
        before += n;
        if (n == 0 || c0 != c1) f8_join(a, b, hk, n, c0, c1, slot0);
    }
}

int f8_ctas_per_sm(int G, int D) {
    const size_t smem = (size_t)2 * kF8Stages * kF8Tile * D + (size_t)4 * G * 32 * 4 + 1024;
    // an SM has 228 KB, a CTA takes 2.25 KB more for its static part and the system's
    return std::min(G <= 8 ? kF8MaxCtasPerSm : 2, (int)((228 * 1024) / (smem + 2304)));
}

template <int D, int NT>
cudaError_t decode_f8_for(const AttnF8Args& a, cudaStream_t stream) {
    const int G = a.n_heads / a.n_kv_heads;
    const size_t smem = (size_t)2 * kF8Stages * kF8Tile * D + (size_t)4 * G * 32 * 4 + 1024;
    const size_t smem_max = (size_t)2 * kF8Stages * kF8Tile * D + (size_t)4 * 8 * NT * 32 * 4 + 1024;
    const void* kernel = (const void*)attn_decode_f8_kernel<D, NT>;
    cudaError_t e = ensure_func_attr(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_max,
                                     "cudaFuncSetAttribute(attn_decode_f8_kernel)");
    if (e == cudaSuccess)
        e = ensure_func_attr(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared,
                             "cudaFuncSetAttribute(attn_decode_f8_kernel carveout)");
    if (e != cudaSuccess) return e;
    const int sms = std::min(device_sm_count(), kF8MaxSms);
    if (sms <= 0) return record(cudaErrorNoDevice, "attn_decode_f8");
    const long long most = (long long)a.batch * a.n_kv_heads *
                           (((long long)a.max_blocks * a.block_size + kF8Tile - 1) / kF8Tile);
    const int P = (int)std::min<long long>(most, (long long)sms * f8_ctas_per_sm(G, D));
    CUtensorMap tmK, tmV;
    const uint64_t lines = (uint64_t)a.num_blocks * a.n_kv_heads * a.block_size * D / 128;
    const uint32_t box = (uint32_t)(std::min(a.block_size, kF8Tile) * D / 128);
    if (!make_tmap_u8_sw128(&tmK, a.k_pool, lines, box) || !make_tmap_u8_sw128(&tmV, a.v_pool, lines, box))
        return cudaErrorInvalidValue;
    trace_before("attn_decode_f8", stream);
    e = launch_pdl(attn_decode_f8_kernel<D, NT>, dim3((unsigned)P), dim3(kF8Threads), smem, stream, 1, tmK, tmV, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "attn_decode_f8_kernel launch");
    trace_before("attn_decode_f8_join", stream);
    const dim3 grid((unsigned)a.n_kv_heads, (unsigned)std::min(a.batch, kF8JoinRuns));
    e = launch_pdl(a.batch > kF8JoinRuns ? attn_decode_f8_join_runs_kernel : attn_decode_f8_join_kernel, grid, dim3(kF8JoinThreads), 0,
                   stream, 1, a, P);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "attn_decode_f8_join_kernel launch");
}

}  // namespace

// Two partials per CTA, G rows each; the bound takes the largest grid on any device.
size_t attn_decode_f8_scratch_bytes(int batch, int n_heads, int n_kv_heads, int head_dim) {
    const int G = n_heads / n_kv_heads;
    const size_t rows = (size_t)2 * kF8MaxSms * f8_ctas_per_sm(G, head_dim) * G;
    (void)batch;
    return rows * head_dim * sizeof(float) + rows * sizeof(float2);
}

cudaError_t launch_attn_decode_f8(AttnF8Args a, void* workspace, cudaStream_t stream) {
    const int G = a.n_heads / a.n_kv_heads, D = a.head_dim;
    const size_t rows = (size_t)2 * kF8MaxSms * f8_ctas_per_sm(G, D) * G;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * D);
    if (D == 128) return G <= 8 ? decode_f8_for<128, 1>(a, stream) : decode_f8_for<128, 2>(a, stream);
    return G <= 8 ? decode_f8_for<64, 1>(a, stream) : decode_f8_for<64, 2>(a, stream);
}

}  // namespace ll
