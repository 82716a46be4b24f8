// Prefill attention over a paged cache of e4m3 codes with one scale per block and KV head, on the
// tcgen05 tensor cores: a ragged batch of new tokens, each attending causally to its own sequence.
//
// A work item is one KV head of one sequence and a tile of 128 query rows: floor(128 / G) consecutive
// tokens times the G query heads that share the KV head, so that a tile of keys is brought in and
// converted once for the whole group.  One CTA per item, 128 keys at a time up to the tile's last
// position, items with the most keys first.  Two CTAs share an SM (256 TMEM columns and 98 KB of shared
// memory each): while one computes its softmax the other has the tensor core, and one's start and end
// hide behind the other.
//
// Roles (288 threads):
//  * warps 0-3, softmax: one thread per query row.  First they stage Q in shared memory as FP16.  Per key
//    tile they read S from TMEM twice (row maximum; then probabilities), write P over S as FP16 and, where
//    the maximum has grown by more than 2^8, scale the running O in TMEM.  At the end O / l goes out.
//  * warps 4-7, keys and values: the codes come straight from global memory into registers, one tile
//    ahead (L2 mostly, since all row tiles of a KV head read the same codes), become FP16 and are stored as
//    the 128-byte-swizzled operand tiles.  There is one K and one V buffer: K of the next tile is stored
//    while the softmax works, V while the next S is computed.
//  * warp 8, one thread: S = Q K^T (both from shared memory), O += P V (P from TMEM).
//
// Precision.  Codes are exact in FP16.  A query row is scaled by a power of two so that its largest element
// lies in [2^14, 2^15); its factor and the block's K scale multiply the float32 score, 16 keys at a time
// (a block holds whole 16-key chunks), so they cost nothing per element but the multiply-add there already
// is.  P is one FP16 (relative error 2^-11, an eighth of the BF16 output's half step), relative to an
// exponent base that keeps it below 2^14.  V carries its block's scale relative to the largest scale of the
// item's keys, times 2^6: exact for powers of two down to 2^-21 of that scale (values below about 2^-31 of
// the largest are lost).  Row maxima, sums, S and O are float32.
#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kPfThreads = 288;
constexpr int kPfRows = 128;             // query rows per item
constexpr int kPfKeys = 128;             // keys per tile
constexpr int kPfChunks = kPfKeys / 16;
constexpr float kPfLog2e = 1.4426950408889634f;
constexpr int kPfShift = 6;              // V enters P V times 2^6
constexpr float kPfBase = 6.f;           // and P times 2^6

template <int D>
struct PfLayout {
    static constexpr uint32_t TILE = kPfRows * D * 2;       // [D / 64][128 rows][128 B] FP16
    static constexpr uint32_t OFF_Q = 0, OFF_K = TILE, OFF_V = 2 * TILE, TOTAL = 3 * TILE;
    static constexpr uint32_t TMEM_S = 0, TMEM_O = 128, TMEM_COLS = 256;
};

// kind::f16 instruction descriptor, FP16 A and B, float32 D; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// MN-major operand with the 128-byte swizzle (V as the B operand of P V): rows of 128 bytes hold 64 head
// dims of a key, the next 8 keys are 1024 bytes on, the next 64 head dims `mn_atom_stride` bytes on.
LL_DEVINL uint64_t pf_desc_mn(uint32_t smem_addr, uint32_t mn_atom_stride) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((mn_atom_stride >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

// byte offset of 16-byte chunk c (8 FP16) of row r in a swizzled tile
LL_DEVINL uint32_t pf_off(int r, int c) {
    return (uint32_t)(c >> 3) * (kPfRows * 128u) + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
}

LL_DEVINL void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

LL_DEVINL void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// What a work item covers: new tokens t0 .. t0 + nt - 1 of sequence b (rows tok0 + t of q), the first at
// position pos0; keys 0 .. kv_end - 1.
struct PfItem {
    int b, hk, tok0, nt, pos0, kv_end;
};

LL_DEVINL bool pf_item(const AttnF8Args& a, int n_mt, int tt, bool flag, PfItem& it) {
    // latest tiles (the most keys) first, KV heads fastest
    int i = blockIdx.x;
    it.hk = i % a.n_kv_heads;
    i /= a.n_kv_heads;
    it.b = i % a.batch;
    const int mt = n_mt - 1 - i / a.batch;
    const int c0 = a.cu_new[it.b], c1 = a.cu_new[it.b + 1], ctx = a.context_lens[it.b];
    const long long n = (long long)c1 - c0;
    if (n == 0) return false;
    if (c0 < 0 || n < 0 || c1 > a.tokens || n > a.max_new || n > ctx || ctx > a.max_blocks * a.block_size) {
        if (flag) flag_status(a.status, LL_DEV_BAD_POSITION);
        return false;
    }
    const int t0 = mt * tt;
    if (t0 >= n) return false;
    it.tok0 = c0 + t0;
    it.nt = min(tt, (int)n - t0);
    it.pos0 = ctx - (int)n + t0;
    it.kv_end = it.pos0 + it.nt;
    return true;
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 2) attn_prefill_f8_kernel(const AttnF8Args a, int n_mt, int tt) {
    using L = PfLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // per key tile j.  k_ready has a barrier per parity because the softmax threads wait for it too, and
    // tile j + 1 may be ready before the last of them has looked at tile j.
    __shared__ uint64_t q_ready, k_ready[2], v_ready, s_full, p_ready, pv_done, o_done, drain;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    __shared__ float ks_s[2][kPfChunks];                    // per parity and 16-key chunk: K scale
    __shared__ uint32_t ok_s[2];                            // per parity: bit c = chunk c is backed by a valid block
    __shared__ int vexp_w[4], vexp_s;                       // exponent of the item's largest V scale

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* status = a.status;
    if (threadIdx.x == 0) {
        mbar_init(&q_ready, 128);
        mbar_init(&k_ready[0], 128);
        mbar_init(&k_ready[1], 128);
        mbar_init(&v_ready, 128);
        mbar_init(&s_full, 1);
        mbar_init(&p_ready, 128);
        mbar_init(&pv_done, 1);
        mbar_init(&o_done, 1);
        mbar_init(&drain, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    PfItem it;
    if (!pf_item(a, n_mt, tt, threadIdx.x == 0, it)) return;
    if (warp == 8) {
        tmem_alloc(&tmem_base_s, L::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int G = a.n_heads / a.n_kv_heads;
    const int n_kt = (it.kv_end + kPfKeys - 1) / kPfKeys;

    if (warp == 8) {
        if (lane == 0) {
            // ------------------------------------------------ MMA issuer
            const uint32_t id_s = idesc_f16(kPfRows, kPfKeys, false);
            const uint32_t id_o = idesc_f16(kPfRows, D, true);
            const uint32_t sq = smem_u32(smem + L::OFF_Q), sk = smem_u32(smem + L::OFF_K), sv = smem_u32(smem + L::OFF_V);
            bool ok = mbar_wait_bounded(&q_ready, 0, &abort_s, status);
            for (int j = 0; j < n_kt && ok; ++j) {
                if (!mbar_wait_bounded(&k_ready[j & 1], (uint32_t)(j >> 1) & 1u, &abort_s, status)) break;
                tc_fence_after();
                // S overwrites P of tile j - 1: MMAs of one thread run in order
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (uint32_t)(kk >> 2) * (kPfRows * 128) + (uint32_t)(kk & 3) * 32;
                    tc_mma_bf16(tmem + L::TMEM_S, umma_desc_sw128(sq + off), umma_desc_sw128(sk + off), id_s, kk > 0 ? 1u : 0u);
                }
                tc_commit(&s_full);
                if (!mbar_wait_bounded(&v_ready, (uint32_t)j & 1u, &abort_s, status)) break;
                if (!mbar_wait_bounded(&p_ready, (uint32_t)j & 1u, &abort_s, status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kPfKeys / 16; ++kk)
                    tc_mma_bf16_ts(tmem + L::TMEM_O, tmem + L::TMEM_S + (uint32_t)kk * 8u,
                                   pf_desc_mn(sv + (uint32_t)kk * 2048u, kPfRows * 128), id_o, (j > 0 || kk > 0) ? 1u : 0u);
                tc_commit(&pv_done);
            }
            tc_commit(&o_done);
            tc_commit(&drain);
            volatile int never = 0;
            mbar_wait_bounded(&drain, 0, &never, status);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------- keys and values (warps 4-7)
        constexpr int LANES = D / 16, ROWS = 128 / LANES, PER = kPfKeys / ROWS;   // lanes per row, rows per step, steps
        const int tid = threadIdx.x - 128;
        const int c16 = tid % LANES, rsub = tid / LANES;
        const int32_t* table_row = a.block_table + (size_t)it.b * a.max_blocks;
        // lane c < 8 of each warp looks after 16-key chunk c of a tile: its block (-1: none) and scales
        auto block_of = [&](int j) {
            const int key = j * kPfKeys + (lane & 7) * 16;
            int blk = -1;
            if (key < it.kv_end) {
                blk = table_row[key / a.block_size];
                if (blk < 0 || blk >= a.num_blocks) {
                    flag_status(status, LL_DEV_BAD_BLOCK);
                    blk = -1;
                }
            }
            return blk;
        };
        auto scale_of = [&](const float* scales, int blk) {
            return blk >= 0 ? scales[(size_t)blk * a.n_kv_heads + it.hk] : 0.f;
        };
        auto load = [&](const uint8_t* pool, int j, int blk_lane, uint4 (&w)[PER]) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = i * ROWS + rsub, key = j * kPfKeys + r;
                const int blk = __shfl_sync(0xffffffffu, blk_lane, r >> 4);
                w[i] = make_uint4(0u, 0u, 0u, 0u);         // also rows that hold no key: 0 * stale stays 0
                if (blk >= 0 && key < it.kv_end)
                    w[i] = *reinterpret_cast<const uint4*>(
                        pool + (((size_t)blk * a.n_kv_heads + it.hk) * a.block_size + (key % a.block_size)) * D + c16 * 16);
            }
        };
        auto store = [&](uint8_t* tile, const uint4 (&w)[PER], bool scaled, float ratio_lane) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = i * ROWS + rsub;
                uint32_t h[8];
                e4m3x4_to_f16x4(w[i].x, h[0], h[1]);
                e4m3x4_to_f16x4(w[i].y, h[2], h[3]);
                e4m3x4_to_f16x4(w[i].z, h[4], h[5]);
                e4m3x4_to_f16x4(w[i].w, h[6], h[7]);
                if (scaled) {
                    const __half2 f = __float2half2_rn(__shfl_sync(0xffffffffu, ratio_lane, r >> 4));
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[x]), f);
                        h[x] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                }
                // the two 16-byte chunks, the upper half of the head dims starting with its second one: the
                // two halves' tiles share their banks
                const int c = 2 * c16, odd = (c >> 3) & 1;
                const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                *reinterpret_cast<uint4*>(tile + pf_off(r, c + odd)) = odd ? hi : lo;
                *reinterpret_cast<uint4*>(tile + pf_off(r, c + 1 - odd)) = odd ? lo : hi;
            }
            fence_async_smem();
        };
        uint4 kw[PER], vw[PER];
        int blk = block_of(0);
        load(a.k_pool, 0, blk, kw);
        load(a.v_pool, 0, blk, vw);
        float ks = scale_of(a.k_scale, blk), vs = scale_of(a.v_scale, blk);
        int E = 0;
        for (int j = 0; j < n_kt; ++j) {
            const int blk_next = j + 1 < n_kt ? block_of(j + 1) : -1;
            // (whole warps leave: the loads below shuffle)
            if (j > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(&s_full, (uint32_t)(j - 1) & 1u, &abort_s, status))) break;
            if (warp == 4) {
                const uint32_t m = __ballot_sync(0xffffffffu, blk >= 0);
                if (lane < kPfChunks) ks_s[j & 1][lane] = ks;
                if (lane == 0) ok_s[j & 1] = m & ((1u << kPfChunks) - 1u);
            }
            __syncwarp();
            store(smem + L::OFF_K, kw, false, 0.f);
            mbar_arrive(&k_ready[j & 1]);
            if (j + 1 < n_kt) load(a.k_pool, j + 1, blk_next, kw);
            if (j == 0) {
                // exponent of the largest V scale of the item's keys
                const int n = (it.kv_end + a.block_size - 1) / a.block_size;
                float top = 0.f;
                for (int i = tid; i < n; i += 128) {
                    const int x = table_row[i];
                    if (x >= 0 && x < a.num_blocks) top = fmaxf(top, a.v_scale[(size_t)x * a.n_kv_heads + it.hk]);
                }
                const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
                if (lane == 0) vexp_w[warp - 4] = (int)(bits >> 23) - 127;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                E = max(max(vexp_w[0], vexp_w[1]), max(vexp_w[2], vexp_w[3]));
                if (tid == 0) vexp_s = E;
            }
            if (j > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(&pv_done, (uint32_t)(j - 1) & 1u, &abort_s, status))) break;
            store(smem + L::OFF_V, vw, true, scalbnf(vs, kPfShift - E));
            mbar_arrive(&v_ready);
            if (j + 1 < n_kt) {
                load(a.v_pool, j + 1, blk_next, vw);
                ks = scale_of(a.k_scale, blk_next);
                vs = scale_of(a.v_scale, blk_next);
                blk = blk_next;
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- softmax (warps 0-3)
        const int r = threadIdx.x;                          // query row = TMEM lane
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const int tok = r / G, head = it.hk * G + r % G;
        const bool live = tok < it.nt;
        const size_t row = ((size_t)it.tok0 + tok) * a.n_heads + head;
        float qf;                                           // score factor but for the K scale
        {
            uint4 w[D / 8];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                w[c] = make_uint4(0u, 0u, 0u, 0u);
                if (live) w[c] = *reinterpret_cast<const uint4*>(a.q + row * D + c * 8);
                m = max(m, max(max(max(w[c].x & 0x7fffu, (w[c].x >> 16) & 0x7fffu), max(w[c].y & 0x7fffu, (w[c].y >> 16) & 0x7fffu)),
                               max(max(w[c].z & 0x7fffu, (w[c].z >> 16) & 0x7fffu), max(w[c].w & 0x7fffu, (w[c].w >> 16) & 0x7fffu))));
            }
            int ex = (int)(m >> 7) - 127;                   // zeros, infinities and NaN: as they are
            if (m == 0u || m >= 0x7f80u) ex = 14;
            const int e0 = (14 - ex) / 2, e1 = 14 - ex - e0;
            const float u0 = __uint_as_float((uint32_t)(e0 + 127) << 23), u1 = __uint_as_float((uint32_t)(e1 + 127) << 23);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                uint4 o;
                o.x = pack_f16x2(bf16_lo(w[c].x) * u0 * u1, bf16_hi(w[c].x) * u0 * u1);
                o.y = pack_f16x2(bf16_lo(w[c].y) * u0 * u1, bf16_hi(w[c].y) * u0 * u1);
                o.z = pack_f16x2(bf16_lo(w[c].z) * u0 * u1, bf16_hi(w[c].z) * u0 * u1);
                o.w = pack_f16x2(bf16_lo(w[c].w) * u0 * u1, bf16_hi(w[c].w) * u0 * u1);
                *reinterpret_cast<uint4*>(smem + L::OFF_Q + pf_off(r, c)) = o;
            }
            qf = scalbnf(a.scale * kPfLog2e, ex - 14);
            fence_async_smem();
            mbar_arrive(&q_ready);
        }
        const int my_pos = it.pos0 + tok;                   // rows beyond the tokens mask nothing that is kept
        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n_kt; ++j) {
            ok = mbar_wait_bounded(&k_ready[j & 1], (uint32_t)(j >> 1) & 1u, &abort_s, status) &&
                 mbar_wait_bounded(&s_full, (uint32_t)j & 1u, &abort_s, status);
            ok = __all_sync(0xffffffffu, ok);               // the TMEM accesses are warp-collective
            if (!ok) break;
            tc_fence_after();
            const uint32_t ts = tmem + lane_base + L::TMEM_S;
            const uint32_t chunks = ok_s[j & 1];
            const int last = my_pos - j * kPfKeys;          // last key of the tile that this row sees
            const bool full = __all_sync(0xffffffffu, last >= kPfKeys - 1 && chunks == (1u << kPfChunks) - 1u);
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < kPfKeys / 32; ++c) {
                float s[32];
                tmem_ld32(ts + (uint32_t)c * 32u, s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int ch = 2 * c + h;
                    float mc = -INFINITY;
                    if (full) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) mc = fmaxf(mc, s[16 * h + i]);
                    } else {
                        const int lim = (chunks >> ch) & 1u ? last - ch * 16 : -1;
#pragma unroll
                        for (int i = 0; i < 16; ++i) mc = i <= lim ? fmaxf(mc, s[16 * h + i]) : mc;
                    }
                    // factor >= 0; a row without a key here keeps -inf (0 * -inf would be NaN)
                    mx = fmaxf(mx, mc == -INFINITY ? mc : mc * (qf * ks_s[j & 1][ch]));
                }
            }
            const bool move = mx > m_used + 8.f;            // false while the row has no key
            if (__any_sync(0xffffffffu, move)) {
                const float f = move ? ex2_approx(m_used - mx) : 1.f;
                if (j > 0) {
                    // S of this tile is complete, so P V of the tile before is in O
                    const uint32_t to = tmem + lane_base + L::TMEM_O;
#pragma unroll
                    for (int c = 0; c < D; c += 16) {
                        float v[16];
                        uint32_t w[16];
                        tmem_ld16(to + (uint32_t)c, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i] * f);
                        tmem_st16(to + (uint32_t)c, w);
                    }
                }
                if (move) {
                    l *= f;
                    m_used = mx;
                }
            }
            const float base = (m_used == -INFINITY ? 0.f : m_used) - kPfBase;
            float rs = 0.f;
#pragma unroll
            for (int c = 0; c < kPfKeys / 32; ++c) {
                float s[32];
                tmem_ld32(ts + (uint32_t)c * 32u, s);
                uint32_t p[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int ch = 2 * c + h;
                    const float f = qf * ks_s[j & 1][ch];
                    const int lim = (chunks >> ch) & 1u ? last - ch * 16 : -1;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float p0 = ex2_approx(fmaf(s[16 * h + 2 * i], f, -base));
                        float p1 = ex2_approx(fmaf(s[16 * h + 2 * i + 1], f, -base));
                        if (!full) {
                            p0 = 2 * i <= lim ? p0 : 0.f;
                            p1 = 2 * i + 1 <= lim ? p1 : 0.f;
                        }
                        rs += p0 + p1;
                        p[8 * h + i] = pack_f16x2(p0, p1);
                    }
                }
                tmem_st16(ts + (uint32_t)c * 16u, p);       // over columns of S already read
            }
            l += rs;
            tc_fence_before();
            mbar_arrive(&p_ready);
        }
        ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&o_done, 0, &abort_s, status));
        if (ok) {
            tc_fence_after();
            // vexp_s was written before v_ready of tile 0, which the P V behind o_done waited for
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int E = *const_cast<volatile int*>(&vexp_s) - kPfShift;
            const float up = E < -126 ? 0.f : __uint_as_float((uint32_t)(E + 127) << 23);
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                float v[16];
                tmem_ld16(tmem + lane_base + L::TMEM_O + (uint32_t)c, v);
                if (live) {
                    uint4 o[2];
                    uint32_t x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = pack_bf16x2(v[2 * i] * inv * up, v[2 * i + 1] * inv * up);
                    o[0] = make_uint4(x[0], x[1], x[2], x[3]);
                    o[1] = make_uint4(x[4], x[5], x[6], x[7]);
                    uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + c);
                    dst[0] = o[0];
                    dst[1] = o[1];
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, L::TMEM_COLS);
}

template <int D>
cudaError_t prefill_f8_for(const AttnF8Args& a, cudaStream_t stream) {
    using L = PfLayout<D>;
    const size_t smem = L::TOTAL + 1024;
    const void* kernel = (const void*)attn_prefill_f8_kernel<D>;
    cudaError_t e = ensure_func_attr(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem,
                                     "cudaFuncSetAttribute(attn_prefill_f8_kernel)");
    if (e == cudaSuccess)
        e = ensure_func_attr(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared,
                             "cudaFuncSetAttribute(attn_prefill_f8_kernel carveout)");
    if (e != cudaSuccess) return e;
    const int tt = kPfRows / (a.n_heads / a.n_kv_heads);    // tokens per item
    const int n_mt = (a.max_new + tt - 1) / tt;
    const long long items = (long long)a.batch * n_mt * a.n_kv_heads;
    if (items > (1LL << 30)) {
        set_last_error("attn_prefill_f8", "too many (sequence, KV head, query tile) items");
        return cudaErrorInvalidValue;
    }
    trace_before("attn_prefill_f8", stream);
    e = launch_pdl(attn_prefill_f8_kernel<D>, dim3((unsigned)items), dim3(kPfThreads), smem, stream, 1, a, n_mt, tt);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "attn_prefill_f8_kernel launch");
}

}  // namespace

size_t attn_prefill_f8_scratch_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_attn_prefill_f8(const AttnF8Args& a, void* workspace, cudaStream_t stream) {
    (void)workspace;
    if (a.tokens <= 0) return cudaSuccess;
    return a.head_dim == 128 ? prefill_f8_for<128>(a, stream) : prefill_f8_for<64>(a, stream);
}

}  // namespace ll
