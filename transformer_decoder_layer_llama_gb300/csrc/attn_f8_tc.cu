// Prefill attention over a paged cache of e4m3 codes with one scale per block and KV head, on the
// tcgen05 tensor cores: a ragged batch of new tokens, each attending causally to its own sequence.
//
// A work item is one KV head of one sequence and two tiles (A, B) of 128 query rows each: a tile is
// floor(128 / G) consecutive tokens times the G query heads that share the KV head, so a tile of 128 keys is
// brought in and converted once for 256 rows.  The key tiles of all items form one list; each CTA of a
// persistent grid, one per SM, takes an equal run of it, whatever the lengths: a run that ends inside an item
// leaves a float32 partial (at most two per CTA), which the join kernel merges by the log-sum-exp.  So a
// single chunk behind a long prefix fills the GPU, and no SM waits for the longest item.
//
// Roles (512 threads):
//  * warps 0-3 and 4-7, softmax of tile A and B: one thread per query row.  They stage the item's Q in shared
//    memory as FP16 (the next item's before the output of the one before).  Per key tile: the row of S from
//    TMEM into registers, its maximum, probabilities written over S as FP16; where the maximum has grown by
//    more than 2^8 the running O in TMEM is scaled.  At the end O / l goes out.
//  * warps 8-11, keys and values: the codes come straight from global memory into registers, a tile
//    ahead (L2 mostly, since all items of a KV head read the same codes), become FP16 and are stored as the
//    128-byte-swizzled operand tiles, two buffers each for K and V.  Block ids are read two tiles ahead.
//  * warp 14, one thread: writes the run's segments (a run of key tiles of one item) to a ring that the other
//    roles read.
//  * warps 12 and 13, one thread each: S = Q K^T (both from shared memory) and O += P V (P from TMEM) of
//    tile A and B, so that the tensor core works for one tile while the other's softmax runs.  (One thread
//    for both spent as long between its groups of MMAs as in them.)
//
// Precision.  Codes are exact in FP16.  A query row is scaled by a power of two so that its largest element
// lies in [2^14, 2^15); its factor and the block's K scale multiply the float32 score, 16 keys at a time
// (a block holds whole 16-key chunks), so they cost nothing per element but the multiply-add there already
// is.  P is one FP16 (relative error 2^-11, an eighth of the BF16 output's half step), relative to an
// exponent base that keeps it below 2^14.  V carries its block's scale relative to the largest scale of the
// run's keys, times 2^6: exact for powers of two down to 2^-21 of that scale (values below about 2^-31 of
// the largest are lost).  Row maxima, sums, S and O are float32.
#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kPfThreads = 512;         // four groups of 128: the register split is set per group
constexpr int kPfRows = 128;             // query rows per tile
constexpr int kPfKeys = 128;             // keys per tile
constexpr int kPfChunks = kPfKeys / 16;
constexpr int kPfMeta = 4;               // tiles whose scales are kept
constexpr int kPfSegs = 4;               // segments in the ring
constexpr float kPfLog2e = 1.4426950408889634f;
constexpr int kPfShift = 6;              // V enters P V times 2^6
constexpr float kPfBase = 6.f;           // and P times 2^6

template <int D>
struct PfLayout {
    static constexpr uint32_t TILE = kPfRows * D * 2;       // [D / 64][128 rows][128 B] FP16
    static constexpr uint32_t OFF_Q = 0;                    // A, B
    static constexpr uint32_t OFF_K = 2 * TILE, OFF_V = 4 * TILE, TOTAL = 6 * TILE;   // two buffers each
    static constexpr uint32_t TMEM_S = 0, TMEM_O = 256, TMEM_COLS = 512;              // A, B 128 columns on
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

// 64 consecutive 32-bit TMEM columns of this thread's lane (warp-collective), without waiting; the values may
// be used behind tmem_wait_ld, which takes them through its operands so that no use can move before it.
LL_DEVINL void tmem_ld64_issue(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}
LL_DEVINL void tmem_wait_ld(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
          "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
          "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
          "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
          "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
        :
        : "memory");
}
// 8 columns, stored without waiting; tmem_wait_st waits for all of the thread's stores.
LL_DEVINL void tmem_st8_issue(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
LL_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// This thread's lane, 8 columns of TMEM times f (warp-collective).
LL_DEVINL void tmem_scale8(uint32_t taddr, float f) {
    asm volatile(
        "{\n .reg .f32 a<8>;\n .reg .b32 r<8>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {r0,r1,r2,r3,r4,r5,r6,r7}, [%0];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b32 a0, r0; mov.b32 a1, r1; mov.b32 a2, r2; mov.b32 a3, r3;\n"
        " mov.b32 a4, r4; mov.b32 a5, r5; mov.b32 a6, r6; mov.b32 a7, r7;\n"
        " mul.f32 a0, a0, %1; mul.f32 a1, a1, %1; mul.f32 a2, a2, %1; mul.f32 a3, a3, %1;\n"
        " mul.f32 a4, a4, %1; mul.f32 a5, a5, %1; mul.f32 a6, a6, %1; mul.f32 a7, a7, %1;\n"
        " mov.b32 r0, a0; mov.b32 r1, a1; mov.b32 r2, a2; mov.b32 r3, a3;\n"
        " mov.b32 r4, a4; mov.b32 r5, a5; mov.b32 r6, a6; mov.b32 r7, a7;\n"
        " tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {r0,r1,r2,r3,r4,r5,r6,r7};\n"
        " tcgen05.wait::st.sync.aligned;\n}\n" ::"r"(taddr),
        "f"(f)
        : "memory");
}

// Two float32 operations in one instruction.
LL_DEVINL float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
LL_DEVINL float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
LL_DEVINL float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 16 bytes of global memory that no kernel running now writes, or zeros: predicated, so that a run of such
// loads issues without branches.
LL_DEVINL uint4 load16_if(const void* p, bool take) {
    uint4 v;
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
        " @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)take)
        : "memory");
    return v;
}

// One lane of the (converged) warp, always the same.
LL_DEVINL bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// tcgen05.mma with descriptors in halves: within a tile only the low half (the address) changes.
LL_DEVINL void pf_mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate));
}
LL_DEVINL void pf_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 db;\n mov.b64 db, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate));
}

// The two issuing warps take turns on the tensor core (bounded as the barrier waits are); a turn is P V of
// a key tile with the S of the next.  Interleaved, or in smaller turns, both tiles' S are ready together: both
// softmaxes run at once and the tensor core waits for them.
LL_DEVINL bool turn_take(int* turn, volatile int* abort, int32_t* status) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; atomicCAS_block(turn, 0, 1) != 0; ++it) {
        if ((it & 255u) == 0) {
            if (*abort) return false;
            if (t0 == 0) t0 = global_timer_ns();
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                flag_status(status, LL_DEV_TIMEOUT);
                return false;
            }
        }
    }
    return true;
}
LL_DEVINL void turn_leave(int* turn) { atomicExch_block(turn, 0); }

// A whole 32-byte sector per thread.
LL_DEVINL void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// sum of floor((a i + b) / m) over i = 0 .. n - 1, by the Euclidean recurrence; a n + b < 2^32
LL_DEVINL long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    long long sum = 0;
    while (n > 0) {
        sum += (long long)((unsigned long long)n * (n - 1) / 2) * (a / m) + (long long)n * (b / m);
        a %= m;
        b %= m;
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// One sequence's new tokens: rows c0 .. c0 + n - 1 of q at positions ctx - n .. ctx - 1 (n = 0 where there
// are none, or where the counts do not fit together: flagged).  With step tokens per item, item mt sees
// keys below pos0 + min((mt + 1) step, n).
struct PfSeq {
    int c0, n, pos0;
};
LL_DEVINL PfSeq pf_seq(const AttnF8Args& a, int b, bool flag) {
    PfSeq s;
    s.c0 = a.cu_new[b];
    const int c1 = a.cu_new[b + 1], ctx = a.context_lens[b];
    const long long n = (long long)c1 - s.c0;
    const bool bad = s.c0 < 0 || n < 0 || c1 > a.tokens || n > a.max_new || n > ctx || ctx > a.max_blocks * a.block_size;
    if (bad && n != 0 && flag) flag_status(a.status, LL_DEV_BAD_POSITION);
    s.n = bad ? 0 : (int)n;
    s.pos0 = ctx - s.n;
    return s;
}
LL_DEVINL int pf_items(const PfSeq& s, int step) { return (s.n + step - 1) / step; }
// key tiles of the items before item mt (mt <= items); all items but the last are full
LL_DEVINL long long pf_tiles_before(const PfSeq& s, int step, int mt) {
    const int full = min(mt, s.n / step);
    long long t = floor_sum((uint32_t)full, kPfKeys, (uint32_t)step, (uint32_t)(s.pos0 + step + kPfKeys - 1));
    if (mt > full) t += (s.pos0 + s.n + kPfKeys - 1) / kPfKeys;
    return t;
}

// A place in the list of key tiles: items in the order sequence, KV head, query tiles.
struct PfPlace {
    int b, hk, mt, j;
};

struct PfRun {
    PfPlace at, to;          // where the run begins and ends (valid where that is before the list's end)
    long long begin, end, total;
};

// Key tiles of an item's edge that a run does not split off: a few tiles more or less cost less than a partial.
constexpr int kPfSnap = 2;

// The run of CTA c of P, found by a whole block of nt threads (a multiple of 32, at most 512): the runs are
// equal but for the snap to item edges.
LL_DEVINL void pf_find_run(const AttnF8Args& a, int step, int P, int c, int nt, bool flag, PfRun* out) {
    __shared__ long long sums[16];
    __shared__ PfPlace place[2];
    __shared__ long long place_t[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.batch + nt - 1) / nt;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const PfSeq s = pf_seq(a, b, flag);
        mine += pf_tiles_before(s, step, pf_items(s, step));
    }
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    if (tid < 2) place_t[tid] = -1;
    __syncthreads();
    long long before = x - mine, total = 0;
    for (int w = 0; w < nt / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    before *= a.n_kv_heads;
    total *= a.n_kv_heads;
    const long long q = total / P, r = total - q * P;
    for (int e = 0; e < 2; ++e) {
        const long long t = q * (c + e) + min((long long)(c + e), r);   // the boundary, before the snap
        if (t >= total) {
            if (tid == 0) place_t[e] = total;
        } else if (t >= before && t < before + mine * a.n_kv_heads) {
            long long at = before;
            for (int b = b0; b < b1; ++b) {
                const PfSeq s = pf_seq(a, b, false);
                const int items = pf_items(s, step);
                const long long per_head = pf_tiles_before(s, step, items);
                if (t >= at + per_head * a.n_kv_heads) {
                    at += per_head * a.n_kv_heads;
                    continue;
                }
                PfPlace p;
                p.b = b;
                p.hk = (int)((t - at) / per_head);
                const long long rest = t - at - (long long)p.hk * per_head;
                int lo = 0, hi = items;                    // the item: last one that begins at or before rest
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (pf_tiles_before(s, step, mid) <= rest) lo = mid;
                    else hi = mid;
                }
                p.mt = lo;
                p.j = (int)(rest - pf_tiles_before(s, step, lo));
                const int n_kt = (s.pos0 + min((lo + 1) * step, s.n) + kPfKeys - 1) / kPfKeys;
                long long snapped = t;
                if (p.j <= kPfSnap) {
                    snapped -= p.j;
                    p.j = 0;
                } else if (n_kt - p.j <= kPfSnap) {
                    snapped += n_kt - p.j;
                    p.j = n_kt;                            // (the walk goes on to the next item)
                }
                place[e] = p;
                place_t[e] = snapped;
                break;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        out->at = place[0];
        out->to = place[1];
        out->begin = place_t[0];
        out->end = place_t[1];
        out->total = total;
    }
    __syncthreads();
}

// A run of key tiles j0 .. j1 - 1 (of n_kt) of one item: nt_a and nt_b tokens in the query tiles (rows tok0 + t
// of q, the first at position pos0), which see keys 0 .. end_a - 1 and 0 .. end_b - 1 (0: no tile B).
struct PfSegment {
    int b;                   // -1: the run is over
    int hk, tok0, pos0, nt_a, nt_b, end_a, end_b, j0, j1, n_kt;
};

struct PfWalk {
    PfPlace at;
    long long left;          // key tiles of the run still to do
    LL_DEVINL bool next(const AttnF8Args& a, int tt, PfSegment& g) {
        while (left > 0) {
            const PfSeq s = pf_seq(a, at.b, false);
            const int t0 = at.mt * 2 * tt;
            if (t0 >= s.n) {                  // past the sequence's items: the next head, or sequence
                at.mt = 0;
                at.j = 0;
                if (s.n == 0 || ++at.hk == a.n_kv_heads) {
                    at.hk = 0;
                    ++at.b;
                }
                continue;
            }
            const int rest = s.n - t0;
            g.b = at.b;
            g.hk = at.hk;
            g.tok0 = s.c0 + t0;
            g.pos0 = s.pos0 + t0;
            g.nt_a = min(tt, rest);
            g.nt_b = min(tt, rest - g.nt_a);
            g.end_a = g.pos0 + g.nt_a;
            g.end_b = g.nt_b ? g.end_a + g.nt_b : 0;
            g.n_kt = (max(g.end_a, g.end_b) + kPfKeys - 1) / kPfKeys;
            if (at.j >= g.n_kt) {
                at.j = 0;
                ++at.mt;
                continue;
            }
            g.j0 = at.j;
            g.j1 = (int)min((long long)g.n_kt, g.j0 + left);
            left -= g.j1 - g.j0;
            at.j = g.j1;
            return true;
        }
        return false;
    }
};
// one past the last key tile of the segment that query tile x works on
LL_DEVINL int pf_end(const PfSegment& g, int x) {
    return min(g.j1, ((x ? g.end_b : g.end_a) + kPfKeys - 1) / kPfKeys);
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) attn_prefill_f8_kernel(const AttnF8Args a, int tt) {
    using L = PfLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // Per query tile x, counted over the key tiles it works on: S computed, P stored; over its segments: Q
    // staged, O complete, O read.  Per key buffer, counted over all key tiles: K or V stored (ready), read by
    // both query tiles (empty).  The scales of key tile i of the run sit in slot i & 3: slot and barrier are
    // written again for tile i + 4, after the S of tile i + 2, which waits for the P of tile i + 1.
    __shared__ uint64_t q_ready[2], s_full[2], p_ready[2], o_done[2], o_free[2], k_ready[2], k_empty[2], v_ready[2], v_empty[2];
    __shared__ uint64_t meta_ready[kPfMeta], drain[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, turn_s;
    __shared__ __align__(16) float ks_s[kPfMeta][kPfChunks];   // per 16-key chunk: K scale
    __shared__ uint32_t ok_s[kPfMeta];                      // bit c = chunk c is backed by a valid block
    __shared__ int vexp_s[kPfMeta], vexp_w[2][4];           // exponent of the segment's largest V scale
    __shared__ PfRun run_s;
    __shared__ uint64_t seg_ready[kPfSegs], seg_empty[kPfSegs];
    __shared__ PfSegment seg_s[kPfSegs];
    __shared__ struct {
        long long row0;      // q and out row of the tile's first query row
        int nt, part;        // tokens; partial slot (-1: the whole item)
        int exp, next;       // exponent of V; the run's key tile that the query tile goes on with
    } out_s[8];              // per softmax warp

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* status = a.status;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPfSegs; ++i) {
            mbar_init(&seg_ready[i], 1);
            mbar_init(&seg_empty[i], 14);                   // 8 softmax warps, 4 for keys and values, 2 issuers
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_ready[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&o_free[i], 4);
            mbar_init(&k_ready[i], 4);
            mbar_init(&k_empty[i], 2);
            mbar_init(&v_ready[i], 4);
            mbar_init(&v_empty[i], 2);
            mbar_init(&drain[i], 1);
        }
        for (int i = 0; i < kPfMeta; ++i) mbar_init(&meta_ready[i], 1);
        abort_s = 0;
        turn_s = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(&tmem_base_s, L::TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    pf_find_run(a, 2 * tt, (int)gridDim.x, (int)blockIdx.x, kPfThreads, blockIdx.x == 0, &run_s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int G = a.n_heads / a.n_kv_heads;
    // segment k of the run; false after a timeout
    auto seg_wait = [&](int k) {
        return mbar_wait_bounded(&seg_ready[k & (kPfSegs - 1)], (uint32_t)(k / kPfSegs) & 1u, &abort_s, status);
    };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 14 && lane == 0) {
            // ------------------------------------------------ segments of the run
            PfWalk walk{run_s.at, run_s.end - run_s.begin};
            for (int k = 0;; ++k) {
                PfSegment& g = seg_s[k & (kPfSegs - 1)];
                if (k >= kPfSegs && !mbar_wait_bounded(&seg_empty[k & (kPfSegs - 1)], (uint32_t)(k / kPfSegs - 1) & 1u, &abort_s, status))
                    break;
                const bool some = walk.next(a, tt, g);
                if (!some) g.b = -1;
                mbar_arrive(&seg_ready[k & (kPfSegs - 1)]);
                if (!some) break;
            }
        } else if (warp < 14) {
            // ------------------------------------------------ MMA issuers: warp 12 for tile A, 13 for B
            // The whole warp walks along, one lane issues: addresses stay in uniform registers.  (One thread on a
            // path of its own took twice an MMA's time to issue the next.)
            const int x = warp - 12;
            constexpr uint32_t id_s = idesc_f16(kPfRows, kPfKeys, false), id_o = idesc_f16(kPfRows, D, true);
            const uint64_t dq = umma_desc_sw128(smem_u32(smem + L::OFF_Q) + (uint32_t)x * L::TILE);
            const uint64_t dk = umma_desc_sw128(smem_u32(smem + L::OFF_K));
            const uint64_t dv = pf_desc_mn(smem_u32(smem + L::OFF_V), kPfRows * 128);
            const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32), k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32);
            const uint32_t v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
            const uint32_t t_s = tmem + L::TMEM_S + (uint32_t)x * 128u, t_o = tmem + L::TMEM_O + (uint32_t)x * 128u;
            // key tile i of the run
            auto k_wait = [&](int i) { return mbar_wait_bounded(&k_ready[i & 1], (uint32_t)(i >> 1) & 1u, &abort_s, status); };
            auto v_wait = [&](int i) { return mbar_wait_bounded(&v_ready[i & 1], (uint32_t)(i >> 1) & 1u, &abort_s, status); };
            auto take = [&](bool good) {                    // (all lanes' waits went well, and the turn is the warp's)
                good = __all_sync(0xffffffffu, good);
                if (good && lane == 0) good = turn_take(&turn_s, &abort_s, status);
                good = __all_sync(0xffffffffu, good);
                tc_fence_after();
                return good;
            };
            // S of a key tile, over P of the one before (MMAs of one thread run in order); by the elected lane
            auto issue_s = [&](int i) {
                const uint32_t b = k_lo + (uint32_t)(i & 1) * (L::TILE >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    // the descriptor's address field counts 16 bytes
                    const uint32_t off = ((uint32_t)(kk >> 2) * (kPfRows * 128) + (uint32_t)(kk & 3) * 32) >> 4;
                    pf_mma_ss(t_s, q_lo + off, q_hi, b + off, k_hi, id_s, kk > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[x]);
            };
            auto issue_pv = [&](int i, bool first) {
                const uint32_t b = v_lo + (uint32_t)(i & 1) * (L::TILE >> 4);
#pragma unroll
                for (int kk = 0; kk < kPfKeys / 16; ++kk)
                    pf_mma_ts(t_o, t_s + (uint32_t)kk * 8u, b + (uint32_t)(kk * 2048 >> 4), v_hi, id_o, !first || kk > 0 ? 1u : 0u);
            };
            int i = 0;                                      // key tiles of the run so far
            uint32_t p_par = 0;                             // parity of this query tile's key tiles
            int segs = 0;                                   // and its segments
            bool ok = true;
            for (int k = 0;; ++k) {
                ok = __all_sync(0xffffffffu, seg_wait(k));
                const PfSegment& seg = seg_s[k & (kPfSegs - 1)];
                if (!ok || seg.b < 0) break;
                const int n = max(pf_end(seg, x) - seg.j0, 0), pass = seg.j1 - seg.j0 - n;
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[k & (kPfSegs - 1)]);   // (its numbers are taken)
                if (n > 0) {
                    ok = take(mbar_wait_bounded(&q_ready[x], (uint32_t)segs & 1u, &abort_s, status) && k_wait(i));
                    if (!ok) break;
                    if (elect_one()) {
                        issue_s(i);
                        turn_leave(&turn_s);
                        tc_commit(&k_empty[i & 1]);
                    }
                    __syncwarp();
                }
                // the segment before this one has been read out of O: before O is overwritten, and before buffers
                // pass on unseen by this tile
                ok = segs == 0 || __all_sync(0xffffffffu, mbar_wait_bounded(&o_free[x], (uint32_t)(segs - 1) & 1u, &abort_s, status));
                for (int j = 0; j < n && ok; ++j, ++i, p_par ^= 1u) {
                    // (what is usually there already is waited for first, beside the softmax)
                    const bool more = j + 1 < n;
                    ok = take(v_wait(i) && (!more || k_wait(i + 1)) && mbar_wait_bounded(&p_ready[x], p_par, &abort_s, status));
                    if (!ok) break;
                    if (elect_one()) {
                        issue_pv(i, j == 0);
                        if (more) issue_s(i + 1);
                        turn_leave(&turn_s);
                        tc_commit(&v_empty[i & 1]);
                        if (more) tc_commit(&k_empty[(i + 1) & 1]);
                        else tc_commit(&o_done[x]);
                    }
                    __syncwarp();
                }
                // key tiles that only the other query tile works on
                for (int j = 0; j < pass && ok; ++j, ++i) {
                    ok = __all_sync(0xffffffffu, k_wait(i) && v_wait(i));
                    if (ok && lane == 0) {
                        mbar_arrive(&k_empty[i & 1]);
                        mbar_arrive(&v_empty[i & 1]);
                    }
                }
                if (!ok) break;
                if (n > 0) ++segs;
            }
            if (elect_one()) {
                tc_commit(&drain[x]);
                volatile int never = 0;
                mbar_wait_bounded(&drain[x], 0, &never, status);
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---------------------------------------------------- keys and values (warps 8-11)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        constexpr int LANES = D / 16, ROWS = 128 / LANES, PER = kPfKeys / ROWS;   // lanes per row, rows per step, steps
        const int tid = threadIdx.x - 256;
        // Eight lanes that store together cover four 16-code pieces of two rows: their 16-byte chunks are 0, 2,
        // 4, 6 of an even and an odd row, which the swizzle puts on different banks.
        const int c16 = D == 128 ? (tid & 3) | ((tid >> 1) & 4) : tid & 3;
        const int rsub = D == 128 ? ((tid >> 2) & 1) | ((tid >> 3) & ~1) : tid >> 2;
        const int my_key = (lane & 7) * 16;                 // lane c < 8 looks after 16-key chunk c of a tile
        const int bs_log2 = 31 - __clz(a.block_size);       // (a power of two: no divisions on this path)
        const int32_t* table_row = nullptr;
        int kv_end = 0, hk = 0, j1 = 0;                     // of the segment
        auto entry_of = [&](int j) {                        // its table entry (-1 past the keys)
            const int key = j * kPfKeys + my_key;
            return j < j1 && key < kv_end ? table_row[key >> bs_log2] : -1;
        };
        auto row_of = [&](int j, int entry) {               // its first pool row (-1: no valid block)
            const int key = j * kPfKeys + my_key;
            const bool want = j < j1 && key < kv_end;
            if (want && (entry < 0 || entry >= a.num_blocks)) flag_status(status, LL_DEV_BAD_BLOCK);
            return want && entry >= 0 && entry < a.num_blocks
                       ? ((entry * a.n_kv_heads + hk) << bs_log2) + (key & (a.block_size - 1)) : -1;
        };
        auto scale_of = [&](const float* scales, int row) {
            return row >= 0 ? scales[row >> bs_log2] : 0.f;
        };
        auto load = [&](const uint8_t* pool, int j, int row_lane, uint4 (&w)[PER]) {
            const int left = kv_end - j * kPfKeys;          // keys of the tile
            int row[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) row[i] = __shfl_sync(0xffffffffu, row_lane, (i * ROWS + rsub) >> 4);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = i * ROWS + rsub;             // rows that hold no key become zeros: 0 * stale stays 0
                w[i] = load16_if(pool + (size_t)(uint32_t)(row[i] + (r & 15)) * D + c16 * 16, row[i] >= 0 && r < left);
            }
        };
        const uint32_t st0 = pf_off(rsub, 2 * c16), st1 = pf_off(rsub, 2 * c16 + 1);
        auto store = [&](uint8_t* tile, const uint4 (&w)[PER], bool scaled, float ratio_lane) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                uint32_t h[8];
                e4m3x4_to_f16x4(w[i].x, h[0], h[1]);
                e4m3x4_to_f16x4(w[i].y, h[2], h[3]);
                e4m3x4_to_f16x4(w[i].z, h[4], h[5]);
                e4m3x4_to_f16x4(w[i].w, h[6], h[7]);
                if (scaled) {
                    const __half2 f = __float2half2_rn(__shfl_sync(0xffffffffu, ratio_lane, (i * ROWS + rsub) >> 4));
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[x]), f);
                        h[x] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                }
                *reinterpret_cast<uint4*>(tile + st0 + i * ROWS * 128) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(tile + st1 + i * ROWS * 128) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_async_smem();
            __syncwarp();
        };
        int i = 0;                                          // key tiles of the run so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = __all_sync(0xffffffffu, seg_wait(k));
            const PfSegment& seg = seg_s[k & (kPfSegs - 1)];
            if (!ok || seg.b < 0) break;
            table_row = a.block_table + (size_t)seg.b * a.max_blocks;
            kv_end = max(seg.end_a, seg.end_b);
            hk = seg.hk;
            const int j0 = seg.j0;
            j1 = seg.j1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[k & (kPfSegs - 1)]);
            uint4 kw[PER], vw[PER];
            int row = row_of(j0, entry_of(j0));
            int entry = entry_of(j0 + 1);               // of the tile after the one in registers
            load(a.k_pool, j0, row, kw);
            load(a.v_pool, j0, row, vw);
            float ks = scale_of(a.k_scale, row), vs = scale_of(a.v_scale, row);
            // exponent of the largest V scale of the segment's keys
            float top = 0.f;
            const int e1 = (min(j1 * kPfKeys, kv_end) + a.block_size - 1) >> bs_log2;
            for (int e = (j0 * kPfKeys >> bs_log2) + tid; e < e1; e += 128) {
                const int x = table_row[e];
                if (x >= 0 && x < a.num_blocks) top = fmaxf(top, a.v_scale[(size_t)x * a.n_kv_heads + hk]);
            }
            const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            if (lane == 0) vexp_w[k & 1][warp - 8] = (int)(bits >> 23) - 127;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int E = max(max(vexp_w[k & 1][0], vexp_w[k & 1][1]), max(vexp_w[k & 1][2], vexp_w[k & 1][3]));
            const int h0 = (kPfShift - E) / 2, h1 = kPfShift - E - h0;
            const float up0 = __uint_as_float((uint32_t)(h0 + 127) << 23), up1 = __uint_as_float((uint32_t)(h1 + 127) << 23);
            for (int j = j0; j < j1; ++j, ++i) {
                // (whole warps leave: the loads below shuffle)
                ok = i < 2 || __all_sync(0xffffffffu, mbar_wait_bounded(&k_empty[i & 1], (uint32_t)((i - 2) >> 1) & 1u, &abort_s, status));
                if (!ok) break;
                store(smem + L::OFF_K + (uint32_t)(i & 1) * L::TILE, kw, false, 0.f);
                if (warp == 8) {
                    const int slot = i & (kPfMeta - 1);
                    const uint32_t m = __ballot_sync(0xffffffffu, row >= 0);
                    if (lane < kPfChunks) ks_s[slot][lane] = ks;
                    if (lane == 0) {
                        ok_s[slot] = m & ((1u << kPfChunks) - 1u);
                        vexp_s[slot] = E;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&meta_ready[slot]);
                }
                if (lane == 0) mbar_arrive(&k_ready[i & 1]);
                // Each value is loaded into the variable whose last use is behind it: a copy at the loop's end
                // would wait for the load.
                row = row_of(j + 1, entry);
                entry = entry_of(j + 2);
                load(a.k_pool, j + 1, row, kw);
                ks = scale_of(a.k_scale, row);
                ok = i < 2 || __all_sync(0xffffffffu, mbar_wait_bounded(&v_empty[i & 1], (uint32_t)((i - 2) >> 1) & 1u, &abort_s, status));
                if (!ok) break;
                store(smem + L::OFF_V + (uint32_t)(i & 1) * L::TILE, vw, true, vs * up0 * up1);
                if (lane == 0) mbar_arrive(&v_ready[i & 1]);
                load(a.v_pool, j + 1, row, vw);
                vs = scale_of(a.v_scale, row);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- softmax (warps 0-3: tile A, 4-7: tile B)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int x = warp >> 2;
        const int r = threadIdx.x & 127;                    // query row = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t per_g = 65536u / (uint32_t)G + 1u;   // r / G = r * per_g >> 16 for r < 128
        const uint32_t ts = tmem + lane_base + L::TMEM_S + (uint32_t)x * 128u;
        const uint32_t to = tmem + lane_base + L::TMEM_O + (uint32_t)x * 128u;
        uint8_t* const sq = smem + L::OFF_Q + (uint32_t)x * L::TILE;
        // The warp's 32 rows of an item's Q on their way to their places in shared memory, as they are: D / 8 lanes
        // take a row, 16 bytes each.  (Rolled loops here, in scale_q and at the output: code that runs once per
        // item displaces the loop that matters.)
        auto fetch_q = [&](const PfSegment& g) {
            constexpr int QL = D / 8, QR = 32 / QL;         // lanes per row, rows per step
            const int c = lane % QL, nt = x ? g.nt_b : g.nt_a;
            const size_t row0 = ((size_t)g.tok0 + x * tt) * a.n_heads + g.hk * G;
#pragma unroll 4
            for (int rr = (warp & 3) * 32 + lane / QL; rr < (warp & 3) * 32 + 32; rr += QR) {
                const int tok = (int)((uint32_t)rr * per_g >> 16);
                const bool take = tok < nt;
                cp_async16(sq + pf_off(rr, c), a.q + (take ? (row0 + (size_t)tok * a.n_heads + (rr - tok * G)) * D + c * 8 : 0), take);
            }
            cp_async_commit();
        };
        // Then each thread turns its own row into FP16, scaled so that its largest element lies in [2^14, 2^15).
        // Returns the row's score factor, but for the K scale.
        auto scale_q = [&]() {
            cp_async_wait<0>();
            __syncwarp();
            uint32_t m = 0;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 w = *reinterpret_cast<const uint4*>(sq + pf_off(r, c));
                m = max(m, max(max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu), max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu)),
                               max(max(w.z & 0x7fffu, (w.z >> 16) & 0x7fffu), max(w.w & 0x7fffu, (w.w >> 16) & 0x7fffu))));
            }
            int ex = (int)(m >> 7) - 127;                   // zeros, infinities and NaN: as they are
            if (m == 0u || m >= 0x7f80u) ex = 14;
            const int e0 = (14 - ex) / 2, e1 = 14 - ex - e0;
            const float u0 = __uint_as_float((uint32_t)(e0 + 127) << 23), u1 = __uint_as_float((uint32_t)(e1 + 127) << 23);
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                uint4* at = reinterpret_cast<uint4*>(sq + pf_off(r, c));
                const uint4 w = *at;
                uint4 o;
                o.x = pack_f16x2(bf16_lo(w.x) * u0 * u1, bf16_hi(w.x) * u0 * u1);
                o.y = pack_f16x2(bf16_lo(w.y) * u0 * u1, bf16_hi(w.y) * u0 * u1);
                o.z = pack_f16x2(bf16_lo(w.z) * u0 * u1, bf16_hi(w.z) * u0 * u1);
                o.w = pack_f16x2(bf16_lo(w.w) * u0 * u1, bf16_hi(w.w) * u0 * u1);
                *at = o;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[x]);
            return scalbnf(a.scale * kPfLog2e, ex - 14);
        };
        int i = 0, k = 0;                                   // key tile of the run, segment in hand
        uint32_t s_par = 0, o_par = 0;                      // parity of this query tile's key tiles and segments
        bool more = false, ok = true;
        auto done_with = [&](int kk) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[kk & (kPfSegs - 1)]);
        };
        // on to segment k, and past those that this query tile has no keys in; i: its first key tile
        auto find = [&]() {
            for (;; ++k) {
                ok = ok && __all_sync(0xffffffffu, seg_wait(k));
                const PfSegment& g = seg_s[k & (kPfSegs - 1)];
                more = ok && g.b >= 0;
                if (!more || pf_end(g, x) > g.j0) return;
                // (a segment without keys for tile A is the end of an item: it still owes a partial)
                if ((x ? g.nt_b : g.nt_a) > 0)
                    a.part_ml[(size_t)(2 * (int)blockIdx.x + (i > 0 ? 1 : 0)) * 2 * kPfRows + x * kPfRows + r] = make_float2(-INFINITY, 0.f);
                i += g.j1 - g.j0;
                done_with(k);
            }
        };
        find();
        float qf = 0.f;
        if (more) {
            fetch_q(seg_s[k & (kPfSegs - 1)]);
            qf = scale_q();
        }
        while (more && ok) {
            int last, left;                                 // last key of the tile that this row sees; tiles after this one
            bool first = true;
            {
                // (rows beyond the tokens mask nothing that is kept)
                const PfSegment& g = seg_s[k & (kPfSegs - 1)];
                last = g.pos0 + x * tt + (int)((uint32_t)r * per_g >> 16) - g.j0 * kPfKeys;
                left = pf_end(g, x) - g.j0 - 1;
                __syncwarp();
                // slot 0 of the CTA: the segment holds the run's first key tile; slot 1: its last
                if (lane == 0) out_s[warp].part = g.j0 == 0 && g.j1 == g.n_kt ? -1 : 2 * (int)blockIdx.x + (i > 0 ? 1 : 0);
            }
            float m_used = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            for (; left >= 0; --left, ++i, last -= kPfKeys, first = false) {
                const int slot = i & (kPfMeta - 1);
                ok = mbar_wait_bounded(&meta_ready[slot], (uint32_t)(i / kPfMeta) & 1u, &abort_s, status) &&
                     mbar_wait_bounded(&s_full[x], s_par, &abort_s, status);
                ok = __all_sync(0xffffffffu, ok);           // the TMEM accesses are warp-collective
                if (!ok) break;
                s_par ^= 1u;
                tc_fence_after();
                if (left == 0) {
                    // The item's last S is there, so its Q is no longer needed: the next one's is fetched beside this
                    // tile's softmax.  What the output needs of the segment is kept aside.
                    const PfSegment& g = seg_s[k & (kPfSegs - 1)];
                    if (lane == 0) {
                        out_s[warp].row0 = ((long long)g.tok0 + x * tt) * a.n_heads + g.hk * G;
                        out_s[warp].nt = x ? g.nt_b : g.nt_a;
                        out_s[warp].exp = vexp_s[slot];
                    }
                    const int here = i;
                    i += 1 + g.j1 - pf_end(g, x);
                    done_with(k);
                    ++k;
                    find();
                    if (lane == 0) out_s[warp].next = i;
                    i = here;
                    if (!ok) break;
                    if (more) fetch_q(seg_s[k & (kPfSegs - 1)]);
                }
                const uint32_t chunks = ok_s[slot];
                // score factor of chunk c, kept above 0: times a masked score of -inf it has to stay -inf
                const auto factor = [&](int c) { return fmaxf(ks_s[slot][c] * qf, 1.2e-38f); };
                float s[128];
                {
                    uint32_t s0[64], s1[64];
                    tmem_ld64_issue(ts, s0);
                    tmem_ld64_issue(ts + 64u, s1);
                    tmem_wait_ld(s0);
                    tmem_wait_ld(s1);
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        s[e] = __uint_as_float(s0[e]);
                        s[64 + e] = __uint_as_float(s1[e]);
                    }
                }
                if (!__all_sync(0xffffffffu, last >= kPfKeys - 1 && chunks == (1u << kPfChunks) - 1u)) {
#pragma unroll
                    for (int c = 0; c < kPfChunks; ++c) {
                        const int lim = (chunks >> c) & 1u ? last - c * 16 : -1;
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[16 * c + e] = e <= lim ? s[16 * c + e] : -INFINITY;
                    }
                }
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < kPfChunks; ++c) {
                    float m0 = max3(s[16 * c], s[16 * c + 1], s[16 * c + 2]), m1 = max3(s[16 * c + 3], s[16 * c + 4], s[16 * c + 5]);
                    m0 = max3(m0, s[16 * c + 6], s[16 * c + 7]);
                    m1 = max3(m1, s[16 * c + 8], s[16 * c + 9]);
                    m0 = max3(m0, s[16 * c + 10], s[16 * c + 11]);
                    m1 = max3(m1, s[16 * c + 12], s[16 * c + 13]);
                    m0 = max3(m0, s[16 * c + 14], s[16 * c + 15]);
                    mx = fmaxf(mx, fmaxf(m0, m1) * factor(c));
                }
                const bool move = mx > m_used + 8.f;        // false while the row has no key
                if (__any_sync(0xffffffffu, move)) {
                    const float dn = move ? ex2_approx(m_used - mx) : 1.f;
                    if (!first) {
                        // S of this tile is complete, so P V of the tile before is in O
#pragma unroll
                        for (int c = 0; c < D; c += 8) tmem_scale8(to + (uint32_t)c, dn);
                    }
                    if (move) {
                        l2.x *= dn;
                        l2.y *= dn;
                        m_used = mx;
                    }
                }
                const float base = (m_used == -INFINITY ? 0.f : m_used) - kPfBase;
                const float2 nb = make_float2(-base, -base);
#pragma unroll
                for (int c = 0; c < kPfChunks; ++c) {       // 16 keys: 8 columns of P, over S
                    uint32_t p[8];
                    const float fc = factor(c);
                    const float2 ff = make_float2(fc, fc);
#pragma unroll
                    for (int e2 = 0; e2 < 8; ++e2) {
                        float2 e = fma2(make_float2(s[16 * c + 2 * e2], s[16 * c + 2 * e2 + 1]), ff, nb);
                        e.x = ex2_approx(e.x);
                        e.y = ex2_approx(e.y);
                        l2 = add2(l2, e);
                        p[e2] = pack_f16x2(e.x, e.y);
                    }
                    tmem_st8_issue(ts + (uint32_t)c * 8u, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[x]);
            }
            if (!ok) break;
            __syncwarp();
            i = out_s[warp].next;
            // the next item's Q before this one's output, so that its S runs beside that
            if (more) qf = scale_q();
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&o_done[x], o_par, &abort_s, status));
            if (!ok) break;
            o_par ^= 1u;
            tc_fence_after();
            const float l = l2.x + l2.y;
            const int E6 = out_s[warp].exp - kPfShift;
            const float up = E6 < -126 ? 0.f : __uint_as_float((uint32_t)(E6 + 127) << 23);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float f = inv * up;
            const int tok = (int)((uint32_t)r * per_g >> 16), part = out_s[warp].part;
            const bool live = tok < out_s[warp].nt;
            const size_t qrow = (size_t)out_s[warp].row0 + (size_t)tok * a.n_heads + (r - tok * G);
            const size_t prow = (size_t)max(part, 0) * 2 * kPfRows + x * kPfRows + r;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                float v[16];
                tmem_ld16(to + (uint32_t)c, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= f;
                if (live && part < 0) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
                    uint4* dst = reinterpret_cast<uint4*>(a.out + qrow * D + c);
                    dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                    dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                } else if (live) {
                    uint32_t y[8], z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y[e] = __float_as_uint(v[e]);
                        z[e] = __float_as_uint(v[8 + e]);
                    }
                    store32(a.part_o + prow * D + c, y);
                    store32(a.part_o + prow * D + c + 8, z);
                }
            }
            if (live && part >= 0) a.part_ml[prow] = make_float2(m_used, l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[x]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, L::TMEM_COLS);
}

// Joins the partials of one item: that of boundary c = blockIdx.x + 1 between the grid's P runs, if it lies
// inside an item and is the first one there.  blockIdx.y takes 32 of the item's 256 query rows; a row's D / 4
// lanes hold four head dims each.
constexpr int kPfJoinThreads = 256;
constexpr int kPfJoinRows = 32;
__global__ void __launch_bounds__(kPfJoinThreads) attn_prefill_f8_join_kernel(const AttnF8Args a, int tt, int P) {
    __shared__ PfRun run_s;
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x + 1, D = a.head_dim, step = 2 * tt;
    pf_find_run(a, step, P, c - 1, kPfJoinThreads, false, &run_s);
    if (run_s.end >= run_s.total) return;
    const PfPlace at = run_s.to;
    const PfSeq s = pf_seq(a, at.b, false);
    const int n_kt = (s.pos0 + min((at.mt + 1) * step, s.n) + kPfKeys - 1) / kPfKeys;
    if (at.j == 0 || at.j >= n_kt) return;
    const long long t0 = run_s.end - at.j, t1 = t0 + n_kt;
    if (run_s.begin > t0) return;                          // not the first inside
    const long long q = run_s.total / P, rem = run_s.total - q * P;
    const auto boundary = [&](int k) { return q * k + min((long long)k, rem); };    // before the snap
    const int first_slot = 2 * (c - 1) + (run_s.begin == t0 ? 0 : 1);
    int last = c;                                          // the last run with tiles of the item
    while (last + 1 < P && boundary(last + 1) < t1 - kPfSnap) ++last;
    const int G = a.n_heads / a.n_kv_heads;
    const int lanes = D / 4, rows_at_once = kPfJoinThreads / lanes, lane = threadIdx.x % lanes;
    const int row0 = (int)blockIdx.y * kPfJoinRows;
    for (int i = threadIdx.x / lanes; i < kPfJoinRows; i += rows_at_once) {
        const int row = row0 + i, x = row / kPfRows, r = row % kPfRows;
        const int tok = at.mt * step + x * tt + r / G;
        if (r / G >= tt || tok >= s.n) continue;
        float M = -INFINITY;
        for (int k = c - 1; k <= last; ++k)
            M = fmaxf(M, a.part_ml[(size_t)(k < c ? first_slot : 2 * k) * 2 * kPfRows + row].x);
        const float base = M == -INFINITY ? 0.f : M;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
        for (int k = c - 1; k <= last; ++k) {
            const size_t pr = (size_t)(k < c ? first_slot : 2 * k) * 2 * kPfRows + row;
            const float2 ml = a.part_ml[pr];
            if (ml.y == 0.f) continue;                     // no key there; its row may not be written
            const float w = exp2f(ml.x - base) * ml.y;
            const float4 o = *reinterpret_cast<const float4*>(a.part_o + pr * D + lane * 4);
            num.x += w * o.x;
            num.y += w * o.y;
            num.z += w * o.z;
            num.w += w * o.w;
            den += w;
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        *reinterpret_cast<uint2*>(a.out + ((size_t)(s.c0 + tok) * a.n_heads + (size_t)at.hk * G + r % G) * D + lane * 4) =
            make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
    }
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
    const int sms = std::min(device_sm_count(), kF8MaxSms);
    if (sms <= 0) return record(cudaErrorNoDevice, "attn_prefill_f8");
    const int tt = kPfRows / (a.n_heads / a.n_kv_heads);    // tokens per query tile
    trace_before("attn_prefill_f8", stream);
    e = launch_pdl(attn_prefill_f8_kernel<D>, dim3((unsigned)sms), dim3(kPfThreads), smem, stream, 1, a, tt);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "attn_prefill_f8_kernel launch");
    if (sms == 1) return cudaSuccess;
    trace_before("attn_prefill_f8_join", stream);
    e = launch_pdl(attn_prefill_f8_join_kernel, dim3((unsigned)(sms - 1), 2 * kPfRows / kPfJoinRows), dim3(kPfJoinThreads), 0,
                   stream, 1, a, tt, sms);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "attn_prefill_f8_join_kernel launch");
}

}  // namespace

// Two partials of 256 rows per CTA; sized for the largest grid on any device.
size_t attn_prefill_f8_scratch_bytes(int head_dim) {
    return (size_t)2 * kF8MaxSms * 2 * kPfRows * (head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attn_prefill_f8(AttnF8Args a, void* workspace, cudaStream_t stream) {
    if (a.tokens <= 0) return cudaSuccess;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)2 * kF8MaxSms * 2 * kPfRows * a.head_dim);
    return a.head_dim == 128 ? prefill_f8_for<128>(a, stream) : prefill_f8_for<64>(a, stream);
}

}  // namespace ll
