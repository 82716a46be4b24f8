// Prefill attention over a paged cache of e4m3 codes with one scale per block and KV head, on the
// tcgen05 tensor cores: a ragged batch of new tokens, each attending causally to its own sequence.
//
// A work item is one KV head of one sequence and two tiles (A, B) of 128 query rows each: a tile is
// floor(128 / G) consecutive tokens times the G query heads that share the KV head, so a tile of keys is
// brought in and converted once for 256 rows.  One CTA per SM and item, 128 keys at a time up to the
// item's last position, items with the most keys first.  Where there are at most half as many items as SMs,
// several CTAs share an item's keys and a second kernel joins their float32 partials by the log-sum-exp:
// 16 tokens behind 32768 (64 heads over 8) take 48 us so (L2 cold), 382 with one CTA per item.  (A persistent grid with
// equal shares of all key tiles was slower: its roles need registers for the walk, and a partial is 128 KB.)
//
// Roles (512 threads in four groups of four warps, the registers split by setmaxnreg):
//  * warps 0-3 and 4-7, softmax of tile A and B: one thread per query row.  First they bring Q to shared
//    memory and turn it into FP16 there.  Per key tile: the row of S from TMEM into registers, its maximum, probabilities
//    written over S as FP16; where the maximum has grown by more than 2^8 the running O in TMEM is scaled.
//    At the end O / l goes out.
//  * warps 8-11, converters: the codes of a key tile, as they lie in the pool, become FP16 in the
//    128-byte-swizzled operand tiles, two buffers each for K and V.
//  * warp 14: brings codes (bulk copies of 16 keys) and scales a tile ahead, and looks at how far V scales differ.
//    (Loaded straight into the converters' registers the codes were what the rest waited for: the little L1 that this
//    much shared memory leaves cannot keep a tile's loads in flight.)
//  * warps 12 and 13, one elected lane each: S = Q K^T (both from shared memory) and O += P V (P from TMEM) of
//    tile A and B.  The two tiles take turns, so that the tensor core works for one while the other's softmax runs.
//
// Bound by the chain of one query tile (S out of TMEM, maximum, 128 exponentials per row, P back, P V and the next
// S: about 3100 clocks a key tile, of which the tensor core works 1024 for each of the two query tiles) together with
// the conversion, which shares shared memory with it: leaving out any one of them gains 3 to 10%.  Ragged
// 70B-shaped chunks (589 GFLOP): 428 us, 1.38 PFLOP/s, 74% of the measured BF16 burst; 7B prompt of 2048
// tokens (34 GFLOP, 256 items of 2 to 16 key tiles, of which an SM's one or two start with 5 us of fetching and
// staging): 45 us.  The code of all roles shares the instruction cache: waits in half the instructions and loops
// that are not unrolled took the prompt from 49.2 to 44.7 us.  Two threads per row (768 threads, 96 registers
// for the softmax) took 475 us in place of 434.
//
// Precision.  Codes are exact in FP16.  A query row is scaled by a power of two so that its largest element
// lies in [2^14, 2^15); its factor and the block's K scale multiply the float32 score, 16 keys at a time
// (a block holds whole 16-key chunks), so they cost nothing per element but the multiply-add there already
// is.  P is one FP16 (relative error 2^-11, an eighth of the BF16 output's half step), relative to an
// exponent base that keeps it below 2^14.  Row maxima, sums, S and O are float32.
//
// V scales belong to blocks, and what a row sums is probability times V scale times code.  So P holds such
// terms, 2^(score + log2 of the V scale - t + 6), where t is the largest term that the row itself has met: a
// block that the row does not see, or hardly weighs, takes no bits from the others, however large its V.  The
// sum of the probabilities has a base of its own (m); terms times one power of two per tile are probabilities.
// Where the scales of a tile of keys differ, but by 2^4 at most, V is code times the scale's ratio to one
// power of two for the tile (exact for powers of two), and t at most 4 too large; where they differ by more, the
// tile takes a slower path that gives each 16 keys their own scale.  A term is lost below about 2^-27 of the
// row's largest.  Four chunks of 1000 tokens behind 1000 to 7000 (64 heads over 8), blocks of 16: 445 us with V scales
// alike, 473 with scales up to 2^2 apart, 942 with scales up to 2^12 apart in every tile.
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
constexpr float kPfLog2e = 1.4426950408889634f;
constexpr float kPfShift = 6.f;          // P enters P V times 2^6
constexpr float kPfFloor = 80.f;         // a V scale this far (in powers of two) below the largest term adds nothing

// The V scales of a key tile: all alike; within 2^4 of each other: V enters P V as code times its scale's ratio to a
// power of two that the whole tile has (exact for scales that are powers of two); further apart: V is the bare code,
// and each 16 keys' probabilities carry their own scale.
enum PfScales { kOneScale, kNearScales, kFarScales };
constexpr float kPfSpread = 16.f;
constexpr uint32_t kPfFar = 1u << kPfChunks;   // beside the bits of a tile's chunks

template <int D>
struct PfLayout {
    static constexpr uint32_t TILE = kPfRows * D * 2;       // [D / 64][128 rows][128 B] FP16
    static constexpr uint32_t OFF_Q = 0;                    // A, B
    static constexpr uint32_t OFF_K = 2 * TILE, OFF_V = 4 * TILE;   // two buffers each
    static constexpr uint32_t CODES = kPfKeys * D;          // a tile of codes as it lies in the pool
    static constexpr uint32_t OFF_CK = 6 * TILE, OFF_CV = OFF_CK + CODES, TOTAL = OFF_CV + CODES;
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
// 16 columns, stored without waiting; tmem_wait_st waits for all of the thread's stores.
LL_DEVINL void tmem_st16_issue(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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

// The larger magnitude in each half (a NaN loses to a number).
LL_DEVINL uint32_t max_abs_bf16x2(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
    return r;
}

// Two BF16 times the power of two in both halves of up2 (exact), as FP16.
LL_DEVINL uint32_t scaled_f16x2(uint32_t x, uint32_t up2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(up2));
    return pack_f16x2(bf16_lo(r), bf16_hi(r));
}

// A whole 32-byte sector per thread.
LL_DEVINL void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Waits for the phase with the given parity for at most two seconds, and no longer once *abort is set; false, and
// *abort set, if it did not come.  (mbar_wait_bounded in fewer instructions: twenty of them share this kernel's
// instruction cache.  The kernel's end flags the status.)
LL_DEVINL bool pf_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
    do {
        if (mbar_try_wait(bar, parity)) return true;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    } while (*abort == 0 && t - t0 < 2000000000u);
    *abort = 1;
    return false;
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

// What a work item covers: new tokens t0 .. of sequence b (rows tok0 + t of q), the first at position pos0;
// nt_a and nt_b tokens in the tiles, which see keys 0 .. end_a - 1 and 0 .. end_b - 1 (0: no tile B).
struct PfItem {
    int b, hk, tok0, pos0, tt;
    int nt_a, nt_b, end_a, end_b;
    int n_kt;                // key tiles
};

// One sequence's new tokens: rows c0 .. c0 + n - 1 of q at positions pos0 .. (n = 0 where there are none, or where
// the counts do not fit together: flagged).
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

// Item i of the grid, KV heads fastest; called by whole warps.  Items with the most keys come first, so that the
// last ones to start are short: in a batch of up to 32 sequences the item's place in that order is found by a
// search over the number of key tiles, a lane per sequence; in larger batches the order is by query tile alone
// (latest first).  Ragged 70B-shaped chunks: 529 -> 485 us.
LL_DEVINL bool pf_item(const AttnF8Args& a, int i, int n_mt, int tt, bool flag, PfItem& it) {
    const int step = 2 * tt;
    it.hk = i % a.n_kv_heads;
    const int k = i / a.n_kv_heads;
    int mt;
    PfSeq s;
    if (a.batch == 1 || a.batch > 32) {
        it.b = k % a.batch;
        mt = n_mt - 1 - k / a.batch;
        s = pf_seq(a, it.b, flag);
        if (mt * step >= s.n) return false;
    } else {
        const int lane = threadIdx.x & 31;
        PfSeq mine{0, 0, 0};
        if (lane < a.batch) mine = pf_seq(a, lane, flag && i == 0);
        // x / step for 0 <= x < 2^30, exactly: step <= 256, so x times what 2^38 / step is rounded up by stays below 2^38
        const unsigned long long per = (1ull << 38) / (unsigned)step + 1;
        const auto steps_of = [&](int x) { return (int)((unsigned long long)x * per >> 38); };
        const int items = steps_of(mine.n + step - 1);
        // this lane's items with more than t key tiles: those whose last key lies beyond 128 t
        const auto longer = [&](int t) {
            const int x = t * kPfKeys - mine.pos0;
            return x < 0 ? items : x >= mine.n ? 0 : items - steps_of(x);
        };
        int lo = 0;                                         // (longer than lo - 1: more than k items, or lo = 0)
        int hi = __reduce_max_sync(0xffffffffu, mine.n ? (mine.pos0 + mine.n + kPfKeys - 1) / kPfKeys : 0);
        if (k >= __reduce_add_sync(0xffffffffu, items)) return false;
        while (lo < hi) {                                   // the smallest t that at most k items exceed: item k's key tiles
            const int mid = (lo + hi) >> 1;
            if (__reduce_add_sync(0xffffffffu, longer(mid)) <= k) hi = mid;
            else lo = mid + 1;
        }
        const int more = longer(lo), same = longer(lo - 1) - more;
        const int p = k - __reduce_add_sync(0xffffffffu, more);      // its place among the items as long
        int before = same;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        before -= same;
        const uint32_t who = __ballot_sync(0xffffffffu, p >= before && p < before + same);
        it.b = __ffs(who) - 1;
        mt = __shfl_sync(0xffffffffu, items - more - 1 - (p - before), it.b);
        s.c0 = __shfl_sync(0xffffffffu, mine.c0, it.b);
        s.n = __shfl_sync(0xffffffffu, mine.n, it.b);
        s.pos0 = __shfl_sync(0xffffffffu, mine.pos0, it.b);
    }
    const int t0 = mt * step, left = s.n - t0;
    it.tt = tt;
    it.tok0 = s.c0 + t0;
    it.pos0 = s.pos0 + t0;
    it.nt_a = min(tt, left);
    it.nt_b = min(tt, left - it.nt_a);
    it.end_a = it.pos0 + it.nt_a;
    it.end_b = it.nt_b ? it.end_a + it.nt_b : 0;
    it.n_kt = (max(it.end_a, it.end_b) + kPfKeys - 1) / kPfKeys;
    return true;
}

// Where there are at most half as many items as SMs, ns CTAs share an item's key tiles, each at least kPfLeast of them,
// and leave partials for the join kernel.
constexpr int kPfLeast = 3;
LL_DEVINL int pf_splits(int ns, int n_kt) { return max(1, min(ns, n_kt / kPfLeast)); }

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) attn_prefill_f8_kernel(const AttnF8Args a, int n_mt, int tt, int ns) {
    using L = PfLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // Per query tile x and key tile j (parity j & 1): S computed, P stored.  Per key buffer: K or V stored
    // (ready), read by both query tiles (empty).  Scales of key tile j sit in slot j & 3: slot and barrier are
    // written again for tile j + 4, when K of tile j + 3 is converted, whose buffer was free after the S of tile
    // j + 1, which waited for the P of tile j.
    __shared__ uint64_t q_ready[2], s_full[2], p_ready[2][2], turn_done[2], o_done[2], k_ready[2], k_empty[2], v_ready[2], v_empty[2];
    // Codes of a key tile: brought in (full), read by the converters (empty).
    __shared__ uint64_t meta_ready[kPfMeta], drain[2], c_full[2], c_empty[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    __shared__ __align__(16) float ks_s[kPfMeta][kPfChunks];   // per 16-key chunk: K scale
    __shared__ float v_s[kPfMeta][kPfChunks];               // near scales: ratio of the V scale to the tile's; far: its log2
    __shared__ uint2 tile_s[kPfMeta];                       // log2 of the tile's V scale; ok_s, and whether they are far apart
    __shared__ int near_s[kPfMeta];                         // whether its V scales are near, not alike
    __shared__ uint32_t ok_s[kPfMeta];                      // bit c = chunk c is backed by a valid block

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* status = a.status;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_ready[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i][0], 4);
            mbar_init(&p_ready[i][1], 4);
            mbar_init(&turn_done[i], 1);
            mbar_init(&o_done[i], 1);
            mbar_init(&k_ready[i], 4);
            mbar_init(&k_empty[i], 2);
            mbar_init(&drain[i], 1);
            mbar_init(&v_ready[i], 4);
            mbar_init(&v_empty[i], 2);
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 4);
        }
        for (int i = 0; i < kPfMeta; ++i) mbar_init(&meta_ready[i], 1);
        abort_s = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    PfItem it;
    const int item = (int)blockIdx.x / ns, split = (int)blockIdx.x - item * ns;
    if (!pf_item(a, item, n_mt, tt, warp == 0 && split == 0, it)) return;
    const int splits = pf_splits(ns, it.n_kt);
    if (split >= splits) return;
    const int first = (int)((long long)it.n_kt * split / splits);   // the CTA's first key tile; tiles are counted from it
    const int n_kt = (int)((long long)it.n_kt * (split + 1) / splits) - first;
    const int G = a.n_heads / a.n_kv_heads;
    const int kv_end = max(it.end_a, it.end_b) - first * kPfKeys;   // keys, and table entries, from the CTA's first tile too
    const int32_t* table_row = a.block_table + (size_t)it.b * a.max_blocks;
    const int key0 = first * kPfKeys;
    const int my_key = (lane & 7) * 16;                 // lane c < 8 looks after 16-key chunk c of a tile
    const int bs_log2 = 31 - __clz(a.block_size);       // (a power of two: no divisions on this path)
    auto entry_of = [&](int j) {                        // its table entry (-1 past the keys)
        const int key = j * kPfKeys + my_key;
        return j < n_kt && key < kv_end ? table_row[(key0 + key) >> bs_log2] : -1;
    };
    auto row_of = [&](int j, int entry) {               // its first pool row (-1: no valid block)
        const int key = j * kPfKeys + my_key;
        const bool want = j < n_kt && key < kv_end;
        if (want && (entry < 0 || entry >= a.num_blocks)) flag_status(status, LL_DEV_BAD_BLOCK);
        return want && entry >= 0 && entry < a.num_blocks
                   ? ((entry * a.n_kv_heads + it.hk) << bs_log2) + ((key0 + key) & (a.block_size - 1)) : -1;
    };
    auto scale_of = [&](const float* scales, int row) {
        return row >= 0 ? scales[row >> bs_log2] : 0.f;
    };
    if (warp < 8) {                                         // Q of tile A (warps 0-3) and B, as it is, to its place
        // a warp's 32 rows, D / 8 lanes to a row, 16 bytes each
        constexpr int QL = D / 8, QR = 32 / QL;
        const int x = warp >> 2, c0 = lane % QL, nt = x ? it.nt_b : it.nt_a;
        const uint32_t per_g = 65536u / (uint32_t)G + 1u;   // row / G = row * per_g >> 16 for row < 128
        const size_t row0 = ((size_t)it.tok0 + x * it.tt) * a.n_heads + it.hk * G;
#pragma unroll 4
        for (int rr = (warp & 3) * 32 + lane / QL; rr < (warp & 3) * 32 + 32; rr += QR) {
            const int t = (int)((uint32_t)rr * per_g >> 16);
            cp_async16(smem + L::OFF_Q + (uint32_t)x * L::TILE + pf_off(rr, c0),
                       a.q + (t < nt ? (row0 + (size_t)t * a.n_heads + (rr - t * G)) * D + c0 * 8 : 0), t < nt);
        }
        cp_async_commit();
    }
    int entry = -1, row = -1;                               // of the producer: the next tile's table entry, the tile's row
    float ks = 0.f, vs = 0.f;
    if (warp == 14) {                                       // (what takes a while is on its way before the barrier)
        row = row_of(0, entry_of(0));
        ks = scale_of(a.k_scale, row);
        vs = scale_of(a.v_scale, row);
        entry = entry_of(1);
    }
    if (warp == 12) {
        tmem_alloc(&tmem_base_s, L::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int n_a = min(max((it.end_a + kPfKeys - 1) / kPfKeys - first, 0), n_kt);
    const int n_b = min(max((it.end_b + kPfKeys - 1) / kPfKeys - first, 0), n_kt);

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp < 14) {
            // ------------------------------------------------ MMA issuers: warp 12 for tile A, 13 for B
            // The whole warp walks along, one lane issues: addresses stay in uniform registers.  (One thread on a
            // path of its own took twice an MMA's time to issue the next.)
            const int x = warp - 12;
            const int n_x = x ? n_b : n_a;
            constexpr uint32_t id_s = idesc_f16(kPfRows, kPfKeys, false), id_o = idesc_f16(kPfRows, D, true);
            const uint64_t dq = umma_desc_sw128(smem_u32(smem + L::OFF_Q) + (uint32_t)x * L::TILE);
            const uint64_t dk = umma_desc_sw128(smem_u32(smem + L::OFF_K));
            const uint64_t dv = pf_desc_mn(smem_u32(smem + L::OFF_V), kPfRows * 128);
            const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32), k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32);
            const uint32_t v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
            const uint32_t t_s = tmem + L::TMEM_S + (uint32_t)x * 128u, t_o = tmem + L::TMEM_O + (uint32_t)x * 128u;
            auto k_wait = [&](int i) { return pf_wait(&k_ready[i & 1], (uint32_t)(i >> 1) & 1u, &abort_s); };
            auto v_wait = [&](int i) { return pf_wait(&v_ready[i & 1], (uint32_t)(i >> 1) & 1u, &abort_s); };
            // The two warps take turns, A before B: a turn is P V of a key tile with the S of the next.  Interleaved,
            // both tiles' S would be ready together: both softmaxes would run at once and the tensor core wait for them.
            auto my_turn = [&](int j) {
                const int before = x ? j : j - 1;           // the other's turn, if it has one
                return before < 0 || before >= (x ? n_a : n_b) || pf_wait(&turn_done[x ^ 1], (uint32_t)before & 1u, &abort_s);
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
            // 64 keys of O += P V
            auto issue_pv = [&](int i, int half, bool first) {
                const uint32_t b = v_lo + (uint32_t)(i & 1) * (L::TILE >> 4) + (uint32_t)(half * 4 * 2048 >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    pf_mma_ts(t_o, t_s + (uint32_t)half * 32u + (uint32_t)kk * 8u, b + (uint32_t)(kk * 2048 >> 4), v_hi, id_o,
                              !first || kk > 0 ? 1u : 0u);
            };
            bool ok = true;
            if (n_x > 0) {
                ok = __all_sync(0xffffffffu, pf_wait(&q_ready[x], 0, &abort_s) && k_wait(0));
                tc_fence_after();
                if (ok && elect_one()) {
                    issue_s(0);
                    tc_commit(&k_empty[0]);
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int j = 0; j < n_x && ok; ++j) {
                // (what is usually there already is waited for first, beside the softmax; P comes in halves of 64 keys,
                // so that P V of the first runs while the second is computed)
                const bool more = j + 1 < n_x;
                ok = __all_sync(0xffffffffu, v_wait(j) && (!more || k_wait(j + 1)) && my_turn(j) &&
                                                 pf_wait(&p_ready[x][0], (uint32_t)j & 1u, &abort_s));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) issue_pv(j, 0, j == 0);
                __syncwarp();
                ok = __all_sync(0xffffffffu, pf_wait(&p_ready[x][1], (uint32_t)j & 1u, &abort_s));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_pv(j, 1, false);
                    if (more) issue_s(j + 1);
                    mbar_arrive(&turn_done[x]);
                    tc_commit(&v_empty[j & 1]);
                    if (more) tc_commit(&k_empty[(j + 1) & 1]);
                    else tc_commit(&o_done[x]);
                }
                __syncwarp();
            }
            // past its own last tile a query tile still takes part in the buffers' rounds
#pragma unroll 1
            for (int j = n_x; j < n_kt && ok; ++j) {
                ok = __all_sync(0xffffffffu, k_wait(j) && v_wait(j));
                if (ok && lane == 0) {
                    mbar_arrive(&k_empty[j & 1]);
                    mbar_arrive(&v_empty[j & 1]);
                }
            }
            if (elect_one()) {
                tc_commit(&drain[x]);
                volatile int never = 0;
                pf_wait(&drain[x], 0, &never);
            }
        } else if (warp == 14) {
            // ------------------------------------------------ codes and scales
            auto bring = [&](int which, const uint8_t* pool, int j, int row, uint32_t mask) {
                if (lane == 0) mbar_arrive_expect_tx(&c_full[which], (uint32_t)__popc(mask) * 16u * D);
                __syncwarp();
                if (lane < kPfChunks && row >= 0)
                    bulk_load(smem + (which ? L::OFF_CV : L::OFF_CK) + lane * 16 * D, pool + (size_t)(uint32_t)row * D, 16u * D,
                              &c_full[which]);
            };
            auto taken = [&](int which, int j) {            // by the converters: the codes of the tile before
                return j == 0 || __all_sync(0xffffffffu, pf_wait(&c_empty[which], (uint32_t)(j - 1) & 1u, &abort_s));
            };
            int k_at = -1, v_at = -1;
            float lvr = 0.f;                                // log2 of the tile's V scale
            uint32_t v_at_log = ~0u;                        // the scale whose log2 lvr is
#pragma unroll 1
            for (int j = 0; j < n_kt; ++j) {
                const int slot = j & (kPfMeta - 1);
                if (j) {
                    row = row_of(j, entry);
                    ks = scale_of(a.k_scale, row);
                    vs = scale_of(a.v_scale, row);
                    entry = entry_of(j + 1);
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, lane < kPfChunks && row >= 0);
                if (!taken(0, j)) break;
                if (lane == 0) ok_s[slot] = mask;
                __syncwarp();
                bring(0, a.k_pool, j, row, mask);
                k_at = j;
                const uint32_t vb = __float_as_uint(vs);    // (scales are not negative: ordered as integers)
                const uint32_t hi = __reduce_max_sync(0xffffffffu, lane < kPfChunks && row >= 0 ? vb : 0u);
                const uint32_t lo = __reduce_min_sync(0xffffffffu, lane < kPfChunks && row >= 0 ? vb : hi);
                PfScales kind = kOneScale;
                if (hi != v_at_log || lo != hi) {
                    lvr = f8_log2_scale(__uint_as_float(hi));
                    v_at_log = hi;
                    if (lo != hi) {
                        kind = __uint_as_float(lo) * kPfSpread >= __uint_as_float(hi) ? kNearScales : kFarScales;
                        if (kind == kNearScales) lvr = floorf(lvr);
                        v_at_log = ~0u;
                        if (lane < kPfChunks) v_s[slot][lane] = kind == kNearScales ? scalbnf(vs, -(int)lvr) : f8_log2_scale(vs);
                    }
                }
                if (lane < kPfChunks) ks_s[slot][lane] = ks;
                if (lane == 0) {
                    tile_s[slot] = make_uint2(__float_as_uint(lvr), kind == kFarScales ? mask | kPfFar : mask);
                    near_s[slot] = kind == kNearScales;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&meta_ready[slot]);
                if (!taken(1, j)) break;
                bring(1, a.v_pool, j, row, mask);
                v_at = j;
            }
            // no copy is in flight when the CTA leaves
            volatile int never = 0;
            if (k_at >= 0) pf_wait(&c_full[0], (uint32_t)k_at & 1u, &never);
            if (v_at >= 0) pf_wait(&c_full[1], (uint32_t)v_at & 1u, &never);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---------------------------------------------------- keys and values (warps 8-11)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        constexpr int LANES = D / 16, ROWS = 128 / LANES, PER = kPfKeys / ROWS;   // lanes per row, rows per step, steps
        const int tid = threadIdx.x - 256;
        // Eight lanes that load or store together: D = 128: four 16-code pieces of an even row and the other four of
        // the row behind it; D = 64: two rows.  So the codes' chunks are on different banks, and so are the operand's:
        // 0, 2, 4, 6 of an even and an odd row, which the swizzle tells apart.
        const int c16 = D == 128 ? (tid & 3) | (((tid ^ (tid >> 1)) & 4)) : tid & 3;
        const int rsub = D == 128 ? ((tid >> 3) & ~1) | ((tid >> 2) & 1) : tid >> 2;
        const uint32_t st0 = pf_off(rsub, 2 * c16), st1 = pf_off(rsub, 2 * c16 + 1);
        // Tile j from its codes to the operand tile; rows that hold no key become zeros: 0 * stale stays 0.
        auto convert = [&](uint8_t* tile, const uint8_t* codes, int j, uint64_t* done, bool scaled) {
            const int slot = j & (kPfMeta - 1), left = kv_end - j * kPfKeys;
            const uint32_t chunks = ok_s[slot];
            uint4 w[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) w[i] = *reinterpret_cast<const uint4*>(codes + (i * ROWS + rsub) * D + c16 * 16);
            if (left < kPfKeys || chunks != (1u << kPfChunks) - 1u) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int r = i * ROWS + rsub;
                    if (r >= left || !((chunks >> (r >> 4)) & 1u)) w[i] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                uint32_t h[8];
                e4m3x4_to_f16x4(w[i].x, h[0], h[1]);
                e4m3x4_to_f16x4(w[i].y, h[2], h[3]);
                e4m3x4_to_f16x4(w[i].z, h[4], h[5]);
                e4m3x4_to_f16x4(w[i].w, h[6], h[7]);
                if (scaled) {
                    const __half2 f = __float2half2_rn(v_s[slot][(i * ROWS + rsub) >> 4]);
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
            // Only now may the codes be overwritten: every lane has stored what it loaded.  (An arrive right behind the loads
            // can be seen before they have read.)
            if (lane == 0) mbar_arrive(done);
        };
#pragma unroll 1
        for (int j = 0; j < n_kt; ++j) {
            // (whole warps leave)
            bool ok = (j < 2 || pf_wait(&k_empty[j & 1], (uint32_t)((j - 2) >> 1) & 1u, &abort_s)) &&
                      pf_wait(&c_full[0], (uint32_t)j & 1u, &abort_s);
            if (!__all_sync(0xffffffffu, ok)) break;
            convert(smem + L::OFF_K + (uint32_t)(j & 1) * L::TILE, smem + L::OFF_CK, j, &c_empty[0], false);
            if (lane == 0) mbar_arrive(&k_ready[j & 1]);
            ok = (j < 2 || pf_wait(&v_empty[j & 1], (uint32_t)((j - 2) >> 1) & 1u, &abort_s)) &&
                 pf_wait(&c_full[1], (uint32_t)j & 1u, &abort_s);
            if (!__all_sync(0xffffffffu, ok)) break;
            convert(smem + L::OFF_V + (uint32_t)(j & 1) * L::TILE, smem + L::OFF_CV, j, &c_empty[1], near_s[j & (kPfMeta - 1)] != 0);
            if (lane == 0) mbar_arrive(&v_ready[j & 1]);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- softmax (warps 0-3: tile A, 4-7: tile B)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int x = warp >> 2;
        const int r = threadIdx.x & 127;                    // query row = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int tok = r / G, head = it.hk * G + r % G;
        const int n_x = x ? n_b : n_a;
        const bool live = tok < (x ? it.nt_b : it.nt_a);
        const size_t qrow = ((size_t)it.tok0 + x * it.tt + tok) * a.n_heads + head;
        float qf = 0.f;                                     // score factor but for the K scale
        cp_async_wait<0>();
        __syncwarp();
        if (n_x > 0) {
            // Each thread turns its own row into FP16 in its place.  (Rolled loops here and at the output: code that runs
            // once per item displaces the loop that matters.)
            uint8_t* const sq = smem + L::OFF_Q + (uint32_t)x * L::TILE;
            uint32_t m2 = 0;                                // largest magnitudes of the even and odd elements
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 w = *reinterpret_cast<const uint4*>(sq + pf_off(r, c));
                m2 = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(m2, w.x), w.y), w.z), w.w);
            }
            const uint32_t m = max(m2 & 0xffffu, m2 >> 16);
            // exponent of the largest; zeros, infinities (and NaN alone) stay as they are; below 2^-112 the row is
            // scaled as if at 2^-112, so that the factor is one BF16
            int ex = max((int)(m >> 7) - 127, -112);
            if (m == 0u || m >= 0x7f80u) ex = 14;
            const uint32_t up = (uint32_t)(14 - ex + 127) << 7, up2 = up << 16 | up;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                uint4* at = reinterpret_cast<uint4*>(sq + pf_off(r, c));
                const uint4 w = *at;
                *at = make_uint4(scaled_f16x2(w.x, up2), scaled_f16x2(w.y, up2), scaled_f16x2(w.z, up2), scaled_f16x2(w.w, up2));
            }
            qf = scalbnf(a.scale * kPfLog2e, ex - 14);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[x]);
        }
        const int my_pos = it.pos0 + x * it.tt + tok - first * kPfKeys;   // rows beyond the tokens mask nothing that is kept
        const uint32_t ts = tmem + lane_base + L::TMEM_S + (uint32_t)x * 128u;
        const uint32_t to = tmem + lane_base + L::TMEM_O + (uint32_t)x * 128u;
        // The bases that the probabilities (m) and the terms, probability times V scale (t), are kept to, as powers of two;
        // the sum of the probabilities, 2^m times l.
        float m_used = -INFINITY, t_used = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        // Moves the bases where the row's largest score and term exceed them by more than 2^8 (not while it has no key).
        auto move_bases = [&](float mx, float tx, bool scale_o) {
            const bool move = mx > m_used + 8.f, move_t = tx > t_used + 8.f;
            if (__any_sync(0xffffffffu, move || move_t)) {
                const float dn = move_t ? ex2_approx(t_used - tx) : 1.f, dm = move ? ex2_approx(m_used - mx) : 1.f;
                if (scale_o) {
                    // S of this tile is complete, so P V of the tile before is in O
#pragma unroll 1
                    for (int c = 0; c < D; c += 8) tmem_scale8(to + (uint32_t)c, dn);
                }
                l2.x *= dm;
                l2.y *= dm;
                if (move) m_used = mx;
                if (move_t) t_used = tx;
            }
        };
        auto m_base = [&] { return m_used == -INFINITY ? 0.f : m_used; };
        auto t_base = [&] { return (t_used == -INFINITY ? 0.f : t_used) - kPfShift; };
        auto hand_over = [&](int half) {                    // what is stored of P, to the tensor core
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[x][half]);
        };
        // A key tile whose V scales lie far apart: 16 keys at a time, twice out of TMEM.  In code of its own, reached from
        // the path of masked tiles: factors of 16 keys each on the path of all tiles took the ragged chunks from 423 us to
        // 467, a test of its own there to 455.
        auto far_tile = [&](int slot, uint32_t chunks, int last, bool scale_o) {
            float e[16];
            auto load = [&](int c) {                        // scores, -inf where the row sees no key
                const int lim = (chunks >> c) & 1u ? last - c * 16 : -1;
                const float f = fmaxf(ks_s[slot][c] * qf, 1.17549435e-38f);
                tmem_ld16(ts + (uint32_t)c * 16u, e);
#pragma unroll
                for (int i = 0; i < 16; ++i) e[i] = i <= lim ? e[i] * f : -INFINITY;
            };
            float mx = -INFINITY, tx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kPfChunks; ++c) {
                load(c);
                float mc = e[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) mc = fmaxf(mc, e[i]);
                mx = fmaxf(mx, mc);
                tx = fmaxf(tx, mc + v_s[slot][c]);
            }
            move_bases(mx, tx, scale_o);
            const float mb = m_base(), tb = t_base();
#pragma unroll 1
            for (int c2 = 0; c2 < kPfChunks; c2 += 2) {
                uint32_t p[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    load(c2 + h);
                    const float nb = v_s[slot][c2 + h] - tb;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        l2.x += ex2_approx(e[2 * i] - mb);
                        l2.y += ex2_approx(e[2 * i + 1] - mb);
                        p[8 * h + i] = pack_f16x2(ex2_approx(e[2 * i] + nb), ex2_approx(e[2 * i + 1] + nb));
                    }
                }
                if (c2 == 4) hand_over(0);
                tmem_st16_issue(ts + (uint32_t)c2 * 8u, p);
            }
            hand_over(1);
        };
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j < n_x; ++j) {
            const int slot = j & (kPfMeta - 1);
            ok = pf_wait(&meta_ready[slot], (uint32_t)(j / kPfMeta) & 1u, &abort_s) &&
                 pf_wait(&s_full[x], (uint32_t)j & 1u, &abort_s);
            ok = __all_sync(0xffffffffu, ok);               // the TMEM accesses are warp-collective
            if (!ok) break;
            tc_fence_after();
            const uint2 tile = tile_s[slot];
            const uint32_t chunks = tile.y;
            const int last = my_pos - j * kPfKeys;          // last key of the tile that this row sees
            float f[kPfChunks];
            {
                const float4 f0 = *reinterpret_cast<const float4*>(&ks_s[slot][0]);
                const float4 f1 = *reinterpret_cast<const float4*>(&ks_s[slot][4]);
                f[0] = f0.x * qf; f[1] = f0.y * qf; f[2] = f0.z * qf; f[3] = f0.w * qf;
                f[4] = f1.x * qf; f[5] = f1.y * qf; f[6] = f1.z * qf; f[7] = f1.w * qf;
            }
            float s[128];
            {
                uint32_t s0[64], s1[64];
                tmem_ld64_issue(ts, s0);
                tmem_ld64_issue(ts + 64u, s1);
                tmem_wait_ld(s0);
                tmem_wait_ld(s1);
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    s[i] = __uint_as_float(s0[i]);
                    s[64 + i] = __uint_as_float(s1[i]);
                }
            }
            if (!__all_sync(0xffffffffu, last >= kPfKeys - 1 && chunks == (1u << kPfChunks) - 1u)) {
                if (chunks & kPfFar) {
                    far_tile(slot, chunks, last, j > 0);
                    continue;
                }
#pragma unroll
                for (int c = 0; c < kPfChunks; ++c) {
                    const int lim = (chunks >> c) & 1u ? last - c * 16 : -1;
                    const uint32_t see = lim < 0 ? 0u : 0xffffu >> (15 - min(lim, 15));   // the keys that this row sees
                    // -inf times the factor stays -inf: a factor of 0 (a block of zeros, or scale 0) becomes 2^-126,
                    // which leaves of a sum S (below 2^31) at most 2^-95
                    f[c] = lim < 0 ? 1.f : fmaxf(f[c], 1.17549435e-38f);
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[16 * c + i] = (see >> i) & 1u ? s[16 * c + i] : -INFINITY;
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
                // factor >= 0; a row without a key here keeps -inf (0 * -inf would be NaN)
                const float mc = fmaxf(m0, m1);
                mx = fmaxf(mx, mc == -INFINITY ? mc : mc * f[c]);
            }
            const float lv = __uint_as_float(tile.x);
            move_bases(mx, mx + lv, j > 0);
            // A term is 2^(score + nb); terms times to_p are probabilities.
            const float nb = fmaxf(lv, t_base() - m_base() - kPfFloor) - t_base(), to_p = ex2_approx(-m_base() - nb);
            const float2 nb2 = make_float2(nb, nb), to_p2 = make_float2(to_p, to_p);
#pragma unroll
            for (int c2 = 0; c2 < kPfChunks; c2 += 2) {     // 32 keys: 16 columns of P, over S
                uint32_t p[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = c2 + h;
                    const float2 ff = make_float2(f[c], f[c]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 e = fma2(make_float2(s[16 * c + 2 * i], s[16 * c + 2 * i + 1]), ff, nb2);
                        e.x = ex2_approx(e.x);
                        e.y = ex2_approx(e.y);
                        l2 = fma2(e, to_p2, l2);
                        p[8 * h + i] = pack_f16x2(e.x, e.y);
                    }
                }
                // the first 64 keys are waited for beside the work on the 32 behind them
                if (c2 == 4) hand_over(0);
                tmem_st16_issue(ts + (uint32_t)c2 * 8u, p);
                if (c2 == 6) hand_over(1);
            }
        }
        const size_t prow = (size_t)blockIdx.x * 2 * kPfRows + x * kPfRows + r;
        ok = __all_sync(0xffffffffu, ok && (n_x == 0 || pf_wait(&o_done[x], 0, &abort_s)));
        if (ok && n_x > 0) {
            tc_fence_after();
            const float l = l2.x + l2.y;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // 2^(t - m) as two factors, exact where it is a power of two; a row has a key, so both are finite (or NaN)
            const float ex = l == 0.f ? 0.f : t_used - kPfShift - m_used, ex0 = rintf(0.5f * ex);
            const float up0 = exp2f(ex0), up1 = exp2f(ex - ex0);
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                uint32_t v[64];
                tmem_ld64_issue(to + (uint32_t)c, v);
                tmem_wait_ld(v);
                if (!live) continue;
#pragma unroll
                for (int i = 0; i < 64; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * inv * up0 * up1);
                if (splits == 1) {
#pragma unroll
                    for (int i = 0; i < 64; i += 8)
                        *reinterpret_cast<uint4*>(a.out + qrow * D + c + i) = make_uint4(
                            pack_bf16x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), pack_bf16x2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])),
                            pack_bf16x2(__uint_as_float(v[i + 4]), __uint_as_float(v[i + 5])), pack_bf16x2(__uint_as_float(v[i + 6]), __uint_as_float(v[i + 7])));
                } else {
#pragma unroll
                    for (int i = 0; i < 64; i += 8) {
                        const uint32_t y[8] = {v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]};
                        store32(a.part_o + prow * D + c + i, y);
                    }
                }
            }
            if (live && splits > 1) a.part_ml[prow] = make_float2(m_used, l);
        } else if (ok && live && splits > 1) {
            a.part_ml[prow] = make_float2(-INFINITY, 0.f);  // no key here
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *const_cast<volatile int*>(&abort_s)) flag_status(status, LL_DEV_TIMEOUT);
    if (warp == 12) tmem_dealloc(tmem, L::TMEM_COLS);
}

// Joins the partials of item blockIdx.x: D / 4 lanes to a query row, as many rows per CTA as its threads allow.  A thread
// takes the partials four at a time, so that their loads are in flight together (one after the other, and four rows
// to a thread, 16 tokens behind 32768 of a 70B-shaped layer took 36 us here), and keeps their mean so far, which stays in
// float32's range where the sum of large values would not.
constexpr int kPfJoinThreads = 256;
__global__ void __launch_bounds__(kPfJoinThreads) attn_prefill_f8_join_kernel(const AttnF8Args a, int n_mt, int tt, int ns) {
    pdl_wait();
    pdl_trigger();
    PfItem it;
    if (!pf_item(a, blockIdx.x, n_mt, tt, false, it)) return;
    const int splits = pf_splits(ns, it.n_kt);
    if (splits == 1) return;
    const int D = a.head_dim, G = a.n_heads / a.n_kv_heads;
    const int lanes = D / 4, col = (int)threadIdx.x % lanes * 4;
    const int row = (int)blockIdx.y * (kPfJoinThreads / lanes) + (int)threadIdx.x / lanes, x = row / kPfRows, r = row % kPfRows;
    if (r / G >= (x ? it.nt_b : it.nt_a)) return;
    const size_t pr = (size_t)blockIdx.x * ns * 2 * kPfRows + row;
    float M = -INFINITY, den = 0.f;
    float4 mean = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < splits; k += 4) {
        float2 ml[4];
        float4 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const size_t pk = pr + (size_t)min(k + i, splits - 1) * 2 * kPfRows;
            ml[i] = k + i < splits ? a.part_ml[pk] : make_float2(-INFINITY, 0.f);
            o[i] = *reinterpret_cast<const float4*>(a.part_o + pk * D + col);
        }
        const float mn = fmaxf(M, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
        const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(M - base);
        float w[4], sum = den * old;
        const float before = sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = exp2f(ml[i].x - base) * ml[i].y;
            sum += w[i];
        }
        const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum), keep = before * inv;   // (2^-22 off: the weights need no more)
        mean.x *= keep;
        mean.y *= keep;
        mean.z *= keep;
        mean.w *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ml[i].y == 0.f) continue;                  // no key there: what was read may be anything
            const float part = w[i] * inv;
            mean.x += part * o[i].x;
            mean.y += part * o[i].y;
            mean.z += part * o[i].z;
            mean.w += part * o[i].w;
        }
        M = mn;
        den = sum;
    }
    *reinterpret_cast<uint2*>(a.out + (((size_t)it.tok0 + x * tt + r / G) * a.n_heads + (size_t)it.hk * G + r % G) * D + col) =
        make_uint2(pack_bf16x2(mean.x, mean.y), pack_bf16x2(mean.z, mean.w));
}

// Pairs of query tiles that max_new tokens of a sequence can take.
int pf_query_tiles(int max_new, int tt) { return (int)(((long long)max_new + 2 * tt - 1) / (2 * tt)); }

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
    const int tt = kPfRows / (a.n_heads / a.n_kv_heads);    // tokens per query tile
    const int n_mt = pf_query_tiles(a.max_new, tt);
    const long long items = (long long)a.batch * n_mt * a.n_kv_heads;
    const int sms = std::min(device_sm_count(), kF8MaxSms);
    if (sms <= 0) return record(cudaErrorNoDevice, "attn_prefill_f8");
    // Fewer items than half the SMs (a short chunk behind a long prefix): several CTAs per item.
    const int ns = (int)std::max<long long>(1, sms / items);
    trace_before("attn_prefill_f8", stream);
    e = launch_pdl(attn_prefill_f8_kernel<D>, dim3((unsigned)(items * ns)), dim3(kPfThreads), smem, stream, 1, a, n_mt, tt, ns);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return record(e, "attn_prefill_f8_kernel launch");
    if (ns == 1) return cudaSuccess;
    trace_before("attn_prefill_f8_join", stream);
    e = launch_pdl(attn_prefill_f8_join_kernel, dim3((unsigned)items, 2 * kPfRows * (D / 4) / kPfJoinThreads), dim3(kPfJoinThreads), 0, stream, 1,
                   a, n_mt, tt, ns);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "attn_prefill_f8_join_kernel launch");
}

}  // namespace

// One partial of 256 rows per CTA of a grid of at most as many CTAs as SMs; sized for the largest on any device.
size_t attn_prefill_f8_scratch_bytes(int head_dim) {
    return (size_t)kF8MaxSms * 2 * kPfRows * (head_dim * sizeof(float) + sizeof(float2));
}

bool attn_prefill_f8_fits(int batch, int max_new, int n_heads, int n_kv_heads) {
    return (long long)batch * pf_query_tiles(max_new, kPfRows / (n_heads / n_kv_heads)) * n_kv_heads <= 1LL << 30;
}

cudaError_t launch_attn_prefill_f8(AttnF8Args a, void* workspace, cudaStream_t stream) {
    if (a.tokens <= 0) return cudaSuccess;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)kF8MaxSms * 2 * kPfRows * a.head_dim);
    return a.head_dim == 128 ? prefill_f8_for<128>(a, stream) : prefill_f8_for<64>(a, stream);
}

}  // namespace ll
