// Moving blocks of a paged KV cache: copies in all tensors of a pool set at once, and the plan
// that packs the blocks in use to the front of the pool.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ll {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = 16384;           // one work item: 16 KB of one block of one tensor

// Work item = (pair, tensor, 16 KB piece): every thread moves 64 bytes, all four loads before the
// stores.  Bound by memory: 64 pairs of 1 MB blocks in 16 tensors (2.1 GB moved) take 332 us, 6.5 TB/s (95%
// of the copy bandwidth).  A persistent grid takes the items in order, since the number of pairs may
// only be known on the device.
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyBlocksArgs a) {
    pdl_wait();
    pdl_trigger();
    const int n = a.n_pairs ? min(max(*a.n_pairs, 0), a.max_pairs) : a.max_pairs;
    const long long items = (long long)n * a.pieces[a.n_tensors];
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int pair = (int)(it / a.pieces[a.n_tensors]);
        const int piece = (int)(it - (long long)pair * a.pieces[a.n_tensors]);
        const int2 sd = reinterpret_cast<const int2*>(a.pairs)[pair];
        if (sd.x == -1 && sd.y == -1) continue;                        // padding
        if (sd.x < 0 || sd.x >= a.num_blocks || sd.y < 0 || sd.y >= a.num_blocks) {
            if (threadIdx.x == 0) flag_status(a.status, LL_DEV_BAD_BLOCK);
            continue;
        }
        if (sd.x == sd.y) continue;
        int lo = 0, hi = a.n_tensors;                                  // tensor of the piece
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.pieces[mid] <= piece) lo = mid;
            else hi = mid;
        }
        const long long bytes = a.bytes[lo];
        const long long at = (long long)(piece - a.pieces[lo]) * kCopyBytes;
        const uint8_t* src = static_cast<const uint8_t*>(a.data[lo]) + (size_t)sd.x * bytes + at;
        uint8_t* dst = static_cast<uint8_t*>(a.data[lo]) + (size_t)sd.y * bytes + at;
        const int len = (int)min((long long)kCopyBytes, bytes - at);
        if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | (uintptr_t)len) & 15u) == 0) {
            uint4 w[kCopyBytes / 16 / kCopyThreads];
#pragma unroll
            for (int i = 0; i < kCopyBytes / 16 / kCopyThreads; ++i) {
                const int o = (i * kCopyThreads + (int)threadIdx.x) * 16;
                if (o < len) w[i] = *reinterpret_cast<const uint4*>(src + o);
            }
#pragma unroll
            for (int i = 0; i < kCopyBytes / 16 / kCopyThreads; ++i) {
                const int o = (i * kCopyThreads + (int)threadIdx.x) * 16;
                if (o < len) *reinterpret_cast<uint4*>(dst + o) = w[i];
            }
        } else {                                                       // blocks of a multiple of 4 bytes
            for (int o = threadIdx.x * 4; o < len; o += kCopyThreads * 4)
                *reinterpret_cast<uint32_t*>(dst + o) = *reinterpret_cast<const uint32_t*>(src + o);
        }
    }
}

constexpr int kCompactThreads = 1024;

// Exclusive prefix of v over the block's threads, and the total (warp scans, then one over the warps).
LL_DEVINL int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[kCompactThreads / 32 - 1];
    return x - v + (warp ? warp_sums[warp - 1] : 0);
}

// With U blocks in use, every used block at or behind place U moves to a free place before U, in
// order: the k-th such block to the k-th free place.  That is the fewest moves, and no source is a
// destination.  One CTA: a bitmap of the blocks in use and its running count per word sit in shared
// memory, so a block's rank among the used ones is one lookup and one popcount.  512 blocks and a table of 64 rows
// take 7 us, the copies of the 96 moves in 32 layers (1.6 GB) 250 behind it.
__global__ void __launch_bounds__(kCompactThreads) compact_plan_kernel(const CompactArgs a) {
    extern __shared__ uint32_t sm[];
    __shared__ int warp_sums[32];
    const int words = (a.num_blocks + 31) / 32;
    uint32_t* bits = sm;
    int* before = reinterpret_cast<int*>(sm + words);      // used blocks in the words before this one
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    for (int i = tid; i < words; i += kCompactThreads) bits[i] = 0;
    for (int i = tid; i < a.pair_rows; i += kCompactThreads) reinterpret_cast<int2*>(a.pairs)[i] = make_int2(-1, -1);
    __syncthreads();
    for (long long i = tid; i < a.entries; i += kCompactThreads) {
        const int v = a.table[i];
        if (v >= 0 && v < a.num_blocks) atomicOr(&bits[v >> 5], 1u << (v & 31));
        else if (v >= a.num_blocks) flag_status(a.status, LL_DEV_BAD_BLOCK);
    }
    __syncthreads();
    // running count: each thread owns a run of words
    const int per = (words + kCompactThreads - 1) / kCompactThreads;
    const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
    int U;
    int run = block_scan(mine, warp_sums, U);
    for (int w = w0; w < w1; ++w) {
        before[w] = run;
        run += __popc(bits[w]);
    }
    __syncthreads();
    auto rank = [&](int v) { return before[v >> 5] + __popc(bits[v >> 5] & ((1u << (v & 31)) - 1u)); };
    const int stay = U >= a.num_blocks ? U : rank(U);      // used blocks before place U
    const int moves = U - stay;
    int2* pairs = reinterpret_cast<int2*>(a.pairs);
    for (int v = tid; v < a.num_blocks; v += kCompactThreads) {
        const bool used = (bits[v >> 5] >> (v & 31)) & 1u;
        if (used && v >= U) pairs[rank(v) - stay].x = v;
        if (!used && v < U) pairs[v - rank(v)].y = v;
    }
    __syncthreads();
    auto moved = [&](int v) { return v < U ? v : pairs[rank(v) - stay].y; };
    for (int v = tid; v < a.num_blocks; v += kCompactThreads)
        a.block_map[v] = ((bits[v >> 5] >> (v & 31)) & 1u) ? moved(v) : -1;
    for (long long i = tid; i < a.entries; i += kCompactThreads) {
        const int v = a.table[i];
        a.new_table[i] = v >= 0 && v < a.num_blocks ? moved(v) : v;
    }
    if (tid == 0) {
        a.counts[0] = U;
        a.counts[1] = moves;
    }
}

}  // namespace

int copy_blocks_piece_bytes() { return kCopyBytes; }

cudaError_t launch_copy_blocks(const CopyBlocksArgs& a, cudaStream_t stream) {
    if (a.max_pairs <= 0 || a.n_tensors <= 0) return cudaSuccess;
    const int sms = device_sm_count();
    if (sms <= 0) return record(cudaErrorNoDevice, "copy_blocks");
    const long long items = (long long)a.max_pairs * a.pieces[a.n_tensors];
    const unsigned ctas = (unsigned)std::min<long long>(items, (long long)sms * 8);
    trace_before("copy_blocks", stream);
    cudaError_t e = launch_pdl(copy_blocks_kernel, dim3(ctas), dim3(kCopyThreads), 0, stream, 1, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "copy_blocks_kernel launch");
}

cudaError_t launch_compact_plan(const CompactArgs& a, cudaStream_t stream) {
    const size_t smem = (size_t)((a.num_blocks + 31) / 32) * 8;
    cudaError_t e = ensure_func_attr((const void*)compact_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kCompactMaxBlocks / 4, "cudaFuncSetAttribute(compact_plan_kernel)");
    if (e != cudaSuccess) return e;
    trace_before("compact_plan", stream);
    e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kCompactThreads), smem, stream, 1, a);
    trace_after(stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record(e, "compact_plan_kernel launch");
}

}  // namespace ll
