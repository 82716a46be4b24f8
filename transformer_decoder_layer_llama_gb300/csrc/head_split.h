// How the threads of the normed heads' kernels share a token's heads.  Plain C++: the host compiler tests it too.
#pragma once

#include <algorithm>

#ifdef __CUDACC__
#define LL_HOST_DEVICE __host__ __device__
#else
#define LL_HOST_DEVICE
#endif

namespace ll {

// A head is `lanes` threads of a group of W (a power of two), each with two columns of N elements; a token is `rows`
// groups, each with up to U heads at a time, in `parts` turns; a CTA has `slots` tokens at a time.
struct HeadSplit {
    int lanes, width, rows, parts, slots, threads;
};

inline HeadSplit head_split(int lanes, int heads, int per_thread, int threads) {
    HeadSplit s;
    s.lanes = lanes;
    s.width = 4;
    while (s.width < s.lanes) s.width *= 2;
    const int most = threads / s.width;
    s.parts = (heads + per_thread * most - 1) / (per_thread * most);
    s.rows = (heads + per_thread * s.parts - 1) / (per_thread * s.parts);
    s.slots = std::max(1, most / s.rows);
    s.threads = (s.slots * s.rows * s.width + 31) / 32 * 32;
    return s;
}

// The first head of a token's group `row` in turn `part`; the group's others lie `rows` behind each other.  The turns are
// rounded up: the last one's groups may have no head at all (127 heads of 32 lanes, three at a time: 6 turns of 8 groups,
// and the last group's first head would be the 128th).
LL_HOST_DEVICE inline int first_head(const HeadSplit& s, int part, int row, int per_thread) {
    return part * s.rows * per_thread + row;
}

}  // namespace ll
