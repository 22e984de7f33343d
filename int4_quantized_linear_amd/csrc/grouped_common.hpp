// grouped_common.hpp -- how the kernels over rows sorted by group (expert) find their tiles.  Internal to libconvrot.
//
// Group e owns the rows offsets[e] .. offsets[e + 1] - 1 (int32, in device memory: only the GPU knows them).  A tile holds
// rows of one group.  Every workgroup counts the groups' tiles itself, in LDS, which takes about one memory
// latency and saves a launch; the grid is sized for the largest possible count and units past the real one are
// no work.  Offsets are held to [0, rows], and one below an earlier one counts as that one: whatever they hold, no
// row lies outside the arrays or in two groups, and there are never more tiles than most_group_tiles.
#pragma once
#include "device_common.hpp"

namespace convrot {

constexpr int MAX_GROUPS = 1024;

// The most tiles of bm rows that any offsets can give (groups <= rows beyond which some are empty).
inline int64_t most_group_tiles(int64_t rows, int64_t groups, int bm)
{
    return rows / bm + (groups < rows ? groups : rows);
}

// The groups' table in LDS: first[e] = group e's first row (past the last group: the last one's end), starts[e] =
// tiles of the groups before e (past the last: all).
struct GroupTable {
    int first[MAX_GROUPS], starts[MAX_GROUPS];
};

struct GroupRows {
    int group, first, end;     // rows first .. end - 1 of the group, from the tile's first row on
};

// Fills the table for tiles of bm rows and returns their number.  All NT threads of the workgroup call it; scratch: NT / 32
// ints.  groups < MAX_GROUPS, or the last group's end is `last`.
template <int NT>
__device__ __forceinline__ int group_tiles(const int32_t *offsets, int groups, int rows, int bm, GroupTable &g, int *scratch,
                                           int &last)
{
    constexpr int PER = MAX_GROUPS / NT, NW = NT / 64;
    const int t = (int)threadIdx.x, lane = t & 63, w = t >> 6;
    // prefix maxima of the clamped offsets
    int lo[PER], most = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = PER * t + i;
        most = max(most, e <= groups ? min(max(offsets[e], 0), rows) : 0);
        lo[i] = most;
    }
    last = groups == MAX_GROUPS ? min(max(offsets[MAX_GROUPS], 0), rows) : 0;
    int m = most;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(m, d);
        if (lane >= d) m = max(m, o);
    }
    if (lane == 63) scratch[w] = m;
    m = __shfl_up(m, 1);
    if (lane == 0) m = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < w) m = max(m, scratch[i]);
        last = max(last, scratch[i]);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) g.first[PER * t + i] = lo[i] = max(lo[i], m);
    __syncthreads();
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = PER * t + i;
        const int hi = i + 1 < PER ? lo[i + 1] : e + 1 < MAX_GROUPS ? g.first[e + 1] : last;
        n[i] = e < groups ? (hi - lo[i] + bm - 1) / bm : 0;
        sum += n[i];
    }
    int before = sum;                                    // inclusive scan over the wavefront
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(before, d);
        if (lane >= d) before += o;
    }
    if (lane == 63) scratch[NW + w] = before;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < w) base += scratch[NW + i];
        total += scratch[NW + i];
    }
    before += base - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        g.starts[PER * t + i] = before;
        before += n[i];
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(total);
}

// The group of tile `tile` < total and its rows; every wavefront for itself, from LDS: the last group whose tiles start at
// or before it (empty groups start where the next one does).
__device__ __forceinline__ GroupRows group_of_tile(const GroupTable &t, int bm, int last, int tile)
{
    const int lane = (int)threadIdx.x & 63;
    constexpr int PER = MAX_GROUPS / 64;
    const int block = __builtin_popcountll(__builtin_amdgcn_ballot_w64(t.starts[PER * lane] <= tile)) - 1;
    const int s = t.starts[PER * block + (lane & (PER - 1))];
    const int e = PER * block + __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane < PER && s <= tile)) - 1;
    GroupRows g;
    g.group = __builtin_amdgcn_readfirstlane(e);
    g.first = __builtin_amdgcn_readfirstlane(t.first[g.group] + (tile - t.starts[g.group]) * bm);
    g.end = __builtin_amdgcn_readfirstlane(g.group + 1 < MAX_GROUPS ? t.first[g.group + 1] : last);
    return g;
}

} // namespace convrot
