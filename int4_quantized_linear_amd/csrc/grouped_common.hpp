// grouped_common.hpp -- how the kernels over rows sorted by group (expert) find their tiles.  Internal to libconvrot.
//
// Group e owns the rows offsets[e] .. offsets[e + 1] - 1 (int32, in device memory: only the GPU knows them).  A tile holds
// rows of one group.  Every workgroup counts the groups' tiles itself, in LDS, which takes about one memory
// latency and saves a launch; the grid is sized for the largest possible count and units past the real one are
// no work.  Offsets are held to [0, rows] and to their order, so that no contents of theirs reach past the arrays: a
// group that starts behind its end is empty.
#pragma once
#include "device_common.hpp"

namespace convrot {

constexpr int MAX_GROUPS = 1024;

// The most tiles of bm rows that any offsets can give (groups <= rows beyond which some are empty).
inline int64_t most_group_tiles(int64_t rows, int64_t groups, int bm)
{
    return rows / bm + (groups < rows ? groups : rows);
}

struct GroupRows {
    int group, first, end;     // rows first .. end - 1 of the group, from the tile's first row on
};

__device__ __forceinline__ void group_range(const int32_t *offsets, int e, int rows, int &lo, int &hi)
{
    lo = min(max(offsets[e], 0), rows);
    hi = min(max(offsets[e + 1], lo), rows);
}

// starts[e] = tiles of the groups before e, for e < MAX_GROUPS (past the last group: the total), computed by a
// workgroup of NT >= 64 threads, which all have to call; returns the total.  scratch: NT / 64 ints.
template <int NT>
__device__ __forceinline__ int group_tiles(const int32_t *offsets, int groups, int rows, int bm, int *starts, int *scratch)
{
    constexpr int PER = MAX_GROUPS / NT;
    const int t = (int)threadIdx.x, lane = t & 63;
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = PER * t + i;
        n[i] = 0;
        if (e < groups) {
            int lo, hi;
            group_range(offsets, e, rows, lo, hi);
            n[i] = (hi - lo + bm - 1) / bm;
        }
        sum += n[i];
    }
    int before = sum;                                    // inclusive scan over the wavefront
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(before, d);
        if (lane >= d) before += o;
    }
    if (lane == 63) scratch[t >> 6] = before;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
        if (i < (t >> 6)) base += scratch[i];
        total += scratch[i];
    }
    before += base - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        starts[PER * t + i] = before;
        before += n[i];
    }
    __syncthreads();
    return total;
}

// The group of tile `tile` < total and its rows; every wavefront for itself, two LDS reads: the last group whose
// tiles start at or before it (empty groups start where the next one does).
__device__ __forceinline__ GroupRows group_of_tile(const int32_t *offsets, int rows, int bm, const int *starts, int tile)
{
    const int lane = (int)threadIdx.x & 63;
    constexpr int PER = MAX_GROUPS / 64;
    const int block = __builtin_popcountll(__builtin_amdgcn_ballot_w64(starts[PER * lane] <= tile)) - 1;
    const int s = starts[PER * block + (lane & (PER - 1))];
    const int e = PER * block + __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane < PER && s <= tile)) - 1;
    GroupRows g;
    g.group = __builtin_amdgcn_readfirstlane(e);
    int lo, hi;
    group_range(offsets, g.group, rows, lo, hi);
    g.first = __builtin_amdgcn_readfirstlane(lo + (tile - starts[g.group]) * bm);
    g.end = __builtin_amdgcn_readfirstlane(hi);
    return g;
}

} // namespace convrot
