// tile_common.hpp -- what the tiled matrix kernels share: buffer descriptors, wait counts and the
// order in which workgroups take tiles.  Internal to libconvrot.
#pragma once
#include "device_common.hpp"

namespace convrot {

typedef __attribute__((address_space(3))) void lds_void;

constexpr uint32_t OOB = 0x80000000u;         // buffer offset past num_records: loads return 0, stores drop
constexpr int NUM_RECORDS = 0x7ffffff0;
constexpr int GROUP_M = 4;

// Buffer descriptor from a wave-uniform address and size, built from readfirstlane'd halves so it
// stays in scalar registers.  (readfirstlane returns int: each half goes through uint32_t, so the
// low half is zero-extended, not sign-extended, into the 64-bit address.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(uint64_t a, int bytes)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(((uint64_t)hi << 32) | (uint64_t)lo), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// s_waitcnt immediate (gfx9 encoding) waiting for vmcnt <= n only.
constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0f70; }

// 16 bytes per lane, global -> LDS (lane l to lds + 16 l).  A function of its own, not a template: the
// host pass silently drops a kernel template whose dependent code uses this gfx950-only size.
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t src, void *lds, uint32_t off, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void *)lds, 16, off, soff, 0, 0);
}

// Unit of virtual id pid (= blockIdx.x + k * gridDim.x, gridDim.x a multiple of 8).  Dispatch ids
// are spread round-robin over the 8 XCDs, so pid keeps its XCD.  Units 0..T_dp-1 are the whole
// tiles, then come the split units; each XCD walks a contiguous range of the whole tiles, then a
// contiguous range of the split units (T_dp is a multiple of 8 whenever there are split units, so
// this is a bijection of [0, U)).
__device__ __forceinline__ int unit_of(int pid, int T_dp, int U)
{
    const int xcd = pid & 7, local = pid >> 3;
    const int dper = T_dp >> 3, drem = T_dp & 7;
    const int dn = dper + (xcd < drem);
    if (local < dn) return xcd * dper + min(xcd, drem) + local;
    const int ut = U - T_dp, tper = ut >> 3, trem = ut & 7;
    return T_dp + xcd * tper + min(xcd, trem) + (local - dn);
}

// Tile q of the M-grouped order: groups of GROUP_M tile rows, walked column by column, so the
// tiles an XCD runs at the same time share their weight tiles in its L2.
__device__ __forceinline__ void tile_coords(int q, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int span = GROUP_M * tiles_n;
    const int first_m = (q / span) * GROUP_M;
    const int gsz = min(tiles_m - first_m, GROUP_M);
    const int r = q % span;
    tm = first_m + r % gsz;
    tn = r / gsz;
}

// Position of a 16-byte chunk in a 128-byte LDS row: chunk ^ swz(row) spreads 16 consecutive rows'
// reads of one chunk over all banks.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

} // namespace convrot
