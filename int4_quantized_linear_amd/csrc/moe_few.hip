// moe_few.hip -- the gated expert layer for a few tokens (at most 64 slots): two kernels, or up to two more that quantize
// (gfx950).
//
// With few tokens the layer is its experts' weights streamed once, and the launches around that.  Here
//   moe_few_gate_kernel  h[slot] = bf16(act(g) u):  a workgroup per 16 features and expert
//   moe_few_down_kernel  y = bf16(sum_j weight d + residual):  a workgroup per 16 output channels, all experts
// find the experts' slots from the table of experts themselves (a slot per lane, ballots), and rotate and
// quantize the rows they use themselves, into LDS, where that repeated work is short (FUSED): it runs while the
// workgroup's first weights arrive.  Otherwise the codes come from launch_rotate_quant.
// The weights go from memory to the matrix core's operand registers: v_mfma_i32_16x16x64_i8 takes 16 rows (lane % 16) of 64
// bytes (16 per lane / 16), so four loads per 16 rows fetch 256 contiguous bytes of each; P such chunks are in
// flight per wavefront.  Columns are the rows of x or h of one expert, at most 16 a pass.
// Integer sums are exact and the epilogues are those of the other kernels, so the results are the same bits.
#include "activation.hpp"
#include "device_common.hpp"
#include "launchers.hpp"
#include "rotate_common.hpp"
#include "tile_common.hpp"

namespace convrot {
namespace {

constexpr int MAX_SLOTS = 64;
constexpr int KC = 256;                                  // bytes of a row per chunk

// The expert of slot `lane`, -1 without one (or without a slot).
__device__ __forceinline__ int expert_of_lane(const int32_t *experts, int S, int E)
{
    const int lane = threadIdx.x & 63;
    const int e = lane < S ? experts[lane] : -1;
    return (unsigned)e < (unsigned)E ? e : -1;
}

__device__ __forceinline__ int bits_below(uint64_t m)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// The set bit number first + i of m, for i < min(16, their count - first), in lane i; any number in other lanes.  Every set
// bit's lane sends its own number to the lane of its rank (others to lane 63, where nobody looks).
__device__ __forceinline__ int slot_of_rank(uint64_t m, int first)
{
    const int lane = threadIdx.x & 63, rank = bits_below(m) - first;
    return __builtin_amdgcn_ds_permute(4 * ((m >> lane & 1) && rank >= 0 && rank < 16 ? rank : 63), lane);
}

// One unit of rotation, 256 channels jj of a row, in the 8 lanes of a slot (rotate_common.hpp): requested, and rotated.
template <bool F32>
struct Unit {
    v4u raw[4][F32 ? 2 : 1];
    bool ok;

    __device__ __forceinline__ void fetch(const void *x, int64_t row0, int K, int jj, bool in)
    {
        const int lane = threadIdx.x & 63, qd = lane & 3, h = lane >> 5;
        ok = in;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = 256 * jj + 64 * r + 32 * h + 8 * qd;
            const int64_t at = in && k < K ? row0 + k : 0;           // others read something that is there
            const v4u *src = reinterpret_cast<const v4u *>(static_cast<const uint8_t *>(x) + at * (F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) raw[r][i] = src[i];
        }
    }
    template <int LG>
    __device__ __forceinline__ void rotate(int K, int jj, float (&v)[4][8])
    {
        const int lane = threadIdx.x & 63, qd = lane & 3, h = lane >> 5;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool in = ok && 256 * jj + 64 * r + 32 * h + 8 * qd < K;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float f;
                if constexpr (F32) f = __uint_as_float(raw[r][e >> 2][e & 3]);
                else f = e & 1 ? bf16hi_to_f32(raw[r][0][e >> 1]) : bf16lo_to_f32(raw[r][0][e >> 1]);
                v[r][e] = in ? f : 0.0f;
            }
        }
        fwht_slot<LG>(v, qd);
    }
};

__device__ __forceinline__ float slot_max(const float (&v)[4][8])
{
    float a = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) a = __builtin_fmaxf(a, __builtin_fabsf(v[r][e]));
    a = __builtin_fmaxf(a, dpp_xor1(a));
    a = __builtin_fmaxf(a, dpp_xor2(a));
    uint32_t lo = __float_as_uint(a), hi = lo;
    swap32(lo, hi);
    return __builtin_fmaxf(__uint_as_float(lo), __uint_as_float(hi));
}

struct Rotation {
    float cg, cg_lo;
    double root;
};

template <int LG>
__device__ __forceinline__ float row_scale(float amax, const Rotation &g)
{
    return (LG % 2 == 0 ? amax * g.cg : (float)((double)amax / g.root)) / 127.0f;
}

// Rows of codes in LDS: `stride` bytes each, 16-byte chunk c of every 256 at c ^ row % 16, so that the 16 rows of a fragment
// read fall on distinct banks.
__device__ __forceinline__ uint32_t code_at(int row, int stride, int jj, int chunk)
{
    return (uint32_t)(row * stride + KC * jj + 16 * (chunk ^ (row & 15)));
}

template <int LG>
__device__ __forceinline__ void store_codes(float (&v)[4][8], float sc, const Rotation &g, uint8_t *codes, int row, int stride, int jj)
{
    const int lane = threadIdx.x & 63, qd = lane & 3, h = lane >> 5;
    const float lsign = (((LG > 3 ? qd : 0) ^ (LG > 4 ? qd >> 1 : 0)) & 1) ? -1.0f : 1.0f;
    QuotientRN k = quotient_consts<LG>(sc, lsign, g.cg);
    const bool tiny = sc > 0.0f && sc < 0x1p-100f;       // 1 / sc could overflow: both scaled by 2^64, exactly
    if (__builtin_amdgcn_ballot_w64(tiny) != 0 && tiny) {
        k = quotient_consts<LG>(sc * 0x1p64f, lsign, g.cg);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[r][e] *= 0x1p64f;
    }
    uint32_t c[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        uint32_t t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = rne_bits(quotient_rn<LG>(v[r][e], k, g.cg, g.cg_lo), 1.0f);
        c[r][0] = pack4_i8(t[0], t[1], t[2], t[3]);
        c[r][1] = pack4_i8(t[4], t[5], t[6], t[7]);
    }
    if constexpr (LG > 5) {
#pragma unroll
        for (int r1 = 0; r1 < 2; ++r1) {
            swap32(c[2 * r1][0], c[2 * r1 + 1][0]);
            swap32(c[2 * r1][1], c[2 * r1 + 1][1]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<v2u *>(codes + code_at(row, stride, jj, 4 * r + 2 * h + (qd >> 1)) + 8 * (qd & 1)) = v2u{c[r][0], c[r][1]};
}

// Rows 0 .. n - 1 (row r from element start(r) of x) to codes and scales in LDS, by a workgroup of NW wavefronts; all of it
// calls.  maxima: n words, zeroed.  A wavefront rotates 8 units at a time; its first stay in registers until the
// rows' maxima are known, later ones are rotated again.  requested(): called once the first units are on their way.
template <bool F32, int LG, int NW, typename Start, typename Requested>
__device__ __forceinline__ void quantize_rows(const void *x, Start start, int n, int K, const Rotation &g, uint8_t *codes, int stride,
                                              uint32_t *maxima, float *scales, Requested requested)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, sl = (lane >> 2) & 7;
    const bool lead = (lane & 3) == 0 && lane < 32;
    const int SL = (K + KC - 1) / KC, units = n * SL;
    Unit<F32> unit;
    float kept[4][8];
    auto place = [&](int u0, int &row, int &jj) {
        const int u = u0 + sl;
        row = u < units ? u / SL : 0;
        jj = u - row * SL;
        return u < units;
    };
    auto maximum = [&](const float (&v)[4][8], int row, bool in) {
        const float m = slot_max(v);
        if (lead && in) atomicMax(&maxima[row], __float_as_uint(m));
    };
    int row, jj;
    const bool first = place(8 * w, row, jj);
    unit.fetch(x, start(row), K, jj, first);
    __builtin_amdgcn_sched_barrier(0);
    requested();
    __builtin_amdgcn_sched_barrier(0);
    unit.template rotate<LG>(K, jj, kept);
    maximum(kept, row, first);
    for (int u0 = 8 * (w + NW); u0 < units; u0 += 8 * NW) {
        float v[4][8];
        const bool in = place(u0, row, jj);
        unit.fetch(x, start(row), K, jj, in);
        unit.template rotate<LG>(K, jj, v);
        maximum(v, row, in);
    }
    __syncthreads();
    for (int u0 = 8 * w; u0 < units; u0 += 8 * NW) {
        const bool in = place(u0, row, jj);
        if (u0 != 8 * w) {
            unit.fetch(x, start(row), K, jj, in);
            unit.template rotate<LG>(K, jj, kept);
        }
        const float sc = row_scale<LG>(__uint_as_float(maxima[row]), g);
        if (in) {
            store_codes<LG>(kept, sc, g, codes, row, stride, jj);
            if (jj == 0 && lead) scales[row] = sc;
        }
    }
    __syncthreads();
}

struct FewParams {
    const int32_t *experts;    // [S]
    const float *weights;      // [S]
    const void *x;             // FUSED: the rows to quantize, [tokens, K] (down: h [S, F])
    const int8_t *q;           // otherwise their codes
    const float *qs;           // and scales
    const int8_t *w1, *w2;     // gate, up [E, F, K]; down [E, K, F]
    const float *s1, *s2;
    const uint16_t *residual;  // bf16 [tokens, K] or null
    uint16_t *out;             // h [S, F]; y [tokens, K]
    uint16_t *saved;           // pre [2, S, F]; d [S, K]; or null
    Rotation g;
    int S, E, top, K, F, act, rmax;
};

// ---------------------------------------------------------------------------------------------
// h: workgroup (x, slot); the first slot of each expert does the expert's work, the others end.  It takes the tiles x,
// x + gridDim.x, ... of 16 features, so that the rows are quantized once for several; 4 wavefronts take every fourth chunk of K
// for 16 rows of gate and 16 of up, GP chunks in flight across tiles, and their sums meet in LDS.  One token, 8 of 64 experts,
// 2048 -> 2 x 1024: 12 us, of which the 34 MB of weights would take 7 and a launch, the row's rotation and the end the rest.
constexpr int GNW = 4, GP = 3, GSUMS = GNW * 2 * 4 * 64;

template <bool FUSED, bool F32, int LG>
__global__ void __launch_bounds__(64 * GNW) moe_few_gate_kernel(FewParams p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];       // two tiles' sums, then the codes
    __shared__ uint32_t maxima[16];
    __shared__ float scales[16];
    int32_t *red = reinterpret_cast<int32_t *>(smem);
    uint8_t *codes = smem + 2 * GSUMS * 4;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = p.K, SL = (K + KC - 1) / KC, stride = KC * SL;
    const int mine = expert_of_lane(p.experts, p.S, p.E);
    const int s = blockIdx.y, e = __builtin_amdgcn_readlane(mine, s);
    if (e < 0) return;
    const uint64_t of = __builtin_amdgcn_ballot_w64(mine == e);          // the expert's slots
    if (__builtin_ctzll(of) != s) return;
    const int count = __builtin_popcountll(of);
    const int tiles = (p.F / 16 - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int CW = (SL + GNW - 1) / GNW, L = tiles * CW;                 // chunks per tile of a wavefront, in all
    const __amdgpu_buffer_rsrc_t rq = uniform_rsrc(reinterpret_cast<uint64_t>(p.q), NUM_RECORDS);
    auto feature = [&](int tile) { return 16 * ((int)blockIdx.x + tile * (int)gridDim.x); };
    for (int first = 0; first < count; first += p.rmax) {
        const int n = min(count - first, p.rmax);
        const int slots = slot_of_rank(of, first);
        const int slot = __shfl(slots, min(r, n - 1));   // of this lane's column
        const uint32_t xrow = (uint32_t)(slot / p.top) * (uint32_t)K;
        int ld_tile = 0, ld_c = 0;
        // a chunk's operands: rows r, bytes 256 c + 64 kk + 16 q (past K, and past the last tile: zeros)
        auto load = [&](v4u (&wb)[2][4], v4u (&xb)[4]) {
            const bool any = ld_tile < tiles;
            const int64_t at = ((int64_t)e * p.F + (any ? feature(ld_tile) : 0)) * K;
            const __amdgpu_buffer_rsrc_t rg = uniform_rsrc(reinterpret_cast<uint64_t>(p.w1 + at), any ? 16 * K : 0);
            const __amdgpu_buffer_rsrc_t ru = uniform_rsrc(reinterpret_cast<uint64_t>(p.w2 + at), any ? 16 * K : 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int k = KC * (w + GNW * ld_c) + 64 * kk;
                const uint32_t off = k < K ? (uint32_t)(k + 16 * q) : OOB;
                wb[0][kk] = __builtin_amdgcn_raw_buffer_load_b128(rg, (uint32_t)(r * K) + off, 0, 0);
                wb[1][kk] = __builtin_amdgcn_raw_buffer_load_b128(ru, (uint32_t)(r * K) + off, 0, 0);
                if constexpr (!FUSED) xb[kk] = __builtin_amdgcn_raw_buffer_load_b128(rq, any ? xrow + off : OOB, 0, 0);
            }
            if (++ld_c == CW) {
                ld_c = 0;
                ++ld_tile;
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        v4u wb[GP][2][4], xb[GP][4];
        auto begin = [&] {
#pragma unroll
            for (int i = 0; i < GP; ++i) load(wb[i], xb[i]);
        };
        float sx = FUSED ? 0.0f : p.qs[slot / p.top];
        if constexpr (FUSED) {
            if (threadIdx.x < 16) maxima[threadIdx.x] = 0u;
            __syncthreads();
            quantize_rows<F32, LG, GNW>(p.x, [&](int row) { return (int64_t)(__shfl(slots, row) / p.top) * K; }, n, K, p.g, codes,
                                        stride, maxima, scales, begin);
            sx = scales[min(r, n - 1)];
        } else {
            begin();
        }
        // this thread's output of a tile: row r of the pass, feature 4 q + w
        float sg = 0.0f, su = 0.0f;
        int tile = 0, c = 0;
        v4i acc[2] = {};
        for (int x0 = 0; x0 < L; x0 += GP) {
#pragma unroll
            for (int i = 0; i < GP; ++i) {
                if (c == 0 && tile < tiles) {
                    const int64_t fs = (int64_t)e * p.F + feature(tile) + 4 * q + w;
                    sg = p.s1[fs];
                    su = p.s2[fs];
                }
                const int cc = min(w + GNW * c, SL - 1); // past the end: weights are zeros
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if constexpr (FUSED)
                        xb[i][kk] = *reinterpret_cast<const v4u *>(codes + code_at(min(r, n - 1), stride, cc, 4 * kk + q));
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, wb[i][b][kk]),
                                                                       __builtin_bit_cast(v4i, xb[i][kk]), acc[b], 0, 0, 0);
                }
                load(wb[i], xb[i]);
                if (++c < CW || tile >= tiles) continue;
                // lane: column r, features 4 q + v
                int32_t *to = red + (tile & 1) * GSUMS;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int v = 0; v < 4; ++v) to[((w * 2 + b) * 4 + v) * 64 + lane] = acc[b][v];
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // loads stay in flight
                int32_t ga = 0, ua = 0;
#pragma unroll
                for (int j = 0; j < GNW; ++j) {
                    ga += to[((j * 2 + 0) * 4 + w) * 64 + lane];
                    ua += to[((j * 2 + 1) * 4 + w) * 64 + lane];
                }
                if (r < n) {
                    const float gv = __builtin_fmaf((float)ga, sx * sg, 0.0f), uv = __builtin_fmaf((float)ua, sx * su, 0.0f);
                    const int64_t o = (int64_t)slot * p.F + feature(tile) + 4 * q + w;
                    p.out[o] = (uint16_t)(pack_bf16x2(act_value(gv, p.act) * uv, 0.0f) & 0xffffu);
                    if (p.saved) {
                        const uint32_t gu = pack_bf16x2(gv, uv);
                        p.saved[o] = (uint16_t)(gu & 0xffffu);
                        p.saved[o + (int64_t)p.S * p.F] = (uint16_t)(gu >> 16);
                    }
                }
                acc[0] = acc[1] = v4i{};
                c = 0;
                ++tile;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------
// y: workgroup = 16 output channels, all experts.  A list in LDS holds the experts' products, at most 16 slots each; each
// is cut along F into `parts` of CP chunks, so that 4 wavefronts have about 4 each, and wavefront w takes pieces w, w + 4, ...
// It adds its int32 sums to the slots' in LDS (exact in any order).  Then a thread per token and channel scales,
// weighs and adds up its slots in their order; what that needs from memory is requested at the start.  The same token, 1024
// -> 2048: 11 us, 17 MB: the list, the rotation of 8 rows, one pass of loads and the sums, one after another.
constexpr int DNW = 4, DP = 4;

template <bool FUSED, int LG>
__global__ void __launch_bounds__(64 * DNW) moe_few_down_kernel(FewParams p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];       // FUSED: codes of h
    __shared__ int32_t sums[MAX_SLOTS][16];
    __shared__ float factor[MAX_SLOTS][16];              // down scales of each slot's expert
    __shared__ uint32_t maxima[MAX_SLOTS];
    __shared__ float scales[MAX_SLOTS], share[MAX_SLOTS];
    __shared__ int expert_of[MAX_SLOTS];                 // of a slot
    __shared__ int list_expert[MAX_SLOTS], list_count[MAX_SLOTS];
    __shared__ __attribute__((aligned(16))) uint8_t list_slot[MAX_SLOTS][16];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int F = p.F, SL = (F + KC - 1) / KC, stride = KC * SL;
    const int n0 = 16 * (int)blockIdx.x;
    const int mine = expert_of_lane(p.experts, p.S, p.E);
    // The list, a slot per lane: how many earlier slots have its expert (rank), and the first of its 16 of them.
    int rank = 0, start = lane;
    for (int i = 0; i < p.S; ++i) {
        const bool same = __builtin_amdgcn_readlane(mine, i) == mine && i < lane;
        if (same && rank % 16 == 0) start = i;
        rank += same;
    }
    if (rank % 16 == 0) start = lane;
    const uint64_t starts = __builtin_amdgcn_ballot_w64(mine >= 0 && start == lane);
    const int items = __builtin_popcountll(starts);
    if (w == 0) {
        const int item = __builtin_popcountll(starts & ((1ull << start) - 1));
        expert_of[lane] = mine;
        list_count[lane] = 0;
        *reinterpret_cast<v4u *>(list_slot[lane]) = v4u{};
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (mine >= 0) {
            list_expert[item] = mine;
            list_slot[item][rank % 16] = (uint8_t)lane;
            atomicAdd(&list_count[item], 1);
        }
    }
    for (int i = threadIdx.x; i < p.S * 16; i += 64 * DNW) (&sums[0][0])[i] = 0;
    if ((int)threadIdx.x < p.S) {
        share[threadIdx.x] = p.weights[threadIdx.x];
        if constexpr (FUSED) maxima[threadIdx.x] = 0u;
        else scales[threadIdx.x] = p.qs[threadIdx.x];
    }
    __syncthreads();
    int CP = (items * SL + 4 * DNW - 1) / (4 * DNW);
    CP = min(max(CP, 1), SL);
    const int parts = (SL + CP - 1) / CP, pieces = items * parts;

    const __amdgpu_buffer_rsrc_t rq = uniform_rsrc(reinterpret_cast<uint64_t>(p.q), NUM_RECORDS);
    // A place in this wavefront's walk: piece (item, part) and chunk of the part; past the last piece: nothing.
    struct Place {
        int item, part, c;
    };
    auto step = [&](Place &k) {
        if (++k.c < CP) return;
        k.c = 0;
        k.part += DNW;
        while (k.part >= parts && k.item < items) {
            k.part -= parts;
            ++k.item;
        }
    };
    Place at = {0, w, 0};
    while (at.part >= parts && at.item < items) {
        at.part -= parts;
        ++at.item;
    }
    Place ld = at;
    auto load = [&](v4u (&wb)[4], v4u (&xb)[4]) {
        const bool any = ld.item < items;
        const int i = any ? ld.item : 0, c = ld.part * CP + ld.c;
        const int e = __builtin_amdgcn_readfirstlane(list_expert[i]);
        const __amdgpu_buffer_rsrc_t rw =
            uniform_rsrc(reinterpret_cast<uint64_t>(p.w1 + ((int64_t)e * p.K + n0) * F), any ? 16 * F : 0);
        const uint32_t row = FUSED ? 0u : (uint32_t)list_slot[i][r] * (uint32_t)F;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int k = KC * c + 64 * kk;
            const uint32_t off = k < F ? (uint32_t)(k + 16 * q) : OOB;
            wb[kk] = __builtin_amdgcn_raw_buffer_load_b128(rw, (uint32_t)(r * F) + off, 0, 0);
            if constexpr (!FUSED) xb[kk] = __builtin_amdgcn_raw_buffer_load_b128(rq, any ? row + off : OOB, 0, 0);
        }
        step(ld);
        __builtin_amdgcn_sched_barrier(0);
    };
    v4u wb[DP][4], xb[DP][4];
    auto begin = [&] {
        if (pieces > 0) {
#pragma unroll
            for (int i = 0; i < DP; ++i) load(wb[i], xb[i]);
        }
        for (int i = threadIdx.x; i < p.S * 16; i += 64 * DNW) {
            const int e = expert_of[i >> 4];
            (&factor[0][0])[i] = e < 0 ? 0.0f : p.s1[(int64_t)e * p.K + n0 + (i & 15)];
        }
    };
    if constexpr (FUSED) quantize_rows<false, LG, DNW>(p.x, [&](int row) { return (int64_t)row * F; }, p.S, F, p.g, smem, stride,
                                                       maxima, scales, begin);
    else begin();
    v4i acc = {};
    while (at.item < items) {
#pragma unroll
        for (int i = 0; i < DP; ++i) {
            const bool any = at.item < items;
            const int item = any ? at.item : 0, slot = list_slot[item][r], c = at.part * CP + at.c;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if constexpr (FUSED)
                    xb[i][kk] = *reinterpret_cast<const v4u *>(smem + code_at(slot, stride, any ? min(c, SL - 1) : 0, 4 * kk + q));
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, wb[i][kk]), __builtin_bit_cast(v4i, xb[i][kk]),
                                                            acc, 0, 0, 0);
            }
            if (any && at.c == CP - 1) {
                if (r < list_count[item]) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) atomicAdd(&sums[slot][4 * q + v], acc[v]);
                }
                acc = v4i{};
            }
            step(at);
            load(wb[i], xb[i]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.S / p.top * 16; i += 64 * DNW) {
        const int m = i >> 4, n = i & 15;
        const int64_t o = (int64_t)m * p.K + n0 + n;
        const float res = p.residual ? bf16lo_to_f32(p.residual[o]) : 0.0f;
        float v = 0.0f;
        for (int j = 0; j < p.top; ++j) {
            const int s = m * p.top + j;
            const float d = __builtin_fmaf((float)sums[s][n], scales[s] * factor[s][n], 0.0f);
            if (expert_of[s] < 0) continue;
            v = __builtin_fmaf(share[s], d, v);
            if (p.saved) p.saved[(int64_t)s * p.K + n0 + n] = (uint16_t)(pack_bf16x2(d, 0.0f) & 0xffffu);
        }
        p.out[o] = (uint16_t)(pack_bf16x2(v + res, 0.0f) & 0xffffu);
    }
}

Rotation rotation(int log2g)
{
    Rotation g;
    g.root = __builtin_sqrt((double)(1 << log2g));
    g.cg = (float)(1.0 / g.root);
    g.cg_lo = (float)(1.0 / g.root - (double)g.cg);
    return g;
}

constexpr int GWG = 512;

template <bool F32, int LG>
void launch_gate(const FewParams &p, dim3 grid, size_t lds, hipStream_t stream)
{
    hipLaunchKernelGGL((moe_few_gate_kernel<true, F32, LG>), grid, dim3(64 * GNW), lds, stream, p);
}

#define CONVROT_LOG2G(fn, ...)           \
    switch (log2g) {                     \
    case 0: fn(0, __VA_ARGS__); break;   \
    case 1: fn(1, __VA_ARGS__); break;   \
    case 2: fn(2, __VA_ARGS__); break;   \
    case 3: fn(3, __VA_ARGS__); break;   \
    case 4: fn(4, __VA_ARGS__); break;   \
    case 5: fn(5, __VA_ARGS__); break;   \
    case 6: fn(6, __VA_ARGS__); break;   \
    case 7: fn(7, __VA_ARGS__); break;   \
    default: fn(8, __VA_ARGS__);         \
    }

} // namespace

bool plan_moe_few(int64_t M, int top, int K, int F, MoeFew &plan)
{
    if (M * top > MAX_SLOTS) return false;
    // How many 256-channel units a workgroup may rotate.  x: the rows of one expert, at most 16 at a time (so the codes take at
    // most 32 KiB), under its weights' loads; layer calls, us, apart / fused: 12 tokens, 2 of 8, 2048 -> 512, 96 units 26.5 / 24.1;
    // 4, 2 of 8, 5120 -> 5120, 80 units 113 / 105; 20, 3 of 16, 2048 -> 512, 160 units 34.6 / 31.5; 32, 2 of 8, 2048, 256
    // units 38.6 / 38.6.  h: all slots, in every workgroup; 8 of 64, 2048 -> 1024, 1 token, 32 units 26.5 / 22.1; 2, 64 units
    // 33.2 / 32.7; 3, 96 units 41.0 / 42.2; 4, 128 units 52.1 / 54.7.
    const int slk = (K + KC - 1) / KC, slf = (F + KC - 1) / KC;
    plan.fuse_x = M * slk <= 256 && (M < 16 ? M : 16) * slk <= 128;
    plan.fuse_h = M * top * slf <= 64;
    return true;
}

hipError_t launch_moe_few_gate(const MoeFewArgs &a, const MoeFew &plan, hipStream_t stream)
{
    FewParams p = {};
    p.experts = a.experts;
    p.x = a.x;
    p.q = a.xq;
    p.qs = a.xs;
    p.w1 = a.wq_gate;
    p.w2 = a.wq_up;
    p.s1 = a.gate_scale;
    p.s2 = a.up_scale;
    p.out = a.h;
    p.saved = a.pre;
    p.S = (int)a.M * a.top;
    p.E = a.E;
    p.top = a.top;
    p.K = a.K;
    p.F = a.F;
    p.act = a.act;
    p.rmax = a.M < 16 ? (int)a.M : 16;
    const int log2g = a.log2g;
    p.g = rotation(log2g);
    // about GWG workgroups in all, each with as many tiles
    const int used = p.S < a.E ? p.S : a.E, tiles = a.F / 16, wgs = used < GWG ? (GWG + used - 1) / used : 1;
    const dim3 grid((unsigned)(tiles < wgs ? tiles : wgs), (unsigned)p.S);
    const size_t lds = 2 * GSUMS * 4 + (plan.fuse_x ? (size_t)p.rmax * ((a.K + KC - 1) / KC) * KC : 0);
    if (!plan.fuse_x) {
        hipLaunchKernelGGL((moe_few_gate_kernel<false, false, 0>), grid, dim3(64 * GNW), lds, stream, p);
        return hipGetLastError();
    }
#define CONVROT_GATE(lg, f32)                                   \
    if (f32) launch_gate<true, lg>(p, grid, lds, stream);       \
    else launch_gate<false, lg>(p, grid, lds, stream)
    CONVROT_LOG2G(CONVROT_GATE, a.x_f32)
#undef CONVROT_GATE
    return hipGetLastError();
}

hipError_t launch_moe_few_down(const MoeFewArgs &a, const MoeFew &plan, hipStream_t stream)
{
    FewParams p = {};
    p.experts = a.experts;
    p.weights = a.weights;
    p.x = a.h;
    p.q = a.hq;
    p.qs = a.hs;
    p.w1 = a.wq_down;
    p.s1 = a.down_scale;
    p.residual = a.residual;
    p.out = a.y;
    p.saved = a.d;
    p.S = (int)a.M * a.top;
    p.E = a.E;
    p.top = a.top;
    p.K = a.K;
    p.F = a.F;
    const int log2g = a.log2g_h;
    p.g = rotation(log2g);
    const dim3 grid((unsigned)(a.K / 16)), block(64 * DNW);
    const size_t lds = plan.fuse_h ? (size_t)p.S * ((a.F + KC - 1) / KC) * KC : 0;
    if (!plan.fuse_h) {
        hipLaunchKernelGGL((moe_few_down_kernel<false, 0>), grid, block, 0, stream, p);
        return hipGetLastError();
    }
#define CONVROT_DOWN(lg, unused) hipLaunchKernelGGL((moe_few_down_kernel<true, lg>), grid, block, lds, stream, p)
    CONVROT_LOG2G(CONVROT_DOWN, 0)
#undef CONVROT_DOWN
    return hipGetLastError();
}

#undef CONVROT_LOG2G

} // namespace convrot
