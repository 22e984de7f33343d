// grouped_i8.hip -- products of rows sorted by group (expert) with their group's INT8 weight, and what a
// mixture-of-experts layer needs around them (gfx950).
//
//   moe_order_kernel    slots sorted by expert: the groups' offsets, slot and token of each row, row of each slot
//   grouped_tile_kernel acc[r, n] = sum_k xq[src(r), k] wq[group(r), n, k] with one of three epilogues
//   moe_combine_kernel  y[m] = bf16(sum_j weight[m, j] part[row(m, j)] + residual[m])
#include "activation.hpp"
#include "device_common.hpp"
#include "grouped_common.hpp"
#include "launchers.hpp"
#include "tile_common.hpp"

namespace convrot {
namespace {

// ---------------------------------------------------------------------------------------------
// Slots sorted by expert, in their own order within an expert (a counting sort).  Workgroup e of E + 1 reads all
// slots, counts those of smaller experts, which is where its rows begin, and then writes the rows of its own; the
// last one takes the slots without an expert and the total.  Workgroups need nothing from one another, so this is one
// launch with the same result at every call.  Bound by each workgroup's read of all slots.
struct OrderParams {
    const int32_t *experts;    // [S]
    int32_t *offsets;          // [E + 1]
    int32_t *slot_of, *token_of;   // [S] of each row
    int32_t *row_of;           // [S] of each slot, -1 without an expert
    const float *sx;           // [tokens] or null
    float *sx_of;              // [S] of each row
    int S, E, top;
};

typedef v4i v4i_any __attribute__((aligned(4)));

// Whether a slot with expert x is workgroup e's own (e == E: of none), and whether it has a smaller expert.
__device__ __forceinline__ bool order_mine(const OrderParams &p, int e, int x)
{
    return e == p.E ? (unsigned)x >= (unsigned)p.E : x == e;
}
__device__ __forceinline__ bool order_less(int e, int x) { return (unsigned)x < (unsigned)e; }

// Tokens and scales of the rows that the workgroup has put in their places.
template <int NT>
__device__ __forceinline__ void order_end(const OrderParams &p, int first, int rows)
{
    __syncthreads();
    for (int r = first + (int)threadIdx.x; r < first + rows; r += NT) {
        const int token = p.slot_of[r] / p.top;
        p.token_of[r] = token;
        if (p.sx) p.sx_of[r] = p.sx[token];
    }
}

// Up to 4 HELD <= 32 slots per thread, requested at once and kept between the two passes as a bit each, so that the
// second takes as many steps as the fullest lane has rows (24576 slots of 64 experts: 19 us with a division and a load in
// the second pass's branch over every slot, 10 so).
template <int NT, int HELD>
__global__ void __launch_bounds__(NT) moe_order_kernel(OrderParams p)
{
    __shared__ int2 part[NT / 64];
    const int t = (int)threadIdx.x, lane = t & 63, e = (int)blockIdx.x;
    const int s0 = min(t * 4 * HELD, p.S), s1 = min(s0 + 4 * HELD, p.S);
    v4i held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int s = s0 + 4 * i;
        if (s + 4 <= s1) held[i] = *reinterpret_cast<const v4i_any *>(p.experts + s);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k) held[i][k] = s + k < s1 ? p.experts[s + k] : 0;
    }
    const int n = s1 - s0;
    const uint32_t real = n >= 32 ? ~0u : (1u << n) - 1u;
    uint32_t mask = 0, below = 0;
#pragma unroll
    for (int i = 0; i < 4 * HELD; ++i) {
        mask |= (uint32_t)order_mine(p, e, held[i / 4][i % 4]) << i;
        below |= (uint32_t)order_less(e, held[i / 4][i % 4]) << i;
    }
    mask &= real;
    const int n_mine = __popc(mask);
    int before = n_mine, all = __popc(below & real);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(before, d);
        if (lane >= d) before += o;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) all += __shfl_xor(all, d);
    if (lane == 63) part[t >> 6] = int2{before, all};
    __syncthreads();
    int row = before - n_mine, first = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
        if (i < (t >> 6)) row += part[i].x;
        rows += part[i].x;
        first += part[i].y;
    }
    if (t == 0) p.offsets[e] = first;
    row += first;
    for (; mask; mask &= mask - 1, ++row) {
        const int s = s0 + __ffs(mask) - 1;
        p.row_of[s] = e == p.E ? -1 : row;
        if (e < p.E) p.slot_of[row] = s;
    }
    if (e < p.E) order_end<NT>(p, first, rows);
}

// Any number of slots: each wavefront takes a run of them, 256 at a time (lane l: 4 l .. 4 l + 3), reads it twice and
// ranks its own by ballots.  131072 slots of 256 experts: 42 us, each workgroup's two reads of all slots (with the threads' own
// runs, as above but read twice, 91: a lane's lines are then its own and leave the cache between its reads).
__global__ void __launch_bounds__(1024) moe_order_long_kernel(OrderParams p)
{
    constexpr int NT = 1024, NW = NT / 64, AHEAD = 4;    // blocks requested at once
    __shared__ int2 part[NW];
    const int t = (int)threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), e = (int)blockIdx.x;
    const int run = (((p.S + NW - 1) / NW) + 255) & ~255;
    const int s0 = (int)min((int64_t)w * run, (int64_t)p.S), s1 = min(s0 + run, p.S);
    auto load = [&](int b) {                             // (no branch among lanes: one would wait for each load)
        v4i x = {};
        const int s = b + 4 * lane;
        if (b + 256 <= s1) {
            x = *reinterpret_cast<const v4i_any *>(p.experts + s);
        } else if (b < s1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = p.experts[min(s + k, p.S - 1)];
        }
        return x;
    };
    auto each = [&](auto f) {
        for (int b = s0; b < s1; b += 256 * AHEAD) {
            v4i x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) x[i] = load(b + 256 * i);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (b + 256 * i < s1) f(b + 256 * i + 4 * lane, x[i]);
        }
    };
    int n_mine = 0, n_less = 0;
    each([&](int s, const v4i &x) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            n_mine += s + k < s1 && order_mine(p, e, x[k]);
            n_less += s + k < s1 && order_less(e, x[k]);
        }
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        n_mine += __shfl_xor(n_mine, d);
        n_less += __shfl_xor(n_less, d);
    }
    if (lane == 0) part[w] = int2{n_mine, n_less};
    __syncthreads();
    int row = 0, first = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < w) row += part[i].x;
        rows += part[i].x;
        first += part[i].y;
    }
    if (t == 0) p.offsets[e] = first;
    row += first;
    if (__builtin_amdgcn_readfirstlane(n_mine) > 0)
        each([&](int s, const v4i &x) {
            bool m[4];
            uint64_t lanes[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = s + k < s1 && order_mine(p, e, x[k]);
                lanes[k] = __builtin_amdgcn_ballot_w64(m[k]);
            }
            if ((lanes[0] | lanes[1] | lanes[2] | lanes[3]) == 0) return;
            int at = row;                                // the lane's first
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                at += __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes[k] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes[k], 0u));
                row += __builtin_popcountll(lanes[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (m[k]) {
                    p.row_of[s + k] = e == p.E ? -1 : at;
                    if (e < p.E) p.slot_of[at] = s + k;
                    ++at;
                }
        });
    if (e < p.E) order_end<NT>(p, first, rows);
}

// ---------------------------------------------------------------------------------------------
// The product, BM (64 or 128) rows x 128 weight rows per unit: gemm_i8_tile_kernel's tiles (K in tiles of 128 bytes through
// NST LDS stages, one barrier per K-tile, 4 wavefronts in 2 x 2, two workgroups per CU), walking units blockIdx.x,
// blockIdx.x + gridDim.x, ... of a count that only the GPU knows.  The loads run NST - 1 K-tiles ahead across
// units, so a unit's epilogue (in the stage of its last K-tile) runs while the next one's first K-tiles arrive; what a
// unit's start needs from memory, its source rows, scales and slots, is requested one unit ahead, into registers.
// Few rows per group: bound by the weights' stream; 12 tokens, 8 of 128 experts, 5120 -> 2 x 1280: 166 us, 4.5 TB/s.  301 tokens,
// 3 of 16, 2688 -> 2 x 1344: 39 us, 3 TB/s: a K-tile of all 350 tiles takes 1.4 us, 3.9 TB/s, a tile's start and end 8 us.
constexpr int BN = 128, BK = 128;
constexpr int NTHREADS = 256;

struct GroupedParams {
    const int8_t *xq;          // codes of the source rows
    const float *sx;
    const int32_t *offsets;
    const int32_t *source;     // source row of a row, or null: the row itself
    const int32_t *slot_of;    // where pre and d keep a row, or null: the row itself
    const int8_t *wq, *wq2;    // [groups, N, K]
    const float *sw, *sw2;     // [groups, N]
    uint16_t *y;               // Plain: bf16 [rows, N]; Gated: bf16(act(g) u) [rows, N]
    float *part;               // Part: fp32 [rows, N]
    uint16_t *pre;             // Gated: bf16 [2, pre_rows, N] or null
    uint16_t *d;               // Part: bf16 [slots, N] or null
    int64_t pre_rows;
    int rows, groups, N, K, tiles_n, act;
};

typedef v4u v4u_any __attribute__((aligned(2)));         // 16 bytes at any element (an odd N)

template <Epi E>
constexpr int features() { return E == Epi::Gated ? BN / 2 : BN; }

// Rows of 8 columns n.. to dst, clipped at N (VEC: N % 8 == 0, all exist).
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *dst, int n, int N, const float (&a)[8])
{
    const v4u d = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])};
    if (VEC || n + 8 <= N) {
        *reinterpret_cast<v4u_any *>(dst) = d;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + e < N) dst[e] = (uint16_t)(e & 1 ? d[e >> 1] >> 16 : d[e >> 1] & 0xffffu);
    }
}

template <Epi E, int BM, int NST, bool VEC>
__global__ void __launch_bounds__(NTHREADS, 2) grouped_tile_kernel(GroupedParams p)
{
    constexpr int NF = features<E>();
    constexpr int STAGE = (BN + BM) * BK;
    constexpr int LPK = (BN + BM) / 32;                  // loads per K-tile and wave
    constexpr int XL = LPK - 4;                          // of them rows of x
    constexpr int MB = BM / 32;                          // 16-row blocks per wave
    __shared__ __attribute__((aligned(16))) uint8_t smem[NST * STAGE];
    __shared__ GroupTable table;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = w & 1, wm = w >> 1;
    const int K = p.K;
    const int KT = max((K + BK - 1) / BK, NST - 1);      // at least the K-tiles in flight (past K: zeros)
    int last;
    const int tiles = group_tiles<NTHREADS>(p.offsets, p.groups, p.rows, BM, table, reinterpret_cast<int *>(smem), last);
    const int units = tiles * p.tiles_n;
    if ((int)blockIdx.x >= units) return;
    const int frow = lane & 15, fq = lane >> 4;
    // epilogue: rows of 8 output columns per lane
    constexpr int LPR = NF / 2 / 8, RPI = 64 / LPR;      // lanes per row, rows at a time
    const int lrow = lane / LPR, lcol = lane % LPR;

    struct Unit {
        GroupRows g;
        int n0;
    };
    auto locate = [&](int v) {
        Unit u;
        int tm, tn;
        tile_coords(unit_of(v, 0, units), tiles, p.tiles_n, tm, tn);
        u.g = group_of_tile(table, BM, last, tm);
        u.n0 = tn * NF;
        return u;
    };
    // The load side.  Instruction i of wave w fills LDS rows 8 (4 i + w) .. + 7 (weight rows 0 .. 127, then rows of x);
    // lane -> row + lane / 8 at position lane % 8.
    const int ldr = 8 * w + (lane >> 3), ldc = 16 * ((lane & 7) ^ swz(ldr));   // swz(row) is swz(ldr) for every i
    const uint32_t half = K % BK && ldc >= 64 ? OOB : 0u;
    int src[XL] = {};                                    // source rows of the unit that the load side takes next
    auto request = [&](int v) {
        if (!p.source || v >= units) return;
        const Unit u = locate(v);
#pragma unroll
        for (int i = 0; i < XL; ++i) src[i] = p.source[min(u.g.first + 32 * i + ldr, u.g.end - 1)];
    };
    uint32_t off[LPK], none = 0u;                        // none: OOB past the last unit
    uint64_t wbase = 0, xbase = 0;
    int ld_t = 0;
    // what the epilogue of the load side's unit will need, requested with its first K-tile
    float s1[8], s2[8], sx;
    int slot = 0;
    auto load_unit = [&](int v) {
        ld_t = 0;
        none = v < units ? 0u : OOB;
        if (v >= units) return;
        const Unit u = locate(v);
        const int left = u.g.end - u.g.first;
#pragma unroll
        for (int i = 0; i < LPK; ++i) {
            const int r = 32 * i + ldr;
            if (i < 4) {
                const int wr = E == Epi::Gated ? 16 * (r >> 5) + (r & 15) : r;
                off[i] = u.n0 + wr < p.N ? (uint32_t)(wr * K + ldc) : OOB;
            } else {
                const int rr = r - BN;
                off[i] = rr < left ? (uint32_t)((p.source ? src[i - 4] : rr) * K + ldc) : OOB;
            }
        }
        const int64_t g0 = (int64_t)u.g.group * p.N;
        const int8_t *wsrc = E == Epi::Gated && (w & 2) ? p.wq2 : p.wq;   // rows 16..31 of each 32: up
        wbase = reinterpret_cast<uint64_t>(wsrc + (g0 + u.n0) * K);
        xbase = reinterpret_cast<uint64_t>(p.source ? p.xq : p.xq + (int64_t)u.g.first * K);
        const int n = u.n0 + wn * (NF / 2) + 8 * lcol;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t i = g0 + min(n + e, p.N - 1);
            s1[e] = p.sw[i];
            if constexpr (E == Epi::Gated) s2[e] = p.sw2[i];
        }
        const int row = min(u.g.first + wm * (BM / 2) + lane % (BM / 2), u.g.end - 1);   // lane l: row l of the wave's
        sx = p.sx[row];
        if (E != Epi::Bf16 && p.slot_of) slot = p.slot_of[row];
        request(v + (int)gridDim.x);
    };
    int st = 0;                                          // stage of the compute side's K-tile
    auto issue = [&](int stage) {
        const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(wbase, NUM_RECORDS), rx = uniform_rsrc(xbase, NUM_RECORDS);
        uint8_t *base = smem + stage * STAGE + w * 1024;
        const int k0 = ld_t * BK;
        const uint32_t skip = none | (k0 >= K ? OOB : k0 + BK > K ? half : 0u);
#pragma unroll
        for (int i = 0; i < LPK; ++i)
            load16_to_lds(i < 4 ? rw : rx, base + 4096 * i, off[i] | skip, __builtin_amdgcn_readfirstlane(k0));
        ++ld_t;
    };

    request((int)blockIdx.x);
    load_unit((int)blockIdx.x);
#pragma unroll
    for (int j = 0; j < NST - 1; ++j) issue(j);
    for (int v = blockIdx.x; v < units; v += gridDim.x) {
        const Unit u = locate(v);
        float c1[8], c2[8], csx = 0.0f;                  // this unit's, while the load side moves on
        int cslot = 0;
        v4i acc[4][MB];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[a][b] = v4i{};
        for (int t = 0; t < KT; ++t) {
            // K-tile t has landed once only the NST - 2 after it are in flight
            __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * LPK));
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (t == KT - (NST - 1)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    c1[e] = s1[e];
                    if constexpr (E == Epi::Gated) c2[e] = s2[e];
                }
                csx = sx;
                cslot = slot;
                load_unit(v + (int)gridDim.x);
            }
            issue(st == 0 ? NST - 1 : st - 1);           // the stage read before this one
            const uint8_t *base = smem + st * STAGE;
            const uint8_t *ar = base + (wn * 64 + frow) * BK, *br = base + (BN + wm * (BM / 2) + frow) * BK;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int pos = 16 * ((4 * kk + fq) ^ swz(frow));
                v4i fa[4], fb[MB];
#pragma unroll
                for (int b = 0; b < 4; ++b) fa[b] = *reinterpret_cast<const v4i *>(ar + 16 * b * BK + pos);
#pragma unroll
                for (int b = 0; b < MB; ++b) fb[b] = *reinterpret_cast<const v4i *>(br + 16 * b * BK + pos);
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < MB; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[a], fb[b], acc[a][b], 0, 0, 0);
            }
            if (t + 1 < KT) st = st == NST - 1 ? 0 : st + 1;
        }
        // Lane: row lane % 16 of block b, weight rows 16 a + 4 (lane / 16) + v of the wave's 64.  Each wave passes
        // its 16-row blocks through 4 KiB of the last K-tile's stage (rows of 64 sums, 16-byte chunk c at c ^ row), which every
        // wave has read by now and the loads leave alone until the next unit's first barrier.
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        uint8_t *reg = smem + st * STAGE + w * 4096;
        const int n = u.n0 + wn * (NF / 2) + 8 * lcol, left = u.g.end - u.g.first;
        const int ch = E == Epi::Gated ? 8 * (lcol >> 1) + 2 * (lcol & 1) : 2 * lcol;
#pragma unroll
        for (int b = 0; b < MB; ++b) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
                *reinterpret_cast<v4i *>(reg + frow * 256 + 16 * ((4 * a + fq) ^ frow)) = acc[a][b];
#pragma unroll 1
            for (int q = 0; q < 16 / RPI; ++q) {
                const int r = RPI * q + lrow, rw = 16 * b + r, rl = wm * (BM / 2) + rw;
                const float sxm = __shfl(csx, rw);
                const int64_t to = E != Epi::Bf16 ? __shfl(cslot, rw) : 0;
                if (rl >= left || n >= p.N) continue;
                const int64_t row = u.g.first + rl;
                auto z8 = [&](int chunk, const float (&s)[8], float (&z)[8]) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const v4i d = *reinterpret_cast<const v4i *>(reg + r * 256 + 16 * ((chunk + h) ^ r));
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[4 * h + i] = __builtin_fmaf((float)d[i], sxm * s[4 * h + i], 0.0f);
                    }
                };
                float z[8], g[8];
                z8(ch, c1, z);
                if constexpr (E == Epi::Bf16) store8<VEC>(p.y + row * p.N + n, n, p.N, z);
                if constexpr (E == Epi::Part) {
                    float *dst = p.part + row * p.N + n;
                    *reinterpret_cast<v4f *>(dst) = v4f{z[0], z[1], z[2], z[3]};
                    *reinterpret_cast<v4f *>(dst + 4) = v4f{z[4], z[5], z[6], z[7]};
                    if (p.d) store8<VEC>(p.d + to * p.N + n, n, p.N, z);
                }
                if constexpr (E == Epi::Gated) {
                    z8(ch + 4, c2, g);
                    if (p.pre) {
                        uint16_t *dst = p.pre + to * p.N + n;
                        store8<VEC>(dst, n, p.N, z);
                        store8<VEC>(dst + p.pre_rows * p.N, n, p.N, g);
                    }
                    act_values(z, p.act);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] *= g[e];
                    store8<VEC>(p.y + row * p.N + n, n, p.N, z);
                }
            }
        }
        st = st == NST - 1 ? 0 : st + 1;
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));           // the last loads into LDS
}

// ---------------------------------------------------------------------------------------------
// A thread takes 4 channels of one token; all slots' parts are requested before the first is added, in slot
// order.  Slots without an expert add nothing.  Bound by memory: 4096 tokens of 6 slots, 2048 channels: 40 us, 5.8
// TB/s.  (The parts as 16-bit integers with a scale per 64 channels are half the bytes, 30 us and 5% of that layer, but a channel
// 1000 times smaller than the largest of the 64 then keeps fewer bits than bf16 has.)
struct CombineParams {
    const float *part;         // [rows, K]
    const int32_t *row_of;     // [M, top]
    const float *weights;      // [M, top], or null: 1
    const uint16_t *residual;  // bf16 [M, K] or null
    uint16_t *y;
    int64_t units;             // M K / 4
    int K, top;
};

__global__ void __launch_bounds__(256) moe_combine_kernel(CombineParams p)
{
    constexpr int AHEAD = 8;
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= p.units) return;
    const int per = p.K / 4;
    const int64_t m = u / per;
    const int c = 4 * (int)(u - m * per);
    v2u res = {};
    if (p.residual) res = *reinterpret_cast<const v2u *>(p.residual + m * p.K + c);
    float v[4] = {};
#pragma unroll 1
    for (int j = 0; j < p.top; j += AHEAD) {
        v4f a[AHEAD];
        float w[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            a[i] = v4f{};
            w[i] = 0.0f;
            if (j + i < p.top) {
                const int64_t row = p.row_of[m * p.top + j + i];
                if (row >= 0) {
                    a[i] = *reinterpret_cast<const v4f *>(p.part + row * p.K + c);
                    w[i] = p.weights ? p.weights[m * p.top + j + i] : 1.0f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(w[i], a[i][e], v[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += e & 1 ? bf16hi_to_f32(res[e >> 1]) : bf16lo_to_f32(res[e >> 1]);
    *reinterpret_cast<v2u *>(p.y + m * p.K + c) = v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

constexpr int GRID = 512;                                // two workgroups per CU

template <Epi E, int BM, int NST, bool VEC>
void launch_tiles(const GroupedParams &p, hipStream_t stream)
{
    // a multiple of 8, so that a workgroup's units stay on its XCD
    const int64_t most = most_group_tiles(p.rows, p.groups, BM) * p.tiles_n;
    const unsigned grid = most < GRID ? (unsigned)((most + 7) & ~7) : (unsigned)GRID;
    hipLaunchKernelGGL((grouped_tile_kernel<E, BM, NST, VEC>), dim3(grid), dim3(NTHREADS), 0, stream, p);
}

// Rows per tile, 64, 128 or 256, by a model with measured constants (us).  A CU takes `step` per K-tile and `end` per
// unit of several, a lone workgroup `lone` per K-tile; a group's last tile is half empty; the weights stream at 4.9 TB/s.
// Measured, whole calls, 64 / 128 / 256 rows:
//   linear_grouped, rows, groups, K x N:  2500, 6, 2688 x 1001: 38 / 42 / 67;   2000, 8, 2048 x 2048: 39 / 29 / 36
//     4000, 8, 2688 x 5376: 148 / 107 / 94;   8192, 16, 5376 x 5376: 591 / 388 / 310
//   expert layer, tokens, top of E, K x F:  12, 6 of 64, 2048 x 1408: 100 / 107 / 123;  600, 2 of 8, 2688 x 2688: 111 / 122 / 115
//     (107 with a height for each product);   1000, 4 of 32, 2048 x 1408: 159 / 147 / 140;   1500, 2 of 8, 5120 x 1280:
//     196 / 203 / 165;   4096, 6 of 64, 2048 x 1408: 617 / 488 / 406
int rows_per_tile(int64_t rows, int groups, int64_t N, int K, Epi epi)
{
    const double cols = (double)N * (epi == Epi::Gated ? 2.0 : 1.0), used = (double)(groups < rows ? groups : rows);
    const double stream = used * cols * K / 4.9e6;
    const int KT = (K + BK - 1) / BK;
    int best_bm = 64;
    double best = 1e30;
    for (int bm = 64; bm <= 256; bm *= 2) {
        const double width = bm == 256 ? 256.0 : 128.0;
        const double step = bm == 64 ? 0.55 : bm == 128 ? 0.72 : 1.72, lone = bm == 64 ? 0.85 : bm == 128 ? 1.1 : 1.72;
        const double end = bm == 64 ? 1.5 : bm == 128 ? 2.5 : epi == Epi::Bf16 ? 5.0 : 7.0;
        const double tiles = (double)rows / bm + 0.5 * used;
        const double units = (tiles > used ? tiles : used) * __builtin_ceil(cols / width);
        // rounds: the last one is half full on average (in 256 rows, then it takes less), unless the tiles are surely no more
        // than the CUs
        const double rounds = units < 220.0 ? 1.0 : units / 256.0 + (bm == 256 ? 0.33 : 0.5);
        const double many = rounds * (KT * step + end), one = KT * lone + end;
        double t = many > one ? many : one;
        if (t < stream) t = stream + end;
        if (t < best) {
            best = t;
            best_bm = bm;
        }
    }
    return best_bm;
}

template <Epi E, bool VEC>
void launch_rows(const GroupedParams &p, int bm, hipStream_t stream)
{
    if (bm == 64) launch_tiles<E, 64, 3, VEC>(p, stream);
    else launch_tiles<E, 128, 2, VEC>(p, stream);
}

} // namespace

hipError_t launch_moe_order(const int32_t *experts, int64_t S, int E, int top, const MoeOrder &o, hipStream_t stream)
{
    OrderParams p;
    p.experts = experts;
    p.offsets = o.offsets;
    p.slot_of = o.slot_of;
    p.token_of = o.token_of;
    p.row_of = o.row_of;
    p.sx = o.sx;
    p.sx_of = o.sx_of;
    p.S = (int)S;
    p.E = E;
    p.top = top;
    const dim3 grid(E + 1);
    if (S <= 1024) hipLaunchKernelGGL((moe_order_kernel<256, 1>), grid, dim3(256), 0, stream, p);
    else if (S <= 8192) hipLaunchKernelGGL((moe_order_kernel<1024, 2>), grid, dim3(1024), 0, stream, p);
    else if (S <= 32768) hipLaunchKernelGGL((moe_order_kernel<1024, 8>), grid, dim3(1024), 0, stream, p);
    else hipLaunchKernelGGL(moe_order_long_kernel, grid, dim3(1024), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_grouped_i8(const GroupedArgs &g, Epi epi, hipStream_t stream)
{
    if (g.rows <= 0 || g.N <= 0) return hipSuccess;
    const int bm = rows_per_tile(g.rows, g.groups, g.N, g.K, epi);
    if (bm == 256) return launch_grouped_gemm_i8(g, epi, stream);
    GroupedParams p;
    p.xq = g.xq;
    p.sx = g.sx;
    p.offsets = g.offsets;
    p.source = g.source;
    p.slot_of = g.slot_of;
    p.wq = g.wq;
    p.wq2 = g.wq2;
    p.sw = g.sw;
    p.sw2 = g.sw2;
    p.y = g.y;
    p.part = g.part;
    p.pre = g.pre;
    p.d = g.d;
    p.pre_rows = g.rows;
    p.rows = (int)g.rows;
    p.groups = g.groups;
    p.N = (int)g.N;
    p.K = g.K;
    p.act = g.act;
    const int nf = epi == Epi::Gated ? BN / 2 : BN;
    p.tiles_n = (int)((g.N + nf - 1) / nf);
    const bool vec = g.N % 8 == 0;
    switch (epi) {
    case Epi::Bf16:
        if (vec) launch_rows<Epi::Bf16, true>(p, bm, stream);
        else launch_rows<Epi::Bf16, false>(p, bm, stream);
        break;
    case Epi::Gated:
        if (!vec) return hipErrorInvalidValue;
        launch_rows<Epi::Gated, true>(p, bm, stream);
        break;
    default:
        if (!vec) return hipErrorInvalidValue;
        launch_rows<Epi::Part, true>(p, bm, stream);
    }
    return hipGetLastError();
}

hipError_t launch_moe_combine(const float *part, const int32_t *row_of, const float *weights, const uint16_t *residual,
                              uint16_t *y, int64_t M, int K, int top, hipStream_t stream)
{
    if (M <= 0) return hipSuccess;
    CombineParams p;
    p.part = part;
    p.row_of = row_of;
    p.weights = weights;
    p.residual = residual;
    p.y = y;
    p.units = M * (K / 4);
    p.K = K;
    p.top = top;
    const int64_t blocks = (p.units + 255) / 256;
    if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return hipGetLastError();
}

} // namespace convrot
