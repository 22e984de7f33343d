// grad_i8.hip -- input gradients of the INT8 ConvRot linears, through the frozen weights (gfx950).
//
// Forward: z = (Q(x R) . wq^T) sx sw + b.  With the token quantizer Q taken as the identity (straight
// through) and the weights frozen, a gradient dz of z gives
//   dx[m,k] = sum_k' ( sum_n dz[m,n] sw[n] wq[n,k'] ) R[k',k],     db[n] = sum_m dz[m,n]
// (R symmetric).  Two weights that share the tokens (gate and up) add their products, so they are one
// contraction over their stacked rows.  Three steps:
//   1. grad_prep_kernel: dz from the incoming gradient, the saved pre-activations and the activation's
//      slope; a[m,n] = bf16(dz sw) for the matrix core, fp32 column sums of dz for db.
//   2. grad_gemm_kernel, or grad_tile_kernel for few tokens: a . wq with v_mfma_f32_16x16x32_bf16.  The codes
//      are exact in bf16, so a's rounding (2^-8 of each term at most, what bf16 training rounds its gradients to
//      anyway; dx's error is 1.3 to 1.5 times that of its own rounding alone) is the only one before
//      the fp32 sums.
//   3. the rotation, dx_add and the one rounding to bf16: in the GEMM's epilogue (a tile spans 256
//      channels, whole groups), or in grad_join_kernel where tiles are split along n.
// Grouped: rows sorted by group (expert), each through its own group's weight.  The operand then comes from
// grad_rows_kernel, a tile holds rows of one group, nothing is split, and the result may also go to
// rows that moe_combine_kernel adds up.
#include "activation.hpp"
#include "device_common.hpp"
#include "grouped_common.hpp"
#include "launchers.hpp"
#include "tile_common.hpp"

namespace convrot {
namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i lds_v2i;
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));

constexpr int BM = 256, BC = 256;             // tokens and channels of a tile
constexpr int BN = 64;                        // contraction rows per step
constexpr int MAX_SPLIT = 64;

struct GradParams {
    const uint16_t *a;         // [M, lda] bf16; columns [0, 64 nt1) the first weight's, then the second's
    const int8_t *w1, *w2;     // [N, K]
    const uint16_t *add;       // dx_add [M, K] or null
    uint16_t *dx;              // [M, K]
    float *part;               // split tiles' partial sums: slots of 256 x 256
    int64_t lda;
    int M, N, K, lg;
    int nt1, nt;               // contraction steps of the first weight, in all
    int bm;                    // tokens per tile, 256 or 64
    int tiles_m, tiles_c;
    int T_dp, S;               // whole tiles, then the rest in S slices each
    float norm;                // 2^(-lg / 2)
    GradNext next;             // next.a non-null: the gated product's gradient goes there, not to dx
    // Grouped (M rows in all, w1, w2 [groups, N, K], next's scales [groups, K]; tiles_m, T_dp and S unused):
    const int32_t *offsets;
    const int32_t *slot_of;    // the row of next.pre that a row has, or null: its own
    float *rows;               // non-null: fp32 rows [M, K] instead of dx
    int groups;
};

// What the gated product's gradient reads of a row for 8 channels, and of the group's scales.
struct NextRow {
    v4u g, u;

    __device__ __forceinline__ void fetch(const GradParams &p, int64_t row, int c)
    {
        const int64_t o = row * p.K + c;
        g = *reinterpret_cast<const v4u *>(p.next.pre + o);
        u = *reinterpret_cast<const v4u *>(p.next.pre + (int64_t)p.M * p.K + o);
    }
};
struct NextScales {
    v4f gate[2], up[2];

    __device__ __forceinline__ void fetch(const GradParams &p, int group, int c)
    {
        const int64_t o = (int64_t)group * p.K + c;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                gate[h][e] = p.next.sw_gate[o + 4 * h + e];
                up[h][e] = p.next.sw_up[o + 4 * h + e];
            }
    }
};

// 8 neighbouring channels of dh, to both operands of the next contraction.
__device__ __forceinline__ void next8(const GradParams &p, int m, int c, const float (&v)[8], const NextRow &r,
                                      const NextScales &s)
{
    float g[8], u[8], slope[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        g[e] = e & 1 ? bf16hi_to_f32(r.g[e >> 1]) : bf16lo_to_f32(r.g[e >> 1]);
        u[e] = e & 1 ? bf16hi_to_f32(r.u[e >> 1]) : bf16lo_to_f32(r.u[e >> 1]);
    }
    act_values_slopes(g, slope, p.next.act);
    v4u a, b;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint32_t d = pack_bf16x2(v[e], v[e + 1]);
        const float d0 = bf16lo_to_f32(d), d1 = bf16hi_to_f32(d);
        const int h = e >> 2, i = e & 3;
        a[e >> 1] = pack_bf16x2(d0 * u[e] * slope[e] * s.gate[h][i], d1 * u[e + 1] * slope[e + 1] * s.gate[h][i + 1]);
        b[e >> 1] = pack_bf16x2(d0 * g[e] * s.up[h][i], d1 * g[e + 1] * s.up[h][i + 1]);
    }
    uint16_t *to = p.next.a + (int64_t)m * 2 * p.K + c;
    *reinterpret_cast<v4u *>(to) = a;
    *reinterpret_cast<v4u *>(to + p.K) = b;
}

// 8 rotated channels c .. of token m to where the launch puts them:
//   dx = bf16(v + add), or, for the hidden gradient of a gated block, dh = bf16(v) and on to
//   both operands of the next contraction, bf16(dh u act'(g) sw_gate) and bf16(dh act(g) sw_up), which
//   saves writing dh and reading it back in a pass of its own.
// (16 bytes each; K % 64 == 0, so all 8 exist.)
template <bool GROUPED>
__device__ __forceinline__ void finish8(const GradParams &p, int m, int c, float (&v)[8])
{
    auto load = [](const uint16_t *src, float (&to)[8]) {
        const v4u d = *reinterpret_cast<const v4u *>(src);
#pragma unroll
        for (int e = 0; e < 8; ++e) to[e] = e & 1 ? bf16hi_to_f32(d[e >> 1]) : bf16lo_to_f32(d[e >> 1]);
    };
    auto store = [](uint16_t *dst, const float (&from)[8]) {
        v4u d;
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = pack_bf16x2(from[2 * e], from[2 * e + 1]);
        *reinterpret_cast<v4u *>(dst) = d;
    };
    const int64_t o = (int64_t)m * p.K + c;
    if (GROUPED && p.rows) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<v4f *>(p.rows + o + 4 * h) = v4f{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        return;
    }
    if (!p.next.a) {
        float add[8] = {};
        if (p.add) load(p.add + o, add);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += add[e];
        store(p.dx + o, v);
        return;
    }
    if constexpr (!GROUPED) {                            // (sorted rows' pre is requested ahead, by their kernels)
        NextRow row;
        NextScales scales;
        row.fetch(p, m, c);
        scales.fetch(p, 0, c);
        next8(p, m, c, v, row, scales);
    }
}

// One step of the rotation.  Sums are normalised before the first: |a + b| or |a - b| is at least the larger of |a| and
// |b|, so nothing on the way exceeds the group's largest result and only a result can overflow.
__device__ __forceinline__ void bfly(float &a, float &b)
{
    const float s = a + b;
    b = a - b;
    a = s;
}

// Swap the odd 16-lane rows of a with the even ones of b (v_permlane16_swap).
__device__ __forceinline__ void swap16f(float &a, float &b)
{
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}

// A 16 x 16 block of sums (lane: channels 4 (lane / 16) + v of token lane % 16), normalised and rotated over its 16
// channels: bits 0 and 1 in registers, 2 and 3 across lanes.
__device__ __forceinline__ void rotate16(v4f &x, float norm, int lg)
{
    float x0 = x[0] * norm, x1 = x[1] * norm, x2 = x[2] * norm, x3 = x[3] * norm;
    if (lg > 0) {
        bfly(x0, x1);
        bfly(x2, x3);
    }
    if (lg > 1) {
        bfly(x0, x2);
        bfly(x1, x3);
    }
    if (lg > 2) {
        swap16f(x0, x1);
        bfly(x0, x1);
        swap16f(x0, x1);
        swap16f(x2, x3);
        bfly(x2, x3);
        swap16f(x2, x3);
    }
    if (lg > 3) {
        swap32f(x0, x1);
        bfly(x0, x1);
        swap32f(x0, x1);
        swap32f(x2, x3);
        bfly(x2, x3);
        swap32f(x2, x3);
    }
    x = v4f{x0, x1, x2, x3};
}

// 16 bytes per lane, global -> LDS (lane l to byte lds + 16 l).  Written out because the compiler, which knows the
// builtin to write LDS, waits for every such load in flight before each transposing read: one load latency
// a step.  The kernel's own s_waitcnt and barrier order the two.  It has no output register, and a load the
// compiler issues itself is only waited for longer than it counts.  It writes m0, which the compiler reserves and does
// not let an asm declare, so nothing the compiler emits in these kernels may use m0 (tested on their assembly).
__device__ __forceinline__ void dma16(v4u rsrc, uint32_t lds, uint32_t off, uint32_t soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(rsrc), "s"(soff)
                 : "memory");
}

// The load side of a tile's K loop: the next step to request, its codes' address and the rows left there, all in
// scalar registers.  Rows past N lie past the descriptor's end and read zeros, as everything past the last
// step does.
struct StepLoads {
    int t, rows;
    uint64_t w, x;             // codes of the step, tokens of the tile
    int64_t own;               // where the group's weights begin (0 but for rows sorted by group)

    __device__ __forceinline__ StepLoads(const GradParams &p, int kb, int m0, int c0, int group)
    {
        own = (int64_t)group * p.N * p.K;
        const int first = kb >= p.nt1 ? p.nt1 : 0;
        t = kb;
        rows = p.N - (kb - first) * BN;
        w = reinterpret_cast<uint64_t>((first ? p.w2 : p.w1) + own + (int64_t)(kb - first) * BN * p.K + c0);
        x = reinterpret_cast<uint64_t>(p.a + (int64_t)m0 * p.lda);
    }
    __device__ __forceinline__ v4u codes(int ke, int K, int c0) const
    {
        const int records = t >= ke ? 0 : rows >= BN ? NUM_RECORDS : rows * K - c0;
        return v4u{(uint32_t)w, (uint32_t)(w >> 32) & 0xffffu, (uint32_t)records, 0x00020000u};
    }
    __device__ __forceinline__ v4u tokens(int ke) const
    {
        return v4u{(uint32_t)x, (uint32_t)(x >> 32) & 0xffffu, t < ke ? (uint32_t)NUM_RECORDS : 0u, 0x00020000u};
    }
    __device__ __forceinline__ void advance(const GradParams &p, int c0)
    {
        ++t;
        rows -= BN;
        w += (uint64_t)(BN * p.K);
        if (t == p.nt1) {
            rows = p.N;
            w = reinterpret_cast<uint64_t>(p.w2 + own + c0);
        }
    }
};

// Transposing LDS read: of each 16 lanes, lane 2 r and 2 r + 1 name the two 8-byte halves of row r's 16 bytes,
// and lane c gets byte c of the 8 rows.  (Not a template, like the two below: the host pass drops a kernel
// template whose dependent code uses gfx950-only builtins.)
__device__ __forceinline__ v2i read_transposed(const uint8_t *p)
{
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(const_cast<uint8_t *>(p)));
}

// 8 codes of one channel to bf16, exactly: v_cvt_f32_i32 takes a byte with its sign, and an integer of 8 bits
// leaves the low half of its fp32 empty.  (A byte u = q + 128 placed in a bf16 denormal, u 2^-133, needs one
// permute for two codes and no conversion, but then every sum carries 128 times the sum of the tokens' own
// values, to be taken back at the end.  For gradients of one sign that is most of the sum: a contraction of 51200
// left an error of 3e-4 of dx before its rounding, against 2e-6 with these plain sums.  Of that contraction's time it
// saved 1%.)
__device__ __forceinline__ v8bf16 codes_to_bf16(v2i raw)
{
    v4u d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (uint32_t)raw[i >> 1] >> (16 * (i & 1));
        d[i] = __builtin_amdgcn_perm(__float_as_uint((float)(int8_t)(pair >> 8)), __float_as_uint((float)(int8_t)pair),
                                     0x07060302u);
    }
    return __builtin_bit_cast(v8bf16, d);
}

// 64 rows whose rotation over 64 channels is done, in LDS as rows of 1 KiB with 16-byte chunk c at c ^ row % 16: its last
// two steps and the result, by 32 threads per row, 8 channels each.  For a gradient that goes on to a gated product, the
// first 4 rows' values of pre and the scales are requested before the rotation and each next row's 4 rows ahead (every row's
// own where it is needed: 121 us for an expert layer's 8192 slots, N x K = 2048 x 1408, 108 so).
template <bool GROUPED>
__device__ __forceinline__ void finish_rows(const GradParams &p, const uint8_t *smem, int m0, int end, int c0, int group,
                                            const int *slots, NextRow (&ahead)[4], const NextScales &scales)
{
    const int lg = p.lg, cc = (int)threadIdx.x & 31, c = c0 + 8 * cc, first = (int)threadIdx.x >> 5;
    auto rotated8 = [&](int row, float (&v)[8]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            auto chunk = [&](int i) -> v4f {
                return *reinterpret_cast<const v4f *>(smem + row * 1024 + 16 * (((2 * cc + q) ^ i) ^ (row & 15)));
            };
            v4f x = chunk(0);
            if (lg > 6) x = cc & 8 ? chunk(16) - x : x + chunk(16);
            if (lg > 7) {
                const v4f y = cc & 8 ? chunk(48) - chunk(32) : chunk(32) + chunk(48);
                x = cc & 16 ? y - x : x + y;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
        }
    };
    if constexpr (GROUPED) {
        if (p.next.a) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (m0 + 32 * half >= end) return;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 8 * (4 * half + i) + first, m = m0 + row;
                    if (m < end && c < p.K) {
                        float v[8];
                        rotated8(row, v);
                        next8(p, m, c, v, ahead[i], scales);
                    }
                    if (half == 0) ahead[i].fetch(p, slots[4 + i], c < p.K ? c : 0);
                }
            }
            return;
        }
    }
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
        const int row = 8 * it + first, m = m0 + row;
        if (m >= end || c >= p.K) continue;
        float v[8];
        rotated8(row, v);
        finish8<GROUPED>(p, m, c, v);
    }
}

// 64 tokens x 256 channels, for batches whose 256-token tiles would not fill the GPU or would mostly compute
// padding: 256 threads, 72 KiB of LDS, two workgroups per CU; each of the 4 wavefronts takes 64 channels of all
// 64 tokens.  The codes go to LDS as they are, both operands without passing registers, in three stages
// with two in flight; a transposing read and the conversion above make the fragments.
//   codes   64 rows of 256 bytes as in memory, 16-byte chunk c of row n at c ^ n % 16, so that the rows
//           of a transposing read (16 lanes: 8 rows x 16 bytes) fall on distinct banks;
//   tokens  rows of 128 bytes (64 values), chunk c of row r at c ^ swz(r).
// One barrier a step: it publishes the next stage and frees this one, which is refilled behind it.
// (With the codes converted and transposed in registers, then written to LDS as bf16, us: 300 tokens 5376 x 2688
// 38 against 33, 2688 x 2 * 5376 54 / 46; 512 tokens 5120 x 5120 62 / 52.)  12 tokens 5120 x 8192: 12 us,
// the codes' stream and one load latency, 5120 x 2 * 25600: 54 us, 4.8 TB/s; 300 tokens 5376 x 2688: 20 us, matrix core 13%
// busy, 2688 x 2 * 5376: 28 us, 23%: a step's LDS reads and barrier.
template <bool GROUPED>
__global__ void __launch_bounds__(256, 2) grad_tile_kernel(GradParams p)
{
    constexpr int TM = 64, NST = 3;
    constexpr int WB = BN * BC, TSTAGE = WB + TM * BN * 2;   // codes, then tokens
    constexpr int XL = 2, WL = 4;                        // loads per step and wavefront
    __shared__ __attribute__((aligned(16))) uint8_t smem[NST * TSTAGE];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = p.K;
    int m0, c0, group = 0, end = p.M, kb = 0, ke = p.nt, slot = -1;
    if constexpr (GROUPED) {
        __shared__ GroupTable table;
        int last;
        const int tiles = group_tiles<256>(p.offsets, p.groups, p.M, TM, table, reinterpret_cast<int *>(smem), last);
        const int units = tiles * p.tiles_c;
        if ((int)blockIdx.x >= units) return;            // the grid holds the most units there could be
        int tm, tc;
        tile_coords(unit_of((int)blockIdx.x, 0, units), tiles, p.tiles_c, tm, tc);
        const GroupRows gr = group_of_tile(table, TM, last, tm);
        m0 = gr.first;
        end = gr.end;
        group = gr.group;
        c0 = tc * BC;
    } else {
        const int T = p.tiles_m * p.tiles_c, U = p.T_dp + (T - p.T_dp) * p.S;
        if ((int)blockIdx.x >= U) return;                // the grid is rounded up to a multiple of 8
        const int u = unit_of((int)blockIdx.x, p.T_dp, U);
        int tile = u;
        if (u >= p.T_dp) {
            const int r = T - p.T_dp, v = u - p.T_dp, sl = v / r;
            tile = p.T_dp + v % r;
            kb = (int)((int64_t)sl * p.nt / p.S);
            ke = (int)((int64_t)(sl + 1) * p.nt / p.S);
            slot = v;
        }
        int tm, tc;
        tile_coords(tile, p.tiles_m, p.tiles_c, tm, tc);
        m0 = tm * TM;
        c0 = tc * BC;
    }

    int slots[8];                                        // Grouped: the rows of pre that this thread finishes
    if constexpr (GROUPED) {
        if (p.next.a) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int m = min(m0 + 8 * i + ((int)threadIdx.x >> 5), end - 1);
                slots[i] = p.slot_of ? p.slot_of[m] : m;
            }
        }
    }
    // tokens: instruction i of wave w fills rows 8 (4 i + w) .. + 7 (lane -> row + lane / 8, position lane % 8);
    // codes: rows 4 (4 i + w) .. + 3 (lane -> row + lane / 16, position lane % 16)
    uint32_t offx[XL], offw[WL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = 8 * (4 * i + w) + (lane >> 3);
        offx[i] = m0 + r < end ? (uint32_t)(r * (int)p.lda * 2 + 16 * ((lane & 7) ^ swz(r))) : OOB;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
        const int n = 4 * (4 * i + w) + (lane >> 4), c = 16 * ((lane & 15) ^ (n & 15));
        offw[i] = c0 + c < K ? (uint32_t)(n * K + c) : OOB;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(const lds_void *)smem + (uint32_t)w * 1024u;
    StepLoads ld(p, kb, m0, c0, group);
    uint32_t ld_lds = lds0;
    auto issue = [&]() {
        const v4u rw = ld.codes(ke, K, c0), rx = ld.tokens(ke);
#pragma unroll
        for (int i = 0; i < WL; ++i) dma16(rw, ld_lds + 4096 * i, offw[i], 0);
#pragma unroll
        for (int i = 0; i < XL; ++i) dma16(rx, ld_lds + WB + 4096 * i, offx[i], (uint32_t)ld.t * (BN * 2));
        ld.advance(p, c0);
        ld_lds = ld_lds == lds0 + (NST - 1) * TSTAGE ? lds0 : ld_lds + TSTAGE;
    };

    // codes: rows 32 kk + 8 fq + i / 2 for lane (fq, i), half i % 2 of chunk 4 w + b
    const int frow = lane & 15, fq = lane >> 4;
    const int key = 8 * (fq & 1) + (frow >> 1);
    int awhere[4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
        awhere[b] = (8 * fq + (frow >> 1)) * BC + 16 * ((4 * w + b) ^ key) + 8 * (frow & 1);
    const int bwhere = WB + frow * 128;
    const int bpos[2] = {16 * (fq ^ swz(frow)), 16 * ((4 + fq) ^ swz(frow))};
    v2i raw[2][4];
    v8bf16 fb[2][4];
    auto read_codes = [&](int stage, int kk) {
        const uint8_t *st = smem + stage * TSTAGE + kk * (32 * BC);
#pragma unroll
        for (int b = 0; b < 4; ++b) raw[kk][b] = read_transposed(st + awhere[b]);
    };
    auto read_tokens = [&](int stage, int kk) {
        const uint8_t *st = smem + stage * TSTAGE + bwhere + bpos[kk];
#pragma unroll
        for (int b = 0; b < 4; ++b) fb[kk][b] = *reinterpret_cast<const v8bf16 *>(st + b * 2048);
    };
    v4f acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = v4f{};
    auto mfma_range = [&](int kk, int a0, int a1) {
#pragma unroll
        for (int a = a0; a < a1; ++a) {
            const v8bf16 fa = codes_to_bf16(raw[kk][a]);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb[kk][b], acc[a][b], 0, 0, 0);
        }
    };
    auto fence = [] { __builtin_amdgcn_sched_barrier(0); };

    issue();
    issue();
    issue();
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * (XL + WL)));
    asm volatile("s_barrier" ::: "memory");
    read_codes(0, 0);
    read_tokens(0, 0);
    int st = 0;                                          // this step's stage
    for (int t = kb; t < ke; ++t) {
        const int next = st == NST - 1 ? 0 : st + 1;
        read_codes(st, 1);
        read_tokens(st, 1);
        mfma_range(0, 0, 4);
        fence();
        mfma_range(1, 0, 1);
        fence();
        // the next step has landed: only the one after it is still in flight
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(XL + WL));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        issue();
        read_codes(next, 0);
        read_tokens(next, 0);
        mfma_range(1, 1, 4);
        fence();
        st = next;
    }
    // every load into LDS has landed and every wave is done reading before the epilogue reuses it
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    NextRow ahead[4];
    NextScales scales;
    if constexpr (GROUPED) {
        if (p.next.a) {
            const int cn = c0 + 8 * ((int)threadIdx.x & 31), cl = cn < K ? cn : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) ahead[i].fetch(p, slots[i], cl);
            scales.fetch(p, group, cl);
        }
    }

    // lane: token lane % 16 of block b, channels 16 (4 w + a) + 4 fq + v
    if (!GROUPED && slot >= 0) {
        float *dst = p.part + (int64_t)slot * (TM * BC);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int ml = 16 * b + frow;
            if (m0 + ml < end) {
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    *reinterpret_cast<v4f *>(dst + ml * BC + 16 * (4 * w + a) + 4 * fq) = acc[a][b];
            }
        }
        return;
    }
    // the rotation: channel bits 0, 1 in v, 2, 3 across lanes, 4, 5 in a; 6 and 7 across the
    // four waves
    const int lg = p.lg;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
        for (int a = 0; a < 4; ++a) rotate16(acc[a][b], p.norm, lg);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (lg > 4 + s) {
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    if (!(a & (1 << s))) {
                        const v4f x = acc[a][b], y = acc[a | (1 << s)][b];
                        acc[a][b] = x + y;
                        acc[a | (1 << s)][b] = x - y;
                    }
            }
        }
    }
    // through LDS, rows of 1 KiB with 16-byte chunk c at c ^ row % 16; then 32 threads per token, 8 channels each
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int a = 0; a < 4; ++a)
            *reinterpret_cast<v4f *>(smem + (16 * b + frow) * 1024 + 16 * ((4 * (4 * w + a) + fq) ^ frow)) = acc[a][b];
    __syncthreads();
    finish_rows<GROUPED>(p, smem, m0, end, c0, group, slots, ahead, scales);
}

// The same for 256 tokens x 256 channels, when there are enough of them: 512 threads, one workgroup per CU, 144 KiB of
// LDS in three stages of the same layout.  Each of the 8 wavefronts takes 32 channels of all 256 tokens, so that
// every code is converted once and by one wavefront; the tokens' fragments, which all eight read, come in
// four groups of 8 a step (two halves of the contraction, 128 tokens each), one ahead of the products.  The barrier
// stands before the last group: it publishes the next step, whose first group is read under those products, and
// frees this one, whose last group is in registers by then.  The loads of step t + 2 go out one by one, after
// each half of three groups' products.
// 4096 tokens 5376 x 16128: 553 us, 1280 TFLOP/s, matrix core 62% busy at 1.97 GHz, LDS nearly conflict-free (a library's
// bf16 product of that shape, operands ready in bf16: 887); without the loads (timing only) 14% less.
// Alternatives, us for that call and for the gated block's at 2048 tokens 5120 x 25600 (593, 1311 as it was, on a faster
// card and with the codes as denormals):
// codes converted and transposed in registers and written to LDS as bf16 625, 1392; wavefronts of 64 channels x
// 128 tokens, which read half as much LDS and convert twice as much, 602, 1335; the loads after
// the first and third quarter of a group 603, 1337, or two at once at its end 600, 1321; their descriptors kept
// ready instead of formed at each load 617, 1368.
// The K loop holds everything in registers; the epilogue spills 26 of them (104 bytes a lane), once a tile.
template <bool GROUPED>
__global__ void __launch_bounds__(512, 1) grad_gemm_kernel(GradParams p)
{
    constexpr int NST = 3, XL = 4, WL = 2, LPS = XL + WL;    // loads per step and wavefront
    constexpr int WB = BN * BC, GSTAGE = WB + BM * BN * 2;   // codes, then tokens
    __shared__ __attribute__((aligned(16))) uint8_t smem[NST * GSTAGE];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = p.K;
    int m0, c0, group = 0, end = p.M, kb = 0, ke = p.nt, slot = -1;
    if constexpr (GROUPED) {
        __shared__ GroupTable table;
        int last;
        const int tiles = group_tiles<512>(p.offsets, p.groups, p.M, BM, table, reinterpret_cast<int *>(smem), last);
        const int units = tiles * p.tiles_c;
        if ((int)blockIdx.x >= units) return;            // the grid holds the most units there could be
        int tm, tc;
        tile_coords(unit_of((int)blockIdx.x, 0, units), tiles, p.tiles_c, tm, tc);
        const GroupRows gr = group_of_tile(table, BM, last, tm);
        m0 = gr.first;
        end = gr.end;
        group = gr.group;
        c0 = tc * BC;
    } else {
        const int T = p.tiles_m * p.tiles_c, U = p.T_dp + (T - p.T_dp) * p.S;
        if ((int)blockIdx.x >= U) return;                // the grid is rounded up to a multiple of 8
        const int u = unit_of((int)blockIdx.x, p.T_dp, U);
        int tile = u;
        if (u >= p.T_dp) {
            const int r = T - p.T_dp, v = u - p.T_dp, sl = v / r;
            tile = p.T_dp + v % r;
            kb = (int)((int64_t)sl * p.nt / p.S);
            ke = (int)((int64_t)(sl + 1) * p.nt / p.S);
            slot = v;
        }
        int tm, tc;
        tile_coords(tile, p.tiles_m, p.tiles_c, tm, tc);
        m0 = tm * BM;
        c0 = tc * BC;
    }

    // tokens: instruction i of wave w fills rows 8 (8 i + w) .. + 7; codes: rows 4 (8 i + w) .. + 3
    uint32_t offx[XL], offw[WL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = 8 * (8 * i + w) + (lane >> 3);
        offx[i] = m0 + r < end ? (uint32_t)(r * (int)p.lda * 2 + 16 * ((lane & 7) ^ swz(r))) : OOB;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
        const int n = 4 * (8 * i + w) + (lane >> 4), c = 16 * ((lane & 15) ^ (n & 15));
        offw[i] = c0 + c < K ? (uint32_t)(n * K + c) : OOB;
    }
    // load i of a step: its codes first
    const uint32_t lds0 = (uint32_t)(uintptr_t)(const lds_void *)smem + (uint32_t)w * 1024u;
    StepLoads ld(p, kb, m0, c0, group);
    uint32_t ld_lds = lds0;
    auto issue = [&](int i) {
        if (i < WL) dma16(ld.codes(ke, K, c0), ld_lds + 8192 * i, offw[i], 0);
        else dma16(ld.tokens(ke), ld_lds + WB + 8192 * (i - WL), offx[i - WL], (uint32_t)ld.t * (BN * 2));
        if (i < LPS - 1) return;
        ld.advance(p, c0);
        ld_lds = ld_lds == lds0 + (NST - 1) * GSTAGE ? lds0 : ld_lds + GSTAGE;
    };

    const int frow = lane & 15, fq = lane >> 4;
    const int key = 8 * (fq & 1) + (frow >> 1);
    int awhere[2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
        awhere[a] = (8 * fq + (frow >> 1)) * BC + 16 * ((2 * w + a) ^ key) + 8 * (frow & 1);
    const int bwhere = WB + frow * 128;
    const int bpos[2] = {16 * (fq ^ swz(frow)), 16 * ((4 + fq) ^ swz(frow))};
    v2i raw[2];
    v8bf16 fb[2][8];
    auto read_codes = [&](int stage, int kk) {
        const uint8_t *st = smem + stage * GSTAGE + kk * (32 * BC);
#pragma unroll
        for (int a = 0; a < 2; ++a) raw[a] = read_transposed(st + awhere[a]);
    };
    // group h of a step's half kk: tokens 128 h .. + 127
    auto read_tokens = [&](int stage, int kk, int h) {
        const uint8_t *st = smem + stage * GSTAGE + bwhere + bpos[kk] + h * 16384;
#pragma unroll
        for (int b = 0; b < 8; ++b) fb[h][b] = *reinterpret_cast<const v8bf16 *>(st + b * 2048);
    };
    v4f acc[2][16];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 16; ++b) acc[a][b] = v4f{};
    auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
    // the products of group h; loads i0, i0 + 1 after its first and second half (i0 < 0: none)
    auto products = [&](const v8bf16 (&fa)[2], int h, int i0) {
#pragma unroll
        for (int b = 0; b < 8; ++b) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
                acc[a][8 * h + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[a], fb[h][b], acc[a][8 * h + b], 0, 0, 0);
            if (i0 >= 0 && (b == 3 || b == 7)) {
                fence();
                issue(i0 + (b >> 2));
                fence();
            }
        }
    };

#pragma unroll
    for (int i = 0; i < 2 * LPS + 2; ++i) issue(i % LPS);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(LPS + 2));
    asm volatile("s_barrier" ::: "memory");
    read_codes(0, 0);
    read_tokens(0, 0, 0);
    int st = 0;                                          // this step's stage
    for (int t = kb; t < ke; ++t) {
        const int next = st == NST - 1 ? 0 : st + 1;
        v8bf16 fa[2];
        read_tokens(st, 0, 1);
        fence();
#pragma unroll
        for (int a = 0; a < 2; ++a) fa[a] = codes_to_bf16(raw[a]);
        products(fa, 0, 2);
        fence();
        read_codes(st, 1);
        read_tokens(st, 1, 0);
        fence();
        products(fa, 1, 4);
        fence();
        read_tokens(st, 1, 1);
        fence();
#pragma unroll
        for (int a = 0; a < 2; ++a) fa[a] = codes_to_bf16(raw[a]);
        products(fa, 0, -1);
        fence();
        // the next step has landed: only the one after it is still in flight
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(LPS));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        read_codes(next, 0);
        read_tokens(next, 0, 0);
        fence();
        products(fa, 1, 0);
        fence();
        st = next;
    }
    // every load into LDS has landed and every wave is done reading before the epilogue reuses it
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();

    // lane: token lane % 16 of block b, channels 32 w + 16 a + 4 fq + v
    if (!GROUPED && slot >= 0) {
        float *dst = p.part + (int64_t)slot * (BM * BC);
#pragma unroll
        for (int b = 0; b < 16; ++b) {
            const int ml = 16 * b + frow;
            if (m0 + ml < end) {
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    *reinterpret_cast<v4f *>(dst + ml * BC + 32 * w + 16 * a + 4 * fq) = acc[a][b];
            }
        }
        return;
    }
    // the rotation: channel bits 0, 1 in v, 2, 3 across lanes, 4 in a; 5 .. 7 across the eight waves, through LDS
    const int lg = p.lg;
#pragma unroll
    for (int b = 0; b < 16; ++b) {
#pragma unroll
        for (int a = 0; a < 2; ++a) rotate16(acc[a][b], p.norm, lg);
        if (lg > 4) {
            const v4f x = acc[0][b], y = acc[1][b];
            acc[0][b] = x + y;
            acc[1][b] = x - y;
        }
    }
    // 128 tokens a round, rows of 1 KiB with 16-byte chunk c at c ^ row % 16; then 32 threads per token, 8 channels each
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 8; ++b)
#pragma unroll
            for (int a = 0; a < 2; ++a)
                *reinterpret_cast<v4f *>(smem + (16 * b + frow) * 1024 + 16 * ((8 * w + 4 * a + fq) ^ frow)) =
                    acc[a][8 * pass + b];
        __syncthreads();
        if (lg > 5) {
            // thread: one row, 4 channels at 8 places 32 channels apart, twice
            const int row = (int)threadIdx.x & 127;
#pragma unroll 1
            for (int j = (int)threadIdx.x >> 7; j < 8; j += 4) {
                v4f x[8];
#pragma unroll
                for (int h = 0; h < 8; ++h) x[h] = *reinterpret_cast<const v4f *>(smem + row * 1024 + 16 * ((8 * h + j) ^ (row & 15)));
#pragma unroll
                for (int s = 0; s < 3; ++s) {
                    if (lg > 5 + s) {
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            if (!(h & (1 << s))) {
                                const v4f a = x[h], b = x[h | (1 << s)];
                                x[h] = a + b;
                                x[h | (1 << s)] = a - b;
                            }
                    }
                }
#pragma unroll
                for (int h = 0; h < 8; ++h) *reinterpret_cast<v4f *>(smem + row * 1024 + 16 * ((8 * h + j) ^ (row & 15))) = x[h];
            }
            __syncthreads();
        }
        const int cc = (int)threadIdx.x & 31, c = c0 + 8 * cc, first = (int)threadIdx.x >> 5;
        auto rotated8 = [&](int row, float (&v)[8]) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const v4f x = *reinterpret_cast<const v4f *>(smem + row * 1024 + 16 * ((2 * cc + q) ^ (row & 15)));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
            }
        };
        if constexpr (GROUPED) {
            if (p.next.a) {
                // pre of the next row on its way
                const int cl = c < K ? c : 0;
                auto slot_at = [&](int it) {
                    const int m = min(m0 + 128 * pass + 16 * it + first, end - 1);
                    return p.slot_of ? p.slot_of[m] : m;
                };
                NextScales scales;
                NextRow ahead;
                scales.fetch(p, group, cl);
                ahead.fetch(p, slot_at(0), cl);
                int then = slot_at(1);
#pragma unroll 1
                for (int it = 0; it < 8; ++it) {
                    const int row = 16 * it + first, m = m0 + 128 * pass + row;
                    if (m - first >= end) break;
                    const NextRow now = ahead;
                    ahead.fetch(p, then, cl);
                    then = slot_at(it + 2);
                    if (m >= end || c >= K) continue;
                    float v[8];
                    rotated8(row, v);
                    next8(p, m, c, v, now, scales);
                }
                continue;
            }
        }
#pragma unroll 1
        for (int it = 0; it < 8; ++it) {
            const int row = 16 * it + first, m = m0 + 128 * pass + row;
            if (m >= end || c >= K) continue;
            float v[8];
            rotated8(row, v);
            finish8<GROUPED>(p, m, c, v);
        }
    }
}

// Split tiles: the S partial sums of a token's 256 channels, added in slice order (the same order at
// every call), then the rotation, dx_add and the rounding.  32 lanes per token, 8 channels each:
// channel bits 0 .. 2 in registers, 3 .. 7 across lanes.  Bound by the partial sums' read: 14 us for 4096 x 5376's
// last round, 5 to 8 us (about two memory latencies) for a few hundred tokens.
__global__ void __launch_bounds__(256) grad_join_kernel(GradParams p, int rb)
{
    constexpr int AHEAD = 8;                             // slices in flight (a remainder read one by one: 30 slices 9.1 us, 8.4 so)
    const int i = (int)blockIdx.x / rb;                                 // split tile
    const int ml = ((int)blockIdx.x % rb) * 8 + ((int)threadIdx.x >> 5);
    const int l = (int)threadIdx.x & 31;
    int tm, tc;
    tile_coords(p.T_dp + i, p.tiles_m, p.tiles_c, tm, tc);
    const int m = tm * p.bm + ml, slot = p.bm * BC;
    const int c = tc * BC + 8 * l;
    const bool row_ok = ml < p.bm && m < p.M;
    const int r = p.tiles_m * p.tiles_c - p.T_dp;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (row_ok) {
        const float *src = p.part + (int64_t)i * slot + ml * BC + 8 * l;
#pragma unroll 1
        for (int s = 0; s < p.S; s += AHEAD) {
            v4f a[AHEAD], b[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                a[i] = b[i] = v4f{};
                if (s + i < p.S) {
                    a[i] = *reinterpret_cast<const v4f *>(src);
                    b[i] = *reinterpret_cast<const v4f *>(src + 4);
                    src += (int64_t)r * slot;
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] += a[i][e];
                    v[e + 4] += b[i][e];
                }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= p.norm;
#pragma unroll
    for (int b = 0; b < 3; ++b)
        if (p.lg > b) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!(e & (1 << b))) bfly(v[e], v[e | (1 << b)]);
        }
#pragma unroll
    for (int b = 0; b < 5; ++b)
        if (p.lg > 3 + b) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl_xor(v[e], 1 << b);
                v[e] = (l >> b) & 1 ? o - v[e] : v[e] + o;
            }
        }
    if (row_ok && c < p.K) finish8<false>(p, m, c, v);
}

struct PrepParams {
    const uint16_t *dy;        // [M, N]
    const uint16_t *pre;       // [M, N], or [2, M, N] (gate, up), or null (no activation)
    const float *sw1, *sw2;    // [N]
    uint16_t *a;               // [M, lda], columns Np on the second weight's
    float *sums;               // [chunks][N (2 N)] partial column sums, or null
    float *db1, *db2;          // with one chunk and no sums: the column sums themselves (each may be null)
    int64_t M, N, Np, lda;
    int act, col_blocks, rows; // rows per chunk
};

// A workgroup takes 256 columns and a chunk of rows: 32 lanes of 8 columns, 8 rows at a time.
// Columns from N to Np are zeros.  Bound by memory: 4096 x 16128 with an activation 76 us (396 MB, 5.2 TB/s).
template <bool GATED>
__global__ void __launch_bounds__(256) grad_prep_kernel(PrepParams p)
{
    __shared__ float red[GATED ? 2 : 1][8][256];
    const int cb = (int)blockIdx.x % p.col_blocks, chunk = (int)blockIdx.x / p.col_blocks;
    const int tr = (int)threadIdx.x >> 5, tl = (int)threadIdx.x & 31;
    const int64_t n = (int64_t)cb * 256 + 8 * tl;
    const int64_t r0 = (int64_t)chunk * p.rows, r1 = r0 + p.rows < p.M ? r0 + p.rows : p.M;
    float s1[8], s2[8], sum1[8], sum2[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s1[e] = n + e < p.N ? p.sw1[n + e] : 0.0f;
        s2[e] = GATED && n + e < p.N ? p.sw2[n + e] : 0.0f;
        sum1[e] = sum2[e] = 0.0f;
    }
    // 16 bytes at any element: rows of an odd N start at odd ones, which a vector load takes.  (2001 x 14366: 49 us,
    // element by element 101; 14368 columns 46.)
    const bool whole = n + 8 <= p.N;
    auto load8 = [&](const uint16_t *base, int64_t m, float (&v)[8]) {
        typedef v4u unaligned __attribute__((aligned(2)));
        const uint16_t *src = base + m * p.N + n;
        if (whole) {
            const v4u d = *reinterpret_cast<const unaligned *>(src);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = bf16lo_to_f32(d[e]);
                v[2 * e + 1] = bf16hi_to_f32(d[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = n + e < p.N ? bf16lo_to_f32(src[e]) : 0.0f;
        }
    };
    auto store8 = [&](int64_t m, int64_t col, const float (&v)[8], const float (&s)[8]) {
        *reinterpret_cast<v4u *>(p.a + m * p.lda + col) =
            v4u{pack_bf16x2(v[0] * s[0], v[1] * s[1]), pack_bf16x2(v[2] * s[2], v[3] * s[3]),
                pack_bf16x2(v[4] * s[4], v[5] * s[5]), pack_bf16x2(v[6] * s[6], v[7] * s[7])};
    };
    for (int64_t m = r0 + tr; m < r1; m += 8) {
        float d[8];
        load8(p.dy, m, d);
        if constexpr (GATED) {
            float g[8], u[8];
            load8(p.pre, m, g);
            load8(p.pre + p.M * p.N, m, u);
            float du[8], slope[8];
            act_values_slopes(g, slope, p.act);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                du[e] = d[e] * g[e];
                d[e] = d[e] * u[e] * slope[e];
                sum2[e] += du[e];
            }
            if (n < p.Np) store8(m, p.Np + n, du, s2);
        } else if (p.pre) {
            float z[8], slope[8];
            load8(p.pre, m, z);
            act_values_slopes(z, slope, p.act);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] *= slope[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum1[e] += d[e];
        if (n < p.Np) store8(m, n, d, s1);
    }
    if (!p.sums && !p.db1 && !p.db2) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        red[0][tr][8 * tl + e] = sum1[e];
        if constexpr (GATED) red[1][tr][8 * tl + e] = sum2[e];
    }
    __syncthreads();
    const int64_t col = (int64_t)cb * 256 + threadIdx.x;
    if (col >= p.N) return;
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += red[q][r][threadIdx.x];
        if (p.sums) p.sums[((int64_t)chunk * (GATED ? 2 : 1) + q) * p.N + col] = s;
        else if (float *db = q ? p.db2 : p.db1) db[col] = s;
    }
}

// db[n] = sum of the chunks' partial sums, in chunk order (0 chunks: 0); the second weight's in the grid's second row.
__global__ void __launch_bounds__(256) grad_bias_kernel(const float *sums, int chunks, int parts, int64_t N, float *db1,
                                                        float *db2)
{
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    float *db = blockIdx.y ? db2 : db1;
    if (n >= N || !db) return;
    float s = 0.0f;
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) s += sums[((int64_t)c * parts + blockIdx.y) * N + n];
    db[n] = s;
}

// The operand of a grouped contraction: a[row] = bf16(share dy[source] sw[group]) and, for the slots of a
// mixture-of-experts layer, the gradient of their weights, dweight = sum_n dy[source, n] d[slot, n] in fp32.
// A workgroup takes one row.  MoE (experts non-null): workgroup = slot, its group the slot's expert, its source the
// slot's token, its row where the sort put it; slots without an expert get dweight 0 and no row.  Otherwise the
// workgroup's row itself, and the group whose offsets hold it.  Columns from N to lda are zeros.  Bound by memory: 8192
// slots of 2048 tokens, 2048 channels, with dweights 24 us; 4097 rows of 5376 20 us, 4.4 TB/s.
struct RowsParams {
    const uint16_t *dy;        // [., N]
    const float *sw;           // [groups, N]
    const int32_t *offsets;
    const int32_t *experts, *row_of;   // [slots]
    const float *weights;      // [slots]
    const uint16_t *d;         // bf16 [slots, N] or null
    float *dweights;           // [slots] or null
    uint16_t *a;               // [rows, lda]
    int64_t lda;
    int rows, groups, N, top;
};

__global__ void __launch_bounds__(256) grad_rows_kernel(RowsParams p)
{
    __shared__ float red[4];
    typedef v4u unaligned __attribute__((aligned(2)));
    typedef v4f v4f_any __attribute__((aligned(4)));
    const int s = grid_workgroup(), t = (int)threadIdx.x;
    if (s >= p.rows) return;
    int64_t row = s, source = s;
    int group = -1;
    float share = 1.0f;
    if (p.experts) {
        row = p.row_of[s];
        if (row < 0) {
            if (p.dweights && t == 0) p.dweights[s] = 0.0f;
            return;
        }
        group = p.experts[s];
        source = s / p.top;
        share = p.weights[s];
    } else {
        // the group before the first offset past the row
        group = -2;
        for (int b = 0; b <= p.groups && group == -2; b += 64) {
            const int e = b + (t & 63);
            const uint64_t past = __builtin_amdgcn_ballot_w64(e <= p.groups && p.offsets[min(e, p.groups)] > s);
            if (past) group = b + __builtin_ctzll(past) - 1;
        }
        if (group < 0) return;                           // a row of no group
    }
    const uint16_t *dy = p.dy + source * p.N, *d = p.d ? p.d + (int64_t)s * p.N : nullptr;
    const float *sw = p.sw + (int64_t)group * p.N;
    uint16_t *a = p.a + row * p.lda;
    float sum = 0.0f;
    for (int n = 8 * t; n < p.lda; n += 8 * 256) {
        float v[8], e[8];
        auto load8 = [&](const uint16_t *src, float (&to)[8]) {
            if (n + 8 <= p.N) {
                const v4u x = *reinterpret_cast<const unaligned *>(src + n);
#pragma unroll
                for (int i = 0; i < 8; ++i) to[i] = i & 1 ? bf16hi_to_f32(x[i >> 1]) : bf16lo_to_f32(x[i >> 1]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) to[i] = n + i < p.N ? bf16lo_to_f32(src[n + i]) : 0.0f;
            }
        };
        load8(dy, v);
        if (d) {
            load8(d, e);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[i], e[i], sum);
        }
        if (n + 8 <= p.N) {
            const v4f lo = *reinterpret_cast<const v4f_any *>(sw + n), hi = *reinterpret_cast<const v4f_any *>(sw + n + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * share * (i < 4 ? lo[i & 3] : hi[i & 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = n + i < p.N ? v[i] * share * sw[n + i] : 0.0f;
        }
        *reinterpret_cast<v4u *>(a + n) =
            v4u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
    if (!p.dweights || !d) return;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) sum += __shfl_xor(sum, k);
    if ((t & 63) == 0) red[t >> 6] = sum;
    __syncthreads();
    if (t == 0) p.dweights[s] = (red[0] + red[1]) + (red[2] + red[3]);
}

int cu_count()
{
    static int cus = [] {
        int dev = 0, n = 0;
        if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            n = 256;
        return n >= 8 ? n : 256;
    }();
    return cus;
}

struct Plan {
    int64_t Np, lda;
    int nt1, nt, bm, tiles_m, tiles_c, T_dp, S;
    int chunks;                // of partial column sums
    size_t a_bytes, sum_bytes, part_bytes;
};

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// Tokens per tile and slices of the contraction, by a model with measured constants.  Whole rounds of tiles run
// whole; the rest of the last round may be split so that it fills the GPU.  A step takes 1.6 us of a CU in
// 256-token tiles; in 64-token ones 0.72 us alone and 0.54 us when workgroups share the CU.  The codes stream at
// 4.9 TB/s.  Slices cost their partial sums' round trip (8 bytes per element at 4.5 TB/s) and a launch.
// Measured (us; K x N, 2 N for gate|up, all launches of the call), 256 tokens unsliced / in the best slices / 64
// tokens unsliced / in the best slices:
//   600 tokens 2048 x 8192: 185 / 50 / 93 / 47;    512 tokens 5120 x 5120: 127 / 54 / 71 / 55
//   1024 tokens 5120 x 5120: 128 / 75 / 99 / 89;   2688 x 2 * 5376: 246 / 93 / 130 / 107
void tile_plan(Plan &pl, int64_t M, int64_t N, int K, bool gated)
{
    const int cus = cu_count() & ~7;
    const double stream = (double)N * K * (gated ? 2.0 : 1.0) / 4.9e12;
    double best = 1e30;
    for (int bm = 64; bm <= BM; bm *= 4) {
        const int64_t tiles = (M + bm - 1) / bm * pl.tiles_c;
        if (tiles >= (int64_t)1 << 24) continue;
        // 64 tokens: two workgroups per CU
        const int T = (int)tiles, cap = cus * (bm == 64 ? 2 : 1), r = T % cap;
        const double lone = bm == 64 ? 0.72e-6 : 1.6e-6, shared = bm == 64 ? 0.54e-6 : 1.6e-6;
        for (int S = 1; S <= (r ? MAX_SPLIT : 1); ++S) {
            if (S > 1 && pl.nt / S < 2) break;
            const double per_cu = (double)(((int64_t)r * S + cus - 1) / cus) * shared;
            const double math = (double)(T / cap) * (cap / cus) * pl.nt * shared +
                                (r ? (double)((pl.nt + S - 1) / S) * (per_cu > lone ? per_cu : lone) : 0.0);
            const double rows = (double)(M < bm ? M : bm);
            const double t = (math > stream ? math : stream) + (S > 1 ? (double)r * S * rows * BC * 8.0 / 4.5e12 + 2e-6 : 0.0);
            if (t < best) {
                best = t;
                pl.bm = bm;
                pl.tiles_m = (int)((M + bm - 1) / bm);
                pl.T_dp = S > 1 ? T - r : T;
                pl.S = S;
            }
        }
    }
}

// Rows of a grad_prep workgroup: all up to 16 tokens, so that the column sums need no second launch (15 x 7497: 5.4 us
// against 4.4 and 2.3); 8, one per thread, up to 512, and a multiple of 8 that gives at most about 64 chunks
// beyond (2048 x 5120: 10 us, against 22 with 8 rows; and few partial column sums to add up).
int prep_rows(int64_t M) { return M > 512 ? (int)((M + 511) / 512 * 8) : M > 16 ? 8 : 16; }

Plan make_plan(int64_t M, int64_t N, int K, bool gated)
{
    Plan pl;
    pl.Np = (N + BN - 1) / BN * BN;
    pl.lda = gated ? 2 * pl.Np : pl.Np;
    pl.nt1 = (int)(pl.Np / BN);
    pl.nt = (int)(pl.lda / BN);
    pl.tiles_c = (K + BC - 1) / BC;
    tile_plan(pl, M, N, K, gated);
    const int rows = prep_rows(M);
    pl.chunks = (int)((M + rows - 1) / rows);
    pl.a_bytes = round256((size_t)M * (size_t)pl.lda * 2);
    pl.sum_bytes = round256((size_t)pl.chunks * (size_t)N * (gated ? 8 : 4));
    pl.part_bytes = pl.S > 1 ? (size_t)(pl.tiles_m * pl.tiles_c - pl.T_dp) * pl.S * pl.bm * BC * 4 : 0;
    return pl;
}

} // namespace

size_t grad_workspace_bytes(int64_t M, int64_t N, int K, bool gated, bool a_given)
{
    if (M <= 0 || N <= 0) return 0;
    const Plan pl = make_plan(M, N, K, gated);
    return (a_given ? 0 : pl.a_bytes + pl.sum_bytes) + pl.part_bytes;
}

hipError_t launch_grad_i8(const GradArgs &g, bool gated, hipStream_t stream)
{
    if (g.N <= 0) return hipSuccess;
    const Plan pl = make_plan(g.M, g.N, g.K, gated);
    uint8_t *ws = static_cast<uint8_t *>(g.ws);
    const size_t part_at = g.a ? 0 : pl.a_bytes + pl.sum_bytes;
    if (!g.a) {
        float *sums = reinterpret_cast<float *>(ws + pl.a_bytes);
        const bool bias = g.db1 || g.db2;
        if (g.M > 0) {
            PrepParams q;
            q.dy = g.dy;
            q.pre = g.pre;
            q.sw1 = g.sw1;
            q.sw2 = g.sw2;
            q.a = reinterpret_cast<uint16_t *>(ws);
            q.sums = bias && pl.chunks > 1 ? sums : nullptr;
            q.db1 = pl.chunks > 1 ? nullptr : g.db1;
            q.db2 = pl.chunks > 1 ? nullptr : g.db2;
            q.M = g.M;
            q.N = g.N;
            q.Np = pl.Np;
            q.lda = pl.lda;
            q.act = g.act;
            q.col_blocks = (int)((pl.Np + 255) / 256);
            q.rows = prep_rows(g.M);
            const int64_t blocks = (g.M + q.rows - 1) / q.rows * q.col_blocks;
            if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
            const dim3 grid((unsigned)blocks);
            if (gated) hipLaunchKernelGGL(grad_prep_kernel<true>, grid, dim3(256), 0, stream, q);
            else hipLaunchKernelGGL(grad_prep_kernel<false>, grid, dim3(256), 0, stream, q);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (bias && (g.M <= 0 || pl.chunks > 1)) {
            hipLaunchKernelGGL(grad_bias_kernel, dim3((unsigned)((g.N + 255) / 256), g.db2 ? 2 : 1), dim3(256), 0, stream, sums,
                               g.M > 0 ? pl.chunks : 0, gated ? 2 : 1, g.N, g.db1, g.db2);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    if (g.M <= 0) return hipSuccess;
    GradParams p = {};
    p.a = g.a ? g.a : reinterpret_cast<const uint16_t *>(ws);
    p.w1 = g.wq1;
    p.w2 = gated ? g.wq2 : g.wq1;
    p.add = g.add;
    p.dx = g.dx;
    p.part = reinterpret_cast<float *>(ws + part_at);
    p.lda = pl.lda;
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.K = g.K;
    p.lg = g.log2g;
    p.nt1 = pl.nt1;
    p.nt = pl.nt;
    p.bm = pl.bm;
    p.tiles_m = pl.tiles_m;
    p.tiles_c = pl.tiles_c;
    p.T_dp = pl.T_dp;
    p.S = pl.S;
    p.next = g.next;
    p.norm = (float)(1.0 / __builtin_sqrt((double)(1 << g.log2g)));
    const int T = pl.tiles_m * pl.tiles_c, U = pl.T_dp + (T - pl.T_dp) * pl.S;
    const dim3 grid((unsigned)((U + 7) & ~7));
    if (pl.bm == 64) hipLaunchKernelGGL(grad_tile_kernel<false>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(grad_gemm_kernel<false>, grid, dim3(512), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || pl.S == 1) return e;
    const int rb = (int)((g.M < pl.bm ? g.M : pl.bm) + 7) / 8;
    hipLaunchKernelGGL(grad_join_kernel, dim3((unsigned)(T - pl.T_dp) * (unsigned)rb), dim3(256), 0, stream, p, rb);
    return hipGetLastError();
}

// Rows per tile, 64 or 256, by a model with measured constants (us): a CU takes `step` per contraction step and `end` per
// unit; a group's last tile is half empty, and so is the last round unless the tiles are surely no more than the CUs.
// Measured, whole calls, 64 / 256 rows:
//   linear_grouped_backward, rows, groups, N x K:  1000, 4, 2048 x 2688: 36 / 66;   3000, 12, 2048 x 2048: 52 / 67
//     2000, 8, 2688 x 5376: 92 / 83;   4097, 8, 5376 x 2688: 169 / 153;   8000, 8, 2688 x 2688: 163 / 162
//   expert layer, tokens, top of E, K x F:  2048, 4 of 32, 2048 x 1408: 282 / 343;   4096, 2 of 16, 2688 x 2688: 526 / 505 (the
//     model takes 64 there)
int grouped_rows_per_tile(int64_t rows, int groups, int tiles_c, int nt)
{
    const double used = (double)(groups < rows ? groups : rows);
    double t[2];
    for (int i = 0; i < 2; ++i) {
        const int bm = i ? BM : 64;
        const double step = i ? 1.6 : 0.57, lone = i ? 1.6 : 0.75, end = i ? 12.0 : 3.0;
        const double tiles = (double)rows / bm + 0.5 * used, units = (tiles > used ? tiles : used) * tiles_c;
        const double rounds = units < 235.0 ? 1.0 : units / 256.0 + 0.5;
        const double many = rounds * (nt * step + end), one = nt * lone + end;
        t[i] = many > one ? many : one;
    }
    return t[1] < t[0] ? BM : 64;
}

int64_t grouped_grad_lda(int64_t N) { return (N + BN - 1) / BN * BN; }

hipError_t launch_grouped_rows(const GroupedRowsArgs &g, hipStream_t stream)
{
    if (g.rows <= 0) return hipSuccess;
    RowsParams p;
    p.dy = g.dy;
    p.sw = g.sw;
    p.offsets = g.offsets;
    p.experts = g.experts;
    p.row_of = g.row_of;
    p.weights = g.weights;
    p.d = g.d;
    p.dweights = g.dweights;
    p.a = g.a;
    p.lda = grouped_grad_lda(g.N);
    p.rows = (int)g.rows;
    p.groups = g.groups;
    p.N = (int)g.N;
    p.top = g.top;
    hipLaunchKernelGGL(grad_rows_kernel, workgroup_grid(g.rows), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_grouped_grad(const GroupedGradArgs &g, hipStream_t stream)
{
    if (g.rows <= 0) return hipSuccess;
    GradParams p = {};
    p.a = g.a;
    p.w1 = g.wq1;
    p.w2 = g.wq2 ? g.wq2 : g.wq1;
    p.add = g.add;
    p.dx = g.dx;
    p.rows = g.part;
    p.lda = grouped_grad_lda(g.N) * (g.wq2 ? 2 : 1);
    p.M = (int)g.rows;
    p.N = (int)g.N;
    p.K = g.K;
    p.lg = g.log2g;
    p.nt1 = (int)(grouped_grad_lda(g.N) / BN);
    p.nt = p.nt1 * (g.wq2 ? 2 : 1);
    p.tiles_c = (g.K + BC - 1) / BC;
    p.norm = (float)(1.0 / __builtin_sqrt((double)(1 << g.log2g)));
    p.next = g.next;
    p.offsets = g.offsets;
    p.slot_of = g.slot_of;
    p.groups = g.groups;
    const int bm = grouped_rows_per_tile(g.rows, g.groups, p.tiles_c, p.nt);
    const int64_t most = most_group_tiles(g.rows, g.groups, bm) * p.tiles_c;
    if (most >= ((int64_t)1 << 31) - 8) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((most + 7) & ~7));
    if (bm == 64) hipLaunchKernelGGL(grad_tile_kernel<true>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(grad_gemm_kernel<true>, grid, dim3(512), 0, stream, p);
    return hipGetLastError();
}

} // namespace convrot
