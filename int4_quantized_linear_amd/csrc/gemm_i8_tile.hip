// gemm_i8_tile.hip -- the fused INT8 linears (activation, residual, gate|up product) for batches whose
// 256 x 256 tiles would not fill the GPU (gfx950).
//
// Same contraction and epilogue arithmetic as gemm_i8.hip, so the outputs are the same bits; smaller
// tiles, so that a few hundred tokens still give every CU work, and slices of K where even those are
// few.  A call here streams its weights once and is bound by that (few tokens), or by the time one
// tile's K loop takes (some hundred tokens).
//  * 256 threads compute BM (64 or 128) tokens x 128 weight rows; two workgroups share a CU, so one
//    computes while the other waits for its loads or writes its epilogue.
//  * K goes in tiles of 128 bytes through NST LDS stages, global -> LDS, NST - 1 of them in flight,
//    with one barrier per K-tile: it publishes the K-tile just landed and frees the stage read before.
//  * 4 wavefronts in 2 (weight rows) x 2 (tokens), v_mfma_i32_16x16x64_i8.
//  * Gated: the 128 rows are 64 features of both weights in alternating 16-row blocks, as in
//    gemm_i8.hip.
//  * Split tiles store exact int32 partial sums; tile_reduce_kernel adds them and runs the epilogue.
// Bound by the K loop, 0.7 us per K-tile of 128 tokens, in which the products take 0.3 and the loads'
// way into LDS 0.35 us of issue without overlapping much.  Tried without gain: a fourth stage; the barrier
// between a K-tile's halves with the next half's reads ahead of the products; loads issued one by one
// between products; the epilogue's row scales and residuals requested ahead.
#include "activation.hpp"
#include "device_common.hpp"
#include "launchers.hpp"
#include "tile_common.hpp"

namespace convrot {
namespace {

constexpr int BN = 128, BK = 128;
constexpr int NTHREADS = 256;
constexpr int MAX_SPLIT = 16;

template <Epi E>
constexpr int features() { return E == Epi::Gated ? BN / 2 : BN; }

struct TileParams {
    const int8_t *xq;
    const int8_t *wq;
    const float *sx;
    const float *sw;
    const float *bias;
    uint16_t *y;
    int32_t *part;             // S > 1: slots of BM x BN, slice-major
    int M, N, K;
    int tiles_m, tiles_n, S;
    FusedEpi f;
};

// 16 bytes at any element: rows of an odd N start at odd ones, which vector loads and stores take.  (256 x 2176 x
// 9001: 20.3 us, element by element 23.3; 9000 columns 19.8.)
typedef v4u v4u_any __attribute__((aligned(2)));

// The residual's 8 columns n.. of row m (zeros where there is none).
template <Epi E, bool VEC>
__device__ __forceinline__ v4u residual8(const TileParams &p, int m, int n)
{
    v4u d = {};
    if (E != Epi::Act || !p.f.residual) return d;
    const uint16_t *src = p.f.residual + (int64_t)m * p.N + n;
    if (VEC || n + 8 <= p.N) {
        d = *reinterpret_cast<const v4u_any *>(src);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + e < p.N) d[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
    }
    return d;
}

// Epilogue of 8 consecutive columns n.. of row m (VEC: N % 8 == 0, all exist):
// v the scaled sums of the (gate) weight, u those of up, res the residual.
template <Epi E, bool VEC>
__device__ __forceinline__ void finish8(const TileParams &p, int m, int n, float (&v)[8], float (&u)[8], const v4u &res)
{
    const int64_t o = (int64_t)m * p.N + n;
    auto store = [&](uint16_t *dst, const float (&a)[8]) {
        const v4u d = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])};
        if (VEC || n + 8 <= p.N) {
            *reinterpret_cast<v4u_any *>(dst) = d;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < p.N) dst[e] = (uint16_t)(e & 1 ? d[e >> 1] >> 16 : d[e >> 1] & 0xffffu);
        }
    };
    if (p.f.pre) store(p.f.pre + o, v);
    if constexpr (E == Epi::Gated) {
        if (p.f.pre) store(p.f.pre + (int64_t)p.M * p.N + o, u);
        act_values(v, p.f.act);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= u[e];
    } else {
        act_values(v, p.f.act);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += e & 1 ? bf16hi_to_f32(res[e >> 1]) : bf16lo_to_f32(res[e >> 1]);
    }
    store(p.y + o, v);
}

// Scale and bias of the 8 columns n.. (past N: the last columns', which no caller uses; a branch per column
// costs more than the load: the slices' join 6.0 us with them, 4.1 without, 300 tokens x 2688).
template <bool VEC>
__device__ __forceinline__ void columns8(const float *sw, const float *bias, int n, int N, float (&s)[8], float (&b)[8])
{
    const int first = VEC ? min(n, N - 8) : n;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = VEC ? first + e : min(n + e, N - 1);
        s[e] = sw[i];
        b[e] = 0.0f;
    }
    if (bias) {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = bias[VEC ? first + e : min(n + e, N - 1)];
    }
}

template <Epi E, int BM, int NST, bool VEC>
__global__ void __launch_bounds__(NTHREADS, 2) gemm_i8_tile_kernel(TileParams p)
{
    constexpr int NF = features<E>();
    constexpr int STAGE = (BN + BM) * BK;
    constexpr int LPK = (BN + BM) / 32;                  // loads per K-tile and wave
    constexpr int MB = BM / 32;                          // 16-token blocks per wave
    __shared__ __attribute__((aligned(16))) uint8_t smem[NST * STAGE];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = w & 1, wm = w >> 1;
    const int K = p.K, KT = (K + BK - 1) / BK;
    const int T = p.tiles_m * p.tiles_n, U = T * p.S;
    if ((int)blockIdx.x >= U) return;                    // the grid is rounded up to a multiple of 8
    const int unit = unit_of((int)blockIdx.x, 0, U);
    const int sl = unit / T;
    const int kb = sl * KT / p.S, ke = (sl + 1) * KT / p.S;
    int tm, tn;
    tile_coords(unit - sl * T, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * NF;

    // instruction i of wave w fills LDS rows 8 (4 i + w) .. + 7 (weight rows 0 .. 127, then tokens);
    // lane -> row + lane / 8 at position lane % 8
    uint32_t off[LPK];
#pragma unroll
    for (int i = 0; i < LPK; ++i) {
        const int r = 8 * (4 * i + w) + (lane >> 3), c = 16 * ((lane & 7) ^ swz(r));
        if (i < 4) {
            const int wr = E == Epi::Gated ? 16 * (r >> 5) + (r & 15) : r;
            off[i] = n0 + wr < p.N ? (uint32_t)(wr * K + c) : OOB;
        } else {
            off[i] = m0 + r - BN < p.M ? (uint32_t)((r - BN) * K + c) : OOB;
        }
    }
    const int8_t *wsrc = E == Epi::Gated && (w & 2) ? p.f.wq2 : p.wq;   // rows 16..31 of each 32: up
    const uint64_t wbase = reinterpret_cast<uint64_t>(wsrc + (int64_t)n0 * K);
    const uint64_t xbase = reinterpret_cast<uint64_t>(p.xq + (int64_t)m0 * K);
    // the last K-tile may be half (K % 128 == 64): its chunks 4 .. 7 are past K (the lane's chunk is
    // (lane % 8) ^ swz(row), and swz of rows 8 (4 i + w) + l is swz(8 w + l) for every i)
    const uint32_t half = K % BK && ((lane & 7) ^ swz(8 * w + (lane >> 3))) >= 4 ? OOB : 0u;
    auto issue = [&](int t) {
        const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(wbase, NUM_RECORDS), rx = uniform_rsrc(xbase, NUM_RECORDS);
        uint8_t *base = smem + ((t - kb) % NST) * STAGE + w * 1024;
        const uint32_t skip = t >= ke ? OOB : t == KT - 1 ? half : 0u;
        const int k0 = __builtin_amdgcn_readfirstlane(t < ke ? t * BK : 0);
#pragma unroll
        for (int i = 0; i < LPK; ++i)
            load16_to_lds(i < 4 ? rw : rx, base + 4096 * i, off[i] | skip, k0);
    };

    const int frow = lane & 15, fq = lane >> 4;
    v4i acc[4][MB];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[a][b] = v4i{};
#pragma unroll
    for (int j = 0; j < NST - 1; ++j) issue(kb + j);
    for (int t = kb; t < ke; ++t) {
        // K-tile t has landed once only the NST - 2 after it are in flight
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * LPK));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        issue(t + NST - 1);
        const uint8_t *st = smem + ((t - kb) % NST) * STAGE;
        const uint8_t *ar = st + (wn * 64 + frow) * BK, *br = st + (BN + wm * (BM / 2) + frow) * BK;
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
    }
    // lane: token lane % 16 of block b, weight rows 16 a + 4 (lane / 16) + v of the wave's 64
    if (p.S > 1) {
        int32_t *dst = p.part + (int64_t)unit * (BM * BN);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const int ml = wm * (BM / 2) + 16 * b + frow;
            if (m0 + ml < p.M) {
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    *reinterpret_cast<v4i *>(dst + ml * BN + wn * 64 + 16 * a + 4 * fq) = acc[a][b];
            }
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));       // the last loads into LDS
        return;
    }
    // Each wave passes its 16-token blocks through its own 4 KiB (rows of 64 sums, 16-byte chunk c at
    // c ^ row), then takes row pieces of 8 output columns per lane.
    constexpr int LPR = NF / 2 / 8, RPI = 64 / LPR;      // lanes per row, rows at a time
    const int lrow = lane / LPR, lcol = lane % LPR;
    const int n = n0 + wn * (NF / 2) + 8 * lcol;
    const int ch = E == Epi::Gated ? 8 * (lcol >> 1) + 2 * (lcol & 1) : 2 * lcol;
    float s1[8], b1[8], s2[8], b2[8];
    columns8<VEC>(p.sw, p.bias, n, p.N, s1, b1);
    if constexpr (E == Epi::Gated) columns8<VEC>(p.f.sw2, p.f.bias2, n, p.N, s2, b2);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    uint8_t *reg = smem + w * 4096;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
            *reinterpret_cast<v4i *>(reg + frow * 256 + 16 * ((4 * a + fq) ^ frow)) = acc[a][b];
#pragma unroll 1
        for (int q = 0; q < 16 / RPI; ++q) {
            const int r = RPI * q + lrow, m = m0 + wm * (BM / 2) + 16 * b + r;
            if (m >= p.M || n >= p.N) continue;
            const float sxm = p.sx[m];
            auto z8 = [&](int chunk, const float (&s)[8], const float (&bi)[8], float (&v)[8]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const v4i d = *reinterpret_cast<const v4i *>(reg + r * 256 + 16 * ((chunk + h) ^ r));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[4 * h + i] = __builtin_fmaf((float)d[i], sxm * s[4 * h + i], bi[4 * h + i]);
                }
            };
            float v[8], u[8];
            z8(ch, s1, b1, v);
            if constexpr (E == Epi::Gated) z8(ch + 4, s2, b2, u);
            finish8<E, VEC>(p, m, n, v, u, residual8<E, VEC>(p, m, n));
        }
    }
}

// Split tiles: adds a row piece's S partial sums (exact) and runs the same epilogue.
template <Epi E, int BM, bool VEC>
__global__ void __launch_bounds__(256) tile_reduce_kernel(TileParams p, int rb)
{
    constexpr int NF = features<E>(), TPR = NF / 8, RPW = 256 / TPR;
    const int T = p.tiles_m * p.tiles_n;
    const int i = (int)blockIdx.x / rb;
    const int ml = ((int)blockIdx.x % rb) * RPW + (int)threadIdx.x / TPR, nl = ((int)threadIdx.x % TPR) * 8;
    int tm, tn;
    tile_coords(i, p.tiles_m, p.tiles_n, tm, tn);
    const int m = tm * BM + ml, n = tn * NF + nl;
    if (ml >= BM || m >= p.M || n >= p.N) return;
    // everything is requested before the first sum is used: the kernel is one memory latency long
    const float sxm = p.sx[m];
    const v4u res = residual8<E, VEC>(p, m, n);
    float s1[8], b1[8], s2[8], b2[8];
    columns8<VEC>(p.sw, p.bias, n, p.N, s1, b1);
    if constexpr (E == Epi::Gated) columns8<VEC>(p.f.sw2, p.f.bias2, n, p.N, s2, b2);
    auto sums = [&](int cl, const float (&sc)[8], const float (&bi)[8], float (&v)[8]) {
        int32_t sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const int32_t *src = p.part + (int64_t)i * (BM * BN) + ml * BN + cl;
#pragma unroll 1
        for (int s = 0; s < p.S; s += 8) {
            v4i a[8], b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = b[i] = v4i{};
                if (s + i < p.S) {
                    a[i] = *reinterpret_cast<const v4i *>(src);
                    b[i] = *reinterpret_cast<const v4i *>(src + 4);
                    src += (int64_t)T * (BM * BN);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum[e] += a[i][e];
                    sum[e + 4] += b[i][e];
                }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf((float)sum[e], sxm * sc[e], bi[e]);
    };
    const int cl = E == Epi::Gated ? 32 * (nl >> 4) + (nl & 15) : nl;
    float v[8], u[8];
    sums(cl, s1, b1, v);
    if constexpr (E == Epi::Gated) sums(cl + 16, s2, b2, u);
    finish8<E, VEC>(p, m, n, v, u, res);
}

template <Epi E, int BM, int NST, bool VEC>
void launch_tiles(const TileParams &p, hipStream_t stream)
{
    const int U = p.tiles_m * p.tiles_n * p.S;
    hipLaunchKernelGGL((gemm_i8_tile_kernel<E, BM, NST, VEC>), dim3((unsigned)((U + 7) & ~7)), dim3(NTHREADS), 0, stream,
                       p);
    if (p.S == 1) return;
    constexpr int rpw = 256 / (features<E>() / 8);
    const int rows = p.M < BM ? p.M : BM, rb = (rows + rpw - 1) / rpw;
    hipLaunchKernelGGL((tile_reduce_kernel<E, BM, VEC>), dim3((unsigned)(p.tiles_m * p.tiles_n) * (unsigned)rb), dim3(256),
                       0, stream, p, rb);
}

constexpr int CUS = 256;

// 64 tokens: three stages, 72 KiB.  128 tokens: two, 64 KiB, so that two workgroups share a CU, but
// three (96 KiB, one workgroup) when there is at most one per CU anyway: 39 us against 45 at 128 tokens,
// 25600 x 5120, in 6 slices; with 400 workgroups (128 tokens, 5120 x 2 * 25600) 74 us against 71.
template <Epi E, bool VEC>
void launch_epi(const TileParams &p, int bm, hipStream_t stream)
{
    if (bm == 64) launch_tiles<E, 64, 3, VEC>(p, stream);
    else if (p.tiles_m * p.tiles_n * p.S <= CUS) launch_tiles<E, 128, 3, VEC>(p, stream);
    else launch_tiles<E, 128, 2, VEC>(p, stream);
}

int64_t tiles_of(int64_t M, int64_t N, int bm, bool gated)
{
    const int64_t nf = gated ? BN / 2 : BN;
    return ((M + bm - 1) / bm) * ((N + nf - 1) / nf);
}

} // namespace

// The fastest of 256 x 256 tiles, and 64- and 128-token tiles in 1 to 16 slices, by a model with
// measured constants.  A CU takes 0.39 (64 tokens) or 0.61 us (128) per K-tile of a workgroup when it
// has several, and a lone workgroup 0.46 or 0.67 us; the weights stream at 4.9 TB/s; slices add their
// partial sums' round trip (4 TB/s) and a launch; prologue, epilogue and launch take about 4 us.
// Measured (us; K x N, 2 N for gate|up, weights not in cache), 256 x 256 tiles against the choice:
//   5120 x 2 * 25600: 17 tokens 78 / 56, 64: 75 / 61, 128: 82 / 71, 256: 92 / 121 (so 256 x 256 is taken)
//   25600 x 5120: 32 tokens 48 / 30, 128: 61 / 39, 512: 97 / 103 (256 x 256 taken)
//   2688 x 2 * 5376: 300 tokens 37 / 22, 1024: 41 / 47 (taken);   2688 x 1001: 333 tokens 51 / 12
TilePlan plan_gemm_i8_tile(int64_t M, int64_t N, int K, bool gated, bool split)
{
    TilePlan best;
    double t_best = gemm_i8_seconds(M, N, K, gated, split);
    best.part_bytes = split ? gemm_i8_split_bytes(M, N, K, true, gated) : 0;
    const int KT = (K + BK - 1) / BK;
    const double cols = (double)N * (gated ? 2.0 : 1.0);
    const double stream = cols * K / 4.9e12;
    for (int bm = 64; bm <= 128; bm *= 2) {
        const int64_t T = tiles_of(M, N, bm, gated);
        if (T >= (int64_t)1 << 20) continue;
        const double several = bm == 64 ? 0.39e-6 : 0.61e-6, lone = bm == 64 ? 0.46e-6 : 0.67e-6;
        for (int S = 1; S <= (split ? MAX_SPLIT : 1); ++S) {
            const int64_t U = T * S;
            if (S > 1 && (KT / S < 2 || U > 4 * CUS)) break;
            const double per_cu = (double)((U + CUS - 1) / CUS) * several;
            const double math = (double)((KT + S - 1) / S) * (per_cu > lone ? per_cu : lone);
            const double joined = S > 1 ? (double)M * cols * S * 8.0 / 4e12 + 4e-6 : 0.0;
            const double t = (math > stream ? math : stream) + joined + 4e-6;
            if (t < t_best) {
                t_best = t;
                best.bm = bm;
                best.S = S;
                best.part_bytes = S > 1 ? (size_t)U * bm * BN * sizeof(int32_t) : 0;
            }
        }
    }
    return best;
}

hipError_t launch_gemm_i8_tile(const TilePlan &pl, const int8_t *xq, const int8_t *wq, const float *sx, const float *sw,
                               const float *bias, void *y, Epi epi, int64_t M, int64_t N, int K, void *part,
                               hipStream_t stream, const FusedEpi &fused)
{
    if (M <= 0 || N <= 0) return hipSuccess;
    if ((epi != Epi::Act && epi != Epi::Gated) || (pl.bm != 64 && pl.bm != 128)) return hipErrorInvalidValue;
    TileParams p;
    p.xq = xq;
    p.wq = wq;
    p.sx = sx;
    p.sw = sw;
    p.bias = bias;
    p.y = static_cast<uint16_t *>(y);
    p.part = static_cast<int32_t *>(part);
    p.M = (int)M;
    p.N = (int)N;
    p.K = K;
    p.tiles_m = (int)((M + pl.bm - 1) / pl.bm);
    p.tiles_n = (int)(tiles_of(M, N, pl.bm, epi == Epi::Gated) / p.tiles_m);
    p.S = pl.S;
    p.f = fused;
    const bool vec = N % 8 == 0;
    if (epi == Epi::Gated && vec) launch_epi<Epi::Gated, true>(p, pl.bm, stream);
    else if (epi == Epi::Gated) launch_epi<Epi::Gated, false>(p, pl.bm, stream);
    else if (vec) launch_epi<Epi::Act, true>(p, pl.bm, stream);
    else launch_epi<Epi::Act, false>(p, pl.bm, stream);
    return hipGetLastError();
}

} // namespace convrot
