// launchers.hpp -- internal host launchers of the ConvRot HIP kernels (not the public ABI).
// Every launcher assumes its arguments were validated by the C-ABI layer and only returns
// the launch status.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

// Rotate rows of x (bf16 or fp32, [rows, K]) by the grouped Hadamard and quantize:
// bits 8 -> q int8 [rows, K], scale fp32 [rows]; bits 4 -> q uint8 [rows, K/2], scale fp16 [rows, K/256].
hipError_t launch_rotate_quant(const void *x, bool x_f32, int64_t rows, int K, int log2g, int bits, void *q,
                               void *scale, hipStream_t stream);
// The INT4 case (log2g 7 or 8, K % 128 == 0) written straight as the FP6 tiles of the W4A4 GEMM:
// tiles of w4a4_tiled_bytes(rows, 0, K) bytes (rows padded to 32 with zero codes), scale as above.
hipError_t launch_rotate_quant_fp6(const void *x, bool x_f32, int64_t rows, int K, int log2g, uint8_t *tiles,
                                   void *scale, hipStream_t stream);

// Epilogue selector of the integer GEMM / GEMV kernels.
//   Act:   z = acc * sx[m] * sw[n] + bias[n];  y = bf16(act(z) + residual);  pre = bf16(z)
//   Gated: two weights share the tokens: g, u as z;  y = bf16(act(g) * u);  pre = bf16([g; u])
//   Part:  z in fp32, d = bf16(z)  (rows sorted by group only)
enum class Epi { Bf16 = 0, Int32 = 1, Act = 2, Gated = 3, Part = 4 };

// What the Act and Gated epilogues take besides the plain one's arguments (activation.hpp holds
// the codes of act).  residual, pre, bias2: may be null.  residual may be y itself.
struct FusedEpi {
    int act = 0;
    const uint16_t *residual = nullptr;   // bf16 [M, N] (Act)
    uint16_t *pre = nullptr;              // bf16 [M, N] (Act), [2, M, N] gate then up (Gated)
    const int8_t *wq2 = nullptr;          // the up weight [N, K], its scales and bias (Gated)
    const float *sw2 = nullptr;
    const float *bias2 = nullptr;
};

// y[M,N] = bf16(acc * sx[m] * sw[n] + bias[n])  or  acc32[M,N] = acc,   acc = xq . wq^T  (M > 16).
// part: optional scratch for the split-K tail (bf16 output only): when the tiles leave the last
// round of the persistent grid partly idle and part_bytes >= gemm_i8_split_bytes(M, N, K), the
// tail tiles are computed as K-slices whose int32 partial sums meet in `part`, then a second
// kernel sums them and applies the epilogue (bit-identical outputs).  part == nullptr: no split.
hipError_t launch_gemm_i8(const int8_t *xq, const int8_t *wq, const float *sx, const float *sw, const float *bias,
                          void *y, Epi epi, int64_t M, int64_t N, int K, void *part, size_t part_bytes,
                          hipStream_t stream, const FusedEpi &fused = FusedEpi());
// Bytes of `part` the split-K tail uses for this shape on the current device (0: no split).
size_t gemm_i8_split_bytes(int64_t M, int64_t N, int K, bool fused = false, bool gated = false);
// Estimated seconds of launch_gemm_i8's fused epilogues, with or without `part`, for the choice below.
double gemm_i8_seconds(int64_t M, int64_t N, int K, bool gated, bool split);

// The Act and Gated linears in tiles of bm (64 or 128) tokens x 128 weight rows, each in S slices of K
// (part: the plan's part_bytes when S > 1).  Same outputs as launch_gemm_i8, bit for bit.
struct TilePlan {
    int bm = 0, S = 1;         // bm == 0: launch_gemm_i8's 256 x 256 tiles are the better choice
    size_t part_bytes = 0;     // for either
};
TilePlan plan_gemm_i8_tile(int64_t M, int64_t N, int K, bool gated, bool split);
hipError_t launch_gemm_i8_tile(const TilePlan &pl, const int8_t *xq, const int8_t *wq, const float *sx, const float *sw,
                               const float *bias, void *y, Epi epi, int64_t M, int64_t N, int K, void *part,
                               hipStream_t stream, const FusedEpi &fused);

// Same contraction for M <= 16 (weight streaming; K split among the wavefronts of a workgroup,
// no scratch memory).
hipError_t launch_gemv_i8(const int8_t *xq, const int8_t *wq, const float *sx, const float *sw, const float *bias,
                          void *y, Epi epi, int64_t M, int64_t N, int K, hipStream_t stream,
                          const FusedEpi &fused = FusedEpi());

// Input gradient of an INT8 linear, or of two that share their tokens (gated: gate and up):
//   dz = dy act'(pre)  (pre null: dy);   gate/up: dg = dy u act'(g), du = dy act(g), pre = [g; u]
//   dx = bf16((sum_n dz sw wq) R + add),  db = column sums of dz (fp32; null: not computed)
// ws: grad_workspace_bytes(M, N, K, gated) bytes, 256-byte aligned.  M == 0 still writes db.
// next.a: instead of dx, the gradient through a gated product whose h this launch's input was:
// [M, 2 K] bf16, dg sw_gate then du sw_up, from pre = [g; u] ([2, M, K]) and dh = bf16(the gradient).
struct GradNext {
    const uint16_t *pre = nullptr;
    const float *sw_gate = nullptr, *sw_up = nullptr;
    uint16_t *a = nullptr;
    int act = 0;
};
struct GradArgs {
    const uint16_t *dy = nullptr, *pre = nullptr;
    int64_t M = 0, N = 0;
    int K = 0, log2g = 0, act = 0;
    const int8_t *wq1 = nullptr, *wq2 = nullptr;
    const float *sw1 = nullptr, *sw2 = nullptr;
    const uint16_t *add = nullptr;
    uint16_t *dx = nullptr;
    float *db1 = nullptr, *db2 = nullptr;
    const uint16_t *a = nullptr;          // the operand as a previous launch's `next` wrote it: dy, pre
                                          // and the scales are not read, no db
    GradNext next;
    void *ws = nullptr;
};
size_t grad_workspace_bytes(int64_t M, int64_t N, int K, bool gated, bool a_given = false);
hipError_t launch_grad_i8(const GradArgs &g, bool gated, hipStream_t stream);

// ---- mixture of experts (grouped_common.hpp says what offsets hold)
//
// Where the slots (token, j) of M tokens with `top` experts each go when sorted by expert, E <= MAX_GROUPS: rows
// offsets[e] .. offsets[e + 1] - 1 are expert e's, in slot order; slots with an expert outside [0, E) have row -1 and
// take no row.  All in device memory, S = M top entries (offsets: E + 1).
// With sx (fp32 [M]) also each row's token's scale, in sx_of [S].
struct MoeOrder {
    int32_t *offsets = nullptr, *slot_of = nullptr, *token_of = nullptr, *row_of = nullptr;
    const float *sx = nullptr;
    float *sx_of = nullptr;
};
hipError_t launch_moe_order(const int32_t *experts, int64_t S, int E, int top, const MoeOrder &o, hipStream_t stream);

// Products of rows sorted by group with their group's weight, z = acc sx sw:
//   Bf16: y = bf16(z);   Gated: y = bf16(act(g) u), pre = bf16([g; u]);   Part: part = z in fp32, d = bf16(z)
// Rows of no group are neither read nor written.  Gated and Part: N % 8 == 0.
struct GroupedArgs {
    const int8_t *xq = nullptr;           // [rows, K], or with `source` any rows, of fewer than 2^31 bytes in all
    const float *sx = nullptr;            // [rows]
    const int32_t *offsets = nullptr;
    const int32_t *source = nullptr;      // the row of xq that a row takes; null: its own
    const int32_t *slot_of = nullptr;     // the row of pre and d that a row goes to (with pre or d)
    const int8_t *wq = nullptr, *wq2 = nullptr;   // [groups, N, K]
    const float *sw = nullptr, *sw2 = nullptr;    // [groups, N]
    uint16_t *y = nullptr, *pre = nullptr, *d = nullptr;   // pre [2, rows, N] (or null), d [rows, N] (or null)
    float *part = nullptr;                // [rows, N]
    int64_t rows = 0, N = 0;
    int groups = 0, K = 0, act = 0;
};
hipError_t launch_grouped_i8(const GroupedArgs &g, Epi epi, hipStream_t stream);
// The same in 256 x 256 tiles (gemm_i8.hip), for launch_grouped_i8.
hipError_t launch_grouped_gemm_i8(const GroupedArgs &g, Epi epi, hipStream_t stream);

// Gradients of grouped products through the frozen weights, in two steps (contractions of grouped_grad_lda(N) columns
// per weight):
//   rows:  a[row] = bf16(share dy[source] sw[group]);  with `experts` (one workgroup per slot) share, source and row are the
//          slot's weight, token and place in the sort, and dweights[slot] = sum dy[token] d[slot] (0 without an expert)
//   grad:  v = (a . wq[group]) R;  to dx = bf16(v + add), to part = v in fp32, or on to next.a (GradNext, its pre [2, rows, K]
//          read at row slot_of[row], its scales [groups, K])
int64_t grouped_grad_lda(int64_t N);
struct GroupedRowsArgs {
    const uint16_t *dy = nullptr;
    const float *sw = nullptr;
    const int32_t *offsets = nullptr, *experts = nullptr, *row_of = nullptr;
    const float *weights = nullptr;
    const uint16_t *d = nullptr;
    float *dweights = nullptr;
    uint16_t *a = nullptr;
    int64_t rows = 0, N = 0;
    int groups = 0, top = 1;
};
hipError_t launch_grouped_rows(const GroupedRowsArgs &g, hipStream_t stream);
struct GroupedGradArgs {
    const uint16_t *a = nullptr;
    const int32_t *offsets = nullptr, *slot_of = nullptr;
    const int8_t *wq1 = nullptr, *wq2 = nullptr;
    const uint16_t *add = nullptr;
    uint16_t *dx = nullptr;
    float *part = nullptr;                // fp32 [rows, K]
    GradNext next;
    int64_t rows = 0, N = 0;
    int groups = 0, K = 0, log2g = 0;
};
hipError_t launch_grouped_grad(const GroupedGradArgs &g, hipStream_t stream);

// y[m] = bf16(sum_j weights[m, j] part[row_of[m, j]] + residual[m])  (weights null: 1; K % 4 == 0).
hipError_t launch_moe_combine(const float *part, const int32_t *row_of, const float *weights, const uint16_t *residual,
                              uint16_t *y, int64_t M, int K, int top, hipStream_t stream);

// The expert layer for at most 64 slots (moe_few.hip): plan_moe_few says whether it takes the call and which of
// the two kernels quantizes its rows itself; where one does not, its codes and scales (xq, xs of the tokens; hq, hs of h's
// slots) are made by launch_rotate_quant before it.
struct MoeFew {
    bool fuse_x = false, fuse_h = false;
};
struct MoeFewArgs {
    const void *x = nullptr;
    bool x_f32 = false;
    const int8_t *xq = nullptr, *hq = nullptr;
    const float *xs = nullptr, *hs = nullptr;
    const int32_t *experts = nullptr;
    const float *weights = nullptr;
    const int8_t *wq_gate = nullptr, *wq_up = nullptr, *wq_down = nullptr;
    const float *gate_scale = nullptr, *up_scale = nullptr, *down_scale = nullptr;
    const uint16_t *residual = nullptr;
    uint16_t *h = nullptr, *y = nullptr;  // h [S, F] by slot
    uint16_t *pre = nullptr, *d = nullptr;   // bf16 [2, S, F] and [S, K], or null
    int64_t M = 0;
    int top = 0, E = 0, K = 0, F = 0, act = 0, log2g = 0, log2g_h = 0;
};
bool plan_moe_few(int64_t M, int top, int K, int F, MoeFew &plan);
hipError_t launch_moe_few_gate(const MoeFewArgs &a, const MoeFew &plan, hipStream_t stream);
hipError_t launch_moe_few_down(const MoeFewArgs &a, const MoeFew &plan, hipStream_t stream);

// Router: see convrot_moe_route and convrot_moe_route_backward.
struct RouteArgs {
    const void *logits = nullptr;         // [M, E]
    bool f32 = false;
    const float *bias = nullptr;
    int64_t M = 0;
    int E = 0, top = 0, score = 0;
    bool normalize = false;
    float scale = 1.0f;
};
hipError_t launch_moe_route(const RouteArgs &a, int32_t *experts, float *weights, hipStream_t stream);
hipError_t launch_moe_route_backward(const RouteArgs &a, const float *dweights, const int32_t *experts, void *dlogits,
                                     hipStream_t stream);

// W4A4: y = bf16(sum_g acc_g * sx[m,g] * sw[n,g] + bias[n]) with packed int4 operands and
// fp16 group scales (group = 256 or 128, K % group == 0, K >= 256), or the unscaled int32 total
// sum_k cx*cw (scales ignored).
// Both operands run through the FP6 tiles of launch_tile_w4a4: the tokens are re-encoded into
// the start of `ws` unless x_tiled says xq already holds their tiles (launch_rotate_quant_fp6),
// the weights after them unless w_tiled says wq does.  `ws` is scratch of
// w4a4_tiled_bytes(M, w_tiled ? 0 : N, K) bytes (16-byte aligned).
size_t w4a4_tiled_bytes(int64_t M, int64_t N, int K);
// Packed int4 rows [R, K/2] -> FP6 tiles (w4a4_tiled_bytes(R, 0, K) bytes), K % 128 == 0.
hipError_t launch_tile_w4a4(const uint8_t *q, int64_t R, int K, uint8_t *out, hipStream_t stream);
hipError_t launch_gemm_w4a4(const uint8_t *xq, bool x_tiled, const uint8_t *wq, bool w_tiled, const uint16_t *sx,
                            const uint16_t *sw, const float *bias, void *y, Epi epi, int64_t M, int64_t N, int K,
                            int group, void *ws, hipStream_t stream);

// W4A8 decode linear (M <= 16): y = bf16(sx[m] * sum_g sw[g,n] * (qx . cw over group g) + bias[n])
// with INT8 tokens and the weights in the W4A8 block layout (codes and fp16 group scales), made
// once by launch_pack_w4a8 from packed INT4 [N, K/2] and scales [K/group, N] (group 256, or 128
// with two scale sets per 256-channel block); N % 8 == 0.
// No scratch memory: K is split only among the wavefronts of one workgroup.
size_t w4a8_packed_bytes(int64_t N, int K, int group);
hipError_t launch_pack_w4a8(const uint8_t *wq, const uint16_t *sw, int64_t N, int K, int group, uint8_t *out,
                            hipStream_t stream);
int gemv_w4a8_waves(int64_t N, int K);
hipError_t launch_gemv_w4a8(const int8_t *xq, const float *sx, const uint8_t *wp, const float *bias, void *y,
                            int64_t M, int64_t N, int K, int group, hipStream_t stream);

} // namespace convrot
