// convrot_abi.hip -- host side of the libconvrot C-ABI: argument validation, dispatch by
// shape, workspace layout and error reporting.  Every precondition is checked before the first
// HIP call, so a rejected call enqueues nothing.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <string>

#include "../../include/convrot.h"
#include "launchers.hpp"

namespace {

thread_local std::string g_last_error;

int fail(int code, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = std::string(convrot_status_string(code)) + ": " + buf;
    return code;
}

bool pow2_group(int g) { return g >= 1 && g <= 256 && (g & (g - 1)) == 0; }
int log2i(int g)
{
    int l = 0;
    while ((1 << l) < g) ++l;
    return l;
}
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

int check_shape(int64_t M, int64_t N, int64_t K, int group, const char *who)
{
    if (M < 0 || N < 0 || M >= ((int64_t)1 << 31) || N >= ((int64_t)1 << 31))
        return fail(CONVROT_ERR_SHAPE, "%s: M=%lld N=%lld must be in [0, 2^31)", who, (long long)M, (long long)N);
    if (K < 64 || K > CONVROT_MAX_K || K % 64)
        return fail(CONVROT_ERR_SHAPE, "%s: K=%lld must be a multiple of 64 in [64, %d]", who, (long long)K,
                    CONVROT_MAX_K);
    if (!pow2_group(group))
        return fail(CONVROT_ERR_GROUP, "%s: group=%d must be a power of two in [1, 256]", who, group);
    if (K % group) return fail(CONVROT_ERR_SHAPE, "%s: K=%lld is not a multiple of group=%d", who, (long long)K, group);
    return CONVROT_OK;
}

// N limit of the tiled GEMMs (their 32-row output blocks use 32-bit byte offsets).
int check_gemm_n(int64_t N, const char *who)
{
    if (N >= CONVROT_GEMM_MAX_N)
        return fail(CONVROT_ERR_SHAPE, "%s: N=%lld; the tiled GEMM (M > 16, or W4A4) needs N < %d", who, (long long)N,
                    CONVROT_GEMM_MAX_N);
    return CONVROT_OK;
}

// One cached answer per device: is it gfx950?
int check_device()
{
    static std::mutex mu;
    static int known[64];   // 0 unknown, 1 ok, 2 wrong arch
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(CONVROT_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= 64) return fail(CONVROT_ERR_DEVICE, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lk(mu);
    if (!known[dev]) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess) return fail(CONVROT_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
        known[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        if (known[dev] == 2) return fail(CONVROT_ERR_DEVICE, "device %d is %s, libconvrot is built for gfx950", dev, prop.gcnArchName);
    }
    return known[dev] == 1 ? CONVROT_OK : fail(CONVROT_ERR_DEVICE, "device %d is not gfx950", dev);
}

int hip_status(hipError_t e, const char *what)
{
    return e == hipSuccess ? CONVROT_OK : fail(CONVROT_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Workspace layout, each region 256-byte aligned; all of it is scratch (no initial contents):
//   bits 8: [xq int8 M*K][x_scale fp32 M]
//   bits 4: [xq packed M*K/2][x_scale fp16 (K/128)*M, enough for either INT4 group][FP6 tiles of
//           both operands]
struct WsLayout {
    size_t xq = 0, xs = 0, tiles = 0, part = 0, total = 0;
};

// epi: the Act and Gated linears plan their K slices themselves.
WsLayout ws_layout(int64_t M, int64_t N, int64_t K, int bits, convrot::Epi epi = convrot::Epi::Bf16)
{
    WsLayout L;
    size_t off = 0;
    if (bits == 8) {
        L.xq = off;
        off += round256((size_t)(M * K));
        L.xs = off;
        off += round256((size_t)M * 4);
        // optional: the split-K tail's int32 partial sums (GEMM path only)
        L.part = off;
        if (M > 16)
            off += round256(epi == convrot::Epi::Bf16
                                ? convrot::gemm_i8_split_bytes(M, N, (int)K)
                                : convrot::plan_gemm_i8_tile(M, N, (int)K, epi == convrot::Epi::Gated, true).part_bytes);
    } else {
        L.xq = off;
        off += round256((size_t)(M * K / 2));
        L.xs = off;
        off += round256((size_t)(M * ((K + 127) / 128) * 2));
        L.tiles = off;
        off += round256(convrot::w4a4_tiled_bytes(M, N, (int)K));
    }
    L.total = off;
    return L;
}

// W4A8 workspace: [xq int8 M*K][x_scale fp32 M], used when the entry point quantizes x itself.
WsLayout ws_layout_w4a8(int64_t M, int64_t K)
{
    WsLayout L;
    size_t off = 0;
    L.xq = off;
    off += round256((size_t)(M * K));
    L.xs = off;
    off += round256((size_t)M * 4);
    L.total = off;
    return L;
}

// [a, a + an) and [b, b + bn) share a byte (either may be NULL: they share none).
bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + bn && y < x + an;
}

int check_act(int act, const char *who)
{
    return act >= CONVROT_ACT_NONE && act <= CONVROT_ACT_GELU_TANH
               ? CONVROT_OK
               : fail(CONVROT_ERR_ACT, "%s: act=%d is not one of CONVROT_ACT_*", who, act);
}

int quantize_common(const void *x, int dtype, int64_t R, int64_t K, int group, int bits, void *q, void *scale,
                    hipStream_t stream, const char *who)
{
    if (R == 0 && K >= 64 && K <= CONVROT_MAX_K && K % 64 == 0 && pow2_group(group) && K % group == 0)
        return CONVROT_OK;   // empty input: nothing to read or write
    if (!x || !q || !scale) return fail(CONVROT_ERR_NULL, "%s: x, q and scale must be non-NULL", who);
    if (dtype != CONVROT_DTYPE_F32 && dtype != CONVROT_DTYPE_BF16) return fail(CONVROT_ERR_DTYPE, "%s: dtype=%d", who, dtype);
    if (bits != 8 && bits != 4) return fail(CONVROT_ERR_BITS, "%s: bits=%d", who, bits);
    int rc = check_shape(R, 1, K, group, who);
    if (rc) return rc;
    if (bits == 4 && group != 256 && group != 128)
        return fail(CONVROT_ERR_GROUP, "%s: INT4 needs group 256 or 128 (group=%d, K=%lld)", who, group, (long long)K);
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, bits == 8 ? 4 : 2))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    if (R == 0) return CONVROT_OK;
    if ((rc = check_device())) return rc;
    return hip_status(convrot::launch_rotate_quant(x, dtype == CONVROT_DTYPE_F32, R, (int)K, log2i(group), bits, q,
                                                   scale, stream),
                      who);
}

} // namespace

extern "C" {

const char *convrot_status_string(int s)
{
    switch (s) {
    case CONVROT_OK: return "CONVROT_OK";
    case CONVROT_ERR_NULL: return "CONVROT_ERR_NULL";
    case CONVROT_ERR_SHAPE: return "CONVROT_ERR_SHAPE";
    case CONVROT_ERR_GROUP: return "CONVROT_ERR_GROUP";
    case CONVROT_ERR_ALIGN: return "CONVROT_ERR_ALIGN";
    case CONVROT_ERR_DTYPE: return "CONVROT_ERR_DTYPE";
    case CONVROT_ERR_BITS: return "CONVROT_ERR_BITS";
    case CONVROT_ERR_WORKSPACE: return "CONVROT_ERR_WORKSPACE";
    case CONVROT_ERR_HIP: return "CONVROT_ERR_HIP";
    case CONVROT_ERR_DEVICE: return "CONVROT_ERR_DEVICE";
    case CONVROT_ERR_ACT: return "CONVROT_ERR_ACT";
    case CONVROT_ERR_OVERLAP: return "CONVROT_ERR_OVERLAP";
    case CONVROT_ERR_SCORE: return "CONVROT_ERR_SCORE";
    default: return "CONVROT_ERR_UNKNOWN";
    }
}

const char *convrot_last_error(void) { return g_last_error.c_str(); }

int convrot_dynamic_group(int64_t K, int max_group)
{
    if (K <= 0 || !pow2_group(max_group)) return 0;
    int g = max_group;
    while (K % g) g >>= 1;
    return g;
}

int convrot_prepare_weight(const void *w, int w_dtype, int64_t N, int64_t K, int group, int bits, void *wq,
                           void *w_scale, hipStream_t stream)
{
    return quantize_common(w, w_dtype, N, K, group, bits, wq, w_scale, stream, "convrot_prepare_weight");
}

int convrot_quantize_act(const void *x, int x_dtype, int64_t M, int64_t K, int group, int bits, void *xq,
                         void *x_scale, hipStream_t stream)
{
    return quantize_common(x, x_dtype, M, K, group, bits, xq, x_scale, stream, "convrot_quantize_act");
}

size_t convrot_workspace_bytes(int64_t M, int64_t N, int64_t K, int bits)
{
    // the shapes the entry points accept (check_shape), which also keeps every size below in range
    if (M < 0 || N < 0 || M >= ((int64_t)1 << 31) || N >= ((int64_t)1 << 31) || K < 64 || K > CONVROT_MAX_K ||
        K % 64 || (bits != 8 && bits != 4))
        return 0;
    return ws_layout(M, N, K, bits).total;
}

} // extern "C"

namespace {

// Shared by convrot_linear, convrot_linear_act, convrot_linear_gated (caller's workspace) and
// convrot_linear_noalloc (the library's fixed scratch array).  scratch_fn, when given, is called
// only after every precondition holds and returns the scratch buffer (or sets the status), so a
// rejected call touches no device.
int linear_i8(const char *who, const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t M,
              int64_t N, int64_t K, int group, const int8_t *wq, const float *w_scale, const float *bias, void *y,
              void *workspace, size_t workspace_bytes, void *(*scratch_fn)(int *), hipStream_t stream,
              convrot::Epi epi = convrot::Epi::Bf16, const convrot::FusedEpi &f = convrot::FusedEpi())
{
    const bool gated = epi == convrot::Epi::Gated;
    int rc = check_shape(M, N, K, group, who);
    if (rc) return rc;
    if (M > 16 && (rc = check_gemm_n(N, who))) return rc;
    if ((rc = check_act(f.act, who))) return rc;
    if (M == 0 || N == 0) return CONVROT_OK;
    if (!wq || !w_scale || !y) return fail(CONVROT_ERR_NULL, "%s: wq, w_scale and y must be non-NULL", who);
    if (gated && (!f.wq2 || !f.sw2)) return fail(CONVROT_ERR_NULL, "%s: wq_up and up_scale must be non-NULL", who);
    if (!x && (!xq || !x_scale)) return fail(CONVROT_ERR_NULL, "%s: give x, or both xq and x_scale", who);
    if (x && x_dtype != CONVROT_DTYPE_F32 && x_dtype != CONVROT_DTYPE_BF16)
        return fail(CONVROT_ERR_DTYPE, "%s: x_dtype=%d", who, x_dtype);
    if ((x && !aligned(x, 16)) || (!x && (!aligned(xq, 16) || !aligned(x_scale, 4))) || !aligned(wq, 16) ||
        !aligned(w_scale, 4) || !aligned(y, 16) || (bias && !aligned(bias, 4)))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    if (!aligned(f.residual, 16) || !aligned(f.pre, 16) || !aligned(f.wq2, 16) || !aligned(f.sw2, 4) ||
        !aligned(f.bias2, 4))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t out_bytes = (size_t)M * (size_t)N * 2, pre_bytes = out_bytes * (gated ? 2 : 1);
    if ((f.residual != y && overlap(f.residual, out_bytes, y, out_bytes)) || overlap(f.pre, pre_bytes, y, out_bytes) ||
        overlap(f.pre, pre_bytes, f.residual, out_bytes))
        return fail(CONVROT_ERR_OVERLAP, "%s: an output overlaps pre or residual (only residual == y is allowed)", who);
    if (!x && epi != convrot::Epi::Bf16 &&
        (overlap(xq, (size_t)M * (size_t)K, y, out_bytes) || overlap(xq, (size_t)M * (size_t)K, f.pre, pre_bytes) ||
         overlap(x_scale, (size_t)M * 4, y, out_bytes) || overlap(x_scale, (size_t)M * 4, f.pre, pre_bytes)))
        return fail(CONVROT_ERR_OVERLAP, "%s: an output overlaps xq or x_scale", who);
    const WsLayout L = ws_layout(M, N, K, 8, epi);
    if (scratch_fn && x && workspace_bytes < L.part)
        return fail(CONVROT_ERR_WORKSPACE, "%s: M*K = %lld needs %zu bytes of scratch; the fixed scratch holds %zu "
                    "(use convrot_linear with a workspace)", who, (long long)(M * K), L.part, workspace_bytes);
    if (!scratch_fn && x && (!workspace || workspace_bytes < L.part || !aligned(workspace, 256)))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of at least %zu bytes (got %zu)",
                    who, L.part, workspace ? workspace_bytes : (size_t)0);
    if ((rc = check_device())) return rc;
    if (scratch_fn) {
        workspace = scratch_fn(&rc);
        if (rc) return rc;
    }

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    // room past the quantized x lets an under-filled GEMM split its tail tiles in K
    void *part = nullptr;
    size_t part_bytes = 0;
    if (M > 16 && ws && aligned(ws, 256) && L.total > L.part && workspace_bytes >= L.total) {
        part = ws + L.part;
        part_bytes = workspace_bytes - L.part;
    }
    if (x) {
        int8_t *qx = reinterpret_cast<int8_t *>(ws + L.xq);
        float *sx = reinterpret_cast<float *>(ws + L.xs);
        rc = hip_status(convrot::launch_rotate_quant(x, x_dtype == CONVROT_DTYPE_F32, M, (int)K, log2i(group), 8, qx,
                                                     sx, stream),
                        "rotate_quant");
        if (rc) return rc;
        xq = qx;
        x_scale = sx;
    }
    if (M <= 16)
        return hip_status(convrot::launch_gemv_i8(xq, wq, x_scale, w_scale, bias, y, epi, M, N, (int)K, stream, f),
                          "gemv_i8");
    if (epi != convrot::Epi::Bf16) {
        const convrot::TilePlan pl = convrot::plan_gemm_i8_tile(M, N, (int)K, gated, part || L.total == L.part);
        if (pl.bm)
            return hip_status(convrot::launch_gemm_i8_tile(pl, xq, wq, x_scale, w_scale, bias, y, epi, M, N, (int)K, part,
                                                           stream, f),
                              "gemm_i8_tile");
    }
    return hip_status(convrot::launch_gemm_i8(xq, wq, x_scale, w_scale, bias, y, epi, M, N, (int)K, part, part_bytes,
                                              stream, f),
                      "gemm_i8");
}

// Workspace of convrot_ffn_gated: the gated linear's, with h [M, F] bf16 and the down linear's
// after it (the two linears run in stream order, but the second quantizes h while the first's
// region is idle, so only h needs its own room: both layouts start at 0).
struct FfnLayout {
    size_t h = 0, total = 0;
};

FfnLayout ffn_layout(int64_t M, int64_t F, int64_t K)
{
    FfnLayout L;
    const size_t up = ws_layout(M, F, K, 8, convrot::Epi::Gated).total;
    const size_t down = ws_layout(M, K, F, 8, convrot::Epi::Act).total;
    L.h = up > down ? up : down;
    L.total = L.h + round256((size_t)M * (size_t)F * 2);
    return L;
}

// Shapes the backward calls take besides check_shape's rules: the tiles have to be countable in int.
bool grad_shape_ok(int64_t M, int64_t N, int64_t K)
{
    return M >= 0 && M < ((int64_t)1 << 31) && N >= 1 && N < CONVROT_BACKWARD_MAX_N && K >= 64 && K <= CONVROT_MAX_K &&
           K % 64 == 0 && ((M + 255) / 256) * ((K + 255) / 256) < ((int64_t)1 << 24);
}

int check_grad(const char *who, const convrot::GradArgs &g, int64_t K, int group, bool gated, const void *workspace,
               size_t workspace_bytes)
{
    int rc = check_shape(g.M, g.N, K, group, who);
    if (rc) return rc;
    if (!grad_shape_ok(g.M, g.N, K))
        return fail(CONVROT_ERR_SHAPE, "%s: M=%lld N=%lld K=%lld: the backward calls need 1 <= N < %d and at most 2^24 "
                    "tiles of 256 x 256", who, (long long)g.M, (long long)g.N, (long long)K, CONVROT_BACKWARD_MAX_N);
    if ((rc = check_act(g.act, who))) return rc;
    if (g.M == 0) {
        if (!aligned(g.db1, 4) || !aligned(g.db2, 4)) return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
        return CONVROT_OK;
    }
    const bool needs_pre = gated || g.act != CONVROT_ACT_NONE;
    if (!g.dy || !g.wq1 || !g.sw1 || !g.dx || (gated && (!g.wq2 || !g.sw2)) || (needs_pre && !g.pre))
        return fail(CONVROT_ERR_NULL, "%s: the gradient, the weights, their scales, dx and, with an activation, pre must "
                    "be non-NULL", who);
    if (!aligned(g.dy, 16) || !aligned(g.pre, 16) || !aligned(g.wq1, 16) || !aligned(g.wq2, 16) || !aligned(g.sw1, 4) ||
        !aligned(g.sw2, 4) || !aligned(g.add, 16) || !aligned(g.dx, 16) || !aligned(g.db1, 4) || !aligned(g.db2, 4))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t dx_bytes = (size_t)g.M * (size_t)K * 2, db_bytes = (size_t)g.N * 4;
    const size_t dy_bytes = (size_t)g.M * (size_t)g.N * 2, pre_bytes = dy_bytes * (gated ? 2 : 1);
    // with few tokens a bias gradient is written while other workgroups still read dy and pre
    auto shared = [&](const float *db) {
        return overlap(db, db_bytes, g.dx, dx_bytes) || overlap(db, db_bytes, g.add, dx_bytes) ||
               overlap(db, db_bytes, g.dy, dy_bytes) || overlap(db, db_bytes, g.pre, pre_bytes);
    };
    if ((g.add != g.dx && overlap(g.add, dx_bytes, g.dx, dx_bytes)) || shared(g.db1) || shared(g.db2) ||
        overlap(g.db1, db_bytes, g.db2, db_bytes))
        return fail(CONVROT_ERR_OVERLAP, "%s: dx overlaps dx_add (only dx_add == dx is allowed), or a bias gradient another "
                    "array of the call", who);
    const size_t need = convrot::grad_workspace_bytes(g.M, g.N, (int)K, gated);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of at least %zu bytes (got %zu)", who,
                    need, workspace ? workspace_bytes : (size_t)0);
    return CONVROT_OK;
}

int grad_i8(const char *who, convrot::GradArgs g, int64_t K, int group, bool gated, void *workspace,
            size_t workspace_bytes, hipStream_t stream)
{
    int rc = check_grad(who, g, K, group, gated, workspace, workspace_bytes);
    if (rc) return rc;
    if (g.M == 0 && !g.db1 && !g.db2) return CONVROT_OK;
    if ((rc = check_device())) return rc;
    g.K = (int)K;
    g.log2g = log2i(group);
    g.ws = workspace;
    return hip_status(convrot::launch_grad_i8(g, gated, stream), "grad_i8");
}

// Workspace of convrot_ffn_gated_backward.  Without gate and up bias gradients the first step's epilogue
// writes the second step's operand [M, 2 F] bf16; with them (fp32 column sums over the tokens) dh [M, F]
// bf16 goes through the second step's own first pass.  Both: the larger of the two steps' own
// workspaces, then that buffer.
struct FfnGradLayout {
    size_t steps = 0, steps_dh = 0, total = 0;
};

FfnGradLayout ffn_grad_layout(int64_t M, int64_t F, int64_t K)
{
    FfnGradLayout L;
    const size_t down = convrot::grad_workspace_bytes(M, K, (int)F, false);
    const size_t up = convrot::grad_workspace_bytes(M, F, (int)K, true, true);
    const size_t up_dh = convrot::grad_workspace_bytes(M, F, (int)K, true);
    L.steps = round256(up > down ? up : down);
    L.steps_dh = round256(up_dh > down ? up_dh : down);
    const size_t with_a = L.steps + round256((size_t)M * (size_t)F * 4);
    const size_t with_dh = L.steps_dh + round256((size_t)M * (size_t)F * 2);
    L.total = with_a > with_dh ? with_a : with_dh;
    return L;
}

// Scratch of convrot_linear_noalloc: one fixed array per GPU, held until the process ends.  On
// the host the array's name is only a stand-in for its device address: the address each device
// holds is looked up once per device (with that device current) and kept in scratch_ptr.
static __device__ __align__(256) uint8_t scratch[CONVROT_NOALLOC_SCRATCH_BYTES];

constexpr int MAX_DEVICES = 64;

void *scratch_for_current_device(int *rc)
{
    static std::mutex mu;
    static void *scratch_ptr[MAX_DEVICES];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) {
        *rc = fail(CONVROT_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
        return nullptr;
    }
    if (dev < 0 || dev >= MAX_DEVICES) {
        *rc = fail(CONVROT_ERR_DEVICE, "device index %d out of range", dev);
        return nullptr;
    }
    std::lock_guard<std::mutex> lk(mu);
    if (!scratch_ptr[dev]) {
        void *ptr = nullptr;
        e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !ptr) {
            *rc = fail(CONVROT_ERR_HIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev, hipGetErrorString(e));
            return nullptr;
        }
        scratch_ptr[dev] = ptr;
    }
    *rc = CONVROT_OK;
    return scratch_ptr[dev];
}

} // namespace

extern "C" {

int convrot_linear(const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t M, int64_t N,
                   int64_t K, int group, const int8_t *wq, const float *w_scale, const float *bias, void *y,
                   void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return linear_i8("convrot_linear", x, x_dtype, xq, x_scale, M, N, K, group, wq, w_scale, bias, y, workspace,
                     workspace_bytes, nullptr, stream);
}

int convrot_linear_noalloc(const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t M, int64_t N,
                           int64_t K, int group, const int8_t *wq, const float *w_scale, const float *bias, void *y,
                           hipStream_t stream)
{
    return linear_i8("convrot_linear_noalloc", x, x_dtype, xq, x_scale, M, N, K, group, wq, w_scale, bias, y, nullptr,
                     CONVROT_NOALLOC_SCRATCH_BYTES, scratch_for_current_device, stream);
}

int convrot_linear_act(const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t M, int64_t N,
                       int64_t K, int group, const int8_t *wq, const float *w_scale, const float *bias, int act,
                       const void *residual, void *pre, void *y, void *workspace, size_t workspace_bytes,
                       hipStream_t stream)
{
    convrot::FusedEpi f;
    f.act = act;
    f.residual = static_cast<const uint16_t *>(residual);
    f.pre = static_cast<uint16_t *>(pre);
    return linear_i8("convrot_linear_act", x, x_dtype, xq, x_scale, M, N, K, group, wq, w_scale, bias, y, workspace,
                     workspace_bytes, nullptr, stream, convrot::Epi::Act, f);
}

size_t convrot_workspace_bytes_act(int64_t M, int64_t N, int64_t K)
{
    return convrot_workspace_bytes(M, N, K, 8) ? ws_layout(M, N, K, 8, convrot::Epi::Act).total : 0;
}

size_t convrot_workspace_bytes_gated(int64_t M, int64_t N, int64_t K)
{
    return convrot_workspace_bytes(M, N, K, 8) ? ws_layout(M, N, K, 8, convrot::Epi::Gated).total : 0;
}

int convrot_linear_gated(const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t M, int64_t N,
                         int64_t K, int group, const int8_t *wq_gate, const float *gate_scale, const float *gate_bias,
                         const int8_t *wq_up, const float *up_scale, const float *up_bias, int act, void *pre, void *h,
                         void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    convrot::FusedEpi f;
    f.act = act;
    f.pre = static_cast<uint16_t *>(pre);
    f.wq2 = wq_up;
    f.sw2 = up_scale;
    f.bias2 = up_bias;
    return linear_i8("convrot_linear_gated", x, x_dtype, xq, x_scale, M, N, K, group, wq_gate, gate_scale, gate_bias, h,
                     workspace, workspace_bytes, nullptr, stream, convrot::Epi::Gated, f);
}

size_t convrot_workspace_bytes_ffn(int64_t M, int64_t F, int64_t K)
{
    if (!convrot_workspace_bytes(M, F, K, 8) || !convrot_workspace_bytes(M, K, F, 8)) return 0;
    return ffn_layout(M, F, K).total;
}

int convrot_ffn_gated(const void *x, int x_dtype, int64_t M, int64_t F, int64_t K, int group, int group_h,
                      const int8_t *wq_gate, const float *gate_scale, const float *gate_bias, const int8_t *wq_up,
                      const float *up_scale, const float *up_bias, const int8_t *wq_down, const float *down_scale,
                      const float *down_bias, int act, const void *residual, void *pre, void *y, void *workspace,
                      size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_ffn_gated";
    // everything the two linears would reject, before the first of them enqueues anything
    int rc = check_shape(M, F, K, group, who);
    if (rc) return rc;
    if ((rc = check_shape(M, K, F, group_h, who))) return rc;
    if ((rc = check_act(act, who))) return rc;
    if (M == 0) return CONVROT_OK;
    if (!x || !wq_gate || !gate_scale || !wq_up || !up_scale || !wq_down || !down_scale || !y)
        return fail(CONVROT_ERR_NULL, "%s: x, the weights, their scales and y must be non-NULL", who);
    if (x_dtype != CONVROT_DTYPE_F32 && x_dtype != CONVROT_DTYPE_BF16)
        return fail(CONVROT_ERR_DTYPE, "%s: x_dtype=%d", who, x_dtype);
    if (!aligned(x, 16) || !aligned(wq_gate, 16) || !aligned(wq_up, 16) || !aligned(wq_down, 16) || !aligned(y, 16) ||
        !aligned(pre, 16) || !aligned(residual, 16) || !aligned(gate_scale, 4) || !aligned(up_scale, 4) ||
        !aligned(down_scale, 4) || !aligned(gate_bias, 4) || !aligned(up_bias, 4) || !aligned(down_bias, 4))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t y_bytes = (size_t)M * (size_t)K * 2, pre_bytes = (size_t)M * (size_t)F * 4;
    const size_t x_bytes = (size_t)M * (size_t)K * (x_dtype == CONVROT_DTYPE_F32 ? 4 : 2);
    // pre and h are written before the residual is read
    if ((residual != y && overlap(residual, y_bytes, y, y_bytes)) || overlap(pre, pre_bytes, y, y_bytes) ||
        overlap(pre, pre_bytes, residual, y_bytes) || overlap(pre, pre_bytes, x, x_bytes))
        return fail(CONVROT_ERR_OVERLAP, "%s: an output overlaps pre, x or residual (only residual == y is allowed)", who);
    const FfnLayout L = ffn_layout(M, F, K);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of at least %zu bytes (got %zu)", who,
                    L.total, workspace ? workspace_bytes : (size_t)0);
    if ((rc = check_device())) return rc;
    void *h = static_cast<uint8_t *>(workspace) + L.h;
    rc = convrot_linear_gated(x, x_dtype, nullptr, nullptr, M, F, K, group, wq_gate, gate_scale, gate_bias, wq_up,
                              up_scale, up_bias, act, pre, h, workspace, L.h, stream);
    if (rc) return rc;
    return convrot_linear_act(h, CONVROT_DTYPE_BF16, nullptr, nullptr, M, K, F, group_h, wq_down, down_scale, down_bias,
                              CONVROT_ACT_NONE, residual, nullptr, y, workspace, L.h, stream);
}

size_t convrot_workspace_bytes_backward(int64_t M, int64_t N, int64_t K)
{
    return grad_shape_ok(M, N, K) ? convrot::grad_workspace_bytes(M, N, (int)K, false) : 0;
}

size_t convrot_workspace_bytes_gated_backward(int64_t M, int64_t N, int64_t K)
{
    return grad_shape_ok(M, N, K) ? convrot::grad_workspace_bytes(M, N, (int)K, true) : 0;
}

size_t convrot_workspace_bytes_ffn_backward(int64_t M, int64_t F, int64_t K)
{
    return grad_shape_ok(M, F, K) && grad_shape_ok(M, K, F) ? ffn_grad_layout(M, F, K).total : 0;
}

int convrot_linear_act_backward(const void *dy, const void *pre, int64_t M, int64_t N, int64_t K, int group,
                                const int8_t *wq, const float *w_scale, int act, const void *dx_add, void *dx,
                                float *dbias, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    convrot::GradArgs g;
    g.dy = static_cast<const uint16_t *>(dy);
    g.pre = act == CONVROT_ACT_NONE ? nullptr : static_cast<const uint16_t *>(pre);
    g.M = M;
    g.N = N;
    g.act = act;
    g.wq1 = wq;
    g.sw1 = w_scale;
    g.add = static_cast<const uint16_t *>(dx_add);
    g.dx = static_cast<uint16_t *>(dx);
    g.db1 = dbias;
    return grad_i8("convrot_linear_act_backward", g, K, group, false, workspace, workspace_bytes, stream);
}

int convrot_linear_gated_backward(const void *dh, const void *pre, int64_t M, int64_t N, int64_t K, int group,
                                  const int8_t *wq_gate, const float *gate_scale, const int8_t *wq_up,
                                  const float *up_scale, int act, const void *dx_add, void *dx, float *dgate_bias,
                                  float *dup_bias, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    convrot::GradArgs g;
    g.dy = static_cast<const uint16_t *>(dh);
    g.pre = static_cast<const uint16_t *>(pre);
    g.M = M;
    g.N = N;
    g.act = act;
    g.wq1 = wq_gate;
    g.sw1 = gate_scale;
    g.wq2 = wq_up;
    g.sw2 = up_scale;
    g.add = static_cast<const uint16_t *>(dx_add);
    g.dx = static_cast<uint16_t *>(dx);
    g.db1 = dgate_bias;
    g.db2 = dup_bias;
    return grad_i8("convrot_linear_gated_backward", g, K, group, true, workspace, workspace_bytes, stream);
}

int convrot_ffn_gated_backward(const void *dy, const void *pre, int64_t M, int64_t F, int64_t K, int group, int group_h,
                               const int8_t *wq_gate, const float *gate_scale, const int8_t *wq_up,
                               const float *up_scale, const int8_t *wq_down, const float *down_scale, int act,
                               const void *dx_add, void *dx, float *dgate_bias, float *dup_bias, float *ddown_bias,
                               void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_ffn_gated_backward";
    int rc = check_shape(M, F, K, group, who);
    if (rc) return rc;
    if ((rc = check_shape(M, K, F, group_h, who))) return rc;
    // the second call's checks first, on everything but dh, which is the library's own
    convrot::GradArgs down, up;
    const FfnGradLayout L = grad_shape_ok(M, F, K) && grad_shape_ok(M, K, F) ? ffn_grad_layout(M, F, K) : FfnGradLayout();
    if (M > 0 && (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of at least %zu bytes (got %zu)", who,
                    L.total, workspace ? workspace_bytes : (size_t)0);
    const bool sums = dgate_bias || dup_bias;
    const size_t steps = sums ? L.steps_dh : L.steps;
    uint16_t *dh = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(workspace) + steps);
    down.dy = static_cast<const uint16_t *>(dy);
    down.M = up.M = M;
    down.N = K;
    down.act = CONVROT_ACT_NONE;
    down.wq1 = wq_down;
    down.sw1 = down_scale;
    down.dx = dh;
    down.db1 = ddown_bias;
    up.dy = dh;
    up.pre = static_cast<const uint16_t *>(pre);
    up.N = F;
    up.act = act;
    up.wq1 = wq_gate;
    up.sw1 = gate_scale;
    up.wq2 = wq_up;
    up.sw2 = up_scale;
    up.add = static_cast<const uint16_t *>(dx_add);
    up.dx = static_cast<uint16_t *>(dx);
    up.db1 = dgate_bias;
    up.db2 = dup_bias;
    if ((rc = check_grad(who, up, K, group, true, workspace, L.steps_dh))) return rc;
    if ((rc = check_grad(who, down, F, group_h, false, workspace, L.steps_dh))) return rc;
    const size_t dx_bytes = (size_t)M * (size_t)K * 2;
    // what the two steps' own checks do not see: each step knows its own bias gradients only, and dy is the first's
    if (overlap(ddown_bias, (size_t)K * 4, dx, dx_bytes) || overlap(ddown_bias, (size_t)K * 4, dx_add, dx_bytes) ||
        overlap(ddown_bias, (size_t)K * 4, dgate_bias, (size_t)F * 4) ||
        overlap(ddown_bias, (size_t)K * 4, dup_bias, (size_t)F * 4) ||
        overlap(ddown_bias, (size_t)K * 4, pre, (size_t)M * (size_t)F * 4) ||
        overlap(dgate_bias, (size_t)F * 4, dy, dx_bytes) || overlap(dup_bias, (size_t)F * 4, dy, dx_bytes))
        return fail(CONVROT_ERR_OVERLAP, "%s: a bias gradient overlaps another array of the call", who);
    if (!sums) {
        down.next.pre = up.pre;
        down.next.sw_gate = gate_scale;
        down.next.sw_up = up_scale;
        down.next.act = act;
        down.next.a = dh;
        up.a = dh;
    }
    if ((rc = grad_i8(who, down, F, group_h, false, workspace, L.steps_dh, stream))) return rc;
    return grad_i8(who, up, K, group, true, workspace, L.steps_dh, stream);
}

int convrot_gemm_i8_i32(const int8_t *xq, const int8_t *wq, int64_t M, int64_t N, int64_t K, int32_t *acc,
                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_gemm_i8_i32";
    int rc = check_shape(M, N, K, 1, who);
    if (rc) return rc;
    if (M > 16 && (rc = check_gemm_n(N, who))) return rc;
    if (M == 0 || N == 0) return CONVROT_OK;
    if (!xq || !wq || !acc) return fail(CONVROT_ERR_NULL, "%s: xq, wq and acc must be non-NULL", who);
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(acc, 16)) return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    (void)workspace;
    (void)workspace_bytes;
    if ((rc = check_device())) return rc;
    if (M <= 16) {
        return hip_status(convrot::launch_gemv_i8(xq, wq, nullptr, nullptr, nullptr, acc, convrot::Epi::Int32, M, N,
                                                  (int)K, stream),
                          "gemv_i8");
    }
    return hip_status(
        convrot::launch_gemm_i8(xq, wq, nullptr, nullptr, nullptr, acc, convrot::Epi::Int32, M, N, (int)K, nullptr, 0,
                                stream),
        "gemm_i8");
}

} // extern "C"

namespace {

// Shared by convrot_linear_w4a4 (packed INT4 weights, re-encoded on every call) and
// convrot_linear_w4a4_packed (weights re-encoded once by convrot_pack_weight_w4a4).
int linear_w4a4(const char *who, const void *x, int x_dtype, const uint8_t *xq, const uint16_t *x_scale, int64_t M,
                int64_t N, int64_t K, int group, const uint8_t *w, bool w_tiled, const uint16_t *w_scale,
                const float *bias, void *y, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    int rc = check_shape(M, N, K, group, who);
    if (rc) return rc;
    if ((rc = check_gemm_n(N, who))) return rc;
    if ((group != 256 && group != 128) || K % group)
        return fail(CONVROT_ERR_GROUP, "%s: W4A4 needs group 256 or 128 dividing K (group=%d, K=%lld)", who, group,
                    (long long)K);
    if (K < 256) return fail(CONVROT_ERR_SHAPE, "%s: K=%lld; W4A4 needs K >= 256", who, (long long)K);
    if (N % 8) return fail(CONVROT_ERR_SHAPE, "%s: N=%lld must be a multiple of 8", who, (long long)N);
    if (M == 0 || N == 0) return CONVROT_OK;
    if (!w || !w_scale || !y) return fail(CONVROT_ERR_NULL, "%s: the weights, w_scale and y must be non-NULL", who);
    if (!x && (!xq || !x_scale)) return fail(CONVROT_ERR_NULL, "%s: give x, or both xq and x_scale", who);
    if (x && x_dtype != CONVROT_DTYPE_F32 && x_dtype != CONVROT_DTYPE_BF16)
        return fail(CONVROT_ERR_DTYPE, "%s: x_dtype=%d", who, x_dtype);
    if ((x && !aligned(x, 16)) || (!x && (!aligned(xq, 16) || !aligned(x_scale, 2))) || !aligned(w, 16) ||
        !aligned(w_scale, 8) || !aligned(y, 16) || (bias && !aligned(bias, 4)))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer (w_scale needs 8 bytes)", who);
    const WsLayout L = ws_layout(M, w_tiled ? 0 : N, K, 4);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of %zu bytes", who, L.total);
    if ((rc = check_device())) return rc;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (x) {
        // rotate + quantize straight into the GEMM's FP6 token tiles (no packed INT4 copy)
        rc = hip_status(convrot::launch_rotate_quant_fp6(x, x_dtype == CONVROT_DTYPE_F32, M, (int)K, log2i(group),
                                                         ws + L.tiles, ws + L.xs, stream),
                        "rotate_quant_fp6");
        if (rc) return rc;
        xq = ws + L.tiles;
        x_scale = reinterpret_cast<const uint16_t *>(ws + L.xs);
    }
    return hip_status(convrot::launch_gemm_w4a4(xq, x != nullptr, w, w_tiled, x_scale, w_scale, bias, y,
                                                convrot::Epi::Bf16, M, N, (int)K, group, ws + L.tiles, stream),
                      "gemm_w4a4");
}

} // namespace

extern "C" {

int convrot_linear_w4a4(const void *x, int x_dtype, const uint8_t *xq, const uint16_t *x_scale, int64_t M,
                        int64_t N, int64_t K, int group, const uint8_t *wq, const uint16_t *w_scale,
                        const float *bias, void *y, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return linear_w4a4("convrot_linear_w4a4", x, x_dtype, xq, x_scale, M, N, K, group, wq, false, w_scale, bias, y,
                       workspace, workspace_bytes, stream);
}

size_t convrot_packed_bytes_w4a4(int64_t N, int64_t K)
{
    if (N < 0 || N >= ((int64_t)1 << 31) || K <= 0 || K % 128 || K > CONVROT_MAX_K) return 0;
    return convrot::w4a4_tiled_bytes(0, N, (int)K);
}

int convrot_pack_weight_w4a4(const uint8_t *wq, int64_t N, int64_t K, void *w_packed, hipStream_t stream)
{
    const char *who = "convrot_pack_weight_w4a4";
    int rc = check_shape(N, 1, K, 128, who);
    if (rc) return rc;
    if (K % 128) return fail(CONVROT_ERR_GROUP, "%s: K=%lld must be a multiple of 128", who, (long long)K);
    if (N == 0) return CONVROT_OK;
    if (!wq || !w_packed) return fail(CONVROT_ERR_NULL, "%s: wq and w_packed must be non-NULL", who);
    if (!aligned(wq, 16) || !aligned(w_packed, 16)) return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    if ((rc = check_device())) return rc;
    return hip_status(convrot::launch_tile_w4a4(wq, N, (int)K, static_cast<uint8_t *>(w_packed), stream), "tile_w4a4");
}

int convrot_linear_w4a4_packed(const void *x, int x_dtype, const uint8_t *xq, const uint16_t *x_scale, int64_t M,
                               int64_t N, int64_t K, int group, const void *w_packed, const uint16_t *w_scale,
                               const float *bias, void *y, void *workspace, size_t workspace_bytes,
                               hipStream_t stream)
{
    return linear_w4a4("convrot_linear_w4a4_packed", x, x_dtype, xq, x_scale, M, N, K, group,
                       static_cast<const uint8_t *>(w_packed), true, w_scale, bias, y, workspace, workspace_bytes,
                       stream);
}

size_t convrot_workspace_bytes_w4a8(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || M > CONVROT_W4A8_MAX_M || N < 0 || K <= 0 || K % 128 || K > CONVROT_MAX_K) return 0;
    return ws_layout_w4a8(M, K).total;
}

size_t convrot_packed_bytes_w4a8_group(int64_t N, int64_t K, int group)
{
    if (N < 0 || N >= ((int64_t)1 << 31) || K <= 0 || K > CONVROT_MAX_K || (group != 256 && group != 128) ||
        K % group)
        return 0;
    return convrot::w4a8_packed_bytes(N, (int)K, group);
}

size_t convrot_packed_bytes_w4a8(int64_t N, int64_t K) { return convrot_packed_bytes_w4a8_group(N, K, 256); }

} // extern "C"

namespace {

int pack_w4a8(const char *who, const uint8_t *wq, const uint16_t *w_scale, int64_t N, int64_t K, int group,
              void *w_packed, hipStream_t stream)
{
    int rc = check_shape(N, 1, K, group, who);
    if (rc) return rc;
    if ((group != 256 && group != 128) || K % group)
        return fail(CONVROT_ERR_GROUP, "%s: W4A8 needs group 256 or 128 dividing K (group=%d, K=%lld)", who, group,
                    (long long)K);
    if (N == 0) return CONVROT_OK;
    if (!wq || !w_scale || !w_packed) return fail(CONVROT_ERR_NULL, "%s: wq, w_scale and w_packed must be non-NULL", who);
    if (!aligned(wq, 16) || !aligned(w_scale, 2) || !aligned(w_packed, 16))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    if ((rc = check_device())) return rc;
    return hip_status(
        convrot::launch_pack_w4a8(wq, w_scale, N, (int)K, group, static_cast<uint8_t *>(w_packed), stream),
        "pack_w4a8");
}

} // namespace

extern "C" {

int convrot_pack_weight_w4a8(const uint8_t *wq, const uint16_t *w_scale, int64_t N, int64_t K, void *w_packed,
                             hipStream_t stream)
{
    return pack_w4a8("convrot_pack_weight_w4a8", wq, w_scale, N, K, 256, w_packed, stream);
}

int convrot_pack_weight_w4a8_group(const uint8_t *wq, const uint16_t *w_scale, int64_t N, int64_t K, int group,
                                   void *w_packed, hipStream_t stream)
{
    return pack_w4a8("convrot_pack_weight_w4a8_group", wq, w_scale, N, K, group, w_packed, stream);
}

int convrot_linear_w4a8(const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t M, int64_t N,
                        int64_t K, int group, const void *w_packed, size_t w_packed_bytes, const float *bias, void *y,
                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_linear_w4a8";
    int rc = check_shape(M, N, K, group, who);
    if (rc) return rc;
    if ((group != 256 && group != 128) || K % group)
        return fail(CONVROT_ERR_GROUP, "%s: W4A8 needs group 256 or 128 dividing K (group=%d, K=%lld); the weights "
                    "must be packed with the same group", who, group, (long long)K);
    if (M > CONVROT_W4A8_MAX_M)
        return fail(CONVROT_ERR_SHAPE, "%s: M=%lld tokens; the W4A8 kernel is the decode path (M <= %d)", who,
                    (long long)M, CONVROT_W4A8_MAX_M);
    if (N % 8) return fail(CONVROT_ERR_SHAPE, "%s: N=%lld must be a multiple of 8", who, (long long)N);
    if (M == 0 || N == 0) return CONVROT_OK;
    if (!w_packed || !y) return fail(CONVROT_ERR_NULL, "%s: w_packed and y must be non-NULL", who);
    // the packed size depends on the group (8320 or 8448 bytes per 64 x 256 block): a buffer packed
    // with the other group has another size, and would be read past its end or misread
    const size_t need = convrot_packed_bytes_w4a8_group(N, K, group);
    if (w_packed_bytes != need)
        return fail(CONVROT_ERR_SHAPE, "%s: w_packed_bytes=%zu, but weights packed for N=%lld K=%lld group=%d take %zu "
                    "bytes (were they packed with the other group?)", who, w_packed_bytes, (long long)N, (long long)K,
                    group, need);
    if (!x && (!xq || !x_scale)) return fail(CONVROT_ERR_NULL, "%s: give x, or both xq and x_scale", who);
    if (x && x_dtype != CONVROT_DTYPE_F32 && x_dtype != CONVROT_DTYPE_BF16)
        return fail(CONVROT_ERR_DTYPE, "%s: x_dtype=%d", who, x_dtype);
    if ((x && !aligned(x, 16)) || (!x && (!aligned(xq, 16) || !aligned(x_scale, 4))) || !aligned(w_packed, 16) ||
        !aligned(y, 16) || (bias && !aligned(bias, 4)))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const WsLayout L = ws_layout_w4a8(M, K);
    if (x && (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of %zu bytes (got %zu)", who, L.total,
                    workspace ? workspace_bytes : (size_t)0);
    if ((rc = check_device())) return rc;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (x) {
        int8_t *qx = reinterpret_cast<int8_t *>(ws + L.xq);
        float *sx = reinterpret_cast<float *>(ws + L.xs);
        rc = hip_status(convrot::launch_rotate_quant(x, x_dtype == CONVROT_DTYPE_F32, M, (int)K, log2i(group), 8, qx, sx, stream),
                        "rotate_quant");
        if (rc) return rc;
        xq = qx;
        x_scale = sx;
    }
    return hip_status(convrot::launch_gemv_w4a8(xq, x_scale, static_cast<const uint8_t *>(w_packed), bias, y, M, N,
                                                (int)K, group, stream),
                      "gemv_w4a8");
}

int convrot_gemm_i4_i32(const uint8_t *xq, const uint8_t *wq, int64_t M, int64_t N, int64_t K, int32_t *acc,
                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_gemm_i4_i32";
    int rc = check_shape(M, N, K, 256, who);
    if (rc) return rc;
    if ((rc = check_gemm_n(N, who))) return rc;
    if (K % 256 || N % 8) return fail(CONVROT_ERR_SHAPE, "%s: needs K %% 256 == 0 and N %% 8 == 0", who);
    if (M == 0 || N == 0) return CONVROT_OK;
    if (!xq || !wq || !acc) return fail(CONVROT_ERR_NULL, "%s: xq, wq and acc must be non-NULL", who);
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(acc, 16)) return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const WsLayout L = ws_layout(M, N, K, 4);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of %zu bytes", who, L.total);
    if ((rc = check_device())) return rc;
    return hip_status(convrot::launch_gemm_w4a4(xq, false, wq, false, nullptr, nullptr, nullptr, acc, convrot::Epi::Int32, M, N,
                                                (int)K, 256, static_cast<uint8_t *>(workspace) + L.tiles, stream),
                      "gemm_w4a4");
}

} // extern "C"

// ---------------------------------------------------------------------------------------------
// Mixture of experts
namespace {

int check_route(const char *who, int dtype, int64_t M, int64_t E, int top, int score)
{
    if (M < 0 || M >= CONVROT_GROUPED_MAX_ROWS || E < 1 || E > CONVROT_MAX_GROUPS || top < 1 || top > E ||
        top > CONVROT_MOE_MAX_TOP || M * top >= CONVROT_GROUPED_MAX_ROWS)
        return fail(CONVROT_ERR_SHAPE, "%s: M=%lld E=%lld top=%d: E must be in [1, %d], top in [1, min(E, %d)], M * top in "
                    "[0, %d)", who, (long long)M, (long long)E, top, CONVROT_MAX_GROUPS, CONVROT_MOE_MAX_TOP,
                    CONVROT_GROUPED_MAX_ROWS);
    if (dtype != CONVROT_DTYPE_F32 && dtype != CONVROT_DTYPE_BF16) return fail(CONVROT_ERR_DTYPE, "%s: dtype=%d", who, dtype);
    if (score != CONVROT_SCORE_SOFTMAX && score != CONVROT_SCORE_SIGMOID)
        return fail(CONVROT_ERR_SCORE, "%s: score=%d is not one of CONVROT_SCORE_*", who, score);
    return CONVROT_OK;
}

convrot::RouteArgs route_args(const void *logits, int dtype, const float *bias, int64_t M, int64_t E, int top, int score,
                              int normalize, float scale)
{
    convrot::RouteArgs a;
    a.logits = logits;
    a.f32 = dtype == CONVROT_DTYPE_F32;
    a.bias = bias;
    a.M = M;
    a.E = (int)E;
    a.top = top;
    a.score = score;
    a.normalize = normalize != 0;
    a.scale = scale;
    return a;
}

// Rows sorted by group: the rules of check_shape, the limits of the group table, units (of 64 rows and, forward, 64
// features) that int can count, and, backward, tiles (of at least 64 rows x 256 channels, 256 threads) that one launch can hold.
bool grouped_shape_ok(int64_t rows, int64_t groups, int64_t N, int64_t K, bool backward)
{
    if (rows < 0 || rows >= CONVROT_GROUPED_MAX_ROWS || groups < 1 || groups > CONVROT_MAX_GROUPS || N < 1 ||
        N >= (backward ? CONVROT_BACKWARD_MAX_N : CONVROT_GEMM_MAX_N) || K < 64 || K > CONVROT_MAX_K || K % 64)
        return false;
    if (backward && (rows / 64 + groups) * ((K + 255) / 256) > ((int64_t)1 << 24) - 8) return false;
    return (rows / 64 + groups) * (((backward ? K : N) + 63) / 64) < ((int64_t)1 << 30);
}

int check_grouped(const char *who, int64_t rows, int64_t groups, int64_t N, int64_t K, int group, bool backward)
{
    int rc = check_shape(0, N, K, group, who);
    if (rc) return rc;
    if (!grouped_shape_ok(rows, groups, N, K, backward))
        return fail(CONVROT_ERR_SHAPE, "%s: rows=%lld groups=%lld N=%lld: rows must be in [0, %d), groups in [1, %d], N in "
                    "[1, %d), and the tiles fewer than 2^30 (backward, of 64 rows by 256 channels, than 2^24)", who,
                    (long long)rows, (long long)groups, (long long)N, CONVROT_GROUPED_MAX_ROWS, CONVROT_MAX_GROUPS,
                    backward ? CONVROT_BACKWARD_MAX_N : CONVROT_GEMM_MAX_N);
    return CONVROT_OK;
}

// [xq int8 rows*K][x_scale fp32 rows]
size_t grouped_bytes(int64_t rows, int64_t K) { return round256((size_t)rows * (size_t)K) + round256((size_t)rows * 4); }

size_t grouped_backward_bytes(int64_t rows, int64_t N)
{
    return round256((size_t)rows * (size_t)convrot::grouped_grad_lda(N) * 2);
}

int check_workspace(const char *who, const void *workspace, size_t bytes, size_t need)
{
    if (!workspace || bytes < need || !aligned(workspace, 256))
        return fail(CONVROT_ERR_WORKSPACE, "%s: need a 256-byte aligned workspace of at least %zu bytes (got %zu)", who, need,
                    workspace ? bytes : (size_t)0);
    return CONVROT_OK;
}

// The expert layer's workspace: the sort's arrays, then, forward, the codes and scales of x, each row's scale, h, its codes and
// scales, and d; backward, the two contractions' operands, and dx's parts over the first.  (d and the parts in fp32.)
struct MoeLayout {
    size_t offsets = 0, slot_of = 0, token_of = 0, row_of = 0;
    size_t xq = 0, xs = 0, rs = 0, h = 0, hq = 0, hs = 0;
    size_t a = 0, a2 = 0;
    size_t part = 0, total = 0;
};

MoeLayout moe_layout(int64_t M, int top, int64_t E, int64_t F, int64_t K, bool backward)
{
    MoeLayout L;
    const size_t S = (size_t)M * (size_t)top;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round256(bytes);
        return at;
    };
    L.offsets = take((size_t)(E + 1) * 4);
    L.slot_of = take(S * 4);
    L.token_of = take(S * 4);
    L.row_of = take(S * 4);
    if (backward) {
        L.a2 = take(S * (size_t)F * 4);
        L.a = L.part = take(S * (size_t)K * 4);
    } else {
        L.xq = take((size_t)M * (size_t)K);
        L.xs = take((size_t)M * 4);
        L.rs = take(S * 4);
        L.h = take(S * (size_t)F * 2);
        L.hq = take(S * (size_t)F);
        L.hs = take(S * 4);
        L.part = take(S * (size_t)K * 4);
    }
    L.total = off;
    return L;
}

bool moe_shape_ok(int64_t M, int top, int64_t E, int64_t F, int64_t K, bool backward)
{
    if (M < 0 || M >= CONVROT_GROUPED_MAX_ROWS || E < 1 || E > CONVROT_MAX_GROUPS || top < 1 || top > E ||
        top > CONVROT_MOE_MAX_TOP)
        return false;
    return grouped_shape_ok(M * top, E, F, K, backward) && grouped_shape_ok(M * top, E, K, F, backward) &&
           M * K < ((int64_t)1 << 31);
}

int check_moe(const char *who, int64_t M, int top, int64_t E, int64_t F, int64_t K, int group, int group_h, int act,
              bool backward)
{
    int rc = check_shape(M, F, K, group, who);
    if (rc) return rc;
    if ((rc = check_shape(M, K, F, group_h, who))) return rc;
    if ((rc = check_act(act, who))) return rc;
    if (!moe_shape_ok(M, top, E, F, K, backward))
        return fail(CONVROT_ERR_SHAPE, "%s: M=%lld top=%d E=%lld F=%lld K=%lld: E must be in [1, %d], top in [1, min(E, %d)], "
                    "M * top below %d, M * K below 2^31", who, (long long)M, top, (long long)E, (long long)F, (long long)K,
                    CONVROT_MAX_GROUPS, CONVROT_MOE_MAX_TOP, CONVROT_GROUPED_MAX_ROWS);
    return CONVROT_OK;
}

convrot::MoeOrder moe_order(uint8_t *ws, const MoeLayout &L)
{
    convrot::MoeOrder o;
    o.offsets = reinterpret_cast<int32_t *>(ws + L.offsets);
    o.slot_of = reinterpret_cast<int32_t *>(ws + L.slot_of);
    o.token_of = reinterpret_cast<int32_t *>(ws + L.token_of);
    o.row_of = reinterpret_cast<int32_t *>(ws + L.row_of);
    return o;
}

} // namespace

extern "C" {

int convrot_moe_route(const void *logits, int dtype, int64_t M, int64_t E, int top, int score, int normalize,
                      float scale, const float *bias, int32_t *experts, float *weights, hipStream_t stream)
{
    const char *who = "convrot_moe_route";
    int rc = check_route(who, dtype, M, E, top, score);
    if (rc) return rc;
    if (M == 0) return CONVROT_OK;
    if (!logits || !experts || !weights) return fail(CONVROT_ERR_NULL, "%s: logits, experts and weights must be non-NULL", who);
    if (!aligned(logits, dtype == CONVROT_DTYPE_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(experts, 4) || !aligned(weights, 4))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t out = (size_t)M * (size_t)top * 4, in = (size_t)M * (size_t)E * (dtype == CONVROT_DTYPE_F32 ? 4 : 2);
    if (overlap(experts, out, weights, out) || overlap(experts, out, logits, in) || overlap(weights, out, logits, in) ||
        overlap(experts, out, bias, (size_t)E * 4) || overlap(weights, out, bias, (size_t)E * 4))
        return fail(CONVROT_ERR_OVERLAP, "%s: an output overlaps another array of the call", who);
    if ((rc = check_device())) return rc;
    return hip_status(convrot::launch_moe_route(route_args(logits, dtype, bias, M, E, top, score, normalize, scale), experts,
                                                weights, stream),
                      "moe_route");
}

int convrot_moe_route_backward(const float *dweights, const void *logits, int dtype, int64_t M, int64_t E, int top,
                               int score, int normalize, float scale, const int32_t *experts, void *dlogits,
                               hipStream_t stream)
{
    const char *who = "convrot_moe_route_backward";
    int rc = check_route(who, dtype, M, E, top, score);
    if (rc) return rc;
    if (M == 0) return CONVROT_OK;
    if (!dweights || !logits || !experts || !dlogits)
        return fail(CONVROT_ERR_NULL, "%s: dweights, logits, experts and dlogits must be non-NULL", who);
    const uintptr_t es = dtype == CONVROT_DTYPE_F32 ? 4 : 2;
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(experts, 4) || !aligned(dweights, 4))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t small = (size_t)M * (size_t)top * 4, in = (size_t)M * (size_t)E * es;
    if ((dlogits != logits && overlap(dlogits, in, logits, in)) || overlap(dlogits, in, experts, small) ||
        overlap(dlogits, in, dweights, small))
        return fail(CONVROT_ERR_OVERLAP, "%s: dlogits overlaps an input (only dlogits == logits is allowed)", who);
    if ((rc = check_device())) return rc;
    return hip_status(convrot::launch_moe_route_backward(route_args(logits, dtype, nullptr, M, E, top, score, normalize, scale),
                                                         dweights, experts, dlogits, stream),
                      "moe_route_backward");
}

size_t convrot_workspace_bytes_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K)
{
    return grouped_shape_ok(rows, groups, N, K, false) ? grouped_bytes(rows, K) : 0;
}

int convrot_linear_grouped(const void *x, int x_dtype, const int8_t *xq, const float *x_scale, int64_t rows, int64_t N,
                           int64_t K, int group, const int32_t *offsets, int64_t groups, const int8_t *wq,
                           const float *w_scale, void *y, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_linear_grouped";
    int rc = check_grouped(who, rows, groups, N, K, group, false);
    if (rc) return rc;
    if (rows == 0) return CONVROT_OK;
    if (!offsets || !wq || !w_scale || !y) return fail(CONVROT_ERR_NULL, "%s: offsets, wq, w_scale and y must be non-NULL", who);
    if (!x && (!xq || !x_scale)) return fail(CONVROT_ERR_NULL, "%s: give x, or both xq and x_scale", who);
    if (x && x_dtype != CONVROT_DTYPE_F32 && x_dtype != CONVROT_DTYPE_BF16)
        return fail(CONVROT_ERR_DTYPE, "%s: x_dtype=%d", who, x_dtype);
    if ((x && !aligned(x, 16)) || (!x && (!aligned(xq, 16) || !aligned(x_scale, 4))) || !aligned(offsets, 4) ||
        !aligned(wq, 16) || !aligned(w_scale, 4) || !aligned(y, 16))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t y_bytes = (size_t)rows * (size_t)N * 2;
    if (overlap(y, y_bytes, offsets, (size_t)(groups + 1) * 4) ||
        (!x && (overlap(y, y_bytes, xq, (size_t)rows * (size_t)K) || overlap(y, y_bytes, x_scale, (size_t)rows * 4))))
        return fail(CONVROT_ERR_OVERLAP, "%s: y overlaps xq, x_scale or offsets", who);
    if (x && (rc = check_workspace(who, workspace, workspace_bytes, grouped_bytes(rows, K)))) return rc;
    if ((rc = check_device())) return rc;
    if (x) {
        int8_t *qx = static_cast<int8_t *>(workspace);
        float *sx = reinterpret_cast<float *>(qx + round256((size_t)rows * (size_t)K));
        rc = hip_status(convrot::launch_rotate_quant(x, x_dtype == CONVROT_DTYPE_F32, rows, (int)K, log2i(group), 8, qx, sx,
                                                     stream),
                        "rotate_quant");
        if (rc) return rc;
        xq = qx;
        x_scale = sx;
    }
    convrot::GroupedArgs g;
    g.xq = xq;
    g.sx = x_scale;
    g.offsets = offsets;
    g.wq = wq;
    g.sw = w_scale;
    g.y = static_cast<uint16_t *>(y);
    g.rows = rows;
    g.N = N;
    g.groups = (int)groups;
    g.K = (int)K;
    return hip_status(convrot::launch_grouped_i8(g, convrot::Epi::Bf16, stream), "grouped_i8");
}

size_t convrot_workspace_bytes_grouped_backward(int64_t rows, int64_t groups, int64_t N, int64_t K)
{
    return grouped_shape_ok(rows, groups, N, K, true) ? grouped_backward_bytes(rows, N) : 0;
}

int convrot_linear_grouped_backward(const void *dy, int64_t rows, int64_t N, int64_t K, int group,
                                    const int32_t *offsets, int64_t groups, const int8_t *wq, const float *w_scale,
                                    const void *dx_add, void *dx, void *workspace, size_t workspace_bytes,
                                    hipStream_t stream)
{
    const char *who = "convrot_linear_grouped_backward";
    int rc = check_grouped(who, rows, groups, N, K, group, true);
    if (rc) return rc;
    if (rows == 0) return CONVROT_OK;
    if (!dy || !offsets || !wq || !w_scale || !dx)
        return fail(CONVROT_ERR_NULL, "%s: dy, offsets, wq, w_scale and dx must be non-NULL", who);
    if (!aligned(dy, 16) || !aligned(offsets, 4) || !aligned(wq, 16) || !aligned(w_scale, 4) || !aligned(dx_add, 16) ||
        !aligned(dx, 16))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t dx_bytes = (size_t)rows * (size_t)K * 2;
    if ((dx_add != dx && overlap(dx_add, dx_bytes, dx, dx_bytes)) || overlap(dx, dx_bytes, offsets, (size_t)(groups + 1) * 4))
        return fail(CONVROT_ERR_OVERLAP, "%s: dx overlaps dx_add (only dx_add == dx is allowed) or offsets", who);
    if ((rc = check_workspace(who, workspace, workspace_bytes, grouped_backward_bytes(rows, N)))) return rc;
    if ((rc = check_device())) return rc;
    convrot::GroupedRowsArgs r;
    r.dy = static_cast<const uint16_t *>(dy);
    r.sw = w_scale;
    r.offsets = offsets;
    r.a = static_cast<uint16_t *>(workspace);
    r.rows = rows;
    r.N = N;
    r.groups = (int)groups;
    if ((rc = hip_status(convrot::launch_grouped_rows(r, stream), "grouped_rows"))) return rc;
    convrot::GroupedGradArgs g;
    g.a = r.a;
    g.offsets = offsets;
    g.wq1 = wq;
    g.add = static_cast<const uint16_t *>(dx_add);
    g.dx = static_cast<uint16_t *>(dx);
    g.rows = rows;
    g.N = N;
    g.groups = (int)groups;
    g.K = (int)K;
    g.log2g = log2i(group);
    return hip_status(convrot::launch_grouped_grad(g, stream), "grouped_grad");
}

size_t convrot_workspace_bytes_moe_ffn(int64_t M, int top, int64_t E, int64_t F, int64_t K)
{
    return moe_shape_ok(M, top, E, F, K, false) ? moe_layout(M, top, E, F, K, false).total : 0;
}

int convrot_moe_ffn_gated(const void *x, int x_dtype, const int32_t *experts, const float *weights, int64_t M, int top,
                          int64_t E, int64_t F, int64_t K, int group, int group_h, const int8_t *wq_gate,
                          const float *gate_scale, const int8_t *wq_up, const float *up_scale, const int8_t *wq_down,
                          const float *down_scale, int act, const void *residual, void *pre, void *d, void *y,
                          void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_moe_ffn_gated";
    int rc = check_moe(who, M, top, E, F, K, group, group_h, act, false);
    if (rc) return rc;
    if (M == 0) return CONVROT_OK;
    if (!x || !experts || !weights || !wq_gate || !gate_scale || !wq_up || !up_scale || !wq_down || !down_scale || !y)
        return fail(CONVROT_ERR_NULL, "%s: x, experts, weights, the expert weights, their scales and y must be non-NULL", who);
    if (x_dtype != CONVROT_DTYPE_F32 && x_dtype != CONVROT_DTYPE_BF16)
        return fail(CONVROT_ERR_DTYPE, "%s: x_dtype=%d", who, x_dtype);
    if (!aligned(x, 16) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(wq_gate, 16) || !aligned(wq_up, 16) ||
        !aligned(wq_down, 16) || !aligned(gate_scale, 4) || !aligned(up_scale, 4) || !aligned(down_scale, 4) ||
        !aligned(residual, 16) || !aligned(pre, 16) || !aligned(d, 16) || !aligned(y, 16))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t S = (size_t)M * (size_t)top, y_bytes = (size_t)M * (size_t)K * 2, small = S * 4;
    const size_t x_bytes = (size_t)M * (size_t)K * (x_dtype == CONVROT_DTYPE_F32 ? 4 : 2);
    const size_t pre_bytes = S * (size_t)F * 4, d_bytes = S * (size_t)K * 2;
    // y is written last, when only weights, residual and the workspace are still read; pre and d before that
    auto saved = [&](const void *q, size_t n) {
        return overlap(q, n, y, y_bytes) || overlap(q, n, residual, y_bytes) || overlap(q, n, x, x_bytes) ||
               overlap(q, n, experts, small) || overlap(q, n, weights, small);
    };
    if ((residual != y && overlap(residual, y_bytes, y, y_bytes)) || overlap(y, y_bytes, experts, small) ||
        overlap(y, y_bytes, weights, small) || saved(pre, pre_bytes) || saved(d, d_bytes) || overlap(pre, pre_bytes, d, d_bytes))
        return fail(CONVROT_ERR_OVERLAP, "%s: y, pre or d overlaps another array of the call (only residual == y is allowed)",
                    who);
    const MoeLayout L = moe_layout(M, top, E, F, K, false);
    if ((rc = check_workspace(who, workspace, workspace_bytes, L.total))) return rc;
    if ((rc = check_device())) return rc;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    convrot::MoeOrder o = moe_order(ws, L);
    int8_t *xq = reinterpret_cast<int8_t *>(ws + L.xq), *hq = reinterpret_cast<int8_t *>(ws + L.hq);
    float *xs = reinterpret_cast<float *>(ws + L.xs), *hs = reinterpret_cast<float *>(ws + L.hs);
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + L.h);
    float *part = reinterpret_cast<float *>(ws + L.part);
    convrot::MoeFew few;
    if (convrot::plan_moe_few(M, top, (int)K, (int)F, few)) {
        convrot::MoeFewArgs a;
        a.x = x;
        a.x_f32 = x_dtype == CONVROT_DTYPE_F32;
        a.xq = xq;
        a.xs = xs;
        a.hq = hq;
        a.hs = hs;
        a.experts = experts;
        a.weights = weights;
        a.wq_gate = wq_gate;
        a.gate_scale = gate_scale;
        a.wq_up = wq_up;
        a.up_scale = up_scale;
        a.wq_down = wq_down;
        a.down_scale = down_scale;
        a.residual = static_cast<const uint16_t *>(residual);
        a.h = h;
        a.y = static_cast<uint16_t *>(y);
        a.pre = static_cast<uint16_t *>(pre);
        a.d = static_cast<uint16_t *>(d);
        a.M = M;
        a.top = top;
        a.E = (int)E;
        a.K = (int)K;
        a.F = (int)F;
        a.act = act;
        a.log2g = log2i(group);
        a.log2g_h = log2i(group_h);
        if (!few.fuse_x &&
            (rc = hip_status(convrot::launch_rotate_quant(x, a.x_f32, M, (int)K, a.log2g, 8, xq, xs, stream), "rotate_quant")))
            return rc;
        if ((rc = hip_status(convrot::launch_moe_few_gate(a, few, stream), "moe_few_gate"))) return rc;
        if (!few.fuse_h &&
            (rc = hip_status(convrot::launch_rotate_quant(h, false, (int64_t)S, (int)F, a.log2g_h, 8, hq, hs, stream),
                             "rotate_quant")))
            return rc;
        return hip_status(convrot::launch_moe_few_down(a, few, stream), "moe_few_down");
    }
    o.sx = xs;
    o.sx_of = reinterpret_cast<float *>(ws + L.rs);
    rc = hip_status(convrot::launch_rotate_quant(x, x_dtype == CONVROT_DTYPE_F32, M, (int)K, log2i(group), 8, xq, xs, stream),
                    "rotate_quant");
    if (rc) return rc;
    if ((rc = hip_status(convrot::launch_moe_order(experts, (int64_t)S, (int)E, top, o, stream), "moe_order"))) return rc;
    convrot::GroupedArgs g;
    g.xq = xq;
    g.sx = o.sx_of;
    g.offsets = o.offsets;
    g.source = o.token_of;
    g.slot_of = o.slot_of;
    g.wq = wq_gate;
    g.wq2 = wq_up;
    g.sw = gate_scale;
    g.sw2 = up_scale;
    g.y = h;
    g.pre = static_cast<uint16_t *>(pre);
    g.rows = (int64_t)S;
    g.N = F;
    g.groups = (int)E;
    g.K = (int)K;
    g.act = act;
    if ((rc = hip_status(convrot::launch_grouped_i8(g, convrot::Epi::Gated, stream), "grouped_i8"))) return rc;
    // (rows past the last slot with an expert hold anything; their codes are never read)
    if ((rc = hip_status(convrot::launch_rotate_quant(h, false, (int64_t)S, (int)F, log2i(group_h), 8, hq, hs, stream),
                         "rotate_quant")))
        return rc;
    convrot::GroupedArgs w;
    w.xq = hq;
    w.sx = hs;
    w.offsets = o.offsets;
    w.slot_of = o.slot_of;
    w.wq = wq_down;
    w.sw = down_scale;
    w.part = part;
    w.d = static_cast<uint16_t *>(d);
    w.rows = (int64_t)S;
    w.N = K;
    w.groups = (int)E;
    w.K = (int)F;
    if ((rc = hip_status(convrot::launch_grouped_i8(w, convrot::Epi::Part, stream), "grouped_i8"))) return rc;
    return hip_status(convrot::launch_moe_combine(part, o.row_of, weights, static_cast<const uint16_t *>(residual),
                                                  static_cast<uint16_t *>(y), M, (int)K, top, stream),
                      "moe_combine");
}

size_t convrot_workspace_bytes_moe_ffn_backward(int64_t M, int top, int64_t E, int64_t F, int64_t K)
{
    return M > 0 && moe_shape_ok(M, top, E, F, K, true) ? moe_layout(M, top, E, F, K, true).total : 0;
}

int convrot_moe_ffn_gated_backward(const void *dy, const void *pre, const void *d, const int32_t *experts,
                                   const float *weights, int64_t M, int top, int64_t E, int64_t F, int64_t K, int group,
                                   int group_h, const int8_t *wq_gate, const float *gate_scale, const int8_t *wq_up,
                                   const float *up_scale, const int8_t *wq_down, const float *down_scale, int act,
                                   const void *dx_add, void *dx, float *dweights, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream)
{
    const char *who = "convrot_moe_ffn_gated_backward";
    int rc = check_moe(who, M, top, E, F, K, group, group_h, act, true);
    if (rc) return rc;
    if (M == 0) return CONVROT_OK;
    if (!dy || !pre || !experts || !weights || !wq_gate || !gate_scale || !wq_up || !up_scale || !wq_down || !down_scale ||
        !dx || (dweights && !d))
        return fail(CONVROT_ERR_NULL, "%s: dy, pre, experts, weights, the expert weights, their scales, dx and, with dweights, "
                    "d must be non-NULL", who);
    if (!aligned(dy, 16) || !aligned(pre, 16) || !aligned(d, 16) || !aligned(experts, 4) || !aligned(weights, 4) ||
        !aligned(wq_gate, 16) || !aligned(wq_up, 16) || !aligned(wq_down, 16) || !aligned(gate_scale, 4) ||
        !aligned(up_scale, 4) || !aligned(down_scale, 4) || !aligned(dx_add, 16) || !aligned(dx, 16) || !aligned(dweights, 4))
        return fail(CONVROT_ERR_ALIGN, "%s: misaligned pointer", who);
    const size_t S = (size_t)M * (size_t)top, x_bytes = (size_t)M * (size_t)K * 2, small = S * 4;
    if ((dx_add != dx && overlap(dx_add, x_bytes, dx, x_bytes)) || overlap(dweights, small, dx, x_bytes) ||
        overlap(dweights, small, dx_add, x_bytes) || overlap(dweights, small, dy, x_bytes) ||
        overlap(dweights, small, pre, S * (size_t)F * 4) || overlap(dweights, small, d, S * (size_t)K * 2) ||
        overlap(dweights, small, experts, small) || overlap(dweights, small, weights, small))
        return fail(CONVROT_ERR_OVERLAP, "%s: dx overlaps dx_add (only dx_add == dx is allowed), or dweights another array of "
                    "the call", who);
    const MoeLayout L = moe_layout(M, top, E, F, K, true);
    if ((rc = check_workspace(who, workspace, workspace_bytes, L.total))) return rc;
    if ((rc = check_device())) return rc;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const convrot::MoeOrder o = moe_order(ws, L);
    float *part = reinterpret_cast<float *>(ws + L.part);
    if ((rc = hip_status(convrot::launch_moe_order(experts, (int64_t)S, (int)E, top, o, stream), "moe_order"))) return rc;
    convrot::GroupedRowsArgs r;
    r.dy = static_cast<const uint16_t *>(dy);
    r.sw = down_scale;
    r.experts = experts;
    r.row_of = o.row_of;
    r.weights = weights;
    r.d = dweights ? static_cast<const uint16_t *>(d) : nullptr;
    r.dweights = dweights;
    r.a = reinterpret_cast<uint16_t *>(ws + L.a);
    r.rows = (int64_t)S;
    r.N = K;
    r.groups = (int)E;
    r.top = top;
    if ((rc = hip_status(convrot::launch_grouped_rows(r, stream), "grouped_rows"))) return rc;
    convrot::GroupedGradArgs down;
    down.a = r.a;
    down.offsets = o.offsets;
    down.slot_of = o.slot_of;
    down.wq1 = wq_down;
    down.next.pre = static_cast<const uint16_t *>(pre);
    down.next.sw_gate = gate_scale;
    down.next.sw_up = up_scale;
    down.next.act = act;
    down.next.a = reinterpret_cast<uint16_t *>(ws + L.a2);
    down.rows = (int64_t)S;
    down.N = K;
    down.groups = (int)E;
    down.K = (int)F;
    down.log2g = log2i(group_h);
    if ((rc = hip_status(convrot::launch_grouped_grad(down, stream), "grouped_grad"))) return rc;
    convrot::GroupedGradArgs up;
    up.a = down.next.a;
    up.offsets = o.offsets;
    up.wq1 = wq_gate;
    up.wq2 = wq_up;
    up.part = part;
    up.rows = (int64_t)S;
    up.N = F;
    up.groups = (int)E;
    up.K = (int)K;
    up.log2g = log2i(group);
    if ((rc = hip_status(convrot::launch_grouped_grad(up, stream), "grouped_grad"))) return rc;
    return hip_status(convrot::launch_moe_combine(part, o.row_of, nullptr, static_cast<const uint16_t *>(dx_add),
                                                  static_cast<uint16_t *>(dx), M, (int)K, top, stream),
                      "moe_combine");
}

} // extern "C"
