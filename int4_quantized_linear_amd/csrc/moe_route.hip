// moe_route.hip -- the router of a mixture-of-experts layer: the top experts of each token and their weights, and the
// gradient of the logits (gfx950).
//
//   s = softmax(l) or sigmoid(l) over the E experts;   key = l, or with a bias s + bias
//   experts = the `top` largest keys (ties to the lowest index), never a key of -inf (a masked expert)
//   w_j = scale s_j,  or with normalize  scale s_j / sum over the chosen of s
// Without a bias the logits themselves order the experts (both scores grow with them), exactly; with one the keys
// are taken in 64 bits, since two of them may be closer than fp32 can tell.
// Normalised weights come from the chosen logits alone: a softmax over log s (l itself, up to a constant, for
// softmax), so they stay defined where every s is 0 in fp32.  They and their gradients are formed in 64 bits:
// a handful of values per token, next to differences that cancel.
//
// One wavefront per token, PER logits per lane.  A choice is the largest of the lanes' largest keys' 32 high bits, by six DPP
// steps and a ballot; only where several lanes have it the low bits and the index decide.  The winner's lane drops it.
// One token's choice, 8 of 64: 3 us, latency.  8192 tokens, 8 of 256, with a bias: 14 us, bound by instructions, about 1000
// per token of which the 256 keys take 400 and a choice 45 (both halves of the key reduced and the logits carried: 15.5);
// their logits are 8 MB, 2 us.  Its gradient, 6 of 128 in bf16: 7.7 us.
#include "device_common.hpp"
#include "launchers.hpp"

namespace convrot {
namespace {

constexpr int WAVES = 4;

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *experts;
    float *weights;
    int64_t M;
    int E, top;
    float scale;
    bool f32, sigmoid, normalize;
};

__device__ __forceinline__ float load_logit(const void *p, bool f32, int64_t i)
{
    return f32 ? static_cast<const float *>(p)[i] : bf16lo_to_f32(static_cast<const uint16_t *>(p)[i]);
}

// Logits 64 r + lane of token m, -inf past the last: every load at once, without a branch between them.
template <int PER>
__device__ __forceinline__ void load_row(const void *logits, bool f32, int64_t m, int E, int lane, float (&l)[PER])
{
    if (f32) {
        const float *src = static_cast<const float *>(logits) + m * E;
#pragma unroll
        for (int r = 0; r < PER; ++r) l[r] = src[min(64 * r + lane, E - 1)];
    } else {
        const uint16_t *src = static_cast<const uint16_t *>(logits) + m * E;
        uint32_t raw[PER];
#pragma unroll
        for (int r = 0; r < PER; ++r) raw[r] = src[min(64 * r + lane, E - 1)];
#pragma unroll
        for (int r = 0; r < PER; ++r) l[r] = bf16lo_to_f32(raw[r]);
    }
#pragma unroll
    for (int r = 0; r < PER; ++r) l[r] = 64 * r + lane < E ? l[r] : -__builtin_inff();
}

// v of another lane by DPP control CTRL, `none` where that control has no source.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float none, float v)
{
    return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(none), __float_as_uint(v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double none, double v)
{
    const uint64_t a = __builtin_bit_cast(uint64_t, none), b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp<CTRL, ROWS>((uint32_t)a, (uint32_t)b), hi = dpp<CTRL, ROWS>((uint32_t)(a >> 32), (uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ float last_lane(float v) { return __uint_as_float(last_lane(__float_as_uint(v))); }
__device__ __forceinline__ double from_lane(double v, int lane)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double last_lane(double v) { return from_lane(v, 63); }

// op over the wavefront, in every lane: within rows of 16 lanes by row_shr 1, 2, 4, 8, then row_bcast 15 and 31.  (Exchanges
// through LDS take several times as long, and the choice is a chain of them.)
template <typename T, typename Op>
__device__ __forceinline__ T wave_all(T v, T none, Op op)
{
    v = op(v, dpp<0x111, 0xf>(none, v));
    v = op(v, dpp<0x112, 0xf>(none, v));
    v = op(v, dpp<0x114, 0xf>(none, v));
    v = op(v, dpp<0x118, 0xf>(none, v));
    v = op(v, dpp<0x142, 0xa>(none, v));
    v = op(v, dpp<0x143, 0xc>(none, v));
    return last_lane(v);
}
__device__ __forceinline__ float wave_max(float v)
{
    return wave_all(v, -__builtin_inff(), [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ double wave_max(double v)
{
    return wave_all(v, -__builtin_inf(), [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    return wave_all(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ double wave_sum(double v)
{
    return wave_all(v, 0.0, [](double a, double b) { return a + b; });
}

// Unsigned integers in the order of the floats (-0 as 0; 0 for NaN and -inf, which no choice takes).
__device__ __forceinline__ uint32_t ordered(float v)
{
    if (!(v > -__builtin_inff())) return 0u;
    const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v)
{
    if (!(v > -__builtin_inf())) return 0u;
    const uint64_t b = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);
    return b & 0x8000000000000000u ? ~b : b | 0x8000000000000000u;
}

// log sigmoid(l), whose exponential is the score up to rounding for every l.
__device__ __forceinline__ double log_sigmoid(double l) { return l < 0.0 ? l - log1p(exp(l)) : -log1p(exp(-l)); }

// The weights' common part for lane j < n, which holds the chosen logit l (other lanes: nothing): with normalize the
// softmax of log s, else s itself.  zmax, z: the row's largest logit and sum of exponentials (softmax scores).  With normalize,
// lead: a lane with the largest share.
__device__ __forceinline__ double chosen_share(bool sigmoid, bool normalize, double l, bool valid, float zmax, double z, int &lead)
{
    lead = 0;
    if (!normalize) {
        if (!valid) return 0.0;
        return sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)zmax) / z;
    }
    const double v = sigmoid ? log_sigmoid(l) : l;
    const double most = wave_max(valid ? v : -__builtin_inf());
    const uint64_t first = __builtin_amdgcn_ballot_w64(valid && v == most);
    if (first) lead = __builtin_ctzll(first);
    const double e = valid ? exp(v - most) : 0.0;
    return e / wave_sum(e);
}

template <typename KEY, int PER>
__global__ void __launch_bounds__(64 * WAVES) moe_route_kernel(RouteParams p)
{
    constexpr bool BIAS = sizeof(KEY) == 8;
    const int lane = threadIdx.x & 63;
    const int64_t m = (int64_t)grid_workgroup() * WAVES + (threadIdx.x >> 6);
    if (m >= p.M) return;
    float l[PER], bias[BIAS ? PER : 1];
    if constexpr (BIAS) {
#pragma unroll
        for (int r = 0; r < PER; ++r) bias[r] = p.bias[min(64 * r + lane, p.E - 1)];
    }
    load_row(p.logits, p.f32, m, p.E, lane, l);
    bool bad = false, infinite = false;
    float most = -__builtin_inff();
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        bad |= l[r] != l[r];
        if constexpr (BIAS) bad |= bias[r] != bias[r];
        infinite |= l[r] == __builtin_inff();
        most = __builtin_fmaxf(most, l[r]);
    }
    // a softmax has no shares next to an infinite logit: the row's weights are NaN, and the logits order its experts
    infinite = !p.sigmoid && __builtin_amdgcn_ballot_w64(infinite) != 0;
    bad = infinite || __builtin_amdgcn_ballot_w64(bad) != 0;
    double z = 1.0;
    if (!p.sigmoid && (BIAS || !p.normalize)) {
        most = wave_max(most);
        double sum = 0.0;
#pragma unroll
        for (int r = 0; r < PER; ++r)
            if (l[r] > -__builtin_inff()) sum += BIAS ? exp((double)l[r] - (double)most) : (double)expf(l[r] - most);
        z = wave_sum(sum);
    }
    KEY key[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        if constexpr (BIAS) {
            const double x = (double)l[r];
            const double s = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)most) / z;
            const double v = infinite && bias[r] > -__builtin_inff() ? x : s + (double)bias[r];
            key[r] = l[r] > -__builtin_inff() ? ordered(v) : 0u;
        } else {
            key[r] = ordered(l[r]);
        }
    }
    int chosen = -1;                                     // lane j: the j-th expert
    for (int j = 0; j < p.top; ++j) {
        KEY best = key[0];                               // the lane's own, the lowest index of equal ones
        int at = lane;
#pragma unroll
        for (int r = 1; r < PER; ++r) {
            const bool more = key[r] > best;
            best = more ? key[r] : best;
            at = more ? 64 * r + lane : at;
        }
        const uint32_t high = (uint32_t)(best >> (BIAS ? 32 : 0)), most_high = wave_max(high);
        if (most_high == 0u) break;                      // nothing left that may be chosen
        uint64_t lanes = __builtin_amdgcn_ballot_w64(high == most_high);
        if (lanes & (lanes - 1)) {                       // several: by the low half, then by index
            bool first = high == most_high;
            if constexpr (BIAS) {
                const uint32_t low = first ? (uint32_t)best : 0u, most_low = wave_max(low);
                first = first && low == most_low;
            }
            at = (int)~wave_max(first ? ~(uint32_t)at : 0u);
        } else {
            at = __builtin_amdgcn_readlane(at, __builtin_ctzll(lanes));
        }
#pragma unroll
        for (int r = 0; r < PER; ++r)
            if (at == 64 * r + lane) key[r] = 0u;
        if (lane == j) chosen = at;
    }
    const float value = chosen >= 0 ? load_logit(p.logits, p.f32, m * p.E + chosen) : 0.0f;
    int lead;
    const double share = chosen_share(p.sigmoid, p.normalize, (double)value, chosen >= 0, most, z, lead);
    if (lane < p.top) {
        p.experts[m * p.top + lane] = chosen;
        p.weights[m * p.top + lane] = bad ? __builtin_nanf("") : chosen < 0 ? 0.0f : (float)(share * (double)p.scale);
    }
}

struct RouteGradParams {
    const void *logits;
    const int32_t *experts;    // [M, top]
    const float *dweights;     // [M, top]
    void *dlogits;             // logits' type
    int64_t M;
    int E, top;
    float scale;
    bool f32, sigmoid, normalize;
};

// With q the shares above, g = scale dweights and G_i the sum of g over the slots that chose i (0 without one):
//   softmax:  dl_i = s_i (G_i - sum_k s_k G_k)
//   softmax normalised: dl_t = q_t (g_t - sum_j q_j g_j);   sigmoid: dl_t = s_t (1 - s_t) g_t, normalised
//   q_t (1 - s_t) (g_t - sum_j q_j g_j);   the logits that no slot chose get 0, and one chosen twice the sum.
// Where one share is nearly 1 the two terms of its difference agree in all but their last digits, 18 logits ahead of the rest in
// all that fp32 has, 37 ahead in all of 64 bits.  Both are therefore taken relative to the leading logit's own G (or g), which leaves
// every difference as it is: the leader's term of the sum is then 0 and the others are small by themselves.  All of it in 64
// bits, rounded once.
template <int PER>
__global__ void __launch_bounds__(64 * WAVES) moe_route_backward_kernel(RouteGradParams p)
{
    const bool all = !p.sigmoid && !p.normalize;         // every logit has a gradient
    const int lane = threadIdx.x & 63;
    const int64_t m = (int64_t)grid_workgroup() * WAVES + (threadIdx.x >> 6);
    if (m >= p.M) return;
    float row[PER] = {};
    if (all) load_row(p.logits, p.f32, m, p.E, lane, row);
    int chosen = -1;
    double g = 0.0, l = 0.0;
    if (lane < p.top) {
        chosen = p.experts[m * p.top + lane];
        if ((unsigned)chosen >= (unsigned)p.E) chosen = -1;
        if (chosen >= 0) {
            g = (double)p.dweights[m * p.top + lane] * (double)p.scale;
            l = (double)load_logit(p.logits, p.f32, m * p.E + chosen);
            if (l == -__builtin_inf()) chosen = -1;      // masked: its weight is a constant 0
        }
    }
    const bool valid = chosen >= 0;
    double d = valid ? g : 0.0;                          // what the slot adds to its logit's entry: G's part, or the gradient
    if (!all) {
        int lead;
        const double share = chosen_share(p.sigmoid, p.normalize, l, valid, 0.0f, 1.0, lead);
        if (p.normalize) {
            d = g - from_lane(g, lead);
            d -= wave_sum(valid ? share * d : 0.0);
        }
        d *= share;
        if (p.sigmoid) d *= 1.0 / (1.0 + exp(l));        // 1 - s
        if (!valid) d = 0.0;
    }
    double v[PER] = {};
    // in slot order, so that an expert chosen twice gets the same sum at every call
    for (int j = 0; j < p.top; ++j) {
        const int at = __builtin_amdgcn_readlane(chosen, j);
        const double add = from_lane(d, j);
#pragma unroll
        for (int r = 0; r < PER; ++r)
            if (at == 64 * r + lane) v[r] += add;
    }
    if (all) {
        float most = -__builtin_inff();
#pragma unroll
        for (int r = 0; r < PER; ++r) most = __builtin_fmaxf(most, row[r]);
        most = wave_max(most);
        double e[PER], sum = 0.0, lead = 0.0;
        bool leads = false;
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            e[r] = row[r] == -__builtin_inff() ? 0.0 : exp((double)row[r] - (double)most);   // a NaN stays one
            sum += e[r];
            const bool first = row[r] == most && !leads;
            lead = first ? v[r] : lead;
            leads |= first;
        }
        const double z = wave_sum(sum);
        const uint64_t lanes = __builtin_amdgcn_ballot_w64(leads);
        lead = from_lane(lead, lanes ? __builtin_ctzll(lanes) : 0);
        sum = 0.0;
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            v[r] -= lead;
            sum += e[r] * v[r];
        }
        // (z == 0: a row masked whole; with a NaN in the row it is one)
        const double inv = z == 0.0 ? 0.0 : 1.0 / z, mean = wave_sum(sum) * inv;
#pragma unroll
        for (int r = 0; r < PER; ++r) v[r] = e[r] * inv * (v[r] - mean);
    }
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = 64 * r + lane;
        if (i >= p.E) continue;
        const float out = (float)v[r];
        if (p.f32) static_cast<float *>(p.dlogits)[m * p.E + i] = out;
        else static_cast<uint16_t *>(p.dlogits)[m * p.E + i] = (uint16_t)(pack_bf16x2(out, 0.0f) & 0xffffu);
    }
}

int per_lane(int E) { return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16; }

template <typename KEY>
void route_per(const RouteParams &p, dim3 grid, hipStream_t stream)
{
    const dim3 block(64 * WAVES);
    switch (per_lane(p.E)) {
    case 1: hipLaunchKernelGGL((moe_route_kernel<KEY, 1>), grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL((moe_route_kernel<KEY, 2>), grid, block, 0, stream, p); break;
    case 4: hipLaunchKernelGGL((moe_route_kernel<KEY, 4>), grid, block, 0, stream, p); break;
    case 8: hipLaunchKernelGGL((moe_route_kernel<KEY, 8>), grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL((moe_route_kernel<KEY, 16>), grid, block, 0, stream, p);
    }
}

} // namespace

hipError_t launch_moe_route(const RouteArgs &a, int32_t *experts, float *weights, hipStream_t stream)
{
    if (a.M <= 0) return hipSuccess;
    const RouteParams p = {a.logits, a.bias, experts, weights, a.M, a.E, a.top, a.scale, a.f32, a.score != 0, a.normalize};
    const dim3 grid = workgroup_grid((a.M + WAVES - 1) / WAVES);
    if (a.bias) route_per<uint64_t>(p, grid, stream);
    else route_per<uint32_t>(p, grid, stream);
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const RouteArgs &a, const float *dweights, const int32_t *experts, void *dlogits,
                                     hipStream_t stream)
{
    if (a.M <= 0) return hipSuccess;
    const RouteGradParams p = {a.logits, experts, dweights, dlogits, a.M, a.E, a.top, a.scale, a.f32, a.score != 0, a.normalize};
    const dim3 grid = workgroup_grid((a.M + WAVES - 1) / WAVES);
    const dim3 block(64 * WAVES);
    switch (per_lane(a.E)) {
    case 1: hipLaunchKernelGGL(moe_route_backward_kernel<1>, grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL(moe_route_backward_kernel<2>, grid, block, 0, stream, p); break;
    case 4: hipLaunchKernelGGL(moe_route_backward_kernel<4>, grid, block, 0, stream, p); break;
    case 8: hipLaunchKernelGGL(moe_route_backward_kernel<8>, grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL(moe_route_backward_kernel<16>, grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

} // namespace convrot
