// rotate_common.hpp -- the rotation and the quantizer's quotient on registers, for the kernels that quantize rows
// (gfx950).  Internal to libconvrot.
//
// Data layout in registers.  A row is cut into "slots" of 256 consecutive channels.  Inside a
// wavefront, lane bits 4:2 select one of 8 slots and the 8 lanes of a slot hold its 256
// values as 4 chunks x 8 channels each:
//     channel bits 2:0 -> element inside a chunk (one 16-byte bf16 load = 8 channels)
//     channel bits 4:3 -> lane bits 1:0   (butterfly partners reached with DPP quad_perm)
//     channel bit  5   -> lane bit 5      (moved into a register with v_permlane32_swap)
//     channel bits 7:6 -> chunk index r   (registers)
// so the 8-stage fast Walsh-Hadamard transform runs 6 stages in registers and 2 across lanes
// with no LDS traffic.  Each load instruction reads 128 contiguous bytes per slot.
#pragma once
#include "device_common.hpp"

namespace convrot {

// The code is rint of the correctly rounded fp32 quotient of the normalised value v = fp32(vu /
// sqrt(g)) by the stored scale s, as its definition states, not of a product with a rounded
// reciprocal: rotated sums of bf16 values often carry few significant bits, so exact half-integer
// quotients are common (3-5e-4 of the codes of N(0, 0.02) bf16 weight rows at g = 1 or 2, and of
// small-integer activations at g = 256) and a rounded reciprocal breaks those ties either way.
//
// Quotient: m = RN(1 / s), q0 = RN(v m) is within an ulp of v / s, the remainder v - q0 s is
// exact in one fma, and one correction step q0 + (v - q0 s) m rounds correctly (Markstein's
// theorem).  The sign the lane-exchange butterflies left on this lane's values goes into both
// factors, and for even log2 g so does 1/sqrt(g) = cg, a power of two (a = sign cg m, b = s /
// (sign cg): exact scalings), so the unnormalised sum vu enters directly.  For odd log2 g, the
// normalised magnitude is vu cg + vu cg_lo in one fma, the correctly rounded product unless
// vu / sqrt(g) lies within ~2^-47 of a rounding midpoint, with a = sign m, b = sign s.  s == 0
// comes with a = b = 0 and vu == 0: the code is 0.
struct QuotientRN {
    float a, b;
};

template <int LG>
__device__ __forceinline__ QuotientRN quotient_consts(float s, float sign, float cg)
{
    const float m = s > 0.0f ? 1.0f / s : 0.0f;
    if constexpr (LG % 2 == 0) return {m * (sign * cg), s > 0.0f ? s / (sign * cg) : 0.0f};
    else return {sign * m, sign * s};
}

// the scale s back from the constants (exact)
template <int LG>
__device__ __forceinline__ float quotient_scale(QuotientRN k, float cg)
{
    return LG % 2 == 0 ? __builtin_fabsf(k.b) * cg : __builtin_fabsf(k.b);
}

// fp32 of the quotient (before rint) for an unnormalised rotated value vu
template <int LG>
__device__ __forceinline__ float quotient_rn(float vu, QuotientRN k, float cg, float cg_lo)
{
    float v = vu;
    if constexpr (LG % 2 != 0) v = __builtin_fmaf(vu, cg, vu * cg_lo);
    const float q0 = v * k.a;
    const float r = __builtin_fmaf(-q0, k.b, v);
    return __builtin_fmaf(r, k.a, q0);
}

__device__ __forceinline__ void bfly(float &a, float &b)
{
    const float s = a + b;
    b = a - b;
    a = s;
}

// Unnormalised Walsh-Hadamard transform of one slot held as 4 chunks x 8 values per lane (the
// register layout above), on channel bits < LG.  qd = lane & 3.
template <int LG>
__device__ __forceinline__ void fwht_slot(float (&v)[4][8], int qd)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            if (LG > b) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!(e & (1 << b))) bfly(v[r][e], v[r][e | (1 << b)]);
            }
        }
    }
    // channel bits 6 and 7: chunk registers
    if constexpr (LG > 6) {
#pragma unroll
        for (int e = 0; e < 8; ++e) { bfly(v[0][e], v[1][e]); bfly(v[2][e], v[3][e]); }
    }
    if constexpr (LG > 7) {
#pragma unroll
        for (int e = 0; e < 8; ++e) { bfly(v[0][e], v[2][e]); bfly(v[1][e], v[3][e]); }
    }
    // channel bit 5: swap it with chunk bit 0 (channel bit 6) between lane halves, then butterfly
    // in registers.  Afterwards v[2*r1 + c5][e] holds channel bit 5 = c5 and channel bit 6 =
    // lane bit 5.
    if constexpr (LG > 5) {
#pragma unroll
        for (int r1 = 0; r1 < 2; ++r1)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                swap32f(v[2 * r1][e], v[2 * r1 + 1][e]);
                bfly(v[2 * r1][e], v[2 * r1 + 1][e]);
            }
    }
    // channel bits 3 and 4, last: partner is lane ^ 1 / lane ^ 2.  Each stage is one
    // v_fmac_f32_dpp per value: self + partner * c, c = +1 on the lower lane (a + b, correct) and
    // -1 on the upper lane (b - a, the negated result).  Running the two lane stages after all
    // others keeps that sign error out of every other butterfly: the final value of a lane is off
    // by the sign (-1)^(bit0 ^ bit1) of its quad position, which is folded into the quantization
    // multiplier and does not change |v|.
    if constexpr (LG > 3) {
        const float c = (qd & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) fmac_dpp8_xor1_(v[r], c);
    }
    if constexpr (LG > 4) {
        const float c = (qd & 2) ? -1.0f : 1.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) fmac_dpp8_xor2_(v[r], c);
    }
}

} // namespace convrot
