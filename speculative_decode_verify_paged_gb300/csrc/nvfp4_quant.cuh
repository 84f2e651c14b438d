// NVFP4 quantisation of one 16-element block against a cache's decode scale,
// shared by the kernels that write a cache.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace spec_attn {

__device__ __forceinline__ void st_global_v2(void* p, uint32_t a, uint32_t b) {
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}

// binary32 -> E4M3 byte, nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3_rn_sat(float x) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(x), "f"(x));
    return d & 0xFFu;
}

// Four pairs (t[2k] even element, t[2k+1] odd) -> four E2M1 code bytes, the
// even element in each low nibble; nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x8_rn_sat(const float (&t)[8]) {
    uint32_t d;
    asm("{ .reg .b8 c0, c1, c2, c3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"   // first operand -> high nibble
        "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
        "mov.b32 %0, {c0, c1, c2, c3}; }"
        : "=r"(d)
        : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
    return d;
}

// (a call: the rare path of a block stays out of its caller's code)
static __device__ __noinline__ float quotient(float x, float y) { return __fdiv_rn(x, y); }

// The block's 16 bf16 elements (a, then b) -> 8 code bytes (c0, c1) and the
// scale byte sb: scale = E4M3(amax / (6 g)), den = scale * g, code = den == 0 ?
// 0 : E2M1(x / den), every product and quotient in binary32 to nearest even.
//
// The 16 quotients share their divisor.  With r = 1 / den to nearest, q = x r
// is close to x / den, its residual x - q den is exact in one fused multiply-add
// or nearly so, and q + r (x - q den) in another is the quotient rounded to
// nearest (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) while nothing overflows or loses bits below
// the normal range: three instructions for each element instead of a division.
// The theorem asks for a q within an ulp, and here it is within 1.5; but only a
// quotient within an ulp or two of a rounding border of E2M1 could change its
// code, x has 8 significant bits, and for every such x and every divisor in
// reach of a border the result is the division's (checked in rational
// arithmetic, tests/test_nvfp4_quotients_host.py).
// The theorem excludes a divisor whose significand is all ones.  Such a den, one
// outside 2^-60 .. 2^60, and a block whose largest quotient passes 2^20 take the
// division itself; elements below 2^-40 den are far from every rounding border.
__device__ __forceinline__ void nvfp4_block(const uint4& a, const uint4& b, float g, uint32_t& c0, uint32_t& c1,
                                            uint32_t& sb) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        amax = fmaxf(amax, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1])));
    }
    sb = e4m3_rn_sat(__fdiv_rn(amax, __fmul_rn(6.0f, g)));
    const float den = __fmul_rn(e4m3_to_float(sb), g);
    c0 = c1 = 0u;
    if (den != 0.f) {
        float t0[8], t1[8];
        const bool plain = den >= 8.673617379884035e-19f && den <= 1.152921504606847e18f && amax <= den * 1048576.0f &&
                           (__float_as_uint(den) & 0x7FFFFFu) != 0x7FFFFFu;
        if (plain) {
            const float r = __frcp_rn(den);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q0 = __fmul_rn(x[e], r), q1 = __fmul_rn(x[8 + e], r);
                t0[e] = __fmaf_rn(__fmaf_rn(-q0, den, x[e]), r, q0);
                t1[e] = __fmaf_rn(__fmaf_rn(-q1, den, x[8 + e]), r, q1);
                // (a zero keeps its sign)
                if (x[e] == 0.f) t0[e] = x[e];
                if (x[8 + e] == 0.f) t1[e] = x[8 + e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t0[e] = quotient(x[e], den);
                t1[e] = quotient(x[8 + e], den);
            }
        }
        c0 = e2m1x8_rn_sat(t0);
        c1 = e2m1x8_rn_sat(t1);
    }
}

}  // namespace spec_attn
