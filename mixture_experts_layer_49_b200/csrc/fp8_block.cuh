// fp8_block.cuh -- the activations of the block-scaled e4m3 experts, the same for
// one or two tokens (fp8_block_decode.cu) and for more (fp8_block_sm100.cu).
#pragma once

#include <stdint.h>

namespace moe {

__device__ __forceinline__ float fb_silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// Two fp32 numbers in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a Phi(a) and b Phi(b), for |a|, |b| <= 9 within 49 * 2^-24 of their values: a block
// of hidden values is scaled by its largest, so where all of a block lie in the
// negative tail an absolute error is not enough (1 + erf leaves 2e-5 of the value at
// -3 and 0.1 at -5.4).  With x = |v| the smaller tail is Phi(-x) = t P(t) exp(-x^2 / 2),
// t = 1 / (1 + 0.3 x); P of degree 7 is fitted by least squares, reweighted towards
// the largest relative error, over 0 <= x <= 14.5: off by 2.8 * 2^-24.  t is off by 3
// of them, the polynomial and products by 7, exp2 by 4; x^2 / 2 log2(e) up to 58 is
// rounded once (22) and its constant is off by 9 there.  Two at a time, because the
// multiply-adds of pairs halve a GELU tile's epilogue.
__device__ __forceinline__ void fb_gelu2(float &a, float &b) {
    const float xa = min_nan(fabsf(a), 15.f), xb = min_nan(fabsf(b), 15.f);      // further out the tail is 0
    const uint64_t x = pack2(xa, xb), nx = pack2(-xa, -xb);
    float da, db;
    unpack2(fma2(pack2(0.3f, 0.3f), x, pack2(1.f, 1.f)), da, db);
    const uint64_t t = pack2(__fdividef(1.f, da), __fdividef(1.f, db));
    uint64_t p = pack2(0.035423725843429565f, 0.035423725843429565f);
#define FB_TERM(c) p = fma2(p, t, pack2(c, c));
    FB_TERM(-0.15615838766098022f) FB_TERM(0.2045566588640213f) FB_TERM(-0.052033912390470505f)
    FB_TERM(0.12769171595573425f) FB_TERM(0.10017596185207367f) FB_TERM(0.12071213871240616f)
    FB_TERM(0.11963201314210892f)
#undef FB_TERM
    constexpr float kHalfLog2e = 0.7213475108146667f;
    const uint64_t nm = mul2(nx, x), lost = fma2(x, x, nm);          // -x^2 rounded, and what that took away
    float ea, eb;
    unpack2(fma2(nm, pack2(kHalfLog2e, kHalfLog2e), mul2(lost, pack2(-kHalfLog2e, -kHalfLog2e))), ea, eb);
    const uint64_t q = mul2(mul2(t, p), pack2(exp2_fast(ea), exp2_fast(eb)));
    unpack2(fma2(nx, q, pack2(fmaxf(a, 0.f), fmaxf(b, 0.f))), a, b);             // a NaN comes through x
}
__device__ __forceinline__ float fb_gelu(float v) {
    float w = v;
    fb_gelu2(v, w);
    return v;
}

}  // namespace moe
