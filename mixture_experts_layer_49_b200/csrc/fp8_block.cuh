// fp8_block.cuh -- the activations of the block-scaled e4m3 experts, the same for
// one or two tokens (fp8_block_decode.cu) and for more (fp8_block_sm100.cu).
#pragma once

#include <stdint.h>

namespace moe {

__device__ __forceinline__ float fb_silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// v Phi(v), for any v within 17 * 2^-24 of its value: a block of hidden values is
// scaled by its largest, so where all of a block lie in the negative tail an
// absolute error is not enough (1 + erf leaves 2e-5 of it at -3 and 0.1 at -5.4).
// With x = |v| the smaller tail is Phi(-x) = t P(t) exp(-x^2 / 2), t = 1 / (1 +
// 0.35 x); P of degree 8 is fitted by least squares, reweighted towards the
// largest relative error, over 0 <= x <= 14.5: off by 2^-24.9.  What the argument
// of exp2 loses to rounding is made good by its first-order term.
__device__ __forceinline__ float fb_gelu(float v) {
    const float x = fminf(fabsf(v), 15.f);                 // further out the tail is 0
    const float t = __fdividef(1.f, fmaf(0.35f, x, 1.f));
    float p = -0.029157884418964386f;
    p = fmaf(p, t, 0.14403092861175537f);
    p = fmaf(p, t, -0.2558390200138092f);
    p = fmaf(p, t, 0.15931972861289978f);
    p = fmaf(p, t, -0.02321236953139305f);
    p = fmaf(p, t, 0.10555250942707062f);
    p = fmaf(p, t, 0.11982128769159317f);
    p = fmaf(p, t, 0.1398635059595108f);
    p = fmaf(p, t, 0.139621302485466f);
    constexpr float kHi = 0.7213475108146667f, kLo = 9.629815167500055e-09f;     // log2(e) / 2
    const float m = x * x, z = m * kHi;
    const float lost = fmaf(fmaf(x, x, -m), kHi, fmaf(m, kLo, fmaf(m, kHi, -z)));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-z));
    e = fmaf(e * lost, -0.6931471805599453f, e);
    const float q = t * p * e;
    return v * (v < 0.f ? q : 1.f - q);
}

}  // namespace moe
