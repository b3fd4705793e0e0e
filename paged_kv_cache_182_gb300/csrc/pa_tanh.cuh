// pa_tanh.cuh -- tanh of a thread's block of capped scores.
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "pa_ptx.cuh"

namespace pa {

// Whether scores scale * dot can be computed under this cap (0: none) as
// cap * tanh(dot * (scale / cap)) in float32: both factors are normal numbers far
// from either end of the range (a cap of 1e37 has a scale / cap that has lost
// bits, one of 2.4e38 no finite cap * log2(e)).
inline bool softcap_ok(float cap, float scale)
{
    if (cap == 0.f)
        return true;
    if (!(cap > 0.f) || !std::isfinite(cap * 1.4426950408889634f))
        return false;
    const float f = std::fabs(scale / cap);
    return scale == 0.f || (f >= 0x1p-100f && f <= 0x1p100f);
}

// tanh of N scores (times 1 / cap), N even: an odd polynomial of degree 11
// where every score of the warp is within 0.7 -- fitted here for the least
// largest relative error of tanh(y) / y in y^2, 1.4e-8 (with its roundings
// 1.2e-7, measured) -- two scores an instruction and no special-function
// operation (the exponentials of the softmax fill that unit); elsewhere (1 - e) / (1 + e) with e = exp(-2 |y|),
// whose relative error is about 2^-22.  The hardware's tanh is not used: its
// relative error of 2^-11 would move a score of 10 under a cap of 50 by 0.005,
// and every weight with it.
// One block per warp (the branch is taken together).  A score within 0.7 gets the
// polynomial by the same operations on both sides: its result does not depend on
// the block's other scores, hidden ones among them.
template <int N>
__device__ __forceinline__ void tanh_block(float (&y)[N])
{
    constexpr float kMax = 0.7f;
    constexpr float kC[6] = {0.999999986f, -0.333331304f, 0.133284148f, -0.0535260093f, 0.0200244578f, -0.00508833599f};
    float top = 0.f;  // (a NaN gives NaN either way)
#pragma unroll
    for (int j = 0; j < N; j += 2)
        top = fmaxf(top, fmaxf(fabsf(y[j]), fabsf(y[j + 1])));
    // two loops, not a test per pair: a branch between the pairs would keep their
    // chains from overlapping
    if (!__any_sync(0xffffffffu, top > kMax)) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 v = make_float2(y[j], y[j + 1]);
            const float2 z = __fmul2_rn(v, v);
            float2 a = make_float2(kC[5], kC[5]);
#pragma unroll
            for (int e = 4; e >= 0; --e)
                a = __ffma2_rn(a, z, make_float2(kC[e], kC[e]));
            a = __fmul2_rn(a, v);
            y[j] = a.x;
            y[j + 1] = a.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float x = y[j], z = x * x;
            const float e = fast_exp2(fabsf(x) * -2.8853900817779268f);  // 2 log2(e)
            const float far = copysignf(__fdividef(1.f - e, 1.f + e), x);
            float a = kC[5];
#pragma unroll
            for (int k = 4; k >= 0; --k)
                a = fmaf(a, z, kC[k]);
            y[j] = fabsf(x) > kMax ? far : a * x;
        }
    }
}

// The same for raw dot products under a cap, out tanh(f x), with both factors in
// the polynomial's coefficients: of degree 7 for |f x| <= 0.5 (largest relative
// error 5.4e-7, 6.3e-7 with its roundings, a thousandth of the 16-bit rounding of the weights that follow),
// five operations a score.  The backward's kernels use it: they are bound by
// the arithmetic of their scores, and by the size of their code (a third path
// for factors whose powers leave float32's range cost 21 and 8 us of the two
// kernels of a capped [4, 32/8, 2048, 128] call without being run; those take
// the second one here).
struct TanhScaled {
    float2 c[4];  // c_k f^(2 k + 1) out, twice
    float f, out;
    float top;    // 0.5 / |f|; negative: never the polynomial
};

inline TanhScaled tanh_scaled(float f, float out)
{
    constexpr float kC[4] = {0.999999456f, -0.333263179f, 0.131902966f, -0.0444022255f};
    TanhScaled t{};
    t.f = f;
    t.out = out;
    const float a = f < 0.f ? -f : f, o = out < 0.f ? -out : out;
    if (!(a >= 1e-5f && a <= 1e4f && o >= 0.1f && o <= 1e6f)) {
        t.top = -1.f;
        return t;
    }
    t.top = 0.5f / a;
    float pw = f * out;  // f^7 out stays within 1e-36 and 1e34
    for (int k = 0; k < 4; ++k, pw *= f * f)
        t.c[k] = make_float2(kC[k] * pw, kC[k] * pw);
    return t;
}

template <int N>
__device__ __forceinline__ void tanh_block_scaled(float (&x)[N], const TanhScaled& t)
{
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < N; j += 2)
        top = fmaxf(top, fmaxf(fabsf(x[j]), fabsf(x[j + 1])));
    if (!__any_sync(0xffffffffu, top > t.top)) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 v = make_float2(x[j], x[j + 1]);
            const float2 z = __fmul2_rn(v, v);
            float2 a = __ffma2_rn(t.c[3], z, t.c[2]);
            a = __ffma2_rn(a, z, t.c[1]);
            a = __ffma2_rn(a, z, t.c[0]);
            a = __fmul2_rn(a, v);
            x[j] = a.x;
            x[j + 1] = a.y;
        }
    } else {
        // (1 - e) / (1 + e) with e = exp(-2 |y|); y - y^3 / 3 up to 0.05, where
        // 1 - e cancels.  Relative errors: 8.7e-7 below it; just above, where e's own
        // error counts twenty times, 2.1e-6 by the bound of the hardware's exp2 (2^-22.5)
        // and 1.1e-6 measured; 2.5e-7 from 0.5 on
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float y = x[j] * t.f;
            const float e = fast_exp2(fabsf(y) * -2.8853900817779268f);  // 2 log2(e)
            const float far = copysignf(__fdividef(1.f - e, 1.f + e), y);
            const float near = fmaf(y * y, y * -0.333333333f, y);
            x[j] = (fabsf(y) > 0.05f ? far : near) * t.out;
        }
    }
}

}  // namespace pa
