// pa_tanh.cuh -- tanh of a thread's block of capped scores.
#pragma once

#include <cuda_runtime.h>

#include "pa_ptx.cuh"

namespace pa {

// y *= f, two an instruction.
template <int N>
__device__ __forceinline__ void scale_block(float (&y)[N], float f)
{
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const float2 r = __fmul2_rn(make_float2(y[j], y[j + 1]), make_float2(f, f));
        y[j] = r.x;
        y[j + 1] = r.y;
    }
}

// tanh of N scores (times 1 / cap), N even: an odd polynomial of degree 11
// where every score of the warp is within 0.7 -- fitted here for the least
// largest relative error of tanh(y) / y in y^2, 1.4e-8 -- two scores an
// instruction and no special-function operation (the exponentials of the
// softmax fill that unit); elsewhere (1 - e) / (1 + e) with e = exp(-2 |y|),
// whose relative error is about 2^-22.  The hardware's tanh is not used: its
// relative error of 2^-11 would move a score of 10 under a cap of 50 by 0.005,
// and every weight with it.
// One block per warp (the branch is taken together).
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

}  // namespace pa
