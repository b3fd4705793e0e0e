// pa_scored.cu -- the weight that each key got in a decode with modified scores
// (include/pa_scored.h): the softmax weights of all heads and new rows, summed
// per key.
//
// The partition kernel leaves its modified scores ([segment][token][row],
// 4 bytes beside the 4 D bytes or more of the key's K and V) and the rows'
// softmax denominators; a second pass over K would cost half the decode.
// Here every key's scores are read once, 2^(score - lse) summed in a fixed
// order (no atomics: the result does not depend on the split).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_ptx.cuh"
#include "pa_vjp.cuh"

namespace pa {
namespace {

constexpr int kWThreads = 128;

// grid (token tiles, B): one thread a key.  With whole vectors of rows (R a
// multiple of 4) a key's scores of one head are 16-byte loads, the heads' loads
// in flight together.
template <bool kVec>
__global__ void __launch_bounds__(kWThreads) pa_key_weights(const __grid_constant__ KeyWeightParams p)
{
    grid_dependents_launch();
    grid_dependency_wait();
    const int b = blockIdx.y;
    const int n = min(max(__ldg(p.seq_lens + b), 0), p.cap);
    const int j = blockIdx.x * kWThreads + static_cast<int>(threadIdx.x);
    if (j >= n + p.NQ || j >= p.cap)
        return;
    const size_t at = static_cast<size_t>(b) * p.cap + j;
    const float old = p.in && j < n ? p.in[at] : 0.f;
    // the stages that the partition kernel left out
    const int pl = p.prefix ? min(max(__ldg(p.prefix + b), 0), n + p.NQ) : 0;
    const int P = (pl + p.TT - 1) & ~(p.TT - 1);
    const int lo = max(n - p.window + 1, 0) & ~(p.TT - 1);
    float w = 0.f;
    if (j < P || j >= lo) {
        const size_t seg0 = static_cast<size_t>(b) * p.KV;
        const size_t step = static_cast<size_t>(p.score_tokens) * p.R;
        const float* s = p.scores + seg0 * step + static_cast<size_t>(j) * p.R;
        const float* l = p.lse + seg0 * p.R;
        if constexpr (kVec) {
            const int n4 = p.R >> 2, total = p.KV * n4;  // vectors of the key, head by head
            constexpr int U = 8;
            for (int i0 = 0; i0 < total; i0 += U) {
                float4 a[U], c[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < total) {
                        const int kh = (i0 + u) / n4, r4 = (i0 + u) - kh * n4;
                        a[u] = __ldcg(reinterpret_cast<const float4*>(s + kh * step) + r4);
                        c[u] = __ldg(reinterpret_cast<const float4*>(l) + i0 + u);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < total)
                        w += (exp2f(a[u].x - c[u].x) + exp2f(a[u].y - c[u].y)) +
                             (exp2f(a[u].z - c[u].z) + exp2f(a[u].w - c[u].w));
            }
        } else {
            for (int kh = 0; kh < p.KV; ++kh)
                for (int r = 0; r < p.R; ++r)
                    w += exp2f(__ldcg(s + kh * step + r) - __ldg(l + kh * p.R + r));
        }
    }
    if (p.in && j < n)
        w = fmaf(p.decay, old, w);
    p.out[at] = w;
}

}  // namespace

int launch_key_weights(const KeyWeightParams& w, cudaStream_t st)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((w.cap + kWThreads - 1) / kWThreads, w.B);
    cfg.blockDim = dim3(kWThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KeyWeightParams p = w;
    void* args[1] = {&p};
    const void* fn = w.R % 4 == 0 ? reinterpret_cast<const void*>(pa_key_weights<true>)
                                  : reinterpret_cast<const void*>(pa_key_weights<false>);
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(1);
    return PA_OK;
}

}  // namespace pa
