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

// grid (token tiles, B): one thread a key.
__global__ void __launch_bounds__(kWThreads) pa_key_weights(const __grid_constant__ KeyWeightParams p)
{
    grid_dependency_wait();
    const int b = blockIdx.y;
    const int n = min(max(__ldg(p.seq_lens + b), 0), p.cap);
    const int j = blockIdx.x * kWThreads + static_cast<int>(threadIdx.x);
    if (j >= n + p.NQ || j >= p.cap)
        return;
    // the stages that the partition kernel left out
    const int pl = p.prefix ? min(max(__ldg(p.prefix + b), 0), n + p.NQ) : 0;
    const int P = (pl + p.TT - 1) & ~(p.TT - 1);
    const int lo = max(n - p.window + 1, 0) & ~(p.TT - 1);
    float w = 0.f;
    if (j < P || j >= lo) {
        for (int kh = 0; kh < p.KV; ++kh) {
            const size_t seg = static_cast<size_t>(b) * p.KV + kh;
            const float* s = p.scores + (seg * p.score_tokens + j) * p.R;
            const float* l = p.lse + seg * p.R;
            for (int r = 0; r < p.R; ++r)
                w += exp2f(__ldcs(s + r) - __ldg(l + r));
        }
    }
    const size_t at = static_cast<size_t>(b) * p.cap + j;
    if (p.in && j < n)
        w = fmaf(p.decay, p.in[at], w);
    p.out[at] = w;
}

}  // namespace

int launch_key_weights(const KeyWeightParams& w, cudaStream_t st)
{
    pa_key_weights<<<dim3((w.cap + kWThreads - 1) / kWThreads, w.B), kWThreads, 0, st>>>(w);
    if (cudaGetLastError() != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(1);
    return PA_OK;
}

}  // namespace pa
