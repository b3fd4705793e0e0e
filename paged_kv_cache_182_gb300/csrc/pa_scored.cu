// pa_scored.cu -- the weight that each key got in a decode with modified scores
// (include/pa_scored.h): the softmax weights of all heads and new rows, summed
// per key.
//
// The partition kernel leaves its modified scores ([segment][token][row],
// 4 bytes beside the 4 D bytes or more of the key's K and V) and the rows'
// softmax denominators; a second pass over K would cost half the decode.
// Here every key's scores are read once, 2^(score - lse) summed in a fixed
// order (no atomics; the denominators' own sums do go by the split).  Bound by
// latency after the decode's last CTA: about 4 us of a call (B = 8, 512-4096
// tokens, 32 heads: 25.3 us without the weights, 29 with; 32768 tokens: 34.8
// and 39.7).
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

// grid (CTAs a sequence, B): tiles of keys dealt to a sequence's CTAs, as many
// as it has (a table may hold far more tokens than a sequence); L threads a
// key, each a share of its rows, in vectors of four where R is whole vectors;
// the heads' loads are in flight together.
template <bool kVec, int L>
__global__ void __launch_bounds__(kWThreads) pa_key_weights(const __grid_constant__ KeyWeightParams p)
{
    // in this order: a kernel that is let off here may read its inputs before this one
    // has ended (pa_opts.inputs_unchanged), and the partition kernel's out be among them
    grid_dependency_wait();
    grid_dependents_launch();
    constexpr int W = kVec ? 4 : 1, U = 4, KEYS = kWThreads / L;
    const int b = blockIdx.y;
    const int n = min(max(__ldg(p.seq_lens + b), 0), p.cap);
    const int end = min(n + p.NQ, p.cap);
    const int sub = static_cast<int>(threadIdx.x) % L;
    // the stages that the partition kernel left out
    const int pl = p.prefix ? min(max(__ldg(p.prefix + b), 0), n + p.NQ) : 0;
    const int P = (pl + p.TT - 1) & ~(p.TT - 1);
    const int lo = max(n - p.window + 1, 0) & ~(p.TT - 1);
    const size_t seg0 = static_cast<size_t>(b) * p.KV;
    const size_t step = static_cast<size_t>(p.score_tokens) * p.R;
    const float* l = p.lse + seg0 * p.R;
    const int per = p.R / W, total = p.KV * per;  // (vectors of) rows of a key, head by head
    for (int j0 = blockIdx.x * KEYS; j0 < end; j0 += gridDim.x * KEYS) {
        const int j = j0 + static_cast<int>(threadIdx.x) / L;
        const size_t at = static_cast<size_t>(b) * p.cap + j;
        const float old = p.in && sub == 0 && j < n ? p.in[at] : 0.f;
        float w = 0.f;
        if (j < end && (j < P || j >= lo)) {
            const float* s = p.scores + seg0 * step + static_cast<size_t>(j) * p.R;
            for (int i0 = sub; i0 < total; i0 += U * L) {
                float a[U][W], c[U][W];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * L;
                    if (i < total) {
                        const int kh = i / per, r = i - kh * per;
                        const float* x = s + kh * step + r * W;
                        if constexpr (kVec) {
                            *reinterpret_cast<float4*>(a[u]) = __ldcg(reinterpret_cast<const float4*>(x));
                            *reinterpret_cast<float4*>(c[u]) = __ldg(reinterpret_cast<const float4*>(l) + i);
                        } else {
                            a[u][0] = __ldcg(x);
                            c[u][0] = __ldg(l + i);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u * L < total) {
#pragma unroll
                        for (int e = 0; e < W; ++e)
                            w += exp2f(a[u][e] - c[u][e]);
                    }
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
            w += __shfl_xor_sync(0xffffffffu, w, o);
        if (j < end && sub == 0)
            p.out[at] = p.in && j < n ? fmaf(p.decay, old, w) : w;
    }
}

}  // namespace

int launch_key_weights(const KeyWeightParams& w, cudaStream_t st)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    // a few loads a thread: 32 heads on 8 KV heads (8 loads a key) took 28.7 us with
    // the decode on four threads a key, 31.7 on one
    const bool vec = w.R % 4 == 0;
    const long long loads = static_cast<long long>(w.KV) * (vec ? w.R / 4 : w.R);
    const int L = loads <= 4 ? 1 : loads <= 16 ? 4 : 16;
    const int keys = kWThreads / L;
    const int tiles = (w.cap + keys - 1) / keys, most = (152 * 16 + w.B - 1) / w.B;
    cfg.gridDim = dim3(tiles < most ? tiles : most, w.B);
    cfg.blockDim = dim3(kWThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KeyWeightParams p = w;
    void* args[1] = {&p};
    using Fn = void (*)(KeyWeightParams);
    const Fn fn1 = vec ? pa_key_weights<true, 1> : pa_key_weights<false, 1>;
    const Fn fn4 = vec ? pa_key_weights<true, 4> : pa_key_weights<false, 4>;
    const Fn fn16 = vec ? pa_key_weights<true, 16> : pa_key_weights<false, 16>;
    const void* fn = reinterpret_cast<const void*>(L == 1 ? fn1 : L == 4 ? fn4 : fn16);
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess)
        return PA_ERR_CUDA;
    count_launches(1);
    return PA_OK;
}

}  // namespace pa
