// pa_vjp.cuh -- shared declarations of the attention backward kernels
// (pa_vjp.cu: checks, CUDA-core kernels, dispatch; pa_vjp_tc.cu: tcgen05
// kernels).
#pragma once

#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "pa_tanh.cuh"

namespace pa {

constexpr float kVjpLog2e = 1.4426950408889634f;
// Row statistics (lse2, delta) of each (batch, query head) start at a
// multiple of this many rows, so a 128-row tile of them is one aligned copy.
constexpr int kVjpRowPad = 128;

struct VjpParams {
    const void* q;
    const void* k;
    const void* v;
    const void* y;
    const void* g;
    const void* mask;
    void* dq;
    void* dk;
    void* dv;
    float* lse;     // [B][HQ][sqp] log2 of the softmax denominator, +inf on empty rows
    float* delta;   // [B][HQ][sqp] rowsum(y * g)
    float* dq_acc;  // [B][HQ][SQ][D] float32 dq accumulator; NULL when dq itself is float32
    float* dq_sum;  // where dq is accumulated: dq_acc, or dq when it is float32
    int* status;
    unsigned long long wait_ns;
    int B, HQ, HK, SQ, SK, D, groups, sqp, causal, mask_kind;
    int md[4];  // mask dims MB, MH, MQ, W
    float scale, scale_log2;
};

// Modified scores (pa_attention_vjp_scored):
//   t = scale q.k; under a cap t = cap tanh(t / cap); t -= slopes[h] |i - j|;
//   key j visible to row i when j < prefix[b], or within the causal rule and
//   |i - j| < window.
// The cap leaves the factor 1 - tanh^2 on ds; bias and masks leave none.
struct VjpScoredParams : VjpParams {
    const float* slopes;    // [HQ], or NULL
    const int32_t* prefix;  // [B], or NULL
    float cap_in, cap_out;  // scale / cap, cap * log2(e); 0 without a cap
    TanhScaled tanh, tanh_cap;  // of cap_in; the same times cap_out
    int bounded;            // a cap of at most 69 and no slopes: 2^|score| needs no maximum taken off
    int window;             // INT_MAX: none
    // tensor cores, split: one CTA per query head instead of per group, its dk and
    // dv in part[0] and part[1] [groups][B][HK][SK][D], summed in group order after
    int split;
    float* part[2];
};

template <int kMod>
using VjpParamsOf = std::conditional_t<kMod != 0, VjpScoredParams, VjpParams>;

// Keys below are visible to every row of sequence b.
__device__ __forceinline__ int vjp_prefix(const VjpScoredParams& p, int b)
{
    return p.prefix ? min(max(__ldg(p.prefix + b), 0), p.SK) : 0;
}

__device__ __forceinline__ bool vjp_seen(const VjpScoredParams& p, int pl, int i, int j)
{
    return j < pl || ((!p.causal || j <= i) && abs(i - j) < p.window);
}

// Additive bias of score (b, h, i, j) in natural-log units: the causal rule
// (key j hidden from row i when j > i), then the mask (boolean: 0 or -inf;
// additive: the value; keys at or past a width W > 1 hidden).
__device__ __forceinline__ float vjp_bias(const VjpParams& p, int b, int h, int i, int j, bool causal)
{
    if (causal && j > i)
        return -INFINITY;
    if (p.mask_kind == 0)
        return 0.f;
    int jj = 0;
    if (p.md[3] != 1) {
        if (j >= p.md[3])
            return -INFINITY;
        jj = j;
    }
    const int64_t idx =
        ((static_cast<int64_t>(p.md[0] == 1 ? 0 : b) * p.md[1] + (p.md[1] == 1 ? 0 : h)) * p.md[2] +
         (p.md[2] == 1 ? 0 : i)) * p.md[3] + jj;
    if (p.mask_kind == 1)
        return static_cast<const uint8_t*>(p.mask)[idx] ? 0.f : -INFINITY;
    return static_cast<const float*>(p.mask)[idx];
}

// Tensor-core path (pa_vjp_tc.cu): whether these sizes take it, and its
// launches (row statistics and the backward; dq rounding is left to the
// caller).  Returns PA_OK or a PA_ERR_* code.
bool vjp_tc_supported(int dtype, int D, int groups, int mask_kind);
int launch_vjp_tc(const VjpParams& p, int dtype, bool f32_out, cudaStream_t st, uint64_t* launches);
int launch_vjp_tc_scored(const VjpScoredParams& p, int dtype, bool f32_out, cudaStream_t st, uint64_t* launches);
// Whether that launch splits its groups (VjpScoredParams::split) on a device of `sms`.
bool vjp_tc_splits(int B, int HQ, int HK, int SK, int sms);

// Adds to the library's count of kernel launches (pa_kernel_launches).
void count_launches(uint64_t n);

// Lets `fn` have as much dynamic shared memory on the current device as a block may
// opt in to: the same limit whatever a call needs, so that no call of another host
// thread lowers it between this one and its launch.
bool allow_shared_memory(const void* fn);

}  // namespace pa
