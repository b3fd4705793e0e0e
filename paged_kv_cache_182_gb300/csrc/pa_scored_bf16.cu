// pa_scored_bf16.cu -- the partition kernels with modified scores, bf16 caches.
#include "pa_kernels.cuh"

namespace pa {

ScoredFn pick_scored_bf16(bool f32_out, int D, int MT)
{
    return f32_out ? pick_scored_mma<__nv_bfloat16, float>(D, MT) : pick_scored_mma<__nv_bfloat16, __nv_bfloat16>(D, MT);
}

}  // namespace pa
