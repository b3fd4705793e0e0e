// pa_scored_f16.cu -- the partition kernels with modified scores, f16 caches.
#include "pa_kernels.cuh"

namespace pa {

ScoredFn pick_scored_f16(bool f32_out, int D, int MT)
{
    return f32_out ? pick_scored_mma<__half, float>(D, MT) : pick_scored_mma<__half, __half>(D, MT);
}

}  // namespace pa
