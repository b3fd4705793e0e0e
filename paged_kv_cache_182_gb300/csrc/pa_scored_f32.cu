// pa_scored_f32.cu -- the partition kernels with modified scores, float32 caches.
#include "pa_kernels.cuh"

namespace pa {

ScoredFn pick_scored_f32(int D) { return pick_scored_simt<float, float>(D); }

}  // namespace pa
