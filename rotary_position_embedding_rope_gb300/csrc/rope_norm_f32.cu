// rope_norm_f32.cu -- the kernels of rope_norm.cuh for float rows (one translation
// unit per element type, compiled in parallel).
#include "rope_norm.cuh"

namespace rope {

cudaError_t launch_norm_f32(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st)
{
    return launch_norm_type<float>(a, layout, backward, st);
}

}  // namespace rope
