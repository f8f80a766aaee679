// rope_norm_f16.cu -- the kernels of rope_norm.cuh for fp16 rows (one translation
// unit per element type, compiled in parallel).
#include "rope_norm.cuh"

namespace rope {

cudaError_t launch_norm_f16(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st)
{
    return launch_norm_type<__half>(a, layout, backward, st);
}

cudaError_t launch_norm_append_f16(const NormAppendArgs &a, int32_t D, int32_t layout, cudaStream_t st)
{
    return launch_norm_append_type<__half>(a, D, layout, st);
}

}  // namespace rope
