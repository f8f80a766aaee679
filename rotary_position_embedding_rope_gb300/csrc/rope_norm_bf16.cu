// rope_norm_bf16.cu -- the kernels of rope_norm.cuh for bf16 rows (one translation
// unit per element type, compiled in parallel).
#include "rope_norm.cuh"

namespace rope {

cudaError_t launch_norm_bf16(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st)
{
    return launch_norm_type<__nv_bfloat16>(a, layout, backward, st);
}

cudaError_t launch_norm_append_bf16(const NormAppendArgs &a, int32_t D, int32_t layout, cudaStream_t st)
{
    return launch_norm_append_type<__nv_bfloat16>(a, D, layout, st);
}

}  // namespace rope
