// rope_attention_paged_bf16.cu -- the kernels of rope_attention_paged.cuh for bf16
// (one translation unit per element type, compiled in parallel).
#include "rope_attention_paged.cuh"

namespace rope {

cudaError_t launch_paged_bf16(const PagedCall &c, const PagedLayout &lay, int32_t D, int32_t layout,
                              cudaStream_t st)
{
    return launch_paged_type<__nv_bfloat16>(c, lay, D, layout, st);
}

}  // namespace rope
