// rope_attention_paged_f16.cu -- the kernels of rope_attention_paged.cuh for fp16
// (one translation unit per element type, compiled in parallel).
#include "rope_attention_paged.cuh"

namespace rope {

cudaError_t launch_paged_f16(const PagedCall &c, const PagedLayout &lay, int32_t D, int32_t layout,
                              cudaStream_t st)
{
    return launch_paged_type<__half>(c, lay, D, layout, st);
}

}  // namespace rope
