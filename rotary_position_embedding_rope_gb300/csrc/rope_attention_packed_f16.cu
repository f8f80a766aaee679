// rope_attention_packed_f16.cu -- the kernels of rope_attention_packed.cuh for
// f16 (one translation unit per element type, compiled in parallel).
#include "rope_attention_packed.cuh"

namespace rope {

cudaError_t launch_packed_f16(const PackedArgs &c, const PackedLayout &lay, int32_t D, int32_t layout,
                               cudaStream_t st)
{
    return launch_packed_type<__half>(c, lay, D, layout, st);
}

}  // namespace rope
