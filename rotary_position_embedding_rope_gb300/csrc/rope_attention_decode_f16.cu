// rope_attention_decode_f16.cu -- the kernels of rope_attention_decode.cuh for
// f16 (one translation unit per element type, compiled in parallel).
#include "rope_attention_decode.cuh"

namespace rope {

cudaError_t launch_decode_f16(const DecodeCall &c, const DecodeLayout &lay, int32_t D, int32_t layout,
                               cudaStream_t st)
{
    return launch_decode_type<__half>(c, lay, D, layout, st);
}

}  // namespace rope
