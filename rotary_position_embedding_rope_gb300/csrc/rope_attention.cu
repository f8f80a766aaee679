// rope_attention.cu -- the attention entry point of librope without an
// attn_mask (the kernels of rope_attention.cuh instantiated with MASK = false;
// rope_attention_masked.cu holds the masked ones, compiled in parallel), and
// the probe of the bounded-wait expiry path.
#include "rope_attention.cuh"

namespace rope {

cudaError_t launch_attention(const AttnArgs &a, int32_t D, int32_t layout, int32_t dtype,
                             cudaStream_t st)
{
    if (a.mask_kind != 0)
        return launch_attention_masked(a, D, layout, dtype, st);
    return launch_attention_t<false>(a, D, layout, dtype, st);
}

// Probe of the expiry path: a thread and a warp wait, one with each of the
// attention kernels' bounded waits, on a barrier that nothing arrives at: for
// `cycles` clock cycles, and for as many tries as those should last.  When both
// have given up, the counted wait no sooner than after an eighth of the cycles (one
// that did would cut real waits short), a thread records the expiry as those
// kernels do (bit 1 of the device flag).  Nothing else runs, so nothing stalls.
constexpr long long kTryCycles = 8000;         // of a failed try: 4.05 us, 7964 cycles
__global__ void rope_wait_probe_kernel(int32_t *flag, long long cycles)
{
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort = 0;
    }
    __syncthreads();
    bool expired = true;
    if (threadIdx.x == 0) {
        expired = !attn_wait(&bar, 0u, nullptr, cycles);
    } else if (threadIdx.x >= 32) {            // (together, as the roles wait)
        const long long tries = cycles / kTryCycles + 1, t0 = clock64();
        expired = !role_wait(&bar, 0u, &abort, (int)(tries < kRoleTries ? tries : kRoleTries)) &&
                  clock64() - t0 >= cycles / 8;
    }
    expired = __syncthreads_and(expired);
    if (threadIdx.x == 0 && expired)
        atomicOr(flag, 2);
}

cudaError_t launch_wait_probe(int32_t *flag, long long cycles, cudaStream_t st)
{
    rope_wait_probe_kernel<<<1, 64, 0, st>>>(flag, cycles);
    return cudaGetLastError();
}


}  // namespace rope
