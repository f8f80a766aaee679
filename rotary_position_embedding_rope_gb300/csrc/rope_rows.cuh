// rope_rows.cuh -- rows of packed sequences: which sequence a token belongs
// to, and the rotation of a head row by a group of D / 16 lanes.  Shared by
// the kernels that write rotated keys (rope_cache.cu, the prepare kernel of
// rope_attention_packed.cuh) and the decode kernels' queries
// (rope_attention_decode.cuh).
#pragma once

#include <cuda_runtime.h>

#include "rope_kernels.cuh"

namespace rope {

// Bits of the device flag word.
constexpr int32_t kFlagPosition = 1;           // position outside the table
constexpr int32_t kFlagTimeout = 2;            // a bounded wait expired
constexpr int32_t kFlagIndex = 4;              // sequence offset, length or page out of range

// The sequence of token t: the last b in [0, n) with cu[b] <= t (0 when there
// is none).  Ends after log2(n) steps whatever cu holds; the caller checks
// that t really lies in [cu[b], cu[b + 1]).
__device__ __forceinline__ int32_t find_sequence(const int32_t *cu, int32_t n, int64_t t)
{
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The part of a head row of D features that lane j of D / 16 owns: two
// 16-byte vectors at element offsets o0 and o1.  rot: a rotated pair of
// vectors, whose eight cos and sin values start at table column 8 j in either
// layout (split-half: vector j of each half of the span; interleaved: vectors
// 2j and 2j + 1); otherwise two vectors past the rotary span, copied.
struct RowPart {
    int32_t o0, o1;
    bool rot;
};

template <int LAYOUT>
__device__ __forceinline__ RowPart row_part(int j, int rotary_dim)
{
    RowPart p;
    p.rot = 16 * j < rotary_dim;
    if (LAYOUT == 0 && p.rot) {
        p.o0 = 8 * j;
        p.o1 = rotary_dim / 2 + 8 * j;
    } else {
        p.o0 = 16 * j;
        p.o1 = 16 * j + 8;
    }
    return p;
}

// Eight cos and eight sin values of a table, from element `at` (a multiple of 8).
__device__ __forceinline__ void table_values(const float *cos, const float *sin, int64_t at, float (&c)[8],
                                             float (&s)[8])
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(cos + at) + q);
        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(sin + at) + q);
        c[4 * q] = c4.x; c[4 * q + 1] = c4.y; c[4 * q + 2] = c4.z; c[4 * q + 3] = c4.w;
        s[4 * q] = s4.x; s[4 * q + 1] = s4.y; s[4 * q + 2] = s4.z; s[4 * q + 3] = s4.w;
    }
}

// Rotates the two vectors of a RowPart with rot set.
template <typename T, int LAYOUT>
__device__ __forceinline__ void rotate_part(uint4 &x0, uint4 &x1, const float (&c)[8],
                                            const float (&s)[8])
{
    float f0[8], f1[8];
    Elt<T>::unpack(x0, f0);
    Elt<T>::unpack(x1, f1);
    if constexpr (LAYOUT == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            rotate_pair(f0[e], f1[e], c[e], s[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            rotate_pair(f0[2 * e], f0[2 * e + 1], c[e], s[e]);
            rotate_pair(f1[2 * e], f1[2 * e + 1], c[4 + e], s[4 + e]);
        }
    }
    x0 = Elt<T>::pack(f0);
    x1 = Elt<T>::pack(f1);
}

}  // namespace rope
