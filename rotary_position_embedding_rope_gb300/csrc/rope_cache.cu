// rope_cache.cu -- rope_cache_append: new keys, rotated, and values written
// into the pages of a cache.
//
// Token t of sequence b (cu[b] <= t < cu[b + 1]) is the sequence's slot
// s = cache_lens[b] + t - cu[b]; it goes to row s mod page of page
// table[b][s / page].  The key is rotated with table row pos[t], or
// pos_offset + s, so the cache holds rotated keys and the attention that
// reads it rotates only its one query.
//
// What bounds it: every key and value is read once and written once, a few
// flops each: HBM bandwidth for a prompt, latency for a decode step.  A group
// of D / 16 lanes owns four heads of one token: its 16 loads of 16 bytes are
// issued before anything else, so the search for the sequence, the page and
// the table row (dependent loads) hides behind them, and the cos/sin values
// are read once for the four heads.
#include "rope_rows.cuh"
#include "rope_serving.cuh"

namespace rope {

constexpr int kRowThreads = 128;
constexpr int kRowHeads = 4;                   // heads of a token per lane group
constexpr int kCuCached = 1024;                // sequence offsets kept in shared memory

template <typename T, int LAYOUT, int D>
__global__ void __launch_bounds__(kRowThreads) rope_cache_append_kernel(const RowsArgs a)
{
    constexpr int L = D / 16;                  // lanes of a group
    constexpr int kGroups = kRowThreads / L;
    __shared__ int32_t s_cu[kCuCached];
    const int tid = threadIdx.x, j = tid % L;
    const int32_t chunks = (a.Hk + kRowHeads - 1) / kRowHeads;
    const int64_t unit = (int64_t)blockIdx.x * kGroups + tid / L;
    const int64_t t = unit / chunks;
    const int32_t h0 = (int32_t)(unit - t * chunks) * kRowHeads;
    const bool live = t < a.total;
    const RowPart part = row_part<LAYOUT>(j, a.rotary_dim);

    pdl_wait();
    pdl_trigger();
    uint4 k0[kRowHeads], k1[kRowHeads], v0[kRowHeads], v1[kRowHeads];
    const T *ks = static_cast<const T *>(a.k) + t * a.k_stride;
    const T *vs = static_cast<const T *>(a.v) + t * a.v_stride;
#pragma unroll
    for (int i = 0; i < kRowHeads; ++i) {
        if (live && h0 + i < a.Hk) {
            const int32_t h = (h0 + i) * D;
            k0[i] = __ldcs(reinterpret_cast<const uint4 *>(ks + h + part.o0));
            k1[i] = __ldcs(reinterpret_cast<const uint4 *>(ks + h + part.o1));
            v0[i] = __ldcs(reinterpret_cast<const uint4 *>(vs + h + part.o0));
            v1[i] = __ldcs(reinterpret_cast<const uint4 *>(vs + h + part.o1));
        }
    }
    // the token's sequence
    const bool cached = a.n_seqs + 1 <= kCuCached;
    if (cached) {
        for (int32_t i = tid; i <= a.n_seqs; i += kRowThreads)
            s_cu[i] = __ldg(a.cu + i);
        __syncthreads();
    }
    const int32_t *cu = cached ? s_cu : a.cu;
    if (blockIdx.x == 0) {                     // the offsets themselves: 0 <= cu[i] <= cu[i + 1] <= total
        bool bad = false;
        for (int32_t i = tid; i < a.n_seqs; i += kRowThreads)
            bad = bad || cu[i] < 0 || cu[i] > cu[i + 1] || cu[i + 1] > a.total;
        if (bad)
            atomicOr(a.flag, kFlagIndex);
    }
    if (!live)
        return;
    const int32_t b = find_sequence(cu, a.n_seqs, t);
    const int32_t start = cu[b];
    if (t < start || t >= cu[b + 1])
        return;                                // a row of no sequence: nothing to write
    const int64_t have = __ldg(a.cache_lens + b);
    const int64_t slot = have + (t - start);
    const int64_t block = slot >> a.page_shift;
    int64_t page = -1;
    if (have >= 0 && block < a.table_stride)
        page = __ldg(a.table + b * a.table_stride + block);
    if (page < 0 || page >= a.n_pages) {
        if (j == 0)
            atomicOr(a.flag, kFlagIndex);
        return;
    }
    int64_t row = a.pos != nullptr ? (int64_t)__ldg(a.pos + t) : a.pos_offset + slot;
    if (row < 0 || row >= a.table_rows) {
        if (j == 0 && !(a.pos != nullptr && row == -1))
            atomicOr(a.flag, kFlagPosition);
        row = -1;                              // not rotated
    }
    if (part.rot && row >= 0) {
        float c[8], s[8];
        table_values(a.cos, a.sin, row * (a.rotary_dim / 2) + 8 * j, c, s);
#pragma unroll
        for (int i = 0; i < kRowHeads; ++i)
            if (h0 + i < a.Hk)
                rotate_part<T, LAYOUT>(k0[i], k1[i], c, s);
    }
    const int64_t in_page = slot & (((int64_t)1 << a.page_shift) - 1);
    T *kp = static_cast<T *>(a.k_out), *vp = static_cast<T *>(a.v_out);
#pragma unroll
    for (int i = 0; i < kRowHeads; ++i) {
        if (h0 + i < a.Hk) {
            const int64_t at = (((page * a.Hk + h0 + i) << a.page_shift) + in_page) * D;
            __stcs(reinterpret_cast<uint4 *>(kp + at + part.o0), k0[i]);
            __stcs(reinterpret_cast<uint4 *>(kp + at + part.o1), k1[i]);
            __stcs(reinterpret_cast<uint4 *>(vp + at + part.o0), v0[i]);
            __stcs(reinterpret_cast<uint4 *>(vp + at + part.o1), v1[i]);
        }
    }
}

template <typename T, int LAYOUT, int D>
static cudaError_t append_t(const RowsArgs &a, cudaStream_t st)
{
    const int64_t chunks = (a.Hk + kRowHeads - 1) / kRowHeads;
    const int64_t groups = kRowThreads / (D / 16);
    const int64_t blocks = (a.total * chunks + groups - 1) / groups;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    return launch_hot(rope_cache_append_kernel<T, LAYOUT, D>, dim3((unsigned)blocks), dim3(kRowThreads), 0, st, a);
}

template <typename T>
static cudaError_t append_d(const RowsArgs &a, int32_t D, int32_t layout, cudaStream_t st)
{
    if (layout == 0)
        return D == 64 ? append_t<T, 0, 64>(a, st) : append_t<T, 0, 128>(a, st);
    return D == 64 ? append_t<T, 1, 64>(a, st) : append_t<T, 1, 128>(a, st);
}

cudaError_t launch_cache_append(const RowsArgs &a, int32_t D, int32_t layout, int32_t dtype,
                                cudaStream_t st)
{
    return dtype == 1 ? append_d<__nv_bfloat16>(a, D, layout, st)
                      : append_d<__half>(a, D, layout, st);
}

}  // namespace rope
