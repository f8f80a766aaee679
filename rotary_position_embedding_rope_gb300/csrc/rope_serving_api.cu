// rope_serving_api.cu -- the C ABI of the serving operators (include/rope.h):
// argument checks.  Everything the host can see is checked here, before
// anything is enqueued; offsets, lengths and page numbers are checked by the
// kernels.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include <cuda_runtime.h>

#include "rope.h"
#include "rope_serving.cuh"

namespace rope {
namespace {

struct Range {
    const void *p;
    int64_t bytes;
};

bool overlap(const Range &a, const Range &b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a * b * ... of non-negative sizes, or -1 on overflow (or a -1 among them)
int64_t product(std::initializer_list<int64_t> xs)
{
    int64_t r = 1;
    for (int64_t x : xs)
        if (r < 0 || x < 0 || __builtin_mul_overflow(r, x, &r))
            return -1;
    return r;
}

// Bytes from the first to the last element of a [total, H, D] view with the
// given token stride, 16-bit elements; -1 on overflow.
int64_t view_bytes(int64_t total, int64_t stride, int64_t row)
{
    if (total == 0)
        return 0;
    const int64_t lead = product({total - 1, stride});
    int64_t n = 0;
    if (lead < 0 || row < 0 || __builtin_add_overflow(lead, row, &n))
        return -1;
    return product({n, 2});
}

rope_status check_shape(int32_t dtype, int32_t layout, int32_t D, int32_t rotary_dim)
{
    if (dtype != ROPE_BF16 && dtype != ROPE_F16)
        return ROPE_ERR_UNSUPPORTED;
    if (layout != ROPE_SPLIT_HALF && layout != ROPE_INTERLEAVED)
        return ROPE_ERR_UNSUPPORTED;
    if (D != 64 && D != 128)
        return ROPE_ERR_UNSUPPORTED;
    if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 != 0)
        return ROPE_ERR_UNSUPPORTED;
    return ROPE_OK;
}

// log2 of a supported page size, else -1
int32_t page_shift(int32_t page_size)
{
    for (int32_t s = 4; s <= 7; ++s)
        if (page_size == 1 << s)
            return s;
    return -1;
}

constexpr int64_t kMaxInt32 = 0x7fffffff;

}  // namespace
}  // namespace rope

using namespace rope;

extern "C" {

rope_status rope_cache_append(const void *k, const void *v, void *k_pages, void *v_pages,
                              const int32_t *block_table, const int32_t *cu_seqlens,
                              const int32_t *cache_lens, const float *cos, const float *sin,
                              const int32_t *pos, int64_t pos_offset, int64_t n_seqs,
                              int64_t total, int64_t k_stride, int64_t v_stride, int32_t Hk,
                              int32_t D, int32_t rotary_dim, int32_t layout, int32_t page_size,
                              int64_t n_pages, int64_t max_blocks, int32_t dtype,
                              int64_t table_rows, void *stream)
{
    rope_status st = check_shape(dtype, layout, D, rotary_dim);
    if (st != ROPE_OK)
        return st;
    const int32_t shift = page_shift(page_size);
    if (shift < 0)
        return ROPE_ERR_UNSUPPORTED;
    if (n_seqs < 0 || n_seqs >= kMaxInt32 || total < 0 || total > kMaxInt32 || Hk < 0 ||
        n_pages < 0 || n_pages > kMaxInt32 || max_blocks < 0 || table_rows < 0 || pos_offset < 0 ||
        pos_offset > kMaxInt32)
        return ROPE_ERR_INVALID_ARG;
    const int64_t row = (int64_t)Hk * D;
    if (k_stride < row || v_stride < row)
        return ROPE_ERR_INVALID_ARG;
    const int64_t kb = view_bytes(total, k_stride, row), vb = view_bytes(total, v_stride, row);
    const int64_t pool = product({n_pages, Hk, page_size, D, 2});
    const int64_t tab = product({table_rows, rotary_dim / 2, 4});
    const int64_t blocks = product({n_seqs, max_blocks, 4});
    if (kb < 0 || vb < 0 || pool < 0 || tab < 0 || blocks < 0)
        return ROPE_ERR_INVALID_ARG;
    if (total == 0 || n_seqs == 0 || Hk == 0)
        return ROPE_OK;
    if (!k || !v || !cu_seqlens || !cache_lens || !cos || !sin || table_rows < 1 || n_pages < 1 ||
        max_blocks < 1 || !k_pages || !v_pages || !block_table)
        return ROPE_ERR_INVALID_ARG;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(cos, 16) || !aligned(sin, 16))
        return ROPE_ERR_UNSUPPORTED;
    if (!aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(cache_lens, 4) ||
        !aligned(pos, 4))
        return ROPE_ERR_INVALID_ARG;
    const Range outs[2] = {{k_pages, pool}, {v_pages, pool}};
    const Range ins[8] = {{k, kb}, {v, vb}, {block_table, blocks}, {cu_seqlens, 4 * (n_seqs + 1)},
                          {cache_lens, 4 * n_seqs}, {cos, tab}, {sin, tab}, {pos, 4 * total}};
    if (overlap(outs[0], outs[1]))
        return ROPE_ERR_INVALID_ARG;
    for (const Range &o : outs)
        for (const Range &i : ins)
            if (overlap(o, i))
                return ROPE_ERR_INVALID_ARG;
    RowsArgs a;
    std::memset(&a, 0, sizeof a);
    a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride;
    a.k_out = k_pages; a.v_out = v_pages;
    a.cu = cu_seqlens; a.pos = pos; a.cos = cos; a.sin = sin;
    a.table_rows = table_rows; a.total = total;
    a.n_seqs = (int32_t)n_seqs; a.Hk = Hk; a.rotary_dim = rotary_dim;
    a.table = block_table; a.cache_lens = cache_lens; a.table_stride = max_blocks;
    a.n_pages = n_pages; a.page_shift = shift; a.pos_offset = pos_offset;
    if (device_flag(&a.flag) != cudaSuccess)
        return ROPE_ERR_CUDA;
    return launch_cache_append(a, D, layout, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ROPE_OK
               : ROPE_ERR_CUDA;
}

}  // extern "C"
