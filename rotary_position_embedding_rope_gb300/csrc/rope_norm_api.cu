// rope_norm_api.cu -- the C ABI of the norm of query and key heads with the
// rotation in the same pass (include/rope.h): argument checks.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "rope.h"
#include "rope_checks.h"
#include "rope_norm_internal.cuh"

namespace rope {
namespace {

struct Sizes {
    int64_t B, S, pos_stride, table_rows;
    int32_t D, rotary_dim, layout, seq_before_head, dtype, weight_dtype;
    float eps;
    int64_t size() const { return dtype == ROPE_F32 ? 4 : 2; }
};

rope_status check_sizes(const Sizes &z)
{
    if ((z.dtype != ROPE_F32 && z.dtype != ROPE_BF16 && z.dtype != ROPE_F16) ||
        (z.weight_dtype != ROPE_F32 && z.weight_dtype != z.dtype) ||
        (z.layout != ROPE_SPLIT_HALF && z.layout != ROPE_INTERLEAVED))
        return ROPE_ERR_UNSUPPORTED;
    if (z.D < 16 || z.D > 256 || z.D % 16 != 0 || z.rotary_dim < 16 || z.rotary_dim > z.D || z.rotary_dim % 16 != 0)
        return ROPE_ERR_UNSUPPORTED;
    if (z.B < 0 || z.S < 0 || z.pos_stride < 0 || z.table_rows < 0 || (z.seq_before_head != 0 && z.seq_before_head != 1) ||
        !(z.eps >= 0.0f) || !std::isfinite(z.eps))
        return ROPE_ERR_INVALID_ARG;
    const int64_t tokens = product({z.B, z.S});
    if (tokens < 0 || tokens > kMaxInt32)
        return ROPE_ERR_INVALID_ARG;
    return ROPE_OK;
}

// Bytes between the first and the last element of a [B, S, H, D] view with
// strides of batch, token and head; -1 on overflow or a stride that is negative
// or (for more than one entry) zero.
int64_t view4_bytes(const Sizes &z, int64_t H, const int64_t (&st)[3])
{
    const int64_t n[3] = {z.B, z.S, H};
    int64_t at = z.D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1)
            continue;
        const int64_t lead = st[i] > 0 ? product({n[i] - 1, st[i]}) : -1;
        if (lead < 0 || __builtin_add_overflow(at, lead, &at))
            return -1;
    }
    return product({at, z.size()});
}

// Strides of a dense tensor, [B, S, H, D] or [B, H, S, D].
void dense_strides(const Sizes &z, int64_t H, int64_t (&st)[3])
{
    st[0] = z.S * H * z.D;
    st[1] = z.seq_before_head ? H * z.D : z.D;
    st[2] = z.seq_before_head ? z.D : z.S * z.D;
}

// Fills one tensor and its ranges; in: x, weights (and the gradient), out: y (and dw).
struct Tensor {
    const void *x, *g, *w;
    void *y, *dw;
    int32_t heads;
    const int64_t *strides;
};

rope_status check_tensor(const Sizes &z, const Tensor &in, bool backward, NormTensor *t, Range (&ins)[3], Range (&outs)[2])
{
    std::memset(t, 0, sizeof *t);
    t->x = in.x; t->g = in.g; t->w = in.w; t->y = in.y; t->dw = in.dw; t->heads = in.heads;
    dense_strides(z, in.heads, t->ys);
    for (int i = 0; i < 3; ++i)
        t->xs[i] = in.strides != nullptr ? in.strides[i] : t->ys[i];
    const int64_t dense = product({z.B, z.S, in.heads, z.D, z.size()}), wide = view4_bytes(z, in.heads, t->xs);
    const int64_t wb = z.D * (z.weight_dtype == ROPE_F32 ? 4 : 2);
    if (dense < 0 || wide < 0)
        return ROPE_ERR_INVALID_ARG;
    const int64_t n[3] = {z.B, z.S, in.heads};
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1)
            t->xs[i] = 0;                      // never used
        if (t->xs[i] * z.size() % 16 != 0)
            return ROPE_ERR_UNSUPPORTED;
    }
    if (in.x == nullptr || in.y == nullptr || (backward && in.g == nullptr))
        return ROPE_ERR_INVALID_ARG;
    if (!aligned(in.x, 16) || !aligned(in.g, 16) || !aligned(in.y, 16) || !aligned(in.w, 16) || !aligned(in.dw, 4))
        return ROPE_ERR_UNSUPPORTED;
    ins[0] = {in.x, wide};
    ins[1] = {in.g, dense};
    ins[2] = {in.w, wb};
    outs[0] = {in.y, dense};
    outs[1] = {in.dw, wb};
    return ROPE_OK;
}

bool same_strides(const Sizes &z, const NormTensor &t)
{
    const int64_t n[3] = {z.B, z.S, t.heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && t.xs[i] != t.ys[i])
            return false;
    return true;
}

rope_status norm_call(const Sizes &z, const Tensor (&in)[2], const float *cos, const float *sin, const int32_t *pos,
                      bool backward, void *workspace, int64_t workspace_bytes, cudaStream_t st)
{
    rope_status e = check_sizes(z);
    if (e != ROPE_OK)
        return e;
    if (in[0].heads < 0 || in[1].heads < 0 || workspace_bytes < 0)
        return ROPE_ERR_INVALID_ARG;
    const int64_t tokens = z.B * z.S, tab = product({z.table_rows, z.rotary_dim / 2, 4});
    if (tab < 0 || (pos != nullptr && z.pos_stride != 0 && z.pos_stride < z.S))
        return ROPE_ERR_INVALID_ARG;
    const bool sums = backward && (in[0].dw != nullptr || in[1].dw != nullptr);
    const int64_t heads = (int64_t)in[0].heads + in[1].heads;
    if ((heads == 0 || tokens == 0) && !sums)
        return ROPE_OK;
    NormArgs a;
    std::memset(&a, 0, sizeof a);
    Range ins[2][3] = {}, outs[2][2] = {};
    for (int i = 0; i < 2; ++i) {
        if (in[i].heads == 0 || tokens == 0) { // no rows: dw alone is written, zeros
            const int64_t wb = z.D * (z.weight_dtype == ROPE_F32 ? 4 : 2);
            a.t[i].dw = in[i].dw;
            a.t[i].heads = in[i].heads;
            if (!aligned(in[i].dw, 4))
                return ROPE_ERR_UNSUPPORTED;
            ins[i][2] = {in[i].w, wb};
            outs[i][1] = {in[i].dw, wb};
            continue;
        }
        e = check_tensor(z, in[i], backward, &a.t[i], ins[i], outs[i]);
        if (e != ROPE_OK)
            return e;
    }
    if (tokens > 0 && heads > 0 && (cos == nullptr || sin == nullptr || z.table_rows < 1))
        return ROPE_ERR_INVALID_ARG;
    if (!aligned(cos, 16) || !aligned(sin, 16))
        return ROPE_ERR_UNSUPPORTED;
    if (!aligned(pos, 4))
        return ROPE_ERR_INVALID_ARG;
    const int64_t need = sums ? rope_norm_qk_workspace(z.D) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return ROPE_ERR_INVALID_ARG;
    if (need > 0 && !aligned(workspace, 16))
        return ROPE_ERR_UNSUPPORTED;
    const int64_t positions = pos == nullptr ? 0 : 4 * (z.pos_stride == 0 ? z.S : (z.B - 1) * z.pos_stride + z.S);
    const Range more[4] = {{cos, tab}, {sin, tab}, {pos, positions}, {workspace, need}};
    const Range all_outs[5] = {outs[0][0], outs[1][0], outs[0][1], outs[1][1], more[3]};
    for (int o = 0; o < 5; ++o) {
        for (int p = 0; p < o; ++p)
            if (overlap(all_outs[o], all_outs[p]))
                return ROPE_ERR_INVALID_ARG;
        for (int i = 0; i < 2; ++i)
            for (int r = 0; r < 3; ++r)
                // in place: every row is read before the same group writes it
                if (overlap(all_outs[o], ins[i][r]) &&
                    !(!backward && o == i && r == 0 && in[i].x == in[i].y && same_strides(z, a.t[i])))
                    return ROPE_ERR_INVALID_ARG;
        for (int r = 0; r < 3; ++r)
            if (overlap(all_outs[o], more[r]))
                return ROPE_ERR_INVALID_ARG;
    }
    a.cos = cos; a.sin = sin; a.pos = pos; a.pos_stride = z.pos_stride; a.table_rows = z.table_rows;
    a.tokens = tokens; a.B = z.B; a.S = z.S > 0 ? z.S : 1;
    a.D = z.D; a.rotary_dim = z.rotary_dim;
    a.w_f32 = z.weight_dtype == ROPE_F32;
    a.eps = z.eps; a.inv_d = 1.0f / (float)z.D;
    for (int i = 0; i < 2; ++i)
        if (backward && in[i].dw != nullptr)
            a.t[i].partial = static_cast<float *>(workspace) + (int64_t)i * kNormPartials * z.D;
    if (device_flag(&a.flag) != cudaSuccess)
        return ROPE_ERR_CUDA;
    const cudaError_t c = z.dtype == ROPE_F32    ? launch_norm_f32(a, z.layout, backward, st)
                          : z.dtype == ROPE_BF16 ? launch_norm_bf16(a, z.layout, backward, st)
                                                 : launch_norm_f16(a, z.layout, backward, st);
    return c == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA;
}

}  // namespace
}  // namespace rope

using namespace rope;

extern "C" {

int64_t rope_norm_qk_workspace(int32_t D)
{
    return D < 16 || D > 256 || D % 16 != 0 ? -1 : (int64_t)2 * kNormPartials * D * 4;
}

rope_status rope_norm_qk_fwd(const void *q, const void *k, void *q_out, void *k_out, const void *wq, const void *wk,
                             const float *cos, const float *sin, const int32_t *pos_idx, int64_t pos_batch_stride,
                             int64_t B, int32_t Hq, int32_t Hk, int64_t S, int32_t D, const int64_t *q_strides,
                             const int64_t *k_strides, int32_t rotary_dim, int32_t layout, int32_t seq_before_head,
                             float eps, int32_t dtype, int32_t weight_dtype, int64_t table_rows, void *stream)
{
    const Sizes z = {B, S, pos_batch_stride, table_rows, D, rotary_dim, layout, seq_before_head, dtype, weight_dtype, eps};
    const Tensor in[2] = {{q, nullptr, wq, q_out, nullptr, Hq, q_strides}, {k, nullptr, wk, k_out, nullptr, Hk, k_strides}};
    return norm_call(z, in, cos, sin, pos_idx, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

rope_status rope_norm_qk_bwd(const void *q, const void *k, const void *gq, const void *gk, void *dq, void *dk,
                             const void *wq, const void *wk, void *dwq, void *dwk, const float *cos, const float *sin,
                             const int32_t *pos_idx, int64_t pos_batch_stride, int64_t B, int32_t Hq, int32_t Hk,
                             int64_t S, int32_t D, const int64_t *q_strides, const int64_t *k_strides,
                             int32_t rotary_dim, int32_t layout, int32_t seq_before_head, float eps, int32_t dtype,
                             int32_t weight_dtype, int64_t table_rows, void *workspace, int64_t workspace_bytes,
                             void *stream)
{
    const Sizes z = {B, S, pos_batch_stride, table_rows, D, rotary_dim, layout, seq_before_head, dtype, weight_dtype, eps};
    const Tensor in[2] = {{q, gq, wq, dq, dwq, Hq, q_strides}, {k, gk, wk, dk, dwk, Hk, k_strides}};
    return norm_call(z, in, cos, sin, pos_idx, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

rope_status rope_norm_cache_append(const void *q, const void *k, const void *v, void *q_out, void *k_pages, void *v_pages,
                                   const void *wq, const void *wk, const int32_t *block_table,
                                   const int32_t *cu_seqlens, const int32_t *cache_lens, const float *cos,
                                   const float *sin, const int32_t *pos, int64_t pos_offset, int64_t n_seqs,
                                   int64_t total, int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t Hq,
                                   int32_t Hk, int32_t D, int32_t rotary_dim, int32_t layout, float eps,
                                   int32_t page_size, int64_t n_pages, int64_t max_blocks, int32_t dtype,
                                   int32_t weight_dtype, int64_t table_rows, void *stream)
{
    rope_status st = check_shape(dtype, layout, D, rotary_dim);
    if (st != ROPE_OK)
        return st;
    const int32_t shift = page_shift(page_size);
    if (shift < 0 || (weight_dtype != ROPE_F32 && weight_dtype != dtype))
        return ROPE_ERR_UNSUPPORTED;
    if (n_seqs < 0 || n_seqs >= kMaxInt32 || total < 0 || total > kMaxInt32 || Hq < 0 || Hk < 0 || n_pages < 0 ||
        n_pages > kMaxInt32 || max_blocks < 0 || table_rows < 0 || pos_offset < 0 || pos_offset > kMaxInt32 ||
        !(eps >= 0.0f) || !std::isfinite(eps))
        return ROPE_ERR_INVALID_ARG;
    const int64_t qrow = (int64_t)Hq * D, row = (int64_t)Hk * D;
    if (q_stride < qrow || k_stride < row || v_stride < row)
        return ROPE_ERR_INVALID_ARG;
    const int64_t qb = view_bytes(total, q_stride, qrow), kb = view_bytes(total, k_stride, row),
                  vb = view_bytes(total, v_stride, row), ob = product({total, qrow, 2});
    const int64_t pool = product({n_pages, Hk, page_size, D, 2});
    const int64_t tab = product({table_rows, rotary_dim / 2, 4});
    const int64_t blocks = product({n_seqs, max_blocks, 4}), wb = D * (weight_dtype == ROPE_F32 ? 4 : 2);
    if (qb < 0 || kb < 0 || vb < 0 || ob < 0 || pool < 0 || tab < 0 || blocks < 0)
        return ROPE_ERR_INVALID_ARG;
    if (total == 0 || n_seqs == 0 || (Hq == 0 && Hk == 0))
        return ROPE_OK;
    if (!cu_seqlens || !cache_lens || !cos || !sin || table_rows < 1 || (Hq > 0 && (!q || !q_out)) ||
        (Hk > 0 && (!k || !v || !k_pages || !v_pages || !block_table || n_pages < 1 || max_blocks < 1)))
        return ROPE_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(q, 16) || !aligned(q_out, 16) ||
        !aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(wq, 16) ||
        !aligned(wk, 16) || !aligned(cos, 16) || !aligned(sin, 16))
        return ROPE_ERR_UNSUPPORTED;
    if (!aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(cache_lens, 4) || !aligned(pos, 4))
        return ROPE_ERR_INVALID_ARG;
    const Range outs[3] = {{k_pages, pool}, {v_pages, pool}, {q_out, ob}};
    const Range ins[11] = {{q, qb}, {k, kb}, {v, vb}, {wq, wb}, {wk, wb}, {block_table, blocks},
                           {cu_seqlens, 4 * (n_seqs + 1)}, {cache_lens, 4 * n_seqs}, {cos, tab}, {sin, tab},
                           {pos, 4 * total}};
    for (int o = 0; o < 3; ++o) {
        for (int p = 0; p < o; ++p)
            if (overlap(outs[o], outs[p]))
                return ROPE_ERR_INVALID_ARG;
        for (int i = 0; i < 11; ++i)
            // queries in place: every row is read before the same group writes it
            if (overlap(outs[o], ins[i]) && !(o == 2 && i == 0 && q == q_out && (q_stride == qrow || total == 1)))
                return ROPE_ERR_INVALID_ARG;
    }
    NormAppendArgs a;
    std::memset(&a, 0, sizeof a);
    RowsArgs &r = a.rows;
    r.k = k; r.v = v; r.k_stride = k_stride; r.v_stride = v_stride;
    r.k_out = k_pages; r.v_out = v_pages;
    r.cu = cu_seqlens; r.pos = pos; r.cos = cos; r.sin = sin;
    r.table_rows = table_rows; r.total = total;
    r.n_seqs = (int32_t)n_seqs; r.Hk = Hk; r.rotary_dim = rotary_dim;
    r.table = block_table; r.cache_lens = cache_lens; r.table_stride = max_blocks;
    r.n_pages = n_pages; r.page_shift = shift; r.pos_offset = pos_offset;
    a.q = q; a.q_stride = q_stride; a.q_out = q_out; a.wq = wq; a.wk = wk;
    a.Hq = Hq; a.w_f32 = weight_dtype == ROPE_F32; a.eps = eps;
    if (device_flag(&r.flag) != cudaSuccess)
        return ROPE_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == ROPE_BF16 ? launch_norm_append_bf16(a, D, layout, s)
                                             : launch_norm_append_f16(a, D, layout, s);
    return e == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA;
}

}  // extern "C"
