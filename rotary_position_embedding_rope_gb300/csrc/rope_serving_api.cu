// rope_serving_api.cu -- the C ABI of the serving operators (include/rope.h):
// argument checks.  Everything the host can see is checked here, before
// anything is enqueued; offsets, lengths and page numbers are checked by the
// kernels.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "rope.h"
#include "rope_checks.h"
#include "rope_serving.cuh"

namespace rope {

int32_t packed_group_heads(int32_t Hq, int32_t Hk)
{
    int32_t gp = 1;
    while (gp < 16 && Hq / Hk % (2 * gp) == 0)
        gp *= 2;
    return gp;
}

bool packed_layout(int64_t n_seqs, int64_t total_q, int64_t total_k, int32_t Hq, int32_t Hk,
                   int32_t D, PackedLayout *out)
{
    // a sequence of n tokens has at most n / tokens + 1 query tiles, and the
    // empty ones have none
    const int64_t tokens = 256 / packed_group_heads(Hq, Hk);
    out->tiles = total_q / tokens + (n_seqs < total_q ? n_seqs : total_q);
    const int64_t entries = product({out->tiles, 32}), maps = product({n_seqs, 128});
    const int64_t keys = product({total_k, Hk, D, 2});
    if (entries < 0 || maps < 0 || keys < 0 || entries > (1ll << 60) || maps > (1ll << 60) ||
        keys > (1ll << 60))
        return false;
    out->entries = 128;
    out->maps = round_up(out->entries + entries, 128);
    out->keys = out->maps + maps;
    out->bytes = out->keys + keys;
    return true;
}

constexpr int32_t kSms = kDecodeSms;

bool decode_layout(int64_t B, int32_t Hq, int32_t Hk, int32_t D, int32_t page_shift, int64_t max_blocks,
                   int64_t n_prefix, DecodeLayout *out)
{
    std::memset(out, 0, sizeof *out);
    const int32_t group = Hq / Hk, gp = packed_group_heads(Hq, Hk);
    const int64_t rows = product({B, Hq});
    if (rows < 0 || rows > kMaxInt32)
        return false;
    out->rows = group < 16 ? group : 16;
    out->row_groups = (group + out->rows - 1) / out->rows;
    // With no more than 16 rows per key head (one mma tile) the prefix is one
    // more sequence of the suffix kernel.
    const int64_t tiles = (n_prefix + 127) / 128;
    out->fold = n_prefix > 0 && B * group <= 16;
    out->slot_rows = out->fold ? (int32_t)(B * group) : out->rows;
    // Otherwise clusters of 256 rows take its (row tile, head unit, key tile)s:
    // at most one cluster per pair of SMs, and per group of row tiles one part
    // for each head unit it touches.
    out->row_tiles = (int32_t)((B + 256 / gp - 1) / (256 / gp));
    const int64_t head_units = Hq / gp, work = product({out->row_tiles, head_units, tiles});
    if (work < 0 || work > kMaxInt32 - 128)
        return false;
    out->clusters = (int32_t)(work < kSms / 2 ? (work > 0 ? work : 1) : kSms / 2);
    const int64_t groups = out->clusters / out->row_tiles > 0 ? out->clusters / out->row_tiles : 1;
    const int64_t parts = n_prefix > 0 && !out->fold ? groups + head_units : 0;
    // The suffixes: a CTA for every 256 keys of a pair, up to one an SM, whose eight
    // warps take runs of at least two chunks.  Chunks of 64 features are of 32 keys,
    // so half the warps of a small call have no run then; with a CTA for 512 keys
    // fewer SMs copy (one sequence of 2000 keys, 16 heads of 64: 11.3 us, so 10.2).
    int64_t chunks = product({B, max_blocks, (int64_t)1 << page_shift >> 4});
    if (chunks < 0 || chunks > kMaxInt32)
        return false;
    if (out->fold)
        chunks += (n_prefix + 15) / 16;
    const int64_t heads = product({Hk, out->row_groups}), all = product({chunks, heads});
    const int64_t pairs = product({B + 1, heads});
    if (chunks > kMaxInt32 || all < 0 || pairs < 0 || pairs > kMaxInt32 - (kSms + 1) * 8)
        return false;
    const int64_t ctas = (all + 15) / 16;
    out->suffix_ctas = (int32_t)(ctas < kSms ? ctas : kSms);
    // (beside a prefix kernel, warps of up to that many CTAs and its own)
    const int64_t most = out->suffix_ctas + 2 * out->clusters < kSms ? out->suffix_ctas + 2 * out->clusters : kSms;
    const int64_t slots = out->suffix_ctas > 0 ? (most + 1) * 8 + pairs : 0;
    const int64_t o = product({slots, out->slot_rows, D, 4}), s = product({slots, out->slot_rows, 8});
    const int64_t po = product({parts, B, gp, D, 4}), ps = product({parts, B, gp, 8});
    if (o < 0 || s < 0 || po < 0 || ps < 0 || o > (1ll << 60) || po > (1ll << 60))
        return false;
    out->chunk_start = 128;
    out->out = round_up(out->chunk_start + 4 * (B + 2), 128);
    out->stats = out->out + o;
    out->prefix_out = round_up(out->stats + s, 128);
    out->prefix_stats = out->prefix_out + po;
    out->bytes = round_up(out->prefix_stats + ps, 128);
    return true;
}

bool paged_layout(int64_t n_seqs, int64_t total_q, int32_t Hq, int32_t Hk, int32_t D, int32_t page_shift,
                  int64_t max_blocks, PagedLayout *out)
{
    const int64_t group = Hq / Hk, few = group < 16 ? 16 / group : 1;
    const int64_t chunks = product({n_seqs, max_blocks, (int64_t)1 << page_shift >> 4});
    const int64_t keys = product({max_blocks, (int64_t)1 << page_shift});
    if (chunks < 0 || chunks > kMaxInt32 - 16 * kMaxDecodeBatch || keys < 0 || keys > kMaxInt32 - 256)
        return false;
    const int64_t few_tokens = total_q < n_seqs * few ? total_q : n_seqs * few;
    out->few_rows = few_tokens * Hq;
    // tiles: a sequence has at most tokens / tile + 1 of them; none where all the
    // call's rows of a key head are few
    const int64_t tile = 256 / packed_group_heads(Hq, Hk);
    const bool tiles = total_q > 1 && total_q * group > 16;
    const int64_t entries = tiles ? total_q / tile + (n_seqs < total_q ? n_seqs : total_q) : 0;
    // at most two pieces of 256 rows for each cluster that the plan may use, and 16 rows for
    // each run of few-row chunks
    const int64_t units = product({entries, Hq / packed_group_heads(Hq, Hk)});
    const int64_t weight = product({units, keys / 128 + 1 + kPagedUnitTiles});   // (tiles of 128 keys)
    const int64_t charge = product({chunks + kFewPairCost * n_seqs, Hk, (group + 15) / 16});
    if (units < 0 || weight < 0 || charge < 0)
        return false;
    const int64_t runs = weight / kPagedMinRun, clusters = std::min<int64_t>(kDecodeSms / 2, std::max(units, runs));
    const int64_t parts = clusters * 2 * 256;
    const int64_t part_rows = 16 * std::min<int64_t>(kFewWarps * kDecodeSms, charge / kFewMinRun + 1) + out->few_rows;
    const int64_t few_out = product({part_rows, D, 4});
    if (entries > (1ll << 31) || few_out < 0)
        return false;
    out->entries = kPagedHead;
    out->maps = round_up(out->entries + entries * 32, 128);
    out->chunk_start = out->maps + n_seqs * 128;
    out->few_start = out->chunk_start + 4 * (n_seqs + 1);
    out->few_seq = out->few_start + 4 * (n_seqs + 1);
    out->few_out = round_up(out->few_seq + 4 * few_tokens, 128);
    out->few_stats = out->few_out + few_out;
    out->out = round_up(out->few_stats + 8 * part_rows, 128);
    out->stats = out->out + parts * D * 4;
    out->bytes = round_up(out->stats + parts * 8, 128);
    return true;
}

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

int64_t rope_attention_packed_workspace(int64_t n_seqs, int64_t total_q, int64_t total_k, int32_t Hq,
                                        int32_t Hk, int32_t D)
{
    PackedLayout lay;
    if (n_seqs < 0 || n_seqs >= kMaxInt32 || total_q < 0 || total_q > kMaxInt32 || total_k < 0 ||
        total_k > kMaxInt32 || Hq < 0 || Hk < 0 || (D != 64 && D != 128))
        return -1;
    if (n_seqs == 0 || total_q == 0 || Hq == 0)
        return 0;
    if (Hk == 0 || Hq % Hk != 0 || !packed_layout(n_seqs, total_q, total_k, Hq, Hk, D, &lay))
        return -1;
    return lay.bytes;
}

rope_status rope_attention_packed_fwd(const void *q, const void *k, const void *v, void *o,
                                      const float *cos, const float *sin, const int32_t *pos_q,
                                      const int32_t *pos_k, const int32_t *cu_seqlens_q,
                                      const int32_t *cu_seqlens_k, int64_t n_seqs, int64_t total_q,
                                      int64_t total_k, int64_t q_stride, int64_t k_stride,
                                      int64_t v_stride, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t rotary_dim, int32_t layout, int32_t causal,
                                      float softmax_scale, int32_t dtype, int64_t table_rows,
                                      void *workspace, int64_t workspace_bytes, void *stream)
{
    rope_status st = check_shape(dtype, layout, D, rotary_dim);
    if (st != ROPE_OK)
        return st;
    if ((causal != 0 && causal != 1) || softmax_scale != softmax_scale || n_seqs < 0 ||
        n_seqs >= kMaxInt32 || total_q < 0 || total_q > kMaxInt32 || total_k < 0 ||
        total_k > kMaxInt32 || Hq < 0 || Hk < 0 || table_rows < 0 || workspace_bytes < 0)
        return ROPE_ERR_INVALID_ARG;
    if (Hq > 0 && (Hk == 0 || Hq % Hk != 0))
        return ROPE_ERR_INVALID_ARG;
    const int64_t qrow = (int64_t)Hq * D, krow = (int64_t)Hk * D;
    if (q_stride < qrow || k_stride < krow || v_stride < krow)
        return ROPE_ERR_INVALID_ARG;
    const int64_t qb = view_bytes(total_q, q_stride, qrow), kb = view_bytes(total_k, k_stride, krow),
                  vb = view_bytes(total_k, v_stride, krow), ob = product({total_q, qrow, 2}),
                  tab = product({table_rows, rotary_dim / 2, 4});
    if (qb < 0 || kb < 0 || vb < 0 || ob < 0 || tab < 0)
        return ROPE_ERR_INVALID_ARG;
    if (total_q == 0 || n_seqs == 0 || Hq == 0)
        return ROPE_OK;                                  // no output rows
    if (!q || !o || !cos || !sin || !cu_seqlens_q || !cu_seqlens_k || (total_k > 0 && (!k || !v)) ||
        table_rows < 1)
        return ROPE_ERR_INVALID_ARG;
    PackedLayout lay;
    if (!packed_layout(n_seqs, total_q, total_k, Hq, Hk, D, &lay) || !workspace ||
        workspace_bytes < lay.bytes)
        return ROPE_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(q, 16) ||
        !aligned(o, 16) || !aligned(cos, 16) || !aligned(sin, 16) || !aligned(workspace, 128) ||
        (total_k > 0 && (!aligned(k, 16) || !aligned(v, 16))))
        return ROPE_ERR_UNSUPPORTED;
    if (!aligned(pos_q, 4) || !aligned(pos_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
        return ROPE_ERR_INVALID_ARG;
    const Range outs[2] = {{o, ob}, {workspace, lay.bytes}};
    const Range ins[9] = {{q, qb}, {k, kb}, {v, vb}, {cos, tab}, {sin, tab}, {pos_q, 4 * total_q},
                          {pos_k, 4 * total_k}, {cu_seqlens_q, 4 * (n_seqs + 1)},
                          {cu_seqlens_k, 4 * (n_seqs + 1)}};
    if (overlap(outs[0], outs[1]))
        return ROPE_ERR_INVALID_ARG;
    for (const Range &out : outs)
        for (const Range &in : ins)
            if (overlap(out, in))
                return ROPE_ERR_INVALID_ARG;
    PackedArgs a;
    std::memset(&a, 0, sizeof a);
    RowsArgs &r = a.keys;
    r.k = k; r.v = v; r.k_stride = k_stride; r.v_stride = v_stride;
    r.cu = cu_seqlens_k; r.pos = pos_k; r.cos = cos; r.sin = sin;
    r.table_rows = table_rows; r.total = total_k;
    r.n_seqs = (int32_t)n_seqs; r.Hk = Hk; r.rotary_dim = rotary_dim;
    if (device_flag(&r.flag) != cudaSuccess)
        return ROPE_ERR_CUDA;
    a.q = q; a.q_stride = q_stride; a.o = o;
    a.cu_q = cu_seqlens_q; a.pos_q = pos_q; a.total_q = total_q;
    a.Hq = Hq; a.causal = causal; a.workspace = workspace;
    const double scale = softmax_scale > 0.0f ? softmax_scale : 1.0 / std::sqrt((double)D);
    a.scale_log2 = (float)(scale * 1.4426950408889634);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == ROPE_BF16 ? launch_packed_bf16(a, lay, D, layout, s)
                                             : launch_packed_f16(a, lay, D, layout, s);
    return e == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA;
}

int64_t rope_attention_decode_workspace(int64_t B, int32_t Hq, int32_t Hk, int32_t D, int32_t page_size,
                                        int64_t max_blocks, int64_t prefix_len)
{
    const int32_t shift = page_shift(page_size);
    DecodeLayout lay;
    if (B < 0 || B > kMaxDecodeBatch || Hq < 0 || Hk < 0 || (D != 64 && D != 128) || shift < 0 ||
        max_blocks < 0 || prefix_len < 0 || prefix_len > kMaxInt32 - 128)
        return -1;
    if (B == 0 || Hq == 0)
        return 0;
    if (Hk == 0 || Hq % Hk != 0 || !decode_layout(B, Hq, Hk, D, shift, max_blocks, prefix_len, &lay))
        return -1;
    return lay.bytes;
}

rope_status rope_attention_decode_fwd(const void *q, const void *k_pages, const void *v_pages, void *o,
                                      const int32_t *block_table, const int32_t *seq_lens,
                                      const int32_t *prefix_table, int64_t prefix_len,
                                      const float *cos, const float *sin, const int32_t *pos_q,
                                      int64_t B, int64_t q_stride, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t rotary_dim, int32_t layout, float softmax_scale,
                                      int32_t page_size, int64_t n_pages, int64_t max_blocks,
                                      int32_t dtype, int64_t table_rows, void *workspace,
                                      int64_t workspace_bytes, void *stream)
{
    rope_status st = check_shape(dtype, layout, D, rotary_dim);
    if (st != ROPE_OK)
        return st;
    const int32_t shift = page_shift(page_size);
    if (shift < 0)
        return ROPE_ERR_UNSUPPORTED;
    if (softmax_scale != softmax_scale || B < 0 || Hq < 0 || Hk < 0 || n_pages < 0 || max_blocks < 0 ||
        prefix_len < 0 || prefix_len > kMaxInt32 - 128 || table_rows < 0 || workspace_bytes < 0)
        return ROPE_ERR_INVALID_ARG;
    if (B > kMaxDecodeBatch)
        return ROPE_ERR_UNSUPPORTED;
    if (Hq > 0 && (Hk == 0 || Hq % Hk != 0))
        return ROPE_ERR_INVALID_ARG;
    const int64_t row = (int64_t)Hq * D;
    if (q_stride < row)
        return ROPE_ERR_INVALID_ARG;
    const int64_t z = product({n_pages, Hk});
    const int64_t qb = view_bytes(B, q_stride, row), ob = product({B, row, 2});
    const int64_t pool = product({n_pages, Hk, page_size, D, 2});
    const int64_t tab = product({table_rows, rotary_dim / 2, 4}), blocks = product({B, max_blocks, 4});
    if (z < 0 || z > kMaxInt32 - 1 || qb < 0 || ob < 0 || pool < 0 || tab < 0 || blocks < 0)
        return ROPE_ERR_INVALID_ARG;
    if (B == 0 || Hq == 0)
        return ROPE_OK;
    const bool any_keys = prefix_len > 0 || max_blocks > 0;
    if (!q || !o || !seq_lens || !cos || !sin || table_rows < 1 || (any_keys && (!k_pages || !v_pages)) ||
        (any_keys && n_pages < 1) || (max_blocks > 0 && !block_table) || (prefix_len > 0 && !prefix_table))
        return ROPE_ERR_INVALID_ARG;
    DecodeLayout lay;
    if (!decode_layout(B, Hq, Hk, D, shift, max_blocks, prefix_len, &lay) || !workspace ||
        workspace_bytes < lay.bytes)
        return ROPE_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || !aligned(q, 16) || !aligned(o, 16) || !aligned(cos, 16) || !aligned(sin, 16) ||
        !aligned(workspace, 128) || !aligned(k_pages, 16) || !aligned(v_pages, 16))
        return ROPE_ERR_UNSUPPORTED;
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(prefix_table, 4) || !aligned(pos_q, 4))
        return ROPE_ERR_INVALID_ARG;
    const Range outs[2] = {{o, ob}, {workspace, lay.bytes}};
    const int64_t prefix_blocks = (prefix_len + page_size - 1) / page_size;
    const Range ins[9] = {{q, qb}, {k_pages, pool}, {v_pages, pool}, {block_table, blocks},
                          {seq_lens, 4 * B}, {prefix_table, 4 * prefix_blocks}, {cos, tab}, {sin, tab},
                          {pos_q, 4 * B}};
    if (overlap(outs[0], outs[1]))
        return ROPE_ERR_INVALID_ARG;
    for (const Range &out : outs)
        for (const Range &in : ins)
            if (overlap(out, in))
                return ROPE_ERR_INVALID_ARG;
    DecodeCall c;
    std::memset(&c, 0, sizeof c);
    c.q = q; c.q_stride = q_stride; c.k_pages = k_pages; c.v_pages = v_pages; c.o = o;
    c.table = block_table; c.lens = seq_lens; c.prefix_table = prefix_table; c.pos_q = pos_q;
    c.cos = cos; c.sin = sin; c.table_rows = table_rows; c.n_pages = n_pages; c.max_blocks = max_blocks;
    c.B = (int32_t)B; c.Hq = Hq; c.Hk = Hk; c.rotary_dim = rotary_dim; c.page_shift = shift;
    c.n_prefix = (int32_t)prefix_len; c.workspace = workspace;
    const double scale = softmax_scale > 0.0f ? softmax_scale : 1.0 / std::sqrt((double)D);
    c.scale_log2 = (float)(scale * 1.4426950408889634);
    if (device_flag(&c.flag) != cudaSuccess)
        return ROPE_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == ROPE_BF16 ? launch_decode_bf16(c, lay, D, layout, s)
                                             : launch_decode_f16(c, lay, D, layout, s);
    return e == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA;
}

int64_t rope_attention_paged_workspace(int64_t n_seqs, int64_t total_q, int32_t Hq, int32_t Hk, int32_t D,
                                       int32_t page_size, int64_t max_blocks)
{
    const int32_t shift = page_shift(page_size);
    PagedLayout lay;
    if (n_seqs < 0 || n_seqs > kMaxDecodeBatch || total_q < 0 || total_q > kMaxInt32 || Hq < 0 || Hk < 0 ||
        (D != 64 && D != 128) || shift < 0 || max_blocks < 0)
        return -1;
    if (n_seqs == 0 || total_q == 0 || Hq == 0)
        return 0;
    if (Hk == 0 || Hq % Hk != 0 || !paged_layout(n_seqs, total_q, Hq, Hk, D, shift, max_blocks, &lay))
        return -1;
    return lay.bytes;
}

rope_status rope_attention_paged_fwd(const void *q, const void *k_pages, const void *v_pages, void *o,
                                     const int32_t *block_table, const int32_t *cu_seqlens_q,
                                     const int32_t *seq_lens, const float *cos, const float *sin,
                                     const int32_t *pos_q, int64_t n_seqs, int64_t total_q, int64_t q_stride,
                                     int32_t Hq, int32_t Hk, int32_t D, int32_t rotary_dim, int32_t layout,
                                     int32_t causal, float softmax_scale, int32_t page_size, int64_t n_pages,
                                     int64_t max_blocks, int32_t dtype, int64_t table_rows, void *workspace,
                                     int64_t workspace_bytes, void *stream)
{
    const bool rotate = cos != nullptr || sin != nullptr;
    rope_status st = check_shape(dtype, layout, D, rotate ? rotary_dim : D);
    if (st != ROPE_OK)
        return st;
    const int32_t shift = page_shift(page_size);
    if (shift < 0)
        return ROPE_ERR_UNSUPPORTED;
    if ((causal != 0 && causal != 1) || softmax_scale != softmax_scale || n_seqs < 0 || total_q < 0 ||
        total_q > kMaxInt32 || Hq < 0 || Hk < 0 || n_pages < 0 || max_blocks < 0 || table_rows < 0 || workspace_bytes < 0)
        return ROPE_ERR_INVALID_ARG;
    if (n_seqs > kMaxDecodeBatch)
        return ROPE_ERR_UNSUPPORTED;
    if (Hq > 0 && (Hk == 0 || Hq % Hk != 0))
        return ROPE_ERR_INVALID_ARG;
    const int64_t row = (int64_t)Hq * D;
    if (q_stride < row)
        return ROPE_ERR_INVALID_ARG;
    const int64_t z = product({n_pages, Hk});
    const int64_t qb = view_bytes(total_q, q_stride, row), ob = product({total_q, row, 2});
    const int64_t pool = product({n_pages, Hk, page_size, D, 2});
    const int64_t tab = rotate ? product({table_rows, rotary_dim / 2, 4}) : 0, blocks = product({n_seqs, max_blocks, 4});
    if (z < 0 || z > kMaxInt32 - 1 || qb < 0 || ob < 0 || pool < 0 || tab < 0 || blocks < 0)
        return ROPE_ERR_INVALID_ARG;
    if (n_seqs == 0 || total_q == 0 || Hq == 0)
        return ROPE_OK;                                  // no output rows
    if (!q || !o || !cu_seqlens_q || !seq_lens || (rotate && (!cos || !sin || table_rows < 1)) ||
        (max_blocks > 0 && (!block_table || !k_pages || !v_pages || n_pages < 1)))
        return ROPE_ERR_INVALID_ARG;
    PagedLayout lay;
    if (!paged_layout(n_seqs, total_q, Hq, Hk, D, shift, max_blocks, &lay) || !workspace || workspace_bytes < lay.bytes)
        return ROPE_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || !aligned(q, 16) || !aligned(o, 16) || !aligned(cos, 16) || !aligned(sin, 16) ||
        !aligned(workspace, 128) || !aligned(k_pages, 16) || !aligned(v_pages, 16))
        return ROPE_ERR_UNSUPPORTED;
    if (!aligned(block_table, 4) || !aligned(cu_seqlens_q, 4) || !aligned(seq_lens, 4) || !aligned(pos_q, 4))
        return ROPE_ERR_INVALID_ARG;
    const Range outs[2] = {{o, ob}, {workspace, lay.bytes}};
    const Range ins[9] = {{q, qb}, {k_pages, pool}, {v_pages, pool}, {block_table, blocks},
                          {cu_seqlens_q, 4 * (n_seqs + 1)}, {seq_lens, 4 * n_seqs}, {cos, tab}, {sin, tab},
                          {pos_q, 4 * total_q}};
    if (overlap(outs[0], outs[1]))
        return ROPE_ERR_INVALID_ARG;
    for (const Range &out : outs)
        for (const Range &in : ins)
            if (overlap(out, in))
                return ROPE_ERR_INVALID_ARG;
    PagedCall c;
    std::memset(&c, 0, sizeof c);
    c.q = q; c.q_stride = q_stride; c.k_pages = k_pages; c.v_pages = v_pages; c.o = o;
    c.table = block_table; c.cu = cu_seqlens_q; c.lens = seq_lens; c.pos_q = pos_q;
    c.cos = cos; c.sin = sin; c.table_rows = table_rows; c.total_q = total_q; c.n_pages = n_pages;
    c.max_blocks = max_blocks;
    c.n_seqs = (int32_t)n_seqs; c.Hq = Hq; c.Hk = Hk; c.rotary_dim = rotate ? rotary_dim : D; c.page_shift = shift;
    c.causal = causal; c.workspace = workspace;
    const double scale = softmax_scale > 0.0f ? softmax_scale : 1.0 / std::sqrt((double)D);
    c.scale_log2 = (float)(scale * 1.4426950408889634);
    if (device_flag(&c.flag) != cudaSuccess)
        return ROPE_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == ROPE_BF16 ? launch_paged_bf16(c, lay, D, layout, s)
                                             : launch_paged_f16(c, lay, D, layout, s);
    return e == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA;
}

}  // extern "C"
