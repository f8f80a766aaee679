// rope_serving.cuh -- declarations of the serving operators: cache append,
// attention over packed sequences, attention over a shared prefix.
// Not part of the public ABI (include/rope.h is).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rope_internal.cuh"

namespace rope {

// The device's flag word (rope_api.cu), reported by rope_check_errors.
cudaError_t device_flag(int32_t **flag);

// Rows of packed keys (and values), to be rotated and written either into
// cache pages or, for attention over packed sequences, into a dense
// [Hk][total][D] workspace (k_out).
struct RowsArgs {
    const void *k, *v;               // [total][Hk][D], token strides in elements
    int64_t k_stride, v_stride;
    void *k_out, *v_out;             // pools [n_pages][Hk][page][D], or the workspace
    const int32_t *cu;               // [n_seqs + 1]
    const int32_t *pos;              // [total] or nullptr
    const float *cos, *sin;
    int64_t table_rows;
    int64_t total;
    int32_t n_seqs, Hk, rotary_dim;
    // pages
    const int32_t *table;            // [n_seqs][table_stride]
    const int32_t *cache_lens;       // [n_seqs]
    int64_t table_stride;            // blocks of a sequence
    int64_t n_pages;
    int32_t page_shift;              // page size = 1 << page_shift
    int64_t pos_offset;
    int32_t *flag;
};

cudaError_t launch_cache_append(const RowsArgs &a, int32_t D, int32_t layout, int32_t dtype,
                                cudaStream_t st);

// Attention over packed sequences (rope_attention_packed.cuh).
struct PackedArgs {
    RowsArgs keys;                   // k -> the rotated-key workspace
    const void *q;                   // [total_q][Hq][D]
    int64_t q_stride;
    void *o;                         // [total_q][Hq][D], dense
    const int32_t *cu_q;
    const int32_t *pos_q;            // [total_q] or nullptr
    int64_t total_q;
    int32_t Hq;
    int32_t causal;
    float scale_log2;
    void *workspace;
};

// Bytes of the workspace of a packed call, and of its parts.
struct PackedLayout {
    int64_t tiles;                   // most query tiles of all sequences
    int64_t entries, maps, keys;     // byte offsets
    int64_t bytes;
};
// Query heads of one group that share a tile: the largest power of two, up to
// 16, that divides Hq / Hk.
int32_t packed_group_heads(int32_t Hq, int32_t Hk);
// False when a size overflows.
bool packed_layout(int64_t n_seqs, int64_t total_q, int64_t total_k, int32_t Hq, int32_t Hk,
                   int32_t D, PackedLayout *out);
cudaError_t launch_packed_bf16(const PackedArgs &c, const PackedLayout &lay, int32_t D, int32_t layout,
                               cudaStream_t st);
cudaError_t launch_packed_f16(const PackedArgs &c, const PackedLayout &lay, int32_t D, int32_t layout,
                              cudaStream_t st);

// Attention of one token per sequence over a shared prefix and a suffix each
// (rope_attention_decode.cuh).
constexpr int32_t kMaxDecodeBatch = 4096;      // sequences of a call (their scan fits an SM)
// The SMs a decode call is dealt out to, at most (its workspace has slots for
// their warps); fewer give the same results, less evenly spread.
constexpr int32_t kDecodeSms = 152;
struct DecodeCall {
    const void *q;                   // [B][Hq][D], row stride q_stride
    int64_t q_stride;
    const void *k_pages, *v_pages;   // [n_pages][Hk][page][D]
    void *o;                         // [B][Hq][D]
    const int32_t *table, *lens;     // [B][max_blocks], [B]
    const int32_t *prefix_table;
    const int32_t *pos_q;            // [B] or nullptr
    const float *cos, *sin;
    int64_t table_rows, n_pages, max_blocks;
    int32_t B, Hq, Hk, rotary_dim, page_shift, n_prefix;
    float scale_log2;
    void *workspace;
    int32_t *flag;
};

// How a decode call is split, and its workspace.
struct DecodeLayout {
    int32_t fold;                                    // the prefix runs with the suffixes
    int32_t row_tiles, clusters;                     // prefix: tiles of rows, most clusters
    int32_t row_groups, rows, slot_rows, suffix_ctas;
    int64_t chunk_start, out, stats, prefix_out, prefix_stats;   // byte offsets
    int64_t bytes;
};
// False when a size overflows or is not taken.
bool decode_layout(int64_t B, int32_t Hq, int32_t Hk, int32_t D, int32_t page_shift, int64_t max_blocks,
                   int64_t n_prefix, DecodeLayout *out);
// Attention of new tokens over a paged cache (rope_attention_paged.cuh).
struct PagedCall {
    const void *q;                   // [total_q][Hq][D], token stride q_stride
    int64_t q_stride;
    const void *k_pages, *v_pages;   // [n_pages][Hk][page][D]
    void *o;                         // [total_q][Hq][D]
    const int32_t *table, *cu, *lens;    // [n_seqs][max_blocks], [n_seqs + 1], [n_seqs]
    const int32_t *pos_q;            // [total_q] or nullptr
    const float *cos, *sin;          // nullptr: queries as they are
    int64_t table_rows, total_q, n_pages, max_blocks;
    int32_t n_seqs, Hq, Hk, rotary_dim, page_shift, causal;
    float scale_log2;
    void *workspace;
    int32_t *flag;
};
// What a unit costs besides its key tiles, in tiles (its query tile's way in and
// its output's way out: about 4 us of 0.9 a tile).
constexpr int32_t kPagedUnitTiles = 4;
// Least weight of a cluster's run where there are more clusters than units: shorter runs
// leave more pieces than they save.  (Two units one after the other take longer than either
// alone.  Clusters by the weight alone, and no fewer than units, us: 84 rows of eight key heads
// after 300 keys beside three single tokens, seven and eight clusters, 23.3, 21.1; four chunks of
// 40 after up to 300 keys 19.6, 18.2, eight of them 20.9, 20.0, 16 of them 23.4, 23.5; three of 30
// with heads of 64 17.4, 15.4; 24 of 20 29.1, 29.0; 64 prompts of 40 47.5 either way.)
constexpr int64_t kPagedMinRun = 2 * kPagedUnitTiles;
// What a pair (sequence, key head) of a few-row sequence counts for besides its chunks, in
// chunks: its queries' way in and its outputs' way out, several loads one after the other.
// Without it the warps that got the short sequences ended last.  0, 2, 5, 12 of them (us): 40
// drafts of up to five tokens, heads of 64, contexts to 3k 70, 48.7, 47.7, 47.8; 64 of four
// tokens, groups of four, contexts to 4k 119, 111, 109, 108; 64 single tokens, contexts to 8k
// 175.5, 172, 170.5, 171.4; 1024 after up to 300 keys 155 (0), 143 (6), 147.
constexpr int32_t kFewPairCost = 5;
// Warps of an SM that take few-row sequences, and the least charge of such a warp's run.
constexpr int kFewWarps = 12;
constexpr int64_t kFewMinRun = 2;
constexpr int64_t kPagedHead = 1024;           // bytes of the plan's head: a cut for every cluster
struct PagedLayout {
    int64_t few_rows;                // most rows (token, head) of few-row sequences
    int64_t entries, maps, chunk_start, few_start, few_seq, few_out, few_stats, out, stats;    // byte offsets
    int64_t bytes;
};
// False when a size overflows or is not taken.
bool paged_layout(int64_t n_seqs, int64_t total_q, int32_t Hq, int32_t Hk, int32_t D, int32_t page_shift,
                  int64_t max_blocks, PagedLayout *out);
cudaError_t launch_paged_bf16(const PagedCall &c, const PagedLayout &lay, int32_t D, int32_t layout,
                              cudaStream_t st);
cudaError_t launch_paged_f16(const PagedCall &c, const PagedLayout &lay, int32_t D, int32_t layout,
                             cudaStream_t st);

cudaError_t launch_decode_bf16(const DecodeCall &c, const DecodeLayout &lay, int32_t D, int32_t layout,
                               cudaStream_t st);
cudaError_t launch_decode_f16(const DecodeCall &c, const DecodeLayout &lay, int32_t D, int32_t layout,
                              cudaStream_t st);

}  // namespace rope
