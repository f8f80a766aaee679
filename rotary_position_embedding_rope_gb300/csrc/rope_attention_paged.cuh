// rope_attention_paged.cuh -- attention of every sequence's new tokens, one or a
// chunk of a prompt, over its keys in a paged cache (rope_attention_paged_fwd).
//
//   o_i = softmax(scale * rot(q_i) K_b^T, j <= i + Lk - Lq) V_b
//
// for the Lq new tokens i of sequence b, whose Lk keys (the new tokens' own among
// them, rotated when they were appended) lie in pages.  A step of a serving loop
// mixes sequences of a single token with chunks of hundreds, so a call has two
// kinds of work, side by side in one launch:
//   tiles   sequences of more rows (token, head) per key head run on
//           rope_attn_packed_kernel, whose units here are (query tile, head unit)
//           pairs.  The key tiles of all units, each unit's with a fixed charge for
//           its start and end, laid end to end, are cut into equal runs, one per
//           cluster, wherever the cuts fall: a long context of one sequence and a
//           batch of ragged chunks both keep every cluster busy to the end.  A unit
//           that lies in one run is written by it; a cut one leaves an fp32 (O, m,
//           l) per piece;
//   few     the others, of at most 16 rows, or a single token, are dealt out as
//           the suffixes of the shared-prefix decode: equal runs of 16-key (32 for
//           heads of 64) chunks for all warps of the SMs that have no tiles, an fp32
//           (O, m, l) for each pair (sequence, key head) that a run touches.
// Three launches:
//   1. rope_paged_plan_kernel checks the offsets and lengths, lists the units and
//      cuts them, decides how many SMs each kind gets (plan_ns's estimate), and
//      writes a tensor map for the last, partly filled page of a sequence (rows
//      past its end arrive as zeros: what lies there must not meet a probability of
//      zero);
//   2. the attention;
//   3. rope_paged_merge_kernel joins the pieces.
// The split depends on the sizes and the lengths alone: the same call gives the
// same bits.
//
// Roundings: for the tiles, and for sequences of nine to 16 rows, rot(q), and P before
// P V, to the element type (operands of a 16-bit product, whose issue is the bound), as in
// the packed attention; for at most eight rows they go into the products as two 16-bit
// parts (few_pair).  Everything else is fp32 until o.
#pragma once

#include "rope_attention_decode.cuh"

namespace rope {

// One query tile of a sequence, 256 / GP tokens; `before`: the weight of the
// units of all entries before it.
struct alignas(16) PagedEntry {
    int32_t seq, tok0, Lq, Lk;
    int32_t q_start, n_tiles;
    int64_t before;
};

// A place among the units' key tiles: entry, head unit, key tile.
struct PagedCut {
    int32_t entry, hu, kt;
    __device__ __forceinline__ bool before(const PagedCut &o) const
    {
        return entry != o.entry ? entry < o.entry : hu != o.hu ? hu < o.hu : kt < o.kt;
    }
    __device__ __forceinline__ bool same_unit(const PagedCut &o) const { return entry == o.entry && hu == o.hu; }
};

constexpr int kPagedPlanThreads = 512;
constexpr int32_t kPagedClusters = kDecodeSms / 2;   // at most
static_assert(kDecMinChunks >= kFewMinRun, "the workspace's runs");
// Bytes of a few-row warp's eight padded query rows, and of a CTA's warps.
template <int D>
static constexpr int kFewQuery = 8 * kDecQStride<D>;
template <int D>
static constexpr int kFewSmem = kFewWarps * (kDecStages<D> * kDecStageBytes<D> + kFewQuery<D>);
static_assert(kFewSmem<128> <= 225 * 1024 && kFewSmem<64> <= 225 * 1024, "a CTA's shared memory");

// The plan, at the start of the workspace.
struct PagedDeal {
    int32_t clusters;                              // with tiles
    int32_t chunks;                                // of the few-row sequences, per pair, charges included
    int32_t few_tokens;                            // of the few-row sequences
    int64_t per;                                   // chunks of a warp
    PagedCut cut[kPagedClusters + 1];              // cluster c: cut[c] .. cut[c + 1]
};
static_assert(sizeof(PagedDeal) <= kPagedHead, "the plan's place in the workspace");

struct PagedPlan {
    const int32_t *cu, *lens;
    int32_t n_seqs, group, tile_tokens, head_units, heads;
    int64_t total_q, most_keys;
    int32_t causal, chunk_shift, page_shift, chunk_bytes, tile_ns, grid;
    PagedDeal *deal;
    PagedEntry *entries;
    int32_t *chunk_start, *few_start;              // [n_seqs + 1]: chunks, tokens of the few-row sequences before b
    int32_t *few_seq;                              // sequence of each token of those
    CUtensorMap *maps;                             // [n_seqs]: of a sequence's last page
    int32_t *flag;
};

// Sequences that run as few-row ones: of at most 16 rows (token, head) per key head, or,
// where a token alone has more, of that token, its heads in groups of 16.
__device__ __forceinline__ bool paged_few(int32_t Lq, int32_t group)
{
    return Lq == 1 || (int64_t)Lq * group <= 16;
}

// A sequence's new tokens and keys; false when an offset or the length is out of range.
__device__ __forceinline__ bool paged_sequence(const int32_t *cu, const int32_t *lens, int32_t b, int64_t total_q,
                                               int64_t most, int32_t &Lq, int32_t &Lk)
{
    const int32_t q0 = __ldg(cu + b), q1 = __ldg(cu + b + 1);
    Lk = __ldg(lens + b);
    Lq = q1 - q0;
    return q0 >= 0 && q0 <= q1 && q1 <= total_q && Lk >= 0 && Lk <= most;
}

// Inclusive sums over the CTA of two 32-bit and one 64-bit number; returns the totals.
struct PagedSums {
    int32_t a, b;
    int64_t c;
};
__device__ __forceinline__ PagedSums paged_scan(PagedSums x, PagedSums &total, PagedSums *warp_sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t a = __shfl_up_sync(0xffffffffu, x.a, d), b = __shfl_up_sync(0xffffffffu, x.b, d);
        const int64_t c = __shfl_up_sync(0xffffffffu, x.c, d);
        if (lane >= d) {
            x.a += a;
            x.b += b;
            x.c += c;
        }
    }
    __syncthreads();                               // the last scan's sums are read
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    total = {0, 0, 0};
    for (int w = 0; w < kPagedPlanThreads / 32; ++w) {
        const PagedSums s = warp_sum[w];
        if (w < warp) {
            x.a += s.a;
            x.b += s.b;
            x.c += s.c;
        }
        total.a += s.a;
        total.b += s.b;
        total.c += s.c;
    }
    return x;
}

// Where position p of the weights falls in the units; a cut that would leave a piece
// of less than two key tiles goes to the unit's start or to the next one's.
__device__ __forceinline__ PagedCut paged_cut(const PagedPlan &p, int64_t pos, int32_t n_entries)
{
    int32_t lo = 0, hi = n_entries - 1;            // the last entry that starts at pos or before
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (p.entries[mid].before <= pos)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int32_t n = p.entries[lo].n_tiles, weight = n + kPagedUnitTiles;
    const int64_t in = pos - p.entries[lo].before;
    PagedCut c;
    c.entry = lo;
    c.hu = (int32_t)divide(in, weight);
    const int32_t off = (int32_t)(in - (int64_t)c.hu * weight), kt = off - kPagedUnitTiles / 2;
    c.kt = kt < 2 ? 0 : kt;
    if (n < 4 ? 2 * off >= weight : kt > n - 2) {
        c.kt = 0;
        ++c.hu;
    } else if (n < 4) {
        c.kt = 0;
    }
    if (c.hu == p.head_units) {
        c.hu = 0;
        ++c.entry;
    }
    return c;
}

// Bytes a ns of an SM's few-row warps beside tiles (an SM alone copies faster than when all
// share the memory).  Taken as 53, as 65, as 70: 48 single tokens beside 2107 of chunks 262, 255,
// 266 us; 100 beside a prompt of 2048 192, 168, 166; 16 beside two chunks of 512 129, 133, 137.
constexpr float kFewRate = 65.0f;
// A cluster's time a key tile beside them, for heads of 128 (of 64).  Taken as 900 (700), 1100
// (900), 1300 (1050), 1500 (1200), us: 48 single tokens beside 2107 of chunks 250, 246, 263, 286;
// 16 beside two chunks of 512 61.8, 55.5, 60.0, 64.2; 30 beside two of 300 71, 63, 63, 66; 64
// beside four of 512 129, 117, 115, 118; 100 beside a prompt of 2048 159, 152, 152, 149; groups of
// 16, 64 beside a chunk of 1024 80, 85, 91, 96; heads of 64, 16 beside two of 512 46.0, 44.3, 43.3,
// 45.6, 48 beside a prompt of 2048 70, 65, 66, 69.  (Tiles alone take all clusters whatever it is.)
template <int D>
constexpr int32_t kPagedTileNs = D == 128 ? 1100 : 900;

// Estimated time, in ns, with c clusters on the tiles and the few-row chunks on the
// SMs left over (as plan_ns: an estimate that is off costs balance, never a result).
__device__ __forceinline__ float paged_ns(const PagedPlan &p, int32_t c, float weight, float chunks)
{
    const float bytes = chunks * (float)p.heads * (float)p.chunk_bytes;
    const float tiles = c > 0 ? weight * (float)p.tile_ns / (float)c : 0.0f;
    if (bytes == 0.0f)
        return tiles;
    if (2 * c >= p.grid)
        return tiles + 10000.0f + bytes / fminf(6600.0f, kFewRate * (float)p.grid);
    const float few = bytes / fminf(6600.0f, kFewRate * (float)(p.grid - 2 * c));
    return fmaxf(tiles, few) + 0.05f * fminf(tiles, few);
}

static __device__ void paged_plan(const PagedPlan &p)
{
    __shared__ int32_t entry_start[kMaxDecodeBatch + 1];
    __shared__ PagedSums warp_sum[kPagedPlanThreads / 32];
    __shared__ uint32_t best[kPagedPlanThreads / 32][2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool bad = false;
    for (int32_t b = tid; b < p.n_seqs; b += kPagedPlanThreads) {
        int32_t Lq, Lk;
        bad = bad || !paged_sequence(p.cu, p.lens, b, p.total_q, p.most_keys, Lq, Lk);
    }
    bad = __syncthreads_or(bad);
    if (bad) {                                     // nothing is written
        if (tid == 0) {
            atomicOr(p.flag, kFlagIndex);
            p.deal->clusters = 0;
            p.deal->chunks = 0;
            p.deal->few_tokens = 0;
            p.deal->per = 1;
        }
        return;
    }
    // entries, chunks and few-row tokens of the sequences before each
    PagedSums carry = {0, 0, 0};                   // chunks, few-row tokens, entries
    for (int32_t b0 = 0; b0 < p.n_seqs; b0 += kPagedPlanThreads) {
        const int32_t b = b0 + tid;
        PagedSums x = {0, 0, 0};
        if (b < p.n_seqs) {
            int32_t Lq, Lk;
            paged_sequence(p.cu, p.lens, b, p.total_q, p.most_keys, Lq, Lk);
            if (Lq > 0 && paged_few(Lq, p.group)) {
                x.a = (int32_t)(((int64_t)Lk + (1 << p.chunk_shift) - 1) >> p.chunk_shift);
                x.a += x.a > 0 ? kFewPairCost : 0;
                x.b = Lq;
            } else {
                x.c = ((int64_t)Lq + p.tile_tokens - 1) / p.tile_tokens;
            }
        }
        PagedSums total;
        const PagedSums inc = paged_scan(x, total, warp_sum);
        if (b < p.n_seqs) {
            p.chunk_start[b] = carry.a + inc.a - x.a;
            p.few_start[b] = carry.b + inc.b - x.b;
            for (int32_t i = 0; i < x.b; ++i)
                p.few_seq[carry.b + inc.b - x.b + i] = b;
            entry_start[b] = (int32_t)(carry.c + inc.c - x.c);
        }
        carry.a += total.a;
        carry.b += total.b;
        carry.c += total.c;
    }
    const int32_t n_entries = (int32_t)carry.c;
    if (tid == 0) {
        p.chunk_start[p.n_seqs] = carry.a;
        p.few_start[p.n_seqs] = carry.b;
        entry_start[p.n_seqs] = n_entries;
    }
    __syncthreads();
    // the entries, and their weights' sums
    int64_t weight = 0;
    for (int32_t e0 = 0; e0 < n_entries; e0 += kPagedPlanThreads) {
        const int32_t e = e0 + tid;
        PagedEntry x = {};
        PagedSums w = {0, 0, 0};
        if (e < n_entries) {
            x.seq = find_sequence(entry_start, p.n_seqs + 1, e);
            paged_sequence(p.cu, p.lens, x.seq, p.total_q, p.most_keys, x.Lq, x.Lk);
            x.q_start = __ldg(p.cu + x.seq);
            x.tok0 = (e - entry_start[x.seq]) * p.tile_tokens;
            x.n_tiles = packed_key_tiles(x.tok0, p.tile_tokens, x.Lq, x.Lk, p.causal);
            w.c = (int64_t)p.head_units * (x.n_tiles + kPagedUnitTiles);
        }
        PagedSums total;
        const PagedSums inc = paged_scan(w, total, warp_sum);
        if (e < n_entries) {
            x.before = weight + inc.c - w.c;
            p.entries[e] = x;
        }
        weight += total.c;
    }
    // clusters for the tiles
    const int64_t units = (int64_t)n_entries * p.head_units, runs = weight / kPagedMinRun, most = runs > units ? runs : units;
    const int32_t top = weight == 0 ? 0 : (int32_t)(most < p.grid / 2 ? most : p.grid / 2);
    if (warp * 32 < kPagedClusters) {
        const int32_t c = tid + 1;
        const uint32_t t = c <= top ? __float_as_uint(paged_ns(p, c, (float)weight, (float)carry.a)) : 0xffffffffu;
        const uint32_t m = __reduce_min_sync(0xffffffffu, t);
        const uint32_t at = __reduce_min_sync(0xffffffffu, t == m ? (uint32_t)c : 0xffffffffu);
        if (lane == 0) {
            best[warp][0] = m;
            best[warp][1] = at;
        }
    }
    __syncthreads();                               // (the entries are written, too)
    uint32_t m = best[0][0], at = best[0][1];
    for (int w = 1; w * 32 < kPagedClusters; ++w) {
        if (best[w][0] < m) {
            m = best[w][0];
            at = best[w][1];
        }
    }
    const int32_t clusters = weight == 0 ? 0 : (int32_t)at;
    if (tid <= clusters && clusters > 0) {
        const int64_t per = (weight + clusters - 1) / clusters, pos = per * tid;
        PagedCut c = {n_entries, 0, 0};
        if (pos < weight && tid < clusters)
            c = paged_cut(p, pos, n_entries);
        p.deal->cut[tid] = c;
    }
    if (tid == 0) {
        const int32_t used = 2 * clusters < p.grid ? 2 * clusters : 0;
        p.deal->clusters = clusters;
        p.deal->chunks = carry.a;
        p.deal->few_tokens = carry.b;
        p.deal->per = decode_per_warp((int64_t)carry.a * p.heads, (p.grid - used) * kFewWarps);
    }
}

// The plan (CTA 0), and the maps of last pages (the others, a sequence a warp).
static __global__ void __launch_bounds__(kPagedPlanThreads)
    rope_paged_plan_kernel(const PagedPlan p, const __grid_constant__ CUtensorMap tmpl)
{
    __shared__ __align__(128) CUtensorMap buf[kPagedPlanThreads / 32];
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) {
        paged_plan(p);
        return;
    }
    constexpr int kWarps = kPagedPlanThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    CUtensorMap *mine = &buf[warp];
    for (int32_t b = ((int)blockIdx.x - 1) * kWarps + warp; b < p.n_seqs; b += ((int)gridDim.x - 1) * kWarps) {
        int32_t Lq, Lk;
        const int32_t page = 1 << p.page_shift;
        if (!paged_sequence(p.cu, p.lens, b, p.total_q, p.most_keys, Lq, Lk) || Lq == 0 || paged_few(Lq, p.group) ||
            (Lk & (page - 1)) == 0)
            continue;
        reinterpret_cast<uint32_t *>(mine)[lane] = reinterpret_cast<const uint32_t *>(&tmpl)[lane];
        __syncwarp();
        if (lane == 0)
            asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;"
                         ::"r"(attn_smem_u32(mine)), "r"(Lk & (page - 1))
                         : "memory");
        __syncwarp();
        asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync."
                     "aligned [%0], [%1], 128;"
                     ::"l"(p.maps + b), "r"(attn_smem_u32(mine))
                     : "memory");
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// the few-row sequences: what their runs (ChunkAt, suffix_run, SuffixCopies) and few_pair ask

struct PagedFew {
    AttnArgs a;                                // cos, sin (null: queries as they are), table_rows, scale, flag
    CUtensorMap k_map, v_map;                  // boxes of 64 features x a chunk's keys, or a page's
    const void *q;                             // [total_q][Hq][D], token stride q_stride
    int64_t q_stride;
    const int32_t *table, *lens, *cu, *pos_q;
    int64_t max_blocks, n_pages;
    int32_t n_seqs, Hq, Hk, page_shift, chunk_shift, row_groups, rows;
    const int32_t *chunk_start, *few_start;
    float *out;                                // [rows of all parts][D]
    float2 *stats;

    static constexpr int32_t kPairCost = kFewPairCost;
    __device__ __forceinline__ int32_t sequences() const { return n_seqs; }
    __device__ __forceinline__ int32_t heads() const { return Hk * row_groups; }
    __device__ __forceinline__ int64_t most_keys() const { return max_blocks << page_shift; }
    __device__ __forceinline__ int32_t tokens(int32_t b) const { return __ldg(cu + b + 1) - __ldg(cu + b); }
    // (offsets and lengths are in range: otherwise the plan has no chunks)
    __device__ __forceinline__ int32_t keys(int32_t b, int64_t) const
    {
        const int32_t Lq = tokens(b);
        return Lq > 0 && paged_few(Lq, Hq / Hk) ? __ldg(lens + b) : 0;
    }
    __device__ __forceinline__ const int32_t *blocks(int32_t b, int64_t &listed) const
    {
        listed = max_blocks;
        return table + b * max_blocks;
    }
    // Rows of a pair: heads of a token, token after token; with more than 16 heads in
    // a group 16 of one token.
    template <typename T, int D>
    __device__ __forceinline__ const T *query(int32_t b, int32_t hr, int32_t r, int32_t &token) const
    {
        const int32_t kv = hr / row_groups, group = Hq / Hk, h0 = (hr - kv * row_groups) * rows;
        const int32_t start = __ldg(cu + b), Lq = __ldg(cu + b + 1) - start;
        const int32_t tok = r / rows, h = h0 + r - tok * rows;
        token = start + tok;
        return tok < Lq && h < group ? static_cast<const T *>(q) + token * q_stride + (int64_t)(kv * group + h) * D
                                     : nullptr;
    }
    __device__ __forceinline__ int64_t query_turn(int32_t b, int32_t token, int64_t) const
    {
        return row_of(token, (int64_t)__ldg(lens + b) - (__ldg(cu + b + 1) - token));
    }
    // Table row of a token: pos_q's, or its index among its sequence's keys.  -1: as it is.
    __device__ __forceinline__ int64_t row_of(int32_t token, int64_t index) const
    {
        if (a.cos == nullptr)
            return -1;
        const int64_t row = pos_q != nullptr ? (int64_t)__ldg(pos_q + token) : index;
        if (row >= 0 && row < a.table_rows)
            return row;
        // (a token before the sequence's first key sees none when causal: its row does not matter)
        if (pos_q != nullptr ? row != -1 : !(a.causal && row < 0))
            atomicOr(a.flag, kFlagPosition);
        return -1;
    }
    __device__ __forceinline__ int32_t limit(int32_t b, int32_t r, int32_t n) const
    {
        if (!a.causal)
            return n;
        const int32_t seen = n - tokens(b) + r / rows + 1;
        return seen < n ? seen : n;
    }
    // Whether a sequence's pairs fill a product's eight columns twice.
    __device__ __forceinline__ bool wide(int32_t b) const { return tokens(b) * (Hq / Hk) > 8; }
    // A run's part of a pair has as many rows as the pair, at row 16 w + the rows of the
    // pairs before it: the run w, the pair or both grow from one part to the next, a pair
    // has at most 16 rows, so parts do not meet.
    __device__ __forceinline__ int64_t part_row(int32_t w, int32_t b, int32_t hr) const
    {
        const int32_t kv = hr / row_groups, group = Hq / Hk;
        const int64_t in = row_groups > 1 ? (int64_t)kv * group + (hr - kv * row_groups) * rows
                                          : (int64_t)kv * group * tokens(b);
        return 16 * (int64_t)w + (int64_t)__ldg(few_start + b) * Hq + in;
    }
    __device__ __forceinline__ int32_t part_rows(int32_t b, int32_t hr) const
    {
        const int32_t kv = hr / row_groups, group = Hq / Hk, left = group - (hr - kv * row_groups) * rows;
        return row_groups > 1 ? (left < rows ? left : rows) : group * tokens(b);
    }
    __device__ __forceinline__ void publish(const int32_t *, int64_t) const {}     // (the plan has done so)
};

// The products are turned round, keys and features being the 16 rows of an mma and the
// pair's rows its eight columns,
//   S^T = K q^T (16 keys x 8 rows),  O^T += V^T P^T (16 features x 8 rows),
// so that a product, an exponential or an accumulator is spent on eight rows, not on 16:
// with a row of S per thread as in decode_suffixes, one token of a group of four used a
// quarter of each (48 single tokens beside 2107 of chunks 308 us, 260 so).  P leaves S^T's
// accumulators in 16 bits and gets to its operand's place by movmatrix.
//
// Every product comes twice.  A pair of at most eight rows has its rot(q) and P in two 16-bit
// parts, the rounded value and what it leaves, so nothing is rounded to 16 bits on the way; a
// wide one has its second eight rows in the parts' place, rounded.  Either way the loop still
// waits for its copies (drafts in wide pairs, 64 of four tokens in groups of four: 109 us, 133
// as tiles; 64 of twelve, heads of 64: 107 and 213).
__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// a and b rounded to 16 bits in one word, and the word of what that leaves.
template <typename T>
__device__ __forceinline__ uint32_t split2(float a, float b, uint32_t &low)
{
    const uint32_t high = Elt<T>::f2_to_word(a, b);
    const float2 h = Elt<T>::word_to_f2(high);
    low = Elt<T>::f2_to_word(a - h.x, b - h.y);
    return high;
}

// Rows first .. first + 7 of the queries of pair (b, hr) (zeros past its rows): a lane's
// words of them, rotated in fp32 and split into two 16-bit parts.
template <typename T, int LAYOUT, int D>
struct FewQueries {
    static constexpr int L = D / 16, kAtOnce = 32 / L, kSteps = 8 / kAtOnce;
    uint4 x0[kSteps], x1[kSteps], y0[kSteps], y1[kSteps];      // the rounded values, and what they leave
    int64_t trow[kSteps];
    __device__ __forceinline__ void request(const PagedFew &g, const ChunkAt &at, int64_t most, const RowPart &part, int first)
    {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
            trow[i] = -1;
            int32_t token;
            const T *row = g.template query<T, D>(at.b, at.hr, first + i * kAtOnce + (threadIdx.x & 31) / L, token);
            if (row != nullptr) {
                x0[i] = __ldg(reinterpret_cast<const uint4 *>(row + part.o0));
                x1[i] = __ldg(reinterpret_cast<const uint4 *>(row + part.o1));
                if (part.rot)
                    trow[i] = g.query_turn(at.b, token, most);
            }
        }
    }
    __device__ __forceinline__ void turn(const PagedFew &g)
    {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            y0[i] = y1[i] = make_uint4(0, 0, 0, 0);
            if (trow[i] >= 0) {
                float c[8], s[8], f0[8], f1[8];
                table_values(g.a.cos, g.a.sin, trow[i] * (g.a.rotary_dim / 2) + 8 * ((threadIdx.x & 31) % L), c, s);
                Elt<T>::unpack(x0[i], f0);
                Elt<T>::unpack(x1[i], f1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (LAYOUT == 0)
                        rotate_pair(f0[e], f1[e], c[e], s[e]);
                    else if (e < 4)
                        rotate_pair(f0[2 * e], f0[2 * e + 1], c[e], s[e]);
                    else
                        rotate_pair(f1[2 * e - 8], f1[2 * e - 7], c[e], s[e]);
                }
                uint32_t *h0 = &x0[i].x, *h1 = &x1[i].x, *l0 = &y0[i].x, *l1 = &y1[i].x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h0[e] = split2<T>(f0[2 * e], f0[2 * e + 1], l0[e]);
                    h1[e] = split2<T>(f1[2 * e], f1[2 * e + 1], l1[e]);
                }
            }
        }
    }
    // Through the warp's tile into the B operand of every 16-feature step.
    static __device__ __forceinline__ void operand(const uint4 (&a)[kSteps], const uint4 (&b)[kSteps], const RowPart &part,
                                                   uint8_t *tile, uint32_t (&f)[D / 16][2])
    {
        const int lane = threadIdx.x & 31;
        __syncwarp();                          // the tile's last readers are done
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            uint8_t *to = tile + (i * kAtOnce + lane / L) * kDecQStride<D>;
            *reinterpret_cast<uint4 *>(to + part.o0 * 2) = a[i];
            *reinterpret_cast<uint4 *>(to + part.o1 * 2) = b[i];
        }
        __syncwarp();
        // lanes 8 m ..: rows 0-7, features 8 m .. of two steps
        const uint32_t addr = attn_smem_u32(tile) + (lane & 7) * kDecQStride<D> + (lane >> 3) * 16;
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
            uint32_t r[4];
            ldsm4(addr + k * 32, r);
            f[k][0] = r[0]; f[k][1] = r[1]; f[k + 1][0] = r[2]; f[k + 1][1] = r[3];
        }
    }
};

// A pair's queries as the two operands of few_pair.
template <typename T, int LAYOUT, int D, bool WIDE>
__device__ __forceinline__ void load_few_queries(const PagedFew &g, const ChunkAt &at, int64_t most, uint8_t *tile,
                                                 uint32_t (&qa)[D / 16][2], uint32_t (&qb)[D / 16][2])
{
    using Q = FewQueries<T, LAYOUT, D>;
    const RowPart part = row_part<LAYOUT>((threadIdx.x & 31) % Q::L, g.a.rotary_dim);
    Q q, second;
    q.request(g, at, most, part, 0);
    if constexpr (WIDE)
        second.request(g, at, most, part, 8);
    q.turn(g);
    Q::operand(q.x0, q.x1, part, tile, qa);
    if constexpr (WIDE) {
        second.turn(g);
        Q::operand(second.x0, second.x1, part, tile, qb);
    } else {
        Q::operand(q.y0, q.y1, part, tile, qb);
    }
}

// The softmax of a thread's two columns (rows r0 and r0 + 1 of eight).
struct FewColumns {
    float m[2], l[2];
    __device__ __forceinline__ void clear()
    {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
    }
    // The reference maxima move only when a key exceeds them by more than 8 (a factor of
    // 256), so the lanes of a row seldom have to agree on its maximum.  True (for all lanes):
    // what is accumulated has to be scaled by f.
    template <int kGroups>
    __device__ __forceinline__ bool maxima(const float (&s)[kGroups][4], float scale_log2, float (&f)[2])
    {
        float x[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            x[c] = fmaxf(s[0][c], s[0][2 + c]);
#pragma unroll
            for (int n = 1; n < kGroups; ++n)
                x[c] = fmaxf(x[c], fmaxf(s[n][c], s[n][2 + c]));
            x[c] *= scale_log2;                // (the scale is positive)
        }
        if (!__any_sync(0xffffffffu, x[0] > m[0] + 8.0f || x[1] > m[1] + 8.0f))
            return false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                x[c] = fmaxf(x[c], __shfl_xor_sync(0xffffffffu, x[c], d));
            const bool up = x[c] > m[c] + 8.0f;
            f[c] = up ? (m[c] == -INFINITY ? 0.0f : fast_exp2(m[c] - x[c])) : 1.0f;
            m[c] = up ? x[c] : m[c];
            l[c] *= f[c];
        }
        return true;
    }
    __device__ __forceinline__ void weights(const float (&s)[4], float scale_log2, float (&p)[4])
    {
        const float n0 = m[0] == -INFINITY ? 0.0f : -m[0], n1 = m[1] == -INFINITY ? 0.0f : -m[1];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = fast_exp2(fmaf(s[i], scale_log2, i & 1 ? n1 : n0));
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
    }
    __device__ __forceinline__ void sums()
    {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
        }
    }
};

// A warp's way through its stages.
struct FewStages {
    uint64_t *bar;
    uint8_t *stages;
    int st;
    uint32_t ph;
    int64_t issued, done;
};

// `count` chunks of pair (at.b, at.hr), from chunk at.ch on, and their part of the pair; false
// after an expired wait.  The two operands, their outputs and softmax: rows 0-7 rounded, and
// what that leaves of them, or (WIDE) rows 8-15.
template <typename T, int LAYOUT, int D, bool WIDE>
__device__ __forceinline__ bool few_pair(const PagedFew &g, SuffixCopies<D, PagedFew> &copies, FewStages &f, uint8_t *qtile,
                                         ChunkAt &at, int32_t count, int32_t w, int64_t most, volatile int *abort)
{
    constexpr int kStages = kDecStages<D>, kStage = kDecStageBytes<D>, kKeys = kDecKeys<D>;
    constexpr int kBox = kKeys * 128, kGroups = kKeys / 16, kSets = WIDE ? 2 : 1;
    const int lane = threadIdx.x & 31;
    const int r0 = 2 * (lane & 3), k0 = lane >> 2;             // S^T: keys k0 and k0 + 8 of 16
    // ldmatrix rows: K (two 8-key halves x two 8-feature halves of a step), V (the same,
    // turned: two 8-feature halves x two 8-key halves)
    const int k_row = lane & 15, k_half = lane >> 4;
    const int v_row = (lane & 7) + ((lane >> 4) << 3), v_half = lane >> 3 & 1;
    const uint32_t base = attn_smem_u32(f.stages);
    const int32_t keys = g.keys(at.b, most), low = g.limit(at.b, 0, keys);     // of the pair; that all rows see
    int32_t lim[kSets][2];                                     // that the thread's rows see
#pragma unroll
    for (int x = 0; x < kSets; ++x) {
        lim[x][0] = g.limit(at.b, 8 * x + r0, keys);
        lim[x][1] = g.limit(at.b, 8 * x + r0 + 1, keys);
    }
    uint32_t qa[D / 16][2], qb[D / 16][2];
    load_few_queries<T, LAYOUT, D, WIDE>(g, at, most, qtile, qa, qb);
    float o[kSets][D / 16][4];                                 // features lane / 4 and + 8 of 16, rows r0 and r0 + 1
    FewColumns soft[kSets];
#pragma unroll
    for (int x = 0; x < kSets; ++x) {
        soft[x].clear();
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.0f;
    }
    for (; count > 0; --count, ++at.ch, ++f.done) {
        if (!__all_sync(0xffffffffu, attn_wait(&f.bar[f.st], f.ph, abort)))
            return false;
        const uint32_t kb = base + f.st * kStage, vb = kb + kStage / 2;
        float s[2][kGroups][4];                                // (key k0, rows r0, r0 + 1), (key k0 + 8, the same)
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[0][n][i] = s[1][n][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t a[4];
                const int chunk = (k & 3) * 2 + k_half;
                ldsm4(kb + (k >> 2) * kBox + (n * 16 + k_row) * 128 + ((chunk ^ (k_row & 7)) << 4), a);
                mma16816<T>(s[0][n], a, qa[k][0], qa[k][1]);
                mma16816<T>(s[1][n], a, qb[k][0], qb[k][1]);
            }
            if constexpr (!WIDE) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[0][n][i] += s[1][n][i];
            }
        }
        if (low - at.ch * kKeys < kKeys) {                     // keys that some row does not see
#pragma unroll
            for (int x = 0; x < kSets; ++x) {
                const int32_t n0 = lim[x][0] - at.ch * kKeys, n1 = lim[x][1] - at.ch * kKeys;
#pragma unroll
                for (int n = 0; n < kGroups; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n * 16 + k0 + (i >> 1) * 8 >= (i & 1 ? n1 : n0))
                            s[x][n][i] = -INFINITY;
                }
            }
            // what lies behind the last key (anything) must not meet a zero
            const int32_t nk = keys - at.ch * kKeys;
            if (nk < kKeys) {
                constexpr int kWords = D / 8;                  // 16-byte words of a value
                for (int i = nk * kWords + lane; i < kKeys * kWords; i += 32)
                    *reinterpret_cast<uint4 *>(f.stages + f.st * kStage + kStage / 2 + (i % kWords / 8) * kBox +
                                               i / kWords * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next copy
                __syncwarp();
            }
        }
#pragma unroll
        for (int x = 0; x < kSets; ++x) {
            float by[2];
            if (soft[x].maxima(s[x], g.a.scale_log2, by)) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[x][i][e] *= by[e & 1];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
            float p[4];
            uint32_t a0, a1, b0, b1;
            soft[0].weights(s[0][n], g.a.scale_log2, p);
            if constexpr (WIDE) {
                a0 = Elt<T>::f2_to_word(p[0], p[1]);
                a1 = Elt<T>::f2_to_word(p[2], p[3]);
                soft[kSets - 1].weights(s[1][n], g.a.scale_log2, p);
                b0 = Elt<T>::f2_to_word(p[0], p[1]);
                b1 = Elt<T>::f2_to_word(p[2], p[3]);
            } else {
                a0 = split2<T>(p[0], p[1], b0);
                a1 = split2<T>(p[2], p[3], b1);
            }
            a0 = transpose8(a0);
            a1 = transpose8(a1);
            b0 = transpose8(b0);
            b1 = transpose8(b1);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t a[4];
                const int chunk = (i & 3) * 2 + v_half;
                ldsm4_t(vb + (i >> 2) * kBox + (n * 16 + v_row) * 128 + ((chunk ^ (v_row & 7)) << 4), a);
                mma16816<T>(o[0][i], a, a0, a1);
                mma16816<T>(o[kSets - 1][i], a, b0, b1);
            }
        }
        __syncwarp();                                          // the stage is read
        if (copies.left > 0) {
            copies.load(f.st);
            ++f.issued;
        }
        if (++f.st == kStages) {
            f.st = 0;
            f.ph ^= 1u;
        }
    }
    const int64_t row0 = g.part_row(w, at.b, at.hr);
    const int32_t rows = g.part_rows(at.b, at.hr);
#pragma unroll
    for (int x = 0; x < kSets; ++x) {
        soft[x].sums();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = 8 * x + r0 + half;
            if (r < rows) {
                float *dst = g.out + (row0 + r) * D + k0;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    dst[16 * i] = o[x][i][half];
                    dst[16 * i + 8] = o[x][i][2 + half];
                }
                if (k0 == 0)
                    g.stats[row0 + r] = make_float2(soft[x].m[half], soft[x].l[half]);
            }
        }
    }
    return true;
}

// One warp's run of chunks; smem: kFewSmem bytes of the CTA.
template <typename T, int LAYOUT, int D>
__device__ __forceinline__ void paged_few_run(const PagedFew &g, uint8_t *smem, const SuffixRun &run,
                                              SuffixShared<D, kFewWarps> &sh)
{
    constexpr int kStages = kDecStages<D>, kStage = kDecStageBytes<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t most = g.most_keys();
    int64_t left = run.left;
    ChunkAt at = run.at;
    if (left <= 0)
        return;
    FewStages f = {sh.bar[warp], smem + warp * kStages * kStage, 0, 0, 0, 0};
    uint8_t *qtile = smem + kFewWarps * kStages * kStage + warp * kFewQuery<D>;
    volatile int *abort = &sh.abort_flag;
    SuffixCopies<D, PagedFew> copies(g, run, most, f.stages, f.bar);
    bool ok = true;
    for (int st = 0; st < kStages && copies.left > 0; ++st, ++f.issued)
        copies.load(st);
    while (ok && left > 0) {
        const int32_t here = at.n - at.ch, count = here < left ? here : (int32_t)left;
        left -= count;
        ok = g.wide(at.b) ? few_pair<T, LAYOUT, D, true>(g, copies, f, qtile, at, count, run.w, most, abort)
                          : few_pair<T, LAYOUT, D, false>(g, copies, f, qtile, at, count, run.w, most, abort);
        if (ok && left > 0) {
            --at.ch;
            at.next(g, most);
            left -= kFewPairCost;
        }
    }
    if (!ok) {
        *abort = 1;
        if (lane == 0)
            atomicOr(g.a.flag, kFlagTimeout);
        // one more bounded wait for the copies in flight
        for (int64_t i = f.done; i < f.issued; ++i)
            (void)attn_wait(&f.bar[i % kStages], (uint32_t)(i / kStages) & 1u);
    }
}

// ---------------------------------------------------------------------------
// the tiles, with the few-row sequences beside or behind them

struct PagedSource {
    static constexpr bool kFullUnroll = true;
    static constexpr bool kParts = true, kAllParts = false;
    static constexpr bool kFinish = true;
    template <int D>
    static constexpr int smem_bytes()
    {
        const int tiles = (int)kPackedSmem<D> + 4 * (kMaxDecodeBatch + 2);
        return tiles > kFewSmem<D> ? tiles : kFewSmem<D>;
    }
    AttnArgs a;                                // o, Hq, cos, sin, table_rows, rotary_dim, scale, causal, flag
    CUtensorMap k_map, v_map, q_map, o_map;    // the pools; queries and outputs of all sequences
    PagedFew few;
    const PagedDeal *deal;
    const PagedEntry *entries;
    const CUtensorMap *maps;                   // [n_seqs]: last pages
    float *out;                                // [2 clusters][256][D]: a run's first piece and its last
    float2 *stats;
    int32_t head_units, units_per_kv, tile_tokens;

    using Cursor = PagedCut;
    struct Walk {
        PagedCut begin, end;
        int32_t cid, clusters, chunks;
    };
    template <int D>
    __device__ __forceinline__ Walk walk(int64_t cid, int64_t, uint8_t *) const
    {
        Walk w;
        w.cid = (int32_t)cid;
        w.clusters = __ldg(&deal->clusters);
        w.chunks = __ldg(&deal->chunks);
        w.begin = w.end = {0, 0, 0};
        if (w.cid < w.clusters) {
            w.begin = load_cut(w.cid);
            w.end = load_cut(w.cid + 1);
        }
        return w;
    }
    __device__ __forceinline__ PagedCut load_cut(int32_t i) const
    {
        const PagedCut *c = deal->cut + i;
        return {__ldg(&c->entry), __ldg(&c->hu), __ldg(&c->kt)};
    }
    __device__ __forceinline__ Cursor first(const Walk &w) const { return w.begin; }
    __device__ __forceinline__ bool valid(const Walk &w, const Cursor &c) const { return c.before(w.end); }
    __device__ __forceinline__ int32_t tiles(const Walk &w, const Cursor &c) const
    {
        const int32_t n = c.same_unit(w.end) ? w.end.kt : __ldg(&entries[c.entry].n_tiles);
        return n - c.kt;
    }
    __device__ __forceinline__ void next(const Walk &w, Cursor &c) const
    {
        if (c.same_unit(w.end)) {
            c.kt = w.end.kt;
            return;
        }
        c.kt = 0;
        if (++c.hu == head_units) {
            c.hu = 0;
            ++c.entry;
        }
    }
    __device__ __forceinline__ PackedUnit unit(const Walk &w, const Cursor &c, int lg) const
    {
        const int4 x = __ldg(reinterpret_cast<const int4 *>(entries + c.entry));
        const int2 y = __ldg(reinterpret_cast<const int2 *>(entries + c.entry) + 2);
        PackedUnit u;
        u.seq = x.x; u.tok0 = x.y; u.tokens = x.z; u.n_keys = x.w;
        u.q_start = y.x; u.k_start = 0;
        u.first = c.kt;
        const bool ends = c.same_unit(w.end);      // the run's cut goes through this unit
        u.n_tiles = (ends ? w.end.kt : y.y) - c.kt;
        u.head0 = c.hu << lg;
        u.kv = c.hu / units_per_kv;
        u.part = c.kt == 0 && !ends ? -1 : 2 * w.cid + (c.same_unit(w.begin) ? 0 : 1);
        return u;
    }
    __device__ __forceinline__ int64_t table_row(const PackedUnit &u, int32_t t) const
    {
        return few.row_of(u.q_start + t, (int64_t)u.n_keys - u.tokens + t);
    }

    // z of page i of the unit's sequence in the pools' maps; past the last page, and for
    // a bad page number, an index that arrives as zeros
    __device__ __forceinline__ int32_t page_z(const PackedUnit &u, int32_t i) const
    {
        const int32_t none = (int32_t)(few.n_pages * few.Hk);
        if ((int64_t)i << few.page_shift >= u.n_keys)
            return none;
        const int32_t p = __ldg(few.table + u.seq * few.max_blocks + i);
        if (p < 0 || p >= few.n_pages) {
            atomicOr(a.flag, kFlagIndex);
            return none;
        }
        return p * few.Hk + u.kv;
    }
    // (keys that other units read too stay in L2)
    __device__ __forceinline__ uint64_t policy(const PackedUnit &u) const
    {
        return u.tokens > tile_tokens || units_per_kv > 1 ? l2_keep() : l2_once();
    }
    template <int D>
    __device__ __forceinline__ int32_t key_place(const PackedUnit &u, int32_t kt, uint32_t rank, int lane) const
    {
        const int32_t shift = few.page_shift < 6 ? few.page_shift : 6;  // keys of a box: a page or half of one
        const int32_t key = (u.first + kt) * kAttnKeys + 64 * (int)rank + (lane / (D / 64) << shift);
        return lane < (64 >> shift) * (D / 64) ? page_z(u, key >> few.page_shift) : 0;
    }
    template <int D>
    __device__ __forceinline__ int32_t value_place(const PackedUnit &u, int32_t kt, int lane) const
    {
        return lane < kAttnKeys >> few.page_shift
                   ? page_z(u, ((u.first + kt) * kAttnKeys >> few.page_shift) + lane)
                   : 0;
    }
    __device__ __forceinline__ void acquire(const PackedUnit &u, int32_t &seq) const
    {
        if (u.seq != seq && (u.n_keys & ((1 << few.page_shift) - 1)) != 0)
            acquire_map(maps + u.seq);
        seq = u.seq;
    }
    template <int D>
    __device__ __forceinline__ void load_keys(const PackedUnit &u, int32_t, int32_t z, uint8_t *dst,
                                              uint64_t *bar, uint32_t rank, int lane) const
    {
        const int32_t shift = few.page_shift < 6 ? few.page_shift : 6;
        if (lane < (64 >> shift) * (D / 64)) {
            const int32_t i = lane / (D / 64), x = lane % (D / 64);
            load_half_box_l2(dst + x * 8192 + (i << shift) * 128, &k_map, x * 64,
                             (64 * (int)rank + (i << shift)) & ((1 << few.page_shift) - 1), z, bar, rank,
                             policy(u));
        }
    }
    template <int D>
    __device__ __forceinline__ void load_values(const PackedUnit &u, int32_t kt, int32_t z, uint8_t *dst,
                                                uint64_t *bar, uint32_t rank, int lane) const
    {
        if (lane < kAttnKeys >> few.page_shift) {
            const int32_t page = ((u.first + kt) * kAttnKeys >> few.page_shift) + lane;
            // the last, partly filled page: rows past the sequence's end arrive as zeros
            const bool tail = page == u.n_keys >> few.page_shift && (u.n_keys & ((1 << few.page_shift) - 1)) != 0;
            load_half_box_l2(dst + (lane << few.page_shift) * D, tail ? maps + u.seq : &v_map,
                             D / 2 * (int)rank, 0, z, bar, rank, policy(u));
        }
    }
    // One helper warp: its rows' O, m and l of a piece, in fp32
    template <int D>
    __device__ __forceinline__ void store_rows(const PackedUnit &u, uint32_t o_base, int32_t y0, int lane,
                                               int lg, float2 stat) const
    {
        const int64_t row = (int64_t)u.part * (2 * kAttnRows) + ((y0 - u.tok0) << lg) + lane;
        const bool live = y0 + (lane >> lg) < u.tokens;
        if (live)
            stats[row] = stat;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
            float ov[32];
            tmem_ld32(o_base + c0, ov);
            if (live) {
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                    *reinterpret_cast<float4 *>(out + row * D + c0 + c) =
                        make_float4(ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
            }
        }
    }
    // The few-row sequences, on the CTAs without tiles, or on all behind them (as
    // PrefixSource::finish).
    template <typename T, int LAYOUT, int D>
    __device__ __forceinline__ void finish(const Walk &w, uint8_t *smem, bool failed) const
    {
        __shared__ SuffixShared<D, kFewWarps> sh;
        const int32_t used = 2 * w.clusters < (int32_t)gridDim.x ? 2 * w.clusters : 0;
        const int32_t cta = (int32_t)blockIdx.x - used;
        // (after an expired wait copies may still be on their way: no work)
        if (w.chunks == 0 || cta < 0 || failed)
            return;
        int32_t *start = reinterpret_cast<int32_t *>(smem + kPackedSmem<D>);
        for (int32_t b = threadIdx.x; b <= few.n_seqs; b += kPackedThreads)
            start[b] = __ldg(few.chunk_start + b);
        __syncthreads();
        const int32_t ctas = (int32_t)gridDim.x - used;
        const SuffixRun run = suffix_run<D>(few, start, w.chunks, cta, ctas, sh);
        // registers: from the roles' 240 / 112 / 104 to 168 for all
        if (threadIdx.x < 128)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 168;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        paged_few_run<T, LAYOUT, D>(few, smem, run, sh);
    }
};

// ---------------------------------------------------------------------------
// the merge: rows of cut units, a warp each, and rows of few-row sequences, W warps
// each (W > 1 where there are few of them: merge_parts)

struct PagedMerge {
    PagedFew few;
    const PagedDeal *deal;
    const PagedEntry *entries;
    const float *out;
    const float2 *stats;
    void *o;
    const int32_t *few_seq;
    int32_t lg;
};

// A row of the few-row sequences: its parts, 16 rows from one to the next, and its output.
struct FewRow {
    int64_t from, to;
    int32_t n;
    __device__ __forceinline__ void find(const PagedMerge &g, int64_t row)
    {
        const PagedFew &f = g.few;
        const int32_t group = f.Hq / f.Hk, heads = f.heads();
        const int32_t t = (int32_t)divide(row, f.Hq), h = (int32_t)(row - (int64_t)t * f.Hq);
        const int32_t b = __ldcg(g.few_seq + t), tok = t - __ldcg(f.few_start + b);
        const int32_t kv = h / group, in_group = h - kv * group, rg = in_group / f.rows;
        const int32_t hr = kv * f.row_groups + rg, r = tok * f.rows + in_group - rg * f.rows;
        const int64_t c0 = __ldcg(f.chunk_start + b), c1 = __ldcg(f.chunk_start + b + 1), per = __ldcg(&g.deal->per);
        const int64_t at = c0 * heads + hr * (c1 - c0), first = divide(at + kFewPairCost, per);
        n = c1 > c0 ? (int32_t)(divide(at + (c1 - c0) - 1, per) - first + 1) : 0;
        from = f.part_row((int32_t)first, b, hr) + r;
        to = ((int64_t)__ldcg(f.cu + b) + tok) * f.Hq + h;
    }
};

template <typename T, int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) rope_paged_merge_kernel(const __grid_constant__ PagedMerge g)
{
    constexpr int kWarps = W == 1 ? 4 : W;
    const int warp = threadIdx.x >> 5;
    const PagedFew &f = g.few;
    constexpr int kRows = W == 1 ? kWarps : 1;                 // few-row rows of a CTA at once
    // The plan is complete before the attention's CTAs let this kernel start (they wait for it
    // first), so what it says of the first row is looked up beside their end; in L2, since
    // nothing before the wait below orders it against what this SM's L1 may hold.
    const int32_t clusters = __ldcg(&g.deal->clusters);
    const int64_t rows = (int64_t)__ldcg(&g.deal->few_tokens) * f.Hq;
    int64_t row = (int64_t)blockIdx.x * kRows + (W == 1 ? warp : 0);
    FewRow few = {};
    if (row < rows)
        few.find(g, row);
    pdl_wait();
    pdl_trigger();
    // Cut i, where it goes through a unit that no earlier cut goes through: that unit's
    // 256 rows, a warp each.
    constexpr int kSteps = 256 / kWarps;
    for (int32_t item = blockIdx.x; item < (clusters - 1) * kSteps; item += gridDim.x) {
        const int32_t i = 1 + item / kSteps, r = (item % kSteps) * kWarps + warp;
        const PagedCut *cut = g.deal->cut;
        const PagedCut c = cut[i], before = cut[i - 1];
        const bool shared = before.same_unit(c);
        if (c.kt == 0 || (shared && before.kt > 0))
            continue;
        const PagedEntry e = g.entries[c.entry];
        const int32_t tok = e.tok0 + (r >> g.lg);
        if (tok >= e.Lq)
            continue;
        int32_t n = 2;                                         // pieces
        for (int32_t j = i + 1; j < clusters && cut[j].same_unit(c) && cut[j].kt > 0; ++j)
            ++n;
        const int32_t first = 2 * (i - 1) + (shared ? 0 : 1);
        const int64_t to = (int64_t)(e.q_start + tok) * f.Hq + (c.hu << g.lg) + (r & ((1 << g.lg) - 1));
        merge_parts<T, D, 1>(n, g.o, to, [&](int32_t p, float2 &stat) {
            const int64_t at = (int64_t)(p == 0 ? first : 2 * (i + p - 1)) * 256 + r;
            stat = __ldg(g.stats + at);
            return g.out + at * D;
        });
    }
    // The few-row sequences: (token, head).
    for (; row < rows; row += (int64_t)gridDim.x * kRows) {
        if (row >= (int64_t)gridDim.x * kRows)
            few.find(g, row);
        if constexpr (W > 1)
            __syncthreads();                                   // the last row's parts are read
        merge_parts<T, D, W>(few.n, g.o, few.to, [&](int32_t p, float2 &stat) {
            const int64_t at = few.from + (int64_t)p * 16;
            stat = __ldg(f.stats + at);
            return (const float *)f.out + at * D;
        });
    }
}

// ---------------------------------------------------------------------------
// host side
template <typename T, int LAYOUT, int D>
static cudaError_t launch_paged(const PagedCall &c, const PagedLayout &lay, cudaStream_t st)
{
    EncodeTiledFn enc = encode_tiled();
    if (enc == nullptr)
        return cudaErrorNotSupported;
    const CUtensorMapDataType dt = std::is_same<T, __nv_bfloat16>::value
                                       ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    uint8_t *ws = static_cast<uint8_t *>(c.workspace);
    const int64_t page = (int64_t)1 << c.page_shift, z = c.n_pages * c.Hk;
    const int32_t group = c.Hq / c.Hk, gp = packed_group_heads(c.Hq, c.Hk), lg = __builtin_ctz((unsigned)gp);
    int sms = 0, dev = 0;
    cudaError_t e = sm_count(&sms, &dev);
    if (e != cudaSuccess)
        return e;
    const int32_t clusters = (sms < kDecodeSms ? sms : kDecodeSms) / 2;

    PagedSource s;
    memset(&s, 0, sizeof s);
    AttnArgs &a = s.a;
    a.o = c.o; a.Hq = c.Hq;
    a.cos = c.cos; a.sin = c.sin; a.rotary_dim = c.rotary_dim; a.table_rows = c.table_rows;
    a.scale_log2 = c.scale_log2; a.causal = c.causal; a.flag = c.flag;
    PagedFew &f = s.few;
    f.a = a;
    f.q = c.q; f.q_stride = c.q_stride;
    f.table = c.table; f.lens = c.lens; f.cu = c.cu; f.pos_q = c.pos_q;
    f.max_blocks = c.max_blocks; f.n_pages = c.n_pages;
    f.n_seqs = c.n_seqs; f.Hq = c.Hq; f.Hk = c.Hk; f.page_shift = c.page_shift;
    f.chunk_shift = __builtin_ctz((unsigned)kDecKeys<D>);
    f.rows = group < 16 ? group : 16;
    f.row_groups = (group + f.rows - 1) / f.rows;
    f.chunk_start = reinterpret_cast<int32_t *>(ws + lay.chunk_start);
    f.few_start = reinterpret_cast<int32_t *>(ws + lay.few_start);
    f.out = reinterpret_cast<float *>(ws + lay.few_out);
    f.stats = reinterpret_cast<float2 *>(ws + lay.few_stats);
    const uint32_t chunk_box = (uint32_t)(page < kDecKeys<D> ? page : kDecKeys<D>), box = (uint32_t)(page < 64 ? page : 64);
    const uint32_t g = (uint32_t)gp;
    // (without pages the pools' maps stand on the workspace, and no key is ever copied)
    const void *kp = z > 0 ? c.k_pages : ws, *vp = z > 0 ? c.v_pages : ws;
    const int64_t zs = z > 0 ? z : 1;
    if (!encode_3d(enc, &f.k_map, kp, dt, {D, page, zs}, {D * 2, page * D * 2}, {64, chunk_box, 1}, sw) ||
        !encode_3d(enc, &f.v_map, vp, dt, {D, page, zs}, {D * 2, page * D * 2}, {64, chunk_box, 1}, sw) ||
        !encode_3d(enc, &s.k_map, kp, dt, {D, page, zs}, {D * 2, page * D * 2}, {64, box, 1}, sw) ||
        !encode_3d(enc, &s.v_map, vp, dt, {D, page, zs}, {D * 2, page * D * 2}, {(uint32_t)D / 2, (uint32_t)page, 1},
                   D == 128 ? sw : CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_3d(enc, &s.q_map, c.q, dt, {D, c.Hq, c.total_q}, {D * 2, c.q_stride * 2}, {64, g, kAttnRows / g}, sw) ||
        !encode_3d(enc, &s.o_map, c.o, dt, {D, c.Hq, c.total_q}, {D * 2, (int64_t)c.Hq * D * 2}, {64, g, 32 / g}, sw))
        return cudaErrorInvalidValue;
    s.deal = reinterpret_cast<PagedDeal *>(ws);
    s.entries = reinterpret_cast<PagedEntry *>(ws + lay.entries);
    s.maps = reinterpret_cast<CUtensorMap *>(ws + lay.maps);
    s.out = reinterpret_cast<float *>(ws + lay.out);
    s.stats = reinterpret_cast<float2 *>(ws + lay.stats);
    s.head_units = c.Hq / gp; s.units_per_kv = group / gp; s.tile_tokens = 2 * kAttnRows / gp;

    PagedPlan p;
    memset(&p, 0, sizeof p);
    p.cu = c.cu; p.lens = c.lens; p.n_seqs = c.n_seqs; p.group = group; p.tile_tokens = s.tile_tokens;
    p.head_units = s.head_units; p.heads = c.Hk * f.row_groups;
    p.total_q = c.total_q; p.most_keys = c.max_blocks << c.page_shift;
    p.causal = c.causal; p.chunk_shift = f.chunk_shift; p.page_shift = c.page_shift;
    p.chunk_bytes = kDecStageBytes<D>; p.tile_ns = kPagedTileNs<D>; p.grid = 2 * clusters;
    p.deal = reinterpret_cast<PagedDeal *>(ws);
    p.entries = reinterpret_cast<PagedEntry *>(ws + lay.entries);
    p.chunk_start = reinterpret_cast<int32_t *>(ws + lay.chunk_start);
    p.few_start = reinterpret_cast<int32_t *>(ws + lay.few_start);
    p.few_seq = reinterpret_cast<int32_t *>(ws + lay.few_seq);
    p.maps = reinterpret_cast<CUtensorMap *>(ws + lay.maps);
    p.flag = c.flag;
    constexpr int32_t kWarps = kPagedPlanThreads / 32;
    e = launch_hot(rope_paged_plan_kernel, dim3((unsigned)(1 + (c.n_seqs + kWarps - 1) / kWarps)),
                   dim3(kPagedPlanThreads), 0, st, p, s.v_map);
    if (e != cudaSuccess)
        return e;
    e = launch_packed_kernel<T, LAYOUT, D>(s, clusters, lg, st);
    if (e != cudaSuccess)
        return e;
    PagedMerge m;
    memset(&m, 0, sizeof m);
    m.few = f; m.deal = s.deal; m.entries = s.entries; m.out = s.out; m.stats = s.stats; m.o = c.o;
    m.few_seq = p.few_seq; m.lg = lg;
    const unsigned grid = 4 * kDecodeSms;
    if (lay.few_rows * 8 <= kMergeWarps)
        return launch_hot(rope_paged_merge_kernel<T, D, 8>, dim3(grid), dim3(256), 0, st, m);
    if (lay.few_rows * 4 <= kMergeWarps)
        return launch_hot(rope_paged_merge_kernel<T, D, 4>, dim3(2 * grid), dim3(128), 0, st, m);
    return launch_hot(rope_paged_merge_kernel<T, D, 1>, dim3(2 * grid), dim3(128), 0, st, m);
}

template <typename T>
cudaError_t launch_paged_type(const PagedCall &c, const PagedLayout &lay, int32_t D, int32_t layout, cudaStream_t st)
{
    if (layout == 0)
        return D == 64 ? launch_paged<T, 0, 64>(c, lay, st) : launch_paged<T, 0, 128>(c, lay, st);
    return D == 64 ? launch_paged<T, 1, 64>(c, lay, st) : launch_paged<T, 1, 128>(c, lay, st);
}

}  // namespace rope
