// rope_attention_decode.cuh -- attention of one new token per sequence over a
// prefix that all sequences share and a suffix of each one's own, both in the
// pages of a cache (rope_attention_decode_fwd).
//
//   o_b = softmax(scale * rot(q_b) [K_prefix; K_b]^T) [V_prefix; V_b]
//
// A softmax over a concatenation is a merge of the parts' softmaxes: with part
// i's maximum m_i, sum l_i = sum_j 2^(s_j - m_i) and output O_i = sum_j 2^(s_j -
// m_i) v_j, and M = max m_i,
//   o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// So the parts run apart:
//   1. the prefix, for the whole batch: its rows (sequence, head) are the rows of
//      rope_attn_packed_kernel's tiles (the batch is a "sequence" of B tokens), its
//      keys come from pages, its key tiles are dealt out evenly to clusters; every
//      piece of a head's keys leaves an fp32 (O, m, l).  A key is read once for each
//      tile of 256 rows: GP heads of a group, GP the largest power of two that
//      divides the group's size (16 at most), and 256 / GP sequences;
//   2. the suffixes (decode_suffixes): every warp an equal run of chunks (16 keys, 32
//      of 64 features) of all suffixes, laid end to end, so that ragged lengths
//      balance; a key is read once for up to 16 heads of its group;
//   3. rope_decode_merge_kernel.
// 1 and 2 do not depend on one another and share a launch: every CTA works out
// from the suffixes' lengths how many clusters the prefix gets (plan_clusters);
// those run 1, the SMs of the others run 2 beside them.  (As two launches the
// parts ran one after the other, or the second kernel's last CTAs started behind
// the first: 64 sequences, 8k prefix, 70 us, so 55 then and 53 now.)  When the batch has no
// more than 16 rows per key head, the prefix is one more sequence of 2, with all
// the rows of the batch, in a kernel of 2 alone.
//
// Roundings: rot(q), and P before P V, to the element type (the operands of a 16-bit
// product), as a prompt's, so that a token's output does not tell whether it came
// with a prompt or in a step; everything else is fp32 until o.
//
// What bounds it: bytes -- the prefix once a row tile (from L2 where the batch has
// several), every suffix once; from about 300 rows per key head on, the prefix
// products.
#pragma once

#include "rope_attention_packed.cuh"

namespace rope {

// ---------------------------------------------------------------------------
// How a call is dealt out to the SMs.

constexpr int kDecWarps = 8;                       // suffix warps of an SM
// Keys of a suffix chunk: 16 of 128 features or 32 of 64, 8 KB of keys and values
// (16 keys of 64 features left a warp's chain of dependent steps too little work:
// 48 sequences, 16 heads of 64: 39 us, now 34.5).
template <int D>
static constexpr int kDecKeys = D == 128 ? 16 : 32;

// The sizes decode_plan goes by.
struct PlanSizes {
    int32_t row_tiles, head_units, tiles;          // the prefix: cluster tiles of all units
    int32_t clusters, sms;                         // most prefix clusters; SMs
    int32_t tile_ns;                               // a cluster's time per key tile
    int32_t heads, chunk_bytes;                    // pairs of a sequence; keys and values of a chunk
    float sm_rate;                                 // copies of an SM, bytes/ns
};

// The prefix on c clusters: `groups` of them (one cluster per row tile in each)
// take `per` consecutive (head unit, key tile) each.
struct PrefixDeal {
    int32_t clusters, groups, per;
};

__host__ __device__ inline PrefixDeal prefix_deal(const PlanSizes &p, int32_t c)
{
    PrefixDeal d;
    d.clusters = c;
    d.groups = c / p.row_tiles > 0 ? c / p.row_tiles : 1;
    d.per = (p.head_units * p.tiles + d.groups - 1) / d.groups;
    return d;
}

// Estimated time, in ns, with c clusters on the prefix and the suffixes' chunks
// (of one pair per sequence) on the SMs left over -- or, with every cluster on
// the prefix, behind it.  Measured here: tile_ns a cluster tile, 4 us from one
// unit to the next, sm_rate bytes/ns for the copies of one SM and 6600 for all.
// Where one side is over long before the other, a little less of it is better
// (the last term).  An estimate that is off costs balance, never a result.
// Forced to c clusters, whole calls took (us):
//   64 sequences, 8k prefix:    c = 8: 72   12: 58   16: 52.5  20: 55   76: 64
//   256 sequences, 4k prefix:   c = 4: 330  8: 332   12: 335   20: 375  76: 353
//   32 sequences, 128k prefix:  c = 60: 128 68: 117  71: 113   72: 117  76: 118
//   48 sequences, 1k prefix, heads of 64:  c = 4: 46  8: 31  12: 31.4  20: 33
// where this picks 16, 12, 72 and 14.
__host__ __device__ inline float plan_ns(const PlanSizes &p, int32_t c, float chunks)
{
    const PrefixDeal d = prefix_deal(p, c);
    const int32_t rounds = (p.row_tiles + c - 1) / c;
    const float bytes = chunks * (float)p.heads * (float)p.chunk_bytes;
    const float prefix = (float)rounds * ((float)d.per * (float)p.tile_ns +
                                          4000.0f * (float)(1 + d.per / p.tiles));
    if (bytes == 0.0f)
        return prefix;
    if (2 * c >= p.sms)
        return prefix + 10000.0f + bytes / fminf(6600.0f, p.sm_rate * (float)p.sms);
    const float suffix = bytes / fminf(6600.0f, p.sm_rate * (float)(p.sms - 2 * c));
    return fmaxf(prefix, suffix) + 0.05f * fminf(prefix, suffix);
}

// Clusters for the prefix, by every thread of a CTA (best: 2 words a warp).
__device__ __forceinline__ int32_t plan_clusters(const PlanSizes &p, int64_t chunks, uint32_t (*best)[2])
{
    const int32_t c = threadIdx.x + 1, warp = threadIdx.x >> 5;
    if (warp * 32 < p.clusters) {
        // positive floats order as their bits do
        const uint32_t t = c <= p.clusters ? __float_as_uint(plan_ns(p, c, (float)chunks)) : 0xffffffffu;
        const uint32_t m = __reduce_min_sync(0xffffffffu, t);
        const uint32_t at = __reduce_min_sync(0xffffffffu, t == m ? (uint32_t)c : 0xffffffffu);
        if ((threadIdx.x & 31) == 0) {
            best[warp][0] = m;
            best[warp][1] = at;
        }
    }
    __syncthreads();
    uint32_t m = best[0][0], at = best[0][1];
    for (int w = 1; w * 32 < p.clusters; ++w) {
        if (best[w][0] < m) {
            m = best[w][0];
            at = best[w][1];
        }
    }
    return (int32_t)at;
}

// What the merge has to know of the deal, in the workspace.
struct DecodeDeal {
    int64_t suffix_per;                            // chunks of a warp
    int32_t prefix_per, pad;                       // (head unit, key tile)s of a group
};

// The keys of sequence b's suffix; a length out of range raises the flag and
// is cut to the range.
__device__ __forceinline__ int32_t suffix_keys(const int32_t *lens, int32_t b, int64_t most, int32_t *flag)
{
    const int32_t n = __ldg(lens + b);
    if (n < 0 || n > most) {
        atomicOr(flag, kFlagIndex);
        return n < 0 ? 0 : (int32_t)most;
    }
    return n;
}

// Table row of sequence b's query: pos_q, or the index of its last key (which
// is the new token's); -1: not rotated.
__device__ __forceinline__ int64_t query_row(const int32_t *pos_q, int32_t b, int64_t keys,
                                             int64_t table_rows, int32_t *flag)
{
    const int64_t r = pos_q != nullptr ? (int64_t)__ldg(pos_q + b) : keys - 1;
    if (r == -1)
        return -1;
    if (r < 0 || r >= table_rows) {
        atomicOr(flag, kFlagPosition);
        return -1;
    }
    return r;
}

// ---------------------------------------------------------------------------
// 2. the suffixes
//
// A pair is (sequence, key head, row group): up to 16 query heads of one group,
// the 16 rows of an mma.  The chunks of all pairs, sequence after sequence, form
// one long list; warp w of the grid owns chunks [w * per, (w +
// 1) * per) of it, whatever pairs they belong to, and leaves an fp32 (O, m, l)
// for each pair it touches in slot w + pair (either index grows by one from
// one slot to the next, so slots are distinct).  Nothing waits on anything
// between warps.
//
// mma.sync (m16n8k16) instead of tcgen05: a decode step has at most 16 rows per
// key here, the work is one pass over the keys, and a warp that owns its keys,
// its stages and its softmax needs no barrier but the copies' own.  K and V
// arrive by TMA (boxes of 64 features x the chunk's keys, or a page's where that
// is less, 128-byte swizzle, so ldmatrix reads without conflicts), two stages a
// warp, eight warps an SM: 128 KB in flight or in use.  Three stages were slower:
// 256 sequences of 2080 keys on average without a prefix (2.2 GB) 352 us, with two
// 326 (now 328, 6.6 TB/s); so were six or seven warps of three stages (342, 344).
constexpr int kDecThreads = 32 * kDecWarps;
template <int D>
static constexpr int kDecStages = 2;
template <int D>
static constexpr int kDecStageBytes = 2 * kDecKeys<D> * D * 2;
template <int D>
static constexpr int kDecQStride = D * 2 + 16;                 // padded rows of the query tile
template <int D>
static constexpr int kDecSmem = kDecWarps * (kDecStages<D> * kDecStageBytes<D> + 16 * kDecQStride<D>);

struct DecodeArgs {
    AttnArgs a;                                // cos, sin, table_rows, rotary_dim, scale, flag
    CUtensorMap k_map, v_map;                  // boxes of 64 features x a chunk's keys, or a page's
    const void *q;                             // [B][Hq][D], row stride q_stride
    int64_t q_stride;
    void *o;                                   // [B][Hq][D]
    const int32_t *table, *prefix_table, *lens, *pos_q;
    int64_t max_blocks, n_pages;
    int32_t B, Hq, Hk, page_shift, n_prefix;
    int32_t chunk_shift;                       // log2 of a chunk's keys
    int32_t fold;                              // 1: the prefix is sequence B of the suffix kernel
    int32_t row_groups, rows;                  // of a key head's query heads; rows of a group
    int32_t slot_rows;                         // rows kept per slot (with fold also B * group)
    int32_t lg;                                // log2 of the heads of a prefix tile's token
    // partial results
    DecodeDeal *deal;
    int32_t *chunk_start;                      // [B + fold + 1]: chunks per pair of the sequences before b
    float *out;                                // [slots][slot_rows][D]
    float2 *stats;                             // [slots][slot_rows]
    const float *prefix_out;                   // PrefixSource::out
    const float2 *prefix_stats;
    int32_t prefix_tiles;                      // key tiles of the prefix kernel (0: it does not run)
    int32_t suffix;                            // 1: the suffix kernel runs
};

// Chunks of a warp: an equal share, and no less than two, so that few warps'
// results meet in the merge.
constexpr int kDecMinChunks = 2;
// a / b of non-negative numbers, in 32 bits when they fit (a quarter of the time)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return (uint32_t)a / (uint32_t)b;
    return a / b;
}
__device__ __forceinline__ int64_t decode_per_warp(int64_t chunks, int32_t warps)
{
    const int64_t per = divide(chunks + warps - 1, warps);
    return per < kDecMinChunks ? kDecMinChunks : per;
}

// Keys, and chunks, of sequence b, the folded prefix (b = B) included.
__device__ __forceinline__ int32_t decode_keys(const DecodeArgs &g, int32_t b, int64_t most)
{
    return b < g.B ? suffix_keys(g.lens, b, most, g.a.flag) : g.n_prefix;
}
__device__ __forceinline__ int32_t decode_chunks(const DecodeArgs &g, int32_t b, int64_t most)
{
    const int32_t n = decode_keys(g, b, most);
    return (n >> g.chunk_shift) + ((n & ((1 << g.chunk_shift) - 1)) != 0);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                     "{%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                     "{%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A place in the list of chunks.
struct ChunkAt {
    int32_t b, hr, ch, n;                      // sequence, key head and row group, chunk of n
    __device__ __forceinline__ void next(const DecodeArgs &g, int64_t most)
    {
        if (++ch < n)
            return;
        ch = 0;
        if (++hr < g.Hk * g.row_groups)
            return;
        hr = 0;
        do {
            if (++b >= g.B + g.fold) {
                n = 0;
                return;
            }
            n = decode_chunks(g, b, most);
        } while (n == 0);
    }
};

// 16 rows of rotated queries of pair (b, hr) into the warp's tile (zeros past
// the pair's rows), then as the A operand of every 16-feature step.  The rows
// are heads of one sequence, or, for the folded prefix, of the whole batch.
template <typename T, int LAYOUT, int D>
__device__ __forceinline__ void load_query_rows(const DecodeArgs &g, const ChunkAt &at, int64_t most,
                                                uint8_t *tile, uint32_t (&qf)[D / 16][4])
{
    constexpr int L = D / 16, kAtOnce = 32 / L, kSteps = 16 / kAtOnce;
    const int lane = threadIdx.x & 31, j = lane % L;
    const int32_t kv = at.hr / g.row_groups, group = g.Hq / g.Hk;
    const int32_t r0 = (at.hr - kv * g.row_groups) * g.rows;
    const RowPart part = row_part<LAYOUT>(j, g.a.rotary_dim);
    uint4 x0[kSteps], x1[kSteps];
    int64_t trow[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        int32_t r = i * kAtOnce + lane / L, b = at.b;
        bool live = r < g.rows && r0 + r < group;
        if (b == g.B) {                        // the folded prefix
            b = r / group;
            r -= b * group;
            live = b < g.B;
        }
        x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
        trow[i] = -1;
        if (live) {
            const T *row = static_cast<const T *>(g.q) + b * g.q_stride + (int64_t)(kv * group + r0 + r) * D;
            x0[i] = __ldg(reinterpret_cast<const uint4 *>(row + part.o0));
            x1[i] = __ldg(reinterpret_cast<const uint4 *>(row + part.o1));
            if (part.rot)
                trow[i] = query_row(g.pos_q, b,
                                    g.pos_q != nullptr ? 0
                                                       : (int64_t)g.n_prefix +
                                                             suffix_keys(g.lens, b, most, g.a.flag),
                                    g.a.table_rows, g.a.flag);
        }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (trow[i] < 0)
            continue;
        float c[8], s[8];
        table_values(g.a.cos, g.a.sin, trow[i] * (g.a.rotary_dim / 2) + 8 * j, c, s);
        rotate_part<T, LAYOUT>(x0[i], x1[i], c, s);
    }
    __syncwarp();                              // the tile's last readers are done
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int r = i * kAtOnce + lane / L;
        *reinterpret_cast<uint4 *>(tile + r * kDecQStride<D> + part.o0 * 2) = x0[i];
        *reinterpret_cast<uint4 *>(tile + r * kDecQStride<D> + part.o1 * 2) = x1[i];
    }
    __syncwarp();
    // lanes 0-15: rows 0-15, features 0-7 of the step; lanes 16-31: features 8-15
    const uint32_t addr = attn_smem_u32(tile) + (lane & 15) * kDecQStride<D> + (lane >> 4) * 16;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
        ldsm4(addr + k * 32, qf[k]);
}

// Chunks of the sequences before b, for all b (start: B + fold + 1 entries of
// shared memory), by all NT threads of a CTA; returns the number of all.
template <int NT>
__device__ __forceinline__ int32_t scan_chunks(const DecodeArgs &g, int32_t *start, int32_t *warp_sum)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t n_seqs = g.B + g.fold;
    const int64_t most = g.max_blocks << g.page_shift;
    int32_t carry = 0;
    for (int32_t b0 = 0; b0 < n_seqs; b0 += NT) {
        const int32_t b = b0 + tid;
        const int32_t n = b < n_seqs ? decode_chunks(g, b, most) : 0;
        int32_t inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d)
                inc += o;
        }
        if (lane == 31)
            warp_sum[warp] = inc;
        __syncthreads();
        int32_t before = carry;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            before += w < warp ? warp_sum[w] : 0;
            carry += warp_sum[w];
        }
        if (b < n_seqs)
            start[b] = before + inc - n;
        __syncthreads();
    }
    if (tid == 0)
        start[n_seqs] = carry;
    __syncthreads();
    return carry;
}

// A warp's run of chunks.
struct SuffixRun {
    ChunkAt at;
    int32_t w;                                 // the warp among all
    int64_t left;                              // chunks
};

// Barriers of the suffix warps of a CTA.
template <int D>
struct SuffixShared {
    uint64_t bar[kDecWarps][kDecStages<D>];
    int abort_flag;
};

// What the merge has to know of the suffixes' deal.  One CTA writes it, whether or
// not its waits expired: the merge runs in either case, and finds the parts'
// places by it.
__device__ __forceinline__ void publish_suffixes(const DecodeArgs &g, const int32_t *start, int64_t per)
{
    for (int32_t b = threadIdx.x; b <= g.B + g.fold; b += blockDim.x)
        g.chunk_start[b] = start[b];
    if (threadIdx.x == 0)
        g.deal->suffix_per = per;
}

// The suffixes' share of CTA `cta` of `ctas`, whose first eight warps work:
// every thread of the CTA calls this, then the working ones decode_suffixes.
template <int D>
__device__ __forceinline__ SuffixRun suffix_run(const DecodeArgs &g, const int32_t *start, int32_t carry,
                                                int32_t cta, int32_t ctas, SuffixShared<D> &sh)
{
    constexpr int kStages = kDecStages<D>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t n_seqs = g.B + g.fold;
    if (tid < kDecWarps * kStages)
        mbar_init(&sh.bar[0][0] + tid, 1);
    if (tid == 0)
        sh.abort_flag = 0;
    if (lane == 0 && warp < 2)                 // the maps, before the first copies need them
        asm volatile("prefetch.tensormap [%0];" ::"l"(warp ? &g.v_map : &g.k_map) : "memory");
    const int32_t heads = g.Hk * g.row_groups;
    const int64_t total = (int64_t)carry * heads;
    const int64_t per = decode_per_warp(total, ctas * kDecWarps);
    if (cta == 0)
        publish_suffixes(g, start, per);
    SuffixRun run;
    // (consecutive runs on different SMs: with few of them every SM copies; on few
    // SMs 4 sequences after 500 keys took 13.6 us, so 12.5)
    run.w = warp * ctas + cta;
    run.at = {0, 0, 0, 0};
    const int64_t c = run.w * per;
    run.left = warp >= kDecWarps ? 0 : total - c < per ? total - c : per;
    if (run.left > 0) {
        const int32_t b = find_sequence(start, n_seqs + 1, divide(c, heads));
        // (the last b whose start is at most c / heads has chunks)
        run.at.b = b;
        run.at.n = start[b + 1] - start[b];
        const int64_t in = c - (int64_t)start[b] * heads;
        run.at.hr = (int32_t)divide(in, run.at.n);
        run.at.ch = (int32_t)(in - (int64_t)run.at.hr * run.at.n);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();                           // start[] is read: its memory may become stages
    return run;
}

// One warp's run; smem: kDecSmem bytes of the CTA.
template <typename T, int LAYOUT, int D>
__device__ __forceinline__ void decode_suffixes(const DecodeArgs &g, uint8_t *smem, const SuffixRun &run,
                                                SuffixShared<D> &sh)
{
    constexpr int kStages = kDecStages<D>, kStage = kDecStageBytes<D>, kKeys = kDecKeys<D>;
    constexpr int kBox = kKeys * 128, kGroups = kKeys / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t most = g.max_blocks << g.page_shift;
    const int32_t heads = g.Hk * g.row_groups, w = run.w;
    int64_t left = run.left;
    ChunkAt at = run.at;
    if (left <= 0)
        return;
    uint64_t *bar = sh.bar[warp];
    uint8_t *stages = smem + warp * kStages * kStage;
    uint8_t *qtile = smem + kDecWarps * kStages * kStage + warp * 16 * kDecQStride<D>;
    volatile int *abort = &sh.abort_flag;
    // The copies run kStages chunks ahead.  Lane i holds the page of block base +
    // i of sequence `of`, so that a step seldom waits for the block list.
    ChunkAt ahead = at;
    int64_t to_load = left;
    int32_t pages = 0, of = -1;
    int64_t base_block = 0;
    // (several row groups of a key head read the same keys)
    const uint64_t policy = g.row_groups > 1 ? l2_keep() : l2_once();
    const int32_t box_shift = g.page_shift < g.chunk_shift ? g.page_shift : g.chunk_shift;
    const int32_t boxes = kKeys >> box_shift;                  // of a chunk's keys: its pages, or one
    auto load = [&](int st) {
        const int64_t key = (int64_t)ahead.ch * kKeys, block = key >> g.page_shift;
        if (of != ahead.b || block < base_block || block + boxes > base_block + 32) {
            of = ahead.b;
            base_block = block;
            const int64_t blocks = (((int64_t)ahead.n * kKeys - 1) >> g.page_shift) + 1;
            const int64_t listed = of < g.B ? g.max_blocks : ((int64_t)g.n_prefix - 1 >> g.page_shift) + 1;
            const int32_t *list = of < g.B ? g.table + of * g.max_blocks : g.prefix_table;
            // (a chunk's last page may lie behind the list: its keys are not visible)
            pages = block + lane < (blocks < listed ? blocks : listed) ? __ldg(list + block + lane) : -1;
        }
        if (lane == 0)
            mbar_expect_tx(&bar[st], kStage);
        // a lane's box: keys or values, 64 features, a page's keys
        const int x = lane % (D / 64), v = lane / (D / 64) & 1, i = lane / (2 * (D / 64));
        const int32_t page = __shfl_sync(0xffffffffu, pages, (int)(block - base_block) + (i < boxes ? i : 0));
        if (i < boxes) {
            int32_t z = page * g.Hk + ahead.hr / g.row_groups;
            if (page < 0 || page >= g.n_pages) {
                // (a page without visible keys may have any number)
                if (key + ((int64_t)i << box_shift) < decode_keys(g, ahead.b, most))
                    atomicOr(g.a.flag, kFlagIndex);
                z = (int32_t)(g.n_pages * g.Hk);               // arrives as zeros
            }
            const int32_t y = (int32_t)(key + ((int64_t)i << box_shift)) & ((1 << g.page_shift) - 1);
            tma_load_3d_l2(stages + st * kStage + v * (kStage / 2) + x * kBox + (i << box_shift) * 128,
                           v ? &g.v_map : &g.k_map, x * 64, y, z, &bar[st], policy);
        }
        --to_load;
        ahead.next(g, most);
    };
    bool ok = true;
    int64_t issued = 0, done = 0;
    for (int st = 0; st < kStages && to_load > 0; ++st, ++issued)
        load(st);

    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;   // rows lane / 4 and + 8
    int32_t keys = 0;                                          // of the pair's suffix
    bool fresh = true;
    int st = 0;
    uint32_t ph = 0;
    // ldmatrix rows: K (two 8-key tiles x two 8-feature halves of a step), V (two
    // 8-key halves x two 8-feature tiles)
    const int k_row = (lane & 7) + ((lane >> 4) << 3), k_half = (lane >> 3) & 1;
    const int v_row = lane & 15, v_half = lane >> 4;
    const uint32_t base = attn_smem_u32(stages);
    for (; ok && left > 0; --left, ++done) {
        if (fresh) {
            keys = decode_keys(g, at.b, most);
            load_query_rows<T, LAYOUT, D>(g, at, most, qtile, qf);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.0f;
            fresh = false;
        }
        ok = __all_sync(0xffffffffu, attn_wait(&bar[st], ph, abort));
        if (!ok)
            break;
        const uint32_t kb = base + st * kStage, vb = kb + kStage / 2;
        // S = q K^T: 16 rows x the chunk's keys.  Lane: rows lane / 4 (sc) and + 8
        // (sd), keys 2 (lane mod 4) + {0, 1} of each 8-key tile.
        float sc[4 * kGroups], sd[4 * kGroups];
#pragma unroll
        for (int k16 = 0; k16 < kGroups; ++k16) {
            float s0[4] = {0, 0, 0, 0}, s1[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                const int chunk = (k & 3) * 2 + k_half;
                ldsm4(kb + (k >> 2) * kBox + (k16 * 16 + k_row) * 128 + ((chunk ^ (k_row & 7)) << 4), b);
                mma16816<T>(s0, qf[k], b[0], b[1]);
                mma16816<T>(s1, qf[k], b[2], b[3]);
            }
            float *c = sc + 4 * k16, *d = sd + 4 * k16;
            c[0] = s0[0]; c[1] = s0[1]; c[2] = s1[0]; c[3] = s1[1];
            d[0] = s0[2]; d[1] = s0[3]; d[2] = s1[2]; d[3] = s1[3];
        }
        const int32_t nk = keys - at.ch * kKeys;               // visible keys of the chunk
        const int c0 = 2 * (lane & 3);
        uint32_t vis[2 * kGroups];                             // value rows: halves of a register
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i)
            vis[i] = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < 4 * kGroups; ++i) {
            sc[i] *= g.a.scale_log2;
            sd[i] *= g.a.scale_log2;
        }
        if (nk < kKeys) {
#pragma unroll
            for (int i = 0; i < 4 * kGroups; ++i) {
                const int key = c0 + (i & 1) + (i >> 1) * 8;
                if (key >= nk) {
                    sc[i] = sd[i] = -INFINITY;
                    // what lies behind the last key (anything) must not meet a zero
                    vis[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
                }
            }
        }
        float x0 = sc[0], x1 = sd[0];
#pragma unroll
        for (int i = 1; i < 4 * kGroups; ++i) {
            x0 = fmaxf(x0, sc[i]);
            x1 = fmaxf(x1, sd[i]);
        }
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        // the reference maxima move only when exceeded by more than 8 (a factor
        // of 256), so O is seldom rescaled
        const bool up0 = x0 > m0 + 8.0f, up1 = x1 > m1 + 8.0f;
        if (__any_sync(0xffffffffu, up0 || up1)) {
            const float f0 = up0 ? (m0 == -INFINITY ? 0.0f : fast_exp2(m0 - x0)) : 1.0f;
            const float f1 = up1 ? (m1 == -INFINITY ? 0.0f : fast_exp2(m1 - x1)) : 1.0f;
            m0 = up0 ? x0 : m0;
            m1 = up1 ? x1 : m1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][0] *= f0;
                o[i][1] *= f0;
                o[i][2] *= f1;
                o[i][3] *= f1;
            }
        }
        const float n0 = m0 == -INFINITY ? 0.0f : m0, n1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
        for (int i = 0; i < 4 * kGroups; ++i) {
            sc[i] = fast_exp2(sc[i] - n0);
            sd[i] = fast_exp2(sd[i] - n1);
        }
#pragma unroll
        for (int k16 = 0; k16 < kGroups; ++k16) {
            const float *c = sc + 4 * k16, *d = sd + 4 * k16;
            l0 += (c[0] + c[1]) + (c[2] + c[3]);
            l1 += (d[0] + d[1]) + (d[2] + d[3]);
            // P rounded to the element type for the P V product (the sums keep fp32)
            const uint32_t p[4] = {Elt<T>::f2_to_word(c[0], c[1]), Elt<T>::f2_to_word(d[0], d[1]),
                                   Elt<T>::f2_to_word(c[2], c[3]), Elt<T>::f2_to_word(d[2], d[3])};
            const uint32_t vis0 = vis[2 * k16], vis1 = vis[2 * k16 + 1];
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                const int chunk = (n & 3) * 2 + v_half;
                ldsm4_t(vb + (n >> 2) * kBox + (k16 * 16 + v_row) * 128 + ((chunk ^ (v_row & 7)) << 4), b);
                mma16816<T>(o[2 * n], p, b[0] & vis0, b[1] & vis1);
                mma16816<T>(o[2 * n + 1], p, b[2] & vis0, b[3] & vis1);
            }
        }
        __syncwarp();                                          // the stage is read
        if (to_load > 0) {
            load(st);
            ++issued;
        }
        if (++st == kStages) {
            st = 0;
            ph ^= 1u;
        }
        const int32_t pair = at.b * heads + at.hr;
        const int64_t slot = (int64_t)w + pair;
        const ChunkAt was = at;
        at.next(g, most);
        if (left == 1 || at.b != was.b || at.hr != was.hr) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const int r = lane >> 2;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int rr = r + 8 * half;
                if (rr < g.slot_rows) {
                    float *dst = g.out + (slot * g.slot_rows + rr) * D + c0;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<float2 *>(dst + 8 * i) =
                            make_float2(o[i][2 * half], o[i][2 * half + 1]);
                    if ((lane & 3) == 0)
                        g.stats[slot * g.slot_rows + rr] = half ? make_float2(m1, l1) : make_float2(m0, l0);
                }
            }
            fresh = true;
        }
    }
    if (!ok) {
        *abort = 1;
        if (lane == 0)
            atomicOr(g.a.flag, kFlagTimeout);
        // one more bounded wait for the copies in flight
        for (int64_t i = done; i < issued; ++i)
            (void)attn_wait(&bar[i % kStages], (uint32_t)(i / kStages) & 1u);
    }
}

// The suffixes (and a folded prefix) alone.
template <typename T, int LAYOUT, int D>
__global__ void __launch_bounds__(kDecThreads, 1) rope_decode_suffix_kernel(const __grid_constant__ DecodeArgs g)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int32_t warp_sum[kDecWarps];
    __shared__ SuffixShared<D> sh;
    int32_t *start = reinterpret_cast<int32_t *>(smem);
    pdl_wait();
    pdl_trigger();
    const int32_t carry = scan_chunks<kDecThreads>(g, start, warp_sum);
    const SuffixRun run = suffix_run<D>(g, start, carry, blockIdx.x, gridDim.x, sh);
    decode_suffixes<T, LAYOUT, D>(g, smem, run, sh);
}

// ---------------------------------------------------------------------------
// 1. the prefix, with the suffixes beside or behind it
struct PrefixSource {
    static constexpr bool kPrefix = true;
    template <int D>
    static constexpr int smem_bytes()
    {
        const int prefix = (int)kPackedSmem<D> + 4 * (kMaxDecodeBatch + 2);
        return prefix > kDecSmem<D> ? prefix : kDecSmem<D>;
    }
    AttnArgs a;                                // cos, sin, table_rows, rotary_dim, scale, flag
    CUtensorMap k_map, v_map, v_tail, q_map;   // v_tail: pages of n_keys mod page rows
    DecodeArgs g;                              // the suffixes
    PlanSizes sizes;
    const int32_t *pages;                      // the prefix's block list
    float *out;                                // [parts][B][GP][D]: part group + head unit
    float2 *stats;                             // [parts][B][GP] (m, l)
    int64_t n_pages;
    int32_t n_keys, B, Hk, page_shift, units_per_kv;

    // Virtual cluster v: row tile v mod row_tiles of group v / row_tiles, whose
    // range of (head unit, key tile) is cut at the heads; a cluster takes v = cid,
    // cid + clusters, ...  The clusters of a group read the same keys at about the
    // same time.
    struct Cursor {
        int32_t v, at, end;
    };
    struct Walk {
        int32_t cid, clusters, groups, per;
        int32_t chunks;                        // of the suffixes
    };
    // Behind the prefix's shared memory: the scan of the suffixes' chunks.
    template <int D>
    static __device__ __forceinline__ int32_t *chunk_starts(uint8_t *smem)
    {
        return reinterpret_cast<int32_t *>(smem + kPackedSmem<D>);
    }
    template <int D>
    __device__ __forceinline__ Walk walk(int64_t cid, int64_t, uint8_t *smem) const
    {
        __shared__ uint32_t best[kPackedThreads / 32][2];
        __shared__ int32_t warp_sum[kPackedThreads / 32];
        const int32_t chunks = scan_chunks<kPackedThreads>(g, chunk_starts<D>(smem), warp_sum);
        const PrefixDeal d = prefix_deal(sizes, plan_clusters(sizes, chunks, best));
        if (blockIdx.x == 0 && threadIdx.x == 0)
            g.deal->prefix_per = d.per;
        return {(int32_t)cid, d.clusters, d.groups, d.per, chunks};
    }
    // The suffixes, on the CTAs without prefix work, or on all behind it: two
    // warpgroups, with 216 registers a thread (after the roles' 240 / 112 / 104).
    template <typename T, int LAYOUT, int D>
    __device__ __forceinline__ void finish(const Walk &w, uint8_t *smem, bool failed) const
    {
        __shared__ SuffixShared<D> sh;
        const int32_t used = 2 * w.clusters < (int32_t)gridDim.x ? 2 * w.clusters : 0;
        const int32_t cta = (int32_t)blockIdx.x - used;
        if (!g.suffix || cta < 0)
            return;
        if (failed) {                          // copies may still be on their way: no work,
            // but what the merge needs; the scan lies behind the roles' memory
            if (cta == 0)
                publish_suffixes(g, chunk_starts<D>(smem),
                                 decode_per_warp((int64_t)w.chunks * g.Hk * g.row_groups,
                                                 ((int32_t)gridDim.x - used) * kDecWarps));
            return;
        }
        const SuffixRun run =
            suffix_run<D>(g, chunk_starts<D>(smem), w.chunks, cta, (int32_t)gridDim.x - used, sh);
        const int warp = threadIdx.x >> 5;
        if (warp < 8) {
            if (warp < 4)
                asm volatile("setmaxnreg.dec.sync.aligned.u32 216;");
            else
                asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            decode_suffixes<T, LAYOUT, D>(g, smem, run, sh);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        }
    }
    __device__ __forceinline__ Cursor start(const Walk &w, int32_t v) const
    {
        const int32_t all = sizes.head_units * sizes.tiles;
        Cursor c;
        c.v = v;
        c.at = v / sizes.row_tiles * w.per;
        c.end = all - c.at < w.per ? all : c.at + w.per;
        return c;
    }
    __device__ __forceinline__ Cursor first(const Walk &w) const
    {
        // (a cluster past the plan's starts behind the last virtual one)
        return start(w, w.cid < w.clusters ? w.cid : w.groups * sizes.row_tiles);
    }
    __device__ __forceinline__ bool valid(const Walk &w, const Cursor &c) const
    {
        return c.v < w.groups * sizes.row_tiles && c.at < c.end;
    }
    __device__ __forceinline__ int32_t tiles(const Walk &, const Cursor &c) const
    {
        const int32_t head_end = sizes.tiles - c.at % sizes.tiles;
        return c.end - c.at < head_end ? c.end - c.at : head_end;
    }
    __device__ __forceinline__ void next(const Walk &w, Cursor &c) const
    {
        c.at += tiles(w, c);
        if (c.at >= c.end)
            c = start(w, c.v + w.clusters);
    }
    __device__ __forceinline__ PackedUnit unit(const Walk &w, const Cursor &c, int lg) const
    {
        const int32_t hu = c.at / sizes.tiles, group = c.v / sizes.row_tiles;
        PackedUnit u;
        u.tok0 = (c.v - group * sizes.row_tiles) * (2 * kAttnRows >> lg);
        u.seq = 0; u.q_start = 0; u.k_start = 0; u.tokens = B; u.n_keys = n_keys;
        u.head0 = hu << lg;
        u.kv = hu / units_per_kv;
        u.first = c.at - hu * sizes.tiles;
        u.n_tiles = tiles(w, c);
        u.part = group + hu;
        return u;
    }
    __device__ __forceinline__ int64_t table_row(const PackedUnit &, int32_t t) const
    {
        return query_row(g.pos_q, t,
                         g.pos_q != nullptr
                             ? 0
                             : (int64_t)n_keys + suffix_keys(g.lens, t, g.max_blocks << page_shift, a.flag),
                         a.table_rows, a.flag);
    }

    // z of a prefix page in the pools' maps; past the last page, and for a bad
    // page number, an index that arrives as zeros
    __device__ __forceinline__ int32_t page_z(int32_t i, int32_t kv) const
    {
        const int32_t none = (int32_t)(n_pages * Hk);
        if ((int64_t)i << page_shift >= n_keys)
            return none;
        const int32_t p = __ldg(pages + i);
        if (p < 0 || p >= n_pages) {
            atomicOr(a.flag, kFlagIndex);
            return none;
        }
        return p * Hk + kv;
    }
    // (with several row tiles the prefix is read by as many clusters at about the
    // same time.  The head units of one key head read it one after the other, long
    // after one another: kept for them, 32 sequences of 24 heads over 8 after 128k
    // keys took 289 us, so 286, and of 48 over 2 102, so 91)
    __device__ __forceinline__ uint64_t policy() const { return sizes.row_tiles > 1 ? l2_keep() : l2_once(); }
    // Where this lane's boxes of a tile lie, looked up before the stage is waited
    // for: keys (box i of a half, features 64 x ..) and values (page i).
    template <int D>
    __device__ __forceinline__ int32_t key_place(const PackedUnit &u, int32_t kt, uint32_t rank, int lane) const
    {
        const int32_t shift = page_shift < 6 ? page_shift : 6;      // keys of a box: a page or half of one
        const int32_t key = (u.first + kt) * kAttnKeys + 64 * (int)rank + (lane / (D / 64) << shift);
        return lane < (64 >> shift) * (D / 64) ? page_z(key >> page_shift, u.kv) : 0;
    }
    template <int D>
    __device__ __forceinline__ int32_t value_place(const PackedUnit &u, int32_t kt, int lane) const
    {
        return lane < kAttnKeys >> page_shift
                   ? page_z(((u.first + kt) * kAttnKeys >> page_shift) + lane, u.kv)
                   : 0;
    }
    template <int D>
    __device__ __forceinline__ void load_keys(const PackedUnit &, int32_t, int32_t z, uint8_t *dst,
                                              uint64_t *bar, uint32_t rank, int lane) const
    {
        const int32_t shift = page_shift < 6 ? page_shift : 6;
        if (lane < (64 >> shift) * (D / 64)) {
            const int32_t i = lane / (D / 64), x = lane % (D / 64);
            load_half_box_l2(dst + x * 8192 + (i << shift) * 128, &k_map, x * 64,
                             (64 * (int)rank + (i << shift)) & ((1 << page_shift) - 1), z, bar, rank,
                             policy());
        }
    }
    template <int D>
    __device__ __forceinline__ void load_values(const PackedUnit &u, int32_t kt, int32_t z, uint8_t *dst,
                                                uint64_t *bar, uint32_t rank, int lane) const
    {
        if (lane < kAttnKeys >> page_shift) {
            const int32_t page = ((u.first + kt) * kAttnKeys >> page_shift) + lane;
            // the last, partly filled page: rows past the prefix arrive as zeros
            const bool tail = page == n_keys >> page_shift;
            load_half_box_l2(dst + (lane << page_shift) * D, tail ? &v_tail : &v_map, D / 2 * (int)rank, 0,
                             z, bar, rank, policy());
        }
    }
    // One helper warp: its rows' O, m and l, in fp32
    template <int D>
    __device__ __forceinline__ void store_rows(const PackedUnit &u, uint32_t o_base, int32_t y0, int lane,
                                               int lg, float2 stat) const
    {
        const int32_t tok = y0 + (lane >> lg);
        const int64_t row = (((int64_t)u.part * B + tok) << lg) + (lane & ((1 << lg) - 1));
        if (tok < B)
            stats[row] = stat;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
            float ov[32];
            tmem_ld32(o_base + c0, ov);
            if (tok < B) {
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                    *reinterpret_cast<float4 *>(out + row * D + c0 + c) =
                        make_float4(ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// 3. the merge: W warps per (sequence, query head), a lane per D / 32 features
//
// Bound by latency: a few dependent reads, then a row's parts, which are many when
// few sequences hold many keys (one sequence, 8 key heads: 125).  With few rows W
// warps share a row's parts and join theirs in shared memory.  Whole calls with W = 1 / 4 / 8
// (us; heads of 128, 32 over 8): 1 sequence, 8k prefix 39.2 / 22.3 / 19.5; 4, 500
// 14.4 / 12.6 / 12.3; 16, 2k 29.7 / 27.5 / 27.5; 32, 1k 35.5 / 34.0 / 36.8; 64,
// 8k 53.5 / 54.9 / 59.4.  So the most warps that 4096 allow, of 8, 4 and 1.  Four
// parts at a time, the first of them beside their statistics; with eight the
// registers keep CTAs out: 8 % less for the first of these, 4 to 9 % more for the
// next three.
constexpr int64_t kMergeWarps = 4096;
template <typename T, int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) rope_decode_merge_kernel(const __grid_constant__ DecodeArgs g)
{
    constexpr int V = D / 32, kAtOnce = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = W == 1 ? 0 : warp;
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (row >= (int64_t)g.B * g.Hq)
        return;
    const int32_t b = (int32_t)(row / g.Hq), h = (int32_t)(row - (int64_t)b * g.Hq);
    const int32_t group = g.Hq / g.Hk, kv = h / group, in_group = h - kv * group;
    const int32_t rg = in_group / g.rows, r = in_group - rg * g.rows;
    const int32_t heads = g.Hk * g.row_groups;
    // the parts: groups of the prefix kernel, slots of the pair, slots of the
    // folded prefix
    int32_t n0 = 0, n1 = 0, n2 = 0;
    int64_t first0 = 0, first1 = 0, first2 = 0;
    const DecodeDeal deal = *g.deal;
    if (g.prefix_tiles > 0) {
        const int32_t hu = h >> g.lg;
        first0 = hu * g.prefix_tiles / deal.prefix_per + hu;
        n0 = (int32_t)(((hu + 1) * g.prefix_tiles - 1) / deal.prefix_per + hu - first0 + 1);
    }
    if (g.suffix) {
        auto slots = [&](int32_t seq, int32_t hr, int64_t &first, int32_t &n) {
            const int64_t c0 = g.chunk_start[seq], c1 = g.chunk_start[seq + 1];
            if (c1 == c0)
                return;
            const int64_t at = c0 * heads + hr * (c1 - c0), pair = (int64_t)seq * heads + hr;
            first = divide(at, deal.suffix_per) + pair;
            n = (int32_t)(divide(at + (c1 - c0) - 1, deal.suffix_per) + pair - first + 1);
        };
        slots(b, kv * g.row_groups + rg, first1, n1);
        if (g.fold)
            slots(g.B, kv, first2, n2);
    }
    // part p: its row among the statistics, and whose
    auto part = [&](int32_t p, bool &prefix) -> int64_t {
        prefix = p < n0;
        if (prefix)
            return (((first0 + p) * g.B + b) << g.lg) + (h & ((1 << g.lg) - 1));
        p -= n0;
        if (p < n1)
            return (first1 + p) * g.slot_rows + r;
        return (first2 + p - n1) * g.slot_rows + b * group + in_group;
    };
    // Batches of 32 of the warp's parts: lane i holds part i's maximum and sum, so
    // the loads of a batch do not wait for one another.
    const int32_t all = n0 + n1 + n2, n_parts = (all - share + W - 1) / W;   // parts share, share + W, ...
    float m = -INFINITY, l = 0.0f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        o[i] = 0.0f;
    for (int32_t p0 = 0; p0 < n_parts; p0 += 32) {
        const int n = n_parts - p0 < 32 ? n_parts - p0 : 32;
        float2 mine = make_float2(-INFINITY, 0.0f);
        const float *src = nullptr;
        if (lane < n) {
            bool prefix;
            const int64_t at = part((p0 + lane) * W + share, prefix);
            mine = __ldg((prefix ? g.prefix_stats : g.stats) + at);
            src = (prefix ? g.prefix_out : g.out) + at * D;
        }
        float v[kAtOnce][V];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const float *x = reinterpret_cast<const float *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i0 + j));
#pragma unroll
                for (int e = 0; e < V; ++e)
                    v[j][e] = 0.0f;
                if (i0 + j < n) {
                    if constexpr (V == 4) {
                        const float4 t = __ldg(reinterpret_cast<const float4 *>(x + lane * V));
                        v[j][0] = t.x; v[j][1] = t.y; v[j][2] = t.z; v[j][3] = t.w;
                    } else {
                        const float2 t = __ldg(reinterpret_cast<const float2 *>(x + lane * V));
                        v[j][0] = t.x; v[j][1] = t.y;
                    }
                }
            }
        };
        fetch(0);
        float top = mine.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m);
        const float ref = top == -INFINITY ? 0.0f : top;       // no key so far (or NaN)
        const float w = exp2f(mine.x - ref), f = exp2f(m - ref);
        float sum = w * mine.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * f + sum;
#pragma unroll
        for (int i = 0; i < V; ++i)
            o[i] *= f;
        m = top;
        for (int i0 = 0; i0 < n; i0 += kAtOnce) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const float wi = __shfl_sync(0xffffffffu, w, i0 + j);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] += wi != 0.0f ? wi * v[j][e] : 0.0f;   // (past the last part: 0)
            }
            if (i0 + kAtOnce < n)
                fetch(i0 + kAtOnce);
        }
    }
    if constexpr (W > 1) {
        __shared__ float2 stat[W];
        __shared__ __align__(16) float part_o[W][D];
        if (lane == 0)
            stat[warp] = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < V; ++i)
            part_o[warp][lane * V + i] = o[i];
        __syncthreads();
        if (warp != 0)
            return;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < W; ++i)
            top = fmaxf(top, stat[i].x);
        const float ref = top == -INFINITY ? 0.0f : top;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            o[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float w = exp2f(stat[i].x - ref);
            l += w * stat[i].y;
#pragma unroll
            for (int e = 0; e < V; ++e)
                o[e] += w != 0.0f ? w * part_o[i][lane * V + e] : 0.0f;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T *dst = static_cast<T *>(g.o) + row * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(Elt<T>::f2_to_word(o[0] * inv, o[1] * inv),
                                                     Elt<T>::f2_to_word(o[2] * inv, o[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(dst) = Elt<T>::f2_to_word(o[0] * inv, o[1] * inv);
}

// ---------------------------------------------------------------------------
// host side
template <typename T, int LAYOUT, int D>
static cudaError_t launch_decode(const DecodeCall &c, const DecodeLayout &lay, cudaStream_t st)
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
    AttnArgs a;
    memset(&a, 0, sizeof a);
    a.cos = c.cos; a.sin = c.sin; a.rotary_dim = c.rotary_dim; a.table_rows = c.table_rows;
    a.scale_log2 = c.scale_log2; a.flag = c.flag;

    const int32_t gp = packed_group_heads(c.Hq, c.Hk), lg = __builtin_ctz((unsigned)gp);
    const bool prefix_kernel = c.n_prefix > 0 && !lay.fold;
    const int32_t tiles = (c.n_prefix + kAttnKeys - 1) / kAttnKeys;
    int sms = 0, dev = 0;
    cudaError_t e = sm_count(&sms, &dev);
    if (e != cudaSuccess)
        return e;

    DecodeArgs g;
    memset(&g, 0, sizeof g);
    g.a = a;
    g.q = c.q; g.q_stride = c.q_stride; g.o = c.o;
    g.table = c.table; g.prefix_table = c.prefix_table; g.lens = c.lens; g.pos_q = c.pos_q;
    g.max_blocks = c.max_blocks; g.n_pages = c.n_pages;
    g.B = c.B; g.Hq = c.Hq; g.Hk = c.Hk; g.page_shift = c.page_shift; g.n_prefix = c.n_prefix;
    g.fold = lay.fold; g.row_groups = lay.row_groups; g.rows = lay.rows; g.slot_rows = lay.slot_rows;
    g.lg = lg;
    g.deal = reinterpret_cast<DecodeDeal *>(ws);
    g.chunk_start = reinterpret_cast<int32_t *>(ws + lay.chunk_start);
    g.out = reinterpret_cast<float *>(ws + lay.out);
    g.stats = reinterpret_cast<float2 *>(ws + lay.stats);
    g.prefix_out = reinterpret_cast<float *>(ws + lay.prefix_out);
    g.prefix_stats = reinterpret_cast<float2 *>(ws + lay.prefix_stats);
    g.prefix_tiles = prefix_kernel ? tiles : 0;
    g.suffix = lay.suffix_ctas > 0;
    g.chunk_shift = __builtin_ctz((unsigned)kDecKeys<D>);
    const uint32_t chunk_box = (uint32_t)(page < kDecKeys<D> ? page : kDecKeys<D>);
    if (g.suffix &&
        (!encode_3d(enc, &g.k_map, c.k_pages, dt, {D, page, z}, {D * 2, page * D * 2}, {64, chunk_box, 1}, sw) ||
         !encode_3d(enc, &g.v_map, c.v_pages, dt, {D, page, z}, {D * 2, page * D * 2}, {64, chunk_box, 1}, sw)))
        return cudaErrorInvalidValue;

    if (prefix_kernel) {
        const uint32_t box = (uint32_t)(page < 64 ? page : 64), tail = (uint32_t)(c.n_prefix % page);
        PrefixSource s;
        memset(&s, 0, sizeof s);
        s.a = a;
        s.g = g;
        if (!encode_3d(enc, &s.k_map, c.k_pages, dt, {D, page, z}, {D * 2, page * D * 2}, {64, box, 1}, sw) ||
            !encode_3d(enc, &s.v_map, c.v_pages, dt, {D, page, z}, {D * 2, page * D * 2},
                       {(uint32_t)D / 2, (uint32_t)page, 1}, D == 128 ? sw : CU_TENSOR_MAP_SWIZZLE_64B) ||
            !encode_3d(enc, &s.v_tail, c.v_pages, dt, {D, tail > 0 ? tail : page, z}, {D * 2, page * D * 2},
                       {(uint32_t)D / 2, (uint32_t)page, 1}, D == 128 ? sw : CU_TENSOR_MAP_SWIZZLE_64B) ||
            !encode_3d(enc, &s.q_map, c.q, dt, {D, c.Hq, c.B}, {D * 2, c.q_stride * 2},
                       {64, (uint32_t)gp, (uint32_t)(kAttnRows / gp)}, sw))
            return cudaErrorInvalidValue;
        // clusters for the prefix and for the suffixes, as far as the SMs go
        int32_t clusters = lay.clusters + (lay.suffix_ctas + 1) / 2;
        const int32_t pairs = (sms < kDecodeSms ? sms : kDecodeSms) / 2;
        clusters = clusters < pairs ? clusters : pairs;
        s.sizes.row_tiles = lay.row_tiles; s.sizes.head_units = c.Hq / gp; s.sizes.tiles = tiles;
        s.sizes.clusters = lay.clusters < clusters ? lay.clusters : clusters;
        s.sizes.sms = 2 * clusters;
        s.sizes.tile_ns = D == 128 ? 850 : 700;
        s.sizes.heads = c.Hk * lay.row_groups; s.sizes.chunk_bytes = kDecStageBytes<D>;
        s.sizes.sm_rate = D == 128 ? 53.0f : 48.0f;
        s.pages = c.prefix_table;
        s.out = reinterpret_cast<float *>(ws + lay.prefix_out);
        s.stats = reinterpret_cast<float2 *>(ws + lay.prefix_stats);
        s.n_pages = c.n_pages;
        s.n_keys = c.n_prefix;
        s.B = c.B; s.Hk = c.Hk; s.page_shift = c.page_shift;
        s.units_per_kv = c.Hq / c.Hk / gp;
        e = launch_packed_kernel<T, LAYOUT, D>(s, clusters, lg, st);
    } else if (g.suffix) {
        static std::atomic<uint64_t> raised{0};
        auto *kernel = rope_decode_suffix_kernel<T, LAYOUT, D>;
        e = raise_smem(reinterpret_cast<const void *>(kernel), kDecSmem<D>, dev, raised);
        if (e == cudaSuccess)
            e = launch_hot(kernel, dim3((unsigned)lay.suffix_ctas), dim3(kDecThreads), (size_t)kDecSmem<D>, st, g);
    }
    if (e != cudaSuccess)
        return e;
    const int64_t rows = (int64_t)c.B * c.Hq;
    if (rows * 8 <= kMergeWarps)
        return launch_hot(rope_decode_merge_kernel<T, D, 8>, dim3((unsigned)rows), dim3(256), 0, st, g);
    if (rows * 4 <= kMergeWarps)
        return launch_hot(rope_decode_merge_kernel<T, D, 4>, dim3((unsigned)rows), dim3(128), 0, st, g);
    return launch_hot(rope_decode_merge_kernel<T, D, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, g);
}

template <typename T>
cudaError_t launch_decode_type(const DecodeCall &c, const DecodeLayout &lay, int32_t D, int32_t layout,
                               cudaStream_t st)
{
    if (layout == 0)
        return D == 64 ? launch_decode<T, 0, 64>(c, lay, st) : launch_decode<T, 0, 128>(c, lay, st);
    return D == 64 ? launch_decode<T, 1, 64>(c, lay, st) : launch_decode<T, 1, 128>(c, lay, st);
}

}  // namespace rope