// rope_attention_packed.cuh -- attention forward over packed sequences of
// different lengths, with rotary Q/K (rope_attention_packed_fwd), on pairs of
// SMs (tcgen05 with cta_group::2, TMEM, TMA).
//
//   o_i = sum_j softmax_j(scale * rot(q_i) . rot(k_j)) v_j
//
// over the keys j of token i's own sequence, j <= i + Lk - Lq when causal.
// Two launches:
//   1. rope_packed_prepare_kernel rotates the keys into the workspace
//      ([Hk][total_k][D]), lists the query tiles of all sequences, longest
//      first, and writes four tensor maps per sequence (rotated K, V, Q, O);
//   2. rope_attn_packed_kernel walks the list, one cluster of two CTAs per
//      pair of SMs.
//
// Why maps per sequence: a map whose row count is the sequence's length makes
// the copy engine itself end every tile where the sequence ends.  Keys, values
// and queries past it arrive as zeros (so an infinity or NaN of the next
// sequence never meets a zero probability), and output rows past it are not
// written.  Nothing in the tile loop asks where a sequence ends, except the
// score mask.
//
// Rows of a tile: GP heads of one group and consecutive tokens, row = token *
// GP + head, GP the largest power of two (up to 16) that divides the group
// size Hq / Hk.  A cluster's 256 rows are then 256 / GP tokens, so a short
// sequence fills a tile with heads instead of padding, and the tile at the
// causal diagonal spans fewer tokens.  A Q or O box is 64 features x GP heads
// x tokens.
//
// The cluster's roles, barriers and phases are those of rope_attn_2sm_kernel
// (rope_attention.cuh): 224 threads a CTA, warps 0-3 the softmax of its 128
// rows, the leader's warps 4 and 5 the S = Q K^T and O += P V products of both
// CTAs, warp 6 the CTA's copies; three S buffers in TMEM, released by the
// products that read P from them.  What differs:
//   * the work list and the maps come from the workspace;
//   * warp 6 also fetches the cos/sin rows of the tile's tokens, one bulk copy
//     per row at any position (pos_q), into the same barrier as the query tile;
//   * D = 64 runs here too (V halves of 32 features, 64-byte swizzle).
#pragma once

#include "rope_attention.cuh"
#include "rope_rows.cuh"
#include "rope_serving.cuh"

namespace rope {

// One query tile of a sequence: tokens tok0 .. of sequence seq.
struct alignas(16) PackedEntry {
    int32_t seq, tok0, Lq, Lk;
    int32_t q_start, n_tiles, pad0, pad1;      // n_tiles: key tiles the tile's rows can see
};

constexpr int kPackedMaps = 4;                 // K, V, Q, O of a sequence
constexpr int kPackedPrepThreads = 128;
constexpr int kPackedBins = 2048;              // key-tile counts told apart when sorting

struct PackedPlan {
    const int32_t *cu_q, *cu_k;
    int32_t n_seqs;
    int64_t total_q, total_k;
    int32_t causal, tile_tokens;               // 256 / GP
    int32_t check_q_rows, check_k_rows;        // positions are indices: lengths must fit the table
    int64_t table_rows;
    int32_t *n_entries;                        // [1]
    PackedEntry *entries;
    CUtensorMap *maps;                         // [n_seqs][kPackedMaps]
    int64_t base[kPackedMaps];                 // address of token 0
    int64_t step[kPackedMaps];                 // bytes from token to token
    int32_t *flag;
    int32_t map_blocks;                        // grid: the planner, the maps, then the rotation
};

struct PackedKernelArgs {
    AttnArgs a;                                // cos, sin, table_rows, rotary_dim, scale, causal, flag
    const PackedEntry *entries;
    const int32_t *n_entries;
    const CUtensorMap *maps;
    const int32_t *pos_q;
    int32_t head_units;                        // Hq / GP
    int32_t units_per_kv;                      // (Hq / Hk) / GP
};

struct PackedMapTemplates {
    CUtensorMap m[kPackedMaps];
};

// ---------------------------------------------------------------------------
// 1. the plan

// Sequence b's offsets are in order and inside the tensors, and (when its
// positions are indices) its lengths fit the table.
__device__ __forceinline__ bool packed_sequence_ok(const PackedPlan &p, int32_t b, bool &fits)
{
    const int32_t q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    fits = (!p.check_q_rows || (int64_t)q1 - q0 <= p.table_rows) &&
           (!p.check_k_rows || (int64_t)k1 - k0 <= p.table_rows);
    return q0 >= 0 && q0 <= q1 && q1 <= p.total_q && k0 >= 0 && k0 <= k1 && k1 <= p.total_k;
}

// Key tiles that the rows of the tile at token t can see.
__device__ __forceinline__ int32_t packed_key_tiles(int32_t t, int32_t tokens, int32_t Lq, int32_t Lk,
                                                    int32_t causal)
{
    int64_t keys = Lk;
    if (causal) {
        const int64_t last = (int64_t)t + tokens - 1 < Lq - 1 ? (int64_t)t + tokens - 1 : Lq - 1;
        const int64_t seen = last + Lk - Lq + 1;
        keys = seen < 0 ? 0 : (seen < keys ? seen : keys);
    }
    return (int32_t)((keys + kAttnKeys - 1) / kAttnKeys);
}

// The list of query tiles, sorted by key tiles, most first (a counting sort;
// ties and counts past the last bin in any order, which changes nothing but
// the order of work).  One CTA.  When an offset is bad the list stays empty.
static __device__ void packed_list(const PackedPlan &p, int32_t *bins)
{
    __shared__ int32_t warp_sum[kPackedPrepThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = kPackedPrepThreads / 32;
    bool bad = false, small = false;
    for (int32_t b = tid; b < p.n_seqs; b += kPackedPrepThreads) {
        bool fits;
        bad = bad || !packed_sequence_ok(p, b, fits);
        small = small || !fits;
    }
    bad = __syncthreads_or(bad);
    small = __syncthreads_or(small);
    if (bad || small) {
        if (tid == 0) {
            atomicOr(p.flag, bad ? kFlagIndex : kFlagPosition);
            *p.n_entries = 0;
        }
        return;
    }
    for (int i = tid; i < kPackedBins; i += kPackedPrepThreads)
        bins[i] = 0;
    __syncthreads();
    // bin of a count: most key tiles in bin 0
    auto bin_of = [](int32_t n) { return kPackedBins - 1 - (n < kPackedBins - 1 ? n : kPackedBins - 1); };
    for (int pass = 0; pass < 2; ++pass) {
        // short sequences have few tiles: a warp takes 32 sequences at a time,
        // one per lane, then all lanes the tiles of each of them in turn
        for (int32_t b0 = warp * 32; b0 < p.n_seqs; b0 += kWarps * 32) {
            const int32_t mine = b0 + lane;
            int32_t q0 = 0, Lq = 0, Lk = 0;
            if (mine < p.n_seqs) {
                q0 = p.cu_q[mine];
                Lq = p.cu_q[mine + 1] - q0;
                Lk = p.cu_k[mine + 1] - p.cu_k[mine];
            }
            const int n = p.n_seqs - b0 < 32 ? p.n_seqs - b0 : 32;
            for (int s = 0; s < n; ++s) {
                const int32_t sq0 = __shfl_sync(0xffffffffu, q0, s), sLq = __shfl_sync(0xffffffffu, Lq, s),
                              sLk = __shfl_sync(0xffffffffu, Lk, s);
                for (int64_t t = (int64_t)lane * p.tile_tokens; t < sLq; t += 32 * (int64_t)p.tile_tokens) {
                    const int32_t nt = packed_key_tiles((int32_t)t, p.tile_tokens, sLq, sLk, p.causal);
                    const int32_t at = atomicAdd(&bins[bin_of(nt)], 1);
                    if (pass == 1) {
                        PackedEntry e = {b0 + s, (int32_t)t, sLq, sLk, sq0, nt, 0, 0};
                        p.entries[at] = e;
                    }
                }
            }
        }
        __syncthreads();
        if (pass == 0) {
            // counts -> first index of each bin
            constexpr int kPer = kPackedBins / kPackedPrepThreads;
            int32_t sum = 0;
            for (int i = 0; i < kPer; ++i)
                sum += bins[tid * kPer + i];
            int32_t inc = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d)
                    inc += o;
            }
            if (lane == 31)
                warp_sum[warp] = inc;
            __syncthreads();
            int32_t at = inc - sum;
            for (int w = 0; w < warp; ++w)
                at += warp_sum[w];
            for (int i = 0; i < kPer; ++i) {
                const int32_t n = bins[tid * kPer + i];
                bins[tid * kPer + i] = at;
                at += n;
            }
            if (tid == kPackedPrepThreads - 1)
                *p.n_entries = at;
            __syncthreads();
        }
    }
}

// The four maps of sequence b, one warp: the template with the sequence's
// address and row count, made in shared memory and published to global memory
// for the tensor-map proxy.
static __device__ void packed_maps(const PackedPlan &p, const PackedMapTemplates &tmpl, int32_t b,
                            CUtensorMap *buf)
{
    const int lane = threadIdx.x & 31;
    const int32_t q0 = p.cu_q[b], k0 = p.cu_k[b];
    const int32_t nq = p.cu_q[b + 1] - q0, nk = p.cu_k[b + 1] - k0;
    for (int i = 0; i < kPackedMaps; ++i) {
        const bool keys = i < 2;
        const int32_t start = keys ? k0 : q0, rows = keys ? nk : nq;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(&tmpl.m[i]);
        reinterpret_cast<uint32_t *>(buf)[lane] = src[lane];
        __syncwarp();
        if (lane == 0) {
            const uint32_t s = attn_smem_u32(buf);
            asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;"
                         ::"r"(s), "l"(p.base[i] + (int64_t)start * p.step[i])
                         : "memory");
            // rows are the second dimension of K and V, the third of Q and O
            if (keys)
                asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;"
                             ::"r"(s), "r"(rows < 1 ? 1 : rows)
                             : "memory");
            else
                asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 2, %1;"
                             ::"r"(s), "r"(rows < 1 ? 1 : rows)
                             : "memory");
        }
        __syncwarp();
        asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync."
                     "aligned [%0], [%1], 128;"
                     ::"l"(p.maps + (int64_t)b * kPackedMaps + i), "r"(attn_smem_u32(buf))
                     : "memory");
        __syncwarp();
    }
}

// The list (CTA 0), the maps (the next map_blocks CTAs), and the keys of the
// packed sequences rotated into [Hk][total][D] (the others; a group of D / 16
// lanes owns up to four heads of a token).
template <typename T, int LAYOUT, int D>
__global__ void __launch_bounds__(kPackedPrepThreads)
    rope_packed_prepare_kernel(const RowsArgs a, const PackedPlan p,
                               const __grid_constant__ PackedMapTemplates tmpl)
{
    constexpr int L = D / 16, kGroups = kPackedPrepThreads / L, kHeads = 4;
    __shared__ __align__(128) CUtensorMap buf[kPackedPrepThreads / 32];
    __shared__ int32_t bins[kPackedBins];      // the planner's; else the first offsets
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        packed_list(p, bins);
        return;
    }
    if ((int)blockIdx.x <= p.map_blocks) {
        constexpr int kWarps = kPackedPrepThreads / 32;
        for (int64_t b = (int64_t)(blockIdx.x - 1) * kWarps + (tid >> 5); b < p.n_seqs;
             b += (int64_t)p.map_blocks * kWarps) {
            bool fits;
            if (packed_sequence_ok(p, (int32_t)b, fits))
                packed_maps(p, tmpl, (int32_t)b, &buf[tid >> 5]);
        }
        return;
    }
    const int j = tid % L;
    const int32_t chunks = (a.Hk + kHeads - 1) / kHeads;
    const int64_t unit = (int64_t)(blockIdx.x - 1 - p.map_blocks) * kGroups + tid / L;
    const int64_t t = unit / chunks;
    const int32_t h0 = (int32_t)(unit - t * chunks) * kHeads;
    const bool live = t < a.total;
    const RowPart part = row_part<LAYOUT>(j, a.rotary_dim);
    uint4 x0[kHeads], x1[kHeads];
    const T *ks = static_cast<const T *>(a.k) + t * a.k_stride;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (live && h0 + i < a.Hk) {
            x0[i] = __ldg(reinterpret_cast<const uint4 *>(ks + (h0 + i) * D + part.o0));
            x1[i] = __ldg(reinterpret_cast<const uint4 *>(ks + (h0 + i) * D + part.o1));
        }
    }
    int64_t row;
    if (a.pos != nullptr) {
        row = live ? __ldg(a.pos + t) : -1;
    } else {
        const bool cached = a.n_seqs + 1 <= kPackedBins;
        if (cached) {
            for (int32_t i = tid; i <= a.n_seqs; i += kPackedPrepThreads)
                bins[i] = __ldg(a.cu + i);
            __syncthreads();
        }
        const int32_t *cu = cached ? bins : a.cu;
        row = t - cu[find_sequence(cu, a.n_seqs, t)];
    }
    if (!live)
        return;
    if (row < 0 || row >= a.table_rows) {
        // indices past the table refuse the whole call in the plan; rows of no
        // sequence are not read
        if (j == 0 && a.pos != nullptr && row != -1)
            atomicOr(a.flag, kFlagPosition);
        row = -1;
    }
    if (part.rot && row >= 0) {
        float c[8], s[8];
        const int64_t at = row * (a.rotary_dim / 2) + 8 * j;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(a.cos + at) + q);
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(a.sin + at) + q);
            c[4 * q] = c4.x; c[4 * q + 1] = c4.y; c[4 * q + 2] = c4.z; c[4 * q + 3] = c4.w;
            s[4 * q] = s4.x; s[4 * q + 1] = s4.y; s[4 * q + 2] = s4.z; s[4 * q + 3] = s4.w;
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h0 + i < a.Hk)
                rotate_part<T, LAYOUT>(x0[i], x1[i], c, s);
    }
    T *out = static_cast<T *>(a.k_out);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (h0 + i < a.Hk) {
            T *dst = out + ((int64_t)(h0 + i) * a.total + t) * D;
            *reinterpret_cast<uint4 *>(dst + part.o0) = x0[i];
            *reinterpret_cast<uint4 *>(dst + part.o1) = x1[i];
        }
    }
}

// ---------------------------------------------------------------------------
// 2. the attention

// Shared memory of a CTA: the query tile, the stages of key and value halves,
// the cos and the sin rows of the tile's tokens, the output tile.  A token's
// table row of 2 * rotary_dim bytes sits at packed_table_offset: 16 bytes of
// padding after every second row spread the rows over the banks (a full row
// of padding each would not fit the 227 KB with 128 tokens a tile).
constexpr int kPackedStages = k2Stages;
__host__ __device__ constexpr uint32_t packed_table_offset(uint32_t t, uint32_t row_bytes)
{
    return t * row_bytes + (t >> 1) * 16;
}
template <int D>
constexpr uint32_t kPackedTile = kAttnRows * D * 2;
template <int D>
constexpr uint32_t kPackedHalf = 64 * D * 2;   // 64 keys of D features, or 128 of D / 2
template <int D>
constexpr uint32_t kPackedTable = packed_table_offset(kAttnRows, 2 * D);
template <int D>
constexpr uint32_t kPackedSmem = 2 * kPackedTile<D> + kPackedStages * 2 * kPackedHalf<D> +
                                 2 * kPackedTable<D>;

// V's MN-major operand: D = 128: 64 features x 128 keys, 128-byte swizzle;
// D = 64: 32 features x 128 keys, 64-byte swizzle (descriptor layout 4), 8-row
// groups of 512 bytes.
template <int D>
__device__ __forceinline__ uint64_t packed_v_desc(uint32_t addr, int kk)
{
    return D == 128 ? umma_desc(addr + kk * 2048u, kBoxBytes, 1024u, kSwizzle128)
                    : umma_desc(addr + kk * 1024u, 64u * 128u, 512u, 4u);
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(attn_smem_u32(dst)), "l"(src), "r"(bytes), "r"(attn_smem_u32(bar))
                 : "memory");
}

// A map written by the prepare kernel, before this thread's first copy with it.
__device__ __forceinline__ void acquire_map(const CUtensorMap *m)
{
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(m) : "memory");
}

// Rotates the query tile in place: rows r = token * GP + head, table rows of
// the tokens in sC / sS.  Tokens past Lq hold zeros, tokens that are not
// rotated (position -1 or out of range) have no table row.
template <typename T, int LAYOUT, int NF>
__device__ __forceinline__ void rotate_packed_tile(uint8_t *sQ, const uint8_t *sC, const uint8_t *sS,
                                                   int32_t tok0, int32_t Lq, int lg,
                                                   const int32_t *pos, const AttnArgs &a, int tid)
{
    constexpr int NQ = LAYOUT == 0 ? 2 : 1;
    const int rd = a.rotary_dim, h8 = rd / 16;
    const int per_row = LAYOUT == 0 ? rd / 16 : rd / 8;
    const int tok = tid >> lg;                 // a thread owns one row of the tile
    bool rot = tok0 + tok < Lq;
    if (rot && pos != nullptr) {
        const int32_t r = __ldg(pos + tok0 + tok);
        rot = r >= 0 && r < a.table_rows;
    }
    if (!rot)
        return;
    const uint8_t *c0 = sC + packed_table_offset(tok, 2 * rd), *s0 = sS + packed_table_offset(tok, 2 * rd);
#pragma unroll 1
    for (int p = 0; p < per_row; p += NF) {
        KeyItem it[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if (f == 0 || p + f < per_row) {
                it[f].o1 = sw128(tid, p + f);
                it[f].o2 = sw128(tid, p + f + h8);
                it[f].rot = true;
                it[f].x1 = *reinterpret_cast<const uint4 *>(sQ + it[f].o1);
                if (LAYOUT == 0)
                    it[f].x2 = *reinterpret_cast<const uint4 *>(sQ + it[f].o2);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(c0 + ((p + f) * NQ + q) * 16);
                    const float4 s4 = *reinterpret_cast<const float4 *>(s0 + ((p + f) * NQ + q) * 16);
                    it[f].cs[4 * q] = c4.x; it[f].cs[4 * q + 1] = c4.y;
                    it[f].cs[4 * q + 2] = c4.z; it[f].cs[4 * q + 3] = c4.w;
                    it[f].sn[4 * q] = s4.x; it[f].sn[4 * q + 1] = s4.y;
                    it[f].sn[4 * q + 2] = s4.z; it[f].sn[4 * q + 3] = s4.w;
                }
            }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f)
            if (f == 0 || p + f < per_row)
                store_key_item<T, LAYOUT>(it[f], sQ);
    }
}

template <typename T, int LAYOUT, int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(k2Threads, 1)
    rope_attn_packed_kernel(const PackedKernelArgs g_args, const int lg)
{
    constexpr uint32_t kTile = kPackedTile<D>, kHalf = kPackedHalf<D>;
    constexpr uint32_t ab_format = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    const AttnArgs &a = g_args.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem;
    uint8_t *sStages = sQ + kTile;
    uint8_t *sO = sStages + kPackedStages * 2 * kHalf;
    uint8_t *sC = sO + kTile;
    uint8_t *sS = sC + kPackedTable<D>;
    auto sK = [&](int st) { return sStages + st * 2 * kHalf; };
    auto sV = [&](int st) { return sStages + st * 2 * kHalf + kHalf; };
    // as in rope_attn_2sm_kernel: both CTAs' key / value halves landed (leader
    // only); S buffer ready, which releases key stage b (multicast); P ready
    // (leader only, each row warp of both CTAs); O += P V done, which releases
    // value stage b (multicast); query tile and table rows landed; both query
    // tiles rotated (leader only); every MMA of an issuer finished.  Every
    // parity wait is for the phase right after the last one known complete.
    __shared__ __align__(8) uint64_t bar_kfull[kPackedStages], bar_vfull[kPackedStages],
        bar_s[k2SBufs], bar_p[k2SBufs], bar_o[k2SBufs], bar_q, bar_qr, bar_drain[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const bool leader = rank == 0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool math = warp < 4;
    const int tokens = kAttnRows >> lg;            // of a CTA's tile
    // The work units: unit L is entry L / head_units of the list (longest
    // first) for head unit L mod head_units.  Cluster c takes unit
    // r * clusters + c in even rounds r and r * clusters + clusters - 1 - c in
    // odd ones, so a cluster that got the longer work of one round gets the
    // shorter of the next.
    const int64_t n_units = (int64_t)__ldg(g_args.n_entries) * g_args.head_units;
    const int64_t clusters = gridDim.x >> 1, cid = blockIdx.x >> 1;
    auto unit_at = [&](int64_t r) {
        return r * clusters + ((r & 1) ? clusters - 1 - cid : cid);
    };
    struct Unit {
        PackedEntry e;
        int32_t head0, kv;
    };
    auto unit_work = [&](int64_t r) {
        const int64_t L = unit_at(r);
        const int64_t i = L / g_args.head_units;
        const int32_t hu = (int32_t)(L - i * g_args.head_units);
        Unit u;
        const int4 x = __ldg(reinterpret_cast<const int4 *>(g_args.entries + i));
        const int2 y = __ldg(reinterpret_cast<const int2 *>(g_args.entries + i) + 2);
        u.e.seq = x.x; u.e.tok0 = x.y; u.e.Lq = x.z; u.e.Lk = x.w;
        u.e.q_start = y.x; u.e.n_tiles = y.y;
        u.head0 = hu << lg;
        u.kv = hu / g_args.units_per_kv;
        return u;
    };
    auto unit_tiles = [&](int64_t r) { return __ldg(&g_args.entries[unit_at(r) / g_args.head_units].n_tiles); };

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(attn_smem_u32(&tmem_base)), "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < kPackedStages; ++s) {
            mbar_init(&bar_kfull[s], 1);
            mbar_init(&bar_vfull[s], 1);
        }
        for (int b = 0; b < k2SBufs; ++b) {
            mbar_init(&bar_s[b], 1);
            mbar_init(&bar_p[b], 2 * (kAttnRows / 32));
            mbar_init(&bar_o[b], 1);
        }
        mbar_init(&bar_q, 1);
        mbar_init(&bar_qr, 2 * (kAttnRows / 32));
        mbar_init(&bar_drain[0], 1);
        mbar_init(&bar_drain[1], 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync_all();                            // barriers and TMEM of both CTAs ready
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base;
    volatile int *abort = &abort_flag;
    const uint32_t peer_abort = peer_addr(&abort_flag, rank ^ 1u);
    auto raise_abort = [&]() {
        *abort = 1;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_abort), "r"(1) : "memory");
    };
    bool ok = true;

    if (math) {
        // ---- the row block.  Pass r: the key tiles of unit r, then the query
        // tile of unit r + 1, then the epilogue of unit r, so that the next
        // unit's first S products run while the epilogue waits for the last
        // O += P V.  The first pass (r = -1) only rotates the first query tile.
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const uint32_t o_base = tmem + k2OCol + lanes;
        uint32_t sb = 0, s_ph = 0;                 // S buffer of this tile and its phase parity
        uint32_t ob = 0, o_ph = 0;                 // the same for the previous tile (O barriers)
        uint32_t qn = 0;                           // units with key tiles so far
        int32_t o_seq = -1;                        // the sequence whose O map was acquired
        for (int64_t r = -1; ok && (r < 0 || unit_at(r) < n_units); ++r) {
            const bool real = r >= 0;
            int32_t n_tiles = 0, sk = 0;
            int64_t qi = 0, shift = 0;
            if (real) {
                const Unit u = unit_work(r);
                n_tiles = u.e.n_tiles;
                sk = u.e.Lk;
                shift = (int64_t)u.e.Lk - u.e.Lq;
                qi = u.e.tok0 + (int)rank * tokens + (tid >> lg);
            }
            float m_ref = -INFINITY, l_run = 0.0f;
            for (int32_t kt = 0; kt < n_tiles; ++kt) {
                const uint32_t b = sb;
                ok = __all_sync(0xffffffffu, attn_wait(&bar_s[b], s_ph, abort));
                if (!ok)
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                bool o_ok = true;
                auto o_ready = [&]() {
                    o_ok = __all_sync(0xffffffffu, attn_wait(&bar_o[ob], o_ph, abort));
                    return o_ok;
                };
                softmax_tile<T, D, true, false>(tmem + (uint32_t)b * kAttnKeys + lanes, o_base, qi,
                                                (int64_t)kt * kAttnKeys, shift, a, 0, kt > 0, m_ref,
                                                l_run, o_ready, (int64_t)sk);
                ok = o_ok;
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(&bar_p[b]);
                    else
                        mbar_arrive_remote(peer_addr(&bar_p[b], 0));
                }
                ob = sb;
                o_ph = s_ph;
                if (++sb == k2SBufs) {
                    sb = 0;
                    s_ph ^= 1u;
                }
                if (!ok)
                    break;
            }
            if (!ok)
                break;
            // the next unit's query tile, once it has landed: rotated in place
            if (unit_at(r + 1) < n_units && unit_tiles(r + 1) > 0) {
                const Unit n = unit_work(r + 1);
                ok = __all_sync(0xffffffffu, attn_wait(&bar_q, qn & 1u, abort));
                if (!ok)
                    break;
                rotate_packed_tile<T, LAYOUT, 2>(
                    sQ, sC, sS, n.e.tok0 + (int)rank * tokens, n.e.Lq, lg,
                    g_args.pos_q != nullptr ? g_args.pos_q + n.e.q_start : nullptr, a, tid);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_remote(peer_addr(&bar_qr, 0));
                ++qn;
            }
            if (!real)
                continue;
            if (n_tiles > 0)
                ok = __all_sync(0xffffffffu, attn_wait(&bar_o[ob], o_ph, abort));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (!ok)
                break;
            // O / l of the warp's 32 rows, staged and stored by TMA (boxes of
            // 64 features x GP heads x 32 / GP tokens; tokens past Lq are not
            // written, and a box that starts past it is not issued)
            if (lane == 0)
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
            stage_o_row<T, D>(o_base, sO, tid, n_tiles > 0, l_run);
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            const Unit u = unit_work(r);
            const int32_t y0 = u.e.tok0 + (int)rank * tokens + warp * (32 >> lg);
            if (lane == 0 && y0 < u.e.Lq) {
                const CUtensorMap *om = g_args.maps + (int64_t)u.e.seq * kPackedMaps + 3;
                if (u.e.seq != o_seq)
                    acquire_map(om);
                o_seq = u.e.seq;
#pragma unroll
                for (int bx = 0; bx < D / 64; ++bx)
                    tma_store_3d(om, sO + bx * kBoxBytes + warp * 32 * 128, bx * 64, u.head0, y0);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        drain_o_stores();
        if (!ok)
            raise_abort();
    } else if (warp == k2SIssueWarp && leader) {
        // ---- S = Q K^T for both CTAs into S buffer g mod 3
        const uint32_t idesc = umma_idesc(256, kAttnKeys, ab_format, 0);
        const uint32_t q_addr = attn_smem_u32(sQ);
        uint32_t sb = 0, ph = 0, qn = 0;           // buffer (and stage) of tile g, its parity
        bool first = true;                         // the first pass over the buffers
        for (int64_t r = 0; ok && unit_at(r) < n_units; ++r) {
            const int32_t n_tiles = unit_tiles(r);
            if (n_tiles == 0)
                continue;
            ok = __all_sync(0xffffffffu, attn_wait(&bar_qr, qn & 1u, abort));
            ++qn;
            for (int32_t kt = 0; ok && kt < n_tiles; ++kt) {
                ok = __all_sync(0xffffffffu, attn_wait(&bar_kfull[sb], ph, abort) &&
                                                 (first || attn_wait(&bar_o[sb], ph ^ 1u, abort)));
                if (!ok)
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (lane == 0) {
                    const uint32_t k_addr = attn_smem_u32(sK(sb));
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma2_ss(tmem + sb * kAttnKeys,
                                 umma_desc(q_addr + (kk >> 2) * kBoxBytes + (kk & 3) * 32u, 16u,
                                           1024u, kSwizzle128),
                                 umma_desc(k_addr + (kk >> 2) * 8192u + (kk & 3) * 32u, 16u,
                                           1024u, kSwizzle128),
                                 idesc, kk > 0);
                    umma2_commit(&bar_s[sb], 3);
                }
                __syncwarp();
                if (++sb == k2SBufs) {
                    sb = 0;
                    ph ^= 1u;
                    first = false;
                }
            }
        }
        if (lane == 0)
            umma2_commit(&bar_drain[0], 1);
        __syncwarp();
        if (!__all_sync(0xffffffffu, attn_wait(&bar_drain[0], 0u)))
            ok = false;
        if (!ok)
            raise_abort();
    } else if (warp == k2PVIssueWarp && leader) {
        // ---- O += P V for both CTAs once both P are in TMEM
        const uint32_t idesc = umma_idesc(256, D, ab_format, 1);
        uint32_t sb = 0, ph = 0;
        for (int64_t r = 0; ok && unit_at(r) < n_units; ++r) {
            const int32_t n_tiles = unit_tiles(r);
            for (int32_t kt = 0; ok && kt < n_tiles; ++kt) {
                ok = __all_sync(0xffffffffu, attn_wait(&bar_p[sb], ph, abort) &&
                                                 attn_wait(&bar_vfull[sb], ph, abort));
                if (!ok)
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (lane == 0) {
                    const uint32_t v_addr = attn_smem_u32(sV(sb));
#pragma unroll
                    for (int kk = 0; kk < kAttnKeys / 16; ++kk)
                        umma2_ts(tmem + k2OCol, tmem + sb * kAttnKeys + kk * 8,
                                 packed_v_desc<D>(v_addr, kk), idesc, (kt > 0 || kk > 0) ? 1u : 0u);
                    umma2_commit(&bar_o[sb], 3);
                }
                __syncwarp();
                if (++sb == k2SBufs) {
                    sb = 0;
                    ph ^= 1u;
                }
            }
        }
        if (lane == 0)
            umma2_commit(&bar_drain[1], 1);
        __syncwarp();
        if (!__all_sync(0xffffffffu, attn_wait(&bar_drain[1], 0u)))
            ok = false;
        if (!ok)
            raise_abort();
    } else if (warp == k2TmaWarp) {
        // ---- per unit: the query tile and its tokens' table rows once the
        // previous unit's last S has read the old one, then this CTA's halves
        // of key and value tile g into stage g mod 3 once tile g - 3 released it
        uint32_t sb = 0, ph = 0, qn = 0;
        uint32_t pb = 0, p_ph = 0;                 // the previous tile's buffer and parity
        bool first = true, any = false;
        uint32_t k_ph[kPackedStages], v_ph[kPackedStages];   // parity of the last copy (2: none)
#pragma unroll
        for (int s = 0; s < kPackedStages; ++s)
            k_ph[s] = v_ph[s] = 2;
        int32_t seq = -1;
        const uint32_t row_bytes = 2u * (uint32_t)a.rotary_dim;
        for (int64_t r = 0; ok && unit_at(r) < n_units; ++r) {
            const Unit u = unit_work(r);
            const int32_t n_tiles = u.e.n_tiles;
            if (n_tiles == 0)
                continue;
            const CUtensorMap *maps = g_args.maps + (int64_t)u.e.seq * kPackedMaps;
            if (u.e.seq != seq) {
                acquire_map(maps);
                acquire_map(maps + 1);
                acquire_map(maps + 2);
                seq = u.e.seq;
            }
            // the table rows of this lane's tokens (-1: none)
            const int32_t tok0 = u.e.tok0 + (int)rank * tokens;
            int32_t trow[4];
            uint32_t n_rows = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = lane + 32 * i;
                trow[i] = -1;
                if (t < tokens && tok0 + t < u.e.Lq) {
                    trow[i] = tok0 + t;
                    if (g_args.pos_q != nullptr) {
                        trow[i] = __ldg(g_args.pos_q + u.e.q_start + tok0 + t);
                        if (trow[i] < 0 || trow[i] >= a.table_rows) {
                            if (trow[i] != -1)
                                atomicOr(a.flag, kFlagPosition);
                            trow[i] = -1;
                        }
                    }
                }
                n_rows += trow[i] >= 0 ? 1u : 0u;
            }
            n_rows = __reduce_add_sync(0xffffffffu, n_rows);
            if (any)
                ok = __all_sync(0xffffffffu, attn_wait(&bar_s[pb], p_ph, abort));
            if (!ok)
                break;
            if (lane == 0)
                mbar_expect_tx(&bar_q, kTile + n_rows * 2u * row_bytes);
            __syncwarp();
            if (lane < D / 64)
                tma_load_3d(sQ + lane * kBoxBytes, maps + 2, lane * 64, u.head0, tok0, &bar_q);
            // (a box that starts past Lq arrives as zeros)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (trow[i] >= 0) {
                    const uint32_t at = packed_table_offset(lane + 32 * i, row_bytes);
                    const int64_t src = (int64_t)trow[i] * (a.rotary_dim / 2);
                    bulk_load(sC + at, a.cos + src, row_bytes, &bar_q);
                    bulk_load(sS + at, a.sin + src, row_bytes, &bar_q);
                }
            }
            ++qn;
            for (int32_t kt = 0; ok && kt < n_tiles; ++kt) {
                const int k0 = kt * kAttnKeys;
                if (!first)
                    ok = __all_sync(0xffffffffu, attn_wait(&bar_s[sb], ph ^ 1u, abort));
                if (!ok)
                    break;
                // keys k0 + 64 rank .. + 63; both CTAs' bytes complete the
                // leader's barrier
                if (leader && lane == 0)
                    mbar_expect_tx(&bar_kfull[sb], 2 * kHalf);
                __syncwarp();
                if (lane < D / 64) {
                    if (leader)
                        tma_load_3d(sK(sb) + lane * 8192, maps, lane * 64, k0, u.kv, &bar_kfull[sb]);
                    else
                        tma_load_3d_to_leader(sK(sb) + lane * 8192, maps, lane * 64, k0 + 64, u.kv,
                                              peer_addr(&bar_kfull[sb], 0));
                }
                k_ph[sb] = ph;
                if (!first)
                    ok = __all_sync(0xffffffffu, attn_wait(&bar_o[sb], ph ^ 1u, abort));
                if (!ok)
                    break;
                // features D/2 rank .. of the tile's 128 keys
                if (lane == 0) {
                    if (leader) {
                        mbar_expect_tx(&bar_vfull[sb], 2 * kHalf);
                        tma_load_3d(sV(sb), maps + 1, 0, k0, u.kv, &bar_vfull[sb]);
                    } else {
                        tma_load_3d_to_leader(sV(sb), maps + 1, D / 2, k0, u.kv,
                                              peer_addr(&bar_vfull[sb], 0));
                    }
                }
                __syncwarp();
                v_ph[sb] = ph;
                pb = sb;
                p_ph = ph;
                any = true;
                if (++sb == k2SBufs) {
                    sb = 0;
                    ph ^= 1u;
                    first = false;
                }
            }
        }
        if (!ok) {
            raise_abort();
            // one more bounded wait for the last query tile and, in the leader
            // (its barriers count both CTAs' bytes), the last copies into each stage
            if (qn > 0)
                (void)attn_wait(&bar_q, (qn - 1) & 1u);
#pragma unroll
            for (int s = 0; s < kPackedStages; ++s) {
                if (leader && k_ph[s] < 2)
                    (void)attn_wait(&bar_kfull[s], k_ph[s]);
                if (leader && v_ph[s] < 2)
                    (void)attn_wait(&bar_vfull[s], v_ph[s]);
            }
        }
    }
    // every role has left its loops; the pair meets once more before TMEM is
    // freed, so no MMA of the leader still reads the follower's memory
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync_all();
    if (tid == 0 && *abort)
        atomicOr(a.flag, kFlagTimeout);
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
}

// ---------------------------------------------------------------------------
// host side

// A rank-3 map of 16-bit elements; box of the given extents, no out-of-range
// fill but zeros.
static bool encode_3d(EncodeTiledFn enc, CUtensorMap *m, const void *base, CUtensorMapDataType dt,
                      const int64_t (&dims)[3], const int64_t (&strides)[2], const uint32_t (&box)[3],
                      CUtensorMapSwizzle swizzle)
{
    const cuuint64_t d[3] = {(cuuint64_t)dims[0], (cuuint64_t)dims[1], (cuuint64_t)dims[2]};
    const cuuint64_t s[2] = {(cuuint64_t)strides[0], (cuuint64_t)strides[1]};
    const cuuint32_t b[3] = {box[0], box[1], box[2]};
    const cuuint32_t e[3] = {1, 1, 1};
    return enc(m, dt, 3, const_cast<void *>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int LAYOUT, int D>
static cudaError_t launch_packed(const PackedArgs &c, const PackedLayout &lay, cudaStream_t st)
{
    EncodeTiledFn enc = encode_tiled();
    if (enc == nullptr)
        return cudaErrorNotSupported;
    const CUtensorMapDataType dt = std::is_same<T, __nv_bfloat16>::value
                                       ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const RowsArgs &k = c.keys;
    uint8_t *ws = static_cast<uint8_t *>(c.workspace);
    const int32_t gp = packed_group_heads(c.Hq, k.Hk);
    const int lg = __builtin_ctz((unsigned)gp);
    const int64_t total_k = k.total > 0 ? k.total : 1;

    // map templates: rotated K, V, Q, O (without keys K and V stand on the
    // workspace and are never used)
    PackedMapTemplates tmpl;
    const void *v = k.total > 0 ? k.v : ws;
    const int64_t vs = k.total > 0 ? k.v_stride : (int64_t)k.Hk * D;
    const uint32_t g = (uint32_t)gp;
    if (!encode_3d(enc, &tmpl.m[0], ws + lay.keys, dt, {D, total_k, k.Hk}, {D * 2, total_k * D * 2},
                   {64, 64, 1}, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_3d(enc, &tmpl.m[1], v, dt, {D, total_k, k.Hk}, {vs * 2, D * 2},
                   {(uint32_t)D / 2, (uint32_t)kAttnKeys, 1},
                   D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_3d(enc, &tmpl.m[2], c.q, dt, {D, c.Hq, c.total_q}, {D * 2, c.q_stride * 2},
                   {64, g, kAttnRows / g}, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_3d(enc, &tmpl.m[3], c.o, dt, {D, c.Hq, c.total_q}, {D * 2, (int64_t)c.Hq * D * 2},
                   {64, g, 32 / g}, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;

    PackedPlan p;
    memset(&p, 0, sizeof p);
    p.cu_q = c.cu_q; p.cu_k = k.cu; p.n_seqs = k.n_seqs;
    p.total_q = c.total_q; p.total_k = k.total;
    p.causal = c.causal; p.tile_tokens = 2 * kAttnRows / gp;
    p.check_q_rows = c.pos_q == nullptr; p.check_k_rows = k.pos == nullptr;
    p.table_rows = k.table_rows;
    p.n_entries = reinterpret_cast<int32_t *>(ws);
    p.entries = reinterpret_cast<PackedEntry *>(ws + lay.entries);
    p.maps = reinterpret_cast<CUtensorMap *>(ws + lay.maps);
    p.base[0] = (int64_t)(ws + lay.keys); p.step[0] = D * 2;
    p.base[1] = (int64_t)v; p.step[1] = vs * 2;
    p.base[2] = (int64_t)c.q; p.step[2] = c.q_stride * 2;
    p.base[3] = (int64_t)c.o; p.step[3] = (int64_t)c.Hq * D * 2;
    p.flag = k.flag;
    // four warps a CTA, one sequence a warp, 256 CTAs at most
    const int64_t map_blocks = (k.n_seqs + 3) / 4;
    p.map_blocks = (int32_t)(map_blocks < 256 ? map_blocks : 256);
    RowsArgs rows = k;
    rows.k_out = ws + lay.keys;
    const int64_t groups = kPackedPrepThreads / (D / 16);
    const int64_t units = k.total * ((k.Hk + 3) / 4);
    const int64_t blocks = (units + groups - 1) / groups + 1 + p.map_blocks;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    rope_packed_prepare_kernel<T, LAYOUT, D><<<(unsigned)blocks, kPackedPrepThreads, 0, st>>>(rows, p, tmpl);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;

    PackedKernelArgs ka;
    memset(&ka, 0, sizeof ka);
    ka.a.cos = k.cos; ka.a.sin = k.sin; ka.a.rotary_dim = k.rotary_dim; ka.a.table_rows = k.table_rows;
    ka.a.scale_log2 = c.scale_log2; ka.a.causal = c.causal; ka.a.flag = k.flag;
    ka.entries = p.entries; ka.n_entries = p.n_entries; ka.maps = p.maps;
    ka.pos_q = c.pos_q;
    ka.head_units = c.Hq / gp;
    ka.units_per_kv = c.Hq / k.Hk / gp;

    static std::atomic<uint64_t> raised{0};        // bit d: shared-memory limit raised on device d
    static std::atomic<int> sm_count[64];          // multiprocessors of device d (0: not read yet)
    // at least 120 KB, so that one CTA holds an SM (and its TMEM)
    constexpr int kSmem = kPackedSmem<D> > 120 * 1024 ? (int)kPackedSmem<D> : 120 * 1024;
    auto *kernel = rope_attn_packed_kernel<T, LAYOUT, D>;
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    int sms = sm_count[dev].load(std::memory_order_acquire);
    if (sms == 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        sm_count[dev].store(sms, std::memory_order_release);
    }
    const uint64_t bit = (uint64_t)1 << dev;
    if (!(raised.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess)
            return e;
        raised.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int64_t most = lay.tiles * ka.head_units;
    const int64_t clusters = most < sms / 2 ? most : sms / 2;
    kernel<<<dim3((unsigned)(2 * clusters)), k2Threads, kSmem, st>>>(ka, lg);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_packed_type(const PackedArgs &c, const PackedLayout &lay, int32_t D, int32_t layout,
                               cudaStream_t st)
{
    if (layout == 0)
        return D == 64 ? launch_packed<T, 0, 64>(c, lay, st) : launch_packed<T, 0, 128>(c, lay, st);
    return D == 64 ? launch_packed<T, 1, 64>(c, lay, st) : launch_packed<T, 1, 128>(c, lay, st);
}

}  // namespace rope
