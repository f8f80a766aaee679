// rope_attention_packed.cuh -- attention forward over packed sequences of
// different lengths, with rotary Q/K (rope_attention_packed_fwd), on pairs of
// SMs (tcgen05 with cta_group::2, TMEM, TMA).
//
//   o_i = sum_j softmax_j(scale * rot(q_i) . rot(k_j)) v_j
//
// over the keys j of token i's own sequence, j <= i + Lk - Lq when causal.
// Scores, maxima, sums and O are fp32.  Rotated queries and keys, and P before
// P V, are rounded to the element type: a kind::f16 product takes both operands
// in one 16-bit type, and two parts of each would be two to four products where
// their issue is the bound.  The dense attention rounds at the same places, so
// sequences of one length get its bits.
// Two launches:
//   1. rope_packed_prepare_kernel rotates the keys into the workspace
//      ([Hk][total_k][D]), lists the query tiles of all sequences, longest
//      first, and writes a tensor map of each sequence's values;
//   2. rope_attn_packed_kernel walks the list, one cluster of two CTAs per
//      pair of SMs.
//
// Where a sequence ends: a map whose row count is the sequence's length makes
// the copy engine itself end a value tile there, with zeros, so an infinity or
// NaN of the next sequence never meets a zero probability.  Only the values need
// that: keys past the end become scores that the mask replaces, and queries past
// it become rows of their own, which are not written.  (A map that a kernel wrote
// has to be acquired, about a microsecond for the next copy.  With maps of keys,
// queries and outputs too, the helpers did that twice a unit: 64 prompts of 50
// tokens 61 us, so 52; 256 of 20 tokens 176 and 159.)
//
// Rows of a tile: GP heads of one group and consecutive tokens, row = token *
// GP + head, GP the largest power of two (up to 16) that divides the group
// size Hq / Hk.  A cluster's 256 rows are then 256 / GP tokens, so a short
// sequence fills a tile with heads instead of padding, and the tile at the
// causal diagonal spans fewer tokens.  A Q or O box is 64 features x GP heads
// x tokens.
//
// The products, their TMEM buffers and the stages are those of
// rope_attn_2sm_kernel (rope_attention.cuh): M = 256 over the pair, three S
// buffers released by the products that read P from them.  D = 64 runs here too
// (V halves of 32 features, 64-byte swizzle).
#pragma once

#include "rope_attention.cuh"
#include "rope_launch.cuh"
#include "rope_rows.cuh"
#include "rope_serving.cuh"

namespace rope {

// One query tile of a sequence: tokens tok0 .. of sequence seq.
struct alignas(16) PackedEntry {
    int32_t seq, tok0, Lq, Lk;
    int32_t q_start, n_tiles, k_start, pad;    // n_tiles: key tiles the tile's rows can see
};

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
    CUtensorMap *maps;                         // [n_seqs]: of the values
    int64_t base, step;                        // values: address of token 0, bytes from token to token
    int32_t *flag;
    int32_t map_blocks;                        // grid: the planner, the maps, then the rotation
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
    __shared__ int32_t warp_sum[kPackedPrepThreads / 32], warp_most[kPackedPrepThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = kPackedPrepThreads / 32;
    bool bad = false, small = false;
    int32_t most = 0;                          // keys of a sequence
    for (int32_t b = tid; b < p.n_seqs; b += kPackedPrepThreads) {
        bool fits;
        bad = bad || !packed_sequence_ok(p, b, fits);
        small = small || !fits;
        const int32_t keys = p.cu_k[b + 1] - p.cu_k[b];
        most = keys > most ? keys : most;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0)
        warp_most[warp] = most;
    bad = __syncthreads_or(bad);
    small = __syncthreads_or(small);
    if (bad || small) {
        if (tid == 0) {
            atomicOr(p.flag, bad ? kFlagIndex : kFlagPosition);
            *p.n_entries = 0;
        }
        return;
    }
    // a bin for each count there is (all 2048: eight short prompts 22.1 us, so 20.5)
    for (int w = 0; w < kWarps; ++w)
        most = warp_most[w] > most ? warp_most[w] : most;
    const int64_t counts = ((int64_t)most + kAttnKeys - 1) / kAttnKeys + 1;
    const int32_t per = counts < kPackedBins
                            ? ((int32_t)counts + kPackedPrepThreads - 1) / kPackedPrepThreads
                            : kPackedBins / kPackedPrepThreads,
                  used = per * kPackedPrepThreads;
    for (int i = tid; i < used; i += kPackedPrepThreads)
        bins[i] = 0;
    __syncthreads();
    // bin of a count: most key tiles in bin 0
    auto bin_of = [used](int32_t n) { return used - 1 - (n < used - 1 ? n : used - 1); };
    const int32_t share = (p.n_seqs + kWarps - 1) / kWarps, group = share < 32 ? share : 32;
    constexpr int32_t kOwnTiles = 4;
    for (int pass = 0; pass < 2; ++pass) {
        // a warp takes up to 32 sequences at a time, one per lane: a lane the tiles
        // of its own where they are few, all lanes those of the others in turn
        // (all lanes for every sequence: 64 prompts of 50 tokens 52 us, so 44; 2000 of
        // 8 tokens 1150 and 968)
        auto take = [&](int32_t seq, int32_t q0, int32_t k0, int32_t Lq, int32_t Lk, int64_t t) {
            const int32_t nt = packed_key_tiles((int32_t)t, p.tile_tokens, Lq, Lk, p.causal);
            const int32_t at = atomicAdd(&bins[bin_of(nt)], 1);
            if (pass == 1) {
                PackedEntry e = {seq, (int32_t)t, Lq, Lk, q0, nt, k0, 0};
                p.entries[at] = e;
            }
        };
        for (int32_t b0 = warp * group; b0 < p.n_seqs; b0 += kWarps * group) {
            const int32_t mine = b0 + lane;
            int32_t q0 = 0, k0 = 0, Lq = 0, Lk = 0;
            if (lane < group && mine < p.n_seqs) {
                q0 = p.cu_q[mine];
                k0 = p.cu_k[mine];
                Lq = p.cu_q[mine + 1] - q0;
                Lk = p.cu_k[mine + 1] - k0;
            }
            const bool few = Lq <= kOwnTiles * p.tile_tokens;
            if (few)
                for (int64_t t = 0; t < Lq; t += p.tile_tokens)
                    take(mine, q0, k0, Lq, Lk, t);
            for (uint32_t rest = __ballot_sync(0xffffffffu, !few); rest != 0; rest &= rest - 1) {
                const int s = __ffs(rest) - 1;
                const int32_t sq0 = __shfl_sync(0xffffffffu, q0, s), sLq = __shfl_sync(0xffffffffu, Lq, s),
                              sLk = __shfl_sync(0xffffffffu, Lk, s), sk0 = __shfl_sync(0xffffffffu, k0, s);
                for (int64_t t = (int64_t)lane * p.tile_tokens; t < sLq; t += 32 * (int64_t)p.tile_tokens)
                    take(b0 + s, sq0, sk0, sLq, sLk, t);
            }
        }
        __syncthreads();
        if (pass == 0) {
            // counts -> first index of each bin
            int32_t sum = 0;
            for (int i = 0; i < per; ++i)
                sum += bins[tid * per + i];
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
            for (int i = 0; i < per; ++i) {
                const int32_t n = bins[tid * per + i];
                bins[tid * per + i] = at;
                at += n;
            }
            if (tid == kPackedPrepThreads - 1)
                *p.n_entries = at;
            __syncthreads();
        }
    }
}

// The map of sequence b's values, one warp: the template with the sequence's
// address and row count, made in shared memory and published to global memory
// for the tensor-map proxy.
static __device__ void packed_map(const PackedPlan &p, const CUtensorMap &tmpl, int32_t b, CUtensorMap *buf)
{
    const int lane = threadIdx.x & 31;
    const int32_t start = p.cu_k[b], rows = p.cu_k[b + 1] - start;
    reinterpret_cast<uint32_t *>(buf)[lane] = reinterpret_cast<const uint32_t *>(&tmpl)[lane];
    __syncwarp();
    if (lane == 0) {
        const uint32_t s = attn_smem_u32(buf);
        asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;"
                     ::"r"(s), "l"(p.base + (int64_t)start * p.step)
                     : "memory");
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;"
                     ::"r"(s), "r"(rows < 1 ? 1 : rows)
                     : "memory");
    }
    __syncwarp();
    asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync."
                 "aligned [%0], [%1], 128;"
                 ::"l"(p.maps + b), "r"(attn_smem_u32(buf))
                 : "memory");
    __syncwarp();
}

// The list (CTA 0), the maps (the next map_blocks CTAs), and the keys of the
// packed sequences rotated into [Hk][total][D] (the others; a group of D / 16
// lanes owns up to four heads of a token).
template <typename T, int LAYOUT, int D>
__global__ void __launch_bounds__(kPackedPrepThreads)
    rope_packed_prepare_kernel(const RowsArgs a, const PackedPlan p,
                               const __grid_constant__ CUtensorMap tmpl)
{
    constexpr int L = D / 16, kGroups = kPackedPrepThreads / L, kHeads = 4;
    __shared__ __align__(128) CUtensorMap buf[kPackedPrepThreads / 32];
    __shared__ int32_t bins[kPackedBins];      // the planner's; else the first offsets
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();                             // the attention's CTAs may set up beside this
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
                packed_map(p, tmpl, (int32_t)b, &buf[tid >> 5]);
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
        // (what stands at tokens of no sequence is not looked at)
        row = live && t >= __ldg(a.cu) && t < __ldg(a.cu + a.n_seqs) ? __ldg(a.pos + t) : -1;
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
        table_values(a.cos, a.sin, row * (a.rotary_dim / 2) + 8 * j, c, s);
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
//
// 384 threads a CTA, three warpgroups:
//   warps 0-3   the softmax of the CTA's 128 rows (thread t = row t), nothing
//               else: a unit's first tile follows the previous unit's last;
//   warps 4-7   the helpers: they rotate the next unit's query tile in the
//               other of two query buffers and write the finished unit's output,
//               both while the softmax warps are busy with key tiles;
//   warps 8-11  the leader's S = Q K^T issue, its O += P V issue, the CTA's
//               copies of queries and keys, and of values.
// The softmax holds a row's 128 scores in registers, so the warpgroups trade
// registers (setmaxnreg): 240 / 112 / 104 of the 168 they start with (240 / 144
// spilled in the tile loop: 340 us against 317 on the prompts below, side by side).
//
// With query rotation and epilogue on the softmax warps' path (their loop then
// ran tiles, rotation, epilogue in turn, 224 threads a CTA) eight causal prompts
// of 16.4k tokens in all, Hq 32, Hk 8, D 128 took 384 us in this kernel; with
// the helpers 336 us, and as it is now 307 us (1250 TFLOP/s).

constexpr int kPackedThreads = 384;
constexpr int kPackedSIssueWarp = 8, kPackedPVIssueWarp = 9, kPackedKeyWarp = 10, kPackedValueWarp = 11;
constexpr int kPackedStages = k2Stages;
constexpr int kPackedStats = 8;                // units whose row statistics are kept
// O buffers in TMEM: beside three S buffers there is room for two of 64 columns,
// or one of 128.  With two, the next unit's first O += P V does not wait for the
// helpers to read the last unit's O.
template <int D>
static constexpr uint32_t kPackedOBufs = D == 64 ? 2 : 1;
template <int D>
static constexpr uint32_t kPackedTile = kAttnRows * D * 2;
template <int D>
static constexpr uint32_t kPackedHalf = 64 * D * 2;   // 64 keys of D features, or 128 of D / 2
// two query tiles, the stages of key and value halves, the output tile, the
// row statistics (max and sum)
template <int D>
static constexpr uint32_t kPackedSmem = 3 * kPackedTile<D> + kPackedStages * 2 * kPackedHalf<D> +
                                        kPackedStats * kAttnRows * 8;

// V's MN-major operand: D = 128: 64 features x 128 keys, 128-byte swizzle;
// D = 64: 32 features x 128 keys, 64-byte swizzle (descriptor layout 4), 8-row
// groups of 512 bytes.
template <int D>
__device__ __forceinline__ uint64_t packed_v_desc(uint32_t addr, int kk)
{
    return D == 128 ? umma_desc(addr + kk * 2048u, kBoxBytes, 1024u, kSwizzle128)
                    : umma_desc(addr + kk * 1024u, 64u * 128u, 512u, 4u);
}

// A map written by the prepare kernel, before this thread's first copy with it.
__device__ __forceinline__ void acquire_map(const CUtensorMap *m)
{
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(m) : "memory");
}

// One box of a key or value half into this CTA's stage; its bytes count on the
// leader's barrier.
__device__ __forceinline__ void load_half_box(uint8_t *dst, const CUtensorMap *map, int x, int y, int z,
                                              uint64_t *bar, uint32_t rank)
{
    if (rank == 0)
        tma_load_3d(dst, map, x, y, z, bar);
    else
        tma_load_3d_to_leader(dst, map, x, y, z, peer_addr(bar, 0));
}

// L2 policies of copies.  Cached keys and values that a call reads once are
// marked to leave L2 first: a decode step streams more than L2 holds, and what
// it needs again (its code, the block lists, the partial results) would be gone.
__device__ __forceinline__ uint64_t l2_once()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t l2_keep()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_3d_l2(void *dst, const CUtensorMap *map, int x, int y, int z,
                                               uint64_t *bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;"
                 ::"r"(attn_smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(attn_smem_u32(bar)),
                   "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void load_half_box_l2(uint8_t *dst, const CUtensorMap *map, int x, int y, int z,
                                                 uint64_t *bar, uint32_t rank, uint64_t policy)
{
    if (rank == 0)
        tma_load_3d_l2(dst, map, x, y, z, bar, policy);
    else
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::"
                     "complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;"
                     ::"r"(attn_smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z),
                       "r"(peer_addr(bar, 0)), "l"(policy)
                     : "memory");
}

// One unit of work of a cluster: the rows (token, head) of tokens tok0 .. and
// heads head0 .. head0 + GP - 1 against the key tiles first .. first + n_tiles - 1
// of key head kv.
struct PackedUnit {
    int32_t seq, tok0, tokens;                 // tokens: of the sequence (or the batch)
    int32_t q_start, k_start;                  // the sequence's first query and key
    int32_t first, n_tiles, n_keys;            // n_keys: of the sequence (or the prefix)
    int32_t head0, kv, part;                   // part: which partial result (prefix)
};

// Where the units come from and where K and V lie.  PackedSource: the list and
// the values' maps that the prepare kernel wrote; rows end in bf16 / fp16 outputs.
struct PackedSource {
    static constexpr bool kFullUnroll = true;  // of the issue loops (see the kernel)
    static constexpr bool kParts = false;      // units may end in fp32 parts (part >= 0, store_rows)
    static constexpr bool kAllParts = false;   // all of them do
    static constexpr bool kFinish = false;     // other work on SMs without units, or behind them
    template <int D>
    static constexpr int smem_bytes()
    {
        return (int)kPackedSmem<D>;
    }
    AttnArgs a;                                // o, Hq, cos, sin, table_rows, rotary_dim, scale, causal, flag
    CUtensorMap k_map, q_map, o_map;           // rotated keys, queries and outputs of all sequences
    const PackedEntry *entries;
    const int32_t *n_entries;
    const CUtensorMap *maps;                   // [n_seqs]: of the values
    const int32_t *pos_q;
    int32_t head_units;                        // Hq / GP
    int32_t units_per_kv;                      // (Hq / Hk) / GP

    // A cluster's way through the units, longest first: unit r * clusters + c of
    // the list in even rounds r and r * clusters + clusters - 1 - c in odd ones,
    // so a cluster that got the longer work of one round gets the shorter of the
    // next.
    // (launch_packed refuses calls of 2^32 units)
    struct Cursor {
        uint32_t r;
    };
    struct Walk {
        uint32_t n_units, clusters, cid;
    };
    template <int D>
    __device__ __forceinline__ Walk walk(int64_t cid, int64_t clusters, uint8_t *) const
    {
        return {(uint32_t)__ldg(n_entries) * (uint32_t)head_units, (uint32_t)clusters, (uint32_t)cid};
    }
    __device__ __forceinline__ uint32_t at(const Walk &w, const Cursor &c) const
    {
        return c.r * w.clusters + ((c.r & 1) ? w.clusters - 1 - w.cid : w.cid);
    }
    __device__ __forceinline__ Cursor first(const Walk &) const { return {0}; }
    __device__ __forceinline__ void next(const Walk &, Cursor &c) const { ++c.r; }
    __device__ __forceinline__ bool valid(const Walk &w, const Cursor &c) const { return at(w, c) < w.n_units; }
    __device__ __forceinline__ int32_t tiles(const Walk &w, const Cursor &c) const
    {
        return __ldg(&entries[at(w, c) / (uint32_t)head_units].n_tiles);
    }
    __device__ __forceinline__ PackedUnit unit(const Walk &w, const Cursor &c, int lg) const
    {
        const uint32_t L = at(w, c);
        const uint32_t i = L / (uint32_t)head_units;
        const int32_t hu = (int32_t)(L - i * (uint32_t)head_units);
        const int4 x = __ldg(reinterpret_cast<const int4 *>(entries + i));
        const int4 y = __ldg(reinterpret_cast<const int4 *>(entries + i) + 1);
        PackedUnit u;
        u.seq = x.x; u.tok0 = x.y; u.tokens = x.z; u.n_keys = x.w;
        u.q_start = y.x; u.n_tiles = y.y; u.k_start = y.z; u.first = 0; u.part = 0;
        u.head0 = hu << lg;
        u.kv = hu / units_per_kv;
        return u;
    }
    // table row of token t of the unit's sequence (-1: not rotated)
    __device__ __forceinline__ int64_t table_row(const PackedUnit &u, int32_t t) const
    {
        return attn_row(pos_q != nullptr ? pos_q + u.q_start : nullptr, t, a.table_rows, a.flag);
    }
    // (the prefix looks its pages up here, before the stage is waited for)
    template <int D>
    __device__ __forceinline__ int32_t key_place(const PackedUnit &, int32_t, uint32_t, int) const
    {
        return 0;
    }
    template <int D>
    __device__ __forceinline__ int32_t value_place(const PackedUnit &, int32_t, int) const
    {
        return 0;
    }
    // the map of the unit's values, before the first copy with it (seq: the last unit's sequence)
    __device__ __forceinline__ void acquire(const PackedUnit &u, int32_t &seq) const
    {
        if (u.seq != seq)
            acquire_map(maps + u.seq);
        seq = u.seq;
    }
    // this CTA's half of key tile kt (64 keys) and of value tile kt (D / 2 features)
    template <int D>
    __device__ __forceinline__ void load_keys(const PackedUnit &u, int32_t kt, int32_t, uint8_t *dst,
                                              uint64_t *bar, uint32_t rank, int lane) const
    {
        if (lane < D / 64)
            load_half_box(dst + lane * 8192, &k_map, lane * 64,
                          u.k_start + kt * kAttnKeys + 64 * (int)rank, u.kv, bar, rank);
    }
    template <int D>
    __device__ __forceinline__ void load_values(const PackedUnit &u, int32_t kt, int32_t, uint8_t *dst,
                                                uint64_t *bar, uint32_t rank, int lane) const
    {
        if (lane == 0)
            load_half_box(dst, maps + u.seq, D / 2 * (int)rank, kt * kAttnKeys, u.kv, bar, rank);
    }
};

// Brings a table row to L1, one 128-byte line after the other, by `parts` threads.
__device__ __forceinline__ void prefetch_table_row(const AttnArgs &a, int64_t trow, int part, int parts)
{
    const int64_t at = trow * (a.rotary_dim / 2);
    for (int i = part * 32; i < a.rotary_dim / 2; i += parts * 32) {
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.cos + at + i));
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.sin + at + i));
    }
}

// Rotates one query tile in place (rows r = token * GP + head; rows of tokens past
// the sequence's end, the next one's queries or zeros, stay as they are): a thread per row, its table row read from global
// memory.  The helpers run this beside the tile loop, so its latency is hidden.
//
// rotate_pairs2 is rotate_pair on two pairs at once (f32x2 instructions, half
// as many: the helpers share the issue slots of the softmax warps).  With w =
// c d rounded, c d - w is exact, so (a b - w) - (c d - w), each fma rounded
// once, is diff_of_products's sum (equal up to the sign of a zero).
__device__ __forceinline__ void rotate_pairs2(uint64_t &x1, uint64_t &x2, uint64_t c, uint64_t s)
{
    const uint64_t minus = 0xbf800000bf800000ull, sign = 0x8000000080000000ull;    // (-1, -1), sign bits
    const uint64_t n2 = x2 ^ sign;
    const uint64_t w1 = mul_f32x2(n2, s), w2 = mul_f32x2(x2, c);       // -(x2 s), -(-x2 c)
    const uint64_t y1 = fma_f32x2(fma_f32x2(x2, s, w1), minus, fma_f32x2(x1, c, w1));
    const uint64_t y2 = fma_f32x2(fma_f32x2(n2, c, w2), minus, fma_f32x2(x1, s, w2));
    x1 = y1;
    x2 = y2;
}

// Eight 16-bit elements as four f32x2 pairs of neighbours, and back.
template <typename T>
__device__ __forceinline__ void unpack_x2(const uint4 &u, uint64_t (&p)[4])
{
    float f[8];
    Elt<T>::unpack(u, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = f32x2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_x2(const uint64_t (&p)[4])
{
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f32x2_split(p[i], f[2 * i], f[2 * i + 1]);
    return Elt<T>::pack(f);
}

template <typename T, int LAYOUT>
__device__ __forceinline__ void rotate_packed_row(uint8_t *sQ, int64_t trow, const AttnArgs &a, int r)
{
    if (trow < 0)
        return;
    const int rd = a.rotary_dim;
    const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(a.cos + trow * (rd / 2));
    const ulonglong2 *s = reinterpret_cast<const ulonglong2 *>(a.sin + trow * (rd / 2));
    if constexpr (LAYOUT == 0) {
        const int h8 = rd / 16;                    // chunk p of one half with chunk p of the other
#pragma unroll 2
        for (int p = 0; p < h8; ++p) {
            uint4 *q1 = reinterpret_cast<uint4 *>(sQ + sw128(r, p));
            uint4 *q2 = reinterpret_cast<uint4 *>(sQ + sw128(r, p + h8));
            const ulonglong2 c0 = __ldg(c + 2 * p), c1 = __ldg(c + 2 * p + 1);
            const ulonglong2 s0 = __ldg(s + 2 * p), s1 = __ldg(s + 2 * p + 1);
            uint64_t x1[4], x2[4];
            unpack_x2<T>(*q1, x1);
            unpack_x2<T>(*q2, x2);
            rotate_pairs2(x1[0], x2[0], c0.x, s0.x);
            rotate_pairs2(x1[1], x2[1], c0.y, s0.y);
            rotate_pairs2(x1[2], x2[2], c1.x, s1.x);
            rotate_pairs2(x1[3], x2[3], c1.y, s1.y);
            *q1 = pack_x2<T>(x1);
            *q2 = pack_x2<T>(x2);
        }
    } else {
#pragma unroll 2
        for (int p = 0; p < rd / 8; ++p) {         // the pairs (0,1) (2,3) (4,5) (6,7) of chunk p
            uint4 *q = reinterpret_cast<uint4 *>(sQ + sw128(r, p));
            const ulonglong2 cv = __ldg(c + p), sv = __ldg(s + p);
            float f[8], g[8];
            Elt<T>::unpack(*q, f);
            uint64_t a0 = f32x2(f[0], f[2]), b0 = f32x2(f[1], f[3]);
            uint64_t a1 = f32x2(f[4], f[6]), b1 = f32x2(f[5], f[7]);
            rotate_pairs2(a0, b0, cv.x, sv.x);
            rotate_pairs2(a1, b1, cv.y, sv.y);
            f32x2_split(a0, g[0], g[2]);
            f32x2_split(b0, g[1], g[3]);
            f32x2_split(a1, g[4], g[6]);
            f32x2_split(b1, g[5], g[7]);
            *q = Elt<T>::pack(g);
        }
    }
}

template <typename T, int LAYOUT, int D, typename Source>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPackedThreads, 1)
    rope_attn_packed_kernel(const __grid_constant__ Source src, const int lg)
{
    constexpr uint32_t kTile = kPackedTile<D>, kHalf = kPackedHalf<D>, kOBufs = kPackedOBufs<D>;
    constexpr uint32_t ab_format = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    // How far the issue loops are unrolled.  Fully unrolled, the prefix's kernel and
    // the D = 64 ones fall into a mode where the softmax step takes twice as long
    // at full clocks and no wait grows (their code and the softmax's loop no longer
    // sit together in the instruction cache, as it seems): 32 sequences after 128k
    // keys 194 us, with 4 / 2 122 us; D = 64 124 and 115 us.  D = 128 over packed
    // sequences is bound by the issue of its products: 4 / 2 costs 1 %.
    constexpr bool kIssueBound = D == 128 && Source::kFullUnroll;
    constexpr int kSUnroll = kIssueBound ? 8 : 4, kPVUnroll = kIssueBound ? 4 : 2;
    const AttnArgs &a = src.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sStages = smem + 2 * kTile;
    uint8_t *sO = sStages + kPackedStages * 2 * kHalf;
    float2 *sStat = reinterpret_cast<float2 *>(sO + kTile);   // [kPackedStats][128] (max, sum)
    auto sQ = [&](uint32_t b) { return smem + b * kTile; };
    auto sK = [&](uint32_t st) { return sStages + st * 2 * kHalf; };
    auto sV = [&](uint32_t st) { return sStages + st * 2 * kHalf + kHalf; };
    // Per tile, modulo three (as in rope_attn_2sm_kernel): both CTAs' key /
    // value halves landed (leader only); S ready, which releases the key stage
    // (multicast); P ready (leader only, each softmax warp of both CTAs); O += P V
    // done, which releases the value stage (multicast).
    // Per unit with key tiles: query tile landed and rotated (leader only, each
    // helper warp of both CTAs), per query buffer; its last O += P V done (multicast) and its O read (leader
    // only, each helper warp of both CTAs), per O buffer; its row statistics
    // written (each softmax warp), per statistics buffer.  At the end: all MMAs
    // of an issuer.
    // A parity wait is sound only for the phase right after the last one known
    // complete: every barrier below is waited for phase by phase, or its next
    // phase cannot complete before the waiter has moved on.
    __shared__ __align__(8) uint64_t bar_kfull[kPackedStages], bar_vfull[kPackedStages],
        bar_s[k2SBufs], bar_p[k2SBufs], bar_o[k2SBufs], bar_q[2], bar_qr[2],
        bar_odone[kOBufs], bar_stat[kPackedStats], bar_ofree[kOBufs], bar_drain[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const bool leader = rank == 0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tokens = kAttnRows >> lg;            // of a CTA's tile

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(attn_smem_u32(&tmem_base)), "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        constexpr uint32_t kBoth = 2 * (kAttnRows / 32);
        for (int s = 0; s < kPackedStages; ++s) {
            mbar_init(&bar_kfull[s], 1);
            mbar_init(&bar_vfull[s], 1);
        }
        for (int b = 0; b < k2SBufs; ++b) {
            mbar_init(&bar_s[b], 1);
            mbar_init(&bar_p[b], kBoth);
            mbar_init(&bar_o[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bar_q[b], 1);
            mbar_init(&bar_qr[b], kBoth);
            mbar_init(&bar_drain[b], 1);
        }
        for (int b = 0; b < kPackedStats; ++b)
            mbar_init(&bar_stat[b], kAttnRows / 32);
        for (uint32_t b = 0; b < kOBufs; ++b) {
            mbar_init(&bar_odone[b], 1);
            mbar_init(&bar_ofree[b], kBoth);
        }
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
    // arrival of a warp on a barrier of the leader
    auto arrive_leader = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) {
            if (leader)
                mbar_arrive(bar);
            else
                mbar_arrive_remote(peer_addr(bar, 0));
        }
    };
    // what ran before this launch (the prepare kernel) is complete from here on
    pdl_wait();
    // (What follows waits for all of this launch, but for the paged merge's look at the plan:
    // that it may start means that every CTA here has waited for it, so no trigger stands
    // before a wait.)
    pdl_trigger();
    const typename Source::Walk walk = src.template walk<D>(blockIdx.x >> 1, gridDim.x >> 1, smem);   // (CTA-wide)
    using Cursor = typename Source::Cursor;
    auto valid = [&](const Cursor &c) { return src.valid(walk, c); };
    auto unit_of = [&](const Cursor &c) { return src.unit(walk, c, lg); };
    // the first unit with key tiles from c on, and the next one after c
    auto with_tiles = [&](Cursor c) {
        while (valid(c) && src.tiles(walk, c) == 0)
            src.next(walk, c);
        return c;
    };
    auto next_with_tiles = [&](Cursor c) {
        src.next(walk, c);
        return with_tiles(c);
    };
    bool ok = true;

    if (warp < 4) {
        // ---- the softmax of this CTA's rows
        asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        uint32_t sb = 0, s_ph = 0;                 // S buffer of this tile and its phase parity
        uint32_t ob = 0, o_ph = 0;                 // the same for the previous tile (O barriers)
        uint32_t stat = 0;                         // statistics buffer; its low bit: O buffer
        // the next unit is looked up a unit early: between units, its loads would
        // be all that the softmax waits for
        Cursor c = with_tiles(src.first(walk));
        PackedUnit un = {};
        if (valid(c))
            un = unit_of(c);
        while (ok && valid(c)) {
            const int32_t n_tiles = un.n_tiles, n_keys = un.n_keys;
            const int64_t shift = (int64_t)un.n_keys - un.tokens;
            const int64_t qi = un.tok0 + (int)rank * tokens + (tid >> lg);
            const int64_t k0 = (int64_t)un.first * kAttnKeys;
            const uint32_t o_base = tmem + k2OCol + lanes + (stat % kOBufs) * D;
            c = next_with_tiles(c);
            const bool more = valid(c);
            if (more)
                un = unit_of(c);
            float m_ref = -INFINITY, l_run = 0.0f;
            for (int32_t kt = 0; kt < n_tiles; ++kt) {
                const uint32_t b = sb;
                ok = __all_sync(0xffffffffu, role_wait(&bar_s[b], s_ph, abort));
                if (!ok)
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                bool o_ok = true;
                auto o_ready = [&]() {
                    o_ok = __all_sync(0xffffffffu, role_wait(&bar_o[ob], o_ph, abort));
                    return o_ok;
                };
                softmax_tile<T, D, true, false>(tmem + b * kAttnKeys + lanes, o_base, qi,
                                                k0 + (int64_t)kt * kAttnKeys, shift, a, 0, kt > 0, m_ref,
                                                l_run, o_ready, (int64_t)n_keys);
                ok = o_ok;
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                arrive_leader(&bar_p[b]);
                ob = sb;
                o_ph = s_ph;
                if (++sb == k2SBufs) {
                    sb = 0;
                    s_ph ^= 1u;
                }
                if (!ok)
                    break;
            }
            // (the buffer's previous unit, eight before this one, is written: this
            // unit's S waited for an O += P V at most three tiles back, and that for
            // the output of the unit one or two before its own)
            sStat[stat * kAttnRows + tid] = make_float2(m_ref, l_run);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar_stat[stat]);
            stat = (stat + 1) % kPackedStats;
            if (!more)
                break;
        }
        if (!ok)
            raise_abort();
    } else if (warp < 8) {
        // ---- the helpers.  A pass: rotate the next unit's query tile, write this
        // unit's output, and (warp 4) request the query tile of the unit after the
        // next: its buffer is this unit's, whose last product has finished.  The
        // first pass requests two tiles and only rotates.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        const int row = tid - 128, wq = warp - 4;  // row of the tile = TMEM lane
        uint32_t qn = 0, un = 0;                   // query tiles rotated, units with tiles written
        Cursor cq = with_tiles(src.first(walk));   // the unit whose query tile is next
        Cursor c = src.first(walk);                // the unit whose output is next
        Cursor cl = cq;                            // the unit whose query tile is requested next
        uint32_t ln = 0;                           // query tiles requested
        auto load_query = [&]() {
            if (wq == 0 && valid(cl)) {
                const PackedUnit u = unit_of(cl);
                const uint32_t b = ln & 1u;
                if (lane == 0)
                    mbar_expect_tx(&bar_q[b], kTile);
                __syncwarp();
                // (rows of tokens past the sequence's end are not looked at)
                if (lane < D / 64)
                    tma_load_3d(sQ(b) + lane * kBoxBytes, &src.q_map, lane * 64, u.head0,
                                u.q_start + u.tok0 + (int)rank * tokens, &bar_q[b]);
                __syncwarp();
                ++ln;
                cl = next_with_tiles(cl);
            }
        };
        load_query();
        load_query();
        for (bool start = true; ok && (start || valid(c)); start = false) {
            // the next query tile, at most one ahead of the unit being written (a
            // second one would wait for products that wait for this output)
            if (valid(cq) && qn < un + 2) {
                const PackedUnit u = unit_of(cq);
                const uint32_t b = qn & 1u;
                const int32_t tok = u.tok0 + (int)rank * tokens + (row >> lg);
                const int64_t trow = tok < u.tokens ? src.table_row(u, tok) : -1;
                if (trow >= 0)
                    prefetch_table_row(a, trow, row & ((1 << lg) - 1), 1 << lg);
                ok = __all_sync(0xffffffffu, role_wait(&bar_q[b], (qn >> 1) & 1u, abort));
                if (!ok)
                    break;
                rotate_packed_row<T, LAYOUT>(sQ(b), trow, a, row);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                arrive_leader(&bar_qr[b]);
                ++qn;
                cq = next_with_tiles(cq);
            }
            if (start)
                continue;
            const PackedUnit u = unit_of(c);
            src.next(walk, c);
            // the staging tile is free once the last store has read it
            if (lane == 0)
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
            float2 stat = make_float2(-INFINITY, 0.0f);
            if (u.n_tiles > 0) {
                // (a wait for a whole unit: its tiles count too)
                ok = __all_sync(0xffffffffu,
                                role_wait(&bar_stat[un % kPackedStats], (un / kPackedStats) & 1u, abort,
                                          kRoleTries + u.n_tiles) &&
                                    role_wait(&bar_odone[un % kOBufs], (un / kOBufs) & 1u, abort));
                if (!ok)
                    break;
                stat = sStat[(un % kPackedStats) * kAttnRows + row];
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            const int32_t y0 = u.tok0 + (int)rank * tokens + wq * (32 >> lg);
            const uint32_t o_base = tmem + k2OCol + ((uint32_t)(wq * 32) << 16) + (un % kOBufs) * D;
            bool parts = false;
            if constexpr (Source::kParts) {
                parts = u.part >= 0;
                if (parts) {
                    src.template store_rows<D>(u, o_base, y0, lane, lg, stat);
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    arrive_leader(&bar_ofree[un % kOBufs]);
                }
            }
            if constexpr (!Source::kAllParts)
            if (!parts) {
                // O / l of the warp's 32 rows, staged and stored by TMA (boxes
                // of 64 features x GP heads x 32 / GP tokens) or, where the
                // sequence ends within them, by the warp.  O is free for the next
                // unit's products as soon as the last of it is in registers.
                const bool none = stat.y == 0.0f;  // a row that saw no key (0 * v may be NaN)
                const float inv = none ? 0.0f : 1.0f / stat.y;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 64) {
                    float ov[64];
                    if (u.n_tiles > 0) {
                        tmem_ld32_nowait(o_base + c0, ov);
                        tmem_ld32_nowait(o_base + c0 + 32, ov + 32);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                        if (c0 + 64 == D) {
                            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                            arrive_leader(&bar_ofree[un % kOBufs]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            ov[i] = 0.0f;
                    }
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = ov[ch * 8 + e] * inv;
                        const uint4 w = Elt<T>::pack(f);
                        *reinterpret_cast<uint4 *>(sO + sw128(row, c0 / 8 + ch)) =
                            none ? make_uint4(0, 0, 0, 0) : w;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (y0 + (32 >> lg) <= u.tokens) {
                    if (lane == 0) {
#pragma unroll
                        for (int bx = 0; bx < D / 64; ++bx)
                            tma_store_3d(&src.o_map, sO + bx * kBoxBytes + wq * 32 * 128, bx * 64, u.head0,
                                         u.q_start + y0);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                } else {
                    // the sequence's last rows, a row by D / 8 lanes
                    constexpr int kRow = D / 8;
                    T *o = static_cast<T *>(a.o) + ((int64_t)(u.q_start + y0) * a.Hq + u.head0) * D;
                    const int live = (u.tokens - y0) << lg;        // rows (none: negative)
                    for (int r = lane / kRow; r < live; r += 32 / kRow)
                        *reinterpret_cast<uint4 *>(o + ((int64_t)(r >> lg) * a.Hq + (r & ((1 << lg) - 1))) * D +
                                                   lane % kRow * 8) =
                            *reinterpret_cast<const uint4 *>(sO + sw128(wq * 32 + r, lane % kRow));
                    __syncwarp();
                }
            }
            if (u.n_tiles > 0) {
                load_query();
                ++un;
            }
        }
        drain_o_stores();
        if (!ok) {
            // one more bounded wait for the query tiles requested
            raise_abort();
            for (uint32_t i = qn; wq == 0 && i < ln; ++i)
                (void)attn_wait(&bar_q[i & 1u], (i >> 1) & 1u);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == kPackedSIssueWarp && leader) {
            // ---- S = Q K^T for both CTAs into S buffer g mod 3
            const uint32_t idesc = umma_idesc(256, kAttnKeys, ab_format, 0);
            uint32_t sb = 0, ph = 0, qn = 0;       // buffer (and stage) of tile g, its parity
            bool first = true;                     // the first pass over the buffers
            for (Cursor c = with_tiles(src.first(walk)); ok && valid(c); c = next_with_tiles(c)) {
                const int32_t n_tiles = src.tiles(walk, c);
                const uint32_t qb = qn & 1u;
                const uint32_t q_addr = attn_smem_u32(sQ(qb));
                ok = __all_sync(0xffffffffu, role_wait(&bar_qr[qb], (qn >> 1) & 1u, abort));
                ++qn;
                for (int32_t kt = 0; ok && kt < n_tiles; ++kt) {
                    ok = __all_sync(0xffffffffu, role_wait(&bar_kfull[sb], ph, abort) &&
                                                     (first || role_wait(&bar_o[sb], ph ^ 1u, abort)));
                    if (!ok)
                        break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (lane == 0) {
                        const uint32_t k_addr = attn_smem_u32(sK(sb));
#pragma unroll kSUnroll
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
            if (qn > 0) {
                if (lane == 0)
                    umma2_commit(&bar_drain[0], 1);
                __syncwarp();
                if (!__all_sync(0xffffffffu, attn_wait(&bar_drain[0], 0u)))
                    ok = false;
            }
        } else if (warp == kPackedPVIssueWarp && leader) {
            // ---- O += P V for both CTAs once both P are in TMEM
            const uint32_t idesc = umma_idesc(256, D, ab_format, 1);
            uint32_t sb = 0, ph = 0, un = 0;
            for (Cursor c = with_tiles(src.first(walk)); ok && valid(c); c = next_with_tiles(c)) {
                const int32_t n_tiles = src.tiles(walk, c);
                // both CTAs have read the O this unit's overwrites
                const uint32_t o_col = k2OCol + (un % kOBufs) * D, ob = un % kOBufs;
                if (un >= kOBufs)
                    ok = __all_sync(0xffffffffu, role_wait(&bar_ofree[ob], (un / kOBufs - 1) & 1u, abort));
                ++un;
                for (int32_t kt = 0; ok && kt < n_tiles; ++kt) {
                    ok = __all_sync(0xffffffffu, role_wait(&bar_p[sb], ph, abort) &&
                                                     role_wait(&bar_vfull[sb], ph, abort));
                    if (!ok)
                        break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (lane == 0) {
                        const uint32_t v_addr = attn_smem_u32(sV(sb));
#pragma unroll kPVUnroll
                        for (int kk = 0; kk < kAttnKeys / 16; ++kk)
                            umma2_ts(tmem + o_col, tmem + sb * kAttnKeys + kk * 8,
                                     packed_v_desc<D>(v_addr, kk), idesc, (kt > 0 || kk > 0) ? 1u : 0u);
                        umma2_commit(&bar_o[sb], 3);
                        if (kt + 1 == n_tiles)
                            umma2_commit(&bar_odone[ob], 3);
                    }
                    __syncwarp();
                    if (++sb == k2SBufs) {
                        sb = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (un > 0) {
                if (lane == 0)
                    umma2_commit(&bar_drain[1], 1);
                __syncwarp();
                if (!__all_sync(0xffffffffu, attn_wait(&bar_drain[1], 0u)))
                    ok = false;
            }
        } else if (warp == kPackedKeyWarp) {
            // ---- this CTA's halves of key tile g into stage g mod 3 once S(g - 3)
            // released it
            uint32_t sb = 0, ph = 0;
            bool first = true;
            uint32_t last_ph[kPackedStages];       // parity of the last copy (2: none)
#pragma unroll
            for (int s = 0; s < kPackedStages; ++s)
                last_ph[s] = 2;
            for (Cursor c = with_tiles(src.first(walk)); ok && valid(c); c = next_with_tiles(c)) {
                const PackedUnit u = unit_of(c);
                for (int32_t kt = 0; ok && kt < u.n_tiles; ++kt) {
                    const int32_t z = src.template key_place<D>(u, kt, rank, lane);
                    if (!first)
                        ok = __all_sync(0xffffffffu, role_wait(&bar_s[sb], ph ^ 1u, abort));
                    if (!ok)
                        break;
                    // keys 64 rank .. + 63 of the tile; both CTAs' bytes
                    // complete the leader's barrier
                    if (leader && lane == 0)
                        mbar_expect_tx(&bar_kfull[sb], 2 * kHalf);
                    __syncwarp();
                    src.template load_keys<D>(u, kt, z, sK(sb), &bar_kfull[sb], rank, lane);
                    last_ph[sb] = ph;
                    if (++sb == k2SBufs) {
                        sb = 0;
                        ph ^= 1u;
                        first = false;
                    }
                }
            }
            if (!ok) {
                // one more bounded wait, in the leader (its barriers count both
                // CTAs' bytes), for the last copies into each stage
                raise_abort();
#pragma unroll
                for (int s = 0; s < kPackedStages; ++s)
                    if (leader && last_ph[s] < 2)
                        (void)attn_wait(&bar_kfull[s], last_ph[s]);
            }
        } else if (warp == kPackedValueWarp) {
            // ---- this CTA's halves of value tile g into stage g mod 3 once
            // O += P V of tile g - 3 released it (a warp of its own: behind the key
            // copies, the next key tile waited for the product)
            uint32_t sb = 0, ph = 0;
            bool first = true;
            uint32_t last_ph[kPackedStages];
#pragma unroll
            for (int s = 0; s < kPackedStages; ++s)
                last_ph[s] = 2;
            int32_t seq = -1;                      // the sequence whose map was acquired
            for (Cursor c = with_tiles(src.first(walk)); ok && valid(c); c = next_with_tiles(c)) {
                const PackedUnit u = unit_of(c);
                src.acquire(u, seq);
                for (int32_t kt = 0; ok && kt < u.n_tiles; ++kt) {
                    const int32_t z = src.template value_place<D>(u, kt, lane);
                    if (!first)
                        ok = __all_sync(0xffffffffu, role_wait(&bar_o[sb], ph ^ 1u, abort));
                    if (!ok)
                        break;
                    // features D/2 rank .. of the tile's 128 keys
                    if (leader && lane == 0)
                        mbar_expect_tx(&bar_vfull[sb], 2 * kHalf);
                    __syncwarp();
                    src.template load_values<D>(u, kt, z, sV(sb), &bar_vfull[sb], rank, lane);
                    __syncwarp();
                    last_ph[sb] = ph;
                    if (++sb == k2SBufs) {
                        sb = 0;
                        ph ^= 1u;
                        first = false;
                    }
                }
            }
            if (!ok) {
                raise_abort();
#pragma unroll
                for (int s = 0; s < kPackedStages; ++s)
                    if (leader && last_ph[s] < 2)
                        (void)attn_wait(&bar_vfull[s], last_ph[s]);
            }
        }
        if (!ok)
            raise_abort();
    }
    // every role has left its loops; the pair meets once more before TMEM is
    // freed, so no MMA of the leader still reads the follower's memory
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    cluster_sync_all();
    const bool failed = *abort != 0;
    if (tid == 0 && failed)
        atomicOr(a.flag, kFlagTimeout);
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    if constexpr (Source::kFinish)
        src.template finish<T, LAYOUT, D>(walk, smem, failed);
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

// The attention kernel over at most `most` units, one cluster per pair of SMs.
template <typename T, int LAYOUT, int D, typename Source>
static cudaError_t launch_packed_kernel(const Source &src, int64_t most, int lg, cudaStream_t st)
{
    static std::atomic<uint64_t> raised{0};
    // at least 120 KB, so that one CTA holds an SM (and its TMEM)
    constexpr int kUsed = Source::template smem_bytes<D>();
    constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    auto *kernel = rope_attn_packed_kernel<T, LAYOUT, D, Source>;
    int sms = 0, dev = 0;
    cudaError_t e = sm_count(&sms, &dev);
    if (e == cudaSuccess)
        e = raise_smem(reinterpret_cast<const void *>(kernel), kSmem, dev, raised);
    if (e != cudaSuccess)
        return e;
    const int64_t clusters = most < sms / 2 ? most : sms / 2;
    return launch_hot(kernel, dim3((unsigned)(2 * clusters)), dim3(kPackedThreads), kSmem, st, src, lg);
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

    // maps of all sequences (without keys K and V stand on the workspace and are
    // never used), V's a template for those of each sequence
    PackedSource ka;
    memset(&ka, 0, sizeof ka);
    CUtensorMap v_map;
    const void *v = k.total > 0 ? k.v : ws;
    const int64_t vs = k.total > 0 ? k.v_stride : (int64_t)k.Hk * D;
    const uint32_t g = (uint32_t)gp;
    if (!encode_3d(enc, &ka.k_map, ws + lay.keys, dt, {D, total_k, k.Hk}, {D * 2, total_k * D * 2},
                   {64, 64, 1}, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_3d(enc, &v_map, v, dt, {D, total_k, k.Hk}, {vs * 2, D * 2},
                   {(uint32_t)D / 2, (uint32_t)kAttnKeys, 1},
                   D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_3d(enc, &ka.q_map, c.q, dt, {D, c.Hq, c.total_q}, {D * 2, c.q_stride * 2},
                   {64, g, kAttnRows / g}, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_3d(enc, &ka.o_map, c.o, dt, {D, c.Hq, c.total_q}, {D * 2, (int64_t)c.Hq * D * 2},
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
    p.base = (int64_t)v; p.step = vs * 2;
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
    cudaError_t e = launch_hot(rope_packed_prepare_kernel<T, LAYOUT, D>, dim3((unsigned)blocks),
                               dim3(kPackedPrepThreads), 0, st, rows, p, v_map);
    if (e != cudaSuccess)
        return e;

    if (lay.tiles * (c.Hq / gp) >= (1ll << 32) - 1024)
        return cudaErrorInvalidConfiguration;
    ka.a.o = c.o; ka.a.Hq = c.Hq;
    ka.a.cos = k.cos; ka.a.sin = k.sin; ka.a.rotary_dim = k.rotary_dim; ka.a.table_rows = k.table_rows;
    ka.a.scale_log2 = c.scale_log2; ka.a.causal = c.causal; ka.a.flag = k.flag;
    ka.entries = p.entries; ka.n_entries = p.n_entries; ka.maps = p.maps;
    ka.pos_q = c.pos_q;
    ka.head_units = c.Hq / gp;
    ka.units_per_kv = c.Hq / k.Hk / gp;

    return launch_packed_kernel<T, LAYOUT, D>(ka, lay.tiles * ka.head_units, lg, st);
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
