// rope_norm.cuh -- the RMS norm of query and key heads with the rotation in
// the same pass: forward, backward, and on the way into a paged cache.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  y = R(t) (w * n)
//
// for every head row x of D features, w one weight per feature (of all query
// heads, or of all key heads), R(t) the rotation of the first rotary_dim
// features by the table's angles.  R is orthogonal, so with g = R(-t) dy
//   dw = sum over rows of g * n,
//   dx = r (w * g - n mean(w * g * n)).
// The backward pass reads x again and forms r anew: that costs nothing beside
// the bytes, and the forward pass has nothing to keep.
//
// What bounds it: bytes.  Forward reads and writes a row once, backward reads
// two and writes one.  A group of L lanes (the power of two from D / 16) owns
// U heads of one token, a lane two vectors of 8 features that hold both
// elements of its pairs (row_part), so the rotation needs no exchange, the mean
// log2(L) shuffles, and the loads of all heads are in flight before the first
// is used.  Cos, sin and weights are read once for the U heads.
//
// All arithmetic is fp32 from the loaded elements on; a result is rounded
// once, when it is stored.
#pragma once

#include "rope_norm_internal.cuh"
#include "rope_rows.cuh"

namespace rope {

constexpr int kNormThreads = 128;
// Heads of a token that a group has in flight: 8 KB of a warp's loads either way.
template <typename T>
static constexpr int kNormHeads = sizeof(T) == 2 ? 4 : 2;

// Eight consecutive features.
template <typename T>
struct Vec8 {
    static constexpr int N = (int)sizeof(T) / 2;   // 16-byte words
    uint4 u[N];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            u[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            __stcs(reinterpret_cast<uint4 *>(p) + i, u[i]);
    }
    __device__ __forceinline__ void unpack(float *f) const
    {
        constexpr int V = Elt<T>::V;
#pragma unroll
        for (int i = 0; i < N; ++i)
            Elt<T>::unpack(u[i], *reinterpret_cast<float(*)[V]>(f + i * V));
    }
    __device__ __forceinline__ void pack(const float *f)
    {
        constexpr int V = Elt<T>::V;
#pragma unroll
        for (int i = 0; i < N; ++i)
            u[i] = Elt<T>::pack(*reinterpret_cast<const float(*)[V]>(f + i * V));
    }
};

// A lane's 16 features of a row: two vectors.
template <typename T>
struct RowVecs {
    Vec8<T> v0, v1;
    __device__ __forceinline__ void load(const T *row, const RowPart &p)
    {
        v0.load(row + p.o0);
        v1.load(row + p.o1);
    }
    __device__ __forceinline__ void store(T *row, const RowPart &p) const
    {
        v0.store(row + p.o0);
        v1.store(row + p.o1);
    }
    __device__ __forceinline__ void unpack(float (&f)[16]) const
    {
        v0.unpack(f);
        v1.unpack(f + 8);
    }
    __device__ __forceinline__ void pack(const float (&f)[16])
    {
        v0.pack(f);
        v1.pack(f + 8);
    }
};

// A lane's 16 weights (ones without any), in fp32 or in the rows' type.
template <typename T>
__device__ __forceinline__ void norm_weights(const void *w, int32_t w_f32, const RowPart &p, float (&f)[16])
{
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            f[i] = 1.0f;
    } else if (w_f32) {
        const float *s = static_cast<const float *>(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = __ldg(reinterpret_cast<const float4 *>(s + (i < 2 ? p.o0 : p.o1)) + (i & 1));
            f[4 * i] = t.x; f[4 * i + 1] = t.y; f[4 * i + 2] = t.z; f[4 * i + 3] = t.w;
        }
    } else if constexpr (sizeof(T) == 2) {
        const T *s = static_cast<const T *>(w);
        Elt<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(s + p.o0)), *reinterpret_cast<float(*)[8]>(f));
        Elt<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(s + p.o1)), *reinterpret_cast<float(*)[8]>(f + 8));
    }
}

// The sum of x over the L lanes of a group, in every lane.
template <int L>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

__device__ __forceinline__ float square_sum(const float (&f)[16])
{
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a = fmaf(f[i], f[i], a);
        b = fmaf(f[8 + i], f[8 + i], b);
    }
    return a + b;
}

// A lane's pairs turned by the angles of (c, s).
template <int LAYOUT>
__device__ __forceinline__ void turn(float (&f)[16], const float (&c)[8], const float (&s)[8], float sign)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (LAYOUT == 0)
            rotate_pair(f[e], f[8 + e], c[e], sign * s[e]);
        else
            rotate_pair(f[2 * e], f[2 * e + 1], c[e], sign * s[e]);
    }
}

// The table row of token t, or -1: not rotated.
__device__ __forceinline__ int64_t norm_row(const NormArgs &a, int64_t t, int64_t b, int64_t s, bool report)
{
    int64_t row = s;
    if (a.pos != nullptr)
        row = __ldg(a.pos + b * a.pos_stride + s);
    if (row < 0 || row >= a.table_rows) {
        if (report && row != -1)
            atomicOr(a.flag, kFlagPosition);
        return -1;
    }
    return row;
}

// Where a group's unit lies: token t, heads h0 .. of tensor i.  With the
// sequence before the heads, neighbouring groups take neighbouring heads; with
// the heads before the sequence, neighbouring tokens: either way a CTA's rows
// lie together.
struct NormUnit {
    int64_t t;
    int32_t h0;
};
__device__ __forceinline__ NormUnit norm_unit(const NormArgs &a, int64_t tile, int32_t g, int32_t groups,
                                              int32_t chunks)
{
    NormUnit u;
    int32_t c;
    if (a.seq_first) {
        const int64_t unit = tile * groups + g;
        u.t = unit / chunks;
        c = (int32_t)(unit - u.t * chunks);
    } else {
        const int64_t tt = tile / chunks;
        c = (int32_t)(tile - tt * chunks);
        u.t = tt * groups + g;
    }
    u.h0 = c * a.chunk_heads;
    return u;
}

// Forward.  One tile (a unit per group) per CTA, the query heads' tiles first:
// the hardware hands them out as CTAs finish.
template <typename T, int LAYOUT, int L>
__global__ void __launch_bounds__(kNormThreads) rope_norm_fwd_kernel(const NormArgs a)
{
    constexpr int U = kNormHeads<T>, kGroups = kNormThreads / L;
    const int tid = threadIdx.x, j = tid % L;
    const bool second = (int64_t)blockIdx.x >= a.tiles[0];
    const NormTensor &x = a.t[second ? 1 : 0];
    const int32_t chunks = (x.heads + U - 1) / U;
    const NormUnit u = norm_unit(a, (int64_t)blockIdx.x - (second ? a.tiles[0] : 0), tid / L, kGroups, chunks);
    const RowPart part = row_part<LAYOUT>(j, a.rotary_dim);
    const bool live = u.t < a.tokens && 16 * j < a.D;
    const int64_t t = u.t < a.tokens ? u.t : 0, b = t / a.S, s = t - b * a.S;

    pdl_wait();
    pdl_trigger();
    RowVecs<T> v[U];
    const T *src = static_cast<const T *>(x.x) + b * x.xs[0] + s * x.xs[1];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (live && u.h0 + i < x.heads)
            v[i].load(src + (u.h0 + i) * x.xs[2], part);
    const int64_t row = norm_row(a, t, b, s, live && j == 0);
    float w[16], c[8], sn[8];
    const bool rot = live && part.rot && row >= 0;
    if (live)
        norm_weights<T>(x.w, a.w_f32, part, w);
    if (rot)
        table_values(a.cos, a.sin, row * (a.rotary_dim / 2) + 8 * j, c, sn);
    T *dst = static_cast<T *>(x.y) + b * x.ys[0] + s * x.ys[1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float f[16];
        float sum = 0.0f;
        if (live && u.h0 + i < x.heads) {
            v[i].unpack(f);
            sum = square_sum(f);
        }
        const float r = __frsqrt_rn(fmaf(group_sum<L>(sum), a.inv_d, a.eps));
        if (live && u.h0 + i < x.heads) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                f[e] = f[e] * r * w[e];
            if (rot)
                turn<LAYOUT>(f, c, sn, 1.0f);
            v[i].pack(f);
            v[i].store(dst + (u.h0 + i) * x.ys[2], part);
        }
    }
}

// Backward.  A CTA takes the tiles blockIdx, blockIdx + grid, ... of the query
// heads, then of the key heads, and keeps its sum of g * n in registers; at the
// end it leaves one row of D partial sums per tensor, which
// rope_norm_weights_kernel adds up in a fixed order (no atomics: the same call
// gives the same bits).
template <typename T, int LAYOUT, int L>
__global__ void __launch_bounds__(kNormThreads) rope_norm_bwd_kernel(const NormArgs a)
{
    constexpr int U = kNormHeads<T> / 2, kGroups = kNormThreads / L;
    const int tid = threadIdx.x, j = tid % L, warp = tid >> 5, lane = tid & 31;
    const RowPart part = row_part<LAYOUT>(j, a.rotary_dim);
    __shared__ float part_sum[kNormThreads / 32][16 * L];
    pdl_wait();
    pdl_trigger();
    for (int k = 0; k < 2; ++k) {
        const NormTensor &x = a.t[k];
        if (x.heads == 0)
            continue;
        const int32_t chunks = (x.heads + U - 1) / U;
        float w[16], acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[e] = 0.0f;
        if (16 * j < a.D)
            norm_weights<T>(x.w, a.w_f32, part, w);
        for (int64_t tile = blockIdx.x; tile < a.tiles[k]; tile += gridDim.x) {
            const NormUnit u = norm_unit(a, tile, tid / L, kGroups, chunks);
            const bool live = u.t < a.tokens && 16 * j < a.D;
            const int64_t t = u.t < a.tokens ? u.t : 0, b = t / a.S, s = t - b * a.S;
            RowVecs<T> v[U], gv[U];
            const T *src = static_cast<const T *>(x.x) + b * x.xs[0] + s * x.xs[1];
            const T *gsrc = static_cast<const T *>(x.g) + b * x.ys[0] + s * x.ys[1];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (live && u.h0 + i < x.heads) {
                    v[i].load(src + (u.h0 + i) * x.xs[2], part);
                    gv[i].load(gsrc + (u.h0 + i) * x.ys[2], part);
                }
            const int64_t row = norm_row(a, t, b, s, live && j == 0);
            float c[8], sn[8];
            const bool rot = live && part.rot && row >= 0;
            if (rot)
                table_values(a.cos, a.sin, row * (a.rotary_dim / 2) + 8 * j, c, sn);
            T *dst = static_cast<T *>(x.y) + b * x.ys[0] + s * x.ys[1];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool on = live && u.h0 + i < x.heads;
                float f[16], g[16];
                float sum = 0.0f, dot = 0.0f;
                if (on) {
                    v[i].unpack(f);
                    gv[i].unpack(g);
                    if (rot)
                        turn<LAYOUT>(g, c, sn, -1.0f);
                    sum = square_sum(f);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        dot = fmaf(g[e] * w[e], f[e], dot);
                }
                const float r = __frsqrt_rn(fmaf(group_sum<L>(sum), a.inv_d, a.eps));
                // mean(w g n) = r mean(w g x)
                const float m = group_sum<L>(dot) * r * a.inv_d;
                if (on) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float n = f[e] * r;
                        acc[e] = fmaf(g[e], n, acc[e]);
                        f[e] = r * fmaf(-n, m, g[e] * w[e]);
                    }
                    v[i].pack(f);
                    v[i].store(dst + (u.h0 + i) * x.ys[2], part);
                }
            }
        }
        if (x.partial == nullptr)
            continue;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
#pragma unroll
            for (int d = L; d < 32; d <<= 1)
                acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], d);
        }
        if (lane < L && 16 * j < a.D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                part_sum[warp][part.o0 + e] = acc[e];
                part_sum[warp][part.o1 + e] = acc[8 + e];
            }
        }
        __syncthreads();
        for (int d = tid; d < a.D; d += kNormThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kNormThreads / 32; ++i)
                sum += part_sum[i][d];
            x.partial[(int64_t)blockIdx.x * a.D + d] = sum;
        }
        __syncthreads();
    }
}

// dw: the sum of the CTAs' rows, 32 features a CTA, eight runs of rows side by side.
template <typename T>
__global__ void __launch_bounds__(256) rope_norm_weights_kernel(const NormArgs a, const int32_t rows)
{
    __shared__ float run[8][32];
    const NormTensor &x = a.t[blockIdx.y];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_trigger();
    if (x.partial == nullptr)
        return;
    float sum = 0.0f;
    if (d < a.D) {
#pragma unroll 8
        for (int i = warp; i < rows; i += 8)
            sum += __ldcg(x.partial + (int64_t)i * a.D + d);
    }
    run[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || d >= a.D)
        return;
#pragma unroll
    for (int i = 1; i < 8; ++i)
        sum += run[i][lane];
    if (a.w_f32)
        static_cast<float *>(x.dw)[d] = sum;
    else
        static_cast<T *>(x.dw)[d] = Elt<T>::from_f(sum);
}

// ---------------------------------------------------------------------------
// Into a paged cache: queries to a dense tensor, keys (the same arithmetic) and
// values to their sequence's pages.  A unit is U heads of one kind of a token;
// which sequence the token belongs to, its page and its table row are looked up
// while the unit's loads are on their way, as in rope_cache_append_kernel.
constexpr int kNormCuCached = 1024;            // sequence offsets kept in shared memory

template <typename T, int LAYOUT, int D>
__global__ void __launch_bounds__(kNormThreads) rope_norm_append_kernel(const NormAppendArgs a)
{
    constexpr int L = D / 16, U = kNormHeads<T>, kGroups = kNormThreads / L;
    __shared__ int32_t s_cu[kNormCuCached];
    const RowsArgs &r = a.rows;
    const int tid = threadIdx.x, j = tid % L;
    const int32_t cq = (a.Hq + U - 1) / U, ck = (r.Hk + U - 1) / U, chunks = cq + 2 * ck;
    const int64_t unit = (int64_t)blockIdx.x * kGroups + tid / L;
    const int64_t t = unit / chunks;
    const int32_t c = (int32_t)(unit - t * chunks);
    const int kind = c < cq ? 0 : (c < cq + ck ? 1 : 2);   // queries, keys, values
    const int32_t h0 = (c - (kind == 0 ? 0 : (kind == 1 ? cq : cq + ck))) * U;
    const int32_t heads = kind == 0 ? a.Hq : r.Hk;
    const bool live = t < r.total;
    const RowPart part = row_part<LAYOUT>(j, r.rotary_dim);

    pdl_wait();
    pdl_trigger();
    RowVecs<T> v[U];
    const T *src = kind == 0 ? static_cast<const T *>(a.q) + t * a.q_stride
                             : (kind == 1 ? static_cast<const T *>(r.k) + t * r.k_stride
                                          : static_cast<const T *>(r.v) + t * r.v_stride);
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (live && h0 + i < heads)
            v[i].load(src + (h0 + i) * D, part);
    const bool cached = r.n_seqs + 1 <= kNormCuCached;
    if (cached) {
        for (int32_t i = tid; i <= r.n_seqs; i += kNormThreads)
            s_cu[i] = __ldg(r.cu + i);
        __syncthreads();
    }
    const int32_t *cu = cached ? s_cu : r.cu;
    if (blockIdx.x == 0) {                     // the offsets themselves: 0 <= cu[i] <= cu[i + 1] <= total
        bool bad = false;
        for (int32_t i = tid; i < r.n_seqs; i += kNormThreads)
            bad = bad || cu[i] < 0 || cu[i] > cu[i + 1] || cu[i + 1] > r.total;
        if (bad)
            atomicOr(r.flag, kFlagIndex);
    }
    bool write = live;
    int64_t slot = 0, page = 0, row = -1;
    if (live) {
        const int32_t b = find_sequence(cu, r.n_seqs, t);
        const int32_t start = cu[b];
        if (t < start || t >= cu[b + 1]) {
            write = false;                     // a row of no sequence
        } else {
            const int64_t have = __ldg(r.cache_lens + b);
            slot = have + (t - start);
            if (kind > 0) {
                const int64_t block = slot >> r.page_shift;
                page = -1;
                if (have >= 0 && block < r.table_stride)
                    page = __ldg(r.table + b * r.table_stride + block);
                if (page < 0 || page >= r.n_pages) {
                    if (j == 0)
                        atomicOr(r.flag, kFlagIndex);
                    write = false;
                }
            }
            if (write && kind < 2) {
                row = r.pos != nullptr ? (int64_t)__ldg(r.pos + t) : r.pos_offset + slot;
                if (row < 0 || row >= r.table_rows) {
                    if (j == 0 && !(r.pos != nullptr && row == -1))
                        atomicOr(r.flag, kFlagPosition);
                    row = -1;                  // not rotated
                }
            }
        }
    }
    float w[16], cs[8], sn[8];
    const bool rot = part.rot && row >= 0;
    if (write && kind < 2)
        norm_weights<T>(kind == 0 ? a.wq : a.wk, a.w_f32, part, w);
    if (rot)
        table_values(r.cos, r.sin, row * (r.rotary_dim / 2) + 8 * j, cs, sn);
    const int64_t in_page = slot & (((int64_t)1 << r.page_shift) - 1);
    T *dst = kind == 0 ? static_cast<T *>(a.q_out) + (t * a.Hq + h0) * D
                       : static_cast<T *>(kind == 1 ? r.k_out : r.v_out) +
                             (((page * r.Hk + h0) << r.page_shift) + in_page) * D;
    const int64_t step = kind == 0 ? D : (int64_t)D << r.page_shift;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const bool on = write && h0 + i < heads;
        float f[16], sum = 0.0f;
        if (on && kind < 2) {
            v[i].unpack(f);
            sum = square_sum(f);
        }
        const float q = __frsqrt_rn(fmaf(group_sum<L>(sum), 1.0f / D, a.eps));
        if (on && kind < 2) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                f[e] = f[e] * q * w[e];
            if (rot)
                turn<LAYOUT>(f, cs, sn, 1.0f);
            v[i].pack(f);
        }
        if (on)
            v[i].store(dst + i * step, part);
    }
}

// ---------------------------------------------------------------------------
// host side
template <typename T, int LAYOUT, int L>
static cudaError_t launch_norm_lanes(NormArgs a, bool backward, cudaStream_t st)
{
    const int64_t groups = kNormThreads / L;
    a.chunk_heads = backward ? kNormHeads<T> / 2 : kNormHeads<T>;
    for (int k = 0; k < 2; ++k) {
        const int64_t chunks = (a.t[k].heads + a.chunk_heads - 1) / a.chunk_heads;
        a.tiles[k] = a.seq_first ? (a.tokens * chunks + groups - 1) / groups
                                 : (a.tokens + groups - 1) / groups * chunks;
    }
    const int64_t tiles = a.tiles[0] + a.tiles[1];
    if (tiles > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    if (!backward)
        return launch_hot(rope_norm_fwd_kernel<T, LAYOUT, L>, dim3((unsigned)tiles), dim3(kNormThreads), 0, st, a);
    const int64_t most = a.tiles[0] > a.tiles[1] ? a.tiles[0] : a.tiles[1];
    // (without rows the sums are zeros)
    const int32_t grid = most < 1 ? 1 : (int32_t)(most < kNormPartials ? most : kNormPartials);
    cudaError_t e = launch_hot(rope_norm_bwd_kernel<T, LAYOUT, L>, dim3((unsigned)grid), dim3(kNormThreads), 0, st, a);
    if (e != cudaSuccess || (a.t[0].partial == nullptr && a.t[1].partial == nullptr))
        return e;
    return launch_hot(rope_norm_weights_kernel<T>, dim3((unsigned)(a.D + 31) / 32, 2), dim3(256), 0, st, a, grid);
}

template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st)
{
    const int lanes = a.D / 16;
#define ROPE_NORM(L)                                                     \
    (layout == 0 ? launch_norm_lanes<T, 0, L>(a, backward, st)           \
                 : launch_norm_lanes<T, 1, L>(a, backward, st))
    return lanes <= 2 ? ROPE_NORM(2) : lanes <= 4 ? ROPE_NORM(4) : lanes <= 8 ? ROPE_NORM(8) : ROPE_NORM(16);
#undef ROPE_NORM
}

template <typename T, int LAYOUT, int D>
static cudaError_t launch_norm_append_t(const NormAppendArgs &a, cudaStream_t st)
{
    constexpr int64_t U = kNormHeads<T>, groups = kNormThreads / (D / 16);
    const int64_t chunks = (a.Hq + U - 1) / U + 2 * ((a.rows.Hk + U - 1) / U);
    const int64_t blocks = (a.rows.total * chunks + groups - 1) / groups;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    return launch_hot(rope_norm_append_kernel<T, LAYOUT, D>, dim3((unsigned)blocks), dim3(kNormThreads), 0, st, a);
}

template <typename T>
cudaError_t launch_norm_append_type(const NormAppendArgs &a, int32_t D, int32_t layout, cudaStream_t st)
{
    if (layout == 0)
        return D == 64 ? launch_norm_append_t<T, 0, 64>(a, st) : launch_norm_append_t<T, 0, 128>(a, st);
    return D == 64 ? launch_norm_append_t<T, 1, 64>(a, st) : launch_norm_append_t<T, 1, 128>(a, st);
}

}  // namespace rope
