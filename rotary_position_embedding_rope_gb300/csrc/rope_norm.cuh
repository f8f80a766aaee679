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
// a token, a lane 16 features of every head that hold both elements of its
// pairs (NormPart), so the rotation needs no exchange and the mean log2(L)
// shuffles.
//
// All arithmetic is fp32 from the loaded elements on; a result is rounded
// once, when it is stored.
#pragma once

#include <cooperative_groups.h>

#include "rope_f32x2.cuh"
#include "rope_launch.cuh"
#include "rope_norm_internal.cuh"
#include "rope_rows.cuh"

namespace rope {

constexpr int kNormThreads = 128;

// The 16 features of a head row that lane j of D / 16 owns: N words of 16 bytes, V
// features each, neighbouring lanes' words side by side.  Rotated lanes (16 j <
// rotary_dim) own pairs: with split halves feature i of the lane's first eight pairs
// with i of its last eight, interleaved 2i with 2i + 1.
template <typename T, int LAYOUT>
struct NormPart {
    static constexpr int N = (int)sizeof(T), V = Elt<T>::V;
    int32_t first, step, second;               // word n lies at first + n step; with split halves
    bool rot;                                  // words N / 2 .. at second + (n - N / 2) step
    __device__ __forceinline__ NormPart(int j, int32_t D, int32_t rotary_dim)
    {
        const int32_t lanes = rotary_dim / 16;
        rot = j < lanes;
        step = (rot ? lanes : D / 16 - lanes) * V;
        first = rot ? j * V : rotary_dim + (j - lanes) * V;
        second = LAYOUT == 0 && rot ? rotary_dim / 2 + first : first + N / 2 * step;
    }
    __device__ __forceinline__ int32_t at(int n) const
    {
        return n < N / 2 ? first + n * step : second + (n - N / 2) * step;
    }
};

// A lane's 16 features as eight pairs (x_i, y_i) that the rotation turns, two at a time:
// x[q] holds x_2q and x_2q+1, y[q] their partners, so everything is done on pairs of fp32
// values, half as many instructions, and alike in both layouts.  (One value at a time, the
// forward kernel issued 16 instructions an element, the backward one 26; now 10 and 17.)
struct Pairs {
    uint64_t x[4], y[4];
    // from and to the lane's features in the order of its words
    template <int LAYOUT>
    __device__ __forceinline__ void set(const float (&f)[16])
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q] = LAYOUT == 0 ? f32x2(f[2 * q], f[2 * q + 1]) : f32x2(f[4 * q], f[4 * q + 2]);
            y[q] = LAYOUT == 0 ? f32x2(f[8 + 2 * q], f[9 + 2 * q]) : f32x2(f[4 * q + 1], f[4 * q + 3]);
        }
    }
    template <int LAYOUT>
    __device__ __forceinline__ void get(float (&f)[16]) const
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x2_split(x[q], f[LAYOUT == 0 ? 2 * q : 4 * q], f[LAYOUT == 0 ? 2 * q + 1 : 4 * q + 2]);
            f32x2_split(y[q], f[LAYOUT == 0 ? 8 + 2 * q : 4 * q + 1], f[LAYOUT == 0 ? 9 + 2 * q : 4 * q + 3]);
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            x[q] = y[q] = 0;
    }
};

// Cos, sin and -sin of the eight pairs.
struct Angles {
    uint64_t c[4], s[4], n[4];
};

template <typename T>
struct RowWords {
    static constexpr int N = (int)sizeof(T), V = Elt<T>::V;
    uint4 u[N];
    template <int LAYOUT>
    __device__ __forceinline__ void store(T *row, const NormPart<T, LAYOUT> &p) const
    {
#pragma unroll
        for (int n = 0; n < N; ++n)
            __stcs(reinterpret_cast<uint4 *>(row + p.at(n)), u[n]);
    }
    template <int LAYOUT>
    __device__ __forceinline__ void unpack(Pairs &p) const
    {
        float f[16];
#pragma unroll
        for (int n = 0; n < N; ++n)
            Elt<T>::unpack(u[n], *reinterpret_cast<float(*)[V]>(f + n * V));
        p.template set<LAYOUT>(f);
    }
    template <int LAYOUT>
    __device__ __forceinline__ void pack(const Pairs &p)
    {
        float f[16];
        p.template get<LAYOUT>(f);
#pragma unroll
        for (int n = 0; n < N; ++n)
            u[n] = Elt<T>::pack(*reinterpret_cast<const float(*)[V]>(f + n * V));
    }
};

// A lane's 16 weights (ones without any), in fp32 or in the rows' type.
template <typename T, int LAYOUT>
__device__ __forceinline__ void norm_weights(const void *w, int32_t w_f32, const NormPart<T, LAYOUT> &p, bool inside, Pairs &to)
{
    constexpr int N = (int)sizeof(T), V = Elt<T>::V;
    float f[16];
    if (w == nullptr || !inside) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            f[i] = 1.0f;
    } else if (w_f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + p.at(4 * i / V) + 4 * i % V));
            f[4 * i] = t.x; f[4 * i + 1] = t.y; f[4 * i + 2] = t.z; f[4 * i + 3] = t.w;
        }
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            Elt<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + p.at(n))),
                           *reinterpret_cast<float(*)[V]>(f + n * V));
    }
    to.set<LAYOUT>(f);
}

// Cos and sin of a rotated lane's eight pairs at a table row.
template <typename T, int LAYOUT, typename Args>
__device__ __forceinline__ void norm_angles(const Args &a, int64_t row, const NormPart<T, LAYOUT> &p, Angles &to)
{
    constexpr int V = Elt<T>::V;
    float c[8], s[8];
    const int64_t at = row * (a.rotary_dim / 2);
    if constexpr (LAYOUT == 1 && V == 4) {     // two pairs a word
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 t = __ldg(reinterpret_cast<const float2 *>(a.cos + at + p.at(n) / 2));
            const float2 u = __ldg(reinterpret_cast<const float2 *>(a.sin + at + p.at(n) / 2));
            c[2 * n] = t.x; c[2 * n + 1] = t.y;
            s[2 * n] = u.x; s[2 * n + 1] = u.y;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            // pairs 4q .. 4q + 3: split halves start at their first features
            const int32_t col = LAYOUT == 0 ? p.at(4 * q / V) + 4 * q % V : p.at(q) / 2;
            const float4 t = __ldg(reinterpret_cast<const float4 *>(a.cos + at + col));
            const float4 u = __ldg(reinterpret_cast<const float4 *>(a.sin + at + col));
            c[4 * q] = t.x; c[4 * q + 1] = t.y; c[4 * q + 2] = t.z; c[4 * q + 3] = t.w;
            s[4 * q] = u.x; s[4 * q + 1] = u.y; s[4 * q + 2] = u.z; s[4 * q + 3] = u.w;
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        to.c[q] = f32x2(c[2 * q], c[2 * q + 1]);
        to.s[q] = f32x2(s[2 * q], s[2 * q + 1]);
        to.n[q] = f32x2(-s[2 * q], -s[2 * q + 1]);
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

__device__ __forceinline__ float pair_sum(uint64_t a)
{
    float lo, hi;
    f32x2_split(a, lo, hi);
    return lo + hi;
}

__device__ __forceinline__ float square_sum(const Pairs &f)
{
    uint64_t a = mul_f32x2(f.x[0], f.x[0]), b = mul_f32x2(f.y[0], f.y[0]);
#pragma unroll
    for (int q = 1; q < 4; ++q) {
        a = fma_f32x2(f.x[q], f.x[q], a);
        b = fma_f32x2(f.y[q], f.y[q], b);
    }
    return pair_sum(add_f32x2(a, b));
}

// (x, y) <- (x c - y s, x s + y c), or by the negated angles
template <bool BACK>
__device__ __forceinline__ void turn(Pairs &f, const Angles &a)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint64_t t = fma_f32x2(f.x[q], a.c[q], mul_f32x2(f.y[q], BACK ? a.s[q] : a.n[q]));
        f.y[q] = fma_f32x2(f.x[q], BACK ? a.n[q] : a.s[q], mul_f32x2(f.y[q], a.c[q]));
        f.x[q] = t;
    }
}

// 1 / sqrt(mean + eps) of a row whose squares sum to `sum`
__device__ __forceinline__ float norm_scale(float sum, float inv_d, float eps) { return rsqrtf(fmaf(sum, inv_d, eps)); }

// f r w
__device__ __forceinline__ void scale(Pairs &f, float r, const Pairs &w)
{
    const uint64_t r2 = f32x2(r, r);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f.x[q] = mul_f32x2(mul_f32x2(f.x[q], r2), w.x[q]);
        f.y[q] = mul_f32x2(mul_f32x2(f.y[q], r2), w.y[q]);
    }
}

// The table row of token (b, s), or -1: not rotated.
__device__ __forceinline__ int64_t norm_row(const NormArgs &a, int64_t b, int64_t s, bool report)
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

// ---------------------------------------------------------------------------
// Forward and backward: one kernel, a ring of stages per thread.
//
// A group of lanes owns a token and walks through its heads, U at a time, with the
// token's cos and sin in registers; a CTA's groups own neighbouring tokens.  A CTA takes
// a run of tiles (U heads of its tokens; all query heads' tiles come before the key
// heads'), from wherever the last CTA's ends, and copies its own words of the tiles to
// come into shared memory, all stages but one ahead.  A thread reads nothing but what it
// copied itself, so nothing is synchronised, and more than 100 KB are on their way to
// every SM whatever the arithmetic is at.
template <bool BACKWARD>
static constexpr int kNormCtas = BACKWARD ? 3 : 4;             // of an SM
template <bool BACKWARD>
static constexpr int kNormStages = BACKWARD ? 4 : 3;
constexpr int kNormWords = 8;                  // 16-byte words of a thread's stage
template <bool BACKWARD>
static constexpr int kNormSmem = kNormStages<BACKWARD> * kNormWords * kNormThreads * 16;

__device__ __forceinline__ void copy16(uint4 *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

// A CTA's sums of g * n for one tensor, into its row of the partial sums.
template <typename T, int LAYOUT, int L>
__device__ __forceinline__ void norm_partials(const NormArgs &a, const NormPart<T, LAYOUT> &part, const Pairs &pairs,
                                              float *to)
{
    __shared__ float sums[kNormThreads / 32][16 * L];
    constexpr int V = Elt<T>::V;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (to == nullptr)
        return;
    float acc[16];
    pairs.get<LAYOUT>(acc);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int d = L; d < 32; d <<= 1)
            acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], d);
    }
    __syncthreads();                           // the last tensor's sums are read
    if (lane < L && 16 * lane < a.D) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            sums[warp][part.at(e / V) + e % V] = acc[e];
    }
    __syncthreads();
    for (int d = tid; d < a.D; d += kNormThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kNormThreads / 32; ++i)
            sum += sums[i][d];
        to[(int64_t)blockIdx.x * a.D + d] = sum;
    }
}

// A group's way through the tiles of one tensor: head h of token (b, s).
struct NormWalk {
    int32_t b, s, h;
    // tile `tile`, of chunks of U heads a token
    __device__ __forceinline__ NormWalk(const NormArgs &a, int64_t tile, int32_t heads, int32_t U, int groups)
    {
        const int32_t chunks = (heads + U - 1) / U;
        const int64_t block = tile / chunks, t = block * groups + threadIdx.x / (kNormThreads / groups);
        h = (int32_t)(tile - block * chunks) * U;
        b = (int32_t)(t / a.S);
        s = (int32_t)(t - b * a.S);
    }
    // true: a new token
    __device__ __forceinline__ bool next(const NormArgs &a, int32_t heads, int32_t U, int groups)
    {
        h += U;
        if (h < heads)
            return false;
        h = 0;
        s += groups;
        while (s >= a.S) {                     // (once, but for sequences shorter than a CTA's tokens)
            s -= (int32_t)a.S;
            ++b;
        }
        return true;
    }
    __device__ __forceinline__ int64_t at(const int64_t (&st)[3]) const
    {
        return b * st[0] + s * st[1] + h * st[2];
    }
};

// The tiles first .. first + n - 1 of tensor x, through the ring.  Backward adds its rows'
// g * n to acc.
template <typename T, int LAYOUT, int L, bool BACKWARD>
__device__ __forceinline__ void norm_run(const NormArgs &a, const NormTensor &x, int64_t first, int32_t n,
                                         const NormPart<T, LAYOUT> &part, uint4 *ring, Pairs &acc)
{
    constexpr int N = (int)sizeof(T), kGroups = kNormThreads / L;
    constexpr int kStages = kNormStages<BACKWARD>, kWords = kNormWords, U = kWords / N / (BACKWARD ? 2 : 1);
    const int j = threadIdx.x % L;
    const bool inside = 16 * j < a.D;
    const int32_t heads = x.heads;
    const T *px = static_cast<const T *>(x.x), *pg = static_cast<const T *>(x.g);
    T *py = static_cast<T *>(x.y);
    NormWalk in(a, first, heads, U, kGroups), out = in;        // the tile copied next, the tile computed next
    const T *src = px + in.at(x.xs), *up = BACKWARD ? pg + in.at(x.ys) : nullptr;
    T *dst = py + out.at(x.ys);
    int32_t to_copy = n;
    auto copy = [&](uint4 *to) {
        if (--to_copy >= 0) {
            if (in.b < a.B && inside) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (in.h + i < heads) {
#pragma unroll
                        for (int w = 0; w < N; ++w) {
                            copy16(to + (i * N + w) * kNormThreads, src + i * x.xs[2] + part.at(w));
                            if constexpr (BACKWARD)
                                copy16(to + ((U + i) * N + w) * kNormThreads, up + i * x.ys[2] + part.at(w));
                        }
                    }
                }
            }
            src += U * x.xs[2];
            if constexpr (BACKWARD)
                up += U * x.ys[2];
            if (in.next(a, heads, U, kGroups)) {
                src = px + in.at(x.xs);
                if constexpr (BACKWARD)
                    up = pg + in.at(x.ys);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    constexpr int kStage = kWords * kNormThreads;
    uint4 *const end = ring + kStages * kStage;
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st)
        copy(ring + st * kStage);
    uint4 *now = ring, *free = end - kStage;   // the stage computed next, the one that the last step has read
    Pairs w;
    Angles angles;
    norm_weights(x.w, a.w_f32, part, inside, w);
    bool rot = false, fresh = true;            // fresh: a new token
    for (; n > 0; --n) {
        const bool live = inside && out.b < a.B;
        if (fresh) {
            const int64_t row = live ? norm_row(a, out.b, out.s, j == 0) : -1;
            rot = part.rot && row >= 0;
            if (rot)
                norm_angles(a, row, part, angles);
        }
        copy(free);
        free = now;
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        // (what a row past the heads or tokens holds is computed, too, and goes nowhere)
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool on = live && out.h + i < heads;
            RowWords<T> v;
            Pairs f, g;
#pragma unroll
            for (int k = 0; k < N; ++k)
                v.u[k] = now[(i * N + k) * kNormThreads];
            v.template unpack<LAYOUT>(f);
            float sum = square_sum(f), dot = 0.0f;
            if constexpr (BACKWARD) {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    v.u[k] = now[((U + i) * N + k) * kNormThreads];
                v.template unpack<LAYOUT>(g);
                if (rot)
                    turn<true>(g, angles);
                uint64_t d0 = 0, d1 = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    d0 = fma_f32x2(mul_f32x2(g.x[q], f.x[q]), w.x[q], d0);
                    d1 = fma_f32x2(mul_f32x2(g.y[q], f.y[q]), w.y[q], d1);
                }
                dot = pair_sum(add_f32x2(d0, d1));
            }
            if (!inside)
                sum = dot = 0.0f;
            const float r = norm_scale(group_sum<L>(sum), a.inv_d, a.eps);
            if constexpr (BACKWARD) {
                // r mean(w g n) n = r^3 mean(w g x) x  (one r at a time: mean(w g x) r is of the
                // size of w g, where r^3 alone leaves fp32's range for rows of 10^13)
                const float m = group_sum<L>(dot) * a.inv_d * r * r * r;
                const uint64_t r2 = f32x2(r, r), m2 = f32x2(-m, -m);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (on) {
                        acc.x[q] = fma_f32x2(mul_f32x2(g.x[q], f.x[q]), r2, acc.x[q]);
                        acc.y[q] = fma_f32x2(mul_f32x2(g.y[q], f.y[q]), r2, acc.y[q]);
                    }
                    f.x[q] = fma_f32x2(mul_f32x2(g.x[q], w.x[q]), r2, mul_f32x2(f.x[q], m2));
                    f.y[q] = fma_f32x2(mul_f32x2(g.y[q], w.y[q]), r2, mul_f32x2(f.y[q], m2));
                }
            } else {
                scale(f, r, w);
                if (rot)
                    turn<false>(f, angles);
            }
            v.template pack<LAYOUT>(f);
            if (on)
                v.store(dst + i * x.ys[2], part);
        }
        now = now + kStage == end ? ring : now + kStage;
        dst += U * x.ys[2];
        fresh = out.next(a, heads, U, kGroups);
        if (fresh)
            dst = py + out.at(x.ys);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Backward keeps a thread's sums of g * n in registers; a CTA leaves one row of D partial
// sums per tensor, which rope_norm_weights_kernel adds up in a fixed order (no atomics: the
// same call gives the same bits).
template <typename T, int LAYOUT, int L, bool BACKWARD>
__global__ void __launch_bounds__(kNormThreads, kNormCtas<BACKWARD>) rope_norm_kernel(const NormArgs a)
{
    extern __shared__ __align__(16) uint4 ring[];
    const NormPart<T, LAYOUT> part(threadIdx.x % L, a.D, a.rotary_dim);
    // this CTA's run of the tiles, the query heads' first
    const int64_t tiles = a.tiles[0] + a.tiles[1];
    const int64_t first = tiles * blockIdx.x / gridDim.x, last = tiles * (blockIdx.x + 1) / gridDim.x;
    pdl_wait();
    pdl_trigger();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const int64_t base = k ? a.tiles[0] : 0, end = base + a.tiles[k];
        const int64_t from = first > base ? first : base, to = last < end ? last : end;
        Pairs acc;
        acc.zero();
        if (from < to)
            norm_run<T, LAYOUT, L, BACKWARD>(a, a.t[k], from - base, (int32_t)(to - from), part, ring + threadIdx.x, acc);
        if constexpr (BACKWARD)
            norm_partials<T, LAYOUT, L>(a, part, acc, a.t[k].partial);
    }
}

// dw: the sum of the CTAs' rows.  A cluster sums 32 features of one tensor, a run of rows
// for each of its 256 warps, in a fixed order: bound by the latency of a few loads one after
// the other, so as many warps as a cluster has share them (1368 rows: the backward call of 16k
// tokens 87.3 us with one CTA, 86.4 so; 12000 tokens of 20 heads of 96, 33.8 and 32.6).
constexpr int kNormSumWarps = 32, kNormSumCtas = 8;
template <typename T>
__global__ void __cluster_dims__(kNormSumCtas, 1, 1) __launch_bounds__(32 * kNormSumWarps)
    rope_norm_weights_kernel(const NormArgs a, const int32_t rows)
{
    __shared__ float run[kNormSumWarps][33], part[32];
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const NormTensor &x = a.t[blockIdx.y];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)cluster.block_rank();
    const int first = blockIdx.x / kNormSumCtas * 32, d = first + lane;
    pdl_wait();
    pdl_trigger();
    if (x.partial == nullptr)                  // (all of the cluster alike)
        return;
    float sum = 0.0f;
    if (d < a.D) {
#pragma unroll 8
        for (int i = rank * kNormSumWarps + warp; i < rows; i += kNormSumCtas * kNormSumWarps)
            sum += __ldcg(x.partial + (int64_t)i * a.D + d);
    }
    run[warp][lane] = sum;
    __syncthreads();
    // warp w: feature w
    sum = run[lane][warp];
#pragma unroll
    for (int i = 16; i > 0; i >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, i);
    if (lane == 0)
        part[warp] = sum;
    cluster.sync();
    if (rank == 0 && warp == 0 && d < a.D) {
        sum = part[lane];
#pragma unroll
        for (int r = 1; r < kNormSumCtas; ++r)
            sum += *cluster.map_shared_rank(&part[lane], r);
        if (a.w_f32)
            static_cast<float *>(x.dw)[d] = sum;
        else
            static_cast<T *>(x.dw)[d] = Elt<T>::from_f(sum);
    }
    cluster.sync();                            // the others' sums are read
}

// ---------------------------------------------------------------------------
// Into a paged cache: queries to a dense tensor, keys (the same arithmetic) and
// values to their sequence's pages.  A unit is U heads of one kind of a token;
// which sequence the token belongs to, its page and its table row are looked up
// while the unit's loads are on their way, as in rope_cache_append_kernel.
constexpr int kNormCuCached = 1024;            // sequence offsets kept in shared memory
constexpr int kNormAppendHeads = 4;            // heads of a token that a group has in flight

template <typename T, int LAYOUT, int D>
__global__ void __launch_bounds__(kNormThreads) rope_norm_append_kernel(const NormAppendArgs a)
{
    constexpr int L = D / 16, U = kNormAppendHeads, N = (int)sizeof(T), kGroups = kNormThreads / L;
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
    const NormPart<T, LAYOUT> part(j, D, r.rotary_dim);

    pdl_wait();
    pdl_trigger();
    RowWords<T> v[U];
    const T *src = kind == 0 ? static_cast<const T *>(a.q) + t * a.q_stride
                             : (kind == 1 ? static_cast<const T *>(r.k) + t * r.k_stride
                                          : static_cast<const T *>(r.v) + t * r.v_stride);
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (live && h0 + i < heads) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                v[i].u[n] = __ldcs(reinterpret_cast<const uint4 *>(src + (h0 + i) * D + part.at(n)));
        }
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
    Pairs w;
    Angles angles;
    const bool rot = part.rot && row >= 0;
    if (write && kind < 2)
        norm_weights(kind == 0 ? a.wq : a.wk, a.w_f32, part, true, w);
    if (rot)
        norm_angles(r, row, part, angles);
    const int64_t in_page = slot & (((int64_t)1 << r.page_shift) - 1);
    T *dst = kind == 0 ? static_cast<T *>(a.q_out) + (t * a.Hq + h0) * D
                       : static_cast<T *>(kind == 1 ? r.k_out : r.v_out) +
                             (((page * r.Hk + h0) << r.page_shift) + in_page) * D;
    const int64_t step = kind == 0 ? D : (int64_t)D << r.page_shift;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const bool on = write && h0 + i < heads;
        Pairs f;
        float sum = 0.0f;
        if (on && kind < 2) {
            v[i].template unpack<LAYOUT>(f);
            sum = square_sum(f);
        }
        const float q = norm_scale(group_sum<L>(sum), 1.0f / D, a.eps);
        if (on && kind < 2) {
            scale(f, q, w);
            if (rot)
                turn<false>(f, angles);
            v[i].template pack<LAYOUT>(f);
        }
        if (on)
            v[i].store(dst + i * step, part);
    }
}

// ---------------------------------------------------------------------------
// host side
template <typename T, int LAYOUT, int L, bool BACKWARD>
static cudaError_t launch_norm_lanes(NormArgs a, cudaStream_t st)
{
    constexpr int64_t groups = kNormThreads / L, U = kNormWords / (int)sizeof(T) / (BACKWARD ? 2 : 1);
    for (int k = 0; k < 2; ++k)
        a.tiles[k] = (a.tokens + groups - 1) / groups * ((a.t[k].heads + U - 1) / U);
    const int64_t tiles = a.tiles[0] + a.tiles[1];
    if (tiles > (1ll << 38))                   // (a run, of a CTA of hundreds, has to fit 32 bits)
        return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> raised{0};
    auto *kernel = rope_norm_kernel<T, LAYOUT, L, BACKWARD>;
    int sms = 0, dev = 0;
    cudaError_t e = sm_count(&sms, &dev);
    if (e == cudaSuccess)
        e = raise_smem(reinterpret_cast<const void *>(kernel), kNormSmem<BACKWARD>, dev, raised);
    if (e != cudaSuccess)
        return e;
    // The CTAs that are resident at once, or twice or three times as many where that leaves
    // runs of some length: the hardware hands them out as others end, which evens out what the
    // SMs and their way to memory take.  Once, twice, three times (us; forward, then backward,
    // 40 heads of 128 unless said): 16k tokens 62.1, 59.1, 56.0 and 96.5, 93.2, 88.3; 8k 30.5, 29.4,
    // 29.6 and 48.0, 47.6, 50.4; 4k 14.2, 16.0, 16.0 and 26.5, 30.0, 32.6; 64k of ten heads 69.6, 65.7,
    // 65.9 and 110, 98, 97; 12000 of 20 heads of 96 18.8, 20.6, 21.2 and 33.6, 36.5, 39.6; 24000 37.6,
    // 36.9, 38.2 and 59.4, 61.1, 61.7; 30000 of 16 heads of 64 20.5, 23.8, 24.5 and 37.3, 40.7, 43.9;
    // 16k of 32 heads of 64 in fp32 46.7, 45.1, 44.0 and 70 each.  The limits below pick within 3 % of
    // the best of each; 8k of 20 heads of 256 are the exception (forward 32.2, 30.7, 30.1: once).
    const int64_t resident = kNormCtas<BACKWARD> * (int64_t)sms;
    int64_t waves = tiles / ((BACKWARD ? 12 : 5) * resident);
    waves = waves < 1 ? 1 : waves > 3 ? 3 : waves;
    int64_t most = waves * resident;
    if (BACKWARD && most > kNormPartials)
        most = kNormPartials;
    // (without rows the sums are zeros)
    const int32_t grid = (int32_t)(tiles < 1 ? 1 : tiles < most ? tiles : most);
    e = launch_hot(kernel, dim3((unsigned)grid), dim3(kNormThreads), (size_t)kNormSmem<BACKWARD>, st, a);
    if (e != cudaSuccess || (a.t[0].partial == nullptr && a.t[1].partial == nullptr))
        return e;
    return launch_hot(rope_norm_weights_kernel<T>, dim3((unsigned)(a.D + 31) / 32 * kNormSumCtas, 2),
                      dim3(32 * kNormSumWarps), 0, st, a, grid);
}

template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, int32_t layout, bool backward, cudaStream_t st)
{
    const int lanes = a.D / 16;
#define ROPE_NORM(L)                                                                                        \
    (layout == 0 ? backward ? launch_norm_lanes<T, 0, L, true>(a, st) : launch_norm_lanes<T, 0, L, false>(a, st) \
                 : backward ? launch_norm_lanes<T, 1, L, true>(a, st) : launch_norm_lanes<T, 1, L, false>(a, st))
    return lanes <= 2 ? ROPE_NORM(2) : lanes <= 4 ? ROPE_NORM(4) : lanes <= 8 ? ROPE_NORM(8) : ROPE_NORM(16);
#undef ROPE_NORM
}

template <typename T, int LAYOUT, int D>
static cudaError_t launch_norm_append_t(const NormAppendArgs &a, cudaStream_t st)
{
    constexpr int64_t U = kNormAppendHeads, groups = kNormThreads / (D / 16);
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
