// rope_tables_scaled.cu -- cos/sin tables of contexts longer than those a
// model was trained on (rope_tables_build_scaled).
//
// Every rule gives pair i a frequency w_i; the table holds cos and sin of p w_i
// for the integer positions p = pos_offset + row.  In turns, p w_i / 2 pi modulo 1
// is all that matters, so the frequency is kept as a fixed-point fraction of a
// turn, F_i = round(w_i / 2 pi * 2^64), and the phase is p * F_i modulo 2^64: one
// 64-bit integer product is the whole range reduction, exact but for F_i's own
// rounding (p 2^-65 turns: 2e-11 radians at a position of 10^8).  A double has 53 bits
// of F_i's 62, and a w_i from pow is off by more (pair 1 at theta 5e5: 704 times 2^-65
// turns a position, 2.6e-7 radians at the last one), so the host computes the
// frequencies with twice as many (Wide).  The nearest
// quarter turn comes off the top two bits, and what is left, at most an eighth of
// a turn either way, goes to fp32 (two roundings of 2^-24) and to the series of sine
// and cosine.  The frequencies go along as kernel arguments: computed in every CTA they
// would cost more than the table.
//
// Off by, at most: p 2^-65 turns for F_i; 2^-57 turns for a rest just below zero, whose two
// parts are rounded before they cancel; and, in units u = 2^-24 of a sine (of a cosine): 2
// (1.6) for the rest's two roundings, 1 (0.7) for the series' last sum, 0.8 (1.1) for what
// comes before it, 0.1 for its end, 2 for the factor's rounding and its product: less than 6.
//
// What bounds it: 8 bytes a pair against some 50 instructions, at 64 pairs a
// row about even: 131072 rows of 64 pairs write 67 MB.  Angles and sincos in 64
// bits (rope_tables_build_ex) would be some 100 64-bit operations a pair, of
// which this GPU does a 64th of its 32-bit ones.
//
// A thread owns four pairs of a row (two 16-byte stores) and keeps their F in
// registers while it walks down the rows.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "rope.h"
#include "rope_checks.h"
#include "rope_f32x2.cuh"
#include "rope_kernels.cuh"

namespace rope {
namespace {

constexpr int kScaledPairs = 256;              // pairs of a row at most
constexpr int kScaledThreads = 256;

struct ScaledArgs {
    uint64_t freq[kScaledPairs];               // fractions of a turn, times 2^64
    float *cos, *sin;
    int64_t rows;
    uint64_t first;                            // position of row 0
    int32_t h;
    float scale;
};

// Cos and sin of two phases, times scale.  Each leaves its nearest quarter turn as a rest of
// at most an eighth of a turn; with y its angle, at most pi / 4, Taylor's series to y^9 and
// y^10 are within 2^-28 of sin y and cos y.  The rounding of y's product with 2 pi goes along
// as `low`, so y is as good as the rest in fp32.
__device__ __forceinline__ void phase_cos_sin(const uint64_t (&phase)[2], float scale, float (&c)[2], float (&s)[2])
{
    uint32_t quarter[2];
    float rest[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t top = (uint32_t)(phase[i] >> 32);
        quarter[i] = (top + 0x20000000u) >> 30;
        rest[i] = fmaf((float)(int32_t)(top - (quarter[i] << 30)), 4294967296.0f, (float)(uint32_t)phase[i]);
    }
    auto both = [](float x) { return f32x2(x, x); };
    constexpr double kTurn = 6.283185307179586477 / 18446744073709551616.0;    // 2 pi / 2^64
    const uint64_t r = f32x2(rest[0], rest[1]), k = both((float)kTurn);
    const uint64_t y = mul_f32x2(r, k);
    const uint64_t low = fma_f32x2(r, both((float)(kTurn - (double)(float)kTurn)),
                                   fma_f32x2(r, k, y ^ 0x8000000080000000ull));
    const uint64_t z = fma_f32x2(add_f32x2(low, low), y, mul_f32x2(y, y));
    uint64_t a = fma_f32x2(z, both(-1.0f / 3628800.0f), both(1.0f / 40320.0f));
    a = fma_f32x2(a, z, both(-1.0f / 720.0f));
    a = fma_f32x2(a, z, both(1.0f / 24.0f));
    a = fma_f32x2(a, z, both(-0.5f));
    a = fma_f32x2(a, z, both(1.0f));
    uint64_t b = fma_f32x2(z, both(1.0f / 362880.0f), both(-1.0f / 5040.0f));
    b = fma_f32x2(b, z, both(1.0f / 120.0f));
    b = fma_f32x2(b, z, both(-1.0f / 6.0f));
    b = add_f32x2(y, fma_f32x2(b, mul_f32x2(y, z), low));
    float x[2], w[2];
    f32x2_split(mul_f32x2(a, both(scale)), x[0], x[1]);
    f32x2_split(mul_f32x2(b, both(scale)), w[0], w[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {              // (cos, sin) of y + quarter * pi / 2
        const bool swap = quarter[i] & 1;
        c[i] = __uint_as_float(__float_as_uint(swap ? w[i] : x[i]) ^ ((quarter[i] + 1) & 2) << 30);
        s[i] = __uint_as_float(__float_as_uint(swap ? x[i] : w[i]) ^ (quarter[i] & 2) << 30);
    }
}

// V: pairs of a thread, 4 where rows are whole 16-byte vectors, else 1.
template <int V>
__global__ void __launch_bounds__(kScaledThreads) rope_tables_scaled_kernel(const __grid_constant__ ScaledArgs a)
{
    const int32_t per_row = a.h / V;           // threads of a row
    const int64_t threads = (int64_t)gridDim.x * kScaledThreads;
    const int64_t at = (int64_t)blockIdx.x * kScaledThreads + threadIdx.x;
    int64_t row = at / per_row;
    const int32_t col = (int32_t)(at - row * per_row) * V;
    const int64_t step = threads / per_row;    // rows the grid takes at once
    if (row >= step)
        return;                                // the grid's last threads, less than a row of them
    uint64_t f[V], phase[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f[i] = a.freq[col + i];
        phase[i] = f[i] * (a.first + (uint64_t)row);
        f[i] *= (uint64_t)step;
    }
    pdl_wait();
    pdl_trigger();
    for (; row < a.rows; row += step) {
        float c[V], s[V];
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const int n = V > 1 ? i + 1 : i;   // (alone: the same twice)
            const uint64_t two[2] = {phase[i], phase[n]};
            float c2[2], s2[2];
            phase_cos_sin(two, a.scale, c2, s2);
            c[i] = c2[0]; c[n] = c2[V > 1];
            s[i] = s2[0]; s[n] = s2[V > 1];
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            phase[i] += f[i];
        if constexpr (V == 4) {
            *reinterpret_cast<float4 *>(a.cos + row * a.h + col) = make_float4(c[0], c[1], c[2], c[3]);
            *reinterpret_cast<float4 *>(a.sin + row * a.h + col) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            a.cos[row * a.h + col] = c[0];
            a.sin[row * a.h + col] = s[0];
        }
    }
}

// Numbers of twice 53 bits: hi + lo, lo at most half a unit of hi.
struct Wide {
    double hi, lo;
};

Wide sum_of(double a, double b)                // exact
{
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}

Wide product_of(double a, double b)            // exact
{
    // (a * b, but no compiler fuses it into a later sum, where its rounding would be lost)
    const double p = std::fma(a, b, 0.0);
    return {p, std::fma(a, b, -p)};
}

// Off by some 2^-104 of the result (the sum: of the larger term).
Wide operator+(Wide a, Wide b)
{
    const Wide s = sum_of(a.hi, b.hi);
    return sum_of(s.hi, s.lo + (a.lo + b.lo));
}
Wide operator-(Wide a, Wide b) { return a + Wide{-b.hi, -b.lo}; }
Wide operator*(Wide a, Wide b)
{
    const Wide p = product_of(a.hi, b.hi);
    return sum_of(p.hi, p.lo + std::fma(a.hi, b.lo, a.lo * b.hi));
}
Wide operator/(Wide a, Wide b)
{
    const double q = a.hi / b.hi;
    const Wide rest = a - b * Wide{q, 0.0};
    return sum_of(q, rest.hi / b.hi);
}

constexpr Wide kOne = {1.0, 0.0};
// 1 / 2 pi: the nearest double, and the nearest to what that leaves
constexpr Wide kPerTurn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};

Wide power(Wide x, int32_t n)                  // x^n, n >= 1
{
    int32_t bit = 1;
    while (bit <= n / 2)
        bit *= 2;
    Wide y = x;
    while ((bit /= 2) > 0) {
        y = y * y;
        if (n & bit)
            y = y * x;
    }
    return y;
}

// x^(-1 / n): a double's power and a step of Newton's method on x y^n = 1
Wide root(double x, int32_t n)
{
    const Wide y = {std::pow(x, -1.0 / n), 0.0};
    return y + y * ((kOne - Wide{x, 0.0} * power(y, n)) / Wide{(double)n, 0.0});
}

// x w, for a weight that goes from `below` at a <= 0 to `above` at a >= span.
Wide ramp(Wide x, Wide a, Wide span, Wide below, Wide above)
{
    if (a.hi <= 0.0)
        return x * below;
    return (a - span).hi >= 0.0 ? x * above : x * (below + a / span * (above - below));
}

// Every pair's turn per position, as a fraction of a turn times 2^64; the factor of all values.
void scaled_frequencies(int32_t kind, double theta, int32_t rd, double factor, int64_t original, double low, double high,
                        uint64_t *freq, double *scale)
{
    const double pi = 3.14159265358979323846;
    const int32_t h = rd / 2;
    double ramp0 = 0.0, ramp1 = 0.0;
    *scale = 1.0;
    if (kind == ROPE_SCALE_YARN) {
        // the pair that makes r turns over the trained context
        auto pair_of = [&](double r) { return rd * std::log((double)original / (r * 2.0 * pi)) / (2.0 * std::log(theta)); };
        ramp0 = std::fmax(std::floor(pair_of(high)), 0.0);
        ramp1 = std::fmin(std::ceil(pair_of(low)), (double)rd - 1.0);
        if (factor > 1.0)
            *scale = 0.1 * std::log(factor) + 1.0;
    }
    Wide ratio = root(theta, h);               // w_i+1 / w_i = theta^(-2 / rd)
    if (kind == ROPE_SCALE_NTK)                // f^(rd / (rd - 2))^(-2 / rd)
        ratio = ratio * root(factor, h - 1);
    const Wide slower = kOne / Wide{factor, 0.0}, trained = Wide{(double)original, 0.0} * kPerTurn, twice = ratio * ratio;
    Wide w[2] = {kOne, ratio};                 // of the next even pair, of the next odd one
    for (int32_t i = 0; i < h; ++i) {
        Wide x = w[i & 1];
        w[i & 1] = x * twice;
        if (kind == ROPE_SCALE_LINEAR)
            x = x * slower;
        else if (kind == ROPE_SCALE_SMOOTH)
            x = ramp(x, trained * x - Wide{low, 0.0}, sum_of(high, -low), slower, kOne);
        else if (kind == ROPE_SCALE_YARN)
            x = ramp(x, {(double)i - ramp0, 0.0}, {ramp1 > ramp0 ? ramp1 - ramp0 : 0.001, 0.0}, kOne, slower);
        // at most 1 / 2 pi of a turn; rounded once, behind hi's whole part
        const Wide turn = x * kPerTurn;
        const double hi = turn.hi * 0x1p64;
        const uint64_t whole = (uint64_t)hi;
        freq[i] = whole + (uint64_t)(int64_t)std::nearbyint(hi - (double)whole + turn.lo * 0x1p64);
    }
}

}  // namespace
}  // namespace rope

using namespace rope;

extern "C" rope_status rope_tables_build_scaled(int32_t kind, double theta, int32_t rotary_dim, int64_t rows,
                                                int64_t pos_offset, double factor, int64_t original_positions,
                                                double low_turns, double high_turns, double value_scale,
                                                float *cos_out, float *sin_out, void *stream)
{
    if (kind != ROPE_SCALE_LINEAR && kind != ROPE_SCALE_NTK && kind != ROPE_SCALE_SMOOTH && kind != ROPE_SCALE_YARN)
        return ROPE_ERR_UNSUPPORTED;
    if (rotary_dim > 2 * kScaledPairs)
        return ROPE_ERR_UNSUPPORTED;
    if (rotary_dim < 2 || (rotary_dim & 1) || (kind == ROPE_SCALE_NTK && rotary_dim == 2) || rows < 0 || pos_offset < 0 ||
        pos_offset > kMaxInt32 || rows > kMaxInt32 - pos_offset)
        return ROPE_ERR_INVALID_ARG;
    // (below 1 a frequency may pass a turn a position, which the fraction does not hold)
    if (!(theta > 1.0) || !std::isfinite(theta) || !(factor >= 1.0) || !std::isfinite(factor) || !std::isfinite(value_scale) ||
        value_scale < 0.0)
        return ROPE_ERR_INVALID_ARG;
    const bool turns = kind == ROPE_SCALE_SMOOTH || kind == ROPE_SCALE_YARN;
    if (turns && (original_positions < 1 || !(low_turns > 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns)))
        return ROPE_ERR_INVALID_ARG;
    if (rows == 0)
        return ROPE_OK;
    const int32_t h = rotary_dim / 2;
    const int64_t bytes = rows * h * 4;
    if (cos_out == nullptr || sin_out == nullptr || overlap({cos_out, bytes}, {sin_out, bytes}) || !aligned(cos_out, 4) ||
        !aligned(sin_out, 4))
        return ROPE_ERR_INVALID_ARG;
    ScaledArgs a;
    double scale;
    scaled_frequencies(kind, theta, rotary_dim, factor, original_positions, low_turns, high_turns, a.freq, &scale);
    for (int32_t i = h; i < kScaledPairs; ++i)
        a.freq[i] = 0;
    a.cos = cos_out; a.sin = sin_out; a.rows = rows; a.first = (uint64_t)pos_offset; a.h = h;
    a.scale = (float)(value_scale > 0.0 ? value_scale : scale);
    const bool wide = h % 4 == 0 && aligned(cos_out, 16) && aligned(sin_out, 16);
    const int64_t threads = rows * (wide ? h / 4 : h);
    int64_t blocks = (threads + kScaledThreads - 1) / kScaledThreads;
    // a few rows a thread for long tables: its frequencies are read once
    const int64_t most = 152 * 8;
    if (blocks > most)
        blocks = most;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        wide ? launch_hot(rope_tables_scaled_kernel<4>, dim3((unsigned)blocks), dim3(kScaledThreads), 0, st, a)
             : launch_hot(rope_tables_scaled_kernel<1>, dim3((unsigned)blocks), dim3(kScaledThreads), 0, st, a);
    return e == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA;
}
