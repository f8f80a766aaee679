// rope_checks.h -- argument checks shared by the C entry points of the serving
// and norm calls (host code).
#pragma once

#include <cstdint>
#include <initializer_list>

#include "rope.h"

namespace rope {

struct Range {
    const void *p;
    int64_t bytes;
};

inline bool overlap(const Range &a, const Range &b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a * b * ... of non-negative sizes, or -1 on overflow (or a -1 among them)
inline int64_t product(std::initializer_list<int64_t> xs)
{
    int64_t r = 1;
    for (int64_t x : xs)
        if (r < 0 || x < 0 || __builtin_mul_overflow(r, x, &r))
            return -1;
    return r;
}

// Bytes from the first to the last element of a [total, H, D] view with the
// given token stride, 16-bit elements; -1 on overflow.
inline int64_t view_bytes(int64_t total, int64_t stride, int64_t row)
{
    if (total == 0)
        return 0;
    const int64_t lead = product({total - 1, stride});
    int64_t n = 0;
    if (lead < 0 || row < 0 || __builtin_add_overflow(lead, row, &n))
        return -1;
    return product({n, 2});
}

inline rope_status check_shape(int32_t dtype, int32_t layout, int32_t D, int32_t rotary_dim)
{
    if (dtype != ROPE_BF16 && dtype != ROPE_F16)
        return ROPE_ERR_UNSUPPORTED;
    if (layout != ROPE_SPLIT_HALF && layout != ROPE_INTERLEAVED)
        return ROPE_ERR_UNSUPPORTED;
    if (D != 64 && D != 128)
        return ROPE_ERR_UNSUPPORTED;
    if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 != 0)
        return ROPE_ERR_UNSUPPORTED;
    return ROPE_OK;
}

// log2 of a supported page size, else -1
inline int32_t page_shift(int32_t page_size)
{
    for (int32_t s = 4; s <= 7; ++s)
        if (page_size == 1 << s)
            return s;
    return -1;
}

constexpr int64_t kMaxInt32 = 0x7fffffff;

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace rope
