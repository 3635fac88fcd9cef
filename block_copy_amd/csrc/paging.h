// paging.h -- where a token of a sequence lives in the pages: integer
// arithmetic shared by the host (argument checks) and the kernels, free of
// HIP so that a CPU build can test it.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define KVC_HD __host__ __device__ __forceinline__
#else
#define KVC_HD inline
#endif

namespace kvc {

// Division of n < 2^31 by a fixed d in 1 .. 2^31 - 1 with one 64-bit product:
// with 2^s >= d and M = ceil(2^(31 + s) / d), M * d exceeds 2^(31 + s) by
// less than d <= 2^s, so floor(n * M / 2^(31 + s)) = floor(n / d) for every
// n < 2^31.  M <= 2^32 - 1 holds since d > 2^(s - 1).
struct Divider {
    uint32_t mul, shift, d;
    KVC_HD uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
    KVC_HD uint32_t mod(uint32_t n, uint32_t q) const { return n - q * d; }
};

inline Divider make_divider(uint32_t d)
{
    uint32_t s = 0;
    while ((1ull << s) < d)
        ++s;
    const uint64_t one = 1ull << (31 + s);
    return Divider{(uint32_t)((one + d - 1) / d), 31 + s, d};
}

// Element offset of (page, place) for one head; the head's own offset is
// added to the base pointer once.
KVC_HD int64_t page_offset(uint32_t page, uint32_t place, int64_t page_stride, int64_t place_stride)
{
    return (int64_t)page * page_stride + (int64_t)place * place_stride;
}

// A slot as the caller gives it: -1 for one to leave out (negative), -2 for
// one beyond the pages, else the slot as 32 bits.
KVC_HD int32_t checked_slot(int64_t slot, uint32_t num_slots)
{
    if (slot < 0)
        return -1;
    return slot < (int64_t)num_slots ? (int32_t)slot : -2;
}

// The first key that a row at `position` may see.  No difference is taken that
// could leave 31 bits: a window may be as large as an int32_t, and a position
// lies before the first key where a sequence has fewer keys than rows.
KVC_HD int32_t first_seen(int32_t position, int32_t window)
{
    return window > 0 && position >= window ? position - window + 1 : 0;
}

// The keys a block of query rows has to look at: rows stand at positions
// first .. last, see keys <= their position and, with a window, > position -
// window; the cache holds `bound` tokens.  [lo, hi) is empty if lo >= hi.
struct KeyRange {
    int32_t lo, hi;
};
KVC_HD KeyRange key_range(int32_t first, int32_t last, int32_t window, int32_t bound)
{
    KeyRange r;
    r.hi = last + 1 < bound ? last + 1 : bound;
    r.lo = first_seen(first, window);
    return r;
}

// Split `split` of such a range: keys base + split * keys .. + keys - 1 of it.
KVC_HD KeyRange split_range(KeyRange r, int32_t base, uint32_t split, uint32_t keys)
{
    const int64_t from = base + (int64_t)split * keys, to = from + keys;
    r.lo = from > r.lo ? (int32_t)(from < r.hi ? from : r.hi) : r.lo;
    r.hi = to < r.hi ? (int32_t)to : r.hi;
    return r;
}

}  // namespace kvc
