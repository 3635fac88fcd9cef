// Checks csrc/paging.h against plain arithmetic: division by every small and
// many large page sizes at the ends of quotients' ranges, slots in and out of
// range, and the key range of blocks of rows against a scan.
#include <stdio.h>
#include <stdlib.h>

#include "paging.h"

static void fail(const char *what, long long a, long long b)
{
    printf("%s: %lld %lld\n", what, a, b);
    exit(1);
}

static void check(const kvc::Divider &v, uint32_t d, uint32_t n)
{
    const uint32_t q = v.div(n);
    if (q != n / d || v.mod(n, q) != n % d)
        fail("division", n, d);
}

int main()
{
    const uint32_t top = (1u << 31) - 1;
    uint64_t seed = 7;
    for (uint32_t i = 1; i < 40000; ++i) {
        seed = seed * 6364136223846793005ull + 1442695040888963407ull;
        const uint32_t d = i < 20000 ? i : 1 + (uint32_t)(seed >> 33) % top;
        const kvc::Divider v = kvc::make_divider(d);
        check(v, d, 0);
        check(v, d, top);
        for (uint64_t m = 1; m < 40; ++m) {
            seed = seed * 6364136223846793005ull + 1442695040888963407ull;
            const uint64_t q = m < 20 ? m : (seed >> 33) % (top / d + 1);
            for (int e = -1; e <= 1; ++e) {
                const uint64_t n = q * d + e;
                if (n <= top)
                    check(v, d, (uint32_t)n);
            }
        }
    }
    const int64_t big = INT64_MAX, small = INT64_MIN;
    const struct { int64_t s; uint32_t n; int32_t want; } slots[] = {
        {0, 1, 0}, {1, 1, -2}, {-1, 1, -1}, {small, 5, -1}, {big, 5, -2}, {4, 5, 4}, {5, 5, -2},
        {1ll << 32, top, -2}, {(1ll << 32) + 1, top, -2}, {top - 1, top, (int32_t)(top - 1)}};
    for (const auto &t : slots)
        if (kvc::checked_slot(t.s, t.n) != t.want)
            fail("slot", t.s, t.n);
    if (kvc::page_offset(3, 5, 1ll << 40, -7) != 3 * (1ll << 40) - 35)
        fail("offset", 0, 0);
    for (int ctx = 0; ctx < 12; ++ctx)
        for (int n = 1; n < 9; ++n)
            for (int w = 0; w < 6; ++w)
                for (int r0 = 0; r0 < n; ++r0)
                    for (int r1 = r0; r1 < n; ++r1) {
                        const int first = ctx - n + r0, last = ctx - n + r1;
                        const kvc::KeyRange k = kvc::key_range(first, last, w, ctx);
                        // every key some row sees is inside, and none is outside the cache
                        for (int r = r0; r <= r1; ++r)
                            for (int t = 0; t < ctx; ++t) {
                                const int p = ctx - n + r;
                                if (t <= p && (w == 0 || t > p - w) && (t < k.lo || t >= k.hi))
                                    fail("range", t, p);
                            }
                        if (k.lo < 0 || k.hi > ctx)
                            fail("bounds", k.lo, k.hi);
                        // splits of it, from its start or from key 0, hold each key once
                        for (int keys = 1; keys < 6; ++keys)
                            for (int base = 0; base <= k.lo; base += k.lo ? k.lo : 1) {
                                int next = k.lo;
                                for (int s = 0; s < 20; ++s) {
                                    const kvc::KeyRange p = kvc::split_range(k, base, s, keys);
                                    if (p.lo >= p.hi)
                                        continue;
                                    if (p.lo != next || p.hi > k.hi || p.hi - p.lo > keys)
                                        fail("split", p.lo, p.hi);
                                    next = p.hi;
                                }
                                if (k.lo < k.hi && next != k.hi)
                                    fail("splits", next, k.hi);
                            }
                    }
    // at the end of 31 bits
    {
        const kvc::KeyRange r = {(int)top - 5000, (int)top - 65536 + 60000};
        const kvc::KeyRange e = kvc::split_range(r, r.lo, 200, 1u << 30);
        if (e.lo < e.hi)
            fail("far split", e.lo, e.hi);
    }
    printf("ok\n");
    return 0;
}
