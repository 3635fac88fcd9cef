// Checks csrc/paging.h's windows against arithmetic in 64 bits: windows up to
// 2^31 - 1, positions before the first key and near the last.
#include <stdio.h>
#include <initializer_list>

#include "paging.h"

int main()
{
    const int32_t top = 0x7fffffff, most = top - 65536;
    const int32_t windows[] = {0, 1, 2, 5, 4096, 1 << 30, most, top - 21, top - 2, top - 1, top};
    const int32_t positions[] = {-most, -65536, -21, -20, -3, -2, -1, 0, 1, 2, 29, 4095, 4096, 1 << 30, most - 1, most};
    for (int32_t w : windows)
        for (int32_t first : positions)
            for (int32_t rows : {1, 2, 50, 4000})
                for (int32_t bound : {0, 1, 30, 5000, most}) {
                    if ((int64_t)first + rows - 1 > most)
                        continue;
                    const int32_t last = first + rows - 1;
                    const kvc::KeyRange k = kvc::key_range(first, last, w, bound);
                    const int64_t from = w > 0 ? (int64_t)first - w + 1 : 0;
                    const int64_t lo = from > 0 ? from : 0, hi = (int64_t)last + 1 < bound ? (int64_t)last + 1 : bound;
                    if (k.lo != lo || k.hi != hi) {
                        printf("key_range(%d, %d, %d, %d): %d %d, not %lld %lld\n", first, last, w, bound, k.lo, k.hi,
                               (long long)lo, (long long)hi);
                        return 1;
                    }
                    if (kvc::first_seen(first, w) != lo) {
                        printf("first_seen(%d, %d)\n", first, w);
                        return 1;
                    }
                }
    printf("ok\n");
    return 0;
}
