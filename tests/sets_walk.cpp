// Walks Sets<K> (csrc/ssc_sets.h), the steps in which the row kernels take a
// token's assignments, as the kernels do, and checks that the items come in
// order, each once and none outside [0, count).
#include <stdio.h>

#include "ssc_sets.h"

template <int K>
static long long wrong(int32_t count) {
    long long bad = 0, next = 0;
    for (ssc::Sets<K> s(count); s.more(); s.next()) {
        if (s.at(0) != next) ++bad;
        const long long here = count - next < K ? count - next : K;
        if (!s.has(static_cast<int>(here) - 1) || (here < K && s.has(static_cast<int>(here)))) ++bad;
        if (s.at(static_cast<int>(here) - 1) >= count) ++bad;
        next += here;
        if (bad) break;
    }
    return bad + (next != (count > 0 ? count : 0));
}

int main() {
    const int32_t most = INT32_MAX;
    const int32_t counts[] = {0, 1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 1000, most - 7, most - 6, most};
    for (int32_t c : counts) {
        const long long bad = wrong<8>(c) + wrong<4>(c) + wrong<2>(c);
        if (bad) {
            printf("%d items: %lld steps wrong\n", c, bad);
            return 1;
        }
    }
    printf("ok\n");
    return 0;
}
