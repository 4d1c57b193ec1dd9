// The steps of a loop over `count` items in sets of K, for any count up to
// INT32_MAX: an int that counts up by K passes the largest int in the last
// step of the largest counts, so the items left are counted down instead. Plain
// C++, so that the host can walk it too.
#pragma once

#include <stdint.h>

namespace ssc {

template <int K>
struct Sets {
    int32_t left;        // items from the set's first one on
    uint32_t first = 0;

    constexpr explicit Sets(int32_t count) : left(count) {}
    constexpr bool more() const { return left > 0; }
    constexpr bool has(int j) const { return j < left; }                  // whether the set has an item j < K,
    constexpr int64_t at(int j) const { return int64_t{first} + j; }      // and which item it is
    constexpr void next() {
        left -= K;
        first += K;
    }
};

}  // namespace ssc
