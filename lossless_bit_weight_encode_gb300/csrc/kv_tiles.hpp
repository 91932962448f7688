// Row tiles of the paged cache's attention launches, and the kernels that there are for them:
// what plans a call and what launches it both ask here.  Host code alone.
#pragma once

#include <algorithm>
#include <cstdint>

namespace w12 {
namespace dev {

constexpr int kTcRows = 128;  // of the tcgen05 kernel

// What a launch has of the spans of a call with shared prefixes: all, the prefixes, or the own
// tokens (then it is the second).
enum KvSpans { kKvAllSpans, kKvPrefixes, kKvOwnSpans };

}  // namespace dev

namespace launch {

// Rows of the tile a launch uses: new tokens times query heads per key head.  Up to
// 8 the warp-level kernel, above 16 the tcgen05 kernel with 128 (more rows take
// several row blocks).  30 rows measured 326 us against 532 with 32-row warp-level
// tiles (64 requests of 8000 tokens, BF16; 8-bit 337 against 547), 128 against 133
// for two requests of 100001.  Between 9 and 16 rows the warp-level kernel is the
// shorter way for few row blocks (12 rows, one request of 777 tokens: 9.1 against
// 10.6 us) and for 8-bit caches (64 x 8000: 325 against 340), the tcgen05 kernel for
// as many blocks as SMs (64 x 8000, BF16: 315 against 343; windows of 1024: 76
// against 81).
inline int attend_rows(int max_new, int group, int kv_heads, int requests, bool q8, int sm_count) {
    const int64_t rows = (int64_t)(max_new < 1 ? 1 : max_new) * group;
    if (rows <= 8) return 8;
    if (rows > 16 || (!q8 && (int64_t)kv_heads * requests >= sm_count)) return dev::kTcRows;
    return 16;
}

// Row tiles of a call with shared prefixes: of the prefixes and of the own tokens, in two
// launches where they differ.
struct SharedTiles {
    int prefix, own;
    int lines() const { return prefix == own ? 1 : 2; }
    dev::KvSpans kind(int line) const {
        return lines() == 1 ? dev::kKvAllSpans : line == 0 ? dev::kKvPrefixes : dev::kKvOwnSpans;
    }
};
inline SharedTiles shared_tiles(int tokens, int max_new, int requests, int groups, int max_requests, int group,
                                int kv_heads, bool q8, int sm_count) {
    const int most = std::max(std::min(max_new, tokens), 1);
    const int together = (int)std::min<int64_t>((int64_t)std::max(max_requests, 1) * most, tokens);
    SharedTiles t;
    t.prefix = t.own = attend_rows(together, group, kv_heads, groups, q8, sm_count);
    // The own tokens in a launch of their own, with their own row tile, for 8-bit caches, whose
    // conversion would be paid for few rows too (8 x 8 beams of 130 tokens behind 6000: 57 us, in
    // one launch 79), and for so many row blocks that the start and end of each in the tcgen05
    // kernel weigh more than a second launch (48 heads over 8: 64 requests of 225 tokens 38
    // against 35, 128 54 against 55, 256 of 100 tokens 68 against 88, 512 118 against 170).
    if (q8 || (int64_t)requests * kv_heads >= 6 * (int64_t)sm_count)
        t.own = attend_rows(most, group, kv_heads, requests, q8, sm_count);
    // Many requests of 9 to 16 rows take the tcgen05 kernel where few groups of as many (fewer
    // are said to be in a group, or have new tokens, than there are requests) would not: one
    // launch with its tile then.
    t.prefix = std::max(t.prefix, t.own);
    return t;
}

// Rows of the kernel that one of a call's launches takes for a tile of `rows`: that, or 0 where
// there is no such kernel.  Of two launches the prefixes' has the larger tile, and of a BF16
// cache the own tokens' has the smallest one.
constexpr int shared_kernel_rows(dev::KvSpans kind, bool q8, int rows) {
    if (rows != 8 && rows != 16 && rows != dev::kTcRows) return 0;
    if (kind == dev::kKvPrefixes) return rows == 8 ? 0 : rows;
    if (kind == dev::kKvOwnSpans) return rows == 8 || (q8 && rows == 16) ? rows : 0;
    return rows;
}

}  // namespace launch
}  // namespace w12
