// sv_launch.hpp -- how the paged-cache calls share pools out to launches: plain
// arithmetic without HIP, so that it can be tested anywhere.
#pragma once

#include <cstdint>

namespace sv {

constexpr int kCacheBlock = 256;
constexpr int kMaxPools = 64;  // pools per launch

// A grid's threads must stay below 2^32.
inline bool grid_fits(int64_t blocks, int block) {
    return blocks <= (int64_t{1} << 32) / block - 1 && blocks <= INT32_MAX;
}

// Pools of a launch: as many as there are, up to kMaxPools, halved until a launch of
// them fits; 0 where one does not.
template <typename Fits>
int pools_per_launch(int32_t pools, Fits fits) {
    int n = pools < kMaxPools ? pools : kMaxPools;
    while (n > 1 && !fits(n)) n /= 2;
    return fits(n) ? n : 0;
}

// Keeping a path: a thread per 16 bytes of a position's heads in n pools (column: per
// pool), counted in 32 bits, in workgroups per sequence; without pools one workgroup
// that leaves the lengths.
inline int64_t keep_blocks(int64_t column, int n) {
    const int64_t blocks = (column * n + kCacheBlock - 1) / kCacheBlock;
    return blocks > 0 ? blocks : 1;
}
inline int keep_pools_per_launch(int64_t column, int32_t batch, int32_t pools) {
    return pools_per_launch(pools, [&](int n) {
        return column * n <= INT32_MAX && grid_fits(keep_blocks(column, n) * batch, kCacheBlock);
    });
}

// Copying pages: a workgroup per row, pool and head.
inline int copy_pools_per_launch(int32_t rows, int32_t heads, int32_t pools) {
    return pools_per_launch(
        pools, [&](int n) { return grid_fits(int64_t{rows} * heads * n, kCacheBlock); });
}

}  // namespace sv
