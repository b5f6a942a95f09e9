// sv_layout.hpp -- where a strided pool's elements lie: whether each has a place of its
// own, in the pool and among other pools of its layout.  Plain host arithmetic.
#pragma once

#include <algorithm>
#include <cstdint>

namespace sv {

// The axes of a pool with more than one element, by falling stride, and what an axis
// and those behind it span together; sizes in bytes.
struct PoolLayout {
    int axes = 0;
    int64_t n[3], stride[3], span[4];
};

// A pool of pages, heads and slots of `unit` bytes.  false: not every element is known
// to lie apart from the others, for which a stride has to reach past all that the
// smaller ones span (every order of whole axes, with gaps or without, does).
inline bool lay_out(const int64_t (&n)[3], const int64_t (&stride)[3], int64_t unit,
                    PoolLayout *p) {
    p->axes = 0;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        int at = p->axes++;
        for (; at > 0 && p->stride[at - 1] < stride[i]; --at) {
            p->n[at] = p->n[at - 1];
            p->stride[at] = p->stride[at - 1];
        }
        p->n[at] = n[i];
        p->stride[at] = stride[i];
    }
    p->span[p->axes] = unit;
    for (int i = p->axes - 1; i >= 0; --i) {
        if (p->stride[i] < p->span[i + 1]) return false;
        p->span[i] = (p->n[i] - 1) * p->stride[i] + p->span[i + 1];
    }
    return true;
}

// Whether two pools of a layout whose bases are d bytes apart share an element, as far
// as axes from `axis` on go.  Along an axis their indexes may differ by any whole number
// below its length, and what remains has to lie within what the inner axes span, at most
// a stride: two numbers do.
inline bool pools_meet(const PoolLayout &p, int64_t d, int axis = 0) {
    if (d >= p.span[axis]) return false;
    if (axis == p.axes) return true;
    const int64_t k = d / p.stride[axis], rest = d - k * p.stride[axis];
    return (k < p.n[axis] && pools_meet(p, rest, axis + 1)) ||
           (k + 1 < p.n[axis] && pools_meet(p, p.stride[axis] - rest, axis + 1));
}

// Whether any two of some pools share an element; of pools that are one and the same
// (twice), only where `twice` says so.  In order of their bases, pools lie behind each
// other, or all within one index of the outermost axis, where the same is asked of the
// axes behind it; any other arrangement is looked at pair by pair.
inline bool any_pools_meet(const PoolLayout &p, void *const *bases, int32_t count, bool twice) {
    constexpr int32_t kSorted = 1024;
    const char *sorted[kSorted];
    auto meet = [&](const char *x, const char *y) {
        return x == y ? twice : pools_meet(p, x < y ? y - x : x - y);
    };
    if (count > kSorted) {  // no room to sort them
        for (int32_t i = 1; i < count; ++i)
            for (int32_t j = 0; j < i; ++j)
                if (meet(static_cast<const char *>(bases[i]), static_cast<const char *>(bases[j])))
                    return true;
        return false;
    }
    for (int32_t i = 0; i < count; ++i) sorted[i] = static_cast<const char *>(bases[i]);
    if (!std::is_sorted(sorted, sorted + count)) std::sort(sorted, sorted + count);
    if (!twice) count = static_cast<int32_t>(std::unique(sorted, sorted + count) - sorted);
    if (count < 2) return false;
    for (int axis = 0;; ++axis) {
        bool behind = true;
        for (int32_t i = 1; i < count; ++i) behind &= sorted[i] - sorted[i - 1] >= p.span[axis];
        if (behind) return false;
        if (axis == p.axes ||
            sorted[count - 1] - sorted[0] > p.stride[axis] - p.span[axis + 1])
            break;
    }
    for (int32_t i = 1; i < count; ++i)
        for (int32_t j = i - 1; j >= 0 && sorted[i] - sorted[j] < p.span[0]; --j)
            if (meet(sorted[i], sorted[j])) return true;
    return false;
}

}  // namespace sv
