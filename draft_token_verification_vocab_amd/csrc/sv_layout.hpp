// sv_layout.hpp -- where a strided pool's elements lie: whether each has a place of its
// own.  Plain host arithmetic.
#pragma once

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

}  // namespace sv
