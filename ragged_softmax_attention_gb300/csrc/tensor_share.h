// Whether two strided tensors have a byte in common.  Views into one buffer
// (columns of a fused projection, the K and V halves of every page) have
// interleaved extents and share nothing, so extents alone do not tell.  Plain
// C++, no CUDA.
#pragma once

#include <cstdint>

#include "fw_attn.h"

namespace fw {

// Bytes from the tensor's first element to one past its last; esz: bytes of an element.
inline int64_t tensor_extent(const fw_tensor_t *t, int64_t esz) {
    int64_t e = 1;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] == 0) return 0;
        e += (t->shape[i] - 1) * t->stride[i];
    }
    return e * esz;
}

inline bool extents_overlap(const fw_tensor_t *a, int64_t esz_a, const fw_tensor_t *b, int64_t esz_b) {
    const char *pa = static_cast<const char *>(a->data), *pb = static_cast<const char *>(b->data);
    const int64_t ea = tensor_extent(a, esz_a), eb = tensor_extent(b, esz_b);
    return ea > 0 && eb > 0 && pa < pb + eb && pb < pa + ea;
}

// The distances from an element run of one tensor to one of another: the bases'
// plus k * stride at every level, lo <= k <= hi.
struct ShareSearch {
    struct Level {
        int64_t stride, lo, hi;
    } level[10];
    int levels = 0;
    int64_t first, last;                  // distances at which two runs meet
    int64_t low[11], high[11];            // what levels i and on can add
    int budget = 4096;

    void add(int64_t stride, int64_t lo, int64_t hi) {
        for (int i = 0; i < levels; ++i)
            if (level[i].stride == stride) {
                level[i].lo += lo;
                level[i].hi += hi;
                return;
            }
        int at = levels++;
        for (; at > 0 && level[at - 1].stride < stride; --at) level[at] = level[at - 1];
        level[at] = Level{stride, lo, hi};
    }
    // The run of consecutive elements a tensor consists of, in bytes; its other
    // dimensions become levels, counted forwards for b and backwards for a.
    int64_t open(const fw_tensor_t *t, int64_t esz, bool backwards) {
        int64_t run = esz;
        int n = t->ndim;
        if (n > 0 && t->stride[n - 1] == 1) run = t->shape[--n] * esz;
        for (int i = 0; i < n; ++i) {
            if (t->shape[i] == 1 || t->stride[i] == 0) continue;
            const int64_t far = t->shape[i] - 1;
            add(t->stride[i] * esz, backwards ? -far : 0, backwards ? 0 : far);
        }
        return run;
    }
    static int64_t floor_div(int64_t x, int64_t y) { return x / y - (x % y != 0 && x < 0); }

    // Whether distance d can reach first .. last through the levels from l on.  Nested
    // strides leave a choice or two a level; a search that finds many gives up and
    // answers yes.
    bool reach(int l, int64_t d) {
        if (l == levels) return d >= first && d <= last;
        const int64_t s = level[l].stride;
        int64_t k0 = -floor_div(-(first - high[l + 1] - d), s), k1 = floor_div(last - low[l + 1] - d, s);
        if (k0 < level[l].lo) k0 = level[l].lo;
        if (k1 > level[l].hi) k1 = level[l].hi;
        for (int64_t k = k0; k <= k1; ++k)
            if (--budget < 0 || reach(l + 1, d + k * s)) return true;
        return false;
    }
};

inline bool tensors_share(const fw_tensor_t *a, int64_t esz_a, const fw_tensor_t *b, int64_t esz_b) {
    if (!extents_overlap(a, esz_a, b, esz_b)) return false;
    ShareSearch s;
    const int64_t run_a = s.open(a, esz_a, true), run_b = s.open(b, esz_b, false);
    s.first = 1 - run_b;
    s.last = run_a - 1;
    s.low[s.levels] = s.high[s.levels] = 0;
    for (int i = s.levels - 1; i >= 0; --i) {
        s.low[i] = s.low[i + 1] + s.level[i].lo * s.level[i].stride;
        s.high[i] = s.high[i + 1] + s.level[i].hi * s.level[i].stride;
    }
    return s.reach(0, static_cast<const char *>(b->data) - static_cast<const char *>(a->data));
}

}  // namespace fw
