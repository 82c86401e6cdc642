// Whether operands share memory, where a kernel that reads the one while it
// writes the other would race.  Host code; addresses, sizes and strides in one unit.
#pragma once

#include <stdint.h>

namespace df11serve {

struct Axis {
    int64_t size, stride;
};

// Whether any of the rows of `own` units from `base` on, along n axes, meets [from, to).
inline bool rows_meet(__int128 from, __int128 to, __int128 base, const Axis *axes, int n, int64_t own)
{
    __int128 span = own;
    for (int i = 0; i < n; i++) {
        if (axes[i].size <= 0) return false;
        span += (__int128)(axes[i].size - 1) * axes[i].stride;
    }
    if (base >= to || base + span <= from) return false;
    if (!n) return true;
    const __int128 stride = axes[0].stride, inner = span - (axes[0].size - 1) * stride;
    if (!stride) return rows_meet(from, to, base, axes + 1, n - 1, own);
    // only those along the first axis that come near
    __int128 i = from - inner - base < 0 ? 0 : (from - inner - base) / stride;
    for (; i < axes[0].size && base + i * stride < to; i++)
        if (rows_meet(from, to, base + i * stride, axes + 1, n - 1, own)) return true;
    return false;
}

// Whether two sets of blocks of `own` units, the second `apart` units behind
// the first and both along the same two axes, meet.  The blocks of a set lie
// apart: the axis of greater stride steps over all that the other one spans.
inline bool sets_meet(__int128 apart, Axis great, Axis small, int64_t own)
{
    if (great.size <= 1) great = Axis{1, 0};
    if (small.size <= 1) small = Axis{1, 0};
    if (great.stride < small.stride) {
        const Axis x = great;
        great = small, small = x;
    }
    // most sets lie one behind the other, which is told without divisions (0.1 us less)
    const __int128 span = (__int128)(great.size - 1) * great.stride + (__int128)(small.size - 1) * small.stride + own;
    if (apart >= span || -apart >= span) return false;
    const auto whole = [](__int128 x, __int128 y) { return x / y - (x % y < 0); };   // rounded down
    // along each axis only the two differences of places around the quotient can meet
    for (int i = 0; i < (great.size > 1 ? 2 : 1); i++) {
        const __int128 a = great.size > 1 ? whole(apart, great.stride) + i : 0;
        if (a >= great.size || -a >= great.size) continue;
        const __int128 rest = apart - a * great.stride;
        for (int j = 0; j < (small.size > 1 ? 2 : 1); j++) {
            const __int128 b = small.size > 1 ? whole(rest, small.stride) + j : 0;
            if (b >= small.size || -b >= small.size) continue;
            const __int128 left = rest - b * small.stride;
            if (left < own && -left < own) return true;
        }
    }
    return false;
}

}  // namespace df11serve
