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

}  // namespace df11serve
