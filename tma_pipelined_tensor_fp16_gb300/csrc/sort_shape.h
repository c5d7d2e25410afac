// sort_shape.h -- the launch of the expert sort: one cluster, every warp of which owns a
// contiguous run of slots.
#pragma once

#include <cstdint>

namespace tg {

constexpr int SORT_CTAS = 16;         // more than the portable 8
constexpr int SORT_PORTABLE_CTAS = 8;
constexpr int SORT_CTA_SLOTS = 1024;  // slots for which another CTA pays

struct SortShape {
    int ctas, warps;
    int run;  // slots per warp, a multiple of 32
    unsigned smem_bytes(int experts) const
    {
        return static_cast<unsigned>(((warps + 2) * (experts + 1) + 33) * 4);
    }
};

// For up to `most` CTAs (a power of two).
inline SortShape sort_shape(int64_t slots, int most)
{
    SortShape s = {1, 32, 0};
    while (s.ctas < most && slots > static_cast<int64_t>(SORT_CTA_SLOTS) * s.ctas) s.ctas *= 2;
    while (s.warps > 8 && slots <= static_cast<int64_t>(s.warps) * 32 * s.ctas) s.warps /= 2;
    const int64_t per_warp = (slots + s.ctas * s.warps - 1) / (s.ctas * s.warps);
    s.run = static_cast<int>((per_warp + 31) / 32 * 32);
    return s;
}

}  // namespace tg
