// experts_rules.hpp - what the experts' step decides with whole numbers alone: the layout of the
// lists in experts_decode's workspace and their bounds.  Plain C++, so that it can be
// checked without a GPU.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define MOE_HOST_DEVICE __host__ __device__
#else
#define MOE_HOST_DEVICE
#endif

namespace moe {

// The work of one pass over an expert's weights: up to a pass's width of its entries.  Slot s
// belongs to expert[s] and has the entries ent[first[s]] .. ent[first[s + 1] - 1].  All
// three, and the number n of slots, are one block of 16-bit words, sized by the number N of
// entries: n, one unused, expert [N], first [N+2], ent [N].
struct ListLayout {
    int N;
    MOE_HOST_DEVICE constexpr int expert() const { return 2; }
    MOE_HOST_DEVICE constexpr int first() const { return 2 + N; }
    MOE_HOST_DEVICE constexpr int ent() const { return 4 + 2 * N; }
    MOE_HOST_DEVICE constexpr int words32() const { return (4 + 3 * N + 1) / 2; }
    // 16-bit word i of a block as it is used, whatever v it holds: n and first at most N, so that
    // first[s + 1] ends every list within ent; ids of experts and entries below E and N.
    MOE_HOST_DEVICE constexpr uint32_t bounded(int i, uint32_t v, int E) const {
        const int most = i >= ent() ? N - 1 : i >= first() || i < expert() ? N : E - 1;
        return v < (uint32_t)most ? v : (uint32_t)most;
    }
};

}  // namespace moe
