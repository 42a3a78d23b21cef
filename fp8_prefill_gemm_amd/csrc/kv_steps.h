// Kernels of the paged cache are compiled for each number of 32-column steps of
// a row, 1 to RZ_KV_MAX_DIM / 32.  Host code, no HIP.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "rz_fp8.h"

namespace rz {

// Calls f(std::integral_constant<int, c>{}); false, and no call, for a c that no
// kernel is compiled for: what follows would read what was never written.
template <int C = 1, typename F>
[[nodiscard]] bool with_steps(uint32_t c, F&& f) {
    if constexpr (C > (int)(RZ_KV_MAX_DIM / 32u)) {
        return false;
    } else {
        if (c != (uint32_t)C) return with_steps<C + 1>(c, f);
        f(std::integral_constant<int, C>{});
        return true;
    }
}

}  // namespace rz
