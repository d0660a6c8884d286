// gdn_checks.h -- what the entry points' checks of their arguments share.
#pragma once

#include "gdn.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <limits>

namespace gdn {
namespace checks {

constexpr int64_t kI32Max = std::numeric_limits<int32_t>::max();

inline bool dtype_ok(int32_t dt) { return dt == GDN_F32 || dt == GDN_F16 || dt == GDN_BF16; }
inline int64_t dtype_size(int32_t dt) { return dt == GDN_F32 ? 4 : 2; }

inline bool aligned(const void *p, int64_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes)) == 0;
}

inline gdn_status launch_status(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

// Validates host cu_seqlens; fills the chunk counts (chunks of `clen` tokens) the
// prefill grid needs.
inline gdn_status check_cu(const int32_t *cu, int32_t n, int32_t total, int clen, int64_t *chunks,
                           int64_t *max_chunks)
{
    if (cu[0] != 0 || cu[n] != total)
        return GDN_ERR_SHAPE;
    int64_t c = 0, mx = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (cu[i + 1] < cu[i])
            return GDN_ERR_SHAPE;
        const int64_t ci = ((int64_t)cu[i + 1] - cu[i] + clen - 1) / clen;
        c += ci;
        if (ci > mx)
            mx = ci;
    }
    *chunks = c;
    *max_chunks = mx;
    return GDN_OK;
}

}  // namespace checks
}  // namespace gdn
