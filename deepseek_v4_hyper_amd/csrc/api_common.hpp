// api_common.hpp -- argument checks that the C ABI's implementation files
// (ds4hc_api.cpp, latent_api.cpp, serve_api.cpp) share. Not installed; not part of the ABI.
#pragma once

#include "ds4hc.h"

#include <stdint.h>

namespace ds4hc {

constexpr int64_t MAX_T = int64_t(1) << 24;  // tokens of one call

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct Range {
    const void *p;
    uint64_t bytes;
};

inline bool overlap(Range a, Range b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Whether any of the outputs overlaps another output or an input.
template <int NI, int NO>
bool clash(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int q = o + 1; q < NO; ++q)
            if (overlap(out[o], out[q])) return true;
    }
    return false;
}

// Keeps the error's text for ds4hc_last_hip_error() on this thread.
ds4hc_status hip_fail(hipError_t e);

}  // namespace ds4hc
