// layer_check.h -- host-side argument checks shared by the C ABI of the layer operators.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/lattice_osr.h"

namespace layer {

inline size_t elem(int dtype) { return dtype == LATTICE_OSR_BF16 ? 2 : 4; }
inline bool dtype_ok(int t) { return t == LATTICE_OSR_F32 || t == LATTICE_OSR_BF16; }

// One buffer argument.  Absent buffers (null) are skipped by every check.
struct Buf {
    const void* p;
    size_t bytes, align;
    bool out;
};

inline int check_buffers(const Buf* b, int n) {
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(b[i].p) % b[i].align != 0) return LATTICE_OSR_ERR_ALIGN;
    for (int i = 0; i < n; ++i) {
        if (!b[i].p || !b[i].out) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(b[i].p), hi = lo + b[i].bytes;
        for (int j = 0; j < n; ++j) {
            if (j == i || !b[j].p) continue;
            const uintptr_t l2 = reinterpret_cast<uintptr_t>(b[j].p), h2 = l2 + b[j].bytes;
            if (lo < h2 && l2 < hi) return LATTICE_OSR_ERR_ALIAS;
        }
    }
    return LATTICE_OSR_OK;
}

}  // namespace layer
