// gated_ff.h -- arguments of the gated feed-forward block's kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rra.h"

namespace rra {

// Gate or up as it is kept for the backward pass: exps and codes (saved.cuh), or
// the values (exps NULL), or nothing (data NULL).
struct Kept {
    int8_t *exps;
    void *data;
};

struct FfArgs {
    const void *x, *wg, *wu;
    long long rows, dim, ff;
    int act;
    void *h;
    Kept gate, up;
};

struct FfGradArgs {
    const void *dh, *x, *wg, *wu;
    Kept gate, up;
    long long rows, dim, ff;
    int act;
    void *dgate, *dup, *h, *dx, *dwg, *dwu;
    int accumulate;
};

} // namespace rra
