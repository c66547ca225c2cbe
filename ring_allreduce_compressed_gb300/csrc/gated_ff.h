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

// A matrix of 16-bit elements, next to each other along its columns.
struct Matrix16 {
    const void *p;
    long long rows, cols, ld;
};

// Can tensor maps read it?  (16-byte aligned rows)
bool gemm_takes(const Matrix16 &x);

// The products on the tensor cores (gated_gemm.cu); operands as gemm_takes has them.
template <typename T>
cudaError_t gemm_forward(const FfArgs &a, const Matrix16 &x, const Matrix16 &wg,
                         const Matrix16 &wu, cudaStream_t st);
template <typename T>
cudaError_t gemm_dx(const FfGradArgs &a, const Matrix16 &dgate, const Matrix16 &dup,
                    const Matrix16 &wg, const Matrix16 &wu, cudaStream_t st);
template <typename T, typename O>
cudaError_t gemm_dw(const FfGradArgs &a, const Matrix16 &dgate, const Matrix16 &dup,
                    const Matrix16 &x, cudaStream_t st);

// Host word that a kernel sets when a wait of its has run out of time.
cudaError_t stalled_word(unsigned **word);

} // namespace rra
