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

// A matrix of 16-bit elements, next to each other along its columns; fp32 ones as three
// planes of bf16, one behind the other.
struct Matrix16 {
    const void *p;
    long long rows, cols, ld;
    int planes;
};

// Can the products read it as it is?  (16-byte aligned rows)
bool gemm_takes(const Matrix16 &x);

// The products on the tensor cores (gated_gemm.cu); operands as gemm_takes has them.
// in: x, w_gate, w_up; dgate, dup, w_gate, w_up, x.  gemm_parts: bytes that a call
// needs `parts_at` bytes from the stream's scratch on.
size_t gemm_parts(const FfArgs &a, bool f32);
size_t gemm_parts(const FfGradArgs &a, bool f32);
template <typename T>
cudaError_t gemm_forward(const FfArgs &a, const Matrix16 (&in)[3], unsigned char *scratch,
                         size_t parts_at, cudaStream_t st);
template <typename T>
cudaError_t gemm_dx(const FfGradArgs &a, const Matrix16 (&in)[5], unsigned char *scratch,
                    size_t parts_at, cudaStream_t st);
template <typename T, typename O>
cudaError_t gemm_dw(const FfGradArgs &a, const Matrix16 (&in)[5], unsigned char *scratch,
                    size_t parts_at, cudaStream_t st);

// Few rows (gated_rows.cu): is the call one of those, and its kernel.
template <typename T> bool few_rows(const FfArgs &a);
template <typename T> rra_status rows_forward(const FfArgs &a, cudaStream_t st);

} // namespace rra
