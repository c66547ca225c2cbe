// layer_norm.cu -- rra_layer_norm and rra_layer_norm_grad.
//
//   mean = sum x / D,  var = sum (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y    = (x - mean) rstd gamma + beta
//
//   xh = (x - mean) rstd,  w = dy gamma
//   dx = rstd (w - mean(w) - xh mean(w xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound by memory: x read and y written; x and dy read and dx written.
#include "op_common.cuh"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float block_sum(float v, float *sm)
{
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sm[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k)
        s += sm[k];
    return s;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
    norm_row_kernel(const T *__restrict__ x, const W *__restrict__ gamma,
                    const W *__restrict__ beta, long long rows, long long dim, float eps, T *y,
                    float *__restrict__ mean, float *__restrict__ rstd)
{
    __shared__ float sm[kWarps];
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *const p = x + r * dim;
        float s = 0.0f;
        for (long long c = threadIdx.x; c < dim; c += kThreads)
            s += to_f32(p[c]);
        const float mu = block_sum(s, sm) / (float)dim;
        s = 0.0f;
        for (long long c = threadIdx.x; c < dim; c += kThreads) {
            const float d = to_f32(p[c]) - mu;
            s = fmaf(d, d, s);
        }
        const float rs = 1.0f / sqrtf(block_sum(s, sm) / (float)dim + eps);
        for (long long c = threadIdx.x; c < dim; c += kThreads) {
            const float g = gamma ? to_f32(gamma[c]) : 1.0f, b = beta ? to_f32(beta[c]) : 0.0f;
            y[r * dim + c] = from_f32<T>(fmaf((to_f32(p[c]) - mu) * rs, g, b));
        }
        if (threadIdx.x == 0) {
            if (mean)
                mean[r] = mu;
            if (rstd)
                rstd[r] = rs;
        }
    }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
    dx_row_kernel(const T *dy, const T *x, const W *__restrict__ gamma,
                  const float *__restrict__ mean, const float *__restrict__ rstd, long long rows,
                  long long dim, T *dx)
{
    __shared__ float sm[kWarps];
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        float a = 0.0f, b = 0.0f;
        for (long long c = threadIdx.x; c < dim; c += kThreads) {
            const float w = to_f32(dy[r * dim + c]) * (gamma ? to_f32(gamma[c]) : 1.0f);
            a += w;
            b = fmaf(w, (to_f32(x[r * dim + c]) - mu) * rs, b);
        }
        a = block_sum(a, sm) / (float)dim;
        b = block_sum(b, sm) / (float)dim;
        for (long long c = threadIdx.x; c < dim; c += kThreads) {
            const float w = to_f32(dy[r * dim + c]) * (gamma ? to_f32(gamma[c]) : 1.0f);
            const float xh = (to_f32(x[r * dim + c]) - mu) * rs;
            dx[r * dim + c] = from_f32<T>(rs * (w - a - xh * b));
        }
    }
}

// Sums over a stretch of rows: a partial row of dgamma and one of dbeta.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    weight_part_kernel(const T *__restrict__ dy, const T *__restrict__ x,
                       const float *__restrict__ mean, const float *__restrict__ rstd,
                       long long rows, long long dim, long long stretch, float *__restrict__ part)
{
    const long long lo = blockIdx.y * stretch, hi = min(lo + stretch, rows);
    for (long long c = (long long)blockIdx.x * kThreads + threadIdx.x; c < dim;
         c += (long long)gridDim.x * kThreads) {
        float g = 0.0f, b = 0.0f;
        for (long long r = lo; r < hi; ++r) {
            const float d = to_f32(dy[r * dim + c]);
            g = fmaf(d, (to_f32(x[r * dim + c]) - mean[r]) * rstd[r], g);
            b += d;
        }
        part[(2LL * blockIdx.y) * dim + c] = g;
        part[(2LL * blockIdx.y + 1) * dim + c] = b;
    }
}

template <typename W>
__global__ void __launch_bounds__(kThreads)
    weight_join_kernel(const float *__restrict__ part, int parts, long long dim, W *dgamma,
                       W *dbeta, int accumulate)
{
    for (long long c = (long long)blockIdx.x * kThreads + threadIdx.x; c < dim;
         c += (long long)gridDim.x * kThreads) {
        float g = 0.0f, b = 0.0f;
        for (int p = 0; p < parts; ++p) {
            g += part[2LL * p * dim + c];
            b += part[(2LL * p + 1) * dim + c];
        }
        if (dgamma)
            dgamma[c] = from_f32<W>(accumulate ? to_f32(dgamma[c]) + g : g);
        if (dbeta)
            dbeta[c] = from_f32<W>(accumulate ? to_f32(dbeta[c]) + b : b);
    }
}

inline unsigned grid_of(long long items, int per_sm)
{
    return (unsigned)std::max(1LL, std::min(items, (long long)num_sms() * per_sm));
}

struct Fwd {
    const void *x, *gamma, *beta;
    long long rows, dim;
    float eps;
    void *y;
    float *mean, *rstd;
};

template <typename T, typename W> void forward(const Fwd &a, cudaStream_t st)
{
    norm_row_kernel<T, W><<<grid_of(a.rows, 8), kThreads, 0, st>>>(
        static_cast<const T *>(a.x), static_cast<const W *>(a.gamma),
        static_cast<const W *>(a.beta), a.rows, a.dim, a.eps, static_cast<T *>(a.y), a.mean,
        a.rstd);
}

constexpr int kMostParts = 128;

struct Bwd {
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    long long rows, dim;
    void *dx, *dgamma, *dbeta;
    int accumulate;
    float *part;
};

template <typename T, typename W> void backward(const Bwd &a, cudaStream_t st)
{
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    const unsigned cols = (unsigned)std::min((a.dim + kThreads - 1) / kThreads, 1LL << 16);
    int parts = 0;
    if (a.dgamma || a.dbeta) {
        if (a.rows > 0) {
            const long long stretch = std::max(16LL, (a.rows + kMostParts - 1) / kMostParts);
            parts = (int)((a.rows + stretch - 1) / stretch);
            weight_part_kernel<T><<<dim3(cols, parts), kThreads, 0, st>>>(
                dy, x, a.mean, a.rstd, a.rows, a.dim, stretch, a.part);
        }
        weight_join_kernel<W><<<cols, kThreads, 0, st>>>(a.part, parts, a.dim,
                                                         static_cast<W *>(a.dgamma),
                                                         static_cast<W *>(a.dbeta), a.accumulate);
    }
    // last: dx may be dy or x
    if (a.dx && a.rows > 0)
        dx_row_kernel<T, W><<<grid_of(a.rows, 8), kThreads, 0, st>>>(
            dy, x, static_cast<const W *>(a.gamma), a.mean, a.rstd, a.rows, a.dim,
            static_cast<T *>(a.dx));
}

constexpr size_t kMostRows = (size_t)1 << 40, kMostDim = (size_t)1 << 31;

bool valid_sizes(size_t rows, size_t dim, rra_dtype t, rra_dtype w)
{
    return valid_dt(t) && valid_dt(w) && dim > 0 && dim <= kMostDim && rows <= kMostRows;
}

// Either apart or the same buffer.
bool apart_or_same(const void *a, size_t na, const void *b, size_t nb)
{
    return a == b || !overlap(a, na, b, nb);
}

} // namespace
} // namespace rra

extern "C" rra_status rra_layer_norm(const void *x, const void *gamma, const void *beta,
                                     size_t rows, size_t dim, rra_dtype dtype,
                                     rra_dtype weight_t, float eps, void *y, float *mean,
                                     float *rstd, void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t) || !(eps >= 0.0f))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es;
    if (rows > 0 && (!x || !y || !aligned_to(x, es) || !aligned_to(y, es)))
        return RRA_ERR_INVALID;
    if (!aligned_to(gamma, ws) || !aligned_to(beta, ws) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4) || !apart_or_same(x, bytes, y, bytes) ||
        overlap(y, bytes, gamma, dim * ws) || overlap(y, bytes, beta, dim * ws) ||
        overlap(y, bytes, mean, rows * 4) || overlap(y, bytes, rstd, rows * 4) ||
        overlap(x, bytes, mean, rows * 4) || overlap(x, bytes, rstd, rows * 4) ||
        overlap(mean, rows * 4, rstd, rows * 4))
        return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    if (rows == 0)
        return RRA_OK;
    const Fwd a{x, gamma, beta, (long long)rows, (long long)dim, eps, y, mean, rstd};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == RRA_F32)
        forward<float, float>(a, st);
    else if (dtype == RRA_F16 && weight_t == RRA_F16)
        forward<__half, __half>(a, st);
    else if (dtype == RRA_F16)
        forward<__half, float>(a, st);
    else if (weight_t == RRA_BF16)
        forward<__nv_bfloat16, __nv_bfloat16>(a, st);
    else
        forward<__nv_bfloat16, float>(a, st);
    return launched(cudaGetLastError());
}

extern "C" rra_status rra_layer_norm_grad(const void *dy, const void *x, const void *gamma,
                                          const float *mean, const float *rstd, size_t rows,
                                          size_t dim, rra_dtype dtype, rra_dtype weight_t,
                                          void *dx, void *dgamma, void *dbeta, int accumulate,
                                          void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t) || (!dx && !dgamma && !dbeta))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es,
                 wb = dim * ws;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !aligned_to(dy, es) || !aligned_to(x, es)))
        return RRA_ERR_INVALID;
    if (!aligned_to(gamma, ws) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(dx, es) || !aligned_to(dgamma, ws) || !aligned_to(dbeta, ws))
        return RRA_ERR_INVALID;
    if (!apart_or_same(dx, bytes, dy, bytes) || !apart_or_same(dx, bytes, x, bytes) ||
        overlap(dgamma, wb, dbeta, wb))
        return RRA_ERR_INVALID;
    for (void *out : {dgamma, dbeta})
        if (overlap(out, wb, dy, bytes) || overlap(out, wb, x, bytes) ||
            overlap(out, wb, gamma, wb) || overlap(out, wb, mean, rows * 4) ||
            overlap(out, wb, rstd, rows * 4) || overlap(out, wb, dx, bytes))
            return RRA_ERR_INVALID;
    if (overlap(dx, bytes, gamma, wb) || overlap(dx, bytes, mean, rows * 4) ||
        overlap(dx, bytes, rstd, rows * 4))
        return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    std::unique_lock<std::mutex> lk;
    unsigned char *scratch = nullptr;
    const rra_status s =
        op_scratch(st, kScratchHead + sizeof(float) * 2 * kMostParts * dim, lk, &scratch);
    if (s != RRA_OK)
        return s;
    const Bwd a{dy, x,      gamma, mean,       rstd, (long long)rows, (long long)dim, dx, dgamma,
                dbeta, accumulate, reinterpret_cast<float *>(scratch + kScratchHead)};
    if (dtype == RRA_F32)
        backward<float, float>(a, st);
    else if (dtype == RRA_F16 && weight_t == RRA_F16)
        backward<__half, __half>(a, st);
    else if (dtype == RRA_F16)
        backward<__half, float>(a, st);
    else if (weight_t == RRA_BF16)
        backward<__nv_bfloat16, __nv_bfloat16>(a, st);
    else
        backward<__nv_bfloat16, float>(a, st);
    return launched(cudaGetLastError());
}
