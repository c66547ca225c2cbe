// layer_norm_saved.cu -- rra_layer_norm_save, rra_layer_norm_restore and
// rra_layer_norm_saved_grad: layer norm whose input is kept in 8 bits (saved.cuh)
// for the backward pass.
//
//   mean = sum x / D,  var = sum (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y    = (x - mean) rstd gamma + beta          codes of x
//
//   v = m 2^(e-6),  xh = (v - mean) rstd         (restored)
//   y  = xh gamma + beta
//   dx = rstd (w - mean(w) - xh mean(w xh)),  w = dy gamma
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound by memory: one pass over what is read and written, 8 bits of the saved
// row among it.
#include "op_common.cuh"
#include "row_group.cuh"
#include "saved.cuh"

namespace rra {
namespace {

// 8 weights as fp32 from column c on, of which n are there.
template <typename W, bool VEC>
__device__ __forceinline__ void weights8(const W *p, long long c, int n, float none, float v[8])
{
    if (p) {
        load8<W, VEC>(p + c, n, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = none;
}

// Elements of a row's pack u: 8, or fewer at the row's end and behind it.
__device__ __forceinline__ int in_pack(long long dim, long long u)
{
    return (int)max(0LL, min((long long)kPack, dim - u * kPack));
}

// ---------------------------------------------------------------- save

struct Save {
    const void *x, *gamma, *beta;
    long long rows, dim;
    float eps;
    void *y;
    int8_t *exps, *codes;
    float *mean, *rstd;
    Group g;
};

constexpr int kSaveThreads = 256;
constexpr int kSaveHeld = 4; // packs of a lane

// A row in the registers of a group of lanes, as in norm_kernel: lane i holds
// packs i, i + lanes, ..., and 16 lanes of a warp a block of codes.
// VEC: every pack is whole and on a 16-byte boundary.
template <typename T, typename W, int K, bool MULTI, bool VEC>
__global__ void __launch_bounds__(MULTI ? 1024 : kSaveThreads) save_kernel(const Save a)
{
    __shared__ __align__(16) float sm[MULTI ? 2 * 32 : 4];
    const T *const x = static_cast<const T *>(a.x);
    T *const y = static_cast<T *>(a.y);
    const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                static_cast<const W *>(a.beta);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, groups = blockDim.x / lanes;
    const int nb = (int)blocks_of(a.dim), packs = nb * kBlockPacks;
    const float n = (float)a.dim, inverse = 1.0f / n;
    GroupOf group = group_of(a.g, sm, 1);
    if (MULTI) {
        if (threadIdx.x < 64)
            sm[threadIdx.x] = 0.0f;
        __syncthreads();
    }
    const int first = threadIdx.x / lanes;
    dependents_wait();
    dependents_launch();
    for (long long base = (long long)blockIdx.x * groups; base < a.rows;
         base += (long long)gridDim.x * groups) {
        // every lane takes part in the sums, some in vain: they read the last row
        const long long r = MULTI ? base : min(base + first, a.rows - 1);
        const bool on = MULTI || base + first < a.rows;
        float v[K][8];
        Sums<1> s{{0.0f}};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = li + k * lanes;
            load8<T, VEC>(x + r * a.dim + (long long)u * kPack, in_pack(a.dim, u), v[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s.v[0] += v[k][j];
        }
        const float mu = quotient(group_sum<MULTI, 1>(s, group).v[0], n, inverse);
        s.v[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int there = in_pack(a.dim, li + k * lanes);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = j < there ? v[k][j] - mu : 0.0f;
                s.v[0] = fmaf(d, d, s.v[0]);
            }
        }
        const float rs = rsqrtf(quotient(group_sum<MULTI, 1>(s, group).v[0], n, inverse) + a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = li + k * lanes, there = in_pack(a.dim, u);
            const int E = block_exponent(half_warp_max(top_bits(v[k])));
            if (!on || u >= packs)
                continue;
            store_codes(a.codes + (r * packs + u) * kPack, encode8(v[k], E));
            if (u % kBlockPacks == 0)
                a.exps[r * nb + u / kBlockPacks] = exponent_byte(E);
            float g[8], b[8];
            weights8<W, VEC>(gamma, (long long)u * kPack, there, 1.0f, g);
            weights8<W, VEC>(beta, (long long)u * kPack, there, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[k][j] = fmaf((v[k][j] - mu) * rs, g[j], b[j]);
            store8<T, VEC>(y + r * a.dim + (long long)u * kPack, there, v[k]);
        }
        if (on && li == 0) {
            a.mean[r] = mu;
            a.rstd[r] = rs;
        }
    }
}

// Rows that no block holds: passes over each, the later ones from L2.
constexpr int kLongThreads = 1024;

template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads) save_long_kernel(const Save a)
{
    __shared__ __align__(16) float sm[2 * 32];
    GroupOf block = group_of(Group{5, kLongThreads / 32}, sm, 1);
    dependents_wait();
    dependents_launch();
    const long long nb = blocks_of(a.dim), packs = nb * kBlockPacks;
    const float n = (float)a.dim;
    const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                static_cast<const W *>(a.beta);
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const p = static_cast<const T *>(a.x) + r * a.dim;
        Sums<1> s{};
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads)
            s.v[0] += to_f32(p[c]);
        const float mu = group_sum<true, 1>(s, block).v[0] / n;
        s.v[0] = 0.0f;
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float d = to_f32(p[c]) - mu;
            s.v[0] = fmaf(d, d, s.v[0]);
        }
        const float rs = rsqrtf(group_sum<true, 1>(s, block).v[0] / n + a.eps);
        // whole warps: a block's 16 lanes take part in its maximum together
        for (long long u0 = threadIdx.x / 32 * 32; u0 < packs; u0 += kLongThreads) {
            const long long u = u0 + threadIdx.x % 32;
            const int there = in_pack(a.dim, u);
            float v[8], g[8], b[8];
            load8<T, false>(p + u * kPack, there, v);
            const int E = block_exponent(half_warp_max(top_bits(v)));
            if (u >= packs)
                continue;
            store_codes(a.codes + (r * packs + u) * kPack, encode8(v, E));
            if (u % kBlockPacks == 0)
                a.exps[r * nb + u / kBlockPacks] = exponent_byte(E);
            weights8<W, false>(gamma, u * kPack, there, 1.0f, g);
            weights8<W, false>(beta, u * kPack, there, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = fmaf((v[j] - mu) * rs, g[j], b[j]);
            store8<T, false>(static_cast<T *>(a.y) + r * a.dim + u * kPack, there, v);
        }
        __syncthreads(); // y may be x: nobody reads the row any more
        if (threadIdx.x == 0) {
            a.mean[r] = mu;
            a.rstd[r] = rs;
        }
    }
}

// Group of 16 lanes (one block of codes), a warp or several.
Group save_group(long long packs, int K)
{
    return {packs <= kBlockPacks ? 4 : 5, (int)((packs + 32 * K - 1) / (32 * K))};
}

template <typename T, typename W, bool VEC> cudaError_t save_rows(Save a, cudaStream_t st)
{
    const long long packs = blocks_of(a.dim) * kBlockPacks;
    if (packs > 1024LL * kSaveHeld)
        return launch_chained(save_long_kernel<T, W>, dim3(grid_of(a.rows, 2)), kLongThreads, st,
                              a);
    const bool few = packs <= 32;
    a.g = save_group(packs, few ? 1 : kSaveHeld);
    if (a.g.warps > 1) {
        const int threads = 32 * a.g.warps;
        return launch_chained(save_kernel<T, W, kSaveHeld, true, VEC>,
                              dim3(grid_of(a.rows, 2048 / threads)), threads, st, a);
    }
    const int per_block = kSaveThreads / a.g.lanes();
    const unsigned grid = grid_of((a.rows + per_block - 1) / per_block, 16);
    return few ? launch_chained(save_kernel<T, W, 1, false, VEC>, dim3(grid), kSaveThreads, st, a)
               : launch_chained(save_kernel<T, W, kSaveHeld, false, VEC>, dim3(grid), kSaveThreads,
                                st, a);
}

// Is every pack of 8 elements of these rows, and of the weights, whole and on
// a 16-byte boundary?
template <typename T>
bool whole_packs(long long dim, std::initializer_list<const void *> arrays)
{
    if (dim % kPack)
        return false;
    for (const void *p : arrays)
        if (p && !aligned_to(p, 16))
            return false;
    return true;
}

template <typename T, typename W> rra_status save(const Save &a, cudaStream_t st)
{
    return launched(whole_packs<T>(a.dim, {a.x, a.y, a.gamma, a.beta})
                        ? save_rows<T, W, true>(a, st)
                        : save_rows<T, W, false>(a, st));
}

// ---------------------------------------------------------------- restore

struct Restore {
    const int8_t *exps, *codes;
    const float *mean, *rstd;
    const void *gamma, *beta;
    long long rows, dim;
    void *y;
    int lanes; // of a row
};

constexpr int kRestoreThreads = 256;

template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kRestoreThreads) restore_kernel(const Restore a)
{
    const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                static_cast<const W *>(a.beta);
    const long long nb = blocks_of(a.dim), packs = (a.dim + kPack - 1) / kPack;
    const int li = threadIdx.x % a.lanes, groups = kRestoreThreads / a.lanes;
    dependents_wait();
    dependents_launch();
    for (long long r = (long long)blockIdx.x * groups + threadIdx.x / a.lanes; r < a.rows;
         r += (long long)gridDim.x * groups) {
        const float mu = a.mean ? a.mean[r] : 0.0f, rs = a.rstd ? a.rstd[r] : 1.0f;
        for (long long u = li; u < packs; u += a.lanes) {
            const int there = in_pack(a.dim, u);
            float v[8], g[8], b[8];
            decode8(load_codes(a.codes + (r * nb * kBlockPacks + u) * kPack),
                    a.exps[r * nb + u / kBlockPacks], v);
            weights8<W, VEC>(gamma, u * kPack, there, 1.0f, g);
            weights8<W, VEC>(beta, u * kPack, there, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = fmaf((v[j] - mu) * rs, g[j], b[j]);
            store8<T, VEC>(static_cast<T *>(a.y) + r * a.dim + u * kPack, there, v);
        }
    }
}

template <typename T, typename W> rra_status restore(Restore a, cudaStream_t st)
{
    a.lanes = 1;
    while (a.lanes < kRestoreThreads && a.lanes * kPack < a.dim)
        a.lanes *= 2;
    const int groups = kRestoreThreads / a.lanes;
    const dim3 grid(grid_of((a.rows + groups - 1) / groups, 8));
    return launched(whole_packs<T>(a.dim, {a.y, a.gamma, a.beta})
                        ? launch_chained(restore_kernel<T, W, true>, grid, kRestoreThreads, st, a)
                        : launch_chained(restore_kernel<T, W, false>, grid, kRestoreThreads, st,
                                         a));
}

// ---------------------------------------------------------------- gradient

struct SavedGrad {
    const void *dy;
    const int8_t *exps, *codes;
    const void *gamma;
    const float *mean, *rstd;
    long long rows, dim;
    void *dx, *dgamma, *dbeta;
    int accumulate;
    float *part; // [parts][2][dim]
    int parts;
    long long stretch; // rows of a partial row
};

// xh of pack u of row r.
__device__ __forceinline__ void normal8(const SavedGrad &a, long long r, long long u, float mu,
                                        float rs, float xh[8])
{
    const long long nb = blocks_of(a.dim);
    decode8(load_codes(a.codes + (r * nb * kBlockPacks + u) * kPack),
            a.exps[r * nb + u / kBlockPacks], xh);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        xh[j] = (xh[j] - mu) * rs;
}

// dx by two passes over a row, the second from L2.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kThreads) saved_dx_kernel(const SavedGrad a)
{
    __shared__ __align__(16) float sm[2 * 2 * 32];
    GroupOf block = group_of(Group{5, kThreads / 32}, sm, 1);
    const T *const dy = static_cast<const T *>(a.dy);
    const W *const gamma = static_cast<const W *>(a.gamma);
    const long long packs = (a.dim + kPack - 1) / kPack;
    const float n = (float)a.dim;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float mu = a.mean[r], rs = a.rstd[r];
        Sums<2> s{};
        for (long long u = threadIdx.x; u < packs; u += kThreads) {
            const int there = in_pack(a.dim, u);
            float xh[8], w[8], g[8];
            normal8(a, r, u, mu, rs, xh);
            load8<T, VEC>(dy + r * a.dim + u * kPack, there, w);
            weights8<W, VEC>(gamma, u * kPack, there, 1.0f, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j < there) {
                    w[j] *= g[j];
                    s.v[0] += w[j];
                    s.v[1] = fmaf(w[j], xh[j], s.v[1]);
                }
            }
        }
        s = group_sum<true, 2>(s, block);
        const float m0 = s.v[0] / n, m1 = s.v[1] / n;
        for (long long u = threadIdx.x; u < packs; u += kThreads) {
            const int there = in_pack(a.dim, u);
            float xh[8], w[8], g[8];
            normal8(a, r, u, mu, rs, xh);
            load8<T, VEC>(dy + r * a.dim + u * kPack, there, w);
            weights8<W, VEC>(gamma, u * kPack, there, 1.0f, g);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = rs * (fmaf(w[j], g[j], -m0) - xh[j] * m1);
            store8<T, VEC>(static_cast<T *>(a.dx) + r * a.dim + u * kPack, there, w);
        }
    }
}

// Partial sums of dgamma and dbeta: a thread adds 8 columns over a stretch of rows.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) saved_weights_kernel(const SavedGrad a)
{
    const T *const dy = static_cast<const T *>(a.dy);
    const long long lo = blockIdx.y * a.stretch, hi = min(lo + a.stretch, a.rows);
    const long long packs = (a.dim + kPack - 1) / kPack;
    for (long long u = (long long)blockIdx.x * kThreads + threadIdx.x; u < packs;
         u += (long long)gridDim.x * kThreads) {
        const int there = in_pack(a.dim, u);
        float g[8] = {}, b[8] = {};
        for (long long r = lo; r < hi; ++r) {
            float xh[8], d[8];
            normal8(a, r, u, a.mean[r], a.rstd[r], xh);
            load8<T, VEC>(dy + r * a.dim + u * kPack, there, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] = fmaf(d[j], xh[j], g[j]);
                b[j] += d[j];
            }
        }
        float *const out = a.part + 2LL * blockIdx.y * a.dim + u * kPack;
        store8<float, false>(out, there, g);
        store8<float, false>(out + a.dim, there, b);
    }
}

template <typename T, typename W, bool VEC>
cudaError_t saved_grad_rows(const SavedGrad &a, cudaStream_t st)
{
    if (a.rows > 0 && (a.dgamma || a.dbeta)) {
        const unsigned cols = (unsigned)std::min((a.dim / kPack + kThreads) / kThreads, 1LL << 16);
        saved_weights_kernel<T, VEC><<<dim3(cols, a.parts), kThreads, 0, st>>>(a);
    }
    if (a.rows > 0 && a.dx) // last: dx may be dy
        saved_dx_kernel<T, W, VEC><<<grid_of(a.rows, 8), kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && (a.dgamma || a.dbeta))
        e = join_parts<W>(Join{a.part, a.parts, a.dim, a.dgamma, a.dbeta, a.accumulate}, false,
                          st);
    return e;
}

template <typename T, typename W> rra_status saved_grad(SavedGrad a, cudaStream_t st)
{
    a.stretch = std::max(16LL, (a.rows + 127) / 128);
    a.parts = (int)((a.rows + a.stretch - 1) / a.stretch);
    std::unique_lock<std::mutex> lk;
    if (a.dgamma || a.dbeta) {
        unsigned char *ws = nullptr;
        const rra_status r =
            op_scratch(st, kScratchHead + sizeof(float) * 2 * a.parts * a.dim, lk, &ws);
        if (r != RRA_OK)
            return r;
        a.part = reinterpret_cast<float *>(ws + kScratchHead);
    }
    return launched(whole_packs<T>(a.dim, {a.dy, a.dx, a.gamma})
                        ? saved_grad_rows<T, W, true>(a, st)
                        : saved_grad_rows<T, W, false>(a, st));
}

// ---------------------------------------------------------------- calls

constexpr size_t kMostRows = (size_t)1 << 40, kMostDim = (size_t)1 << 31;

bool valid_sizes(size_t rows, size_t dim, rra_dtype t, rra_dtype w)
{
    // (fp32 rows are the largest arrays, codes of short rows aside)
    return valid_dt(t) && valid_dt(w) && dim > 0 && dim <= kMostDim && rows <= kMostRows &&
           holdable(rows, dim, 4) && holdable(rows, (size_t)blocks_of((long long)dim) * kBlock, 1);
}

// Do two of `outs` overlap, or one of them one of `ins`?
template <size_t N, size_t M> bool clash(const Span (&outs)[N], const Span (&ins)[M])
{
    for (size_t i = 0; i < N; ++i) {
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return true;
        for (const Span &in : ins)
            if (overlap(outs[i].p, outs[i].bytes, in.p, in.bytes))
                return true;
    }
    return false;
}

// fn<T, W>::call for the types of a call.
template <template <typename, typename> class F, typename A>
rra_status by_types(rra_dtype t, rra_dtype w, const A &a, cudaStream_t st)
{
    if (t == RRA_F32)
        return F<float, float>::call(a, st);
    if (t == RRA_F16)
        return w == RRA_F16 ? F<__half, __half>::call(a, st) : F<__half, float>::call(a, st);
    return w == RRA_BF16 ? F<__nv_bfloat16, __nv_bfloat16>::call(a, st)
                         : F<__nv_bfloat16, float>::call(a, st);
}

template <typename T, typename W> struct SaveCall {
    static rra_status call(const Save &a, cudaStream_t st) { return save<T, W>(a, st); }
};
template <typename T, typename W> struct RestoreCall {
    static rra_status call(const Restore &a, cudaStream_t st) { return restore<T, W>(a, st); }
};
template <typename T, typename W> struct SavedGradCall {
    static rra_status call(const SavedGrad &a, cudaStream_t st) { return saved_grad<T, W>(a, st); }
};

} // namespace
} // namespace rra

extern "C" rra_status rra_layer_norm_save(const void *x, const void *gamma, const void *beta,
                                          size_t rows, size_t dim, rra_dtype dtype,
                                          rra_dtype weight_t, float eps, void *y, int8_t *exps,
                                          int8_t *codes, float *mean, float *rstd, void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t) || !(eps >= 0.0f))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es;
    if (rows > 0 && (!x || !y || !exps || !codes || !mean || !rstd))
        return RRA_ERR_INVALID;
    if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(gamma, ws) ||
        !aligned_to(beta, ws) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(codes, 16) || !apart_or_same(x, bytes, y, bytes))
        return RRA_ERR_INVALID;
    const Span outs[] = {{y, bytes},
                         {exps, exps_bytes(rows, dim)},
                         {codes, codes_bytes(rows, dim)},
                         {mean, rows * 4},
                         {rstd, rows * 4}};
    const Span ins[] = {{x == y ? nullptr : x, bytes}, {gamma, dim * ws}, {beta, dim * ws}};
    if (clash(outs, ins))
        return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    if (rows == 0)
        return RRA_OK;
    const Save a{x,    gamma, beta, (long long)rows, (long long)dim, eps, y, exps,
                 codes, mean,  rstd, {}};
    return by_types<SaveCall>(dtype, weight_t, a, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" rra_status rra_layer_norm_restore(const int8_t *exps, const int8_t *codes,
                                             const float *mean, const float *rstd,
                                             const void *gamma, const void *beta, size_t rows,
                                             size_t dim, rra_dtype dtype, rra_dtype weight_t,
                                             void *y, void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es;
    if (rows > 0 && (!exps || !codes || !y))
        return RRA_ERR_INVALID;
    if (!aligned_to(y, es) || !aligned_to(gamma, ws) || !aligned_to(beta, ws) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(codes, 16))
        return RRA_ERR_INVALID;
    const Span outs[] = {{y, bytes}};
    const Span ins[] = {{exps, exps_bytes(rows, dim)}, {codes, codes_bytes(rows, dim)},
                        {mean, rows * 4},              {rstd, rows * 4},
                        {gamma, dim * ws},             {beta, dim * ws}};
    if (clash(outs, ins))
        return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    if (rows == 0)
        return RRA_OK;
    const Restore a{exps, codes, mean, rstd, gamma, beta, (long long)rows, (long long)dim, y, 1};
    return by_types<RestoreCall>(dtype, weight_t, a, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" rra_status rra_layer_norm_saved_grad(const void *dy, const int8_t *exps,
                                                const int8_t *codes, const void *gamma,
                                                const float *mean, const float *rstd, size_t rows,
                                                size_t dim, rra_dtype dtype, rra_dtype weight_t,
                                                void *dx, void *dgamma, void *dbeta,
                                                int accumulate, void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t) || (!dx && !dgamma && !dbeta))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es,
                 wb = dim * ws;
    if (rows > 0 && (!dy || !exps || !codes || !mean || !rstd))
        return RRA_ERR_INVALID;
    if (!aligned_to(dy, es) || !aligned_to(gamma, ws) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4) || !aligned_to(codes, 16) || !aligned_to(dx, es) ||
        !aligned_to(dgamma, ws) || !aligned_to(dbeta, ws) || !apart_or_same(dx, bytes, dy, bytes))
        return RRA_ERR_INVALID;
    const Span outs[] = {{dx == dy ? nullptr : dx, bytes}, {dgamma, wb}, {dbeta, wb}};
    const Span ins[] = {{dy, bytes},
                        {exps, exps_bytes(rows, dim)},
                        {codes, codes_bytes(rows, dim)},
                        {gamma, wb},
                        {mean, rows * 4},
                        {rstd, rows * 4}};
    if (clash(outs, ins))
        return RRA_ERR_INVALID;
    // in place: apart from the other inputs all the same
    if (dx == dy && any_overlap(ins[0], {ins[1], ins[2], ins[3], ins[4], ins[5]}))
        return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    const SavedGrad a{dy, exps,   codes, gamma,      mean,    rstd, (long long)rows, (long long)dim,
                      dx, dgamma, dbeta, accumulate, nullptr, 0,    0};
    return by_types<SavedGradCall>(dtype, weight_t, a, reinterpret_cast<cudaStream_t>(stream));
}
