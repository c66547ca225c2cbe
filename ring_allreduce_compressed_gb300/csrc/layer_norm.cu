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
#include <initializer_list>

#include "op_common.cuh"

namespace rra {
namespace {

// A row is held in registers by a group of lanes: 2^lg lanes of a warp, or
// all lanes of `warps` warps.  Lane i holds packs i, i + lanes, ... of V
// elements (V: the widest that every row's address allows), so x is read once
// and the variance is the mean of squares about the mean, not a difference.
struct Group {
    int lg;    // one warp or less: 2^lg lanes
    int warps; // more
    __host__ __device__ int lanes() const { return warps > 1 ? 32 * warps : 1 << lg; }
};

// Sums v over the group; every lane gets it.  More than a warp: `sm` holds
// 2 * 32 * N floats of the group's own, and `turn` alternates, so that one
// barrier a sum is enough: a warp that is a sum ahead writes elsewhere.
template <int N> struct Sums {
    float v[N];
};

template <bool MULTI, int N>
__device__ __forceinline__ Sums<N> group_sum(Sums<N> s, const Group &g, float *sm, int &turn,
                                             int barrier)
{
    const int lane = threadIdx.x % 32;
    if constexpr (!MULTI) {
        for (int o = 1 << g.lg >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n)
                s.v[n] += __shfl_xor_sync(kFull, s.v[n], o);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
            s.v[n] = warp_sum(s.v[n]);
        float *const at = sm + turn * (32 * N);
        turn ^= 1;
        const int w = threadIdx.x / 32 % g.warps;
        if (lane == 0)
#pragma unroll
            for (int n = 0; n < N; ++n)
                at[n * 32 + w] = s.v[n];
        asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * g.warps) : "memory");
#pragma unroll
        for (int n = 0; n < N; ++n)
            s.v[n] = warp_sum(lane < g.warps ? at[n * 32 + lane] : 0.0f);
    }
    return s;
}

// V values of type W as fp32, or `none` where there is no array.
template <typename W, int V>
__device__ __forceinline__ void load_weights(const W *p, long long c, float none, float (&v)[V])
{
    if (!p) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = none;
        return;
    }
    W w[V];
    load_values<W, V>(p + c, w);
#pragma unroll
    for (int j = 0; j < V; ++j)
        v[j] = to_f32(w[j]);
}

// ---------------------------------------------------------------- forward

struct Fwd {
    const void *x, *gamma, *beta;
    long long rows, dim;
    float eps;
    void *y;
    float *mean, *rstd;
    Group g;
};

constexpr int kFwdThreads = 256; // of a block, where a group is no more than that

template <typename T, typename W, int V, int K, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 1024 : kFwdThreads, MULTI ? 1 : 4) norm_kernel(const Fwd a)
{
    __shared__ float sm[MULTI ? 2 * 32 : 1]; // a group of several warps is a block
    const T *const x = static_cast<const T *>(a.x);
    T *const y = static_cast<T *>(a.y);
    const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                static_cast<const W *>(a.beta);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, groups = blockDim.x / lanes;
    const long long units = a.dim / V;
    const float n = (float)a.dim;
    int turn = 0;
    for (long long base = (long long)blockIdx.x * groups; base < a.rows;
         base += (long long)gridDim.x * groups) {
        const long long r = base + threadIdx.x / lanes;
        const bool on = r < a.rows; // (every lane takes part in the sums)
        Raw<T, V> v[K];
        Sums<1> s{};
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && li + k * lanes < units)
                v[k].load(x + r * a.dim + (long long)(li + k * lanes) * V);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && li + k * lanes < units)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    s.v[0] += v[k].get(j);
        const float mu = group_sum<MULTI, 1>(s, a.g, sm, turn, 1).v[0] / n;
        s.v[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && li + k * lanes < units)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = v[k].get(j) - mu;
                    s.v[0] = fmaf(d, d, s.v[0]);
                }
        const float rs = 1.0f / sqrtf(group_sum<MULTI, 1>(s, a.g, sm, turn, 1).v[0] / n + a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && li + k * lanes < units) {
                const long long c = (long long)(li + k * lanes) * V;
                float g[V], b[V];
                load_weights<W, V>(gamma, c, 1.0f, g);
                load_weights<W, V>(beta, c, 0.0f, b);
                T o[V];
#pragma unroll
                for (int j = 0; j < V; ++j)
                    o[j] = from_f32<T>(fmaf((v[k].get(j) - mu) * rs, g[j], b[j]));
                store_values<T, V>(y + r * a.dim + c, o);
            }
        if (on && li == 0) {
            if (a.mean)
                a.mean[r] = mu;
            if (a.rstd)
                a.rstd[r] = rs;
        }
    }
}

// Rows that no block holds: three passes over each, the last two from L2.
constexpr int kLongThreads = 1024;

template <int N> __device__ __forceinline__ Sums<N> block_sums(Sums<N> s, float *sm, int &turn)
{
    return group_sum<true, N>(s, Group{5, kLongThreads / 32}, sm, turn, 1);
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const Fwd a)
{
    __shared__ float sm[2 * 32];
    int turn = 0;
    const float n = (float)a.dim;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const p = static_cast<const T *>(a.x) + r * a.dim;
        const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                    static_cast<const W *>(a.beta);
        Sums<1> s{};
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads)
            s.v[0] += to_f32(p[c]);
        const float mu = block_sums<1>(s, sm, turn).v[0] / n;
        s.v[0] = 0.0f;
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float d = to_f32(p[c]) - mu;
            s.v[0] = fmaf(d, d, s.v[0]);
        }
        const float rs = 1.0f / sqrtf(block_sums<1>(s, sm, turn).v[0] / n + a.eps);
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float g = gamma ? to_f32(gamma[c]) : 1.0f, b = beta ? to_f32(beta[c]) : 0.0f;
            static_cast<T *>(a.y)[r * a.dim + c] =
                from_f32<T>(fmaf((to_f32(p[c]) - mu) * rs, g, b));
        }
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = mu;
            if (a.rstd)
                a.rstd[r] = rs;
        }
    }
}

inline unsigned grid_of(long long items, int per_sm)
{
    return (unsigned)std::max(1LL, std::min(items, (long long)num_sms() * per_sm));
}

// Group whose lanes hold `units` packs, K each.
inline Group group_for(long long units, int K)
{
    Group g{0, 1};
    while (g.lg < 5 && ((long long)K << g.lg) < units)
        ++g.lg;
    g.warps = (int)((units + 32 * K - 1) / (32 * K));
    return g;
}

constexpr int kShort = 8, kHeld = 32; // elements that a lane holds

template <typename T, typename W, int V> void forward_packs(Fwd a, cudaStream_t st)
{
    const long long units = a.dim / V;
    if (a.dim > 1024LL * kHeld) {
        norm_long_kernel<T, W><<<grid_of(a.rows, 2), kLongThreads, 0, st>>>(a);
    } else if (a.dim <= 32 * kHeld) {
        // a warp or a part of one; few elements a lane for short rows
        const bool few = a.dim <= 32 * kShort;
        a.g = group_for(units, (few ? kShort : kHeld) / V);
        const int per_block = kFwdThreads / a.g.lanes();
        const unsigned grid = grid_of((a.rows + per_block - 1) / per_block, 16);
        if (few)
            norm_kernel<T, W, V, kShort / V, false><<<grid, kFwdThreads, 0, st>>>(a);
        else
            norm_kernel<T, W, V, kHeld / V, false><<<grid, kFwdThreads, 0, st>>>(a);
    } else {
        a.g = group_for(units, kHeld / V);
        const int threads = 32 * a.g.warps;
        norm_kernel<T, W, V, kHeld / V, true>
            <<<grid_of(a.rows, 2048 / threads), threads, 0, st>>>(a);
    }
}

// Do packs of V elements of x (and of all rows), and of the weights, fit?
template <typename T, typename W, int V>
bool packs_fit(long long dim, std::initializer_list<const void *> rows,
               std::initializer_list<const void *> weights)
{
    for (const void *p : rows)
        if (p && !pack_fits(p, (size_t)dim * sizeof(T), V * sizeof(T)))
            return false;
    for (const void *p : weights)
        if (p && !aligned_to(p, std::min(V * sizeof(W), (size_t)16)))
            return false;
    return true;
}

template <typename T, typename W> void forward(const Fwd &a, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (packs_fit<T, W, V>(a.dim, {a.x, a.y}, {a.gamma, a.beta}))
        forward_packs<T, W, V>(a, st);
    else
        forward_packs<T, W, 1>(a, st);
}

// ---------------------------------------------------------------- backward

// A lane keeps its columns' sums of dgamma and dbeta over all rows of its
// group in registers.  At the end the groups of a block add theirs in shared
// memory, in order, and the block leaves one partial row of each, which
// join_kernel adds.  The next row's packs are read while a row is worked on.
struct Bwd {
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    long long rows, dim;
    void *dx, *dgamma, *dbeta;
    int accumulate;
    float *part; // [parts][2][dim]
    int parts;
    Group g;
};

constexpr int kBwdThreads = 768; // most of a block: 80 registers a thread

// Elements that a lane holds: 32 bytes of x.
template <typename T, int V> constexpr int kBwdHeld = V > 1 ? 32 / sizeof(T) : 8;

template <typename T, typename W, int V, bool MULTI>
__global__ void __launch_bounds__(kBwdThreads) norm_grad_kernel(const Bwd a)
{
    constexpr int K = kBwdHeld<T, V> / V;
    extern __shared__ __align__(16) float sums[];                // [2][dim], if there are several groups
    __shared__ float sm[MULTI ? 24 * 2 * 32 : 1][2]; // of every group
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    T *const dx = static_cast<T *>(a.dx);
    const W *const gamma = static_cast<const W *>(a.gamma);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, group = threadIdx.x / lanes,
              groups = blockDim.x / lanes;
    const long long units = a.dim / V, step = (long long)gridDim.x * groups;
    const float n = (float)a.dim;
    float *const own = MULTI ? sm[group * 64] : sm[0];
    int turn = 0;
    float dg[K][V] = {}, db[K][V] = {};
    Raw<T, V> vx[K], vd[K], nx[K], nd[K];
    float next_mu = 0.0f, next_rs = 0.0f;

    long long base = (long long)blockIdx.x * groups;
    const auto read = [&](long long r) {
        if (r < a.rows) {
            next_mu = a.mean[r];
            next_rs = a.rstd[r];
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (r < a.rows && li + k * lanes < units) {
                const long long at = r * a.dim + (long long)(li + k * lanes) * V;
                nx[k].load(x + at);
                nd[k].load(dy + at);
            }
    };
    read(base + group);
    for (; base < a.rows; base += step) {
        const long long r = base + group;
        const bool on = r < a.rows;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            vx[k] = nx[k];
            vd[k] = nd[k];
        }
        const float mu = next_mu, rs = next_rs;
        read(r + step);
        Sums<2> s{};
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && li + k * lanes < units) {
                float g[V];
                load_weights<W, V>(gamma, (long long)(li + k * lanes) * V, 1.0f, g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = vd[k].get(j), xh = (vx[k].get(j) - mu) * rs, w = d * g[j];
                    s.v[0] += w;
                    s.v[1] = fmaf(w, xh, s.v[1]);
                    dg[k][j] = fmaf(d, xh, dg[k][j]);
                    db[k][j] += d;
                }
            }
        if (!dx)
            continue;
        s = group_sum<MULTI, 2>(s, a.g, own, turn, 1 + group);
        const float m0 = s.v[0] / n, m1 = s.v[1] / n;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && li + k * lanes < units) {
                const long long c = (long long)(li + k * lanes) * V;
                float g[V];
                load_weights<W, V>(gamma, c, 1.0f, g);
                T o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (vx[k].get(j) - mu) * rs;
                    o[j] = from_f32<T>(rs * (fmaf(vd[k].get(j), g[j], -m0) - xh * m1));
                }
                store_values<T, V>(dx + r * a.dim + c, o);
            }
    }
    dependents_launch();
    if (!a.dgamma && !a.dbeta)
        return;

    float *const out = a.part + 2LL * blockIdx.x * a.dim;
    if constexpr (!MULTI) { // the warp's groups first
        for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dg[k][j] += __shfl_xor_sync(kFull, dg[k][j], o);
                    db[k][j] += __shfl_xor_sync(kFull, db[k][j], o);
                }
    }
    const int holders = MULTI ? groups : blockDim.x / 32, me = MULTI ? group : threadIdx.x / 32;
    const bool holds = MULTI || threadIdx.x % 32 < lanes;
    float *const to = holders > 1 ? sums : out;
    for (int h = 0; h < holders; ++h) {
        if (h == me && holds)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (li + k * lanes < units) {
                    const long long c = (long long)(li + k * lanes) * V;
                    if (h > 0) {
                        float p[V], q[V];
                        load_values<float, V>(to + c, p);
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            dg[k][j] += p[j];
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            q[j] = to[a.dim + c + j];
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            db[k][j] += q[j];
                    }
                    store_values<float, V>(to + c, dg[k]);
                    store_values<float, V>(to + a.dim + c, db[k]);
                }
        if (holders > 1)
            __syncthreads();
    }
    if (holders > 1)
        for (long long c = threadIdx.x; c < 2 * a.dim; c += blockDim.x)
            out[c] = sums[c];
}

constexpr int kThreads = 256;

// Long rows: dx by three passes over the row, the weights' sums by columns.
template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads) dx_long_kernel(const Bwd a)
{
    __shared__ float sm[2 * 2 * 32];
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    const W *const gamma = static_cast<const W *>(a.gamma);
    int turn = 0;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float mu = a.mean[r], rs = a.rstd[r], n = (float)a.dim;
        Sums<2> s{};
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float w = to_f32(dy[r * a.dim + c]) * (gamma ? to_f32(gamma[c]) : 1.0f);
            s.v[0] += w;
            s.v[1] = fmaf(w, (to_f32(x[r * a.dim + c]) - mu) * rs, s.v[1]);
        }
        s = block_sums<2>(s, sm, turn);
        const float m0 = s.v[0] / n, m1 = s.v[1] / n;
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float g = gamma ? to_f32(gamma[c]) : 1.0f;
            const float xh = (to_f32(x[r * a.dim + c]) - mu) * rs;
            static_cast<T *>(a.dx)[r * a.dim + c] =
                from_f32<T>(rs * (fmaf(to_f32(dy[r * a.dim + c]), g, -m0) - xh * m1));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) weight_long_kernel(const Bwd a, long long stretch)
{
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    const long long lo = blockIdx.y * stretch, hi = min(lo + stretch, a.rows);
    for (long long c = (long long)blockIdx.x * kThreads + threadIdx.x; c < a.dim;
         c += (long long)gridDim.x * kThreads) {
        float g = 0.0f, b = 0.0f;
#pragma unroll 4
        for (long long r = lo; r < hi; ++r) {
            const float d = to_f32(dy[r * a.dim + c]);
            g = fmaf(d, (to_f32(x[r * a.dim + c]) - a.mean[r]) * a.rstd[r], g);
            b += d;
        }
        a.part[2LL * blockIdx.y * a.dim + c] = g;
        a.part[(2LL * blockIdx.y + 1) * a.dim + c] = b;
    }
}

// Adds the partial rows: a block takes 32 columns of [dgamma, dbeta], its
// warps a stretch of the partial rows each.
constexpr int kWarps = kThreads / 32;

template <typename W> __global__ void __launch_bounds__(kThreads) join_kernel(const Bwd a)
{
    __shared__ float sm[kWarps][32];
    dependents_wait();
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const int lo = (int)((long long)a.parts * w / kWarps),
              hi = (int)((long long)a.parts * (w + 1) / kWarps);
    for (long long c0 = 32LL * blockIdx.x; c0 < 2 * a.dim; c0 += 32LL * gridDim.x) {
        const long long c = c0 + lane;
        float s = 0.0f;
        if (c < 2 * a.dim)
#pragma unroll 8
            for (int p = lo; p < hi; ++p)
                s += a.part[2LL * p * a.dim + c];
        __syncthreads();
        sm[w][lane] = s;
        __syncthreads();
        if (w == 0 && c < 2 * a.dim) {
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
                s += sm[k][lane];
            W *const to = static_cast<W *>(c < a.dim ? a.dgamma : a.dbeta);
            const long long at = c < a.dim ? c : c - a.dim;
            if (to)
                to[at] = from_f32<W>(a.accumulate ? to_f32(to[at]) + s : s);
        }
    }
}

// Launch shape of the backward pass, from which its scratch follows.
struct BwdShape {
    Group g;
    int groups; // of a block
    int parts;  // partial rows: blocks of the first kernel
    bool packs, held;
};

template <typename T, typename W> BwdShape backward_shape(const Bwd &a)
{
    constexpr int V = 16 / sizeof(T);
    BwdShape s;
    s.packs = packs_fit<T, W, V>(a.dim, {a.dy, a.x, a.dx}, {a.gamma});
    const int held = s.packs ? kBwdHeld<T, V> : kBwdHeld<T, 1>;
    s.held = a.dim <= (long long)kBwdThreads * held;
    if (s.held) {
        s.g = group_for(s.packs ? a.dim / V : a.dim, held / (s.packs ? V : 1));
        // one block per SM; groups of a block only where rows are many
        const long long most = std::max(1, (s.g.warps > 1 ? kBwdThreads : kThreads) / s.g.lanes());
        s.groups = (int)std::max(1LL, std::min(most, a.rows / num_sms()));
        if (s.g.warps == 1) { // whole warps
            const int in_warp = 32 / s.g.lanes();
            s.groups = std::max(1, s.groups / in_warp) * in_warp;
        }
        const long long blocks = (a.rows + s.groups - 1) / s.groups;
        s.parts = (int)std::min(blocks, (long long)num_sms() * (s.g.warps == 1 ? 3 : 1));
    } else {
        const long long stretch = std::max(16LL, (a.rows + 127) / 128);
        s.groups = 1;
        s.parts = (int)((a.rows + stretch - 1) / stretch);
    }
    return s;
}

template <typename T, typename W, int V> cudaError_t held_rows(Bwd a, const BwdShape &s,
                                                               cudaStream_t st)
{
    const int threads = s.groups * s.g.lanes();
    const bool several = s.g.warps > 1 ? s.groups > 1 : threads > 32;
    const int smem = several ? (int)(8 * a.dim) : 0;
    const auto fn = s.g.warps > 1 ? norm_grad_kernel<T, W, V, true> : norm_grad_kernel<T, W, V, false>;
    if (smem > 32768) {
        const cudaError_t e =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    fn<<<s.parts, threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename W> cudaError_t backward(Bwd a, const BwdShape &s, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    a.g = s.g;
    a.parts = s.parts;
    if (a.rows > 0) {
        if (s.held) {
            e = s.packs ? held_rows<T, W, 16 / sizeof(T)>(a, s, st) : held_rows<T, W, 1>(a, s, st);
        } else {
            if (a.dgamma || a.dbeta) {
                const unsigned cols =
                    (unsigned)std::min((a.dim + kThreads - 1) / kThreads, 1LL << 16);
                const long long stretch = std::max(16LL, (a.rows + 127) / 128);
                weight_long_kernel<T><<<dim3(cols, s.parts), kThreads, 0, st>>>(a, stretch);
            }
            if (a.dx) // last: dx may be dy or x
                dx_long_kernel<T, W><<<grid_of(a.rows, 2), kLongThreads, 0, st>>>(a);
            e = cudaGetLastError();
        }
    }
    if (e != cudaSuccess || (!a.dgamma && !a.dbeta))
        return e;
    const unsigned grid = (unsigned)std::min((2 * a.dim + 31) / 32, 1LL << 20);
    if (a.rows == 0) {
        join_kernel<W><<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
    return launch_chained(join_kernel<W>, dim3(grid), kThreads, st, a);
}

template <typename T, typename W> rra_status backward_call(Bwd a, cudaStream_t st)
{
    const BwdShape s = backward_shape<T, W>(a);
    std::unique_lock<std::mutex> lk;
    if (a.dgamma || a.dbeta) {
        unsigned char *ws = nullptr;
        const rra_status r =
            op_scratch(st, kScratchHead + sizeof(float) * 2 * s.parts * a.dim, lk, &ws);
        if (r != RRA_OK)
            return r;
        a.part = reinterpret_cast<float *>(ws + kScratchHead);
    }
    return launched(backward<T, W>(a, s, st));
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
    const Fwd a{x, gamma, beta, (long long)rows, (long long)dim, eps, y, mean, rstd, {}};
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
    const Bwd a{dy, x,  gamma,  mean,  rstd,       (long long)rows, (long long)dim,
                dx, dgamma, dbeta, accumulate, nullptr,         0,
                {}};
    if (dtype == RRA_F32)
        return backward_call<float, float>(a, st);
    if (dtype == RRA_F16 && weight_t == RRA_F16)
        return backward_call<__half, __half>(a, st);
    if (dtype == RRA_F16)
        return backward_call<__half, float>(a, st);
    if (weight_t == RRA_BF16)
        return backward_call<__nv_bfloat16, __nv_bfloat16>(a, st);
    return backward_call<__nv_bfloat16, float>(a, st);
}
