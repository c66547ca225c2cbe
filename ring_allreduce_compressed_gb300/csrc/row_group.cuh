// row_group.cuh -- what layer_norm.cu and layer_norm_saved.cu share: rows held
// in registers by groups of lanes, sums over such a group, weights as fp32,
// packs staged in shared memory, partial rows of the weights' gradients joined.
#pragma once

#include "op_common.cuh"

namespace rra {
namespace {

// A row is held in registers by a group of lanes: 2^lg lanes of a warp, or
// all lanes of `warps` warps.  Lane i holds packs i, i + lanes, ... of V
// elements (V: the widest that every row's address allows), so x is read once
// and the variance is the mean of squares about the mean, not a difference.
// 32 elements a lane: a row's own sums, barriers and addresses are some 150
// instructions of every warp, and 16 a lane took 62 us where 32 take 49.
struct Group {
    int lg;    // one warp or less: 2^lg lanes
    int warps; // more
    __host__ __device__ int lanes() const { return warps > 1 ? 32 * warps : 1 << lg; }
};

// s / n for whole n of up to 2^16, where `inverse` is 1 / n correctly rounded
// (after P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990).  q is within 1.5 units of
// its last place, so the remainder s - q n, a multiple of that unit, is exact.
// The sum then misses s / n by less than 2^-45 of it before it is rounded, and no
// s / n is as near as that to the middle of two fp32 numbers (s has not the bits
// to lie on one, and is 2^-25 / n of it away at least): the result is the
// division's.  Below 2^-126 a tie may go to the other side.  Three instructions
// where a division takes some twenty of every warp of a row.
__device__ __forceinline__ float quotient(float s, float n, float inverse)
{
    const float q = s * inverse;
    const float r = fmaf(fmaf(-q, n, s), inverse, q);
    return r == r ? r : q; // (an infinite q)
}

// Sums over the lanes of a group; every lane gets them.  More than a warp:
// `at` holds 2 * 32 * N floats of the group's own, zero behind the warps'
// places, and `turn` alternates, so that one barrier a sum is enough: a warp
// that is a sum ahead writes elsewhere.
template <int N> struct Sums {
    float v[N];
};

struct GroupOf {
    int half;    // of the lanes that a row has in a warp
    int warps;   // of the group
    int warp;    // this one's number
    int barrier; // the group's
    float *at;
    int turn;
};

__device__ __forceinline__ GroupOf group_of(const Group &g, float *at, int barrier)
{
    return {1 << g.lg >> 1, g.warps, (int)(threadIdx.x / 32) % g.warps, barrier, at, 0};
}

template <bool MULTI, int N>
__device__ __forceinline__ Sums<N> group_sum(Sums<N> s, GroupOf &g)
{
    if constexpr (!MULTI) {
        for (int o = g.half; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n)
                s.v[n] += __shfl_xor_sync(kFull, s.v[n], o);
        return s;
    }
    const int lane = threadIdx.x % 32;
    float *const at = g.at + g.turn * (32 * N);
    g.turn ^= 1;
    if constexpr (N == 2) { // each half warp takes one of the two on
        const float mine = lane < 16 ? s.v[0] : s.v[1], other = lane < 16 ? s.v[1] : s.v[0];
        float t = mine + __shfl_xor_sync(kFull, other, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            t += __shfl_xor_sync(kFull, t, o);
        if (lane % 16 == 0)
            at[lane * 2 + g.warp] = t;
    } else {
        s.v[0] = warp_sum(s.v[0]);
        if (lane == 0)
            at[g.warp] = s.v[0];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(g.barrier), "r"(32 * g.warps) : "memory");
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (g.warps <= 8) {
            const float4 a = *reinterpret_cast<const float4 *>(at + n * 32);
            s.v[n] = (a.x + a.y) + (a.z + a.w);
            if (g.warps > 4) {
                const float4 b = *reinterpret_cast<const float4 *>(at + n * 32 + 4);
                s.v[n] += (b.x + b.y) + (b.z + b.w);
            }
        } else {
            s.v[n] = warp_sum(at[n * 32 + lane]);
        }
    }
    return s;
}

// V weights as fp32, or `none` where there is no array.
template <typename W, int V>
__device__ __forceinline__ void load_weights(const W *p, int c, float none,
                                             typename Values<V>::E (&v)[Values<V>::N])
{
    if (!p) {
#pragma unroll
        for (int n = 0; n < Values<V>::N; ++n)
            v[n] = Values<V>::all(none);
        return;
    }
    constexpr int U = V * sizeof(W) > 16 ? 16 / sizeof(W) : V; // of one load
    using P = Values<U>;
#pragma unroll
    for (int i = 0; i < V / U; ++i) {
        Raw<W, U> raw;
        raw.load(p + c + i * U);
#pragma unroll
        for (int n = 0; n < P::N; ++n)
            v[i * P::N + n] = P::get(raw, n);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_vals(T *p, const typename Values<V>::E (&e)[Values<V>::N])
{
    float f[V];
    Values<V>::to_array(e, f);
    T o[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        o[j] = from_f32<T>(f[j]);
    store_values<T, V>(p, o);
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

// One pack to shared memory, asynchronously where it has a size that can be.
template <typename T, int V> __device__ __forceinline__ void stage_pack(T *to, const T *from)
{
    constexpr int bytes = V * sizeof(T);
    if constexpr (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                     : "memory");
    else if constexpr (bytes >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from),
                     "n"(bytes)
                     : "memory");
    else
        *to = *from;
}

// Partial sums of dgamma and dbeta, [parts][2][dim], and where they go (either
// may be NULL).
struct Join {
    const float *part;
    int parts;
    long long dim;
    void *dgamma, *dbeta;
    int accumulate;
};

constexpr int kThreads = 256;

// Adds the partial rows: a block takes 32 columns of [dgamma, dbeta], 32 / V
// threads for each of its 8 V stretches of the partial rows.
template <typename W, int V> __global__ void __launch_bounds__(kThreads) join_kernel(const Join a)
{
    constexpr int kLanes = 32 / V, kStretches = kThreads / kLanes;
    __shared__ float sm[kStretches][33];
    dependents_wait();
    dependents_launch();
    const int t = threadIdx.x % kLanes, s = threadIdx.x / kLanes;
    const int lo = (int)((long long)a.parts * s / kStretches),
              hi = (int)((long long)a.parts * (s + 1) / kStretches);
    for (long long c0 = 32LL * blockIdx.x; c0 < 2 * a.dim; c0 += 32LL * gridDim.x) {
        float sum[V] = {};
        if (c0 + t * V < 2 * a.dim)
#pragma unroll 8
            for (int p = lo; p < hi; ++p) {
                const Pack<float, V> v = load_pack<float, V>(a.part + 2LL * p * a.dim + c0 + t * V);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    sum[j] += v.e[j];
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j)
            sm[s][t * V + j] = sum[j];
        __syncthreads();
        const long long c = c0 + threadIdx.x;
        if (threadIdx.x < 32 && c < 2 * a.dim) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kStretches; ++k)
                v += sm[k][threadIdx.x];
            W *const to = static_cast<W *>(c < a.dim ? a.dgamma : a.dbeta);
            const long long at = c < a.dim ? c : c - a.dim;
            if (to)
                to[at] = from_f32<W>(a.accumulate ? to_f32(to[at]) + v : v);
        }
    }
}

// behind: a kernel of the same call, launched before on `st`, wrote the parts.
template <typename W> cudaError_t join_parts(const Join &a, bool behind, cudaStream_t st)
{
    const unsigned grid = (unsigned)std::min((2 * a.dim + 31) / 32, 1LL << 20);
    const auto fn = a.dim % 4 == 0 ? join_kernel<W, 4> : join_kernel<W, 1>;
    if (!behind) { // nothing of this call to be chained to
        fn<<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
    return launch_chained(fn, dim3(grid), kThreads, st, a);
}

// Either apart or the same buffer.
inline bool apart_or_same(const void *a, size_t na, const void *b, size_t nb)
{
    return a == b || !overlap(a, na, b, nb);
}

} // namespace
} // namespace rra
