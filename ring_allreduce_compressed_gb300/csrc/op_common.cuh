// op_common.cuh -- what the training-step operators (grad_norm.cu,
// embedding.cu, layer_norm.cu) share: packs of elements read and written by
// one instruction, block reductions, argument checks and the scratch memory
// of a stream.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "rra.h"
#include "rra_device.cuh"

namespace rra {

int num_sms();

// ---------------------------------------------------------------- device

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v)
{
    return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// V consecutive elements that one load or store of V * sizeof(T) <= 16 bytes
// moves; the address is a multiple of that size.
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T e[V];
};

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T *p)
{
    return *reinterpret_cast<const Pack<T, V> *>(p);
}

// The same for 16 bytes, from L2 past L1.
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack_l2(const T *p)
{
    static_assert(sizeof(T) * V == 16, "a whole load");
    Pack<T, V> v;
    *reinterpret_cast<uint4 *>(&v) = __ldcg(reinterpret_cast<const uint4 *>(p));
    return v;
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &v)
{
    *reinterpret_cast<Pack<T, V> *>(p) = v;
}

// The same for results that the call does not read again: they leave L2 first.
template <typename T, int V>
__device__ __forceinline__ void stream_pack(T *p, const Pack<T, V> &v)
{
    if constexpr (sizeof(T) * V == 16)
        __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&v));
    else
        store_pack<T, V>(p, v);
}

// A pack as the words that it was loaded in; elements are taken out where they
// are used, so that a pack in flight costs its own size in registers.
template <typename T, int V> struct Raw {
    static constexpr int kWords = V * sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = 0;
    }
    __device__ __forceinline__ void load(const T *p)
    {
        const Pack<uint32_t, kWords> q =
            load_pack<uint32_t, kWords>(reinterpret_cast<const uint32_t *>(p));
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = q.e[i];
    }
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[j]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
        else
            return __half2float(__ushort_as_half((unsigned short)(w[j / 2] >> (16 * (j % 2)))));
    }
};
template <typename T> struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void clear() { v = from_f32<T>(0.0f); }
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
};

// V elements at p in stores (loads) of at most 16 bytes; p is a multiple of
// the lesser of V * sizeof(T) and 16 bytes.
template <typename T, int V> __device__ __forceinline__ void store_values(T *p, const T (&v)[V])
{
    constexpr int W = V * sizeof(T) > 16 ? 16 / sizeof(T) : V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        Pack<T, W> q;
#pragma unroll
        for (int j = 0; j < W; ++j)
            q.e[j] = v[i + j];
        store_pack<T, W>(p + i, q);
    }
}

template <typename T, int V> __device__ __forceinline__ void load_values(const T *p, T (&v)[V])
{
    constexpr int W = V * sizeof(T) > 16 ? 16 / sizeof(T) : V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        const Pack<T, W> q = load_pack<T, W>(p + i);
#pragma unroll
        for (int j = 0; j < W; ++j)
            v[i + j] = q.e[j];
    }
}

// Values of a pack as the arithmetic takes them: pairs for the paired fp32
// instructions (two IEEE operations each), or a single float.
using Pair = unsigned long long;

__device__ __forceinline__ Pair pair_of(float lo, float hi)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void halves(Pair p, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum_of(float a) { return a; }
__device__ __forceinline__ float sum_of(Pair p)
{
    float lo, hi;
    halves(p, lo, hi);
    return lo + hi;
}

// The values of a pack of V elements: N of type E.
template <int V> struct Values {
    using E = Pair;
    static constexpr int N = V / 2;
    static __device__ __forceinline__ E all(float v) { return pair_of(v, v); }
    template <typename R> static __device__ __forceinline__ E get(const R &raw, int n)
    {
        return pair_of(raw.get(2 * n), raw.get(2 * n + 1));
    }
    static __device__ __forceinline__ void to_array(const E (&e)[N], float (&v)[V])
    {
#pragma unroll
        for (int n = 0; n < N; ++n)
            halves(e[n], v[2 * n], v[2 * n + 1]);
    }
};
template <> struct Values<1> {
    using E = float;
    static constexpr int N = 1;
    static __device__ __forceinline__ E all(float v) { return v; }
    template <typename R> static __device__ __forceinline__ E get(const R &raw, int)
    {
        return raw.get(0);
    }
    static __device__ __forceinline__ void to_array(const E (&e)[1], float (&v)[1]) { v[0] = e[0]; }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The next kernel of the stream may start its blocks now, if it was launched
// by launch_chained; what it reads of this one it waits for.
__device__ __forceinline__ void dependents_launch()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Until the kernel before this one has ended and its writes are visible.
__device__ __forceinline__ void dependents_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- host

// A kernel launched so may start before the one ahead of it in the stream has
// ended, if that one lets it in (dependents_launch).  It waits for that one
// (dependents_wait) before it touches memory, except where a comment says why
// it need not: then the one ahead lets it in only when it has itself waited.
// No kernel ends before the ones ahead of it, so what is behind a call finds
// all of the call done.  A launch costs 1 to 2 us less so.
template <typename... P, typename... A>
cudaError_t launch_chained_smem(void (*fn)(P...), dim3 grid, int threads, int smem,
                                cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*fn)(P...), dim3 grid, int threads, cudaStream_t st, A... args)
{
    return launch_chained_smem(fn, grid, threads, 0, st, args...);
}

inline bool valid_dt(rra_dtype t) { return t == RRA_F32 || t == RRA_F16 || t == RRA_BF16; }

// Is an array of a * b elements of es bytes one that a memory could hold?  (64 TB;
// the product of sizes that are each in range may not fit 64 bits.)
inline bool holdable(size_t a, size_t b, size_t es)
{
    return a == 0 || b <= ((size_t)1 << 46) / es / a;
}

// Do [a, a + na) and [b, b + nb) share a byte?
inline bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

__host__ __device__ inline bool aligned_to(const void *p, size_t n)
{
    return reinterpret_cast<uintptr_t>(p) % n == 0;
}

// Are packs of `bytes` bytes aligned in every row, rows of row_bytes lying one
// behind the other from `base` on?
__host__ __device__ inline bool pack_fits(const void *base, size_t row_bytes, size_t bytes)
{
    return aligned_to(base, bytes) && row_bytes % bytes == 0;
}

// Scratch memory of the operators, one buffer per stream (the per-thread
// default stream: one per thread): calls on one stream run in order and share
// it, calls on different streams never do.  Its first kScratchHead bytes are
// zero between calls (tickets that their last user clears).  The lock in `lk`
// is held until the launches of the call are queued.  A buffer that has become
// too small, or whose stream is gone, is freed once the device's work is done,
// but kept if a captured graph may hold its address; sizes at least double.
// RRA_ERR_INVALID: the buffer would have to grow while the stream is being
// captured; RRA_ERR_NOMEM, RRA_ERR_CUDA.
constexpr size_t kScratchHead = 256;
rra_status op_scratch(cudaStream_t st, size_t bytes, std::unique_lock<std::mutex> &lk,
                      unsigned char **out);

// Allows a kernel `smem` bytes of dynamic shared memory, and clusters of more
// than 8 blocks: once per kernel and device, not on every launch.
cudaError_t op_allow(const void *fn, int smem, bool large_clusters = false);

inline rra_status launched(cudaError_t e) { return e == cudaSuccess ? RRA_OK : RRA_ERR_CUDA; }

} // namespace rra
