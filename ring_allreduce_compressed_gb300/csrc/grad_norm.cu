// grad_norm.cu -- rra_grad_norm and rra_grad_clip: the norm of a list of
// gradients taken as one vector, and their scaling to a largest norm.
//
//   norm = (sum |g|^p)^(1/p), p = 1 or 2, or max |g|
//   out  = g * min(1, max_norm / (norm + eps))
//
// Both passes are bound by memory: the norm reads every gradient once, the
// scaling reads it again and writes it.  The list is cut into tiles of 32 KB,
// so that a block works on one tensor at a time and short tensors leave no SM
// with more than its share.  The scaling's blocks start beside the norm's and
// have their first tile in registers when the norm is known.
//
// Measured: 16.2 us for 25 MiB of fp16 (7.7 us to read and write it once), 13.4
// in place; 1125 us for 10^9 elements in 40 tensors of bf16 and fp32 (three
// passes over 2.5 GB, 6.7 TB/s).  Of the 16.2 the norm takes 11 to 12, at a
// third of the memory's rate: 63 registers leave room for four blocks an SM, so
// the 800 tiles run as 608 and a second wave of 192.  Holding the 25 MiB in the SMs'
// shared memory in one cooperative launch took 20.6 us; tiles of 8 and 16 KB,
// 128 and 512 threads, and 5 to 8 blocks an SM were no faster.
#include <math.h>

#include "op_common.cuh"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kTileBytes = 32768;
template <int THREADS> constexpr int kUnroll = kTileBytes / (16 * THREADS); // packs of a thread
constexpr int kMostItems = 512;                       // tensors of one launch
constexpr int kFewItems = 16; // of a launch with short arguments
constexpr int kSmallBytes = 65536; // of a list that one block takes in one launch
constexpr int kGridPerSm = 8; // blocks; the squares' 63 registers hold 4 of them at a time, the
                              // scaling's 48 hold 5, the other norms' 32 hold 8

// One tensor of the list.  Its tiles start at a 16-byte boundary of `in`, so
// that every pack of a tile is aligned; the `head` elements before it belong
// to tile 0.
struct Item {
    const void *in;
    void *out;
    long long n;
    unsigned tile0; // number of the tensor's first tile in the launch
    short head;
    short dtype;
};

// ITEMS: how many tensors there is room for.  Kernel arguments are copied and
// read with every launch: a short list has short ones.
template <int ITEMS> struct Args {
    int items;
    unsigned tiles;
    int slot; // first partial of this launch
    int last; // the launch that joins the partials of all
    float max_norm, eps;
    float4 *partial;  // a slot per block: {sum or maximum, big, small, 0}
    unsigned *ticket; // zero between calls
    float *coef;      // scratch: min(1, max_norm / (norm + eps))
    float *norm;
    Item item[ITEMS];
};

// Sums of squares over the whole range of fp32, without overflow and without
// the loss of small values (J. L. Blue, "A portable Fortran program to find
// the Euclidean norm of a vector", ACM TOMS 4, 1978): three accumulators, for
// packs whose largest magnitude is above 2^44, between, and below 2^-50; the
// first are scaled by 2^-84, the last by 2^90.  A value far below its pack's
// largest loses nothing that the sum could hold.
struct Acc {
    float mid = 0.0f, low = 0.0f; // sum, and what rounding has taken from it
    float big = 0.0f, small = 0.0f;
};
constexpr float kBig = 0x1p44f, kSmall = 0x1p-50f;
constexpr float kBigScale = 0x1p-84f, kSmallScale = 0x1p90f;

template <int V, bool NARROW>
__device__ __forceinline__ void add_squares(Acc &a, const float (&x)[V])
{
    if constexpr (NARROW) { // fp16: every square is in the middle range
#pragma unroll
        for (int i = 0; i < V; ++i)
            a.mid = fmaf(x[i], x[i], a.mid);
        return;
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        m = fmaxf(m, fabsf(x[i]));
    if (m > kBig) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            a.big = fmaf(x[i] * kBigScale, x[i] * kBigScale, a.big);
    } else if (m < kSmall) { // NaN is ignored by fmaxf: a pack of NaN alone comes here
#pragma unroll
        for (int i = 0; i < V; ++i)
            a.small = fmaf(x[i] * kSmallScale, x[i] * kSmallScale, a.small);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            a.mid = fmaf(x[i], x[i], a.mid);
    }
}

template <int KIND, int V, bool NARROW = false>
__device__ __forceinline__ void add_pack(Acc &a, const float (&x)[V])
{
    if constexpr (KIND == RRA_NORM_L2) {
        add_squares<V, NARROW>(a, x);
    } else if constexpr (KIND == RRA_NORM_L1) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            a.mid += fabsf(x[i]);
    } else {
        // magnitudes order like their bit patterns, NaN above infinity
#pragma unroll
        for (int i = 0; i < V; ++i)
            a.mid = __uint_as_float(
                max(__float_as_uint(a.mid), __float_as_uint(x[i]) & 0x7fffffffu));
    }
}

// Adds a tile's sum to the thread's, with the rounding error of every addition
// (D. E. Knuth's two-sum): a thread adds thousands of tiles of a long list.
template <int KIND> __device__ __forceinline__ void add_tile(Acc &to, const Acc &tile)
{
    if (KIND == RRA_NORM_INF) {
        to.mid = __uint_as_float(max(__float_as_uint(to.mid), __float_as_uint(tile.mid)));
        return;
    }
    const float s = to.mid + tile.mid, t = s - to.mid;
    to.low += (to.mid - (s - t)) + (tile.mid - t);
    to.mid = s;
    to.big += tile.big;
    to.small += tile.small;
}

// The item that holds a tile of the launch.
template <typename A> __device__ __forceinline__ int find_item(const A &a, unsigned tile)
{
    int lo = 0, hi = a.items;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (a.item[m].tile0 <= tile)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// Element range [lo, hi) of a tile; lo is a pack boundary.
template <typename T>
__device__ __forceinline__ void tile_range(const Item &it, unsigned tile, long long *lo,
                                           long long *hi)
{
    constexpr long long kElems = kTileBytes / sizeof(T);
    *lo = it.head + (long long)(tile - it.tile0) * kElems;
    *hi = min(*lo + kElems, it.n);
}

template <typename T, int KIND, int THREADS>
__device__ __forceinline__ void norm_tile(const Item &it, unsigned tile, Acc &sum)
{
    Acc acc;
    constexpr int V = 16 / sizeof(T);
    const T *const p = static_cast<const T *>(it.in);
    long long lo, hi;
    tile_range<T>(it, tile, &lo, &hi);
    if (hi - lo == kTileBytes / (int)sizeof(T)) {
        Pack<T, V> v[kUnroll<THREADS>];
#pragma unroll
        for (int u = 0; u < kUnroll<THREADS>; ++u)
            v[u] = load_pack<T, V>(p + lo + (u * THREADS + threadIdx.x) * V);
#pragma unroll
        for (int u = 0; u < kUnroll<THREADS>; ++u) {
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = to_f32(v[u].e[i]);
            add_pack<KIND, V, std::is_same<T, __half>::value>(acc, x);
        }
    } else {
        const long long packs = hi > lo ? (hi - lo) / V : 0;
        for (long long k = threadIdx.x; k < packs; k += THREADS) {
            const Pack<T, V> v = load_pack<T, V>(p + lo + k * V);
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = to_f32(v.e[i]);
            add_pack<KIND, V, std::is_same<T, __half>::value>(acc, x);
        }
        const long long i = lo + packs * V + threadIdx.x;
        if (i < hi) {
            const float x[1] = {to_f32(p[i])};
            add_pack<KIND, 1>(acc, x);
        }
    }
    if (tile == it.tile0 && threadIdx.x < (unsigned)it.head && threadIdx.x < it.n) {
        const float x[1] = {to_f32(p[threadIdx.x])};
        add_pack<KIND, 1>(acc, x);
    }
    add_tile<KIND>(sum, acc);
}

template <int KIND, int THREADS>
__device__ __forceinline__ void norm_any(const Item &it, unsigned tile, Acc &sum)
{
    if (it.dtype == RRA_F32)
        norm_tile<float, KIND, THREADS>(it, tile, sum);
    else if (it.dtype == RRA_F16)
        norm_tile<__half, KIND, THREADS>(it, tile, sum);
    else
        norm_tile<__nv_bfloat16, KIND, THREADS>(it, tile, sum);
}

// A sum of blocks' sums: two floats, exact to about 48 bits (fp64 runs at a
// small part of fp32's rate here: a block of 1024 threads took 10 us to join
// 152 sums in it).
struct Two {
    float hi = 0.0f, lo = 0.0f;
};

template <int KIND> __device__ __forceinline__ Two plus(Two a, float hi, float lo)
{
    if (KIND == RRA_NORM_INF)
        return {__uint_as_float(max(__float_as_uint(a.hi), __float_as_uint(hi))), 0.0f};
    const float s = a.hi + hi, t = s - a.hi;
    return {s, a.lo + lo + ((a.hi - (s - t)) + (hi - t))};
}

__device__ __forceinline__ float value(Two a)
{
    return a.lo == a.lo ? a.hi + a.lo : a.hi; // (an infinite sum has no error)
}

template <int KIND> __device__ __forceinline__ Two warp_join(Two a)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = plus<KIND>(a, __shfl_xor_sync(kFull, a.hi, o), __shfl_xor_sync(kFull, a.lo, o));
    return a;
}

// What the list's norm is, from its sums.
template <int KIND> __device__ __forceinline__ float norm_of(Two mid, float big, float small)
{
    if (KIND != RRA_NORM_L2)
        return value(mid);
    if (big == 0.0f && small == 0.0f)
        return sqrtf(value(mid));
    return (float)sqrt((double)value(mid) + (double)big * 0x1p168 + (double)small * 0x1p-180);
}

__device__ __forceinline__ float coef_of(float norm, float max_norm, float eps)
{
    if (norm == 0.0f)
        return 1.0f;
    if (isinf(norm)) // (an infinite max_norm has no quotient with it)
        return 0.0f;
    const float c = max_norm / (norm + eps);
    return c < 1.0f ? c : (c == c ? 1.0f : c); // a NaN norm: a NaN factor
}

template <int KIND> __device__ __forceinline__ float join(float a, float b)
{
    if (KIND == RRA_NORM_INF)
        return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
    return a + b;
}

// Joins v over the block; the result is valid in the first warp.
template <int KIND, int THREADS> __device__ __forceinline__ float block_join(float v, float *sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = join<KIND>(v, __shfl_xor_sync(kFull, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sm[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < THREADS / 32 ? sm[threadIdx.x] : 0.0f;
#pragma unroll
        for (int o = THREADS / 64; o > 0; o >>= 1)
            v = join<KIND>(v, __shfl_xor_sync(kFull, v, o));
    }
    return v;
}

// A block's sums; big and small ones only where a thread has any.
template <int KIND, int THREADS>
__device__ __forceinline__ float4 block_sums(const Acc &acc, float *sm)
{
    // (an infinite sum has no rounding error)
    const float mine = acc.low == acc.low ? acc.mid + acc.low : acc.mid;
    float4 s = make_float4(block_join<KIND, THREADS>(mine, sm), 0.0f, 0.0f, 0.0f);
    if (KIND == RRA_NORM_L2 && __syncthreads_or(acc.big != 0.0f || acc.small != 0.0f)) {
        s.y = block_join<KIND, THREADS>(acc.big, sm);
        s.z = block_join<KIND, THREADS>(acc.small, sm);
    }
    return s;
}

// First pass.  Every block leaves its sums in a slot; the block that finishes
// last joins them in the order of their slots, so that the result does not
// depend on the order in which blocks ran.
template <int KIND, int ITEMS>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Args<ITEMS> a)
{
    __shared__ float sm[kThreads / 32];
    __shared__ float4 joined[kThreads / 32];
    __shared__ bool last;
    dependents_wait();
    dependents_launch();
    Acc acc;
    for (unsigned t = blockIdx.x; t < a.tiles; t += gridDim.x)
        norm_any<KIND, kThreads>(a.item[find_item(a, t)], t, acc);
    const float4 sums = block_sums<KIND, kThreads>(acc, sm);
    if (threadIdx.x == 0) {
        __stcg(a.partial + a.slot + blockIdx.x, sums);
        last = false;
        if (a.last) {
            __threadfence();
            last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    const int slots = a.slot + gridDim.x;
    Two mid;
    float big = 0.0f, small = 0.0f;
#pragma unroll 4
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        const float4 p = __ldcg(a.partial + s);
        mid = plus<KIND>(mid, p.x, 0.0f);
        big += p.y;
        small += p.z;
    }
    mid = warp_join<KIND>(mid);
    big = warp_sum(big);
    small = warp_sum(small);
    if (threadIdx.x % 32 == 0)
        joined[threadIdx.x / 32] = make_float4(mid.hi, mid.lo, big, small);
    __syncthreads();
    if (threadIdx.x >= 32)
        return;
    const float4 j = threadIdx.x < kThreads / 32 ? joined[threadIdx.x] : make_float4(0, 0, 0, 0);
    const float n = norm_of<KIND>(warp_join<KIND>({j.x, j.y}), warp_sum(j.z), warp_sum(j.w));
    if (threadIdx.x == 0) {
        *a.norm = n;
        *a.coef = coef_of(n, a.max_norm, a.eps);
        *a.ticket = 0;
    }
}

// `factor()` gives the factor, once the norm is known: a whole tile is read
// before.  EARLY: possibly before this kernel's own wait, which alone makes
// another kernel's writes visible to ordinary loads.  The norm's kernel has
// waited for whoever wrote the gradients, so they are in L2 by then; an SM's
// L1, where the norm's kernel may never have run, could hold older ones, so the
// loads pass it by.
template <typename T, int THREADS, bool EARLY, typename F>
__device__ __forceinline__ void scale_tile(const Item &it, unsigned tile, const F &factor)
{
    constexpr int V = 16 / sizeof(T);
    const T *const p = static_cast<const T *>(it.in);
    T *const q = static_cast<T *>(it.out);
    long long lo, hi;
    tile_range<T>(it, tile, &lo, &hi);
    // `out` may start elsewhere between two 16-byte boundaries than `in`
    const bool vec = reinterpret_cast<uintptr_t>(q + lo) % 16 == 0;
    const auto scaled = [](Pack<T, V> v, float c) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v.e[i] = from_f32<T>(to_f32(v.e[i]) * c);
        return v;
    };
    float c;
    if (vec && hi - lo == kTileBytes / (int)sizeof(T)) {
        Pack<T, V> v[kUnroll<THREADS>];
#pragma unroll
        for (int u = 0; u < kUnroll<THREADS>; ++u) {
            const T *const from = p + lo + (u * THREADS + threadIdx.x) * V;
            v[u] = EARLY ? load_pack_l2<T, V>(from) : load_pack<T, V>(from);
        }
        c = factor();
        if (c == 1.0f && it.in == it.out)
            return;
#pragma unroll
        for (int u = 0; u < kUnroll<THREADS>; ++u)
            store_pack<T, V>(q + lo + (u * THREADS + threadIdx.x) * V, scaled(v[u], c));
    } else {
        c = factor();
        if (c == 1.0f && it.in == it.out)
            return;
        const long long packs = vec && hi > lo ? (hi - lo) / V : 0;
        for (long long k = threadIdx.x; k < packs; k += THREADS)
            store_pack<T, V>(q + lo + k * V, scaled(load_pack<T, V>(p + lo + k * V), c));
        for (long long i = lo + packs * V + threadIdx.x; i < hi; i += THREADS)
            q[i] = from_f32<T>(to_f32(p[i]) * c);
    }
    if (tile == it.tile0 && threadIdx.x < (unsigned)it.head && threadIdx.x < it.n)
        q[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * c);
}

template <int THREADS, bool EARLY, typename F>
__device__ __forceinline__ void scale_any(const Item &it, unsigned tile, const F &factor)
{
    if (it.dtype == RRA_F32)
        scale_tile<float, THREADS, EARLY>(it, tile, factor);
    else if (it.dtype == RRA_F16)
        scale_tile<__half, THREADS, EARLY>(it, tile, factor);
    else
        scale_tile<__nv_bfloat16, THREADS, EARLY>(it, tile, factor);
}

// Second pass, from the last tile down: what the first pass read last may
// still be in L2.  In place a factor of 1 leaves nothing to do.
template <int ITEMS>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Args<ITEMS> a)
{
    dependents_launch(); // (every block waits for the norm, if after its first reads)
    bool known = false;
    float c = 0.0f;
    const auto factor = [&]() {
        if (!known) {
            dependents_wait();
            c = __ldcg(a.coef);
            known = true;
        }
        return c;
    };
    for (unsigned t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const unsigned tile = a.tiles - 1 - t;
        scale_any<kThreads, true>(a.item[find_item(a, tile)], tile, factor);
    }
}

// A short list: one block, one launch, the second reading from L1 or L2 (7 us
// a call of 4096 fp32 from Python, 12 us with two launches; the GPU has 3 to do).
template <int KIND, int ITEMS>
__global__ void __launch_bounds__(kThreads) small_kernel(const __grid_constant__ Args<ITEMS> a)
{
    __shared__ float sm[kThreads / 32];
    __shared__ float c;
    dependents_wait();
    dependents_launch();
    Acc acc;
    for (unsigned t = 0; t < a.tiles; ++t)
        norm_any<KIND, kThreads>(a.item[find_item(a, t)], t, acc);
    const float4 s = block_sums<KIND, kThreads>(acc, sm);
    if (threadIdx.x == 0) {
        const float n = norm_of<KIND>({s.x, 0.0f}, s.y, s.z);
        *a.norm = n;
        c = coef_of(n, a.max_norm, a.eps);
    }
    __syncthreads();
    const float factor = c;
    if (a.tiles > 0 && a.item[0].out)
        for (unsigned t = 0; t < a.tiles; ++t)
            scale_any<kThreads, false>(a.item[find_item(a, t)], t, [&]() { return factor; });
}

struct List {
    const void *const *in;
    void *const *out; // nullptr: the norm alone
    const size_t *counts;
    const rra_dtype *dtypes;
    int n;
};

bool valid_list(const List &l, const float *norm)
{
    if (!norm || !aligned_to(norm, sizeof(float)))
        return false;
    if (l.n < 0 || (l.n > 0 && (!l.in || !l.counts || !l.dtypes)))
        return false;
    unsigned long long tiles = 0; // of the whole list: their numbers are 32-bit
    for (int k = 0; k < l.n; ++k) {
        if (!valid_dt(l.dtypes[k]) || l.counts[k] > (size_t)1 << 40)
            return false;
        if (l.counts[k] == 0)
            continue;
        const size_t es = dtype_size(l.dtypes[k]);
        if (!l.in[k] || !aligned_to(l.in[k], es) ||
            overlap(l.in[k], l.counts[k] * es, norm, sizeof(float)))
            return false;
        if (l.out && (!l.out[k] || !aligned_to(l.out[k], es) ||
                      overlap(l.out[k], l.counts[k] * es, norm, sizeof(float)) ||
                      (l.out[k] != l.in[k] &&
                       overlap(l.in[k], l.counts[k] * es, l.out[k], l.counts[k] * es))))
            return false;
        tiles += l.counts[k] * es / kTileBytes + 2;
    }
    return tiles < 1ull << 31;
}

// Fills args with tensors from number k on, as many as one launch takes;
// returns the number of the first that is left.
template <int ITEMS> int fill(Args<ITEMS> &a, const List &l, int k)
{
    unsigned long long tiles = 0;
    a.items = 0;
    for (; k < l.n && a.items < ITEMS; ++k) {
        if (l.counts[k] == 0)
            continue;
        const size_t es = dtype_size(l.dtypes[k]);
        Item &it = a.item[a.items];
        it.in = l.in[k];
        it.out = l.out ? l.out[k] : nullptr;
        it.n = (long long)l.counts[k];
        it.dtype = (short)l.dtypes[k];
        it.head = (short)((16 - reinterpret_cast<uintptr_t>(it.in) % 16) % 16 / es);
        it.tile0 = (unsigned)tiles;
        const long long body = std::max(0LL, it.n - it.head), per = kTileBytes / (long long)es;
        tiles += std::max(1LL, (body + per - 1) / per);
        ++a.items;
    }
    a.tiles = (unsigned)tiles;
    return k;
}

template <int KIND, int ITEMS>
rra_status run(const List &l, bool small, float max_norm, float eps, float *norm, cudaStream_t st)
{
    Args<ITEMS> a;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    a.slot = 0;
    if constexpr (ITEMS == kFewItems) {
        if (small) {
            fill(a, l, 0);
            return launched(launch_chained(small_kernel<KIND, ITEMS>, dim3(1), kThreads, st, a));
        }
    }
    const unsigned most = (unsigned)num_sms() * kGridPerSm;
    const unsigned long long launches = l.n / ITEMS + 1;
    std::unique_lock<std::mutex> lk;
    unsigned char *ws = nullptr;
    const rra_status s =
        op_scratch(st, kScratchHead + 16 + sizeof(float4) * most * launches, lk, &ws);
    if (s != RRA_OK)
        return s;
    a.ticket = reinterpret_cast<unsigned *>(ws);
    a.coef = reinterpret_cast<float *>(ws + kScratchHead);
    a.partial = reinterpret_cast<float4 *>(ws + kScratchHead + 16);
    cudaError_t e = cudaSuccess;
    for (int k = 0;;) {
        k = fill(a, l, k);
        a.last = k >= l.n;
        const unsigned grid = std::max(1u, std::min(a.tiles, most));
        e = launch_chained(norm_kernel<KIND, ITEMS>, dim3(grid), kThreads, st, a);
        if (e != cudaSuccess)
            return RRA_ERR_CUDA;
        a.slot += (int)grid;
        if (a.last)
            break;
    }
    const bool again = l.n > ITEMS; // is what args hold not the whole list?
    for (int k = 0; e == cudaSuccess && l.out && k < l.n;) {
        k = again ? fill(a, l, k) : l.n;
        if (a.tiles == 0)
            continue;
        e = launch_chained(scale_kernel<ITEMS>, dim3(std::min(a.tiles, most)), kThreads, st, a);
    }
    return launched(e);
}

template <int KIND>
rra_status run_kind(const List &l, float max_norm, float eps, float *norm, cudaStream_t st)
{
    size_t bytes = 0;
    for (int k = 0; k < l.n; ++k)
        bytes += std::min(l.counts[k], (size_t)kSmallBytes) * dtype_size(l.dtypes[k]);
    if (l.n <= kFewItems)
        return run<KIND, kFewItems>(l, bytes <= kSmallBytes, max_norm, eps, norm, st);
    return run<KIND, kMostItems>(l, false, max_norm, eps, norm, st);
}

rra_status run(const List &l, rra_norm kind, float max_norm, float eps, float *norm,
               cudaStream_t st)
{
    if (kind == RRA_NORM_L2)
        return run_kind<RRA_NORM_L2>(l, max_norm, eps, norm, st);
    if (kind == RRA_NORM_L1)
        return run_kind<RRA_NORM_L1>(l, max_norm, eps, norm, st);
    return run_kind<RRA_NORM_INF>(l, max_norm, eps, norm, st);
}

bool valid_kind(rra_norm k) { return k == RRA_NORM_L2 || k == RRA_NORM_L1 || k == RRA_NORM_INF; }

} // namespace
} // namespace rra

extern "C" rra_status rra_grad_norm(const void *const *grads, const size_t *counts,
                                    const rra_dtype *dtypes, int ntensors, rra_norm kind,
                                    float *norm, void *stream)
{
    const rra::List l{grads, nullptr, counts, dtypes, ntensors};
    if (!rra::valid_kind(kind) || !rra::valid_list(l, norm))
        return RRA_ERR_INVALID;
    return rra::run(l, kind, 0.0f, 0.0f, norm, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" rra_status rra_grad_clip(const void *const *grads, void *const *out,
                                    const size_t *counts, const rra_dtype *dtypes, int ntensors,
                                    rra_norm kind, float max_norm, float eps, float *norm,
                                    void *stream)
{
    const rra::List l{grads, out, counts, dtypes, ntensors};
    if (!rra::valid_kind(kind) || (ntensors > 0 && !out) || !rra::valid_list(l, norm) ||
        !(max_norm >= 0.0f) || !(eps >= 0.0f) || isinf(eps))
        return RRA_ERR_INVALID;
    return rra::run(l, kind, max_norm, eps, norm, reinterpret_cast<cudaStream_t>(stream));
}
