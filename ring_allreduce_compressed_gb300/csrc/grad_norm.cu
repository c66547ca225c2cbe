// grad_norm.cu -- rra_grad_norm and rra_grad_clip: the norm of a list of
// gradients taken as one vector, and their scaling to a largest norm.
//
//   norm = (sum |g|^p)^(1/p), p = 1 or 2, or max |g|
//   out  = g * min(1, max_norm / (norm + eps))
//
// Both passes are bound by memory: the norm reads every gradient once, the
// scaling reads it again and writes it.  The list is cut into tiles of 32 KB,
// so that a block works on one tensor at a time and short tensors leave no SM
// with more than its share.
#include <math.h>

#include "op_common.cuh"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kTileBytes = 32768;
constexpr int kUnroll = kTileBytes / (16 * kThreads); // 16-byte packs per thread and tile
constexpr int kMostItems = 512;                       // tensors of one launch
constexpr int kGridPerSm = 8;                         // 256-thread blocks: full SMs

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

struct Args {
    int items;
    unsigned tiles;
    int kind; // rra_norm
    int slot; // first partial of this launch
    int last; // the launch that joins the partials of all
    float max_norm, eps;
    float *partial;   // 3 per slot
    unsigned *ticket; // zero between calls
    float *coef;      // scratch: min(1, max_norm / (norm + eps))
    float *norm;
    Item item[kMostItems];
};

// Sums of squares over the whole range of fp32, without overflow and without
// the loss of small values (J. L. Blue, "A portable Fortran program to find
// the Euclidean norm of a vector", ACM TOMS 4, 1978): three accumulators, for
// packs whose largest magnitude is above 2^44, between, and below 2^-50; the
// first are scaled by 2^-84, the last by 2^90.  A value far below its pack's
// largest loses nothing that the sum could hold.
struct Acc {
    float mid = 0.0f, big = 0.0f, small = 0.0f;
};
constexpr float kBig = 0x1p44f, kSmall = 0x1p-50f;
constexpr float kBigScale = 0x1p-84f, kSmallScale = 0x1p90f;

template <int V> __device__ __forceinline__ void add_squares(Acc &a, const float (&x)[V])
{
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

template <int KIND, int V> __device__ __forceinline__ void add_pack(Acc &a, const float (&x)[V])
{
    if constexpr (KIND == RRA_NORM_L2) {
        add_squares<V>(a, x);
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

// The item that holds a tile of the launch.
__device__ __forceinline__ int find_item(const Args &a, unsigned tile)
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

template <typename T, int KIND>
__device__ __forceinline__ void norm_tile(const Item &it, unsigned tile, Acc &acc)
{
    constexpr int V = 16 / sizeof(T);
    const T *const p = static_cast<const T *>(it.in);
    long long lo, hi;
    tile_range<T>(it, tile, &lo, &hi);
    if (hi - lo == kTileBytes / (int)sizeof(T)) {
        Pack<T, V> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = load_pack<T, V>(p + lo + (u * kThreads + threadIdx.x) * V);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = to_f32(v[u].e[i]);
            add_pack<KIND, V>(acc, x);
        }
    } else {
        const long long packs = hi > lo ? (hi - lo) / V : 0;
        for (long long k = threadIdx.x; k < packs; k += kThreads) {
            const Pack<T, V> v = load_pack<T, V>(p + lo + k * V);
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = to_f32(v.e[i]);
            add_pack<KIND, V>(acc, x);
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
}

// What the list's norm is, from its three sums.
template <int KIND> __device__ __forceinline__ float norm_of(double mid, double big, double small)
{
    if (KIND == RRA_NORM_L2)
        return (float)sqrt(mid + big * 0x1p168 + small * 0x1p-180);
    return (float)mid;
}

__device__ __forceinline__ float coef_of(float norm, float max_norm, float eps)
{
    if (norm == 0.0f)
        return 1.0f;
    const float c = max_norm / (norm + eps);
    return c < 1.0f ? c : (c == c ? 1.0f : c); // a NaN norm: a NaN factor
}

template <int KIND> __device__ __forceinline__ double join(double a, double b)
{
    if (KIND == RRA_NORM_INF) // NaN wins
        return a != a || a > b ? a : b;
    return a + b;
}

// Joins v over the block; the result is valid in thread 0.
template <int KIND> __device__ double block_join(double v, double *sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = join<KIND>(v, __shfl_xor_sync(kFull, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sm[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < kThreads / 32 ? sm[threadIdx.x] : 0.0;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            v = join<KIND>(v, __shfl_xor_sync(kFull, v, o));
    }
    return v;
}

// First pass.  Every block leaves three partial sums; the block that finishes
// last joins them in the order of their slots, so that the result does not
// depend on the order in which blocks ran.
template <int KIND>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Args a)
{
    __shared__ double sm[kThreads / 32];
    __shared__ bool last;
    Acc acc;
    for (unsigned t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const Item &it = a.item[find_item(a, t)];
        if (it.dtype == RRA_F32)
            norm_tile<float, KIND>(it, t, acc);
        else if (it.dtype == RRA_F16)
            norm_tile<__half, KIND>(it, t, acc);
        else
            norm_tile<__nv_bfloat16, KIND>(it, t, acc);
    }
    double mid = block_join<KIND>(acc.mid, sm), big = 0, small = 0;
    if (KIND == RRA_NORM_L2) {
        big = block_join<KIND>(acc.big, sm);
        small = block_join<KIND>(acc.small, sm);
    }
    if (threadIdx.x == 0) {
        float *p = a.partial + 3LL * (a.slot + blockIdx.x);
        p[0] = (float)mid;
        p[1] = (float)big;
        p[2] = (float)small;
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
    mid = big = small = 0;
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        mid = join<KIND>(mid, __ldcg(a.partial + 3LL * s));
        if (KIND == RRA_NORM_L2) {
            big += __ldcg(a.partial + 3LL * s + 1);
            small += __ldcg(a.partial + 3LL * s + 2);
        }
    }
    mid = block_join<KIND>(mid, sm);
    if (KIND == RRA_NORM_L2) {
        big = block_join<KIND>(big, sm);
        small = block_join<KIND>(small, sm);
    }
    if (threadIdx.x == 0) {
        const float n = norm_of<KIND>(mid, big, small);
        *a.norm = n;
        *a.coef = coef_of(n, a.max_norm, a.eps);
        *a.ticket = 0;
    }
}

template <typename T>
__device__ __forceinline__ void scale_tile(const Item &it, unsigned tile, float c)
{
    constexpr int V = 16 / sizeof(T);
    const T *const p = static_cast<const T *>(it.in);
    T *const q = static_cast<T *>(it.out);
    long long lo, hi;
    tile_range<T>(it, tile, &lo, &hi);
    // `out` may start elsewhere between two 16-byte boundaries than `in`
    const bool vec = reinterpret_cast<uintptr_t>(q + lo) % 16 == 0;
    if (vec && hi - lo == kTileBytes / (int)sizeof(T)) {
        Pack<T, V> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = load_pack<T, V>(p + lo + (u * kThreads + threadIdx.x) * V);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[u].e[i] = from_f32<T>(to_f32(v[u].e[i]) * c);
            store_pack<T, V>(q + lo + (u * kThreads + threadIdx.x) * V, v[u]);
        }
    } else {
        for (long long i = lo + threadIdx.x; i < hi; i += kThreads)
            q[i] = from_f32<T>(to_f32(p[i]) * c);
    }
    if (tile == it.tile0 && threadIdx.x < (unsigned)it.head && threadIdx.x < it.n)
        q[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * c);
}

// Second pass, from the last tile down: what the first pass read last may
// still be in L2.  In place a factor of 1 leaves nothing to do.
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Args a)
{
    const float c = __ldcg(a.coef);
    for (unsigned t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const unsigned tile = a.tiles - 1 - t;
        const Item &it = a.item[find_item(a, tile)];
        if (c == 1.0f && it.in == it.out)
            continue;
        if (it.dtype == RRA_F32)
            scale_tile<float>(it, tile, c);
        else if (it.dtype == RRA_F16)
            scale_tile<__half>(it, tile, c);
        else
            scale_tile<__nv_bfloat16>(it, tile, c);
    }
}

struct List {
    const void *const *in;
    void *const *out; // nullptr: the norm alone
    const size_t *counts;
    const rra_dtype *dtypes;
    int n;
};

bool valid_list(const List &l)
{
    if (l.n < 0 || (l.n > 0 && (!l.in || !l.counts || !l.dtypes)))
        return false;
    unsigned long long tiles = 0; // of the whole list: their numbers are 32-bit
    for (int k = 0; k < l.n; ++k) {
        if (!valid_dt(l.dtypes[k]) || l.counts[k] > (size_t)1 << 40)
            return false;
        if (l.counts[k] == 0)
            continue;
        const size_t es = dtype_size(l.dtypes[k]);
        if (!l.in[k] || !aligned_to(l.in[k], es))
            return false;
        if (l.out && (!l.out[k] || !aligned_to(l.out[k], es) ||
                      (l.out[k] != l.in[k] &&
                       overlap(l.in[k], l.counts[k] * es, l.out[k], l.counts[k] * es))))
            return false;
        tiles += l.counts[k] * es / kTileBytes + 2;
    }
    return tiles < 1ull << 31;
}

// Fills args with tensors from number k on, as many as one launch takes;
// returns the number of the first that is left.
int fill(Args &a, const List &l, int k)
{
    unsigned long long tiles = 0;
    a.items = 0;
    for (; k < l.n && a.items < kMostItems; ++k) {
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

rra_status run(const List &l, int kind, bool clip, float max_norm, float eps, float *norm,
               cudaStream_t st)
{
    const int most = num_sms() * kGridPerSm;
    const int launches = std::max(1, (l.n + kMostItems - 1) / kMostItems) + 1;
    std::unique_lock<std::mutex> lk;
    unsigned char *ws = nullptr;
    const rra_status s =
        op_scratch(st, kScratchHead + sizeof(float) * (4 + 3ull * most * launches), lk, &ws);
    if (s != RRA_OK)
        return s;
    Args a;
    a.kind = kind;
    a.max_norm = max_norm;
    a.eps = eps;
    a.ticket = reinterpret_cast<unsigned *>(ws);
    a.coef = reinterpret_cast<float *>(ws + kScratchHead);
    a.partial = a.coef + 4;
    a.norm = norm;
    a.slot = 0;
    int k = 0;
    do {
        k = fill(a, l, k);
        a.last = k >= l.n;
        const int grid = (int)std::max(1u, std::min(a.tiles, (unsigned)most));
        if (kind == RRA_NORM_L2)
            norm_kernel<RRA_NORM_L2><<<grid, kThreads, 0, st>>>(a);
        else if (kind == RRA_NORM_L1)
            norm_kernel<RRA_NORM_L1><<<grid, kThreads, 0, st>>>(a);
        else
            norm_kernel<RRA_NORM_INF><<<grid, kThreads, 0, st>>>(a);
        a.slot += grid;
    } while (k < l.n);
    if (clip) {
        for (k = 0; k < l.n;) {
            k = fill(a, l, k);
            if (a.tiles)
                scale_kernel<<<std::min(a.tiles, (unsigned)most), kThreads, 0, st>>>(a);
        }
    }
    return launched(cudaGetLastError());
}

bool valid_kind(rra_norm k) { return k == RRA_NORM_L2 || k == RRA_NORM_L1 || k == RRA_NORM_INF; }

} // namespace
} // namespace rra

extern "C" rra_status rra_grad_norm(const void *const *grads, const size_t *counts,
                                    const rra_dtype *dtypes, int ntensors, rra_norm kind,
                                    float *norm, void *stream)
{
    const rra::List l{grads, nullptr, counts, dtypes, ntensors};
    if (!norm || !rra::valid_kind(kind) || !rra::valid_list(l))
        return RRA_ERR_INVALID;
    return rra::run(l, kind, false, 0.0f, 0.0f, norm, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" rra_status rra_grad_clip(const void *const *grads, void *const *out,
                                    const size_t *counts, const rra_dtype *dtypes, int ntensors,
                                    rra_norm kind, float max_norm, float eps, float *norm,
                                    void *stream)
{
    const rra::List l{grads, out, counts, dtypes, ntensors};
    if (!norm || !rra::valid_kind(kind) || (ntensors > 0 && !out) || !rra::valid_list(l) ||
        !(max_norm >= 0.0f) || !(eps >= 0.0f) || isinf(eps))
        return RRA_ERR_INVALID;
    return rra::run(l, kind, true, max_norm, eps, norm, reinterpret_cast<cudaStream_t>(stream));
}
