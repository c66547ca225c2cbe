// embedding.cu -- rra_embedding and rra_embedding_grad: rows of a table looked
// up by token and scaled, and the table's gradient.
//
//   out[t, :] = scale * W[token[t], :]
//   dW[v, :]  = scale * sum over t with token[t] = v of dout[t, :]
//
// Both are bound by memory.  The gradient sorts the tokens (stable, so that a
// row's terms are added in the order of their positions and the result does
// not depend on the order in which blocks run), after which all terms of a
// row lie side by side.
#include "op_common.cuh"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ---------------------------------------------------------------- lookup

// A group of 2^lg lanes takes `kRun` packs a lane of one row: one run of
// columns.  A token outside the table gives a row of zeros.
constexpr int kRun = 4;

template <typename T, int V, typename I>
__global__ void __launch_bounds__(kThreads)
    lookup_kernel(const T *__restrict__ w, const I *__restrict__ tok, long long n, long long vocab,
                  long long dim, float scale, T *__restrict__ out, int lg, long long runs)
{
    const int lanes = 1 << lg;
    const int lane = threadIdx.x & (lanes - 1);
    const long long units = dim / V; // packs of a row
    const long long total = n * runs;
    const long long step = (long long)gridDim.x * (kThreads >> lg);
    for (long long i = (long long)blockIdx.x * (kThreads >> lg) + (threadIdx.x >> lg); i < total;
         i += step) {
        const long long t = i / runs, c0 = (i - t * runs) * (lanes * kRun) + lane;
        const long long v = (long long)tok[t];
        const bool in = v >= 0 && v < vocab;
        const T *const src = w + (in ? v : 0) * dim;
        T *const dst = out + t * dim;
        Pack<T, V> x[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const long long c = c0 + k * lanes;
            if (in && c < units) {
                x[k] = load_pack<T, V>(src + c * V);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    x[k].e[j] = from_f32<T>(0.0f);
            }
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const long long c = c0 + k * lanes;
#pragma unroll
            for (int j = 0; j < V; ++j)
                x[k].e[j] = from_f32<T>(to_f32(x[k].e[j]) * scale);
            if (c < units)
                store_pack<T, V>(dst + c * V, x[k]);
        }
    }
}

// ---------------------------------------------------------------- sort

// Least significant digit first, 8 bits a pass.  A pass counts the digits of
// every tile, turns the counts into places, and moves the tile's (token,
// position) pairs there; a tile's pairs keep their order.  Tokens that get no
// gradient (outside the table, padding) sort behind all others, as `vocab`.
constexpr int kDigits = 256;
constexpr int kSortTile = 4096;
constexpr int kSortRounds = kSortTile / kThreads;

struct SortArgs {
    const void *tok; // first pass: the tokens
    int wide;        // 64-bit tokens
    const uint32_t *key_in, *pos_in;
    uint32_t *key_out, *pos_out;
    uint32_t *hist;  // [digit][tile]
    uint32_t *total; // [digit]
    long long n, vocab, padding;
    long long tiles;
    int shift;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs &a, long long i)
{
    if (!a.tok)
        return a.key_in[i];
    const long long v = a.wide ? static_cast<const long long *>(a.tok)[i]
                               : (long long)static_cast<const int *>(a.tok)[i];
    return (uint32_t)(v >= 0 && v < a.vocab && v != a.padding ? v : a.vocab);
}

__global__ void __launch_bounds__(kThreads) sort_count_kernel(const SortArgs a)
{
    __shared__ uint32_t cnt[kDigits];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const long long base = (long long)blockIdx.x * kSortTile;
    for (int r = 0; r < kSortRounds; ++r) {
        const long long i = base + r * kThreads + threadIdx.x;
        if (i < a.n)
            atomicAdd(&cnt[(sort_key(a, i) >> a.shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    a.hist[threadIdx.x * a.tiles + blockIdx.x] = cnt[threadIdx.x];
}

// Exclusive sum of v over the block's threads; *sum is the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *sm, uint32_t *sum)
{
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        sm[w] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        before += k < w ? sm[k] : 0;
        all += sm[k];
    }
    __syncthreads();
    *sum = all;
    return before + x - v;
}

// One block per digit: its tiles' counts become the places behind the digit's
// first.
__global__ void __launch_bounds__(kThreads) sort_scan_kernel(const SortArgs a)
{
    __shared__ uint32_t sm[kWarps];
    uint32_t run = 0;
    uint32_t *const h = a.hist + blockIdx.x * a.tiles;
    for (long long b = 0; b < a.tiles; b += kThreads) {
        const long long i = b + threadIdx.x;
        uint32_t sum;
        const uint32_t x = block_scan(i < a.tiles ? h[i] : 0u, sm, &sum);
        if (i < a.tiles)
            h[i] = run + x;
        run += sum;
    }
    if (threadIdx.x == 0)
        a.total[blockIdx.x] = run;
}

__global__ void __launch_bounds__(kThreads) sort_move_kernel(const SortArgs a)
{
    __shared__ uint32_t cnt[kWarps][kDigits];
    __shared__ uint32_t sm[kWarps];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    for (int d = lane; d < kDigits; d += 32)
        cnt[w][d] = 0;
    uint32_t sum;
    const uint32_t first = block_scan(a.total[threadIdx.x], sm, &sum);
    __syncwarp();
    // a warp takes a stretch of the tile, 32 pairs a round
    const long long base = (long long)blockIdx.x * kSortTile + w * (kSortTile / kWarps) + lane;
    uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const long long i = base + r * 32;
        const bool on = i < a.n;
        key[r] = on ? sort_key(a, i) : 0u;
        const uint32_t d = on ? (key[r] >> a.shift) & (kDigits - 1) : kDigits;
        const uint32_t same = __match_any_sync(kFull, d);
        const uint32_t before = __popc(same & ((1u << lane) - 1));
        uint32_t at = 0;
        if (on)
            at = cnt[w][d];
        __syncwarp();
        rank[r] = at + before;
        if (on && before == 0)
            cnt[w][d] = at + __popc(same);
        __syncwarp();
    }
    __syncthreads();
    { // thread d: the places of digit d of every warp's stretch
        uint32_t at = first + a.hist[threadIdx.x * a.tiles + blockIdx.x];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const uint32_t c = cnt[k][threadIdx.x];
            cnt[k][threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const long long i = base + r * 32;
        if (i < a.n) {
            const uint32_t at = cnt[w][(key[r] >> a.shift) & (kDigits - 1)] + rank[r];
            a.key_out[at] = key[r];
            a.pos_out[at] = a.tok ? (uint32_t)i : a.pos_in[i];
        }
    }
}

// ---------------------------------------------------------------- gradient

// First place whose token is not below v.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t *key, uint32_t n, uint32_t v)
{
    uint32_t lo = 0, len = n;
    while (len > 0) {
        const uint32_t h = len / 2;
        if (key[lo + h] < v) {
            lo += h + 1;
            len -= h + 1;
        } else {
            len = h;
        }
    }
    return lo;
}

// A block per row of the table: the row's places are found by bisection.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads)
    row_sum_kernel(const T *__restrict__ dout, const uint32_t *__restrict__ key,
                   const uint32_t *__restrict__ pos, uint32_t n, long long vocab, long long dim,
                   float scale, O *__restrict__ dw, int accumulate)
{
    for (long long v = blockIdx.x; v < vocab; v += gridDim.x) {
        const uint32_t lo = lower_bound(key, n, (uint32_t)v);
        const uint32_t hi = lower_bound(key, n, (uint32_t)v + 1);
        if (accumulate && lo == hi)
            continue;
        for (long long c = threadIdx.x; c < dim; c += kThreads) {
            float s = 0.0f;
            for (uint32_t i = lo; i < hi; ++i)
                s += to_f32(dout[(long long)pos[i] * dim + c]);
            O *const p = dw + v * dim + c;
            *p = from_f32<O>(accumulate ? fmaf(s, scale, to_f32(*p)) : s * scale);
        }
    }
}

inline unsigned grid_of(long long items, int per_sm)
{
    return (unsigned)std::max(1LL, std::min(items, (long long)num_sms() * per_sm));
}

template <typename T, int V>
void lookup(const void *w, const void *tok, long long n, long long vocab, long long dim, bool wide,
            float scale, void *out, cudaStream_t st)
{
    const long long units = dim / V;
    int lg = 0;
    while (lg < 5 && (1LL << lg) * kRun < units)
        ++lg;
    const long long runs = (units + (kRun << lg) - 1) / (kRun << lg);
    const long long per_block = kThreads >> lg;
    const unsigned grid = grid_of((n * runs + per_block - 1) / per_block, 32);
    if (wide)
        lookup_kernel<T, V, long long><<<grid, kThreads, 0, st>>>(
            static_cast<const T *>(w), static_cast<const long long *>(tok), n, vocab, dim, scale,
            static_cast<T *>(out), lg, runs);
    else
        lookup_kernel<T, V, int><<<grid, kThreads, 0, st>>>(
            static_cast<const T *>(w), static_cast<const int *>(tok), n, vocab, dim, scale,
            static_cast<T *>(out), lg, runs);
}

template <typename T>
void lookup_any(const void *w, const void *tok, long long n, long long vocab, long long dim,
                bool wide, float scale, void *out, cudaStream_t st)
{
    const size_t row = (size_t)dim * sizeof(T);
    const auto fits = [&](size_t b) { return pack_fits(w, row, b) && pack_fits(out, row, b); };
    if (fits(16))
        lookup<T, 16 / sizeof(T)>(w, tok, n, vocab, dim, wide, scale, out, st);
    else if (fits(8))
        lookup<T, 8 / sizeof(T)>(w, tok, n, vocab, dim, wide, scale, out, st);
    else if (sizeof(T) == 2 && fits(4))
        lookup<T, 4 / sizeof(T)>(w, tok, n, vocab, dim, wide, scale, out, st);
    else
        lookup<T, 1>(w, tok, n, vocab, dim, wide, scale, out, st);
}

template <typename T, typename O>
void row_sum(const void *dout, const uint32_t *key, const uint32_t *pos, long long n,
             long long vocab, long long dim, float scale, void *dw, int accumulate,
             cudaStream_t st)
{
    row_sum_kernel<T, O><<<grid_of(vocab, 64), kThreads, 0, st>>>(
        static_cast<const T *>(dout), key, pos, (uint32_t)n, vocab, dim, scale,
        static_cast<O *>(dw), accumulate);
}

bool valid_index(rra_index t) { return t == RRA_I32 || t == RRA_I64; }
constexpr size_t kMost = 0x7fffffff; // tokens, rows of the table
constexpr size_t kMostDim = (size_t)1 << 32;

} // namespace
} // namespace rra

extern "C" rra_status rra_embedding(const void *weight, const void *tokens, size_t ntokens,
                                    size_t vocab, size_t dim, rra_dtype dtype, rra_index index,
                                    float scale, void *out, void *stream)
{
    using namespace rra;
    if (!valid_dt(dtype) || !valid_index(index) || vocab == 0 || vocab > kMost || dim == 0 ||
        dim > kMostDim || ntokens > kMost)
        return RRA_ERR_INVALID;
    if (ntokens == 0)
        return RRA_OK;
    const size_t es = dtype_size(dtype), is = index == RRA_I64 ? 8 : 4;
    if (!weight || !tokens || !out || !aligned_to(weight, es) || !aligned_to(out, es) ||
        !aligned_to(tokens, is) || overlap(weight, vocab * dim * es, out, ntokens * dim * es) ||
        overlap(tokens, ntokens * is, out, ntokens * dim * es))
        return RRA_ERR_INVALID;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool wide = index == RRA_I64;
    if (dtype == RRA_F32)
        lookup_any<float>(weight, tokens, ntokens, vocab, dim, wide, scale, out, st);
    else if (dtype == RRA_F16)
        lookup_any<__half>(weight, tokens, ntokens, vocab, dim, wide, scale, out, st);
    else
        lookup_any<__nv_bfloat16>(weight, tokens, ntokens, vocab, dim, wide, scale, out, st);
    return launched(cudaGetLastError());
}

extern "C" rra_status rra_embedding_grad(const void *dout, const void *tokens, size_t ntokens,
                                         size_t vocab, size_t dim, rra_dtype dout_t,
                                         rra_index index, float scale, int64_t padding,
                                         void *dweight, rra_dtype dweight_t, int accumulate,
                                         void *stream)
{
    using namespace rra;
    if (!valid_dt(dout_t) || !valid_dt(dweight_t) || !valid_index(index) || vocab == 0 ||
        vocab > kMost || dim == 0 || dim > kMostDim || ntokens > kMost || !dweight)
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dout_t), os = dtype_size(dweight_t),
                 is = index == RRA_I64 ? 8 : 4;
    if (!aligned_to(dweight, os) ||
        (ntokens > 0 &&
         (!dout || !tokens || !aligned_to(dout, es) || !aligned_to(tokens, is) ||
          overlap(dout, ntokens * dim * es, dweight, vocab * dim * os) ||
          overlap(tokens, ntokens * is, dweight, vocab * dim * os))))
        return RRA_ERR_INVALID;
    if (dweight_t != dout_t && dweight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const long long n = (long long)ntokens, tiles = (n + kSortTile - 1) / kSortTile;
    std::unique_lock<std::mutex> lk;
    unsigned char *ws = nullptr;
    const rra_status s = op_scratch(
        st, kScratchHead + sizeof(uint32_t) * (4ull * n + kDigits * (tiles + 1ull)), lk, &ws);
    if (s != RRA_OK)
        return s;
    SortArgs a{};
    uint32_t *const base = reinterpret_cast<uint32_t *>(ws + kScratchHead);
    uint32_t *const key[2] = {base, base + n}, *const pos[2] = {base + 2 * n, base + 3 * n};
    a.hist = base + 4 * n;
    a.total = a.hist + kDigits * tiles;
    a.n = n;
    a.vocab = (long long)vocab;
    a.padding = padding;
    a.tiles = tiles;
    a.wide = index == RRA_I64;
    int at = 0;
    if (n > 0) {
        for (int shift = 0; shift == 0 || (vocab >> shift) != 0; shift += 8) {
            a.tok = shift == 0 ? tokens : nullptr;
            a.key_in = key[at];
            a.pos_in = pos[at];
            a.key_out = key[at ^ 1];
            a.pos_out = pos[at ^ 1];
            a.shift = shift;
            sort_count_kernel<<<(unsigned)tiles, kThreads, 0, st>>>(a);
            sort_scan_kernel<<<kDigits, kThreads, 0, st>>>(a);
            sort_move_kernel<<<(unsigned)tiles, kThreads, 0, st>>>(a);
            at ^= 1;
        }
    }
#define RRA_SUM(T, O)                                                                             \
    row_sum<T, O>(dout, key[at], pos[at], n, (long long)vocab, (long long)dim, scale, dweight,    \
                  accumulate, st)
    if (dout_t == RRA_F32)
        RRA_SUM(float, float);
    else if (dout_t == RRA_F16 && dweight_t == RRA_F16)
        RRA_SUM(__half, __half);
    else if (dout_t == RRA_F16)
        RRA_SUM(__half, float);
    else if (dweight_t == RRA_BF16)
        RRA_SUM(__nv_bfloat16, __nv_bfloat16);
    else
        RRA_SUM(__nv_bfloat16, float);
#undef RRA_SUM
    return launched(cudaGetLastError());
}
