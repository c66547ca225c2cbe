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
#include "token_sort.cuh"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ---------------------------------------------------------------- lookup

// A group of 2^lg lanes takes `kRun` packs a lane of one row: one run of
// columns.  A token outside the table gives a row of zeros.  The rows are
// streamed out, so that the table's stay in L2 for the tokens to come.  No
// pointer is marked as read alone: the read-only path holds for memory that
// nobody writes while the kernel lives, and this one may begin while the kernel
// ahead still writes the table.
//
// Measured: 30.3 us for 32768 rows of 2048 bf16 out of 128000, 6.0 TB/s of the
// rows read once and written (32.8 us with plain stores; 50 us with 8 packs a
// lane, whose registers leave too few warps).
constexpr int kRun = 4;

template <typename T, int V, typename I>
__global__ void __launch_bounds__(kThreads)
    lookup_kernel(const T *w, const I *tok, long long n, long long vocab, long long dim,
                  float scale, T *out, int lg, long long runs)
{
    dependents_wait();
    dependents_launch();
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
        const float factor = in ? scale : 1.0f; // a row of zeros stays one for every scale
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
                x[k].e[j] = from_f32<T>(to_f32(x[k].e[j]) * factor);
            if (c < units)
                stream_pack<T, V>(dst + c * V, x[k]);
        }
    }
}

// ---------------------------------------------------------------- gradient
//
// The sorted places are cut into tiles of 8, 16 or 32.  A group of 2^lg lanes adds
// the rows of one tile over a slab of 8 columns a lane, all in registers, and
// writes a row of the table when its last term has come.  A row whose terms
// cross a tile's edge leaves a partial sum on either side (slot 0 of a tile:
// the row that came in, slot 1: the row that goes on), which finish_kernel adds
// in the order of the tiles.  So a frequent token's terms are spread over as
// many groups as there are tiles of it.
//
// Measured: 49 us for 16384 x 2048 bf16 into 50000 rows (272 MB, 5.55 TB/s),
// 152 us for 131072 x 1024 bf16 into 128000 fp32 rows (793 MB, 5.2 TB/s): the
// sort's 11 and 31 us, in which only the clears use memory, then near its rate.
//
// Rows of no token are cleared: the table's last rows, where tokens are
// fewest, while the sort runs on 16 of the SMs (and written over by the sums
// where a token has them), the others beside the joins, whose waits they hide.

constexpr int kMostPlaces = 32;
constexpr int kSumThreads = 128; // small blocks: a short last wave
constexpr uint32_t kFew = 16; // partial sums that one warp joins
// Rows in flight: 16 registers a lane.  Twice as many left room for 5 blocks of
// an SM instead of 7: 56 against 53 us at 16384 x 2048 bf16.
template <typename T, int V> constexpr int kBatchOf = sizeof(T) * V >= 4 ? 8 / sizeof(T) : 4;

struct SumArgs {
    const void *dout;
    const uint2 *pair; // (token, position), sorted; goes on to a whole tile
    uint32_t n;
    long long vocab, dim;
    float scale;
    void *dw;
    int accumulate;
    float *part;     // [tile][2][dim]
    uint32_t *present; // a bit for every row that a token has
    uint32_t *joins; // lengths of the two lists
    uint4 *list;     // [2][tiles]: {tile, row, partial sums} of the rows that cross
                     // edges, those of up to kFew partial sums and the others
    uint32_t places; // of a tile
    uint32_t tiles, slabs;
    int lg;
    long long cleared; // rows before which clear_kernel has left the table alone
    int clear_lg;      // 2^clear_lg rows at a time are cleared by a warp
    long long sums;
    unsigned join_blocks; // blocks of the last kernel that join; the others clear
};

// V columns of a finished row of the table.
template <typename O, int V>
__device__ __forceinline__ void put_final(O *q, const float (&s)[V], const SumArgs &a)
{
    O v[V];
    if (a.accumulate) {
        load_values<O, V>(q, v);
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = from_f32<O>(fmaf(s[j], a.scale, to_f32(v[j])));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = from_f32<O>(s[j] * a.scale);
    }
    store_values<O, V>(q, v);
}

template <typename T, typename O, int V>
__device__ __forceinline__ void sum_tile(const SumArgs &a, uint32_t tile, uint32_t slab, int lane)
{
    constexpr int K = 8 / V, kBatch = kBatchOf<T, V>;
    const T *const dout = static_cast<const T *>(a.dout);
    const long long c0 = (long long)slab * (8 << a.lg) + lane * V;
    const int stride = V << a.lg;
    const uint32_t lo = tile * a.places, hi = min(lo + a.places, a.n);
    const uint32_t vocab = (uint32_t)a.vocab;
    if (a.pair[lo].x >= vocab)
        return;
    uint32_t cur = a.pair[lo].x;
    bool head = lo > 0 && a.pair[lo - 1].x == cur;
    float acc[K][V] = {};

    const auto emit = [&](bool tail) {
        if (head || tail) {
            float *const q = a.part + ((long long)tile * 2 + (head ? 0 : 1)) * a.dim;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c0 + k * stride < a.dim)
                    store_values<float, V>(q + c0 + k * stride, acc[k]);
        } else {
            O *const q = static_cast<O *>(a.dw) + (long long)cur * a.dim;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c0 + k * stride < a.dim)
                    put_final<O, V>(q + c0 + k * stride, acc[k], a);
        }
    };

    // pairs are read one batch ahead of the rows
    uint4 ahead[kBatch / 2];
    const auto read_pairs = [&](uint32_t i) {
#pragma unroll
        for (int q = 0; q < kBatch / 2; ++q)
            ahead[q] = reinterpret_cast<const uint4 *>(a.pair + i)[q];
    };
    read_pairs(lo);
    for (uint32_t i = lo; i < hi; i += kBatch) {
        uint32_t key[kBatch], pos[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch / 2; ++q) {
            key[2 * q] = ahead[q].x;
            pos[2 * q] = ahead[q].y;
            key[2 * q + 1] = ahead[q].z;
            pos[2 * q + 1] = ahead[q].w;
        }
        Raw<T, V> x[kBatch][K];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i + b >= hi)
                key[b] = vocab;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (key[b] < vocab && c0 + k * stride < a.dim)
                    x[b][k].load(dout + (long long)pos[b] * a.dim + c0 + k * stride);
        }
        if (i + kBatch < hi)
            read_pairs(i + kBatch);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (key[b] >= vocab)
                break;
            if (key[b] != cur) {
                emit(false);
                cur = key[b];
                head = false;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        acc[k][j] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    acc[k][j] += x[b][k].get(j);
        }
    }
    const bool tail = hi < a.n && a.pair[hi].x == cur;
    emit(tail);
    if (tail && !head && slab == 0 && lane == 0) {
        // the tiles after this one that begin with the row
        uint32_t in = 1, out = 2; // `in` do, if `out` is a tile it does not
        const auto begins = [&](uint32_t k) {
            return k < a.tiles - tile && a.pair[(size_t)(tile + k) * a.places].x == cur;
        };
        while (begins(out)) {
            in = out;
            out *= 2;
        }
        while (out - in > 1) {
            const uint32_t m = in + (out - in) / 2;
            (begins(m) ? in : out) = m;
        }
        const int many = in + 1 > kFew;
        a.list[many * a.tiles + atomicAdd(a.joins + many, 1u)] = make_uint4(tile, cur, in + 1, 0);
    }
}

// Clears the rows that no token has.  A warp takes a few rows of about 4 KB,
// then the next ones a grid further, so that the grid goes through the table
// in order.  Its lanes read the marks of its next 32 turns at once: at every
// turn, behind the writes of a whole GPU, the read cost more than the writes
// (whole gradient at 16384 x 2048 bf16, 4 blocks an SM: 72 against 65 us; with
// 8 blocks 62).
constexpr int kClearBytes = 4096;
constexpr int kClearPerSm = 8; // blocks

template <typename O>
__device__ __forceinline__ void clear_rows(const SumArgs &a, unsigned block, unsigned blocks)
{
    constexpr int V = 16 / sizeof(O);
    const int lane = threadIdx.x % 32;
    const bool vec = pack_fits(a.dw, a.dim * sizeof(O), 16);
    const unsigned long long width = a.dim / (vec ? V : 1); // stores of a row
    const int rows = 1 << a.clear_lg;
    const long long step = (long long)blocks * kWarps << a.clear_lg;
    long long v = (long long)(block * kWarps + threadIdx.x / 32) << a.clear_lg;
    // (past L1, which may hold an earlier call's)
    const auto marks = [&](long long at) {
        return a.n && at < a.cleared ? __ldcg(a.present + at / 32) >> at % 32 : 0u;
    };
    uint32_t ahead = 0;
    for (int turn = 0; v < a.cleared; v += step, ++turn) {
        if (turn % 32 == 0)
            ahead = marks(v + lane * step);
        const uint32_t there = __shfl_sync(kFull, ahead, turn % 32);
        O *const q = static_cast<O *>(a.dw) + v * a.dim;
        if (rows == 1) {
            if (there & 1)
                continue;
            if (vec) {
#pragma unroll 4
                for (unsigned long long u = lane; u < width; u += 32)
                    reinterpret_cast<uint4 *>(q)[u] = make_uint4(0, 0, 0, 0);
            } else {
                for (unsigned long long u = lane; u < width; u += 32)
                    q[u] = from_f32<O>(0.0f);
            }
        } else {
            const unsigned w = (unsigned)width, units = (unsigned)min(a.cleared - v, (long long)rows) * w;
#pragma unroll 4
            for (unsigned u = lane; u < units; u += 32) {
                if (there >> u / w & 1)
                    continue;
                if (vec)
                    reinterpret_cast<uint4 *>(q)[u] = make_uint4(0, 0, 0, 0);
                else
                    q[u] = from_f32<O>(0.0f);
            }
        }
    }
}

template <typename T, typename O, int V>
__global__ void __launch_bounds__(kSumThreads, 7) sum_kernel(const SumArgs a)
{
    // in this order: when finish_kernel starts, the sort has ended
    dependents_wait();
    dependents_launch();
    const long long g = ((long long)blockIdx.x * kSumThreads + threadIdx.x) >> a.lg;
    if (g < a.sums) {
        const uint32_t tile = (uint32_t)(g / a.slabs);
        sum_tile<T, O, V>(a, tile, (uint32_t)(g - (long long)tile * a.slabs),
                          threadIdx.x & ((1 << a.lg) - 1));
    }
}

// The table from row `cleared` on, before the sums are written over it.  (The
// sort has waited for what was before the call when it lets this kernel in.)
__global__ void __launch_bounds__(kThreads) clear_kernel(unsigned char *p, long long bytes)
{
    dependents_launch();
    const long long packs = bytes / 16, step = (long long)gridDim.x * kThreads;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < packs; i += step)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(0, 0, 0, 0);
    if (blockIdx.x == 0 && threadIdx.x < bytes % 16)
        p[packs * 16 + threadIdx.x] = 0;
    // When this kernel has ended, so has the sort.  One block waits for it: the
    // others make room for those that found none beside the sort's.
    if (blockIdx.x == 0)
        dependents_wait();
}

// V * K columns of a lane, `stride` apart, of partial sums p0 .. p1 - 1 of the
// row that begins in tile t.
template <int V, int K>
__device__ __forceinline__ void add_parts(const SumArgs &a, uint32_t t, uint32_t p0, uint32_t p1,
                                          long long c, int stride, float (&acc)[K][V])
{
#pragma unroll 8
    for (uint32_t p = p0; p < p1; ++p) {
        const float *const q = a.part + ((long long)(t + p) * 2 + (p == 0 ? 1 : 0)) * a.dim;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c + k * stride < a.dim) {
                const Pack<float, V> x = load_pack<float, V>(q + c + k * stride);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    acc[k][j] += x.e[j];
            }
    }
}

// Rows of terms that cross tile edges: their partial sums, in the order of
// the tiles.  Up to kFew are added by a warp, for 128 columns.  More by a
// block, for 32 columns: 8 lanes take 32 columns, so the block adds 32
// stretches of the sums at once and then their results.
constexpr int kStretches = kThreads / 8;

template <typename O, int V> __device__ __forceinline__ void join_rows(const SumArgs &a)
{
    constexpr int K = 4 / V;
    __shared__ float sm[kStretches][33];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const uint32_t few_slabs = (uint32_t)((a.dim + 127) / 128),
                   many_slabs = (uint32_t)((a.dim + 31) / 32);
    const unsigned long long few = (unsigned long long)a.joins[0] * few_slabs,
                             many = (unsigned long long)a.joins[1] * many_slabs;

    for (unsigned long long i = blockIdx.x; i < many; i += a.join_blocks) {
        const uint4 e = a.list[a.tiles + i / many_slabs];
        const long long c0 = (long long)(i % many_slabs) * 32;
        const int s = threadIdx.x / 8, at = threadIdx.x % 8 * V;
        float acc[K][V] = {};
        add_parts<V, K>(a, e.x, (uint32_t)((unsigned long long)e.z * s / kStretches),
                        (uint32_t)((unsigned long long)e.z * (s + 1) / kStretches), c0 + at, 8 * V,
                        acc);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
                sm[s][at + k * 8 * V + j] = acc[k][j];
        __syncthreads();
        if (w == 0 && c0 + lane < a.dim) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int q = 0; q < kStretches; ++q)
                sum[0] += sm[q][lane];
            put_final<O, 1>(static_cast<O *>(a.dw) + (long long)e.y * a.dim + c0 + lane, sum, a);
        }
    }
    // from the last block down: the first ones may be at the long rows
    for (unsigned long long i = (unsigned long long)(a.join_blocks - 1 - blockIdx.x) * kWarps + w;
         i < few; i += (unsigned long long)a.join_blocks * kWarps) {
        const uint4 e = a.list[i / few_slabs];
        const long long c = (long long)(i % few_slabs) * 128 + lane * V;
        float acc[K][V] = {};
        add_parts<V, K>(a, e.x, 0, e.z, c, 32 * V, acc);
        O *const q = static_cast<O *>(a.dw) + (long long)e.y * a.dim;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c + k * 32 * V < a.dim)
                put_final<O, V>(q + c + k * 32 * V, acc[k], a);
    }
}

// The joins, for which the sums must have ended, and the clears, which need the
// sort alone: they run beside the sums' last blocks, too.
template <typename O, int V>
__global__ void __launch_bounds__(kThreads) finish_kernel(const SumArgs a)
{
    dependents_launch();
    if (blockIdx.x < a.join_blocks) {
        dependents_wait();
        join_rows<O, V>(a);
    } else {
        clear_rows<O>(a, blockIdx.x - a.join_blocks, gridDim.x - a.join_blocks);
        if (blockIdx.x == 0) // no joins: the sums have ended when this kernel has
            dependents_wait();
    }
}

inline unsigned grid_of(long long items, int per_sm)
{
    return (unsigned)std::max(1LL, std::min(items, (long long)num_sms() * per_sm));
}

template <typename T, int V>
cudaError_t lookup(const void *w, const void *tok, long long n, long long vocab, long long dim, bool wide,
            float scale, void *out, cudaStream_t st)
{
    const long long units = dim / V;
    int lg = 0;
    while (lg < 5 && (1LL << lg) * kRun < units)
        ++lg;
    const long long runs = (units + (kRun << lg) - 1) / (kRun << lg);
    const long long per_block = kThreads >> lg;
    const unsigned grid = grid_of((n * runs + per_block - 1) / per_block, 16);
    if (wide)
        return launch_chained(lookup_kernel<T, V, long long>, dim3(grid), kThreads, st,
                              static_cast<const T *>(w), static_cast<const long long *>(tok), n,
                              vocab, dim, scale, static_cast<T *>(out), lg, runs);
    return launch_chained(lookup_kernel<T, V, int>, dim3(grid), kThreads, st,
                          static_cast<const T *>(w), static_cast<const int *>(tok), n, vocab, dim,
                          scale, static_cast<T *>(out), lg, runs);
}

template <typename T>
cudaError_t lookup_any(const void *w, const void *tok, long long n, long long vocab, long long dim,
                bool wide, float scale, void *out, cudaStream_t st)
{
    const size_t row = (size_t)dim * sizeof(T);
    const auto fits = [&](size_t b) { return pack_fits(w, row, b) && pack_fits(out, row, b); };
    if (fits(16))
        return lookup<T, 16 / sizeof(T)>(w, tok, n, vocab, dim, wide, scale, out, st);
    if (fits(8))
        return lookup<T, 8 / sizeof(T)>(w, tok, n, vocab, dim, wide, scale, out, st);
    if (sizeof(T) == 2 && fits(4))
        return lookup<T, 4 / sizeof(T)>(w, tok, n, vocab, dim, wide, scale, out, st);
    return lookup<T, 1>(w, tok, n, vocab, dim, wide, scale, out, st);
}

// A table that is not worth a launch for its clearing: the joins' kernel does it.
constexpr size_t kSmallTable = 8 << 20;

// Table rows that are cleared during the sort: about what the other SMs write
// in the time that it takes.  A line through two measured sizes (none, 48 MB +
// 1 KB a token: 63, 56 us at 16384 tokens, 169, 152 us at 131072); a sort by
// fewer than 16 blocks was not measured and may leave room for more.
long long cleared_early(const SumArgs &a, size_t row)
{
    if (a.accumulate || a.n == 0 || a.n > kCsMost)
        return 0;
    const unsigned long long bytes = (48ull << 20) + 1024ull * a.n;
    if (a.vocab * row <= kSmallTable)
        return 0;
    return std::min((long long)(bytes / row), a.vocab);
}

template <typename T, typename O, int V> cudaError_t sum_rows(SumArgs a, cudaStream_t st)
{
    const size_t row = (size_t)a.dim * sizeof(O);
    const long long early = cleared_early(a, row);
    a.cleared = a.vocab - early;
    unsigned char *p = static_cast<unsigned char *>(a.dw) + a.cleared * row;
    // from a whole pack on: within 8 rows, or there is none
    for (int k = 0; k < 8 && !aligned_to(p, 16); ++k, ++a.cleared)
        p += row;
    if (early < 8 || !aligned_to(p, 16))
        a.cleared = a.vocab;
    if (a.cleared < a.vocab) {
        const long long bytes = (a.vocab - a.cleared) * (long long)row;
        const cudaError_t e = launch_chained(
            clear_kernel, dim3(grid_of(bytes / (16 * kThreads) + 1, 8)), kThreads, st, p, bytes);
        if (e != cudaSuccess)
            return e;
    }
    if (a.tiles > 0) {
        const cudaError_t e = launch_chained(
            sum_kernel<T, O, V>,
            dim3((unsigned)(((a.sums << a.lg) + kSumThreads - 1) / kSumThreads)), kSumThreads, st,
            a);
        if (e != cudaSuccess)
            return e;
    }
    a.clear_lg = 0;
    while (a.clear_lg < 5 && (row << (a.clear_lg + 1)) <= kClearBytes)
        ++a.clear_lg;
    const long long at_once = (long long)kWarps << a.clear_lg;
    const long long clears =
        a.accumulate || a.cleared == 0
            ? 0
            : grid_of((a.cleared + at_once - 1) / at_once, kClearPerSm);
    // joins wait more than they read: two blocks an SM last as long as the
    // clears beside it, many are better where there are none
    a.join_blocks = a.tiles < 2 ? 0
                                : grid_of((long long)a.tiles * ((a.dim + 127) / 128) / 4,
                                          clears > num_sms() ? 2 : 8);
    const dim3 grid((unsigned)(a.join_blocks + clears));
    if (grid.x == 0)
        return cudaSuccess;
    const bool wide = a.dim % 4 == 0 && aligned_to(a.dw, 4 * sizeof(O));
    const auto fn = wide ? finish_kernel<O, 4> : finish_kernel<O, 1>;
    if (a.tiles == 0) { // nothing of this call to be chained to
        fn<<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
    return launch_chained(fn, grid, kThreads, st, a);
}

template <typename T, typename O> cudaError_t sum_any(const SumArgs &a, cudaStream_t st)
{
    // the widest packs at which every row of dout and of the table is aligned
    const size_t dim = (size_t)a.dim;
    const auto fits = [&](int v) {
        return pack_fits(a.dout, dim * sizeof(T), v * sizeof(T)) &&
               pack_fits(a.dw, dim * sizeof(O), std::min(v * sizeof(O), (size_t)16));
    };
    if (fits(16 / sizeof(T)))
        return sum_rows<T, O, 16 / sizeof(T)>(a, st);
    if (fits(8 / sizeof(T)))
        return sum_rows<T, O, 8 / sizeof(T)>(a, st);
    if (sizeof(T) == 2 && fits(2))
        return sum_rows<T, O, 4 / sizeof(T)>(a, st);
    return sum_rows<T, O, 1>(a, st);
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
    if (!holdable(vocab, dim, es) || !holdable(ntokens, dim, es))
        return RRA_ERR_INVALID;
    if (!weight || !tokens || !out || !aligned_to(weight, es) || !aligned_to(out, es) ||
        !aligned_to(tokens, is) || overlap(weight, vocab * dim * es, out, ntokens * dim * es) ||
        overlap(tokens, ntokens * is, out, ntokens * dim * es))
        return RRA_ERR_INVALID;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool wide = index == RRA_I64;
    if (dtype == RRA_F32)
        return launched(
            lookup_any<float>(weight, tokens, ntokens, vocab, dim, wide, scale, out, st));
    if (dtype == RRA_F16)
        return launched(
            lookup_any<__half>(weight, tokens, ntokens, vocab, dim, wide, scale, out, st));
    return launched(
        lookup_any<__nv_bfloat16>(weight, tokens, ntokens, vocab, dim, wide, scale, out, st));
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
    if (!holdable(vocab, dim, os) || !holdable(ntokens, dim, es))
        return RRA_ERR_INVALID;
    if (!aligned_to(dweight, os) ||
        (ntokens > 0 &&
         (!dout || !tokens || !aligned_to(dout, es) || !aligned_to(tokens, is) ||
          overlap(dout, ntokens * dim * es, dweight, vocab * dim * os) ||
          overlap(tokens, ntokens * is, dweight, vocab * dim * os))))
        return RRA_ERR_INVALID;
    if (dweight_t != dout_t && dweight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const long long n = (long long)ntokens;
    SumArgs sum{};
    sum.n = (uint32_t)n;
    sum.vocab = (long long)vocab;
    sum.dim = (long long)dim;
    // Long tiles leave few partial sums, short ones give every SM work.
    while (sum.lg < 5 && (8ull << sum.lg) < dim)
        ++sum.lg;
    sum.slabs = (uint32_t)((dim + (8 << sum.lg) - 1) / (8 << sum.lg));
    sum.places = kMostPlaces;
    while (sum.places > 8 && n * sum.slabs < (long long)sum.places * 16 * num_sms())
        sum.places /= 2;
    sum.tiles = (uint32_t)((n + sum.places - 1) / sum.places);
    sum.sums = (long long)sum.tiles * sum.slabs;
    const long long places = (n + kMostPlaces - 1) / kMostPlaces * kMostPlaces; // whole tiles
    const bool large = n > kCsMost;
    // every part is a multiple of 128 bytes, so that packs of all are aligned
    const size_t pairs = sizeof(uint2) * places * (large ? 2 : 1),
                 counts = large ? sizeof(uint32_t) * kDigits * (sort_tiles(n) + 1) : 0,
                 marks = accumulate ? 0 : ((size_t)present_words(vocab) * 4 + 127) / 128 * 128,
                 lists = (sizeof(uint4) * (2 * (size_t)sum.tiles + 1) + 127) / 128 * 128,
                 parts = sizeof(float) * 2 * sum.tiles * dim;
    std::unique_lock<std::mutex> lk;
    unsigned char *ws = nullptr;
    const rra_status s = op_scratch(st, kScratchHead + pairs + counts + marks + lists + parts, lk, &ws);
    if (s != RRA_OK)
        return s;
    ws += kScratchHead;
    uint2 *const pair[2] = {reinterpret_cast<uint2 *>(ws), reinterpret_cast<uint2 *>(ws) + places};
    sum.dout = dout;
    sum.scale = scale;
    sum.dw = dweight;
    sum.accumulate = accumulate;
    unsigned char *const after = ws + pairs + counts;
    sum.present = accumulate ? nullptr : reinterpret_cast<uint32_t *>(after);
    sum.joins = reinterpret_cast<uint32_t *>(after + marks);
    sum.list = reinterpret_cast<uint4 *>(after + marks) + 1;
    sum.part = reinterpret_cast<float *>(after + marks + lists);
    const Tokens t{tokens, index == RRA_I64, (uint32_t)n, (long long)vocab, padding};
    cudaError_t e = cudaSuccess;
    if (large) {
        e = many_sort(t, pair, reinterpret_cast<uint32_t *>(ws + pairs), sum.joins, sum.present,
                      &sum.pair, st);
    } else {
        sum.pair = pair[0];
        if (n > 0)
            e = cluster_sort(t, pair[0], sum.joins, sum.present, st);
    }
    if (e != cudaSuccess)
        return RRA_ERR_CUDA;
    if (dout_t == RRA_F32)
        e = sum_any<float, float>(sum, st);
    else if (dout_t == RRA_F16 && dweight_t == RRA_F16)
        e = sum_any<__half, __half>(sum, st);
    else if (dout_t == RRA_F16)
        e = sum_any<__half, float>(sum, st);
    else if (dweight_t == RRA_BF16)
        e = sum_any<__nv_bfloat16, __nv_bfloat16>(sum, st);
    else
        e = sum_any<__nv_bfloat16, float>(sum, st);
    return launched(e);
}
