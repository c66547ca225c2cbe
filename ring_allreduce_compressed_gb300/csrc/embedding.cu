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

// ---------------------------------------------------------------- sort in a cluster
//
// Up to 16 x 8192 tokens are sorted by one cluster of up to 16 blocks in one
// launch: the pairs stay in registers, a pass's counts and the moved pairs go
// through distributed shared memory, and digits of up to 10 bits make two
// passes of a vocabulary below 2^20.

constexpr int kCsThreads = 1024, kCsWarps = kCsThreads / 32;
constexpr int kCsMostBits = 10, kCsMostRounds = 8, kCsMostBlocks = 16;
constexpr long long kCsMost = (long long)kCsMostBlocks * kCsThreads * kCsMostRounds;

struct ClusterSortArgs {
    const void *tok;
    int wide;
    uint32_t n;
    long long vocab, padding;
    uint32_t *key, *pos; // sorted
    int bits, passes;    // of a digit; digits
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_blocks()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// Shared-memory address of the same place in another block of the cluster.
__device__ __forceinline__ uint32_t remote(uint32_t at, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}

// The next kernel of the stream may start its blocks now; what it reads of
// this one it waits for (dependents_wait).
__device__ __forceinline__ void dependents_launch()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Until the kernels before this one have ended and their writes are visible.
__device__ __forceinline__ void dependents_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int R> // rounds: pairs per thread
__global__ void __launch_bounds__(kCsThreads) cluster_sort_kernel(const ClusterSortArgs a)
{
    constexpr uint32_t kLocal = kCsThreads * R; // pairs of a block
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t digits = 1u << a.bits;
    uint2 *const buf = reinterpret_cast<uint2 *>(smem);                   // [kLocal]
    uint32_t *const table = reinterpret_cast<uint32_t *>(buf + kLocal);  // [blocks][digits]
    const uint32_t blocks = cluster_blocks(), me = cluster_rank();
    uint32_t *const base = table + blocks * digits;                      // [digits]
    uint16_t *const cnt = reinterpret_cast<uint16_t *>(base + digits);   // [warp][digits]
    __shared__ uint32_t sums[kCsWarps];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    uint16_t *const mine = cnt + w * digits;
    dependents_launch();

    uint32_t key[R], pos[R], rank[R];
    const uint32_t local = w * (32 * R) + lane, first = me * kLocal + local;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t i = first + r * 32;
        pos[r] = i;
        key[r] = 0;
        if (i < a.n) {
            const long long v = a.wide ? static_cast<const long long *>(a.tok)[i]
                                       : (long long)static_cast<const int *>(a.tok)[i];
            key[r] = (uint32_t)(v >= 0 && v < a.vocab && v != a.padding ? v : a.vocab);
        }
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.bits;
        for (uint32_t d = lane; d < digits; d += 32)
            mine[d] = 0;
        __syncwarp();
        // place of every pair among its warp's pairs of the same digit
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool on = first + r * 32 < a.n;
            const uint32_t d = on ? (key[r] >> shift) & (digits - 1) : digits;
            const uint32_t same = __match_any_sync(kFull, d);
            const uint32_t before = __popc(same & ((1u << lane) - 1));
            uint32_t at = 0;
            if (on)
                at = mine[d];
            __syncwarp();
            rank[r] = at + before;
            if (on && before == 0)
                mine[d] = (uint16_t)(at + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        // thread d: digit d's pairs before each warp, and the block's total,
        // which goes to every block of the cluster
        if (threadIdx.x < digits) {
            uint32_t at = 0;
            for (int k = 0; k < kCsWarps; ++k) {
                const uint32_t c = cnt[k * digits + threadIdx.x];
                cnt[k * digits + threadIdx.x] = (uint16_t)at;
                at += c;
            }
            const uint32_t to = smem_u32(table + me * digits + threadIdx.x);
            for (uint32_t b = 0; b < blocks; ++b)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(to, b)), "r"(at)
                             : "memory");
        }
        cluster_sync();
        { // first place of every digit's pairs of this block
            uint32_t total = 0, before = 0;
            if (threadIdx.x < digits)
                for (uint32_t b = 0; b < blocks; ++b) {
                    const uint32_t c = table[b * digits + threadIdx.x];
                    before += b < me ? c : 0;
                    total += c;
                }
            uint32_t x = total;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kFull, x, o);
                if (lane >= o)
                    x += y;
            }
            if (lane == 31)
                sums[w] = x;
            __syncthreads();
            if (w == 0) {
                const uint32_t v = sums[lane];
                uint32_t y = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t z = __shfl_up_sync(kFull, y, o);
                    if (lane >= o)
                        y += z;
                }
                sums[lane] = y - v;
            }
            __syncthreads();
            if (threadIdx.x < digits)
                base[threadIdx.x] = sums[w] + x - total + before;
        }
        __syncthreads();
        const bool end = pass == a.passes - 1;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (first + r * 32 >= a.n)
                continue;
            const uint32_t d = (key[r] >> shift) & (digits - 1);
            const uint32_t g = base[d] + mine[d] + rank[r];
            if (end) {
                a.key[g] = key[r];
                a.pos[g] = pos[r];
            } else {
                const uint32_t to = remote(smem_u32(buf + g % kLocal), g / kLocal);
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(key[r]),
                             "r"(pos[r])
                             : "memory");
            }
        }
        if (!end) {
            cluster_sync();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint2 p = buf[local + r * 32];
                key[r] = p.x;
                pos[r] = p.y;
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
//
// The sorted places are cut into tiles of kPlaces.  A group of 2^lg lanes adds
// the rows of one tile over a slab of 8 columns a lane, all in registers, and
// writes a row of the table when its last term has come.  A row whose terms
// cross a tile's edge leaves a partial sum on either side (slot 0 of a tile:
// the row that came in, slot 1: the row that goes on), which join_kernel adds
// in the order of the tiles.  So a frequent token's terms are spread over as
// many groups as there are tiles of it.

constexpr int kPlaces = 32;
// Rows in flight: 32 registers a lane.
template <typename T, int V> constexpr int kBatchOf = sizeof(T) * V >= 4 ? 16 / sizeof(T) : 4;

struct SumArgs {
    const void *dout;
    const uint32_t *key, *pos;
    uint32_t n;
    long long vocab, dim;
    float scale;
    void *dw;
    int accumulate;
    float *part; // [tile][2][dim]
    uint32_t tiles, slabs;
    int lg;
    int zero_rows; // table rows of one group that clears what no token has
    long long sums, items;
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
    const uint32_t lo = tile * kPlaces, hi = min(lo + kPlaces, a.n);
    const uint32_t vocab = (uint32_t)a.vocab;
    uint32_t cur = a.key[lo];
    if (cur >= vocab)
        return;
    bool head = lo > 0 && a.key[lo - 1] == cur;
    const uint32_t next = hi < a.n ? a.key[hi] : vocab;
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

    for (uint32_t i = lo; i < hi; i += kBatch) {
        uint32_t key[kBatch], pos[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch / 4; ++q) {
            // the arrays go on to a whole tile
            const uint4 x = *reinterpret_cast<const uint4 *>(a.key + i + 4 * q);
            const uint4 y = *reinterpret_cast<const uint4 *>(a.pos + i + 4 * q);
            key[4 * q] = x.x; key[4 * q + 1] = x.y; key[4 * q + 2] = x.z; key[4 * q + 3] = x.w;
            pos[4 * q] = y.x; pos[4 * q + 1] = y.y; pos[4 * q + 2] = y.z; pos[4 * q + 3] = y.w;
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
    emit(next == cur);
}

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

// A warp clears those of its stretch of table rows that no token has.
template <typename O>
__device__ __forceinline__ void clear_rows(const SumArgs &a, long long v0, int lane)
{
    const long long v = v0 + lane;
    bool absent = false;
    if (lane < a.zero_rows && v < a.vocab) {
        const uint32_t at = lower_bound(a.key, a.n, (uint32_t)v);
        absent = at >= a.n || a.key[at] != (uint32_t)v;
    }
    unsigned left = __ballot_sync(kFull, absent);
    const bool vec = pack_fits(a.dw, a.dim * sizeof(O), 16);
    constexpr int V = 16 / sizeof(O);
    while (left) {
        const int r = __ffs(left) - 1;
        left &= left - 1;
        O *const q = static_cast<O *>(a.dw) + (v0 + r) * a.dim;
        if (vec) {
            for (long long c = lane * V; c < a.dim; c += 32 * V)
                *reinterpret_cast<uint4 *>(q + c) = make_uint4(0, 0, 0, 0);
        } else {
            for (long long c = lane; c < a.dim; c += 32)
                q[c] = from_f32<O>(0.0f);
        }
    }
}

template <typename T, typename O, int V>
__global__ void __launch_bounds__(kThreads, 3) sum_kernel(const SumArgs a)
{
    dependents_launch();
    dependents_wait();
    const long long thread = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long step = (long long)gridDim.x * kThreads;
    // groups add tiles, then warps clear rows
    for (long long g = thread >> a.lg; g < a.sums; g += step >> a.lg) {
        const uint32_t tile = (uint32_t)(g / a.slabs);
        sum_tile<T, O, V>(a, tile, (uint32_t)(g - (long long)tile * a.slabs),
                          threadIdx.x & ((1 << a.lg) - 1));
    }
    for (long long g = thread / 32; g < a.items; g += step / 32)
        clear_rows<O>(a, g * a.zero_rows, threadIdx.x % 32);
}

// Rows of terms that cross an edge.  Warp w of a block looks at the far edge
// of tile 8 b + w: where a row goes on there that began in the tile, its
// partial sums are added in the order of the tiles; more than kFew of them by
// the whole block, an eighth a warp.
constexpr int kFew = 16;
constexpr int kJoinCols = 512; // columns of a block

template <typename O, int V>
__global__ void __launch_bounds__(kThreads) join_kernel(const SumArgs a)
{
    constexpr int K = 4 / V;
    __shared__ uint32_t many[kWarps];
    __shared__ float sm[kWarps][32 * 4];
    dependents_wait();
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const uint32_t tile = blockIdx.x * kWarps + w, vocab = (uint32_t)a.vocab;
    uint32_t parts = 0, v = 0;
    if (tile + 1 < a.tiles) {
        const uint32_t lo = tile * kPlaces;
        v = a.key[lo + kPlaces - 1];
        const bool starts = lo == 0 || a.key[lo - 1] != v;
        if (v < vocab && a.key[lo + kPlaces] == v && (starts || a.key[lo] != v)) {
            // tiles that begin with the row go on with it
            parts = 1;
            for (uint32_t u = tile + 1;; u += 32) {
                const uint32_t t = u + lane;
                const unsigned in =
                    __ballot_sync(kFull, t < a.tiles && a.key[(size_t)t * kPlaces] == v);
                const int run = __ffs(~in) - 1;
                parts += run < 0 ? 32 : run;
                if (run >= 0)
                    break;
            }
        }
    }
    if (lane == 0)
        many[w] = parts > kFew ? parts : 0;
    __syncthreads();
    const long long c_lo = (long long)blockIdx.y * kJoinCols;
    const long long c_hi = min(c_lo + kJoinCols, a.dim);

    // partial p of the row that begins in tile t
    const auto add = [&](uint32_t t, uint32_t p0, uint32_t p1, long long c, float (&acc)[K][V]) {
#pragma unroll 8
        for (uint32_t p = p0; p < p1; ++p) {
            const float *const q = a.part + ((long long)(t + p) * 2 + (p == 0 ? 1 : 0)) * a.dim;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c + k * 32 * V < c_hi) {
                    const Pack<float, V> x = load_pack<float, V>(q + c + k * 32 * V);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        acc[k][j] += x.e[j];
                }
        }
    };
    const auto put = [&](uint32_t row, long long c, const float (&acc)[K][V]) {
        O *const q = static_cast<O *>(a.dw) + (long long)row * a.dim;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c + k * 32 * V < c_hi)
                put_final<O, V>(q + c + k * 32 * V, acc[k], a);
    };

    if (parts > 0 && parts <= kFew)
        for (long long c = c_lo + lane * V; c - lane * V < c_hi; c += 128) {
            float acc[K][V] = {};
            add(tile, 0, parts, c, acc);
            put(v, c, acc);
        }
    for (int k = 0; k < kWarps; ++k) {
        const uint32_t n = many[k];
        if (n == 0)
            continue;
        const uint32_t t = blockIdx.x * kWarps + k;
        for (long long c = c_lo + lane * V; c - lane * V < c_hi; c += 128) {
            float acc[K][V] = {};
            add(t, (uint32_t)((unsigned long long)n * w / kWarps),
                (uint32_t)((unsigned long long)n * (w + 1) / kWarps), c, acc);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    sm[w][(i * V + j) * 32 + lane] = acc[i][j];
            __syncthreads();
            if (w == 0) {
#pragma unroll
                for (int i = 0; i < K; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float s = 0.0f;
                        for (int q = 0; q < kWarps; ++q)
                            s += sm[q][(i * V + j) * 32 + lane];
                        acc[i][j] = s;
                    }
                put(a.key[(size_t)t * kPlaces + kPlaces - 1], c, acc);
            }
        }
    }
}

// Launch after which the next kernel of the stream may start early.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*fn)(P...), dim3 grid, int threads, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute at[1] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <int R> cudaError_t cluster_sort(const ClusterSortArgs &a, int blocks, cudaStream_t st)
{
    const size_t digits = (size_t)1 << a.bits;
    const int smem = (int)(8 * (size_t)kCsThreads * R + 4 * digits * blocks + 4 * digits +
                           2 * digits * kCsWarps);
    cudaError_t e = cudaFuncSetAttribute(cluster_sort_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(cluster_sort_kernel<R>,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kCsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cluster_sort_kernel<R>, a);
}

cudaError_t cluster_sort(ClusterSortArgs a, cudaStream_t st)
{
    int bits = 1;
    while (((unsigned long long)a.vocab >> bits) != 0)
        ++bits;
    a.passes = (bits + kCsMostBits - 1) / kCsMostBits;
    a.bits = (bits + a.passes - 1) / a.passes;
    int blocks = 1, rounds = 1;
    while (blocks < kCsMostBlocks && (long long)blocks * kCsThreads < a.n)
        blocks *= 2;
    while ((long long)blocks * kCsThreads * rounds < a.n)
        rounds *= 2;
    switch (rounds) {
    case 1: return cluster_sort<1>(a, blocks, st);
    case 2: return cluster_sort<2>(a, blocks, st);
    case 4: return cluster_sort<4>(a, blocks, st);
    default: return cluster_sort<8>(a, blocks, st);
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

template <typename T, typename O, int V> cudaError_t sum_rows(SumArgs a, cudaStream_t st)
{
    a.lg = 0;
    while (a.lg < 5 && (8LL << a.lg) < a.dim)
        ++a.lg;
    a.slabs = (uint32_t)((a.dim + (8 << a.lg) - 1) / (8 << a.lg));
    a.sums = (long long)a.tiles * a.slabs;
    a.zero_rows = a.vocab >= 1 << 17 ? 32 : 8;
    a.items = a.accumulate ? 0 : (a.vocab + a.zero_rows - 1) / a.zero_rows;
    const long long warps = std::max(((a.sums << a.lg) + 31) / 32, a.items);
    cudaError_t e = launch_chained(sum_kernel<T, O, V>, dim3(grid_of((warps + kWarps - 1) / kWarps, 32)),
                                   kThreads, st, a);
    if (e != cudaSuccess || a.tiles < 2)
        return e;
    const dim3 grid((a.tiles - 1 + kWarps - 1) / kWarps,
                    (unsigned)((a.dim + kJoinCols - 1) / kJoinCols));
    if (a.dim % 4 == 0 && aligned_to(a.dw, 4 * sizeof(O)))
        return launch_chained(join_kernel<O, 4>, grid, kThreads, st, a);
    return launch_chained(join_kernel<O, 1>, grid, kThreads, st, a);
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
    const long long n = (long long)ntokens;
    const long long places = (n + kPlaces - 1) / kPlaces * kPlaces; // whole tiles
    const long long sort_tiles = (n + kSortTile - 1) / kSortTile;
    const bool large = n > kCsMost;
    const size_t arrays = sizeof(uint32_t) * places * (large ? 4 : 2),
                 counts = large ? sizeof(uint32_t) * kDigits * (sort_tiles + 4) : 0,
                 parts = sizeof(float) * 2 * (places / kPlaces) * dim;
    std::unique_lock<std::mutex> lk;
    unsigned char *ws = nullptr;
    const rra_status s = op_scratch(st, kScratchHead + arrays + counts + parts, lk, &ws);
    if (s != RRA_OK)
        return s;
    SumArgs sum{};
    sum.dout = dout;
    sum.n = (uint32_t)n;
    sum.vocab = (long long)vocab;
    sum.dim = (long long)dim;
    sum.scale = scale;
    sum.dw = dweight;
    sum.accumulate = accumulate;
    sum.tiles = (uint32_t)(places / kPlaces);
    // the arrays of places and the counts are multiples of 128 bytes, so that
    // every pack of them and of the partial sums behind them is aligned
    uint32_t *const key = reinterpret_cast<uint32_t *>(ws + kScratchHead);
    sum.part = reinterpret_cast<float *>(ws + kScratchHead + arrays + counts);
    cudaError_t e = cudaSuccess;
    if (!large) {
        sum.key = key;
        sum.pos = key + places;
        if (n > 0)
            e = cluster_sort({tokens, index == RRA_I64, (uint32_t)n, (long long)vocab, padding,
                              key, key + places, 0, 0},
                             st);
    } else {
        SortArgs a{};
        a.hist = key + 4 * places;
        a.total = a.hist + kDigits * sort_tiles;
        a.n = n;
        a.vocab = (long long)vocab;
        a.padding = padding;
        a.tiles = sort_tiles;
        a.wide = index == RRA_I64;
        int at = 0;
        for (int shift = 0; shift == 0 || (vocab >> shift) != 0; shift += 8) {
            a.tok = shift == 0 ? tokens : nullptr;
            a.key_in = key + at * places;
            a.pos_in = key + (2 + at) * places;
            a.key_out = key + (at ^ 1) * places;
            a.pos_out = key + (2 + (at ^ 1)) * places;
            a.shift = shift;
            sort_count_kernel<<<(unsigned)sort_tiles, kThreads, 0, st>>>(a);
            sort_scan_kernel<<<kDigits, kThreads, 0, st>>>(a);
            sort_move_kernel<<<(unsigned)sort_tiles, kThreads, 0, st>>>(a);
            at ^= 1;
        }
        sum.key = key + at * places;
        sum.pos = key + (2 + at) * places;
        e = cudaGetLastError();
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
