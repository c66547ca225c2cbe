// token_sort.cuh -- stable sort of token numbers for the embedding's gradient:
// (token, position) pairs by token, equal tokens in the order of their
// positions.  Least significant digit first.  Tokens that get no gradient
// (outside the table, padding) sort behind all others, as `vocab`.
//
// Up to 16 x 8192 tokens are sorted by one cluster of up to 16 blocks in one
// launch, in shared memory; more take three launches a digit.
#pragma once

#include "op_common.cuh"

namespace rra {
namespace {

struct Tokens {
    const void *tok;
    int wide; // 64-bit
    uint32_t n;
    long long vocab, padding;
};

__device__ __forceinline__ uint32_t token_key(const Tokens &a, uint32_t i)
{
    const long long v = a.wide ? static_cast<const long long *>(a.tok)[i]
                               : (long long)static_cast<const int *>(a.tok)[i];
    return (uint32_t)(v >= 0 && v < a.vocab && v != a.padding ? v : a.vocab);
}

// Words of a bit for every token.
__host__ __device__ inline uint32_t present_words(long long vocab)
{
    return (uint32_t)((vocab + 31) / 32);
}

// Lanes of the warp with the same digit of `bits` bits; lanes that are not
// `on` stand apart.  One vote a bit.
__device__ __forceinline__ uint32_t same_digit(uint32_t d, int bits, bool on)
{
    uint32_t same = __ballot_sync(kFull, on);
    if (!on)
        same = ~same;
#pragma unroll 4
    for (int b = 0; b < bits; ++b) {
        const bool bit = (d >> b) & 1;
        const uint32_t set = __ballot_sync(kFull, bit);
        same &= bit ? set : ~set;
    }
    return same;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t x)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, x, o);
        if (threadIdx.x % 32 >= o)
            x += y;
    }
    return x;
}

// Exclusive sum of v over the WARPS * 32 threads of a block; *sum: the total.
template <int WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *sm, uint32_t *sum)
{
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const uint32_t x = warp_scan(v);
    if (lane == 31)
        sm[w] = x;
    __syncthreads();
    const uint32_t mine = lane < WARPS ? sm[lane] : 0, upto = warp_scan(mine);
    *sum = __shfl_sync(kFull, upto, WARPS - 1);
    const uint32_t before = __shfl_sync(kFull, upto - mine, w);
    __syncthreads();
    return before + x - v;
}

// ---------------------------------------------------------------- one cluster
//
// The pairs stay in registers.  A pass ranks a warp's pairs by digit, sums
// the counts over the block and, through distributed shared memory, over the
// cluster, and moves every pair to its place: first among the block's own
// pairs, so that pairs of a digit lie side by side and leave for the same
// block in runs (29 us for 131072 tokens; 34 us when they were moved straight
// from the registers, each word of a store to anywhere).  11 us for 16384
// tokens: barriers and the exchange of counts, not bytes.

constexpr int kCsThreads = 1024, kCsWarps = kCsThreads / 32;
constexpr int kCsMostRounds = 8, kCsMostBlocks = 16;
constexpr long long kCsMost = (long long)kCsMostBlocks * kCsThreads * kCsMostRounds;

// Bits of a digit: what the counts leave room for.
constexpr int cs_most_bits(int rounds) { return rounds == kCsMostRounds ? 9 : 10; }

struct ClusterSortArgs {
    Tokens t;
    uint2 *pair;         // sorted
    uint32_t *joins;     // two counts that later kernels use, cleared here
    uint32_t *present;   // a bit for every token < vocab: is it there? May be nullptr
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

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    cluster_wait();
}

// The first half of a barrier that says only that this block has started.
__device__ __forceinline__ void cluster_started()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// Shared-memory address of the same place in another block of the cluster.
__device__ __forceinline__ uint32_t remote(uint32_t at, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}

template <int R> // rounds: pairs per thread
__global__ void __launch_bounds__(kCsThreads) cluster_sort_kernel(const ClusterSortArgs a)
{
    constexpr uint32_t kLocal = kCsThreads * R; // pairs of a block
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t digits = 1u << a.bits, blocks = cluster_blocks(), me = cluster_rank();
    uint2 *const buf = reinterpret_cast<uint2 *>(smem);              // [kLocal], from all blocks
    uint2 *const stage = buf + kLocal;                               // [kLocal], own
    uint32_t *const table = reinterpret_cast<uint32_t *>(stage + kLocal); // [blocks][digits]
    uint32_t *const first_own = table + blocks * digits;             // [digits], in stage
    uint32_t *const first_all = first_own + digits;                  // [digits], less the former
    uint16_t *const cnt = reinterpret_cast<uint16_t *>(first_all + digits); // [warp][digits]
    __shared__ uint32_t sums[kCsWarps];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    uint16_t *const mine = cnt + w * digits;
    const uint32_t n = a.t.n;
    cluster_started();
    dependents_wait();
    dependents_launch();
    if (me == 0 && threadIdx.x < 2)
        a.joins[threadIdx.x] = 0;
    if (a.present) {
        const uint32_t words = present_words(a.t.vocab);
        for (uint32_t i = me * kCsThreads + threadIdx.x; i < words; i += blocks * kCsThreads)
            a.present[i] = 0;
    }

    // a warp holds a stretch of the block's pairs, 32 a round
    uint32_t key[R], pos[R], rank[R];
    const uint32_t local = w * (32 * R) + lane, first = me * kLocal + local;
    const uint32_t held = min(n - min(n, me * kLocal), kLocal); // pairs of this block
    const int used = (held + 32 * R - 1) / (32 * R);            // warps that hold them
#pragma unroll
    for (int r = 0; r < R; ++r) {
        pos[r] = first + r * 32;
        key[r] = pos[r] < n ? token_key(a.t, pos[r]) : 0u;
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.bits;
        if (w < used) {
            for (uint32_t d = lane; d < digits / 2; d += 32)
                reinterpret_cast<uint32_t *>(mine)[d] = 0;
            __syncwarp();
            // place of every pair among its warp's pairs of the same digit
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool on = first + r * 32 < n;
                const uint32_t d = (key[r] >> shift) & (digits - 1);
                const uint32_t same = same_digit(d, a.bits, on);
                const uint32_t before = __popc(same & ((1u << lane) - 1));
                const uint32_t at = on ? mine[d] : 0;
                __syncwarp();
                rank[r] = at + before;
                if (on && before == 0)
                    mine[d] = (uint16_t)(at + __popc(same));
                __syncwarp();
            }
        }
        __syncthreads();
        // A block's shared memory may be written by others once it is known to
        // have started: blocks of a cluster are scheduled together, but nothing
        // says that they have all begun.  The wait's other half stands at the
        // kernel's beginning, so that ranking the first digit hides it.
        if (pass == 0)
            cluster_wait();
        // thread d: digit d's pairs before each warp, and the block's total,
        // which goes to every block of the cluster
        uint32_t own = 0;
        if (threadIdx.x < digits) {
#pragma unroll 8
            for (int k = 0; k < used; ++k) {
                const uint32_t c = cnt[k * digits + threadIdx.x];
                cnt[k * digits + threadIdx.x] = (uint16_t)own;
                own += c;
            }
            const uint32_t to = smem_u32(table + me * digits + threadIdx.x);
            for (uint32_t b = 0; b < blocks; ++b)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(to, b)), "r"(own)
                             : "memory");
        }
        cluster_sync();
        { // first places of the digits: in the block (14 bits) and in all (18 bits)
            uint32_t all = 0, before = 0, sum;
            if (threadIdx.x < digits)
#pragma unroll 4
                for (uint32_t b = 0; b < blocks; ++b) {
                    const uint32_t c = table[b * digits + threadIdx.x];
                    before += b < me ? c : 0;
                    all += c;
                }
            const uint32_t x = block_scan<kCsWarps>(own << 18 | all, sums, &sum);
            if (threadIdx.x < digits) {
                first_own[threadIdx.x] = x >> 18;
                first_all[threadIdx.x] = (x & 0x3ffffu) + before - (x >> 18);
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (first + r * 32 < n) {
                const uint32_t d = (key[r] >> shift) & (digits - 1);
                stage[first_own[d] + mine[d] + rank[r]] = make_uint2(key[r], pos[r]);
            }
        __syncthreads();
        const bool end = pass == a.passes - 1;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t j = r * kCsThreads + threadIdx.x;
            if (j >= held)
                continue;
            const uint2 p = stage[j];
            const uint32_t g = first_all[(p.x >> shift) & (digits - 1)] + j;
            if (end) {
                a.pair[g] = p;
                // the block's pairs are sorted here, too: one of a token's marks it
                if (a.present && p.x < a.t.vocab && (j == 0 || stage[j - 1].x != p.x))
                    atomicOr(a.present + p.x / 32, 1u << p.x % 32);
            } else {
                const uint32_t to = remote(smem_u32(buf + g % kLocal), g / kLocal);
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(p.x),
                             "r"(p.y)
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

template <int R> cudaError_t cluster_sort(ClusterSortArgs a, int key_bits, int blocks,
                                          cudaStream_t st)
{
    a.passes = (key_bits + cs_most_bits(R) - 1) / cs_most_bits(R);
    a.bits = (key_bits + a.passes - 1) / a.passes;
    const size_t digits = (size_t)1 << a.bits;
    const size_t smem = 16 * (size_t)kCsThreads * R + 4 * digits * (blocks + 2) +
                        2 * digits * kCsWarps;
    const cudaError_t e =
        op_allow(reinterpret_cast<const void *>(cluster_sort_kernel<R>), (int)smem, true);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kCsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, cluster_sort_kernel<R>, a);
}

// Up to kCsMost tokens, at least one.
inline cudaError_t cluster_sort(const Tokens &t, uint2 *pair, uint32_t *joins, uint32_t *present,
                                cudaStream_t st)
{
    int key_bits = 1;
    while (((unsigned long long)t.vocab >> key_bits) != 0)
        ++key_bits;
    int blocks = 1, rounds = 1;
    while (blocks < kCsMostBlocks && (long long)blocks * kCsThreads < t.n)
        blocks *= 2;
    while ((long long)blocks * kCsThreads * rounds < t.n)
        rounds *= 2;
    const ClusterSortArgs a{t, pair, joins, present, 0, 0};
    switch (rounds) {
    case 1: return cluster_sort<1>(a, key_bits, blocks, st);
    case 2: return cluster_sort<2>(a, key_bits, blocks, st);
    case 4: return cluster_sort<4>(a, key_bits, blocks, st);
    default: return cluster_sort<8>(a, key_bits, blocks, st);
    }
}

// ---------------------------------------------------------------- many tokens
//
// 8 bits a pass.  A pass counts the digits of every tile, turns the counts
// into places, and moves the tile's pairs there; a tile's pairs keep their
// order.
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kDigits = 256;
constexpr int kSortTile = 4096;
constexpr int kSortRounds = kSortTile / kSortThreads;

struct SortArgs {
    Tokens t;
    const uint2 *in; // nullptr: the tokens
    uint2 *out;
    uint32_t *hist;  // [digit][tile]
    uint32_t *total; // [digit]
    long long tiles;
    int shift;
};

__device__ __forceinline__ uint2 sort_pair(const SortArgs &a, uint32_t i)
{
    return a.in ? a.in[i] : make_uint2(token_key(a.t, i), i);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a)
{
    __shared__ uint32_t cnt[kDigits];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t base = blockIdx.x * kSortTile;
    for (int r = 0; r < kSortRounds; ++r) {
        const uint32_t i = base + r * kSortThreads + threadIdx.x;
        if (i < a.t.n)
            atomicAdd(&cnt[((a.in ? a.in[i].x : token_key(a.t, i)) >> a.shift) & (kDigits - 1)],
                      1u);
    }
    __syncthreads();
    a.hist[threadIdx.x * a.tiles + blockIdx.x] = cnt[threadIdx.x];
}

// One block per digit: its tiles' counts become the places behind the digit's
// first.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(const SortArgs a)
{
    __shared__ uint32_t sm[kSortWarps];
    uint32_t run = 0;
    uint32_t *const h = a.hist + blockIdx.x * a.tiles;
    for (long long b = 0; b < a.tiles; b += kSortThreads) {
        const long long i = b + threadIdx.x;
        uint32_t sum;
        const uint32_t x = block_scan<kSortWarps>(i < a.tiles ? h[i] : 0u, sm, &sum);
        if (i < a.tiles)
            h[i] = run + x;
        run += sum;
    }
    if (threadIdx.x == 0)
        a.total[blockIdx.x] = run;
}

__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const SortArgs a)
{
    __shared__ uint32_t cnt[kSortWarps][kDigits];
    __shared__ uint32_t sm[kSortWarps];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    for (int d = lane; d < kDigits; d += 32)
        cnt[w][d] = 0;
    uint32_t sum;
    const uint32_t first = block_scan<kSortWarps>(a.total[threadIdx.x], sm, &sum);
    __syncwarp();
    // a warp takes a stretch of the tile, 32 pairs a round
    const uint32_t base = blockIdx.x * kSortTile + w * (kSortTile / kSortWarps) + lane;
    uint2 pair[kSortRounds];
    uint16_t rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const bool on = base + r * 32 < a.t.n;
        pair[r] = on ? sort_pair(a, base + r * 32) : make_uint2(0u, 0u);
        const uint32_t d = (pair[r].x >> a.shift) & (kDigits - 1);
        const uint32_t same = same_digit(d, 8, on);
        const uint32_t before = __popc(same & ((1u << lane) - 1));
        const uint32_t at = on ? cnt[w][d] : 0;
        __syncwarp();
        rank[r] = (uint16_t)(at + before);
        if (on && before == 0)
            cnt[w][d] = at + __popc(same);
        __syncwarp();
    }
    __syncthreads();
    { // thread d: the places of digit d of every warp's stretch
        uint32_t at = first + a.hist[threadIdx.x * a.tiles + blockIdx.x];
#pragma unroll
        for (int k = 0; k < kSortWarps; ++k) {
            const uint32_t c = cnt[k][threadIdx.x];
            cnt[k][threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r)
        if (base + r * 32 < a.t.n)
            a.out[cnt[w][(pair[r].x >> a.shift) & (kDigits - 1)] + rank[r]] = pair[r];
}

// Marks the tokens of the sorted pairs.
__global__ void __launch_bounds__(kSortThreads)
    mark_kernel(const uint2 *__restrict__ pair, uint32_t n, long long vocab, uint32_t *present)
{
    const uint32_t i = blockIdx.x * kSortThreads + threadIdx.x;
    if (i < n) {
        const uint32_t v = pair[i].x;
        if (v < vocab && (i == 0 || pair[i - 1].x != v))
            atomicOr(present + v / 32, 1u << v % 32);
    }
}

inline long long sort_tiles(long long n) { return (n + kSortTile - 1) / kSortTile; }

// Any number of tokens up to 2^31 - 1; pair[0] and pair[1] hold n pairs each,
// counts kDigits * (sort_tiles + 1) words; joins and present as above.  *out
// receives the sorted pairs.
inline cudaError_t many_sort(const Tokens &t, uint2 *const pair[2], uint32_t *counts,
                             uint32_t *joins, uint32_t *present, const uint2 **out,
                             cudaStream_t st)
{
    cudaError_t e = cudaMemsetAsync(joins, 0, 2 * sizeof(uint32_t), st);
    if (e == cudaSuccess && present)
        e = cudaMemsetAsync(present, 0, sizeof(uint32_t) * present_words(t.vocab), st);
    if (e != cudaSuccess)
        return e;
    SortArgs a{};
    a.t = t;
    a.tiles = sort_tiles(t.n);
    a.hist = counts;
    a.total = counts + kDigits * a.tiles;
    int at = 0;
    for (a.shift = 0; a.shift == 0 || ((unsigned long long)t.vocab >> a.shift) != 0;
         a.shift += 8) {
        a.in = a.shift == 0 ? nullptr : pair[at];
        a.out = pair[at ^ 1];
        sort_count_kernel<<<(unsigned)a.tiles, kSortThreads, 0, st>>>(a);
        sort_scan_kernel<<<kDigits, kSortThreads, 0, st>>>(a);
        sort_move_kernel<<<(unsigned)a.tiles, kSortThreads, 0, st>>>(a);
        at ^= 1;
    }
    if (present)
        mark_kernel<<<(t.n + kSortThreads - 1) / kSortThreads, kSortThreads, 0, st>>>(
            pair[at], t.n, t.vocab, present);
    *out = pair[at];
    return cudaGetLastError();
}

} // namespace
} // namespace rra
