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
// row among it.  Measured at 16384 x 4096 bf16: save 60 us (338 MB, 5.6 TB/s), restore 37 us
// (202 MB, 5.5 TB/s), gradient 75 us (338 MB, 4.5 TB/s: latency, with 12 warps an SM, one row
// ahead and issue slots busy 56 %; 5 of the 75 for adding the partial rows); 3001 x 1001 fp32:
// restore 7.4 us, gradient 15.6.
#include "op_common.cuh"
#include "ragged.cuh"
#include "row_group.cuh"
#include "saved.cuh"

namespace rra {
namespace {

// 8 weights as fp32 from column c (a multiple of 8) on, of which n are there; VEC: all or
// none, on a 16-byte boundary.
template <typename W, bool VEC>
__device__ __forceinline__ void weights8(const W *p, long long c, int n, float none, float v[8])
{
    if (p) {
        if (VEC || (n == 8 && aligned_to(p, 16)))
            load8<W, true>(p + c, n, v);
        else
            load8<W, false>(p + c, n, v);
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

// The pairs of a pack.
template <typename T> __device__ __forceinline__ Pair pair_in(const uint32_t *w, int j)
{
    return pair_of(element<T>(w, 2 * j), element<T>(w, 2 * j + 1));
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

// Threads of a block, wide rows apart, which need their registers.
constexpr int kSaveThreads = 256;
constexpr int kSaveHeld = 4; // packs of a lane

// Larger of the two halves of each, as unsigned numbers.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bits of the largest magnitudes of the blocks of codes that a lane's P packs are in, as
// fp32.  16-bit numbers are compared as whole numbers, two packs in a word.
template <typename T, int P>
__device__ __forceinline__ void block_tops(const uint32_t (&w)[P][kPackWords<T>], uint32_t (&top)[P])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < P; ++k) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = element<T>(w[k], j);
            top[k] = half_warp_max(top_bits(v));
        }
    } else {
        uint32_t most[P];
#pragma unroll
        for (int k = 0; k < P; ++k) {
            uint32_t m = w[k][0] & 0x7fff7fffu;
#pragma unroll
            for (int j = 1; j < 4; ++j)
                m = max_halves(m, w[k][j] & 0x7fff7fffu);
            most[k] = max_halves(m, m >> 16); // the lower half
        }
#pragma unroll
        for (int k = 0; k < P; k += 2) {
            uint32_t m = k + 1 < P ? __byte_perm(most[k], most[k + 1], 0x5410) : most[k] & 0xffffu;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                m = max_halves(m, __shfl_xor_sync(kFull, m, o));
#pragma unroll
            for (int i = 0; i < 2 && k + i < P; ++i) {
                const uint32_t h = i ? m >> 16 : m & 0xffffu;
                top[k + i] = std::is_same<T, __nv_bfloat16>::value
                                 ? h << 16
                                 : __float_as_uint(__half2float(__ushort_as_half((uint16_t)h)));
            }
        }
    }
}

// Weights of the whole packs of a row, or `none` where there is no array.
template <typename W> __device__ __forceinline__ void whole_weights(const W *p, float none, Pair (&v)[4])
{
    float t[8];
    if (p) {
        load8<W, true>(p, 8, t);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t[j] = none;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = pair_of(t[2 * j], t[2 * j + 1]);
}

// Which pack of a row is a lane's k-th: a warp of several holds 32 K neighbouring ones,
// 32 apart in a lane, so that its K are at constant distances; lanes of less than a warp
// hold every `lanes`-th.
template <int K, bool MULTI> __device__ __forceinline__ int pack_of(int li, int k, int lanes)
{
    return MULTI ? li / 32 * (32 * K) + k * 32 + li % 32 : li + k * lanes;
}

// Rows in the registers of a group of lanes, as in norm_kernel; 16 lanes of a warp hold a
// block of codes.  The next row is on its way while one is worked on (16384 x 4096 bf16:
// 78 us, and 81 without or with two rows at a time; 67 with constant distances and one
// question for special blocks; 62 with the codes in a loop of their own).
// WHOLE: every pack is whole and on a 16-byte boundary.
template <typename T, typename W, int K, bool MULTI, bool WHOLE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kSaveThreads ? 2 : 1)
    save_kernel(const Save a)
{
    constexpr int N = kPackWords<T>;
    __shared__ __align__(16) float sm[MULTI ? 2 * 32 : 4];
    const T *const x = static_cast<const T *>(a.x), *const x_end = x + a.rows * a.dim;
    T *const y = static_cast<T *>(a.y);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, groups = blockDim.x / lanes;
    const int gap = (MULTI ? 32 : lanes) * kPack; // elements between a lane's packs
    const int dim = (int)a.dim, nb = (int)blocks_of(dim), packs = nb * kBlockPacks;
    const float n = (float)dim, inverse = 1.0f / n;
    GroupOf group = group_of(a.g, sm, 1);
    if (MULTI) {
        for (int i = threadIdx.x; i < 2 * 32; i += blockDim.x)
            sm[i] = 0.0f;
        __syncthreads();
    }
    const int first = threadIdx.x / lanes, u0 = pack_of<K, MULTI>(li, 0, lanes);
    const W *const gamma = static_cast<const W *>(a.gamma),
                   *const beta = static_cast<const W *>(a.beta);
    int there[K], next[K]; // elements of the lane's packs, and of the ones behind them
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = u0 * kPack + k * gap;
        there[k] = max(0, min(kPack, dim - c));
        next[k] = max(0, min(kPack, dim - c - kPack));
    }
    const long long step = (long long)gridDim.x * groups;
    dependents_wait();
    dependents_launch();
    uint32_t ahead[K][kChunkWords<T, WHOLE>] = {}; // (what is not there stays zero)
    const auto read = [&](long long base) {
        // every lane takes part in the sums, some in vain: they read the last row
        const T *const row = x + min(base + (MULTI ? 0 : first), a.rows - 1) * dim;
        const bool inside = WHOLE || row_inside(row, dim, x, x_end);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (there[k] > 0)
                load_chunks<T, WHOLE>(row + u0 * kPack + k * gap, there[k], x, x_end, ahead[k],
                                      inside);
    };
    long long base = (long long)blockIdx.x * groups;
    read(base);
    for (; base < a.rows; base += step) {
        const long long r = min(base + (MULTI ? 0 : first), a.rows - 1);
        const bool on = MULTI || base + first < a.rows;
        uint32_t w[K][N];
#pragma unroll
        for (int k = 0; k < K; ++k)
            settle<T, WHOLE>(ahead[k], x + r * dim, there[k], w[k]);
        if (base + step < a.rows)
            read(base + step);
        Pair sum = pair_of(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum = add(sum, pair_in<T>(w[k], j));
        Sums<1> s{{sum_of(sum)}};
        const float mu = quotient(group_sum<MULTI, 1>(s, group).v[0], n, inverse);
        const Pair minus = pair_of(-mu, -mu);
        sum = pair_of(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (there[k] == kPack) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Pair d = add(pair_in<T>(w[k], j), minus);
                    sum = fma(d, d, sum);
                }
            } else if (!WHOLE && there[k] > 0) {
                float t = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = j < there[k] ? element<T>(w[k], j) - mu : 0.0f;
                    t = fmaf(d, d, t);
                }
                sum = add(sum, pair_of(t, 0.0f));
            }
        s.v[0] = sum_of(sum);
        const float rs = rsqrtf(quotient(group_sum<MULTI, 1>(s, group).v[0], n, inverse) + a.eps);
        const Pair scale = pair_of(rs, rs);
        uint32_t top[K];
        block_tops<T, K>(w, top);
        bool special = false;
#pragma unroll
        for (int k = 0; k < K; ++k)
            special = special || special_block(top[k]);
        // (one question a row: asked for every pack, its ways apart cost more than the codes.
        // Packs behind the row are zero, and so special: rows that leave some of a warp's
        // packs empty take the general code, as rows of zeros do.  About 200 MB of bf16: 76 us
        // with rows of 1536, 66 with 1024)
        const bool plain = !__any_sync(kFull, special);
        int8_t *const codes = a.codes + (r * packs + u0) * kPack;
        int8_t *const exps = a.exps + r * nb + u0 / kBlockPacks;
        const auto save_codes = [&](auto encode) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = element<T>(w[k], j);
                if (on && u0 + k * (gap / kPack) < packs) {
                    store_codes(codes + k * gap, encode(v, top[k]));
                    if (li % kBlockPacks == 0)
                        exps[k * gap / kBlock] = exponent_byte(block_exponent(top[k]));
                }
            }
        };
        if (plain)
            save_codes([](const float *v, uint32_t t) { return plain_codes8(v, t); });
        else
            save_codes([](const float *v, uint32_t t) { return encode8(v, t); });
        T *const to = y + r * dim + u0 * kPack;
        Carry<T> carry;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = u0 + k * (gap / kPack);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = element<T>(w[k], j);
            Pair g[4], b[4];
            if (WHOLE) {
                // (behind the row: its first weights, for nothing)
                const int c = there[k] ? u * kPack : 0;
                whole_weights(gamma ? gamma + c : nullptr, 1.0f, g);
                whole_weights(beta ? beta + c : nullptr, 0.0f, b);
            } else {
                float t[8];
                weights8<W, false>(gamma, u * kPack, there[k], 1.0f, t);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    g[j] = pair_of(t[2 * j], t[2 * j + 1]);
                weights8<W, false>(beta, u * kPack, there[k], 0.0f, t);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b[j] = pair_of(t[2 * j], t[2 * j + 1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                halves(fma(mul(add(pair_of(v[2 * j], v[2 * j + 1]), minus), scale), g[j], b[j]),
                       v[2 * j], v[2 * j + 1]);
            uint32_t o[N];
            to_words<T>(v, o);
            store_words<T, WHOLE>(to + k * gap, there[k], next[k], on, min(lanes, 32), o, carry,
                                  k > 0, k == K - 1);
        }
        if (on && li == 0) {
            a.mean[r] = mu;
            a.rstd[r] = rs;
        }
    }
}

// Rows that no block holds: passes over each, the later ones from L2, element by element
// (1024 x 65536 bf16: 190 us).
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
            const uint32_t top = half_warp_max(top_bits(v));
            if (u >= packs)
                continue;
            store_codes(a.codes + (r * packs + u) * kPack, encode8(v, top));
            if (u % kBlockPacks == 0)
                a.exps[r * nb + u / kBlockPacks] = exponent_byte(block_exponent(top));
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

template <typename T, typename W, int K, bool MULTI, bool WHOLE, int THREADS>
cudaError_t save_launch(const Save &a, cudaStream_t st)
{
    const int threads = MULTI ? 32 * a.g.warps : kSaveThreads, rows = threads / a.g.lanes();
    // one wave of blocks, for the rows that they have ahead (16384 x 4096 bf16: 60 us, 62
    // with three waves)
    const int per_sm = std::max(1, (K == 1 ? 1024 : 640) / threads);
    return launch_chained(save_kernel<T, W, K, MULTI, WHOLE, THREADS>,
                          dim3(grid_of((a.rows + rows - 1) / rows, per_sm)), threads, st, a);
}

template <typename T, typename W, bool WHOLE> cudaError_t save_rows(Save a, cudaStream_t st)
{
    const long long packs = blocks_of(a.dim) * kBlockPacks;
    if (packs > 1024LL * kSaveHeld)
        return launch_chained(save_long_kernel<T, W>, dim3(grid_of(a.rows, 2)), kLongThreads, st,
                              a);
    const bool few = packs <= 32;
    a.g = save_group(packs, few ? 1 : kSaveHeld);
    if (a.g.warps > 16)
        return save_launch<T, W, kSaveHeld, true, WHOLE, 1024>(a, st);
    if (a.g.warps > kSaveThreads / 32)
        return save_launch<T, W, kSaveHeld, true, WHOLE, 512>(a, st);
    if (a.g.warps > 1)
        return save_launch<T, W, kSaveHeld, true, WHOLE, kSaveThreads>(a, st);
    return few ? save_launch<T, W, 1, false, WHOLE, kSaveThreads>(a, st)
               : save_launch<T, W, kSaveHeld, false, WHOLE, kSaveThreads>(a, st);
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
    int lanes; // of a row's stretch of columns
};

constexpr int kRestoreThreads = 256;
constexpr int kRestorePack = 16; // elements of a thread in a row: 16 bytes of codes
// Rows of a thread at a time, and blocks an SM: 16384 x 4096 bf16 take 37 us with 2 and 3,
// 44 with 2 and 2, 46 with 3 and 2; 3001 x 1001 fp32, whose packs are shifted, took 9.5 us
// with 3 and 2, 12 with 2 and 3.
template <bool WHOLE> constexpr int kRestoreRows = WHOLE ? 2 : 3;
template <bool WHOLE> constexpr int kRestoreBlocks = WHOLE ? 3 : 2;
constexpr int kRestoreCols = kRestoreThreads * kRestorePack; // of a block, blockIdx.y each

// A thread keeps its columns' weights in registers over all of its rows, and has the
// codes of several rows on their way at a time.
template <typename T, typename W, bool WHOLE>
__global__ void __launch_bounds__(kRestoreThreads, kRestoreBlocks<WHOLE>)
    restore_kernel(const Restore a)
{
    constexpr int E = kRestorePack, R = kRestoreRows<WHOLE>;
    const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                static_cast<const W *>(a.beta);
    T *const y = static_cast<T *>(a.y);
    const long long nb = blocks_of(a.dim), width = nb * kBlock;
    const int groups = kRestoreThreads / a.lanes, mine = threadIdx.x / a.lanes;
    const long long step = (long long)gridDim.x * groups;
    const auto in = [&](long long c) { return (int)max(0LL, min((long long)E, a.dim - c)); };
    dependents_wait();
    dependents_launch();
    for (long long first = (long long)blockIdx.y * kRestoreCols; first < a.dim;
         first += (long long)gridDim.y * kRestoreCols) {
        const long long c0 = first + threadIdx.x % a.lanes * E;
        const int there = in(c0), next = in(c0 + E);
        Pair g[E / 2], b[E / 2];
#pragma unroll
        for (int h = 0; h < E; h += 8) {
            const int n = max(0, min(8, there - h));
            float t[8];
            weights8<W, WHOLE>(gamma, c0 + h, n, 1.0f, t);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                g[h / 2 + j] = pair_of(t[2 * j], t[2 * j + 1]);
            weights8<W, WHOLE>(beta, c0 + h, n, 0.0f, t);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[h / 2 + j] = pair_of(t[2 * j], t[2 * j + 1]);
        }
        // the rows of a block's groups go on together: whole warps store
        long long r = (long long)blockIdx.x * groups + mine; // to read, and to write
        const int8_t *codes = a.codes + r * width + c0, *exps = a.exps + r * nb + c0 / kBlock;
        T *to = y + r * a.dim + c0;
        const long long codes_step = step * width, exps_step = step * nb, to_step = step * a.dim;
        for (long long base = (long long)blockIdx.x * groups; base < a.rows; base += R * step) {
            uint4 c[R];
            int8_t e[R];
            float mu[R], rs[R];
#pragma unroll
            for (int i = 0; i < R; ++i, codes += codes_step, exps += exps_step) {
                const long long at = r + i * step;
                c[i] = make_uint4(0u, 0u, 0u, 0u);
                e[i] = 0;
                mu[i] = 0.0f;
                rs[i] = 1.0f;
                if (at < a.rows && there > 0) {
                    c[i] = *reinterpret_cast<const uint4 *>(codes);
                    e[i] = *exps;
                    if (a.mean)
                        mu[i] = a.mean[at];
                    if (a.rstd)
                        rs[i] = a.rstd[at];
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i, r += step, to += to_step) {
                const Pair minus = pair_of(-mu[i], -mu[i]), scale = pair_of(rs[i], rs[i]);
                const float s = block_scale(e[i]);
                const Pair unit = pair_of(s, s);
                uint32_t o[kPackWords<T, E>];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 f[4];
                    fractions8(h ? Codes8{{c[i].z, c[i].w}} : Codes8{{c[i].x, c[i].y}}, f);
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        halves(fma(mul(fma(pair_of(f[j].x, f[j].y), unit, minus), scale), g[4 * h + j],
                                   b[4 * h + j]),
                               v[2 * j], v[2 * j + 1]);
                    uint32_t w[kPackWords<T>];
                    to_words<T>(v, w);
#pragma unroll
                    for (int j = 0; j < kPackWords<T>; ++j)
                        o[h * kPackWords<T> + j] = w[j];
                }
                if constexpr (WHOLE) { // (8 elements, or 16)
                    if (r < a.rows)
#pragma unroll
                        for (int j = 0; j < kPackWords<T, E>; j += 4)
                            if (j * 4 < there * (int)sizeof(T))
                                *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(to) + j) =
                                    make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                } else {
                    Carry<T, E> carry;
                    store_words<T, false, E>(to, there, next, r < a.rows, min(a.lanes, 32), o, carry);
                }
            }
        }
    }
}

template <typename T, typename W, bool WHOLE> cudaError_t restore_launch(const Restore &a, cudaStream_t st)
{
    const int rows = kRestoreThreads / a.lanes * kRestoreRows<WHOLE>; // of a block at a time
    const long long cols = std::min((a.dim + kRestoreCols - 1) / kRestoreCols, 65535LL);
    // (one wave: a block's weights are read once)
    const long long blocks = std::max(1LL, num_sms() * (long long)kRestoreBlocks<WHOLE> / cols);
    const dim3 grid((unsigned)std::min((a.rows + rows - 1) / rows, blocks), (unsigned)cols);
    return launch_chained(restore_kernel<T, W, WHOLE>, grid, kRestoreThreads, st, a);
}

template <typename T, typename W> rra_status restore(Restore a, cudaStream_t st)
{
    a.lanes = 1;
    while (a.lanes < kRestoreThreads && a.lanes * kRestorePack < a.dim)
        a.lanes *= 2;
    return launched(whole_packs<T>(a.dim, {a.y, a.gamma, a.beta}) ? restore_launch<T, W, true>(a, st)
                                                                  : restore_launch<T, W, false>(a, st));
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
    long long stretch; // long rows: rows of a partial row
    Group g;
};

// A row's packs in the registers and shared memory of a group of lanes, as in
// norm_grad_kernel: a lane keeps its columns' sums of dgamma and dbeta over all rows
// of its group in registers, the packs of the next row are on their way to shared
// memory while a row is worked on, each lane's to slots of its own, and every block
// leaves one partial row of the sums, which join_kernel adds.  A pack of dy that does
// not begin on a 16-byte boundary comes with the chunks that it touches.
constexpr int kGradHeld = 4; // packs of a lane
constexpr int kGradThreads = 384, kGradWide = 512;
constexpr int kGradSums = 2 * 2 * 32; // floats of a group for its rows' sums
constexpr int kMostBarriers = 15;     // of groups: a block has 16, __syncthreads takes one
constexpr int kGradStages = 2;

// 16-byte chunks that a pack's slot has.
template <typename T, bool WHOLE>
constexpr int kChunks = (int)sizeof(T) / 2 + (WHOLE ? 0 : 1);

__device__ __forceinline__ void stage16(void *to, const void *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                 : "memory");
}

template <typename T, typename W, bool MULTI, int THREADS, bool WHOLE>
__global__ void __launch_bounds__(THREADS, 1) saved_grad_kernel(const SavedGrad a)
{
    constexpr int K = kGradHeld, C = kChunks<T, WHOLE>, N = kPackWords<T>;
    // gamma as fp32, the groups' sums, the stages; after the last row: the
    // holders' [2][width]
    extern __shared__ __align__(16) float smem[];
    const T *const dy = static_cast<const T *>(a.dy), *const dy_end = dy + a.rows * a.dim;
    T *const dx = static_cast<T *>(a.dx);
    const W *const gamma = static_cast<const W *>(a.gamma);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, group = threadIdx.x / lanes,
              groups = blockDim.x / lanes;
    const int dim = (int)a.dim, nb = (int)blocks_of(dim), packs = (dim + kPack - 1) / kPack,
              width = packs * kPack;
    const long long step = (long long)gridDim.x * groups;
    const float n = (float)dim, inverse = 1.0f / n;
    float *const weights = smem, *const sums = weights + width;
    GroupOf mine = group_of(a.g, sums + group * kGradSums, 1 + group);
    unsigned char *const stages =
        reinterpret_cast<unsigned char *>(sums + (MULTI ? groups * kGradSums : 0));
    // a stage: chunk c of every thread's k-th pack, then every thread's k-th codes
    constexpr int kRow = THREADS * 16, kCodes = K * C * kRow, kStage = kCodes + K * THREADS * 8;
    unsigned char *const slots = stages + threadIdx.x * 16;
    unsigned char *const codes = stages + kCodes + threadIdx.x * 8;
    const int gap = (MULTI ? 32 : lanes) * kPack; // elements between a lane's packs
    const int u0 = pack_of<K, MULTI>(li, 0, lanes);
    int there[K], next[K]; // elements of the lane's packs, and of the ones behind them
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = u0 * kPack + k * gap;
        there[k] = max(0, min(kPack, dim - c));
        next[k] = max(0, min(kPack, dim - c - kPack));
    }
    dependents_wait();

    const auto stage_row = [&](int stage, long long r) {
        unsigned char *const to = slots + stage * kStage;
        const bool on = r < a.rows;
        const bool inside = WHOLE || row_inside(dy + r * dim, dim, dy, dy_end);
        const T *const row = dy + r * dim + u0 * kPack;
        const int8_t *const row_codes = a.codes + r * nb * kBlock + u0 * kPack;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int in = there[k];
            if (!on || in == 0)
                continue;
            const T *const p = row + k * gap;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                             smem_u32(codes + stage * kStage + k * THREADS * 8)),
                         "l"(row_codes + k * gap)
                         : "memory");
            if (WHOLE) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    stage16(to + (k * C + c) * kRow, reinterpret_cast<const uint4 *>(p) + c);
                continue;
            }
            const int m = (int)(reinterpret_cast<uintptr_t>(p) & 15);
            const uint4 *const from =
                reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - m);
            if (inside || (reinterpret_cast<const T *>(from) >= dy &&
                           reinterpret_cast<const T *>(from + C) <= dy_end)) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    stage16(to + (k * C + c) * kRow, from + c);
            } else { // an end of the array: what is there, zeros behind it
                for (int j = 0; j < kPack; ++j) {
                    const int at = m + j * (int)sizeof(T);
                    *reinterpret_cast<T *>(to + (k * C + at / 16) * kRow + at % 16) =
                        j < in ? p[j] : from_f32<T>(0.0f);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Pair dg[K][4], db[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dg[k][j] = db[k][j] = pair_of(0.0f, 0.0f);
    long long r = (long long)blockIdx.x * groups + group;
    int stage = 0;
    stage_row(0, r);
    float next_mu = 0.0f, next_rs = 0.0f;
    int8_t next_e[K] = {};
    const auto next_row = [&](long long q) {
        if (q >= a.rows)
            return;
        next_mu = a.mean[q];
        next_rs = a.rstd[q];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (there[k] > 0)
                next_e[k] = a.exps[q * nb + (u0 * kPack + k * gap) / kBlock];
    };
    next_row(r);
    for (int i = threadIdx.x; i < width; i += blockDim.x)
        weights[i] = i >= dim ? 0.0f : gamma ? to_f32(gamma[i]) : 1.0f;
    if (MULTI)
        for (int i = threadIdx.x; i < groups * kGradSums; i += blockDim.x)
            sums[i] = 0.0f;
    __syncthreads();
    // a group of several warps has barriers of its own: it ends with its last
    // row; the groups of a warp go on together
    const long long end = MULTI ? a.rows : a.rows + (group - (group & -(32 / lanes)));
    for (; r < end; r += step) {
        const bool on = MULTI || r < a.rows;
        stage_row(stage ^ 1, r + step);
        const int now = stage;
        stage ^= 1;
        const float rs = next_rs;
        const Pair minus = pair_of(-next_mu, -next_mu), scale = pair_of(rs, rs);
        float s_e[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            s_e[k] = block_scale(next_e[k]);
        next_row(r + step);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        // dy and xh of the k-th pack, out of its slot
        const auto take = [&](int k, bool shifted, Pair (&d)[4], Pair (&xh)[4]) {
            unsigned char *const at = slots + now * kStage;
            uint32_t w[N];
            if (WHOLE || shifted) {
#pragma unroll
                for (int c = 0; c < N / 4; ++c) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(at + (k * C + c) * kRow);
                    w[4 * c] = q.x, w[4 * c + 1] = q.y, w[4 * c + 2] = q.z, w[4 * c + 3] = q.w;
                }
            } else {
                uint32_t in[N + 4];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(at + (k * C + c) * kRow);
                    in[4 * c] = q.x, in[4 * c + 1] = q.y, in[4 * c + 2] = q.z, in[4 * c + 3] = q.w;
                }
                shift_bytes(in, (int)(reinterpret_cast<uintptr_t>(dy + r * dim) & 15), w);
                if (there[k] < kPack)
                    keep_first<T>(w, there[k]);
                if (dx) // (for the second time)
#pragma unroll
                    for (int c = 0; c < N / 4; ++c)
                        *reinterpret_cast<uint4 *>(at + (k * C + c) * kRow) =
                            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            }
            const Codes8 q = load_codes(
                reinterpret_cast<const int8_t *>(codes + now * kStage + k * THREADS * 8));
            float2 f[4];
            fractions8(q, f);
            const Pair s = pair_of(s_e[k], s_e[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j] = pair_in<T>(w, j);
                xh[j] = mul(fma(pair_of(f[j].x, f[j].y), s, minus), scale);
            }
        };
        const auto weight = [&](int k, Pair (&g)[4]) {
            const float4 *const p =
                reinterpret_cast<const float4 *>(weights + u0 * kPack + k * gap);
            const float4 lo = p[0], hi = p[1];
            g[0] = pair_of(lo.x, lo.y), g[1] = pair_of(lo.z, lo.w);
            g[2] = pair_of(hi.x, hi.y), g[3] = pair_of(hi.z, hi.w);
        };
        Pair s0 = pair_of(0.0f, 0.0f), s1 = s0;
        if (on) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (there[k] == 0)
                    continue;
                Pair d[4], xh[4], g[4];
                take(k, false, d, xh);
                weight(k, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Pair w = mul(d[j], g[j]);
                    s0 = add(s0, w);
                    s1 = fma(w, xh[j], s1);
                    dg[k][j] = fma(d[j], xh[j], dg[k][j]);
                    db[k][j] = add(db[k][j], d[j]);
                }
            }
        }
        if (!dx)
            continue;
        Sums<2> s{{sum_of(s0), sum_of(s1)}};
        s = group_sum<MULTI, 2>(s, mine);
        // dx = rs w - rs mean(w) - xh rs mean(w xh)
        const float t0 = -rs * quotient(s.v[0], n, inverse), t1 = -rs * quotient(s.v[1], n, inverse);
        const Pair m0 = pair_of(t0, t0), m1 = pair_of(t1, t1);
        Carry<T> carry;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint32_t o[N] = {};
            if (on && there[k] > 0) {
                Pair d[4], xh[4], g[4];
                float v[8];
                take(k, true, d, xh);
                weight(k, g);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    halves(fma(xh[j], m1, fma(mul(d[j], g[j]), scale, m0)), v[2 * j], v[2 * j + 1]);
                to_words<T>(v, o);
            }
            store_words<T, WHOLE>(dx + r * dim + u0 * kPack + k * gap, there[k], next[k], on,
                                  min(lanes, 32), o, carry, k > 0, k == K - 1);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    dependents_launch();
    if (!a.dgamma && !a.dbeta)
        return;

    float *const out = a.part + 2LL * blockIdx.x * a.dim;
    float fg[K][8], fb[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            halves(dg[k][j], fg[k][2 * j], fg[k][2 * j + 1]);
            halves(db[k][j], fb[k][2 * j], fb[k][2 * j + 1]);
        }
    if constexpr (!MULTI) { // the warp's groups first
        for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    fg[k][j] += __shfl_xor_sync(kFull, fg[k][j], o);
                    fb[k][j] += __shfl_xor_sync(kFull, fb[k][j], o);
                }
    }
    const int holders = MULTI ? groups : blockDim.x / 32, me = MULTI ? group : threadIdx.x / 32;
    const bool holds = MULTI || threadIdx.x % 32 < lanes;
    __syncthreads(); // (gamma and the stages are done with)
    float *const own = smem + me * 2 * width;
    if (holds)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (there[k] > 0) {
                store_values<float, 8>(own + u0 * kPack + k * gap, fg[k]);
                store_values<float, 8>(own + width + u0 * kPack + k * gap, fb[k]);
            }
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += blockDim.x) {
        float g = 0.0f, b = 0.0f;
        for (int h = 0; h < holders; ++h) {
            g += smem[h * 2 * width + c];
            b += smem[(h * 2 + 1) * width + c];
        }
        out[c] = g;
        out[dim + c] = b;
    }
}

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

// Rows that no block holds: dx by two passes over a row, the second from L2 (with the
// weights' sums, 1024 x 65536 bf16: 237 us).
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
cudaError_t saved_grad_long(const SavedGrad &a, cudaStream_t st)
{
    if (a.dgamma || a.dbeta) {
        const unsigned cols = (unsigned)std::min((a.dim / kPack + kThreads) / kThreads, 1LL << 16);
        saved_weights_kernel<T, VEC><<<dim3(cols, a.parts), kThreads, 0, st>>>(a);
    }
    if (a.dx) // last: dx may be dy
        saved_dx_kernel<T, W, VEC><<<grid_of(a.rows, 8), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

// Launch shape of the gradient, from which its scratch follows.
struct GradShape {
    Group g;
    int groups;  // of a block
    int parts;   // partial rows
    int threads; // kGradThreads, kGradWide, or 0: rows that no block holds
    bool whole;
};

template <typename T> GradShape grad_shape(const SavedGrad &a)
{
    GradShape s;
    s.whole = whole_packs<T>(a.dim, {a.dy, a.dx, a.gamma});
    const long long packs = (a.dim + kPack - 1) / kPack;
    s.threads = packs <= kGradThreads * kGradHeld ? kGradThreads
                // (fp32 rows off 16-byte boundaries: 512 threads' slots are too many)
                : packs <= kGradWide * kGradHeld && (s.whole || sizeof(T) == 2) ? kGradWide
                                                                                : 0;
    if (!s.threads) {
        const long long stretch = std::max(16LL, (a.rows + 127) / 128);
        s.groups = 1;
        s.parts = (int)((a.rows + stretch - 1) / stretch);
        return s;
    }
    s.g = group_for(packs, kGradHeld);
    // one block per SM; groups of a block only where rows are many
    const long long most = std::min(std::max(1, s.threads / s.g.lanes()),
                                    s.g.warps > 1 ? kMostBarriers : s.threads);
    s.groups = (int)std::max(1LL, std::min(most, a.rows / num_sms()));
    if (s.g.warps == 1) { // whole warps
        const int in_warp = 32 / s.g.lanes();
        s.groups = std::max(1, s.groups / in_warp) * in_warp;
    }
    s.parts = (int)std::min((a.rows + s.groups - 1) / s.groups, (long long)num_sms());
    return s;
}

template <typename T, typename W, bool MULTI, int THREADS, bool WHOLE>
cudaError_t saved_grad_held(const SavedGrad &a, const GradShape &s, cudaStream_t st)
{
    // the slots of a whole block, whatever its size: their distance is a constant
    const size_t stages =
                     (size_t)kGradStages * kGradHeld * (kChunks<T, WHOLE> * 16 + 8) * THREADS,
                 sums = MULTI ? sizeof(float) * kGradSums * s.groups : 0,
                 weights = sizeof(float) * ((a.dim + kPack - 1) / kPack * kPack);
    // at the end: the sums of every holder (a group, or a warp of groups)
    const int holders = MULTI ? s.groups : s.groups * s.g.lanes() / 32;
    const int smem = (int)std::max(weights + sums + stages, 2 * weights * holders);
    const auto fn = saved_grad_kernel<T, W, MULTI, THREADS, WHOLE>;
    const cudaError_t e = op_allow(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess)
        return e;
    return launch_chained_smem(fn, dim3(s.parts), s.groups * s.g.lanes(), smem, st, a);
}

template <typename T, typename W, bool WHOLE>
cudaError_t saved_grad_rows(const SavedGrad &a, const GradShape &s, cudaStream_t st)
{
    if (s.threads == kGradThreads)
        return s.g.warps > 1 ? saved_grad_held<T, W, true, kGradThreads, WHOLE>(a, s, st)
                             : saved_grad_held<T, W, false, kGradThreads, WHOLE>(a, s, st);
    if constexpr (WHOLE || sizeof(T) == 2)
        if (s.threads == kGradWide)
            return saved_grad_held<T, W, true, kGradWide, WHOLE>(a, s, st);
    return saved_grad_long<T, W, WHOLE>(a, st);
}

template <typename T, typename W> rra_status saved_grad(SavedGrad a, cudaStream_t st)
{
    const GradShape s = grad_shape<T>(a);
    a.g = s.g;
    a.parts = s.parts;
    a.stretch = std::max(16LL, (a.rows + 127) / 128);
    std::unique_lock<std::mutex> lk;
    if (a.dgamma || a.dbeta) {
        unsigned char *ws = nullptr;
        const rra_status r =
            op_scratch(st, kScratchHead + sizeof(float) * 2 * a.parts * a.dim, lk, &ws);
        if (r != RRA_OK)
            return r;
        a.part = reinterpret_cast<float *>(ws + kScratchHead);
    }
    cudaError_t e = cudaSuccess;
    if (a.rows > 0)
        e = s.whole ? saved_grad_rows<T, W, true>(a, s, st) : saved_grad_rows<T, W, false>(a, s, st);
    if (e == cudaSuccess && (a.dgamma || a.dbeta))
        e = join_parts<W>(Join{a.part, a.parts, a.dim, a.dgamma, a.dbeta, a.accumulate},
                          a.rows > 0 && s.threads, st);
    return launched(e);
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
                      dx, dgamma, dbeta, accumulate, nullptr, 0,    0,  {}};
    return by_types<SavedGradCall>(dtype, weight_t, a, reinterpret_cast<cudaStream_t>(stream));
}
