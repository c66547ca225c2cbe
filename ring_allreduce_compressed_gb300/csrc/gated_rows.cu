// gated_rows.cu -- the gated feed-forward block of few rows (a step of decoding).
//
//   g = x Wg^T,  u = x Wu^T,  h = a(g) u
//
// Bound by the weights, which are read once: every warp reads 16 rows of them (8 of
// gate, the same 8 of up) straight into registers, 16 bytes a lane, and multiplies
// them with all rows of x, which stay in L1.  4096 x 16384 bf16: 41 us with one row
// (6.5 TB/s), 49 with 16; fp32 82 us with one (6.5 TB/s), 130 with 8.  The large kernel's
// tiles have 128 rows (fp32: 64), which few rows leave empty.
//
// 16 bits: one warp-wide product takes 16 weight rows x 16 elements of k x 8 rows of x.
// Its k may be any 16 as long as both sides agree: a lane's 8 neighbouring elements
// count as those that it holds in two products, so nothing is rearranged.  (The
// large kernel's instruction; with one row its pipe is busy 9 % of the time.)  fp32: paired fp32 operations, the same layout.
#include "gated_ff.h"

#include "gated_act.cuh"
#include "op_common.cuh"
#include "ragged.cuh"
#include "saved.cuh"

namespace rra {
namespace {

constexpr int kWarps = 8, kRowThreads = 32 * kWarps;
constexpr int kUnit = 8;   // columns of h that a block makes at a time
constexpr int kStep = 32;  // elements of k that a warp reads of each row at a time
// steps in flight: 128 bytes a lane
template <typename T> constexpr int kSteps = 8 / (int)sizeof(T);
// blocks an SM
template <typename T, int ROWS> constexpr int kBlocks = ROWS <= 8 && sizeof(T) == 2 ? 3 : 2;

// acc (8 gate and 8 up rows x 8 rows of x) += weights times x, 32 elements of k.
template <typename T>
__device__ __forceinline__ void products(float (&acc)[4], const uint32_t (&wg)[4],
                                         const uint32_t (&wu)[4], const uint32_t (&x)[4])
{
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                         "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                         : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                         : "r"(wg[2 * j]), "r"(wu[2 * j]), "r"(wg[2 * j + 1]), "r"(wu[2 * j + 1]),
                           "r"(x[2 * j]), "r"(x[2 * j + 1]));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                         "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                         : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                         : "r"(wg[2 * j]), "r"(wu[2 * j]), "r"(wg[2 * j + 1]), "r"(wu[2 * j + 1]),
                           "r"(x[2 * j]), "r"(x[2 * j + 1]));
}

// ROWS: rows of x that there is room for (16-bit: a multiple of 8).  TILES: eights of
// columns that a warp makes at a time; two for many rows of x, whose reads from L1 are
// then half as many for a weight.  WHOLE: every 8 elements are on a 16-byte boundary.
template <typename T, int ROWS, int TILES, bool WHOLE>
__global__ void __launch_bounds__(kRowThreads, kBlocks<T, ROWS>)
    rows_kernel(const FfArgs a, long long units, float *wide)
{
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int WORDS = kPackWords<T>, STEPS = kSteps<T> / TILES, N = F32 ? 1 : ROWS / 8;
    constexpr int ACC = F32 ? 2 * ROWS : 4;
    // a warp's sums: [row of x][gate, up][column]
    __shared__ float sums[kWarps][ROWS * 2 * kUnit];
    const int warp = threadIdx.x / 32, g = threadIdx.x % 32 / 4, t = threadIdx.x % 4;
    const T *const x = static_cast<const T *>(a.x), *const x_end = x + a.rows * a.dim;
    const T *const wg = static_cast<const T *>(a.wg), *const wg_end = wg + a.ff * a.dim;
    const T *const wu = static_cast<const T *>(a.wu), *const wu_end = wu + a.ff * a.dim;
    dependents_wait();
    dependents_launch();
    for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const long long row = unit * (kUnit * TILES) + g;
        float acc[TILES][N][ACC];
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int c = 0; c < ACC; ++c)
                    acc[i][n][c] = 0.0f;
        for (long long k0 = (long long)warp * STEPS * kStep; k0 < a.dim;
             k0 += kWarps * STEPS * kStep) {
            uint32_t vg[TILES][STEPS][WORDS], vu[TILES][STEPS][WORDS];
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const long long k = k0 + s * kStep + t * 8;
                    const bool there = row + i * kUnit < a.ff;
                    const int in = there ? (int)max(0LL, min(8LL, a.dim - k)) : 0;
                    const long long at = there ? (row + i * kUnit) * a.dim + k : 0;
                    load_words<T, WHOLE>(wg + at, in, wg, wg_end, vg[i][s]);
                    load_words<T, WHOLE>(wu + at, in, wu, wu_end, vu[i][s]);
                }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const long long k = k0 + s * kStep + t * 8;
                const int in = (int)max(0LL, min(8LL, a.dim - k));
                // (the rows' addresses are made here, one after the other, and not kept in
                // registers all the time)
                long long dim = a.dim;
                asm volatile("" : "+l"(dim));
                const T *p = x + k + (F32 ? 0 : g * dim);
                if constexpr (F32) { // all rows of x; this lane's part of k
#pragma unroll
                    for (int m = 0; m < ROWS; ++m, p += dim) {
                        uint32_t w[WORDS];
                        load_words<T, WHOLE>(p, m < a.rows ? in : 0, x, x_end, w);
                        Pair sg = pair_of(acc[0][0][2 * m], 0.0f),
                             su = pair_of(acc[0][0][2 * m + 1], 0.0f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const Pair xv = pair_of(__uint_as_float(w[2 * j]),
                                                    __uint_as_float(w[2 * j + 1]));
                            sg = fma(xv, pair_of(__uint_as_float(vg[0][s][2 * j]),
                                                 __uint_as_float(vg[0][s][2 * j + 1])), sg);
                            su = fma(xv, pair_of(__uint_as_float(vu[0][s][2 * j]),
                                                 __uint_as_float(vu[0][s][2 * j + 1])), su);
                        }
                        acc[0][0][2 * m] = sum_of(sg);
                        acc[0][0][2 * m + 1] = sum_of(su);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < N; ++n, p += 8 * dim) {
                        uint32_t w[WORDS];
                        load_words<T, WHOLE>(p, n * 8 + g < a.rows ? in : 0, x, x_end, w);
#pragma unroll
                        for (int i = 0; i < TILES; ++i)
                            products<T>(acc[i][n], vg[i][s], vu[i][s], w);
                    }
                }
            }
        }
        float *const mine = sums[warp];
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            __syncthreads(); // (the last sums are read)
            if constexpr (F32) {
#pragma unroll
                for (int m = 0; m < ROWS; ++m)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = acc[i][0][2 * m + c];
                        v += __shfl_xor_sync(kFull, v, 1);
                        v += __shfl_xor_sync(kFull, v, 2);
                        if (t == m % 4)
                            mine[(m * 2 + c) * kUnit + g] = v;
                    }
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) // rows of x 2t, 2t + 1; gate, up
                        mine[((n * 8 + 2 * t + c % 2) * 2 + c / 2) * kUnit + g] = acc[i][n][c];
            }
            __syncthreads();
            for (int q = threadIdx.x; q < ROWS * kUnit; q += kRowThreads) {
                const long long r = q / kUnit, c = (unit * TILES + i) * kUnit + q % kUnit;
                if (r >= a.rows || c >= a.ff)
                    continue;
                float vg = 0.0f, vu = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    vg += sums[w][(q / kUnit * 2) * kUnit + q % kUnit];
                    vu += sums[w][(q / kUnit * 2 + 1) * kUnit + q % kUnit];
                }
                const long long at = r * a.ff + c;
                static_cast<T *>(a.h)[at] = from_f32<T>(act_of<F32>(a.act, vg) * vu);
                if (a.gate.exps)
                    wide[at] = vg;
                else if (a.gate.data)
                    static_cast<T *>(a.gate.data)[at] = from_f32<T>(vg);
                if (a.up.exps)
                    wide[a.rows * a.ff + at] = vu;
                else if (a.up.data)
                    static_cast<T *>(a.up.data)[at] = from_f32<T>(vu);
            }
        }
    }
}

// Gate (blockIdx.y 0) and up (1) into 8 bits: a warp takes two blocks of codes at a time.
__global__ void __launch_bounds__(kRowThreads) codes_kernel(const FfArgs a, const float *wide)
{
    const Kept &to = blockIdx.y == 0 ? a.gate : a.up;
    dependents_wait();
    dependents_launch();
    if (!to.exps)
        return;
    const float *const v0 = wide + (blockIdx.y == 0 ? 0 : a.rows * a.ff), *const end = v0 + a.rows * a.ff;
    const long long nb = blocks_of(a.ff), packs = a.rows * nb * kBlockPacks;
    for (long long i0 = ((long long)blockIdx.x * kWarps + threadIdx.x / 32) * 32; i0 < packs;
         i0 += (long long)gridDim.x * kRowThreads) {
        const long long i = i0 + threadIdx.x % 32, b = i / kBlockPacks, r = b / nb;
        const long long c = (b - r * nb) * kBlock + i % kBlockPacks * kPack;
        const bool there = i < packs;
        uint32_t w[8];
        load_words<float, false>(v0 + (there ? r * a.ff + c : 0),
                                 there ? (int)max(0LL, min(8LL, a.ff - c)) : 0, v0, end, w);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = __uint_as_float(w[j]);
        const uint32_t top = half_warp_max(top_bits(v));
        if (!there)
            continue;
        store_codes(static_cast<int8_t *>(to.data) + i * kPack, encode8(v, top));
        if (i % kBlockPacks == 0)
            to.exps[b] = exponent_byte(block_exponent(top));
    }
}

template <typename T, int ROWS, int TILES = 1>
cudaError_t rows_call(const FfArgs &a, float *wide, cudaStream_t st)
{
    const long long units = (a.ff + kUnit * TILES - 1) / (kUnit * TILES);
    const dim3 grid((unsigned)std::min(units, (long long)num_sms() * kBlocks<T, ROWS>));
    bool whole = a.dim % 8 == 0;
    for (const void *p : {a.x, a.wg, a.wu})
        whole = whole && aligned_to(p, 16);
    const cudaError_t e =
        whole ? launch_chained(rows_kernel<T, ROWS, TILES, true>, grid, kRowThreads, st, a, units, wide)
              : launch_chained(rows_kernel<T, ROWS, TILES, false>, grid, kRowThreads, st, a, units, wide);
    if (e != cudaSuccess || !wide)
        return e;
    const long long packs = a.rows * blocks_of(a.ff) * kBlockPacks;
    return launch_chained(codes_kernel,
                          dim3((unsigned)std::min((packs + kRowThreads - 1) / kRowThreads,
                                                  num_sms() * 4LL),
                               2),
                          kRowThreads, st, a, (const float *)wide);
}

} // namespace

// The large kernel takes over where this one is hardly faster, or already 4 % slower
// (2048 x 8192 fp16: 20 us here with 17 rows, 28 with 48, 36 with 64, 35-37 there with 17
// to 64; 4096 x 16384 bf16: 64, 85, 120 here, 115 there; 512 x 1024: 7 here with 64, 12
// there with 65).  fp32 has no variant for more than 16 rows (4096 x 16384: 380 us
// with 16, 694 there with 17).
template <typename T> bool few_rows(const FfArgs &a) { return a.rows <= (sizeof(T) == 2 ? 64 : 16); }

template <typename T> rra_status rows_forward(const FfArgs &a, cudaStream_t st)
{
    // gate and up whole, where they are kept in 8 bits: blocks of codes are wider than
    // the columns that one of the kernel's blocks makes
    std::unique_lock<std::mutex> lk;
    float *wide = nullptr;
    if (a.gate.exps || a.up.exps) {
        unsigned char *ws = nullptr;
        const rra_status r =
            op_scratch(st, kScratchHead + 2 * (size_t)a.rows * a.ff * sizeof(float), lk, &ws);
        if (r != RRA_OK)
            return r;
        wide = reinterpret_cast<float *>(ws + kScratchHead);
    }
    if constexpr (sizeof(T) == 4)
        return launched(a.rows <= 1   ? rows_call<T, 1>(a, wide, st)
                        : a.rows <= 2 ? rows_call<T, 2>(a, wide, st)
                        : a.rows <= 4 ? rows_call<T, 4>(a, wide, st)
                        : a.rows <= 8 ? rows_call<T, 8>(a, wide, st)
                                      : rows_call<T, 16>(a, wide, st));
    else
        return launched(a.rows <= 8    ? rows_call<T, 8>(a, wide, st)
                        : a.rows <= 16 ? rows_call<T, 16>(a, wide, st)
                        : a.rows <= 32 ? rows_call<T, 32, 2>(a, wide, st)
                        : a.rows <= 48 ? rows_call<T, 48, 2>(a, wide, st)
                                       : rows_call<T, 64, 2>(a, wide, st));
}

#define RRA_ROWS(T)                                                                              \
    template bool few_rows<T>(const FfArgs &);                                                   \
    template rra_status rows_forward<T>(const FfArgs &, cudaStream_t);
RRA_ROWS(float)
RRA_ROWS(__half)
RRA_ROWS(__nv_bfloat16)
#undef RRA_ROWS

} // namespace rra
