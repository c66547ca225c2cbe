// gated_gemm.cu -- the products of the gated feed-forward block on the tensor cores.
//
// A block makes 128 x 256 results (fp32: 64 x 256) of a stretch of k, in registers: eight
// warps, each 64 (32) rows and 64 columns.  Slices of 64 along k are copied to shared memory
// ahead of their use, four of them in a ring.  All waits are for the block's own
// copies and barriers: none depends on another block or launch.
//
// Bound by the tensor cores' older instructions and the waits between them: their pipe is
// at work 58 % of the time, with eight warps an SM (their sums fill the registers).  At 8192
// x 4096 x 16384 bf16 a forward call takes 6.2 ms, 355 TFLOP/s; from 8 bits, the
// gradient 12.7 ms.
#include "gated_ff.h"

#include "gated_act.cuh"
#include "op_common.cuh"
#include "ragged.cuh"
#include "saved.cuh"

namespace rra {
namespace {

constexpr int kWide = 256, kHalf = 128; // columns of a block's results; half of them
constexpr int kSlice = 64;              // elements of k
constexpr int kStages = 4;
constexpr int kGemmThreads = 256, kGemmWarps = kGemmThreads / 32;
template <bool F32> constexpr int kTall = F32 ? 64 : 128; // rows of a block's results
template <bool F32> constexpr int kStageBytes = (kTall<F32> + kWide) * kSlice * 2;
// Tiles along m that share their columns' slices in L2.
constexpr int kGroup = 16;

// fp32 operands come as three planes of bf16, each the next 8 bits of a number, which
// add up to it exactly.  Of the nine products of planes the six largest count (what is
// left out is below 2^-21 of a product, 2^-24 in the mean), the small ones first.  The
// instructions cut sums off and do not round them (every addend 25 bits below the largest,
// the sum to 24: sums of 16,384 products of one sign are off by 2^-13 in fp16, fp32's by
// 2^-20); for fp32 results those of a slice are therefore added up outside of them.
template <bool F32> constexpr int kProducts = F32 ? 6 : 1;
__device__ __forceinline__ int plane_a(int q) { return q == 0 ? 2 : q == 2 || q == 3 ? 1 : 0; }
__device__ __forceinline__ int plane_b(int q) { return q == 1 ? 2 : q == 2 || q == 4 ? 1 : 0; }

// What the products are:
//  kForward: columns 0..127 are gate, 128..255 up, of the same 128 of ff.
//            a = x, b[0] = w_gate, b[1] = w_up, k = dim, all next to each other along k.
//  kDx:      a[i] (dgate, dup) along k = ff, b[i] (w_gate, w_up) along the columns, both
//            pairs one after the other.
//  kDw:      a[i] (dgate, dup) along the rows ff, b = x along the columns, k = rows; the two
//            outputs are tiles one after the other.
enum Mode { kForward, kDx, kDw };

struct Gemm {
    Matrix16 a[2], b[2];
    int tiles_m, tiles_n, tiles; // tiles: of all outputs
    int slices;                  // of one pair of operands
    int splits, per_split;       // parts of the slices, each an item of work; slices of one
    long long m, n;              // of an output
    int act;
    void *out[2]; // h; dx; dw_gate, dw_up
    Kept gate, up;
    int accumulate;
    int first_out; // kDw: the output of the first tiles
    float *parts;  // more than one split: sums, [tile][split][rows of a tile][256 columns]
};

struct TilePlace {
    int which;
    long long m0, n0;
};

// Tiles in groups along m, n by n, so that those at work at one time share
// slices in L2.
template <int MODE, int TALL> __device__ __forceinline__ TilePlace tile_place(const Gemm &g, int t)
{
    TilePlace p;
    const int per = g.tiles_m * g.tiles_n;
    p.which = MODE == kDw ? t / per + g.first_out : 0;
    t %= per;
    const long long wide = (long long)kGroup * g.tiles_n;
    const int group = (int)(t / wide), left = (int)(t - group * wide);
    const int height = min(kGroup, g.tiles_m - group * kGroup);
    p.m0 = (long long)(group * kGroup + left % height) * TALL;
    p.n0 = (long long)(left / height) * (MODE == kForward ? kHalf : kWide);
    return p;
}

// ---------------------------------------------------------------- operands

// 16 bytes of a matrix's plane from (row, col) on to shared memory, col a multiple of 8;
// what is outside of the plane is zero and not read.
__device__ __forceinline__ void copy16(uint32_t to, const Matrix16 &x, int plane, long long row,
                                       long long col)
{
    const long long left = row < x.rows ? min(8LL, x.cols - col) : 0;
    const uint32_t bytes = left > 0 ? (uint32_t)left * 2 : 0;
    const uint16_t *const p = static_cast<const uint16_t *>(x.p);
    const uint16_t *const from = bytes ? p + (plane * x.rows + row) * x.ld + col : p;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_here()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// An operand's slice lies in shared memory as lines of 16-byte chunks: along k a line is
// 64 elements of k of a row, along the rows it is SIZE rows of one k.  A chunk's
// number is turned by its line's, so that eight lines' chunks are in different banks.
template <bool ROWS, int SIZE> __device__ __forceinline__ uint32_t chunk_at(int line, int chunk)
{
    return (uint32_t)(line * (ROWS ? SIZE * 2 : kSlice * 2) + ((chunk ^ (line & 7)) << 4));
}

// COUNT rows (from r0 on; all SIZE of them are the operand's, these from `first` on) of
// a slice from k0 on.
template <bool ROWS, int SIZE, int COUNT>
__device__ __forceinline__ void copy_operand(uint32_t to, const Matrix16 &x, int plane, long long r0,
                                             int first, long long k0)
{
    static_assert(COUNT * 8 % kGemmThreads == 0, "all threads copy as much");
#pragma unroll
    for (int j = 0; j < COUNT * 8 / kGemmThreads; ++j) {
        const int i = j * kGemmThreads + threadIdx.x;
        if (ROWS) {
            const int k = i / (COUNT / 8), c = i % (COUNT / 8);
            copy16(to + chunk_at<true, SIZE>(k, first / 8 + c), x, plane, k0 + k, r0 + c * 8);
        } else {
            const int r = i / 8, c = i % 8;
            copy16(to + chunk_at<false, SIZE>(first + r, c), x, plane, r0 + r, k0 + c * 8);
        }
    }
}

// Four 8 x 8 matrices, a lane giving the address of a line of one.
template <bool TURN> __device__ __forceinline__ void read4(uint32_t at, uint32_t (&r)[4])
{
    if (TURN)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
}

// 16 rows from m on and 16 elements of k of the first operand.
template <bool ROWS, int SIZE>
__device__ __forceinline__ void read_a(uint32_t at, int m, int k, uint32_t (&r)[4])
{
    const int l = threadIdx.x % 32, j = l / 8;
    if (ROWS)
        read4<true>(at + chunk_at<true, SIZE>(k + l % 8 + j / 2 * 8, m / 8 + j % 2), r);
    else
        read4<false>(at + chunk_at<false, SIZE>(m + l % 16, k / 8 + l / 16), r);
}
// 16 columns from n on of the second: r[0], r[1] the first 8, r[2], r[3] the others.
template <bool ROWS, int SIZE>
__device__ __forceinline__ void read_b(uint32_t at, int n, int k, uint32_t (&r)[4])
{
    const int l = threadIdx.x % 32, j = l / 8;
    if (ROWS)
        read4<true>(at + chunk_at<true, SIZE>(k + l % 8 + j % 2 * 8, n / 8 + j / 2), r);
    else
        read4<false>(at + chunk_at<false, SIZE>(n + l % 8 + j / 2 * 8, k / 8 + j % 2), r);
}

template <bool HALF>
__device__ __forceinline__ void multiply(float (&acc)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    if (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- results

template <typename O>
__device__ __forceinline__ void put4(O *p, long long there, bool whole, const float v[4])
{
    if (whole && there >= 4) {
        Pack<O, 4> q;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q.e[j] = from_f32<O>(v[j]);
        store_pack<O, 4>(p, q);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < there)
            p[j] = from_f32<O>(v[j]);
}

template <typename T>
__device__ __forceinline__ void keep4(const Kept &to, long long r, long long n0, long long n,
                                      bool whole, const float v[4])
{
    const int c = threadIdx.x % 32 * 4;
    if (to.exps) { // (all of the warp is here)
        float w[8] = {};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = v[j];
            top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        }
        top = __reduce_max_sync(kFull, top);
        const long long b = r * blocks_of(n) + n0 / kBlock;
        *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(to.data) + b * kBlock + c) =
            encode8(w, top).w[0];
        if (c == 0)
            to.exps[b] = exponent_byte(block_exponent(top));
    } else if (to.data) {
        put4(static_cast<T *>(to.data) + r * n + n0 + c, n - n0 - c, whole, v);
    }
}

// A row of a tile (r < m) to where it goes: a lane has 4 of its first 128 columns and the
// same 4 of its last.
template <typename T, typename O, int MODE, int ACT>
__device__ __forceinline__ void put_row(const Gemm &g, const TilePlace &p, long long r,
                                        float (&v)[2][4])
{
    const int c = threadIdx.x % 32 * 4;
    O *const out = static_cast<O *>(g.out[p.which]);
    const bool whole = pack_fits(out, (size_t)g.n * sizeof(O), 4 * sizeof(O));
    if constexpr (MODE == kForward) {
        const bool kept = whole && (g.gate.exps || aligned_to(g.gate.data, 4 * sizeof(T))) &&
                          (g.up.exps || aligned_to(g.up.data, 4 * sizeof(T)));
        keep4<T>(g.gate, r, p.n0, g.n, kept, v[0]);
        keep4<T>(g.up, r, p.n0, g.n, kept, v[1]);
        float h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = act_value<ACT, sizeof(T) == 4>(v[0][j]) * v[1][j];
        put4(out + r * g.n + p.n0 + c, g.n - p.n0 - c, whole, h);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long col = p.n0 + h * kHalf + c;
            O *const to = out + r * g.n + col;
            if (g.accumulate)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < g.n)
                        v[h][j] += to_f32(to[j]);
            put4(to, g.n - col, whole, v[h]);
        }
    }
}

// f(the activation) where there is one, once.
template <int MODE, typename F> __device__ __forceinline__ void by_mode(const Gemm &g, F f)
{
    if constexpr (MODE == kForward)
        by_act(g.act, f);
    else
        f(std::integral_constant<int, RRA_ACT_RELU>()); // (not used)
}

// ---------------------------------------------------------------- the kernel

constexpr int kRowFloats = kWide + 4; // of a block's results in shared memory

// T: the type of the call's elements; O: of the outputs.
template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ Gemm g)
{
    constexpr bool F32 = sizeof(T) == 4, HALF = std::is_same<T, __half>::value;
    constexpr bool A_ROWS = MODE == kDw, B_ROWS = MODE != kForward;
    constexpr int TALL = kTall<F32>, MT = TALL / 32, kAhead = kStages - 1;
    static_assert(TALL * kRowFloats * 4 <= kStages * kStageBytes<F32>, "results fit");
    extern __shared__ __align__(1024) unsigned char raw[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int wm = warp / 4 * (TALL / 2), wn = warp % 4 * 64; // the warp's results
    const int split = blockIdx.x / g.tiles, tile = blockIdx.x - split * g.tiles;
    const TilePlace p = tile_place<MODE, TALL>(g, tile);
    const int lo = split * g.per_split,
              hi = min(lo + g.per_split, MODE == kDx ? 2 * g.slices : g.slices);
    const int steps = (hi - lo) * kProducts<F32>;

    const auto copy = [&](int step) {
        if (step < steps) {
            const int q = step % kProducts<F32>, k = lo + step / kProducts<F32>;
            const int pa = F32 ? plane_a(q) : 0, pb = F32 ? plane_b(q) : 0;
            const uint32_t a = smem_u32(raw) + step % kStages * kStageBytes<F32>,
                           b = a + TALL * kSlice * 2;
            const int from = MODE == kDx && k >= g.slices ? 1 : 0;
            const long long k0 = (long long)(k - from * g.slices) * kSlice;
            copy_operand<A_ROWS, TALL, TALL>(a, g.a[MODE == kDw ? p.which : from], pa, p.m0, 0, k0);
            if (MODE == kForward) {
                copy_operand<false, kWide, kHalf>(b, g.b[0], pb, p.n0, 0, k0);
                copy_operand<false, kWide, kHalf>(b, g.b[1], pb, p.n0, kHalf, k0);
            } else {
                copy_operand<B_ROWS, kWide, kWide>(b, g.b[from], pb, p.n0, 0, k0);
            }
        }
        copies_sent(); // (an empty one keeps the count)
    };

    float acc[MT][8][4] = {}, sum[F32 ? MT : 1][8][4] = {};
    for (int step = 0; step < kAhead; ++step)
        copy(step);
    for (int step = 0; step < steps; ++step) {
        copies_here<kAhead - 1>();
        __syncthreads(); // all threads' copies of this slice; the last one's stage is free
        copy(step + kAhead);
        const uint32_t a = smem_u32(raw) + step % kStages * kStageBytes<F32>,
                       b = a + TALL * kSlice * 2;
#pragma unroll
        for (int k = 0; k < kSlice; k += 16) {
            uint32_t fa[MT][4], fb[4][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
                read_a<A_ROWS, TALL>(a, wm + 16 * i, k, fa[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                read_b<B_ROWS, kWide>(b, wn + 16 * j, k, fb[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    multiply<HALF>(acc[i][j], fa[i], fb[j / 2][j % 2 * 2], fb[j / 2][j % 2 * 2 + 1]);
        }
        if (F32 && step % kProducts<F32> == kProducts<F32> - 1)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[F32 ? i : 0][j][e] += acc[i][j][e];
                        acc[i][j][e] = 0.0f;
                    }
    }
    copies_here<0>();
    __syncthreads();

    // through shared memory, for rows as they are written
    float *const rows = reinterpret_cast<float *>(raw);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float *const v = F32 ? sum[F32 ? i : 0][j] : acc[i][j];
                *reinterpret_cast<float2 *>(rows + (wm + 16 * i + 8 * e + lane / 4) * kRowFloats +
                                            wn + 8 * j + lane % 4 * 2) =
                    make_float2(v[2 * e], v[2 * e + 1]);
            }
    __syncthreads();
    by_mode<MODE>(g, [&](auto act) {
        for (int row = warp; row < TALL && p.m0 + row < g.m; row += kGemmWarps) {
            float v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 q =
                    *reinterpret_cast<const float4 *>(rows + row * kRowFloats + h * kHalf + lane * 4);
                v[h][0] = q.x, v[h][1] = q.y, v[h][2] = q.z, v[h][3] = q.w;
                if (g.splits > 1) // for finish_kernel
                    *reinterpret_cast<float4 *>(
                        g.parts + (((long long)tile * g.splits + split) * TALL + row) * kWide +
                        h * kHalf + lane * 4) = q;
            }
            if (g.splits == 1)
                put_row<T, O, MODE, decltype(act)::value>(g, p, p.m0 + row, v);
        }
    });
}

// ---------------------------------------------------------------- splits

// The sums of a tile's splits added, in their order, and on to where they go: a warp has
// a row of a tile.  (A launch of its own, with all of the GPU.)
constexpr int kFinishThreads = 256;

template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const __grid_constant__ Gemm g)
{
    constexpr int kWarps = kFinishThreads / 32, kAhead = 4; // splits on their way
    constexpr int TALL = kTall<sizeof(T) == 4>;
    const int c = threadIdx.x % 32 * 4;
    dependents_wait();
    dependents_launch();
    by_mode<MODE>(g, [&](auto act) {
        for (long long i = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
             i < (long long)g.tiles * TALL; i += (long long)gridDim.x * kWarps) {
            const int tile = (int)(i / TALL), row = (int)(i % TALL);
            const TilePlace p = tile_place<MODE, TALL>(g, tile);
            if (p.m0 + row >= g.m)
                continue;
            const float *const from =
                g.parts + ((long long)tile * g.splits * TALL + row) * kWide + c;
            float v[2][4] = {};
            for (int k0 = 0; k0 < g.splits; k0 += kAhead) {
                float4 q[kAhead][2];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        q[k][h] = k0 + k < g.splits
                                      ? __ldcs(reinterpret_cast<const float4 *>(
                                            from + (long long)(k0 + k) * TALL * kWide + h * kHalf))
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        v[h][0] += q[k][h].x, v[h][1] += q[k][h].y;
                        v[h][2] += q[k][h].z, v[h][3] += q[k][h].w;
                    }
            }
            put_row<T, O, MODE, decltype(act)::value>(g, p, p.m0 + row, v);
        }
    });
}

// ---------------------------------------------------------------- host

// (Launched without an early start: it begins when what is ahead of it has ended.)
template <typename T, typename O, int MODE> cudaError_t launch_gemm(const Gemm &g, cudaStream_t st)
{
    const auto fn = gemm_kernel<T, O, MODE>;
    constexpr int smem = kStages * kStageBytes<sizeof(T) == 4>;
    cudaError_t e = op_allow(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess)
        return e;
    fn<<<(unsigned)(g.tiles * g.splits), kGemmThreads, smem, st>>>(g);
    if ((e = cudaGetLastError()) != cudaSuccess || g.splits == 1)
        return e;
    const long long rows = (long long)g.tiles * kTall<sizeof(T) == 4>, warps = kFinishThreads / 32;
    return launch_chained(finish_kernel<T, O, MODE>,
                          dim3((unsigned)std::min((rows + warps - 1) / warps, num_sms() * 8LL)),
                          kFinishThreads, st, g);
}

// Tiles, slices and splits of a product: m x n results (of each output), `total` slices
// for each of them, step_n columns of an output a tile.
struct Plan {
    bool ok; // (an int counts the tiles)
    int tiles_m, tiles_n, tiles, splits, per_split;
    size_t bytes; // of parts
};

// Few tiles with many slices are split along k.  The time of a launch in steps: a
// slice takes 1.8 us a block, as measured (8192 x 4096 x 16384 bf16: 6.2 ms for 54 tiles
// of 64 slices an SM; one of fp32 planes has half of the rows), an item 3 us to write out,
// adding up the splits 4 us and 0.2 more for each.
Plan plan_of(long long m, long long n, int outputs, long long step_n, long long total, bool f32)
{
    Plan p = {};
    const int tall = f32 ? kTall<true> : kTall<false>;
    const long long tm = (m + tall - 1) / tall, tn = (n + step_n - 1) / step_n;
    if (tm > 0x3fffffff || tn > 0x3fffffff || tm * tn * outputs > 0x3fffffff || total > 0x0fffffff)
        return p;
    p.ok = true;
    p.tiles_m = (int)tm;
    p.tiles_n = (int)tn;
    p.tiles = (int)(tm * tn) * outputs;
    const int sms = num_sms();
    const double slice = f32 ? 0.9 * kProducts<true> : 1.8;
    double best = 0;
    for (int s = 1; s <= 64 && (s == 1 || p.tiles * s <= 2 * sms); ++s) {
        const int per = (int)((total + s - 1) / s);
        // (a split has some slices, and none is empty)
        if (s > 1 && (per < 2 || (long long)per * (s - 1) >= total))
            continue;
        const double t = (double)((p.tiles * s + sms - 1) / sms) * (per * slice + 3) +
                         (s > 1 ? 4 + 0.2 * s : 0);
        if (s == 1 || t < best) {
            best = t;
            p.splits = s;
            p.per_split = per;
        }
    }
    if (p.splits > 1)
        p.bytes = (size_t)p.tiles * p.splits * tall * kWide * sizeof(float);
    return p;
}

long long slices_of(long long k) { return (k + kSlice - 1) / kSlice; }

Plan plan_forward(const FfArgs &a, bool f32)
{
    return plan_of(a.rows, a.ff, 1, kHalf, slices_of(a.dim), f32);
}
Plan plan_dx(const FfGradArgs &a, bool f32)
{
    return plan_of(a.rows, a.dim, 1, kWide, 2 * slices_of(a.ff), f32);
}
Plan plan_dw(const FfGradArgs &a, bool f32)
{
    return plan_of(a.ff, a.dim, a.dwg && a.dwu ? 2 : 1, kWide, slices_of(a.rows), f32);
}

// g's tiles by the plan; parts: where they are in the stream's scratch.
bool use_plan(Gemm &g, const Plan &p, long long slices, unsigned char *scratch, size_t parts_at)
{
    g.tiles_m = p.tiles_m;
    g.tiles_n = p.tiles_n;
    g.tiles = p.tiles;
    g.slices = (int)slices;
    g.splits = p.splits;
    g.per_split = p.per_split;
    if (p.splits > 1)
        g.parts = reinterpret_cast<float *>(scratch + parts_at);
    return p.ok;
}

} // namespace

bool gemm_takes(const Matrix16 &x)
{
    return aligned_to(x.p, 16) && x.ld % 8 == 0;
}

size_t gemm_parts(const FfArgs &a, bool f32) { return plan_forward(a, f32).bytes; }

size_t gemm_parts(const FfGradArgs &a, bool f32)
{
    return std::max(a.dx ? plan_dx(a, f32).bytes : 0,
                    a.dwg || a.dwu ? plan_dw(a, f32).bytes : 0);
}

template <typename T>
cudaError_t gemm_forward(const FfArgs &a, const Matrix16 (&in)[3], unsigned char *scratch,
                         size_t parts_at, cudaStream_t st)
{
    Gemm g = {};
    g.m = a.rows;
    g.n = a.ff;
    g.act = a.act;
    g.out[0] = a.h;
    g.gate = a.gate;
    g.up = a.up;
    if (!use_plan(g, plan_forward(a, sizeof(T) == 4), slices_of(a.dim), scratch, parts_at))
        return cudaErrorInvalidValue;
    g.a[0] = in[0];
    g.b[0] = in[1];
    g.b[1] = in[2];
    return launch_gemm<T, T, kForward>(g, st);
}

template <typename T>
cudaError_t gemm_dx(const FfGradArgs &a, const Matrix16 (&in)[5], unsigned char *scratch,
                    size_t parts_at, cudaStream_t st)
{
    Gemm g = {};
    g.m = a.rows;
    g.n = a.dim;
    g.out[0] = a.dx;
    if (!use_plan(g, plan_dx(a, sizeof(T) == 4), slices_of(a.ff), scratch, parts_at))
        return cudaErrorInvalidValue;
    g.a[0] = in[0];
    g.a[1] = in[1];
    g.b[0] = in[2];
    g.b[1] = in[3];
    return launch_gemm<T, T, kDx>(g, st);
}

template <typename T, typename O>
cudaError_t gemm_dw(const FfGradArgs &a, const Matrix16 (&in)[5], unsigned char *scratch,
                    size_t parts_at, cudaStream_t st)
{
    Gemm g = {};
    g.m = a.ff;
    g.n = a.dim;
    g.out[0] = a.dwg;
    g.out[1] = a.dwu;
    g.accumulate = a.accumulate;
    g.first_out = a.dwg ? 0 : 1;
    if (!use_plan(g, plan_dw(a, sizeof(T) == 4), slices_of(a.rows), scratch, parts_at))
        return cudaErrorInvalidValue;
    g.a[0] = in[0];
    g.a[1] = in[1];
    g.b[0] = in[4];
    return launch_gemm<T, O, kDw>(g, st);
}

#define RRA_GEMM(T)                                                                              \
    template cudaError_t gemm_forward<T>(const FfArgs &, const Matrix16 (&)[3], unsigned char *, \
                                         size_t, cudaStream_t);                                  \
    template cudaError_t gemm_dx<T>(const FfGradArgs &, const Matrix16 (&)[5], unsigned char *,  \
                                    size_t, cudaStream_t);                                       \
    template cudaError_t gemm_dw<T, float>(const FfGradArgs &, const Matrix16 (&)[5],            \
                                           unsigned char *, size_t, cudaStream_t);
RRA_GEMM(float)
RRA_GEMM(__half)
RRA_GEMM(__nv_bfloat16)
#undef RRA_GEMM
template cudaError_t gemm_dw<__half, __half>(const FfGradArgs &, const Matrix16 (&)[5],
                                             unsigned char *, size_t, cudaStream_t);
template cudaError_t gemm_dw<__nv_bfloat16, __nv_bfloat16>(const FfGradArgs &,
                                                           const Matrix16 (&)[5], unsigned char *,
                                                           size_t, cudaStream_t);

} // namespace rra
