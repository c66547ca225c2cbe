// gated_gemm.cu -- the products of the gated feed-forward block on the tensor cores.
//
// A pair of blocks makes 256 x 256 results at a time: each block has 128 of the rows
// and half of the other operand's 256 columns in its shared memory, and one
// instruction of the pair multiplies all of it.  Slices of 64 along k come by tensor
// maps, six in flight (5 take the same time); the sums of two results lie in tensor
// memory, so that one is written out while the next is summed.
//
// Bound by the tensor cores, and those by the GPU's power: at 8192 x 4096 x 16384 bf16 the
// SM clock falls from 2.0 to 1.55 GHz and the products run at 1.69-1.76 PFLOP/s (forward,
// nothing kept: 1250-1270 us; gate and up kept whole 1285-1330, in 8 bits 1300-1310), 1.66
// and 1.6 for dx and the weights' gradients (1317 and 1367 us each); the library's plain
// products of these sizes run at 1.79-1.84.
#include "gated_ff.h"

#include "gated_act.cuh"
#include "op_common.cuh"
#include "ragged.cuh"
#include "saved.cuh"
#include "stream_slot.h"
#include "tc.cuh"

namespace rra {
namespace {

constexpr int kSide = 256;      // rows and columns of a pair's results
constexpr int kHalf = 128;      // rows of a block, columns it has in shared memory
constexpr int kSlice = 64;      // elements of k: 128 bytes
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalf * kSlice * 2, kStageBytes = 2 * kOperandBytes;
constexpr int kBoxBytes = kSlice * kSlice * 2; // 64 rows for 64 elements of k
constexpr int kWriters = 8;                    // warps that write results
constexpr int kGemmThreads = 64 + 32 * kWriters; // copies, instructions, and those
// Tiles along m that share their columns' slices in L2 (8192 x 4096 x 16384 bf16: forward
// 1257 us with 16, 1271 with 8; dx 1317 with 8, 1368 with 16, 1381 with 4).
template <int MODE> constexpr int kGroup = MODE == 0 ? 16 : 8;

// fp32 operands come as three planes of bf16, each the next 8 bits of a number, which
// add up to it exactly.  Of the nine products of planes the six largest count (what is
// left out is below 2^-21 of a product, 2^-24 in the mean), the small ones first.  Sums
// in tensor memory are cut off at each step of 16 along k, not rounded: half a unit
// of the last place a step, always towards zero (measured: 4.8e-7 of the result after
// 512 elements of k, 4.4e-6 after 4096).  For fp32 results they are therefore taken out
// after kRun slices and added up there.
constexpr int kRun = 4;
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
    CUtensorMap a[2], b[2];
    int tiles_m, tiles_n, tiles; // tiles: of all outputs
    int slices;                  // of one pair of operands
    int splits, per_split;       // parts of the slices, each an item of work; slices of one
    long long m, n;              // of an output
    int act;
    void *out[2]; // h; dx; dw_gate, dw_up
    Kept gate, up;
    int accumulate;
    int first_out;      // kDw: the output of the first tiles
    float *parts; // more than one split: sums, [tile][split][256 rows][256 columns]
    unsigned *stalled;
};

struct TilePlace {
    int which;
    long long m0, n0;
};

// Tiles in groups along m, n by n, so that those at work at one time share
// slices in L2.
template <int MODE> __device__ __forceinline__ TilePlace tile_place(const Gemm &g, int t)
{
    TilePlace p;
    const int per = g.tiles_m * g.tiles_n;
    p.which = MODE == kDw ? t / per + g.first_out : 0;
    t %= per;
    constexpr int G = kGroup<MODE>;
    const int group = t / (G * g.tiles_n), left = t - group * G * g.tiles_n;
    const int height = min(G, g.tiles_m - group * G);
    p.m0 = (long long)(group * G + left % height) * kSide;
    p.n0 = (long long)(left / height) * (MODE == kForward ? kHalf : kSide);
    return p;
}

// An item of work: a tile and a stretch of its slices.
struct Item {
    int tile, split, lo, hi;
};

template <int MODE> __device__ __forceinline__ Item item_of(const Gemm &g, int i)
{
    const int all = MODE == kDx ? 2 * g.slices : g.slices;
    Item t;
    t.split = i / g.tiles;
    t.tile = i - t.split * g.tiles;
    t.lo = t.split * g.per_split;
    t.hi = min(t.lo + g.per_split, all);
    return t;
}

// Slices whose sums stay in tensor memory.
template <bool F32> __device__ __forceinline__ int run_of(const Item &t) { return F32 ? kRun : t.hi - t.lo; }

// 16 columns from `col` on of a warp's 32 rows (from r0 on; a lane has a row) to an
// output of m x n.  whole: every 16 columns are on a 32-byte boundary.  A lane then
// writes its own 32 or 64 bytes (whole sectors, of which 16 bytes would write halves);
// else they go through shared memory, so that a store has two rows' neighbouring
// elements and not 32 rows' (which takes a cycle a row: 333 x 513 x 1001 fp16, dx: 50 us).
constexpr int kStageRow = 17; // floats: rows begin in different banks
template <typename O>
__device__ __forceinline__ void put_columns(float *stage, O *out, long long m, long long n,
                                            long long r0, long long col, bool whole,
                                            bool accumulate, float (&v)[16])
{
    const int lane = threadIdx.x % 32;
    if (whole && col + 16 <= n) {
        O *const p = out + (r0 + lane) * n + col;
        if (r0 + lane >= m)
            return;
        if (accumulate) {
            float old[16];
            load8<O, true>(p, 8, *reinterpret_cast<float(*)[8]>(&old[0]));
            load8<O, true>(p + 8, 8, *reinterpret_cast<float(*)[8]>(&old[8]));
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] += old[j];
        }
        uint32_t w[kPackWords<O> * 2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t half[kPackWords<O>];
            to_words<O>(v + 8 * i, half);
#pragma unroll
            for (int j = 0; j < kPackWords<O>; ++j)
                w[i * kPackWords<O> + j] = half[j];
        }
#pragma unroll
        for (int i = 0; i < kPackWords<O> * 2; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             reinterpret_cast<uint32_t *>(p) + i),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                         "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                         : "memory");
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
        stage[lane * kStageRow + j] = v[j];
    __syncwarp();
    const long long c = col + lane % 16;
    O *p = out + (r0 + lane / 16) * n + c;
#pragma unroll 8
    for (int i = lane / 16; i < 32; i += 2, p += 2 * n)
        if (r0 + i < m && c < n) {
            const float f = stage[i * kStageRow + lane % 16];
            *p = from_f32<O>(accumulate ? to_f32(*p) + f : f);
        }
    __syncwarp();
}

template <int N>
__device__ __forceinline__ void floats(const uint32_t (&r)[N], int i, float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j)
        v[j] = __uint_as_float(r[i + j]);
}

// ---------------------------------------------------------------- writers

// Writer w has the lanes (rows) 32 (w % 4) .. of tensor memory and one half of the
// columns (in kForward, of gate's and of up's).  kForward's halves of a row meet in
// shared memory where a block of 128 codes needs its largest magnitude.

struct Shared {
    uint64_t full[kStages], empty[kStages], summed[2], written[2];
    uint32_t tmem, stop;
    uint32_t top[2][2][kHalf]; // gate, up; half; row
    float stage[kWriters][32 * kStageRow];
};

// Largest magnitude's bits of 64 columns of this lane's row.
__device__ __forceinline__ uint32_t row_top(uint32_t at)
{
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
        uint32_t r[32];
        tmem_load(at + c, r);
        tmem_loaded();
#pragma unroll
        for (int j = 0; j < 32; ++j)
            top = max(top, r[j] & 0x7fffffffu);
    }
    return top;
}

// One of gate and up, 16 columns from col on.
template <typename T>
__device__ __forceinline__ void keep_columns(const Kept &to, float *stage, uint32_t top,
                                             const Gemm &g, long long r0, long long col, bool whole,
                                             float (&v)[16])
{
    const long long r = r0 + threadIdx.x % 32;
    if (to.exps) {
        if (r >= g.m)
            return;
        const Codes8 a = encode8(v, top), b = encode8(v + 8, top);
        *reinterpret_cast<uint4 *>(static_cast<int8_t *>(to.data) + r * blocks_of(g.n) * kBlock +
                                   col) = make_uint4(a.w[0], a.w[1], b.w[0], b.w[1]);
    } else if (to.data) {
        put_columns(stage, static_cast<T *>(to.data), g.m, g.n, r0, col, whole, false, v);
    }
}

// Gate and up of a warp's rows from r0 on, 64 columns from n0 + 64 half on, to where
// they go.
template <typename T, int ACT>
__device__ __forceinline__ void write_forward(const Gemm &g, Shared &s, float *stage, int half,
                                              int quarter, uint32_t at, long long r0, long long n0,
                                              bool whole)
{
    uint32_t top[2] = {0, 0}; // bits of the blocks' largest magnitudes
    if (g.gate.exps || g.up.exps) {
        const int row = quarter * 32 + threadIdx.x % 32;
        const long long r = r0 + threadIdx.x % 32;
        s.top[0][half][row] = row_top(at + half * 64);
        s.top[1][half][row] = row_top(at + kHalf + half * 64);
        named_barrier(2 + quarter, 64);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = max(s.top[i][0][row], s.top[i][1][row]);
            int8_t *const exps = i == 0 ? g.gate.exps : g.up.exps;
            if (r < g.m && half == 0 && exps)
                exps[r * blocks_of(g.n) + n0 / kBlock] = exponent_byte(block_exponent(top[i]));
        }
        named_barrier(2 + quarter, 64); // (read before the next ones are written)
    }
#pragma unroll 1
    for (int c = half * 64; c < half * 64 + 64; c += 16) {
        uint32_t rg[16], ru[16];
        tmem_load(at + c, rg);
        tmem_load(at + kHalf + c, ru);
        tmem_loaded();
        float vg[16], vu[16];
        floats(rg, 0, vg);
        floats(ru, 0, vu);
        keep_columns<T>(g.gate, stage, top[0], g, r0, n0 + c, whole, vg);
        keep_columns<T>(g.up, stage, top[1], g, r0, n0 + c, whole, vu);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            vg[j] = act_value<ACT, sizeof(T) == 4>(vg[j]) * vu[j];
        put_columns(stage, static_cast<T *>(g.out[0]), g.m, g.n, r0, n0 + c, whole, false, vg);
    }
}

template <typename O>
__device__ __forceinline__ void write_plain(const Gemm &g, float *stage, O *out, int half,
                                            uint32_t at, long long r0, long long n0, bool whole)
{
#pragma unroll 1
    for (int c = half * kHalf; c < half * kHalf + kHalf && n0 + c < g.n; c += 32) {
        uint32_t v[32];
        tmem_load(at + c, v);
        tmem_loaded();
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            float f[16];
            floats(v, i, f);
            put_columns(stage, out, g.m, g.n, r0, n0 + c + i, whole, g.accumulate != 0, f);
        }
    }
}

// to (+)= the sums at `from`, a warp's 128 columns from `first` on.
__device__ __forceinline__ void take_sums(uint32_t from, uint32_t to, int first, bool add)
{
#pragma unroll 1
    for (int c = first; c < first + kHalf; c += 32) {
        uint32_t v[32];
        tmem_load(from + c, v);
        if (add) {
            uint32_t w[32];
            tmem_load(to + c, w);
            tmem_loaded();
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
        } else {
            tmem_loaded();
        }
        tmem_store(to + c, v);
    }
    tmem_stored();
}

// A warp's sums of an item (128 columns from `first` on; `there`: the lane's row is one of
// the output's) to memory, for finish_kernel.
__device__ __forceinline__ void write_part(const Gemm &g, const Item &t, uint32_t at, int row,
                                           int first, bool there)
{
    float *const to = g.parts + (((long long)t.tile * g.splits + t.split) * kSide + row) * kSide;
#pragma unroll 1
    for (int c = first; c < first + kHalf; c += 32) {
        uint32_t v[32];
        tmem_load(at + c, v);
        tmem_loaded();
#pragma unroll
        for (int j = 0; there && j < 32; j += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + c + j),
                         "r"(v[j]), "r"(v[j + 1]), "r"(v[j + 2]), "r"(v[j + 3]), "r"(v[j + 4]),
                         "r"(v[j + 5]), "r"(v[j + 6]), "r"(v[j + 7])
                         : "memory");
    }
}

// ---------------------------------------------------------------- the kernel

// T: the type of the call's elements; O: of the outputs.
template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ Gemm g)
{
    constexpr bool F32 = sizeof(T) == 4;
    constexpr bool A_ROWS = MODE == kDw, B_ROWS = MODE != kForward;
    constexpr uint32_t kKind =
        mma_kind(!std::is_same<T, __half>::value, A_ROWS, B_ROWS, kSide, kSide);
    extern __shared__ unsigned char raw[];
    // swizzled boxes begin on 1024-byte boundaries
    unsigned char *const stages = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    Shared &s = *reinterpret_cast<Shared *>(stages + kStages * kStageBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2, items = g.tiles * g.splits;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.summed[i], 1);
            mbar_init(&s.written[i], 2 * kWriters); // of both blocks
        }
        s.stop = 0;
        mbar_fence_init();
        prefetch_map(&g.a[0]);
        prefetch_map(&g.b[0]);
    }
    __syncwarp();
    if (warp == 1)
        tmem_alloc(&s.tmem);
    tc_fence_before();
    cluster_barrier();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile uint32_t *const stop = &s.stop;
    dependents_wait();
    dependents_launch();

    if (warp == 0) {
        if (lane == 0) {
            uint32_t step = 0;
            bool ok = true;
            // one slice of one product of planes
            const auto load = [&](const TilePlace &p, int k, int pa, int pb) {
                const int m = (int)p.m0 + (int)rank * kHalf, n = (int)p.n0 + (int)rank * kHalf;
                const int i = step % kStages;
                // the first round finds the stages empty
                if (!wait_limited(&s.empty[i], (step / kStages & 1) ^ 1, stop, g.stalled))
                    return false;
                if (rank == 0)
                    mbar_arrive_expect_tx(&s.full[i], 2 * kStageBytes);
                const uint32_t bar = cluster_address(&s.full[i], 0);
                unsigned char *const a = stages + i * kStageBytes, *const b = a + kOperandBytes;
                if (MODE == kForward) {
                    load_box(a, &g.a[0], k * kSlice, m, pa, bar);
                    load_box(b, &g.b[rank], k * kSlice, (int)p.n0, pb, bar);
                } else {
                    const int from = MODE == kDx && k >= g.slices ? 1 : 0;
                    const int at = (k - from * g.slices) * kSlice;
                    if (MODE == kDx) {
                        load_box(a, &g.a[from], at, m, pa, bar);
                    } else {
                        load_box(a, &g.a[p.which], m, at, pa, bar);
                        load_box(a + kBoxBytes, &g.a[p.which], m + kSlice, at, pa, bar);
                    }
                    load_box(b, &g.b[from], n, at, pb, bar);
                    load_box(b + kBoxBytes, &g.b[from], n + kSlice, at, pb, bar);
                }
                ++step;
                return true;
            };
            for (int t = pair; ok && t < items; t += pairs) {
                const Item it = item_of<MODE>(g, t);
                const TilePlace p = tile_place<MODE>(g, it.tile);
                const int run = run_of<F32>(it);
                for (int lo = it.lo; ok && lo < it.hi; lo += run)
                    for (int q = 0; ok && q < kProducts<F32>; ++q)
                        for (int k = lo; ok && k < min(lo + run, it.hi); ++k)
                            ok = load(p, k, F32 ? plane_a(q) : 0, F32 ? plane_b(q) : 0);
            }
            // the other block's arrivals on this one's barriers come before it ends
            for (int i = 0; ok && i < kStages; ++i, ++step)
                ok = wait_limited(&s.empty[step % kStages], (step / kStages & 1) ^ 1, stop,
                                  g.stalled);
            if (!ok) { // what is on its way lands before the block ends
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 20000000)
                    __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t step = 0, made = 0;
            bool ok = true;
            for (int t = pair; ok && t < items; t += pairs) {
                const Item it = item_of<MODE>(g, t);
                const int run = run_of<F32>(it);
                for (int lo = it.lo; ok && lo < it.hi; lo += run, ++made) {
                    // fp32: the second half of tensor memory holds the sums of runs
                    const uint32_t into = F32 ? 0 : made % 2, round = F32 ? made : made / 2;
                    const uint32_t at = tmem + into * kSide;
                    if (!(ok = wait_limited(&s.written[into], (round & 1) ^ 1, stop, g.stalled)))
                        break;
                    tc_fence_after();
                    const int count = kProducts<F32> * (min(lo + run, it.hi) - lo);
                    for (int k = 0; k < count; ++k, ++step) {
                        const int i = step % kStages;
                        if (!(ok = wait_limited(&s.full[i], step / kStages & 1, stop, g.stalled)))
                            break;
                        tc_fence_after();
                        const unsigned char *const pa = stages + i * kStageBytes,
                                            *const pb = pa + kOperandBytes;
                        const uint64_t a =
                            A_ROWS ? operand_along_rows(pa, kBoxBytes) : operand_along_k(pa);
                        const uint64_t b =
                            B_ROWS ? operand_along_rows(pb, kBoxBytes) : operand_along_k(pb);
#pragma unroll
                        for (int j = 0; j < kSlice / 16; ++j)
                            mma_pair(at, a + j * (A_ROWS ? kStepAlongRows : kStepAlongK),
                                     b + j * (B_ROWS ? kStepAlongRows : kStepAlongK), kKind,
                                     k > 0 || j > 0);
                        mma_commit_pair(&s.empty[i]);
                    }
                    if (ok)
                        mma_commit_pair(&s.summed[into]);
                }
            }
        }
    } else {
        const int quarter = warp % 4, half = (warp - 2) / 4;
        const uint32_t lanes = (uint32_t)quarter * 32 << 16;
        uint32_t made = 0;
        bool ok = true;
        const auto wait_sums = [&](uint32_t into, uint32_t round) {
            // (all writers go on or none: they meet at barriers)
            const bool yes = named_all(1, 32 * kWriters,
                                       wait_limited(&s.summed[into], round & 1, stop, g.stalled));
            __syncwarp();
            tc_fence_after();
            return yes;
        };
        const auto release = [&](uint32_t into) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_at(cluster_address(&s.written[into], 0));
        };
        for (int t = pair; ok && t < items; t += pairs) {
            const Item it = item_of<MODE>(g, t);
            const int run = run_of<F32>(it);
            uint32_t into = 0;
            for (int lo = it.lo; ok && lo < it.hi; lo += run, ++made) {
                into = F32 ? 0 : made % 2;
                ok = wait_sums(into, F32 ? made : made / 2);
                if (F32 && ok) {
                    take_sums(tmem + lanes, tmem + lanes + kSide, half * kHalf, lo > it.lo);
                    release(0);
                }
            }
            if (!ok)
                break;
            const uint32_t at = tmem + lanes + (F32 ? kSide : into * kSide);
            const TilePlace p = tile_place<MODE>(g, it.tile);
            const int row = quarter * 32 + lane;
            const long long r0 = p.m0 + rank * kHalf + quarter * 32;
            float *const stage = s.stage[warp - 2];
            if (g.splits > 1) {
                write_part(g, it, at, rank * kHalf + row, half * kHalf, r0 + lane < g.m);
            } else {
                O *const out = static_cast<O *>(g.out[p.which]);
                const bool whole = pack_fits(out, (size_t)g.n * sizeof(O), 32);
                if (MODE == kForward) {
                    if (F32) { // a half has columns whose sums the other has stored
                        tc_fence_before();
                        named_barrier(2 + quarter, 64);
                        tc_fence_after();
                    }
                    by_act(g.act, [&](auto act) {
                        write_forward<T, decltype(act)::value>(
                            g, s, stage, half, quarter, at, r0, p.n0,
                            whole && (g.gate.exps || aligned_to(g.gate.data, 32)) &&
                                (g.up.exps || aligned_to(g.up.data, 32)));
                    });
                } else {
                    write_plain<O>(g, stage, out, half, at, r0, p.n0, whole);
                }
            }
            if (!F32)
                release(into);
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_barrier();
    tc_fence_after();
    if (warp == 1)
        tmem_free(tmem);
}

constexpr int kGemmSmem = kStages * kStageBytes + 1024 + (int)sizeof(Shared);

// ---------------------------------------------------------------- splits

// The sums of a tile's splits added, in their order, and on to where they go: a warp has
// a row of a tile, a lane 4 of its first 128 columns and the same 4 of its last.  (A
// launch of its own, with all of the GPU: the last of a tile's splits to end took 10 us
// for it.)
constexpr int kFinishThreads = 256;

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

template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const __grid_constant__ Gemm g)
{
    constexpr int kWarps = kFinishThreads / 32, kAhead = 4; // splits on their way
    const int c = threadIdx.x % 32 * 4;
    dependents_wait();
    dependents_launch();
    for (long long i = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
         i < (long long)g.tiles * kSide; i += (long long)gridDim.x * kWarps) {
        const int tile = (int)(i / kSide), row = (int)(i % kSide);
        const TilePlace p = tile_place<MODE>(g, tile);
        const long long r = p.m0 + row;
        if (r >= g.m)
            continue;
        const float *const from = g.parts + ((long long)tile * g.splits * kSide + row) * kSide + c;
        float v[2][4] = {};
        for (int k0 = 0; k0 < g.splits; k0 += kAhead) {
            float4 q[kAhead][2];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q[k][h] = k0 + k < g.splits
                                  ? __ldcs(reinterpret_cast<const float4 *>(
                                        from + (long long)(k0 + k) * kSide * kSide + h * kHalf))
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[h][0] += q[k][h].x, v[h][1] += q[k][h].y;
                    v[h][2] += q[k][h].z, v[h][3] += q[k][h].w;
                }
        }
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
                h[j] = act_of<sizeof(T) == 4>(g.act, v[0][j]) * v[1][j];
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
}

// ---------------------------------------------------------------- host

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Boxes of 64 x box_rows elements of the planes of a matrix of 16-bit numbers; what is
// outside of a plane is read as zero.
bool make_map(CUtensorMap *m, bool bf16, const Matrix16 &x, int box_rows)
{
    const EncodeFn fn = encoder();
    if (!fn)
        return false;
    const long long plane = x.planes > 1 ? x.rows * x.ld : x.ld;
    const cuuint64_t dims[3] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows, (cuuint64_t)x.planes},
                     strides[2] = {(cuuint64_t)x.ld * 2, (cuuint64_t)plane * 2};
    const cuuint32_t box[3] = {kSlice, (cuuint32_t)box_rows, 1}, steps[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(x.p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of blocks that the device runs at a time (the kernels' launches are alike).
int resident_pairs()
{
    static std::mutex mu;
    static int cached[64] = {};
    const void *const fn = reinterpret_cast<const void *>(gemm_kernel<__half, __half, kForward>);
    const int most = std::max(1, num_sms() / 2);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64)
        return most;
    std::lock_guard<std::mutex> lk(mu);
    if (!cached[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * most);
        cfg.blockDim = dim3(kGemmThreads);
        cfg.dynamicSmemBytes = kGemmSmem;
        cudaLaunchAttribute at[1] = {};
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (op_allow(fn, kGemmSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = most;
        }
        cached[dev] = std::min(n, most);
    }
    return cached[dev];
}

template <typename T, typename O, int MODE> cudaError_t launch_gemm(Gemm &g, cudaStream_t st)
{
    const auto fn = gemm_kernel<T, O, MODE>;
    cudaError_t e = op_allow(reinterpret_cast<const void *>(fn), kGemmSmem);
    if (e != cudaSuccess)
        return e;
    if ((e = stalled_word(&g.stalled)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * std::min(resident_pairs(), g.tiles * g.splits));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kGemmSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, fn, g)) != cudaSuccess || g.splits == 1)
        return e;
    const long long rows = (long long)g.tiles * kSide, warps = kFinishThreads / 32;
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

// Few tiles with many slices are split along k.  The time of a launch in steps, as
// measured: a slice takes 0.28 us a pair, an item 3 us to write out, adding up the splits
// 4 us and 0.2 more for each.
Plan plan_of(long long m, long long n, int outputs, long long step_n, long long total, bool f32)
{
    Plan p = {};
    const long long tm = (m + kSide - 1) / kSide, tn = (n + step_n - 1) / step_n;
    if (tm * tn * outputs > 0x3fffffff || total > 0x3fffffff)
        return p;
    p.ok = true;
    p.tiles_m = (int)tm;
    p.tiles_n = (int)tn;
    p.tiles = (int)(tm * tn) * outputs;
    const int pairs = resident_pairs();
    const double slice = 0.28 * (f32 ? kProducts<true> : 1);
    double best = 0;
    for (int s = 1; s <= 64 && (s == 1 || p.tiles * s <= 2 * pairs); ++s) {
        const int per = (int)((total + s - 1) / s);
        // (a split has some slices, and none is empty)
        if (s > 1 && (per * (f32 ? kProducts<true> : 1) < 4 || (long long)per * (s - 1) >= total))
            continue;
        const double t = (double)((p.tiles * s + pairs - 1) / pairs) * (per * slice + 3) +
                         (s > 1 ? 4 + 0.2 * s : 0);
        if (s == 1 || t < best) {
            best = t;
            p.splits = s;
            p.per_split = per;
        }
    }
    if (p.splits > 1)
        p.bytes = (size_t)p.tiles * p.splits * kSide * kSide * sizeof(float);
    return p;
}

long long slices_of(long long k) { return (k + kSlice - 1) / kSlice; }

Plan plan_forward(const FfArgs &a, bool f32)
{
    return plan_of(a.rows, a.ff, 1, kHalf, slices_of(a.dim), f32);
}
Plan plan_dx(const FfGradArgs &a, bool f32)
{
    return plan_of(a.rows, a.dim, 1, kSide, 2 * slices_of(a.ff), f32);
}
Plan plan_dw(const FfGradArgs &a, bool f32)
{
    return plan_of(a.ff, a.dim, a.dwg && a.dwu ? 2 : 1, kSide, slices_of(a.rows), f32);
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

// Set by a kernel whose wait has run out of time, in host memory: one word for the
// process, read (and cleared) by the next call.
cudaError_t stalled_word(unsigned **word)
{
    static std::mutex mu;
    static unsigned *p = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!p) {
        const AllocationAllowed allowed;
        void *q = nullptr;
        const cudaError_t e = cudaHostAlloc(&q, 64, cudaHostAllocPortable | cudaHostAllocMapped);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
        p = static_cast<unsigned *>(q);
        *p = 0;
    }
    *word = p;
    return cudaSuccess;
}

bool gemm_takes(const Matrix16 &x)
{
    return aligned_to(x.p, 16) && x.ld % 8 == 0 && x.ld <= (1LL << 38);
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
    constexpr bool bf16 = !std::is_same<T, __half>::value;
    Gemm g = {};
    g.m = a.rows;
    g.n = a.ff;
    g.act = a.act;
    g.out[0] = a.h;
    g.gate = a.gate;
    g.up = a.up;
    if (!use_plan(g, plan_forward(a, sizeof(T) == 4), slices_of(a.dim), scratch, parts_at) ||
        !make_map(&g.a[0], bf16, in[0], kHalf) || !make_map(&g.b[0], bf16, in[1], kHalf) ||
        !make_map(&g.b[1], bf16, in[2], kHalf))
        return cudaErrorInvalidValue;
    return launch_gemm<T, T, kForward>(g, st);
}

template <typename T>
cudaError_t gemm_dx(const FfGradArgs &a, const Matrix16 (&in)[5], unsigned char *scratch,
                    size_t parts_at, cudaStream_t st)
{
    constexpr bool bf16 = !std::is_same<T, __half>::value;
    Gemm g = {};
    g.m = a.rows;
    g.n = a.dim;
    g.out[0] = a.dx;
    if (!use_plan(g, plan_dx(a, sizeof(T) == 4), slices_of(a.ff), scratch, parts_at) ||
        !make_map(&g.a[0], bf16, in[0], kHalf) || !make_map(&g.a[1], bf16, in[1], kHalf) ||
        !make_map(&g.b[0], bf16, in[2], kSlice) || !make_map(&g.b[1], bf16, in[3], kSlice))
        return cudaErrorInvalidValue;
    return launch_gemm<T, T, kDx>(g, st);
}

template <typename T, typename O>
cudaError_t gemm_dw(const FfGradArgs &a, const Matrix16 (&in)[5], unsigned char *scratch,
                    size_t parts_at, cudaStream_t st)
{
    constexpr bool bf16 = !std::is_same<T, __half>::value;
    Gemm g = {};
    g.m = a.ff;
    g.n = a.dim;
    g.out[0] = a.dwg;
    g.out[1] = a.dwu;
    g.accumulate = a.accumulate;
    g.first_out = a.dwg ? 0 : 1;
    if (!use_plan(g, plan_dw(a, sizeof(T) == 4), slices_of(a.rows), scratch, parts_at) ||
        !make_map(&g.a[0], bf16, in[0], kSlice) || !make_map(&g.a[1], bf16, in[1], kSlice) ||
        !make_map(&g.b[0], bf16, in[4], kSlice))
        return cudaErrorInvalidValue;
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
