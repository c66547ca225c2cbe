// gated_gemm.cu -- the products of the gated feed-forward block on the tensor cores
// (16-bit types).
//
// A pair of blocks makes 256 x 256 results at a time: each block has 128 of the rows
// and half of the other operand's 256 columns in its shared memory, and one
// instruction of the pair multiplies all of it.  Slices of 64 along k come by tensor
// maps, six in flight; the sums of two results lie in tensor memory, so that one is
// written out while the next is summed.
#include "gated_ff.h"

#include "gated_act.cuh"
#include "op_common.cuh"
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
constexpr int kGemmThreads = 192; // copies, instructions, four warps that write
constexpr int kGroup = 8;         // tiles along m that share their columns' slices in L2

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
    long long m, n;              // of an output
    int act;
    void *out[2]; // h; dx; dw_gate, dw_up
    Kept gate, up;
    int accumulate;
    int first_out; // kDw: the output of the first tiles
    unsigned *stalled;
};

struct TilePlace {
    int which;
    long long m0, n0;
};

// Tiles in groups of kGroup along m, n by n, so that those at work at one time share
// slices in L2.
template <int MODE> __device__ __forceinline__ TilePlace tile_place(const Gemm &g, int t)
{
    TilePlace p;
    const int per = g.tiles_m * g.tiles_n;
    p.which = MODE == kDw ? t / per + g.first_out : 0;
    t %= per;
    const int group = t / (kGroup * g.tiles_n), left = t - group * kGroup * g.tiles_n;
    const int height = min(kGroup, g.tiles_m - group * kGroup);
    p.m0 = (long long)(group * kGroup + left % height) * kSide;
    p.n0 = (long long)(left / height) * (MODE == kForward ? kHalf : kSide);
    return p;
}

// Eight values next to each other, of which `there` are in the row.
template <typename T>
__device__ __forceinline__ void put8(T *p, int there, bool whole, const float v[8])
{
    if (whole && there == 8)
        store8<T, true>(p, 8, v);
    else
        store8<T, false>(p, there, v);
}

__device__ __forceinline__ void floats(const uint32_t (&r)[32], int i, float v[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __uint_as_float(r[i + j]);
}

// Largest magnitude's bits of 128 columns of this lane's row.
__device__ __forceinline__ uint32_t row_top(uint32_t at)
{
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kHalf; c += 32) {
        uint32_t r[32];
        tmem_load(at + c, r);
        tmem_loaded();
#pragma unroll
        for (int j = 0; j < 32; ++j)
            top = max(top, r[j] & 0x7fffffffu);
    }
    return top;
}

// One of gate and up, 8 columns from c on of row r.
template <typename T>
__device__ __forceinline__ void keep8(const Kept &to, uint32_t top, long long r, long long c, long long ff,
                                      bool whole, const float v[8])
{
    if (to.exps) {
        const long long nb = blocks_of(ff);
        store_codes(static_cast<int8_t *>(to.data) + r * nb * kBlock + c, encode8(v, top));
    } else if (to.data) {
        put8(static_cast<T *>(to.data) + r * ff + c, (int)max(0LL, min(8LL, ff - c)), whole, v);
    }
}

// Rows of a pair's results from tensor memory to where they go: this lane's row r.
template <typename T>
__device__ __forceinline__ void write_forward(const Gemm &g, uint32_t at, long long r, long long n0,
                                              bool whole)
{
    uint32_t eg = 0, eu = 0; // bits of the blocks' largest magnitudes
    if (g.gate.exps)
        eg = row_top(at);
    if (g.up.exps)
        eu = row_top(at + kHalf);
    const bool on = r < g.m;
    const long long nb = blocks_of(g.n);
    if (on && g.gate.exps)
        g.gate.exps[r * nb + n0 / kBlock] = exponent_byte(block_exponent(eg));
    if (on && g.up.exps)
        g.up.exps[r * nb + n0 / kBlock] = exponent_byte(block_exponent(eu));
    for (int c = 0; c < kHalf; c += 32) {
        uint32_t rg[32], ru[32];
        tmem_load(at + c, rg);
        tmem_load(at + kHalf + c, ru);
        tmem_loaded();
        if (!on)
            continue;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            float vg[8], vu[8], h[8];
            floats(rg, i, vg);
            floats(ru, i, vu);
            const long long col = n0 + c + i;
            keep8<T>(g.gate, eg, r, col, g.n, whole, vg);
            keep8<T>(g.up, eu, r, col, g.n, whole, vu);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[j] = act_value<false>(g.act, vg[j]) * vu[j];
            put8(static_cast<T *>(g.out[0]) + r * g.n + col, (int)max(0LL, min(8LL, g.n - col)),
                 whole, h);
        }
    }
}

template <typename O>
__device__ __forceinline__ void write_plain(const Gemm &g, O *out, uint32_t at, long long r,
                                            long long n0, bool whole)
{
    const bool on = r < g.m;
    for (int c = 0; c < kSide; c += 32) {
        uint32_t v[32];
        tmem_load(at + c, v);
        tmem_loaded();
        if (!on)
            continue;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            const long long col = n0 + c + i;
            const int there = (int)max(0LL, min(8LL, g.n - col));
            float f[8];
            floats(v, i, f);
            O *const p = out + r * g.n + col;
            if (g.accumulate) {
                float old[8];
                if (whole && there == 8)
                    load8<O, true>(p, 8, old);
                else
                    load8<O, false>(p, there, old);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] += old[j];
            }
            put8(p, there, whole, f);
        }
    }
}

struct Shared {
    uint64_t full[kStages], empty[kStages], summed[2], written[2];
    uint32_t tmem, stop;
};

template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ Gemm g)
{
    constexpr bool A_ROWS = MODE == kDw, B_ROWS = MODE != kForward;
    constexpr uint32_t kKind =
        mma_kind(std::is_same<T, __nv_bfloat16>::value, A_ROWS, B_ROWS, kSide, kSide);
    extern __shared__ unsigned char raw[];
    // swizzled boxes begin on 1024-byte boundaries
    unsigned char *const stages = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    Shared &s = *reinterpret_cast<Shared *>(stages + kStages * kStageBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.summed[i], 1);
            mbar_init(&s.written[i], 8); // warps that write, of both blocks
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
    const int slices = MODE == kDx ? 2 * g.slices : g.slices;
    dependents_wait();
    dependents_launch();

    if (warp == 0) {
        if (lane == 0) {
            uint32_t step = 0;
            bool ok = true;
            for (int t = pair; ok && t < g.tiles; t += pairs) {
                const TilePlace p = tile_place<MODE>(g, t);
                const int m = (int)p.m0 + (int)rank * kHalf, n = (int)p.n0 + (int)rank * kHalf;
                for (int k = 0; k < slices; ++k, ++step) {
                    const int i = step % kStages;
                    // the first round finds the stages empty
                    if (!(ok = wait_limited(&s.empty[i], (step / kStages & 1) ^ 1, stop, g.stalled)))
                        break;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&s.full[i], 2 * kStageBytes);
                    const uint32_t bar = cluster_address(&s.full[i], 0);
                    unsigned char *const a = stages + i * kStageBytes, *const b = a + kOperandBytes;
                    if (MODE == kForward) {
                        load_box(a, &g.a[0], k * kSlice, m, bar);
                        load_box(b, &g.b[rank], k * kSlice, (int)p.n0, bar);
                    } else {
                        const int from = MODE == kDx && k >= g.slices ? 1 : 0;
                        const int at = (k - from * g.slices) * kSlice;
                        if (MODE == kDx) {
                            load_box(a, &g.a[from], at, m, bar);
                        } else {
                            load_box(a, &g.a[p.which], m, at, bar);
                            load_box(a + kBoxBytes, &g.a[p.which], m + kSlice, at, bar);
                        }
                        load_box(b, &g.b[from], n, at, bar);
                        load_box(b + kBoxBytes, &g.b[from], n + kSlice, at, bar);
                    }
                }
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
            for (int t = pair; ok && t < g.tiles; t += pairs, ++made) {
                const uint32_t into = made % 2, at = tmem + into * kSide;
                if (!(ok = wait_limited(&s.written[into], (made / 2 & 1) ^ 1, stop, g.stalled)))
                    break;
                tc_fence_after();
                for (int k = 0; k < slices; ++k, ++step) {
                    const int i = step % kStages;
                    if (!(ok = wait_limited(&s.full[i], step / kStages & 1, stop, g.stalled)))
                        break;
                    tc_fence_after();
                    const unsigned char *const pa = stages + i * kStageBytes,
                                        *const pb = pa + kOperandBytes;
                    const uint64_t a = A_ROWS ? operand_along_rows(pa, kBoxBytes) : operand_along_k(pa);
                    const uint64_t b = B_ROWS ? operand_along_rows(pb, kBoxBytes) : operand_along_k(pb);
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
    } else {
        const int quarter = warp % 4; // of the lanes of tensor memory, that a warp can read
        uint32_t made = 0;
        for (int t = pair; t < g.tiles; t += pairs, ++made) {
            const uint32_t into = made % 2;
            const bool ok = wait_limited(&s.summed[into], made / 2 & 1, stop, g.stalled);
            if (!__all_sync(kFull, ok))
                break;
            tc_fence_after();
            const TilePlace p = tile_place<MODE>(g, t);
            const long long r = p.m0 + rank * kHalf + quarter * 32 + lane;
            const uint32_t at = tmem + into * kSide + ((uint32_t)quarter * 32 << 16);
            O *const out = static_cast<O *>(g.out[p.which]);
            const bool whole = g.n % 8 == 0 && aligned_to(out, 16);
            if (MODE == kForward)
                write_forward<T>(g, at, r, p.n0,
                                 whole && (g.gate.exps || aligned_to(g.gate.data, 16)) &&
                                     (g.up.exps || aligned_to(g.up.data, 16)));
            else
                write_plain<O>(g, out, at, r, p.n0, whole);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_at(cluster_address(&s.written[into], 0));
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

// Boxes of 64 x box_rows elements of a matrix of 16-bit numbers; what is outside of it
// is read as zero.
bool make_map(CUtensorMap *m, bool bf16, const Matrix16 &x, int box_rows)
{
    const EncodeFn fn = encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows},
                     strides[1] = {(cuuint64_t)x.ld * 2};
    const cuuint32_t box[2] = {kSlice, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void *>(x.p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of blocks that the device runs at a time.
int resident_pairs(const void *fn)
{
    static std::mutex mu;
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64)
        return std::max(1, num_sms() / 2);
    std::lock_guard<std::mutex> lk(mu);
    if (!cached[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_sms() / 2 * 2);
        cfg.blockDim = dim3(kGemmThreads);
        cfg.dynamicSmemBytes = kGemmSmem;
        cudaLaunchAttribute at[1] = {};
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = std::max(1, num_sms() / 2);
        }
        cached[dev] = std::min(n, std::max(1, num_sms() / 2));
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
    cfg.gridDim = dim3(2 * std::min(resident_pairs(reinterpret_cast<const void *>(fn)), g.tiles));
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
    return cudaLaunchKernelEx(&cfg, fn, g);
}

// Tiles of all outputs; false: more than an int counts.
bool set_tiles(Gemm &g, int outputs, long long step_n)
{
    const long long tm = (g.m + kSide - 1) / kSide, tn = (g.n + step_n - 1) / step_n;
    if (tm * tn * outputs > 0x3fffffff)
        return false;
    g.tiles_m = (int)tm;
    g.tiles_n = (int)tn;
    g.tiles = (int)(tm * tn) * outputs;
    return true;
}

int slices_of(long long k) { return (int)((k + kSlice - 1) / kSlice); }

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

template <typename T> cudaError_t gemm_forward(const FfArgs &a, const Matrix16 &x, const Matrix16 &wg,
                                               const Matrix16 &wu, cudaStream_t st)
{
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    Gemm g = {};
    g.m = a.rows;
    g.n = a.ff;
    g.act = a.act;
    g.out[0] = a.h;
    g.gate = a.gate;
    g.up = a.up;
    g.slices = slices_of(a.dim);
    if (!set_tiles(g, 1, kHalf) || !make_map(&g.a[0], bf16, x, kHalf) ||
        !make_map(&g.b[0], bf16, wg, kHalf) || !make_map(&g.b[1], bf16, wu, kHalf))
        return cudaErrorInvalidValue;
    return launch_gemm<T, T, kForward>(g, st);
}

template <typename T>
cudaError_t gemm_dx(const FfGradArgs &a, const Matrix16 &dgate, const Matrix16 &dup,
                    const Matrix16 &wg, const Matrix16 &wu, cudaStream_t st)
{
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    Gemm g = {};
    g.m = a.rows;
    g.n = a.dim;
    g.out[0] = a.dx;
    g.slices = slices_of(a.ff);
    if (!set_tiles(g, 1, kSide) || !make_map(&g.a[0], bf16, dgate, kHalf) ||
        !make_map(&g.a[1], bf16, dup, kHalf) || !make_map(&g.b[0], bf16, wg, kSlice) ||
        !make_map(&g.b[1], bf16, wu, kSlice))
        return cudaErrorInvalidValue;
    return launch_gemm<T, T, kDx>(g, st);
}

template <typename T, typename O>
cudaError_t gemm_dw(const FfGradArgs &a, const Matrix16 &dgate, const Matrix16 &dup,
                    const Matrix16 &x, cudaStream_t st)
{
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    Gemm g = {};
    g.m = a.ff;
    g.n = a.dim;
    g.out[0] = a.dwg;
    g.out[1] = a.dwu;
    g.accumulate = a.accumulate;
    g.first_out = a.dwg ? 0 : 1;
    g.slices = slices_of(a.rows);
    if (!set_tiles(g, a.dwg && a.dwu ? 2 : 1, kSide) || !make_map(&g.a[0], bf16, dgate, kSlice) ||
        !make_map(&g.a[1], bf16, dup, kSlice) || !make_map(&g.b[0], bf16, x, kSlice))
        return cudaErrorInvalidValue;
    return launch_gemm<T, O, kDw>(g, st);
}

#define RRA_GEMM(T)                                                                              \
    template cudaError_t gemm_forward<T>(const FfArgs &, const Matrix16 &, const Matrix16 &,     \
                                         const Matrix16 &, cudaStream_t);                        \
    template cudaError_t gemm_dx<T>(const FfGradArgs &, const Matrix16 &, const Matrix16 &,      \
                                    const Matrix16 &, const Matrix16 &, cudaStream_t);           \
    template cudaError_t gemm_dw<T, T>(const FfGradArgs &, const Matrix16 &, const Matrix16 &,   \
                                       const Matrix16 &, cudaStream_t);                          \
    template cudaError_t gemm_dw<T, float>(const FfGradArgs &, const Matrix16 &,                 \
                                           const Matrix16 &, const Matrix16 &, cudaStream_t);
RRA_GEMM(__half)
RRA_GEMM(__nv_bfloat16)
#undef RRA_GEMM

} // namespace rra
