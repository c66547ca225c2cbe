// gated_ff.cu -- rra_gated_ff and rra_gated_ff_grad.
//
//   g = x Wg^T,  u = x Wu^T,  h = a(g) u
//
//   dup = dh a(g),  dgate = dh u a'(g)
//   dx = dgate Wg + dup Wu,  dWg = dgate^T x,  dWu = dup^T x
//
// with M rows of x, D = dim and F = ff: 4 M F D operations forward, 8 backward.
#include "gated_ff.h"

#include "gated_act.cuh"
#include "op_common.cuh"
#include "saved.cuh"

namespace rra {
namespace {

// ---------------------------------------------------------------- products without tensor cores

// out[m, n] = sum over k of a(m, k) b(k, n), over one or two pairs of operands
// (their sums added), or two outputs of one a.  An operand is read along k or along
// its rows, whichever is next to each other in memory.
//
// A block makes 32 x 128 results, a warp 4 rows of 128 (one block of codes), a
// lane 4 x 4 of each; the operands come in slices of 16 along k.
constexpr int kTileM = 32, kTileN = 128, kTileK = 16, kTileThreads = 256;

struct Operand {
    const void *p;
    long long ld;
};

// A slice of R rows of an operand, [k][row], as fp32.  ALONG: k is next to each other.
template <typename T, int R, bool ALONG>
__device__ __forceinline__ void load_slice(float (&to)[kTileK][R + 4], const Operand &o,
                                           long long row0, long long rows, long long k0,
                                           long long depth)
{
    const T *const p = static_cast<const T *>(o.p);
#pragma unroll
    for (int i = threadIdx.x; i < R * kTileK; i += kTileThreads) {
        const int k = ALONG ? i % kTileK : i / R, r = ALONG ? i / kTileK : i % R;
        const bool there = row0 + r < rows && k0 + k < depth;
        to[k][r] = there ? to_f32(ALONG ? p[(row0 + r) * o.ld + k0 + k] : p[(k0 + k) * o.ld + row0 + r])
                         : 0.0f;
    }
}

__device__ __forceinline__ void add_products(const float (&a)[kTileK][kTileM + 4],
                                             const float (&b)[kTileK][kTileN + 4],
                                             float (&acc)[4][4])
{
    const int m = threadIdx.x / 32 * 4, n = threadIdx.x % 32 * 4;
#pragma unroll
    for (int k = 0; k < kTileK; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(a[k][m + i], b[k][n + j], acc[i][j]);
}

// Gate or up: the values, or their codes.
template <typename T>
__device__ __forceinline__ void keep_row(const Kept &to, long long r, long long c0, long long ff,
                                         const float v[4])
{
    const int c = threadIdx.x % 32 * 4;
    if (to.exps) { // every lane of the warp is here
        uint32_t top = 0;
        float w[8] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = c0 + c + j < ff ? v[j] : 0.0f;
            top = max(top, __float_as_uint(w[j]) & 0x7fffffffu);
        }
        top = __reduce_max_sync(kFull, top);
        const Codes8 q = encode8(w, top);
        const long long nb = blocks_of(ff), b = c0 / kBlock;
        *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(to.data) + (r * nb + b) * kBlock + c) =
            q.w[0];
        if (c == 0)
            to.exps[r * nb + b] = exponent_byte(block_exponent(top));
    } else if (to.data) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c0 + c + j < ff)
                static_cast<T *>(to.data)[r * ff + c0 + c + j] = from_f32<T>(v[j]);
    }
}

template <typename T> __global__ void __launch_bounds__(kTileThreads) ff_plain_kernel(const FfArgs a)
{
    __shared__ float sx[kTileK][kTileM + 4], sg[kTileK][kTileN + 4], su[kTileK][kTileN + 4];
    dependents_wait();
    dependents_launch();
    const long long tn = (a.ff + kTileN - 1) / kTileN, tm = (a.rows + kTileM - 1) / kTileM;
    for (long long t = blockIdx.x; t < tn * tm; t += gridDim.x) {
        const long long m0 = t / tn * kTileM, n0 = t % tn * kTileN;
        float g[4][4] = {}, u[4][4] = {};
        for (long long k0 = 0; k0 < a.dim; k0 += kTileK) {
            __syncthreads();
            load_slice<T, kTileM, true>(sx, {a.x, a.dim}, m0, a.rows, k0, a.dim);
            load_slice<T, kTileN, true>(sg, {a.wg, a.dim}, n0, a.ff, k0, a.dim);
            load_slice<T, kTileN, true>(su, {a.wu, a.dim}, n0, a.ff, k0, a.dim);
            __syncthreads();
            add_products(sx, sg, g);
            add_products(sx, su, u);
        }
        constexpr bool exact = sizeof(T) == 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long r = m0 + threadIdx.x / 32 * 4 + i, c = n0 + threadIdx.x % 32 * 4;
            if (r >= a.rows) // (all of a warp or none)
                continue;
            keep_row<T>(a.gate, r, n0, a.ff, g[i]);
            keep_row<T>(a.up, r, n0, a.ff, u[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < a.ff)
                    static_cast<T *>(a.h)[r * a.ff + c + j] =
                        from_f32<T>(act_value<exact>(a.act, g[i][j]) * u[i][j]);
        }
    }
}

// out (rows x cols) = a1 b1 (+ a2 b2), or += where it accumulates.
struct Product {
    Operand a[2], b[2];
    int pairs;
    long long rows, cols, depth;
    void *out;
    int accumulate;
};

// AK, BK: is a, b next to each other along k?
template <typename T, typename O, bool AK, bool BK>
__global__ void __launch_bounds__(kTileThreads) product_kernel(const Product p)
{
    __shared__ float sa[kTileK][kTileM + 4], sb[kTileK][kTileN + 4];
    const long long tn = (p.cols + kTileN - 1) / kTileN, tm = (p.rows + kTileM - 1) / kTileM;
    for (long long t = blockIdx.x; t < tn * tm; t += gridDim.x) {
        const long long m0 = t / tn * kTileM, n0 = t % tn * kTileN;
        float acc[4][4] = {};
        for (int i = 0; i < p.pairs; ++i)
            for (long long k0 = 0; k0 < p.depth; k0 += kTileK) {
                __syncthreads();
                load_slice<T, kTileM, AK>(sa, p.a[i], m0, p.rows, k0, p.depth);
                load_slice<T, kTileN, BK>(sb, p.b[i], n0, p.cols, k0, p.depth);
                __syncthreads();
                add_products(sa, sb, acc);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long r = m0 + threadIdx.x / 32 * 4 + i, c = n0 + threadIdx.x % 32 * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r < p.rows && c + j < p.cols) {
                    O *const to = static_cast<O *>(p.out) + r * p.cols + c + j;
                    *to = from_f32<O>(p.accumulate ? to_f32(*to) + acc[i][j] : acc[i][j]);
                }
        }
    }
}

template <typename T, typename O, bool AK, bool BK>
cudaError_t product(const Product &p, cudaStream_t st)
{
    const long long tiles = (p.cols + kTileN - 1) / kTileN * ((p.rows + kTileM - 1) / kTileM);
    product_kernel<T, O, AK, BK>
        <<<(unsigned)std::min(tiles, 1LL << 20), kTileThreads, 0, st>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- elementwise part of the gradient

constexpr int kActThreads = 256;

// Packs of 8 elements of a row; SAVED: gate and up in 8 bits.  Every element is read
// before it is written, so outputs may take inputs' places.
template <typename T, bool SAVED, bool VEC>
__global__ void __launch_bounds__(kActThreads) act_grad_kernel(const FfGradArgs a, int lanes)
{
    constexpr bool exact = sizeof(T) == 4;
    const T *const dh = static_cast<const T *>(a.dh);
    const long long nb = blocks_of(a.ff), packs = (a.ff + kPack - 1) / kPack;
    const int li = threadIdx.x % lanes, groups = kActThreads / lanes;
    dependents_wait();
    dependents_launch();
    for (long long r = (long long)blockIdx.x * groups + threadIdx.x / lanes; r < a.rows;
         r += (long long)gridDim.x * groups)
        for (long long u = li; u < packs; u += lanes) {
            const int there = (int)min((long long)kPack, a.ff - u * kPack);
            const long long at = r * a.ff + u * kPack;
            float g[8], v[8], d[8];
            if (SAVED) {
                const long long b = r * nb + u / kBlockPacks, c = (r * nb * kBlockPacks + u) * kPack;
                decode8(load_codes(static_cast<const int8_t *>(a.gate.data) + c), a.gate.exps[b],
                        g);
                decode8(load_codes(static_cast<const int8_t *>(a.up.data) + c), a.up.exps[b], v);
            } else {
                load8<T, VEC>(static_cast<const T *>(a.gate.data) + at, there, g);
                load8<T, VEC>(static_cast<const T *>(a.up.data) + at, there, v);
            }
            load8<T, VEC>(dh + at, there, d);
            float dg[8], h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float slope;
                const float value = act_both<exact>(a.act, g[j], &slope);
                dg[j] = d[j] * v[j] * slope;
                h[j] = value * v[j];
                d[j] *= value;
            }
            store8<T, VEC>(static_cast<T *>(a.dgate) + at, there, dg);
            store8<T, VEC>(static_cast<T *>(a.dup) + at, there, d);
            if (a.h)
                store8<T, VEC>(static_cast<T *>(a.h) + at, there, h);
        }
}

template <typename T> cudaError_t act_grad(const FfGradArgs &a, cudaStream_t st)
{
    bool vec = a.ff % kPack == 0;
    for (const void *p : {a.dh, a.gate.exps ? nullptr : (const void *)a.gate.data,
                          a.up.exps ? nullptr : (const void *)a.up.data, (const void *)a.dgate,
                          (const void *)a.dup, (const void *)a.h})
        vec = vec && (!p || aligned_to(p, 16));
    int lanes = 1;
    while (lanes < kActThreads && lanes * kPack < a.ff)
        lanes *= 2;
    const int groups = kActThreads / lanes;
    const dim3 grid((unsigned)std::max(
        1LL, std::min((a.rows + groups - 1) / groups, (long long)num_sms() * 8)));
    const auto fn = a.gate.exps ? (vec ? act_grad_kernel<T, true, true> : act_grad_kernel<T, true, false>)
                                : (vec ? act_grad_kernel<T, false, true>
                                       : act_grad_kernel<T, false, false>);
    return launch_chained(fn, grid, kActThreads, st, a, lanes);
}

// ---------------------------------------------------------------- operands for tensor maps

// A matrix whose rows do not begin on 16-byte boundaries, copied to rows that do.
template <typename T>
__global__ void __launch_bounds__(kActThreads) align_kernel(const T *from, T *to, long long rows,
                                                            long long cols, long long ld)
{
    const long long packs = ld / kPack, total = rows * packs;
    dependents_wait();
    dependents_launch();
    for (long long i = (long long)blockIdx.x * kActThreads + threadIdx.x; i < total;
         i += (long long)gridDim.x * kActThreads) {
        const long long r = i / packs, c = (i - r * packs) * kPack;
        const int there = (int)min((long long)kPack, cols - c);
        Pack<T, kPack> v;
#pragma unroll
        for (int j = 0; j < kPack; ++j)
            v.e[j] = j < there ? from[r * cols + c + j] : from_f32<T>(0.0f);
        store_pack<T, kPack>(to + r * ld + c, v);
    }
}

// Operands as tensor maps can read them: where they are, or in the stream's scratch.
template <typename T, int N> class Aligned {
public:
    Matrix16 m[N];

    // Plans copies of those that need one; their places follow from take().
    explicit Aligned(const Matrix16 (&given)[N])
    {
        for (int i = 0; i < N; ++i) {
            m[i] = given[i];
            copy_[i] = m[i].p && m[i].rows > 0 && !gemm_takes(m[i]);
            if (copy_[i]) {
                m[i].ld = (m[i].cols + kPack - 1) / kPack * kPack;
                at_[i] = bytes_;
                bytes_ += (size_t)m[i].rows * m[i].ld * sizeof(T) + 255 & ~(size_t)255;
            }
        }
    }
    size_t bytes() const { return bytes_; }
    rra_status take(cudaStream_t st)
    {
        if (!bytes_)
            return RRA_OK;
        const rra_status r = op_scratch(st, kScratchHead + bytes_, lk_, &ws_);
        return r;
    }
    // Copies operand i, once what it holds is there.
    cudaError_t fill(int i, cudaStream_t st)
    {
        if (!copy_[i])
            return cudaSuccess;
        T *const to = reinterpret_cast<T *>(ws_ + kScratchHead + at_[i]);
        const long long packs = m[i].rows * (m[i].ld / kPack);
        const unsigned grid = (unsigned)std::min((packs + kActThreads - 1) / kActThreads,
                                                 (long long)num_sms() * 32);
        const cudaError_t e =
            launch_chained(align_kernel<T>, dim3(grid), kActThreads, st,
                           static_cast<const T *>(m[i].p), to, m[i].rows, m[i].cols, m[i].ld);
        m[i].p = to;
        return e;
    }

private:
    bool copy_[N];
    size_t at_[N], bytes_ = 0;
    unsigned char *ws_ = nullptr;
    std::unique_lock<std::mutex> lk_; // until the call's launches are queued
};

// ---------------------------------------------------------------- calls

// Has a kernel given up waiting since the last call?
rra_status stalled_status()
{
    unsigned *word = nullptr;
    if (stalled_word(&word) != cudaSuccess)
        return RRA_ERR_CUDA;
    volatile unsigned *const w = word;
    if (!*w)
        return RRA_OK;
    *w = 0;
    return RRA_ERR_TIMEOUT;
}

template <typename T> rra_status ff_tensor(const FfArgs &a, cudaStream_t st)
{
    rra_status s = stalled_status();
    if (s != RRA_OK)
        return s;
    Aligned<T, 3> in({{a.x, a.rows, a.dim, a.dim}, {a.wg, a.ff, a.dim, a.dim},
                      {a.wu, a.ff, a.dim, a.dim}});
    if ((s = in.take(st)) != RRA_OK)
        return s;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 3 && e == cudaSuccess; ++i)
        e = in.fill(i, st);
    return launched(e == cudaSuccess ? gemm_forward<T>(a, in.m[0], in.m[1], in.m[2], st) : e);
}

template <typename T, typename O> rra_status ff_grad_tensor(const FfGradArgs &a, cudaStream_t st)
{
    rra_status s = stalled_status();
    if (s != RRA_OK)
        return s;
    const bool weights = a.dwg || a.dwu;
    Aligned<T, 5> in({{a.dgate, a.rows, a.ff, a.ff},
                      {a.dup, a.rows, a.ff, a.ff},
                      {a.dx ? a.wg : nullptr, a.ff, a.dim, a.dim},
                      {a.dx ? a.wu : nullptr, a.ff, a.dim, a.dim},
                      {weights ? a.x : nullptr, a.rows, a.dim, a.dim}});
    if (!a.dx && !weights)
        return launched(act_grad<T>(a, st));
    if ((s = in.take(st)) != RRA_OK)
        return s;
    cudaError_t e = act_grad<T>(a, st);
    for (int i = 0; i < 5 && e == cudaSuccess; ++i)
        e = in.fill(i, st);
    if (e == cudaSuccess && a.dx)
        e = gemm_dx<T>(a, in.m[0], in.m[1], in.m[2], in.m[3], st);
    if (e == cudaSuccess && weights)
        e = gemm_dw<T, O>(a, in.m[0], in.m[1], in.m[4], st);
    return launched(e);
}

template <typename T> rra_status ff(const FfArgs &a, cudaStream_t st)
{
    if constexpr (sizeof(T) == 2)
        return ff_tensor<T>(a, st);
    const long long tiles = (a.ff + kTileN - 1) / kTileN * ((a.rows + kTileM - 1) / kTileM);
    return launched(launch_chained(ff_plain_kernel<T>, dim3((unsigned)std::min(tiles, 1LL << 20)),
                                   kTileThreads, st, a));
}

template <typename T, typename O> rra_status ff_grad(const FfGradArgs &a, cudaStream_t st)
{
    if constexpr (sizeof(T) == 2)
        if (a.rows > 0)
            return ff_grad_tensor<T, O>(a, st);
    cudaError_t e = a.rows > 0 ? act_grad<T>(a, st) : cudaSuccess;
    if (e == cudaSuccess && a.dx && a.rows > 0) {
        const Product p{{{a.dgate, a.ff}, {a.dup, a.ff}},
                        {{a.wg, a.dim}, {a.wu, a.dim}},
                        2,
                        a.rows,
                        a.dim,
                        a.ff,
                        a.dx,
                        0};
        e = product<T, T, true, false>(p, st);
    }
    for (int i = 0; i < 2; ++i) {
        void *const out = i == 0 ? a.dwg : a.dwu;
        if (e != cudaSuccess || !out || (a.rows == 0 && a.accumulate))
            continue;
        const Product p{{{i == 0 ? a.dgate : a.dup, a.ff}},
                        {{a.x, a.dim}},
                        1,
                        a.ff,
                        a.dim,
                        a.rows,
                        out,
                        a.accumulate};
        e = product<T, O, false, false>(p, st);
    }
    return launched(e);
}

constexpr size_t kMost = (size_t)1 << 30; // rows, dim, ff

bool valid_ff(size_t rows, size_t dim, size_t ff, rra_dtype t, rra_act act)
{
    return valid_dt(t) && (unsigned)act <= RRA_ACT_RELU && rows <= kMost && dim > 0 &&
           dim <= kMost && ff > 0 && ff <= kMost && holdable(rows, dim, 4) &&
           holdable(rows, ff, 4) && holdable(ff, dim, 4) &&
           holdable(rows, (size_t)blocks_of((long long)ff) * kBlock, 1);
}

} // namespace
} // namespace rra

extern "C" rra_status rra_gated_ff(const void *x, const void *w_gate, const void *w_up, size_t rows,
                                   size_t dim, size_t ff_, rra_dtype dtype, rra_act act, void *h,
                                   int8_t *gate_exps, void *gate, int8_t *up_exps, void *up,
                                   void *stream)
{
    using namespace rra;
    if (!valid_ff(rows, dim, ff_, dtype, act))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), hb = rows * ff_ * es, xb = rows * dim * es,
                 wb = ff_ * dim * es;
    if (!w_gate || !w_up || (rows > 0 && (!x || !h)))
        return RRA_ERR_INVALID;
    if ((gate_exps && !gate) || (up_exps && !up))
        return RRA_ERR_INVALID;
    if (!aligned_to(x, es) || !aligned_to(w_gate, es) || !aligned_to(w_up, es) ||
        !aligned_to(h, es) || !aligned_to(gate, gate_exps ? 16 : es) ||
        !aligned_to(up, up_exps ? 16 : es))
        return RRA_ERR_INVALID;
    const size_t eb = exps_bytes(rows, ff_), cb = codes_bytes(rows, ff_);
    const Span sh{h, hb}, ge{gate_exps, eb}, gd{gate, gate_exps ? cb : hb}, ue{up_exps, eb},
        ud{up, up_exps ? cb : hb}, sx{x, xb}, sg{w_gate, wb}, su{w_up, wb};
    if (any_overlap(sh, {ge, gd, ue, ud, sx, sg, su}) || any_overlap(ge, {gd, ue, ud, sx, sg, su}) ||
        any_overlap(gd, {ue, ud, sx, sg, su}) || any_overlap(ue, {ud, sx, sg, su}) ||
        any_overlap(ud, {sx, sg, su}))
        return RRA_ERR_INVALID;
    if (rows == 0)
        return RRA_OK;
    const FfArgs a{x, w_gate, w_up, (long long)rows, (long long)dim, (long long)ff_, act, h,
                   {gate_exps, gate}, {up_exps, up}};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == RRA_F32   ? ff<float>(a, st)
           : dtype == RRA_F16 ? ff<__half>(a, st)
                              : ff<__nv_bfloat16>(a, st);
}

extern "C" rra_status rra_gated_ff_grad(const void *dh, const void *x, const void *w_gate,
                                        const void *w_up, const int8_t *gate_exps,
                                        const void *gate, const int8_t *up_exps, const void *up,
                                        size_t rows, size_t dim, size_t ff_, rra_dtype dtype,
                                        rra_act act, void *dgate, void *dup, void *h, void *dx,
                                        void *dw_gate, void *dw_up, rra_dtype dweight_t,
                                        int accumulate, void *stream)
{
    using namespace rra;
    if (!valid_ff(rows, dim, ff_, dtype, act) || !valid_dt(dweight_t))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ds = dtype_size(dweight_t), hb = rows * ff_ * es,
                 xb = rows * dim * es, wb = ff_ * dim * es, db = ff_ * dim * ds;
    const bool weights = dw_gate || dw_up;
    if (rows > 0 && (!dh || !gate || !up || !dgate || !dup || (weights && !x)))
        return RRA_ERR_INVALID;
    if (rows > 0 && dx && (!w_gate || !w_up))
        return RRA_ERR_INVALID;
    if (!gate_exps != !up_exps) // both in 8 bits or neither
        return RRA_ERR_INVALID;
    const size_t kept = gate_exps ? 16 : es;
    for (const void *p : {dh, x, w_gate, w_up, (const void *)dgate, (const void *)dup,
                          (const void *)h, (const void *)dx})
        if (!aligned_to(p, es))
            return RRA_ERR_INVALID;
    if (!aligned_to(gate, kept) || !aligned_to(up, kept) || !aligned_to(dw_gate, ds) ||
        !aligned_to(dw_up, ds))
        return RRA_ERR_INVALID;
    const size_t eb = exps_bytes(rows, ff_), cb = codes_bytes(rows, ff_);
    const Span ge{gate_exps, eb}, gd{gate, gate_exps ? cb : hb}, ue{up_exps, eb},
        ud{up, up_exps ? cb : hb}, sdh{dh, hb}, sx{x, xb}, sg{w_gate, wb}, su{w_up, wb},
        dg{dgate, hb}, du{dup, hb}, sh{h, hb}, sdx{dx, xb}, dwg{dw_gate, db}, dwu{dw_up, db};
    // elementwise outputs: apart from each other; in the place of an elementwise input, or apart
    for (const Span &o : {dg, du, sh}) {
        if (any_overlap(o, {ge, ue, sx, sg, su, sdx, dwg, dwu}))
            return RRA_ERR_INVALID;
        for (const Span &in : {sdh, gd, ud})
            if (overlap(o.p, o.bytes, in.p, in.bytes) &&
                (o.p != in.p || (gate_exps && in.p != dh)))
                return RRA_ERR_INVALID;
    }
    if (any_overlap(dg, {du, sh}) || any_overlap(du, {sh}))
        return RRA_ERR_INVALID;
    for (const Span &o : {sdx, dwg, dwu})
        if (any_overlap(o, {ge, gd, ue, ud, sdh, sx, sg, su}))
            return RRA_ERR_INVALID;
    if (any_overlap(sdx, {dwg, dwu}) || any_overlap(dwg, {dwu}))
        return RRA_ERR_INVALID;
    if (dweight_t != dtype && dweight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    const FfGradArgs a{dh, x, w_gate, w_up,
                       {const_cast<int8_t *>(gate_exps), const_cast<void *>(gate)},
                       {const_cast<int8_t *>(up_exps), const_cast<void *>(up)},
                       (long long)rows, (long long)dim, (long long)ff_, act,
                       dgate, dup, h, dx, dw_gate, dw_up, accumulate};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == RRA_F32)
        return ff_grad<float, float>(a, st);
    if (dtype == RRA_F16)
        return dweight_t == RRA_F16 ? ff_grad<__half, __half>(a, st)
                                    : ff_grad<__half, float>(a, st);
    return dweight_t == RRA_BF16 ? ff_grad<__nv_bfloat16, __nv_bfloat16>(a, st)
                                 : ff_grad<__nv_bfloat16, float>(a, st);
}
