// gated_ff.cu -- rra_gated_ff and rra_gated_ff_grad.
//
//   g = x Wg^T,  u = x Wu^T,  h = a(g) u
//
//   dup = dh a(g),  dgate = dh u a'(g)
//   dx = dgate Wg + dup Wu,  dWg = dgate^T x,  dWu = dup^T x
//
// with M rows of x, D = dim and F = ff: 4 M F D operations forward, 8 backward.
//
// Here: the calls, the elementwise part of the gradient, and operands laid out for the
// products, which stand in gated_gemm.cu and, for few rows, gated_rows.cu.  dgate and dup
// are rounded to the call's type before they are multiplied, as the tensor cores take
// them: an error of half a step of a 16-bit number in each, as large as the results' own.
#include "gated_ff.h"

#include "gated_act.cuh"
#include "op_common.cuh"
#include "ragged.cuh"
#include "saved.cuh"

namespace rra {
namespace {

// ---------------------------------------------------------------- elementwise part of the gradient

constexpr int kActThreads = 256;

// Packs of 8 elements of a row; SAVED: gate and up in 8 bits.  Every element is read
// before it is written, so outputs may take inputs' places.  Bound by memory: 8192 x 16384
// bf16 from 8 bits take 187 us without h (1.08 GB, 5.8 TB/s) and 214 with it (1.34 GB,
// 6.3 TB/s).  WHOLE: every pack is on a 16-byte boundary.
template <typename T, bool SAVED, bool WHOLE, int ACT>
__global__ void __launch_bounds__(kActThreads) act_grad_kernel(const FfGradArgs a, int lanes)
{
    constexpr bool exact = sizeof(T) == 4;
    constexpr int N = kPackWords<T>;
    const long long count = a.rows * a.ff;
    const T *const dh = static_cast<const T *>(a.dh), *const gate = static_cast<const T *>(a.gate.data),
                   *const up = static_cast<const T *>(a.up.data);
    const long long nb = blocks_of(a.ff), packs = (a.ff + kPack - 1) / kPack;
    const int li = threadIdx.x % lanes, groups = kActThreads / lanes, stretch = min(lanes, 32);
    dependents_wait();
    dependents_launch();
    // (all lanes go on together: those of a warp store together)
    for (long long base = (long long)blockIdx.x * groups; base < a.rows;
         base += (long long)gridDim.x * groups) {
        const long long r = base + threadIdx.x / lanes;
#pragma unroll 2
        for (long long u0 = 0; u0 < packs; u0 += lanes) {
            const long long u = u0 + li, at = r * a.ff + u * kPack;
            const bool on = r < a.rows;
            const auto in = [&](long long p) {
                return (int)max(0LL, min((long long)kPack, a.ff - p * kPack));
            };
            const int there = on ? in(u) : 0;
            float g[8], v[8];
            uint32_t d[N];
            load_words<T, WHOLE>(dh + at, there, dh, dh + count, d);
            if (SAVED) {
                const long long b = r * nb + u / kBlockPacks, c = (r * nb * kBlockPacks + u) * kPack;
                Codes8 cg = {{0u, 0u}}, cu = cg;
                int8_t eg = 0, eu = 0;
                if (there > 0) {
                    cg = load_codes(static_cast<const int8_t *>(a.gate.data) + c);
                    cu = load_codes(static_cast<const int8_t *>(a.up.data) + c);
                    eg = a.gate.exps[b];
                    eu = a.up.exps[b];
                }
                decode8(cg, eg, g);
                decode8(cu, eu, v);
            } else {
                uint32_t wg[N], wu[N];
                load_words<T, WHOLE>(gate + at, there, gate, gate + count, wg);
                load_words<T, WHOLE>(up + at, there, up, up + count, wu);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    g[j] = element<T>(wg, j);
                    v[j] = element<T>(wu, j);
                }
            }
            float dg[8], du[8], h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float slope;
                const float value = act_both<ACT, exact>(g[j], &slope), x = element<T>(d, j);
                dg[j] = x * v[j] * slope;
                du[j] = x * value;
                h[j] = value * v[j];
            }
            // (a misaligned store takes neighbours' elements along: all of the warp has read)
            if (!WHOLE)
                __syncwarp();
            uint32_t o[N];
            const int next = in(u + 1);
            Carry<T> none;
            to_words<T>(dg, o);
            store_words<T, WHOLE>(static_cast<T *>(a.dgate) + at, there, next, on, stretch, o, none);
            to_words<T>(du, o);
            store_words<T, WHOLE>(static_cast<T *>(a.dup) + at, there, next, on, stretch, o, none);
            if (a.h) {
                to_words<T>(h, o);
                store_words<T, WHOLE>(static_cast<T *>(a.h) + at, there, next, on, stretch, o, none);
            }
        }
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
    return host_by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        const auto fn = a.gate.exps ? (vec ? act_grad_kernel<T, true, true, ACT>
                                           : act_grad_kernel<T, true, false, ACT>)
                                    : (vec ? act_grad_kernel<T, false, true, ACT>
                                           : act_grad_kernel<T, false, false, ACT>);
        return launch_chained(fn, grid, kActThreads, st, a, lanes);
    });
}

// ---------------------------------------------------------------- operands for the products

// A matrix whose rows do not begin on 16-byte boundaries, copied to rows that do; one
// of fp32 numbers cut into three planes of bf16, 8 bits of each number in the first,
// the next 8 in the second and the rest in the third.  (Cut, not rounded: the three
// add up to the number exactly, and none is larger.)
struct Copies {
    struct {
        const void *from;
        uint32_t *to;
        long long rows, cols, ld;
    } c[5];
};

// blockIdx.y: the matrix.
template <typename T> __global__ void __launch_bounds__(kActThreads) operand_kernel(const Copies all)
{
    const T *const from = static_cast<const T *>(all.c[blockIdx.y].from);
    uint32_t *const to = all.c[blockIdx.y].to;
    const long long rows = all.c[blockIdx.y].rows, cols = all.c[blockIdx.y].cols,
                    ld = all.c[blockIdx.y].ld;
    const long long packs = ld / kPack, total = rows * packs;
    dependents_wait();
    dependents_launch();
    for (long long i = (long long)blockIdx.x * kActThreads + threadIdx.x; i < total;
         i += (long long)gridDim.x * kActThreads) {
        const long long r = i / packs, c = (i - r * packs) * kPack;
        uint32_t w[kPackWords<T>];
        load_words<T, false>(from + r * cols + c, (int)min((long long)kPack, cols - c), from,
                             from + rows * cols, w);
        uint4 *const at = reinterpret_cast<uint4 *>(to) + i;
        if constexpr (sizeof(T) == 2) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint32_t q[3][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = __uint_as_float(w[j]);
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const uint32_t top = __float_as_uint(v) & 0xffff0000u;
                    q[p][j / 2] = j % 2 ? q[p][j / 2] | top : top >> 16;
                    // (what is not finite is all in the first plane; a NaN of the low bits
                    // alone keeps being one)
                    const float rest = v - __uint_as_float(top);
                    if (p == 0 && (w[j] & 0x7f800000u) == 0x7f800000u) {
                        if (w[j] & 0x007fffffu)
                            q[0][j / 2] |= j % 2 ? 0x00400000u : 0x00000040u;
                        v = 0.0f;
                    } else {
                        v = rest;
                    }
                }
            }
#pragma unroll
            for (int p = 0; p < 3; ++p)
                at[p * total] = make_uint4(q[p][0], q[p][1], q[p][2], q[p][3]);
        }
    }
}

// Operands as the products can read them: where they are, or in the stream's scratch,
// where the products' own parts are, too.
template <typename T, int N> class Operands {
public:
    Matrix16 m[N];
    unsigned char *scratch = nullptr;
    size_t parts_at = 0;

    explicit Operands(const Matrix16 (&given)[N])
    {
        size_t at = kScratchHead;
        for (int i = 0; i < N; ++i) {
            m[i] = given[i];
            m[i].planes = sizeof(T) == 4 ? 3 : 1;
            copy_[i] = m[i].p && (sizeof(T) == 4 || !gemm_takes(m[i]));
            if (copy_[i]) {
                m[i].ld = (m[i].cols + kPack - 1) / kPack * kPack;
                at_[i] = at;
                at += ((size_t)m[i].planes * m[i].rows * m[i].ld * 2 + 255) & ~(size_t)255;
            }
        }
        parts_at = at;
    }
    rra_status take(size_t parts, cudaStream_t st)
    {
        if (parts_at + parts == kScratchHead)
            return RRA_OK;
        return op_scratch(st, parts_at + parts, lk_, &scratch);
    }
    // Copies those that need it, once what they hold is there.
    cudaError_t fill(cudaStream_t st)
    {
        Copies all = {};
        int n = 0;
        long long most = 0;
        for (int i = 0; i < N; ++i)
            if (copy_[i]) {
                uint32_t *const to = reinterpret_cast<uint32_t *>(scratch + at_[i]);
                all.c[n++] = {m[i].p, to, m[i].rows, m[i].cols, m[i].ld};
                most = std::max(most, m[i].rows * (m[i].ld / kPack));
                m[i].p = to;
            }
        if (n == 0)
            return cudaSuccess;
        const unsigned grid =
            (unsigned)std::min((most + kActThreads - 1) / kActThreads, (long long)num_sms() * 16);
        return launch_chained(operand_kernel<T>, dim3(grid, n), kActThreads, st, all);
    }

private:
    bool copy_[N];
    size_t at_[N];
    std::unique_lock<std::mutex> lk_; // until the call's launches are queued
};

// ---------------------------------------------------------------- calls

template <typename T> rra_status ff(const FfArgs &a, cudaStream_t st)
{
    if (few_rows<T>(a))
        return rows_forward<T>(a, st);
    rra_status s;
    Operands<T, 3> in({{a.x, a.rows, a.dim, a.dim, 1},
                       {a.wg, a.ff, a.dim, a.dim, 1},
                       {a.wu, a.ff, a.dim, a.dim, 1}});
    if ((s = in.take(gemm_parts(a, sizeof(T) == 4), st)) != RRA_OK)
        return s;
    const cudaError_t e = in.fill(st);
    return launched(e == cudaSuccess ? gemm_forward<T>(a, in.m, in.scratch, in.parts_at, st) : e);
}

template <typename T, typename O> rra_status ff_grad(const FfGradArgs &a, cudaStream_t st)
{
    const bool weights = a.dwg || a.dwu;
    if (a.rows == 0) { // sums over nothing
        cudaError_t e = cudaSuccess;
        for (void *out : {a.dwg, a.dwu})
            if (e == cudaSuccess && out && !a.accumulate)
                e = cudaMemsetAsync(out, 0, (size_t)a.ff * a.dim * sizeof(O), st);
        return launched(e);
    }
    rra_status s = RRA_OK;
    const bool products = a.dx || weights;
    Operands<T, 5> in({{products ? a.dgate : nullptr, a.rows, a.ff, a.ff, 1},
                       {products ? a.dup : nullptr, a.rows, a.ff, a.ff, 1},
                       {a.dx ? a.wg : nullptr, a.ff, a.dim, a.dim, 1},
                       {a.dx ? a.wu : nullptr, a.ff, a.dim, a.dim, 1},
                       {weights ? a.x : nullptr, a.rows, a.dim, a.dim, 1}});
    if (products && (s = in.take(gemm_parts(a, sizeof(T) == 4), st)) != RRA_OK)
        return s;
    cudaError_t e = act_grad<T>(a, st);
    if (e == cudaSuccess && products)
        e = in.fill(st);
    if (e == cudaSuccess && a.dx)
        e = gemm_dx<T>(a, in.m, in.scratch, in.parts_at, st);
    if (e == cudaSuccess && weights)
        e = gemm_dw<T, O>(a, in.m, in.scratch, in.parts_at, st);
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
