// layer_norm.cu -- rra_layer_norm and rra_layer_norm_grad.
//
//   mean = sum x / D,  var = sum (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y    = (x - mean) rstd gamma + beta
//
//   xh = (x - mean) rstd,  w = dy gamma
//   dx = rstd (w - mean(w) - xh mean(w xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound by memory: x read and y written; x and dy read and dx written.
// Measured at 16384 x 4096 bf16: 47 us forward (268 MB, 5.7 TB/s), 73.6 us
// backward (403 MB, 5.5 TB/s; 5 of the 73.6 for adding the partial rows of
// dgamma and dbeta); 15.1 us backward at 3001 x 1001 fp32 (36 MB): 20 rows an
// SM, so a start, an end and 4 turns of a row's latency, and 5 us for the join.
// Backward at 4096 rows of 16384 bf16: 90.5 us (403 MB, 4.45 TB/s).
#include <initializer_list>

#include "op_common.cuh"
#include "row_group.cuh"

namespace rra {
namespace {

// ---------------------------------------------------------------- forward

struct Fwd {
    const void *x, *gamma, *beta;
    long long rows, dim;
    float eps;
    void *y;
    float *mean, *rstd;
    Group g;
};

constexpr int kFwdThreads = 256; // of a block, where a group is no more than that

template <typename T, typename W, int V, int K, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 1024 : kFwdThreads, MULTI ? 1 : 4) norm_kernel(const Fwd a)
{
    __shared__ __align__(16) float sm[MULTI ? 2 * 32 : 4]; // a group of several warps is a block
    const T *const x = static_cast<const T *>(a.x);
    T *const y = static_cast<T *>(a.y);
    const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                static_cast<const W *>(a.beta);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, groups = blockDim.x / lanes;
    using P = Values<V>;
    using E = typename P::E;
    const int units = (int)a.dim / V, apart = lanes * V; // (a held row is short)
    const float n = (float)a.dim, inverse = 1.0f / n;
    bool in[K];  // does the lane hold a k-th pack?
    int col[K]; // its first column; that of the row's last pack if not
#pragma unroll
    for (int k = 0; k < K; ++k) {
        in[k] = li + k * lanes < units;
        col[k] = min(li + k * lanes, units - 1) * V;
    }
    GroupOf group = group_of(a.g, sm, 1);
    if (MULTI) {
        if (threadIdx.x < 64)
            sm[threadIdx.x] = 0.0f;
        __syncthreads();
    }
    const int first = threadIdx.x / lanes;
    dependents_wait();
    dependents_launch();
    for (long long base = (long long)blockIdx.x * groups; base < a.rows;
         base += (long long)gridDim.x * groups) {
        // every lane takes part in the sums, some in vain: they read the last row
        const long long r = MULTI ? base : min(base + first, a.rows - 1);
        const bool on = MULTI || base + first < a.rows;
        const T *const p = x + r * a.dim + li * V;
        Raw<T, V> raw[K];
        E sum = P::all(0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            raw[k].clear();
            if (in[k])
                raw[k].load(p + k * apart);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int m = 0; m < P::N; ++m)
                sum = add(sum, P::get(raw[k], m));
        Sums<1> s{{sum_of(sum)}};
        const float mu = quotient(group_sum<MULTI, 1>(s, group).v[0], n, inverse);
        sum = P::all(0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const E minus = P::all(in[k] ? -mu : 0.0f); // a pack that is not there stays zero
#pragma unroll
            for (int m = 0; m < P::N; ++m) {
                const E d = add(P::get(raw[k], m), minus);
                sum = fma(d, d, sum);
            }
        }
        s.v[0] = sum_of(sum);
        const float rs = rsqrtf(quotient(group_sum<MULTI, 1>(s, group).v[0], n, inverse) + a.eps);
        const E minus = P::all(-mu), scale = P::all(rs);
        T *const q = y + r * a.dim + li * V;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            E g[P::N], b[P::N];
            load_weights<W, V>(gamma, col[k], 1.0f, g);
            load_weights<W, V>(beta, col[k], 0.0f, b);
#pragma unroll
            for (int m = 0; m < P::N; ++m)
                g[m] = fma(mul(add(P::get(raw[k], m), minus), scale), g[m], b[m]);
            if (on && in[k])
                store_vals<T, V>(q + k * apart, g);
        }
        if (on && li == 0) {
            if (a.mean)
                a.mean[r] = mu;
            if (a.rstd)
                a.rstd[r] = rs;
        }
    }
}

// Rows that no block holds: three passes over each, the last two from L2.
constexpr int kLongThreads = 1024;

template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const Fwd a)
{
    __shared__ __align__(16) float sm[2 * 32];
    GroupOf block = group_of(Group{5, kLongThreads / 32}, sm, 1);
    dependents_wait();
    dependents_launch();
    const float n = (float)a.dim;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const p = static_cast<const T *>(a.x) + r * a.dim;
        const W *const gamma = static_cast<const W *>(a.gamma), *const beta =
                                                                    static_cast<const W *>(a.beta);
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
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float g = gamma ? to_f32(gamma[c]) : 1.0f, b = beta ? to_f32(beta[c]) : 0.0f;
            static_cast<T *>(a.y)[r * a.dim + c] =
                from_f32<T>(fmaf((to_f32(p[c]) - mu) * rs, g, b));
        }
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = mu;
            if (a.rstd)
                a.rstd[r] = rs;
        }
    }
}

constexpr int kShort = 8; // elements that a lane holds: of short rows
template <int V> constexpr int kHeld = V > 1 ? 32 : 16;

template <typename T, typename W, int V> cudaError_t forward_packs(Fwd a, cudaStream_t st)
{
    const long long units = a.dim / V;
    if (a.dim > 1024LL * kHeld<V>) {
        return launch_chained(norm_long_kernel<T, W>, dim3(grid_of(a.rows, 2)), kLongThreads, st,
                              a);
    } else if (a.dim <= 32 * kHeld<V>) {
        // a warp or a part of one; few elements a lane for short rows
        const bool few = a.dim <= 32 * kShort;
        a.g = group_for(units, (few ? kShort : kHeld<V>) / V);
        const int per_block = kFwdThreads / a.g.lanes();
        const unsigned grid = grid_of((a.rows + per_block - 1) / per_block, 16);
        if (few)
            return launch_chained(norm_kernel<T, W, V, kShort / V, false>, dim3(grid), kFwdThreads,
                                  st, a);
        return launch_chained(norm_kernel<T, W, V, kHeld<V> / V, false>, dim3(grid), kFwdThreads,
                              st, a);
    } else {
        a.g = group_for(units, kHeld<V> / V);
        const int threads = 32 * a.g.warps;
        return launch_chained(norm_kernel<T, W, V, kHeld<V> / V, true>,
                              dim3(grid_of(a.rows, 2048 / threads)), threads, st, a);
    }
}

// Do packs of V elements of x (and of all rows), and of the weights, fit?
template <typename T, typename W, int V>
bool packs_fit(long long dim, std::initializer_list<const void *> rows,
               std::initializer_list<const void *> weights)
{
    for (const void *p : rows)
        if (p && !pack_fits(p, (size_t)dim * sizeof(T), V * sizeof(T)))
            return false;
    for (const void *p : weights)
        if (p && !aligned_to(p, std::min(V * sizeof(W), (size_t)16)))
            return false;
    return true;
}

template <typename T, typename W> rra_status forward(const Fwd &a, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    return launched(packs_fit<T, W, V>(a.dim, {a.x, a.y}, {a.gamma, a.beta})
                        ? forward_packs<T, W, V>(a, st)
                        : forward_packs<T, W, 1>(a, st));
}

// ---------------------------------------------------------------- backward

// A lane keeps its columns' sums of dgamma and dbeta over all rows of its
// group in registers.  At the end the groups of a block add theirs in shared
// memory, in order, and the block leaves one partial row of each, which
// join_kernel adds.  The packs of the next rows are on their way to shared
// memory while a row is worked on, each lane's to slots of its own, so that
// nothing but the row's two sums crosses lanes.
//
// Rows that do not begin on a 16-byte boundary are still read and written in
// whole packs, but for those at their ends: a block takes rows that all begin
// equally far behind one (every V-th row), so a lane's packs are the same
// columns in all of them.  60000 x 1001 bf16 take 99 us so and took 499 element by
// element; 3001 x 1001 fp32 15.3 and 15.8 (fp32 has 4-byte copies).
struct Bwd {
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    long long rows, dim;
    void *dx, *dgamma, *dbeta;
    int accumulate;
    float *part; // [parts][2][dim]
    int parts;
    int period; // rows between two that begin equally far behind a boundary
    Group g;
};

// Most threads of a block, one block an SM.  384 leave a thread the registers
// for 32 elements of 16 bits (64 bytes of x) and their sums: 75 us at
// 16384 x 4096 bf16, where 512 threads took 84 and 768 with half the elements
// 111 -- a row's own sums, barrier and addresses cost as much for few elements.
// Rows that 384 threads do not hold take 512.
constexpr int kBwdThreads = 384, kBwdWide = 512;
constexpr int kMostBarriers = 15; // of groups: a block has 16, __syncthreads takes one
constexpr int kBwdStages = 2; // rows in shared memory
constexpr int kBwdSums = 2 * 2 * 32; // floats of a group for its rows' sums

// Elements that a lane holds.
template <typename T, int V, int THREADS>
constexpr int kBwdHeld = V > 1 ? 64 / sizeof(T) : THREADS == kBwdThreads ? 8 : 16;

// SHIFT: rows may begin and end inside a pack.
template <typename T, typename W, int V, bool MULTI, int THREADS, bool SHIFT>
__global__ void __launch_bounds__(THREADS, 1) norm_grad_kernel(const Bwd a)
{
    constexpr int K = kBwdHeld<T, V, THREADS> / V;
    // gamma as fp32, the groups' sums, the stages; after the last row: the
    // holders' [2][width]
    extern __shared__ __align__(16) float smem[];
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    T *const dx = static_cast<T *>(a.dx);
    const W *const gamma = static_cast<const W *>(a.gamma);
    const int lanes = a.g.lanes(), li = threadIdx.x % lanes, group = threadIdx.x / lanes,
              groups = blockDim.x / lanes;
    using P = Values<V>;
    using E = typename P::E;
    const int period = SHIFT ? a.period : 1;
    const int dim = (int)a.dim, phase = blockIdx.x % period; // (a held row is short)
    // elements between the last boundary and the row, in all rows of the block
    const int shift =
        SHIFT ? (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T) + (unsigned)(phase * (dim % V))) %
                      V)
              : 0;
    const int units = SHIFT ? (dim + shift + V - 1) / V : dim / V, width = SHIFT ? units * V : dim;
    const long long step = (long long)(gridDim.x / period) * groups * period;
    const float n = (float)dim, inverse = 1.0f / n;
    float *const weights = smem, *const sums = weights + (width + 3) / 4 * 4;
    GroupOf mine = group_of(a.g, sums + group * kBwdSums, 1 + group);
    dependents_wait();
    T *const stages = reinterpret_cast<T *>(sums + (MULTI ? groups * kBwdSums : 0));
    bool in[K];   // does the lane hold a k-th pack?
    bool full[K]; // one that is all in the row?
    int col[K];   // its first place (column + shift); that of the row's last pack if not
    E dg[K][P::N], db[K][P::N];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int u = li + k * lanes;
        in[k] = u < units;
        full[k] = SHIFT ? u * V >= shift && (u + 1) * V <= shift + dim : in[k];
        col[k] = min(u, units - 1) * V;
#pragma unroll
        for (int m = 0; m < P::N; ++m)
            dg[k][m] = db[k][m] = P::all(0.0f);
    }

    // The lane's k-th pack of x is k slots behind the stage's first, that of dy
    // K slots further.  What is not in the row stays zero and adds nothing.
    constexpr int kSlot = THREADS * V, kStage = 2 * K * kSlot;
    const int apart = lanes * V;
    T *const slots = stages + threadIdx.x * V;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (!full[k])
#pragma unroll
            for (int i = 0; i < kBwdStages; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    slots[i * kStage + k * kSlot + j] = slots[i * kStage + (K + k) * kSlot + j] =
                        from_f32<T>(0.0f);
    // Of a pack at an end of the row: its elements in the row, asynchronously
    // in pieces of 4 bytes.  A piece may bring an element of the row beside, if
    // there is one, which forget() clears.
    const auto valid = [&](int place) { return place >= shift && place < shift + dim; };
    const auto stage_end = [&](T *to, const T *from, int place, bool before, bool behind) {
        constexpr int Q = sizeof(T) == 4 ? 1 : 2; // elements of a piece
#pragma unroll
        for (int j = 0; j < V; j += Q) {
            const bool p = valid(place + j), q = valid(place + j + Q - 1);
            if ((p && q) || (p && behind) || (q && before)) {
                stage_pack<T, Q>(to + j, from + j);
            } else if (Q == 2 && p) {
                to[j] = from[j];
            } else if (Q == 2 && q) {
                to[j + Q - 1] = from[j + Q - 1];
            }
        }
    };
    const auto forget = [&](T *stage) {
        if (sizeof(T) == 4)
            return;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in[k] && !full[k])
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (!valid(col[k] + j))
                        stage[k * kSlot + j] = stage[(K + k) * kSlot + j] = from_f32<T>(0.0f);
    };
    const auto stage_row = [&](T *to, long long r, const T *px, const T *pd) {
        const bool there = r < a.rows;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (there && full[k]) {
                stage_pack<T, V>(to + k * kSlot, px + k * apart);
                stage_pack<T, V>(to + (K + k) * kSlot, pd + k * apart);
            } else if (SHIFT && there && in[k]) {
                const bool before = r > 0, behind = r < a.rows - 1;
                stage_end(to + k * kSlot, px + k * apart, col[k], before, behind);
                stage_end(to + (K + k) * kSlot, pd + k * apart, col[k], before, behind);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    long long r = ((long long)(blockIdx.x / period) * groups + group) * period + phase;
    const long long row_step = step * a.dim;
    // The lane's first pack: three pointers, those of x and dy a stage ahead, or
    // one offset where a block is so wide that its threads have 128 registers
    // (16-bit rows of 16384 spill no register then: 90 us against 113 for 4096 of
    // them; narrower blocks, which spill none, take 74 us so at 16384 x 4096 and
    // 76 with an offset).
    constexpr bool kOffset = THREADS == kBwdWide;
    constexpr int kAhead = kBwdStages - 1;
    long long at = r * a.dim - shift + li * V;
    const T *px = x + at, *pd = dy + at;
    T *q = dx + at;
#pragma unroll
    for (int i = 0; i < kAhead; ++i, px += row_step, pd += row_step)
        stage_row(slots + i * kStage, r + i * step, px, pd);
    float next_mu = 0.0f, next_rs = 0.0f;
    if (r < a.rows) {
        next_mu = a.mean[r];
        next_rs = a.rstd[r];
    }
    for (int i = threadIdx.x; i < width; i += blockDim.x) {
        const int c = i - shift;
        weights[i] = c < 0 || c >= dim ? 0.0f : gamma ? to_f32(gamma[c]) : 1.0f;
    }
    if (MULTI)
        for (int i = threadIdx.x; i < groups * kBwdSums; i += blockDim.x)
            sums[i] = 0.0f;
    __syncthreads();
    int stage = 0;
    // a group of several warps has barriers of its own: it ends with its last
    // row; the groups of a warp go on together
    const long long end =
        MULTI ? a.rows : a.rows + (group - (group & -(32 / lanes))) * period;
    for (; r < end; r += step, at += row_step, px += row_step, pd += row_step, q += row_step) {
        const bool on = MULTI || r < a.rows;
        T *const now = slots + stage * kStage;
        // into the stage that the last row was in
        stage_row(slots + (stage == 0 ? kAhead : stage - 1) * kStage, r + kAhead * step,
                  kOffset ? x + at + kAhead * row_step : px,
                  kOffset ? dy + at + kAhead * row_step : pd);
        stage = stage == kBwdStages - 1 ? 0 : stage + 1;
        const E minus = P::all(-next_mu), scale = P::all(next_rs);
        const float rs = next_rs;
        if (r + step < a.rows) {
            next_mu = a.mean[r + step];
            next_rs = a.rstd[r + step];
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        if (SHIFT)
            forget(now);
        E s0 = P::all(0.0f), s1 = s0;
        if (on) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Raw<T, V> vx, vd;
                vx.load(now + k * kSlot);
                vd.load(now + (K + k) * kSlot);
                E g[P::N];
                load_weights<float, V>(weights, col[k], 1.0f, g);
#pragma unroll
                for (int m = 0; m < P::N; ++m) {
                    const E d = P::get(vd, m), xh = mul(add(P::get(vx, m), minus), scale),
                            w = mul(d, g[m]);
                    s0 = add(s0, w);
                    s1 = fma(w, xh, s1);
                    dg[k][m] = fma(d, xh, dg[k][m]);
                    db[k][m] = add(db[k][m], d);
                }
            }
        }
        if (!dx)
            continue;
        Sums<2> s{{sum_of(s0), sum_of(s1)}};
        s = group_sum<MULTI, 2>(s, mine);
        // dx = rs w - rs mean(w) - xh rs mean(w xh)
        const E m0 = P::all(-rs * quotient(s.v[0], n, inverse)),
                m1 = P::all(-rs * quotient(s.v[1], n, inverse));
        T *const to = kOffset ? dx + at : q;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Raw<T, V> vx, vd;
            vx.load(now + k * kSlot);
            vd.load(now + (K + k) * kSlot);
            E g[P::N];
            load_weights<float, V>(weights, col[k], 1.0f, g);
#pragma unroll
            for (int m = 0; m < P::N; ++m) {
                const E xh = mul(add(P::get(vx, m), minus), scale);
                const E w = mul(P::get(vd, m), g[m]);
                g[m] = fma(xh, m1, fma(w, scale, m0));
            }
            if (on && full[k]) {
                store_vals<T, V>(to + k * apart, g);
            } else if (SHIFT && on && in[k]) {
                float o[V];
                P::to_array(g, o);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (valid(col[k] + j))
                        to[k * apart + j] = from_f32<T>(o[j]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    dependents_launch();
    if (!a.dgamma && !a.dbeta)
        return;

    float *const out = a.part + 2LL * blockIdx.x * a.dim;
    float fg[K][V], fb[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        P::to_array(dg[k], fg[k]);
        P::to_array(db[k], fb[k]);
    }
    if constexpr (!MULTI) { // the warp's groups first
        for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    fg[k][j] += __shfl_xor_sync(kFull, fg[k][j], o);
                    fb[k][j] += __shfl_xor_sync(kFull, fb[k][j], o);
                }
    }
    const int holders = MULTI ? groups : blockDim.x / 32, me = MULTI ? group : threadIdx.x / 32;
    const bool holds = MULTI || threadIdx.x % 32 < lanes;
    __syncthreads(); // (gamma and the stages are done with)
    if (!SHIFT && holders == 1) { // nothing to add: 71.7 us against 73.5 at 4096 x 8192 fp32
        if (holds)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in[k]) {
                    store_values<float, V>(out + (li + k * lanes) * V, fg[k]);
                    store_values<float, V>(out + dim + (li + k * lanes) * V, fb[k]);
                }
        return;
    }
    float *const own = smem + me * 2 * width;
    if (holds)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in[k]) {
                store_values<float, V>(own + (li + k * lanes) * V, fg[k]);
                store_values<float, V>(own + width + (li + k * lanes) * V, fb[k]);
            }
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += blockDim.x) {
        float g = 0.0f, b = 0.0f;
        for (int h = 0; h < holders; ++h) {
            g += smem[h * 2 * width + shift + c];
            b += smem[(h * 2 + 1) * width + shift + c];
        }
        out[c] = g;
        out[dim + c] = b;
    }
}


// Long rows: dx by three passes over the row, the weights' sums by columns.
template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads) dx_long_kernel(const Bwd a)
{
    __shared__ __align__(16) float sm[2 * 2 * 32];
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    const W *const gamma = static_cast<const W *>(a.gamma);
    GroupOf block = group_of(Group{5, kLongThreads / 32}, sm, 1);
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float mu = a.mean[r], rs = a.rstd[r], n = (float)a.dim;
        Sums<2> s{};
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float w = to_f32(dy[r * a.dim + c]) * (gamma ? to_f32(gamma[c]) : 1.0f);
            s.v[0] += w;
            s.v[1] = fmaf(w, (to_f32(x[r * a.dim + c]) - mu) * rs, s.v[1]);
        }
        s = group_sum<true, 2>(s, block);
        const float m0 = s.v[0] / n, m1 = s.v[1] / n;
        for (long long c = threadIdx.x; c < a.dim; c += kLongThreads) {
            const float g = gamma ? to_f32(gamma[c]) : 1.0f;
            const float xh = (to_f32(x[r * a.dim + c]) - mu) * rs;
            static_cast<T *>(a.dx)[r * a.dim + c] =
                from_f32<T>(rs * (fmaf(to_f32(dy[r * a.dim + c]), g, -m0) - xh * m1));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) weight_long_kernel(const Bwd a, long long stretch)
{
    const T *const dy = static_cast<const T *>(a.dy), *const x = static_cast<const T *>(a.x);
    const long long lo = blockIdx.y * stretch, hi = min(lo + stretch, a.rows);
    for (long long c = (long long)blockIdx.x * kThreads + threadIdx.x; c < a.dim;
         c += (long long)gridDim.x * kThreads) {
        float g = 0.0f, b = 0.0f;
#pragma unroll 4
        for (long long r = lo; r < hi; ++r) {
            const float d = to_f32(dy[r * a.dim + c]);
            g = fmaf(d, (to_f32(x[r * a.dim + c]) - a.mean[r]) * a.rstd[r], g);
            b += d;
        }
        a.part[2LL * blockIdx.y * a.dim + c] = g;
        a.part[(2LL * blockIdx.y + 1) * a.dim + c] = b;
    }
}

// Launch shape of the backward pass, from which its scratch follows.
struct BwdShape {
    Group g;
    int groups; // of a block
    int parts;  // partial rows: blocks of the first kernel
    int threads; // kBwdThreads, kBwdWide, or 0: rows that no block holds
    int period;
    bool packs, shift;
};

template <typename T, typename W> BwdShape backward_shape(const Bwd &a)
{
    constexpr int V = 16 / sizeof(T);
    BwdShape s;
    // packs at the same places of x, dy and dx
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) % 16;
    s.packs = reinterpret_cast<uintptr_t>(a.dy) % 16 == at &&
              (!a.dx || reinterpret_cast<uintptr_t>(a.dx) % 16 == at);
    s.period = s.packs && a.dim % V != 0 ? V : 1;
    s.shift = s.packs && (at != 0 || s.period > 1);
    // packs that a row touches at most
    const long long units = !s.packs  ? a.dim
                            : s.shift ? (a.dim + 2 * V - 2) / V
                                      : a.dim / V;
    int held = s.packs ? kBwdHeld<T, V, kBwdThreads> / V : kBwdHeld<T, 1, kBwdThreads>;
    s.threads = kBwdThreads;
    if (units > (long long)s.threads * held) {
        held = s.packs ? kBwdHeld<T, V, kBwdWide> / V : kBwdHeld<T, 1, kBwdWide>;
        s.threads = units <= (long long)kBwdWide * held ? kBwdWide : 0;
    }
    if (s.threads) {
        s.g = group_for(units, held);
        // one block per SM; groups of a block only where rows are many
        const long long most = std::min(std::max(1, s.threads / s.g.lanes()),
                                        s.g.warps > 1 ? kMostBarriers : s.threads);
        s.groups = (int)std::max(1LL, std::min(most, a.rows / num_sms()));
        if (s.g.warps == 1) { // whole warps
            const int in_warp = 32 / s.g.lanes();
            s.groups = std::max(1, s.groups / in_warp) * in_warp;
        }
        const long long rows = (a.rows + s.period - 1) / s.period; // of a phase
        s.parts = s.period * (int)std::min((rows + s.groups - 1) / s.groups,
                                           (long long)std::max(1, num_sms() / s.period));
    } else {
        const long long stretch = std::max(16LL, (a.rows + 127) / 128);
        s.groups = 1;
        s.parts = (int)((a.rows + stretch - 1) / stretch);
    }
    return s;
}

template <typename T, typename W, int V, bool MULTI, int THREADS, bool SHIFT>
cudaError_t held_rows(const Bwd &a, const BwdShape &s, cudaStream_t st)
{
    // the slots of a whole block, whatever its size: their distance is a constant
    const size_t stages = (size_t)kBwdStages * 2 * kBwdHeld<T, V, THREADS> * sizeof(T) * THREADS,
                 sums = MULTI ? sizeof(float) * kBwdSums * s.groups : 0,
                 weights = sizeof(float) * ((a.dim + 2 * V + 3) / 4 * 4);
    // at the end: the sums of every holder (a group, or a warp of groups)
    const int holders = MULTI ? s.groups : s.groups * s.g.lanes() / 32;
    const int smem = (int)std::max(weights + sums + stages, 2 * weights * holders);
    const auto fn = norm_grad_kernel<T, W, V, MULTI, THREADS, SHIFT>;
    const cudaError_t e = op_allow(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess)
        return e;
    return launch_chained_smem(fn, dim3(s.parts), s.groups * s.g.lanes(), smem, st, a);
}

template <typename T, typename W, int V>
cudaError_t held_rows(const Bwd &a, const BwdShape &s, cudaStream_t st)
{
    if constexpr (V > 1) // rows that may be shifted
        if (s.shift) {
            if (s.threads == kBwdWide)
                return held_rows<T, W, V, true, kBwdWide, true>(a, s, st);
            return s.g.warps > 1 ? held_rows<T, W, V, true, kBwdThreads, true>(a, s, st)
                                 : held_rows<T, W, V, false, kBwdThreads, true>(a, s, st);
        }
    if (s.threads == kBwdWide)
        return held_rows<T, W, V, true, kBwdWide, false>(a, s, st);
    return s.g.warps > 1 ? held_rows<T, W, V, true, kBwdThreads, false>(a, s, st)
                         : held_rows<T, W, V, false, kBwdThreads, false>(a, s, st);
}

template <typename T, typename W> cudaError_t backward(Bwd a, const BwdShape &s, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    a.g = s.g;
    a.parts = s.parts;
    a.period = s.period;
    if (a.rows > 0) {
        if (s.threads) {
            e = s.packs ? held_rows<T, W, 16 / sizeof(T)>(a, s, st) : held_rows<T, W, 1>(a, s, st);
        } else {
            if (a.dgamma || a.dbeta) {
                const unsigned cols =
                    (unsigned)std::min((a.dim + kThreads - 1) / kThreads, 1LL << 16);
                const long long stretch = std::max(16LL, (a.rows + 127) / 128);
                weight_long_kernel<T><<<dim3(cols, s.parts), kThreads, 0, st>>>(a, stretch);
            }
            if (a.dx) // last: dx may be dy or x
                dx_long_kernel<T, W><<<grid_of(a.rows, 2), kLongThreads, 0, st>>>(a);
            e = cudaGetLastError();
        }
    }
    if (e != cudaSuccess || (!a.dgamma && !a.dbeta))
        return e;
    return join_parts<W>(Join{a.part, a.parts, a.dim, a.dgamma, a.dbeta, a.accumulate},
                         a.rows > 0, st);
}

template <typename T, typename W> rra_status backward_call(Bwd a, cudaStream_t st)
{
    const BwdShape s = backward_shape<T, W>(a);
    std::unique_lock<std::mutex> lk;
    if (a.dgamma || a.dbeta) {
        unsigned char *ws = nullptr;
        const rra_status r =
            op_scratch(st, kScratchHead + sizeof(float) * 2 * s.parts * a.dim, lk, &ws);
        if (r != RRA_OK)
            return r;
        a.part = reinterpret_cast<float *>(ws + kScratchHead);
    }
    return launched(backward<T, W>(a, s, st));
}

constexpr size_t kMostRows = (size_t)1 << 40, kMostDim = (size_t)1 << 31;

bool valid_sizes(size_t rows, size_t dim, rra_dtype t, rra_dtype w)
{
    return valid_dt(t) && valid_dt(w) && dim > 0 && dim <= kMostDim && rows <= kMostRows &&
           holdable(rows, dim, dtype_size(t));
}

} // namespace
} // namespace rra

extern "C" rra_status rra_layer_norm(const void *x, const void *gamma, const void *beta,
                                     size_t rows, size_t dim, rra_dtype dtype,
                                     rra_dtype weight_t, float eps, void *y, float *mean,
                                     float *rstd, void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t) || !(eps >= 0.0f))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es;
    if (rows > 0 && (!x || !y || !aligned_to(x, es) || !aligned_to(y, es)))
        return RRA_ERR_INVALID;
    if (!aligned_to(gamma, ws) || !aligned_to(beta, ws) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4) || !apart_or_same(x, bytes, y, bytes) ||
        overlap(y, bytes, gamma, dim * ws) || overlap(y, bytes, beta, dim * ws) ||
        overlap(y, bytes, mean, rows * 4) || overlap(y, bytes, rstd, rows * 4) ||
        overlap(x, bytes, mean, rows * 4) || overlap(x, bytes, rstd, rows * 4) ||
        overlap(mean, rows * 4, rstd, rows * 4))
        return RRA_ERR_INVALID;
    for (const float *out : {mean, rstd})
        if (overlap(out, rows * 4, gamma, dim * ws) || overlap(out, rows * 4, beta, dim * ws))
            return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    if (rows == 0)
        return RRA_OK;
    const Fwd a{x, gamma, beta, (long long)rows, (long long)dim, eps, y, mean, rstd, {}};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == RRA_F32)
        return forward<float, float>(a, st);
    if (dtype == RRA_F16 && weight_t == RRA_F16)
        return forward<__half, __half>(a, st);
    if (dtype == RRA_F16)
        return forward<__half, float>(a, st);
    if (weight_t == RRA_BF16)
        return forward<__nv_bfloat16, __nv_bfloat16>(a, st);
    return forward<__nv_bfloat16, float>(a, st);
}

extern "C" rra_status rra_layer_norm_grad(const void *dy, const void *x, const void *gamma,
                                          const float *mean, const float *rstd, size_t rows,
                                          size_t dim, rra_dtype dtype, rra_dtype weight_t,
                                          void *dx, void *dgamma, void *dbeta, int accumulate,
                                          void *stream)
{
    using namespace rra;
    if (!valid_sizes(rows, dim, dtype, weight_t) || (!dx && !dgamma && !dbeta))
        return RRA_ERR_INVALID;
    const size_t es = dtype_size(dtype), ws = dtype_size(weight_t), bytes = rows * dim * es,
                 wb = dim * ws;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !aligned_to(dy, es) || !aligned_to(x, es)))
        return RRA_ERR_INVALID;
    if (!aligned_to(gamma, ws) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(dx, es) || !aligned_to(dgamma, ws) || !aligned_to(dbeta, ws))
        return RRA_ERR_INVALID;
    if (!apart_or_same(dx, bytes, dy, bytes) || !apart_or_same(dx, bytes, x, bytes) ||
        overlap(dgamma, wb, dbeta, wb))
        return RRA_ERR_INVALID;
    for (void *out : {dgamma, dbeta})
        if (overlap(out, wb, dy, bytes) || overlap(out, wb, x, bytes) ||
            overlap(out, wb, gamma, wb) || overlap(out, wb, mean, rows * 4) ||
            overlap(out, wb, rstd, rows * 4) || overlap(out, wb, dx, bytes))
            return RRA_ERR_INVALID;
    if (overlap(dx, bytes, gamma, wb) || overlap(dx, bytes, mean, rows * 4) ||
        overlap(dx, bytes, rstd, rows * 4))
        return RRA_ERR_INVALID;
    if (weight_t != dtype && weight_t != RRA_F32)
        return RRA_ERR_UNSUPPORTED;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const Bwd a{dy, x,  gamma,  mean,  rstd,       (long long)rows, (long long)dim,
                dx, dgamma, dbeta, accumulate, nullptr,         0,
                1,  {}};
    if (dtype == RRA_F32)
        return backward_call<float, float>(a, st);
    if (dtype == RRA_F16 && weight_t == RRA_F16)
        return backward_call<__half, __half>(a, st);
    if (dtype == RRA_F16)
        return backward_call<__half, float>(a, st);
    if (weight_t == RRA_BF16)
        return backward_call<__nv_bfloat16, __nv_bfloat16>(a, st);
    return backward_call<__nv_bfloat16, float>(a, st);
}
