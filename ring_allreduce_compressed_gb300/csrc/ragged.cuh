// ragged.cuh -- packs of 8 elements of rows that begin anywhere: read and written in
// whole 16-byte chunks all the same.
//
// A row that begins m bytes behind a 16-byte boundary has every pack m bytes behind
// one.  A lane reads the chunks that its pack touches and shifts the bytes into
// place.  To write, it takes the last 16 bytes of the lane before it, so that the
// bytes of its own pack and that lane's last m fill whole chunks; only the ends of a
// stretch of lanes are written element by element.
#pragma once

#include "op_common.cuh"

namespace rra {

// Words from byte q (0..16, a multiple of 2) of `in` on.
template <int N_IN, int N_OUT>
__device__ __forceinline__ void shift_bytes(const uint32_t (&in)[N_IN], int q, uint32_t (&out)[N_OUT])
{
    static_assert(N_IN == N_OUT + 4, "16 bytes more");
    uint32_t t[N_IN];
#pragma unroll
    for (int i = 0; i < N_IN; ++i)
        t[i] = q & 2 ? __byte_perm(in[i], i + 1 < N_IN ? in[i + 1] : 0u, 0x5432) : in[i];
#pragma unroll
    for (int i = 0; i + 1 < N_IN; ++i)
        t[i] = q & 4 ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i + 2 < N_IN; ++i)
        t[i] = q & 8 ? t[i + 2] : t[i];
#pragma unroll
    for (int i = 0; i < N_OUT; ++i)
        out[i] = q & 16 ? t[i + 4] : t[i];
}

// Words of a pack of 8 elements, or of 16.
template <typename T, int E = 8> constexpr int kPackWords = E * sizeof(T) / 4;

template <typename T> __device__ __forceinline__ float element(const uint32_t *w, int j)
{
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(w[j]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    else
        return __half2float(__ushort_as_half((unsigned short)(w[j / 2] >> (16 * (j % 2)))));
}

template <typename T>
__device__ __forceinline__ void to_words(const float *v, uint32_t (&w)[kPackWords<T>])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = __float_as_uint(v[j]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
}

// The n (0..8) elements at p, zeros behind them; WHOLE: n is 0 or 8 and p on a
// 16-byte boundary.  [begin, end): the array; nothing outside of it is read.
template <typename T, bool WHOLE>
__device__ __forceinline__ void load_words(const T *p, int n, const T *begin, const T *end,
                                           uint32_t (&w)[kPackWords<T>])
{
    constexpr int N = kPackWords<T>;
#pragma unroll
    for (int i = 0; i < N; ++i)
        w[i] = 0;
    if (n == 0)
        return;
    if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 q = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p) + i);
            w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
        }
    } else {
        const int m = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        const uint4 *const c = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - m);
        if (n == 8 && reinterpret_cast<const T *>(c) >= begin &&
            reinterpret_cast<const T *>(c + N / 4 + 1) <= end) {
            uint32_t in[N + 4];
#pragma unroll
            for (int i = 0; i < N + 4; i += 4) {
                const uint4 q = c[i / 4];
                in[i] = q.x, in[i + 1] = q.y, in[i + 2] = q.z, in[i + 3] = q.w;
            }
            shift_bytes(in, m, w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) {
                    if constexpr (sizeof(T) == 4)
                        w[j] = reinterpret_cast<const uint32_t *>(p)[j];
                    else
                        w[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[j]
                                    << (16 * (j % 2));
                }
        }
    }
}

// Writes the n (0..E) elements at p; `next`: how many the next lane's pack has.  A
// stretch of `lanes` (a power of two, at most a warp) lanes holds neighbouring packs
// of one row; all lanes of the warp are here.  on: is the lane's row written at all?
template <typename T, bool WHOLE, int E = 8>
__device__ __forceinline__ void store_words(T *p, int n, int next, bool on, int lanes,
                                            const uint32_t (&w)[kPackWords<T, E>])
{
    constexpr int N = kPackWords<T, E>;
    if constexpr (WHOLE) {
        if (on && n == E)
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(p) + i) =
                    make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
        const int m = (int)(reinterpret_cast<uintptr_t>(p) & 15), s = m / (int)sizeof(T);
        const int place = threadIdx.x % lanes;
        uint32_t in[N + 4], out[N];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            in[i] = __shfl_up_sync(kFull, w[N - 4 + i], 1);
#pragma unroll
        for (int i = 0; i < N; ++i)
            in[4 + i] = w[i];
        shift_bytes(in, 16 - m, out);
        if (!on || n == 0)
            return;
        // chunk i holds elements [16 i / sizeof(T) - s, ...) of the pack
        constexpr int C = 16 / sizeof(T); // elements of a chunk
        unsigned char *const c = reinterpret_cast<unsigned char *>(p) - m;
        const auto one = [&](int j) {
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(p)[j] = w[j];
            else
                reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
        };
        int done = 0;              // elements from the first on that are written
        if (m > 0 && place == 0) { // the chunk's first elements are not this lane's
            done = min(n, C - s);
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (j < done)
                    one(j);
        }
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const int last = (i + 1) * C - s; // elements up to the chunk's end
            if (done < last && n >= last) {
                *reinterpret_cast<uint4 *>(c + 16 * i) =
                    make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                done = last;
            }
        }
        // the rest is the next lane's, which begins with it
        if (m > 0 && n == E && done == E - s && place != lanes - 1 && next >= C - s)
            return;
        // (a chunk that the row ends in has elements of the lane before: it wrote them)
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (j >= done && j < n)
                one(j);
    }
}

} // namespace rra
