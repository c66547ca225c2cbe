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

// Words from byte q (0..16, a multiple of 2) of `in` on.  (A warp with one row has one q,
// and goes one of the five ways: an instruction a word, where selects took three.)
template <int N_IN, int N_OUT>
__device__ __forceinline__ void shift_bytes(const uint32_t (&in)[N_IN], int q, uint32_t (&out)[N_OUT])
{
    static_assert(N_IN == N_OUT + 4, "16 bytes more");
    const uint32_t bits = 8 * (q & 3);
    const auto words = [&](auto from) {
        constexpr int S = decltype(from)::value;
#pragma unroll
        for (int i = 0; i < N_OUT; ++i)
            out[i] = S == 4 ? in[i + 4] : __funnelshift_r(in[i + S], in[i + S + 1], bits);
    };
    switch (q >> 2) {
    case 0:
        words(std::integral_constant<int, 0>());
        break;
    case 1:
        words(std::integral_constant<int, 1>());
        break;
    case 2:
        words(std::integral_constant<int, 2>());
        break;
    case 3:
        words(std::integral_constant<int, 3>());
        break;
    default:
        words(std::integral_constant<int, 4>());
    }
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

// Words of a pack with zeros behind its first n elements.
template <typename T> __device__ __forceinline__ void keep_first(uint32_t (&w)[kPackWords<T>], int n)
{
#pragma unroll
    for (int i = 0; i < kPackWords<T>; ++i) {
        if constexpr (sizeof(T) == 4)
            w[i] = i < n ? w[i] : 0u;
        else
            w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0u;
    }
}

// Are all chunks that packs of a row of dim elements touch in [begin, end)?
template <typename T>
__device__ __forceinline__ bool row_inside(const T *row, long long dim, const T *begin, const T *end)
{
    return row - 16 / (int)sizeof(T) >= begin && row + dim + 8 + 16 / (int)sizeof(T) <= end;
}

// Words of the chunks that a pack touches (WHOLE: of the pack).
template <typename T, bool WHOLE> constexpr int kChunkWords = kPackWords<T> + (WHOLE ? 0 : 4);

// The chunks of the n (1..8) elements at p, still where they are in memory, so that
// nothing waits for them; settle() has the elements.  WHOLE: n is 8 and p on a 16-byte
// boundary.  [begin, end): the array; nothing outside of it is read.  inside: is it known
// that the chunks are?
template <typename T, bool WHOLE>
__device__ __forceinline__ void load_chunks(const T *p, int n, const T *begin, const T *end,
                                            uint32_t (&raw)[kChunkWords<T, WHOLE>],
                                            bool inside = false)
{
    constexpr int N = kPackWords<T>;
    const int m = WHOLE ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4 *const c = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - m);
    if (WHOLE || inside || (reinterpret_cast<const T *>(c) >= begin &&
                            reinterpret_cast<const T *>(c + N / 4 + 1) <= end)) {
#pragma unroll
        for (int i = 0; i < kChunkWords<T, WHOLE>; i += 4) {
            const uint4 q = c[i / 4];
            raw[i] = q.x, raw[i + 1] = q.y, raw[i + 2] = q.z, raw[i + 3] = q.w;
        }
        return;
    }
    if constexpr (!WHOLE) { // an end of the array: as many elements, at the same place
        uint32_t w[N + 8] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if constexpr (sizeof(T) == 4)
                    w[4 + j] = reinterpret_cast<const uint32_t *>(p)[j];
                else
                    w[4 + j / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[j]
                                    << (16 * (j % 2));
            }
        shift_bytes(w, 16 - m, raw);
    }
}

// The elements of load_chunks(p, n, ...), zeros behind them.
template <typename T, bool WHOLE>
__device__ __forceinline__ void settle(const uint32_t (&raw)[kChunkWords<T, WHOLE>], const T *p, int n,
                                       uint32_t (&w)[kPackWords<T>])
{
    if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < kPackWords<T>; ++i)
            w[i] = raw[i];
    } else {
        shift_bytes(raw, (int)(reinterpret_cast<uintptr_t>(p) & 15), w);
        if (n < 8)
            keep_first<T>(w, n);
    }
}

// Both, of n (0..8) elements (WHOLE: 0 or 8).
template <typename T, bool WHOLE>
__device__ __forceinline__ void load_words(const T *p, int n, const T *begin, const T *end,
                                           uint32_t (&w)[kPackWords<T>])
{
#pragma unroll
    for (int i = 0; i < kPackWords<T>; ++i)
        w[i] = 0;
    if (n == 0)
        return;
    uint32_t raw[kChunkWords<T, WHOLE>];
    load_chunks<T, WHOLE>(p, n, begin, end, raw);
    settle<T, WHOLE>(raw, p, n, w);
}

// The first r bytes (even, below 16) of a chunk, or those from byte m (even, above 0) on.
__device__ __forceinline__ void put_begin(unsigned char *c, int r, uint32_t a, uint32_t b, uint32_t x,
                                          uint32_t y)
{
    if (r & 8)
        *reinterpret_cast<uint2 *>(c) = make_uint2(a, b);
    if (r & 4)
        *reinterpret_cast<uint32_t *>(c + (r & 8)) = r & 8 ? x : a;
    if (r & 2)
        *reinterpret_cast<uint16_t *>(c + (r & 12)) =
            (uint16_t)(r & 8 ? (r & 4 ? y : x) : (r & 4 ? b : a));
}
__device__ __forceinline__ void put_end(unsigned char *c, int m, uint32_t a, uint32_t b, uint32_t x,
                                        uint32_t y)
{
    if (m & 2)
        *reinterpret_cast<uint16_t *>(c + m) =
            (uint16_t)((m & 8 ? (m & 4 ? y : x) : (m & 4 ? b : a)) >> 16);
    const int q = (m + 2) & ~3; // whole words from here on
    if (q & 4)
        *reinterpret_cast<uint32_t *>(c + q) = q & 8 ? y : b;
    if (q <= 8)
        *reinterpret_cast<uint2 *>(c + 8) = make_uint2(x, y);
}

// What a lane's last bytes of its pack before are, for the next store_words.
template <typename T, int E = 8> struct Carry {
    uint32_t w[4] = {};
};

// Writes the n (0..E) elements at p.  A stretch of `lanes` (a power of two, at most a
// warp) lanes holds neighbouring packs of one row, and the stretch of the lanes' next
// packs may follow it: `next`: how many elements the pack behind this one has; joined:
// does this stretch follow the one that `carry` is of?  last: does none follow it?  All
// lanes of the warp are here.  on: is the lane's row written at all?
// A chunk with the ends of two packs is the second one's to write.
template <typename T, bool WHOLE, int E = 8>
__device__ __forceinline__ void store_words(T *p, int n, int next, bool on, int lanes,
                                            const uint32_t (&w)[kPackWords<T, E>], Carry<T, E> &carry,
                                            bool joined = false, bool last = true)
{
    constexpr int N = kPackWords<T, E>;
    if constexpr (WHOLE) {
        if (on && n == E)
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(p) + i) =
                    make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
        const int m = (int)(reinterpret_cast<uintptr_t>(p) & 15), place = threadIdx.x % lanes;
        // the lane before; before the first one the last of the stretch before
        const int before = threadIdx.x % 32 - place + (place + lanes - 1) % lanes;
        uint32_t in[N + 4], out[N];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t mine = w[N - 4 + i];
            in[i] = __shfl_sync(kFull, place == lanes - 1 ? carry.w[i] : mine, before);
            carry.w[i] = mine;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            in[4 + i] = w[i];
        shift_bytes(in, 16 - m, out);
        if (!on || n == 0)
            return;
        unsigned char *const c = reinterpret_cast<unsigned char *>(p) - m;
        const int bytes = m + n * (int)sizeof(T); // from the first chunk's begin on
        const bool first = !joined && place == 0 && m > 0; // its first bytes are not this lane's
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            if (16 * (i + 1) <= bytes && !(i == 0 && first))
                *reinterpret_cast<uint4 *>(c + 16 * i) =
                    make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
        if (first) {
            if (bytes < 16) { // a row, or its rest, inside of a chunk
#pragma unroll
                for (int j = 0; j < 16 / (int)sizeof(T); ++j)
                    if (j < n) {
                        if constexpr (sizeof(T) == 4)
                            reinterpret_cast<uint32_t *>(p)[j] = w[j];
                        else
                            reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
                    }
                return;
            }
            put_end(c, m, out[0], out[1], out[2], out[3]);
        }
        const int rest = bytes & 15;
        if (rest > 0 && (next == 0 || (last && place == lanes - 1))) {
            // the chunk that the row or the stretch ends in: one of `out`, or the pack's own
            // last bytes alone
            const uint32_t own[8] = {w[N - 4], w[N - 3], w[N - 2], w[N - 1], 0u, 0u, 0u, 0u};
            uint32_t t[4];
            shift_bytes(own, 16 - m, t);
            const int at = bytes / 16;
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    t[j] = at == i ? out[4 * i + j] : t[j];
            put_begin(c + 16 * at, rest, t[0], t[1], t[2], t[3]);
        }
    }
}

} // namespace rra
