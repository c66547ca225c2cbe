// saved.cuh -- activations held in 8 bits between the two passes of a step.
//
// A row of D elements is cut into blocks of 128; a block has one exponent
// e = floor(log2 max|v|) (-126 for a zero or subnormal maximum) and a code
// m = clamp(rne(v 2^(6-e)), +-127) for each element, which stands for
// m 2^(e-6): the block floating point of rra_bfp_encode, with every row's
// blocks its own.  Codes lie in rows of whole blocks (zeros behind D), so a
// pack of 8 is one 8-byte access in every row whatever D is.
// A block with an infinity or NaN has the exponent byte -128 and codes 0: its
// scale 2^e comes out as infinity, and 0 times that is NaN.
//
// Everywhere a lane holds packs of 8 elements and 16 neighbouring lanes a
// block.
#pragma once

#include "bfp_group.cuh"
#include "op_common.cuh"

namespace rra {

constexpr int kPack = 8;                     // elements
constexpr int kBlockPacks = kBlock / kPack;  // packs that share an exponent

__host__ __device__ inline long long blocks_of(long long dim) { return (dim + kBlock - 1) / kBlock; }

struct Codes8 {
    uint32_t w[2];
};

// Biased exponent of a block from the bits of its largest magnitude (an
// infinity or NaN: 255), and the byte that is stored.
__device__ __forceinline__ int block_exponent(uint32_t top_bits)
{
    return max((int)(top_bits >> 23), 1);
}
__device__ __forceinline__ int8_t exponent_byte(int E) { return (int8_t)(E - 127); }

// Codes of 8 values in a block whose largest magnitude has these bits (two's
// complement).  As in BfpGroup: t = fma(v, 2^(6-e), 1.5 2^23 + 128) holds m + 128 in
// its low byte.
__device__ __forceinline__ Codes8 encode8(const float v[8], uint32_t top)
{
    constexpr float kEnc = kMagic + 128.0f;
    const int E = block_exponent(top);
    if (E == 255)
        return {{0u, 0u}};
    // 2^(6-e), a normal float unless E < 6: such blocks are first scaled by 2^64
    const float s = __int_as_float((E < 6 ? 196 - E : 260 - E) << 23);
    const float2 s2 = make_float2(s, s), c2 = make_float2(kEnc, kEnc);
    float2 t[4];
    if (E < 6) {
        const float2 up = make_float2(1.8446744073709552e19f, 1.8446744073709552e19f);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            t[j] = __ffma2_rn(__fmul2_rn(make_float2(v[2 * j], v[2 * j + 1]), up), s2, c2);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            t[j] = __ffma2_rn(make_float2(v[2 * j], v[2 * j + 1]), s2, c2);
    }
    // m is at most 128, and above 127 only where the block's largest value is 127.5
    // of 128 or more (a subnormal one, which is none, may look like it)
    if ((top & 0x7fffffu) >= 0x7f0000u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            t[j].x = fminf(fmaxf(t[j].x, kEnc - 127.0f), kEnc + 127.0f);
            t[j].y = fminf(fmaxf(t[j].y, kEnc - 127.0f), kEnc + 127.0f);
        }
    }
    Codes8 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 a = t[2 * h], b = t[2 * h + 1];
        c.w[h] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                             __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040),
                             0x5410) ^
                 0x80808080u;
    }
    return c;
}

// Is a block with this largest magnitude one that plain_codes8 cannot take: not finite,
// subnormal or nearly so, or with a value that rounds past 127?
__device__ __forceinline__ bool special_block(uint32_t top)
{
    return (top & 0x7fffffu) >= 0x7f0000u || top - (6u << 23) >= (249u << 23);
}

// encode8 of any other block.
__device__ __forceinline__ Codes8 plain_codes8(const float v[8], uint32_t top)
{
    constexpr float kEnc = kMagic + 128.0f;
    const float s = __uint_as_float((260u << 23) - (top & 0x7f800000u));
    float2 t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        t[j] = __ffma2_rn(make_float2(v[2 * j], v[2 * j + 1]), make_float2(s, s),
                          make_float2(kEnc, kEnc));
    Codes8 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 a = t[2 * h], b = t[2 * h + 1];
        c.w[h] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                             __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040),
                             0x5410) ^
                 0x80808080u;
    }
    return c;
}

// 2^e of a block's exponent byte (an infinity for a block that is not finite).
__device__ __forceinline__ float block_scale(int8_t e)
{
    return __uint_as_float(((uint32_t)(e + 127) & 255u) << 23);
}

// m / 64 of 8 codes, exactly; a value is that times the block's scale.
__device__ __forceinline__ void fractions8(const Codes8 &c, float2 f[4])
{
    constexpr float kOff = -(kMagic + 128.0f) / 64.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = c.w[h] ^ 0x80808080u; // m + 128
#pragma unroll
        for (int j = 0; j < 2; ++j)
            f[2 * h + j] = __ffma2_rn(
                make_float2(__uint_as_float(__byte_perm(x, kMagicBits, 0x7640 + 2 * j)),
                            __uint_as_float(__byte_perm(x, kMagicBits, 0x7641 + 2 * j))),
                make_float2(1.0f / 64, 1.0f / 64), make_float2(kOff, kOff));
    }
}

// The 8 values of codes whose block's exponent byte is e.
__device__ __forceinline__ void decode8(const Codes8 &c, int8_t e, float v[8])
{
    float2 f[4];
    fractions8(c, f);
    const float s = block_scale(e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 r = __fmul2_rn(f[j], make_float2(s, s));
        v[2 * j] = r.x;
        v[2 * j + 1] = r.y;
    }
}

__device__ __forceinline__ Codes8 load_codes(const int8_t *p)
{
    const Pack<uint32_t, 2> q = load_pack<uint32_t, 2>(reinterpret_cast<const uint32_t *>(p));
    return {{q.e[0], q.e[1]}};
}
__device__ __forceinline__ void store_codes(int8_t *p, const Codes8 &c)
{
    Pack<uint32_t, 2> q;
    q.e[0] = c.w[0];
    q.e[1] = c.w[1];
    store_pack<uint32_t, 2>(reinterpret_cast<uint32_t *>(p), q);
}

// Largest magnitude's bits over each half of a warp; every lane takes part.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t bits)
{
    const bool low = threadIdx.x % 32 < 16;
    const uint32_t a = __reduce_max_sync(kFull, low ? bits : 0u);
    const uint32_t b = __reduce_max_sync(kFull, low ? 0u : bits);
    return low ? a : b;
}

// Bits of the largest magnitude of 8 values: infinities and NaN are above all
// finite ones.
__device__ __forceinline__ uint32_t top_bits(const float v[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return m;
}

// n (0..8) elements at p, as fp32, zeros behind them; VEC: n is 0 or 8 and p a
// multiple of 16 bytes.
template <typename T, bool VEC> __device__ __forceinline__ void load8(const T *p, int n, float v[8])
{
    if (VEC) {
        T t[8];
        if (n == 8) {
            load_values<T, 8>(p, t);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = to_f32(t[j]);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = !VEC && j < n ? to_f32(p[j]) : 0.0f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int n, const float v[8])
{
    if (VEC) {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t[j] = from_f32<T>(v[j]);
        if (n == 8)
            store_values<T, 8>(p, t);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                p[j] = from_f32<T>(v[j]);
    }
}

// Exponents and codes of an activation of `rows` rows.
inline size_t exps_bytes(size_t rows, size_t dim) { return rows * (size_t)blocks_of(dim); }
inline size_t codes_bytes(size_t rows, size_t dim) { return rows * (size_t)blocks_of(dim) * kBlock; }

} // namespace rra
