// held.h -- rows of a cache that are held as codes of 8 bits: value = code *
// scale, one fp32 scale for each block of positions and head.
//
// Codes are exact in bf16 and fp32 (e4m3 has 4 significant bits, an integer 8),
// so the matrix instructions take them as they are.  The scales, which differ from
// key to key, are applied in fp32 to the scores and to the softmax weights, or, where
// they are powers of two, in the widening, which stays exact.
#pragma once

#include "exact.h"
#include "tile.h"

namespace sdl {

struct E4M3 { uint8_t code; };      // sign, 4 bits of exponent, 3 of fraction; no infinity; 0x7f, 0xff: NaN
struct Int8 { int8_t code; };

template <class H> inline constexpr bool kCodes = false;
template <> inline constexpr bool kCodes<E4M3> = true;
template <> inline constexpr bool kCodes<Int8> = true;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Values of the four codes in w.
template <class H>
__device__ inline f32x4 wide(uint32_t w)
{
    if constexpr (std::is_same_v<H, E4M3>) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        return f32x4{a[0], a[1], b[0], b[1]};
    } else {
        return f32x4{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)};
    }
}

template <class H>
__device__ inline bf16x4 wide_bf16(uint32_t w)
{
    if constexpr (std::is_same_v<H, E4M3>) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3);
    } else {
        // 8 bits lie in the upper half of a fp32
        const f32x4 x = wide<H>(w);
        const uint32_t a = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302);
        const uint32_t b = __builtin_amdgcn_perm(__float_as_uint(x[3]), __float_as_uint(x[2]), 0x07060302);
        return __builtin_bit_cast(bf16x4, (uint64_t)b << 32 | a);
    }
}

// The same times a scale that is a power of two (or 0, for codes that are 0).
template <class H>
__device__ inline bf16x4 wide_scaled(uint32_t w, float scale)
{
    if constexpr (std::is_same_v<H, E4M3>) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3);
    } else {
        const f32x4 x = wide<H>(w) * scale;
        const uint32_t a = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302);
        const uint32_t b = __builtin_amdgcn_perm(__float_as_uint(x[3]), __float_as_uint(x[2]), 0x07060302);
        return __builtin_bit_cast(bf16x4, (uint64_t)b << 32 | a);
    }
}

// Largest value of a code, and the codes of four values that are divided by
// their scale already (no larger than that, or no number), to nearest even.
template <class H> inline constexpr float kMost = std::is_same_v<H, E4M3> ? 448.0f : 127.0f;

template <class H>
__device__ inline uint32_t narrow(f32x4 x)
{
    if constexpr (std::is_same_v<H, E4M3>) {
        const int low = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
        return __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], low, true);
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w |= ((uint32_t)(int)__builtin_rintf(x[e]) & 0xff) << (8 * e);     // NaN: 0
        return w;
    }
}

// Code number e of w next nearer to zero.
template <class H>
__device__ inline uint32_t smaller(uint32_t w, int e, bool negative)
{
    const uint32_t code = w >> (8 * e) & 0xff;
    const uint32_t to = std::is_same_v<H, Int8> && negative ? code + 1 : code - 1;
    return (w & ~(0xffu << (8 * e))) | (to & 0xff) << (8 * e);
}

// The smallest power of two s >= 2^-126 with top <= kMost s, for a finite top >= 0.
template <class H>
__device__ inline float scale_of_top(float top)
{
    // kMost is 1.75 * 2^8 or 1.984375 * 2^6
    constexpr uint32_t most = std::is_same_v<H, E4M3> ? 0x43e00000 : 0x42fe0000;
    const uint32_t bits = __float_as_uint(top);
    const int e = (int)(bits >> 23) - (int)(most >> 23) + ((bits & 0x7fffff) > (most & 0x7fffff) ? 1 : 0);
    return __uint_as_float((uint32_t)(e > -126 ? e + 127 : 1) << 23);
}

// Division by a scale, rounded once: a product where the scale is a power of
// two, which it is unless another program wrote it.
struct Divide {
    float by, inverse;
    bool power;
    __device__ explicit Divide(float scale) : by(scale)
    {
        const uint32_t bits = __float_as_uint(scale), e = bits >> 23;
        power = (bits & 0x7fffff) == 0 && e >= 1 && e <= 253;
        inverse = __uint_as_float((254 - e) << 23);
    }
    __device__ f32x4 operator()(f32x4 x) const
    {
        if (power)
            return f32x4{x[0] * inverse, x[1] * inverse, x[2] * inverse, x[3] * inverse};
        return f32x4{x[0] / by, x[1] / by, x[2] / by, x[3] / by};
    }
    // Codes of four values.  Next to the end of fp32's range rounding up may lead to a
    // code that times its scale is infinite (from 248 * 2^120 on 256 * 2^120): then the
    // next smaller one, so that what is finite is read as finite.
    template <class H>
    __device__ uint32_t codes(f32x4 x) const
    {
        const f32x4 q = (*this)(x);
        uint32_t w = narrow<H>(q);
        if (by >= 0x1p119f) {                  // below, 448 times the scale is finite
#pragma unroll
            for (int step = 0; step < 2; ++step) {     // (twice: quotients by other scales are rounded)
                const f32x4 code = wide<H>(w);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (finite(q[e]) && !finite(code[e] * by))
                        w = smaller<H>(w, e, code[e] < 0.0f);
            }
        }
        return w;
    }
};

// The larger scale; NaN if either is.
__device__ inline float larger_scale(float a, float b) { return a != a || a >= b ? a : b; }

// A row of codes as a row of values, for exact.h.
template <class H>
struct CodeRow {
    const H *at;
    float scale;
    __device__ CodeRow operator+(int d) const { return {at + d, scale}; }
    __device__ float operator[](int d) const { return wide<H>(*(const uint8_t *)(at + d))[0] * scale; }
};

template <bool ONE, class H>
__device__ inline CodeRow<H> row_of_lane(CodeRow<H> r, int n)
{
    const int scale = __float_as_int(r.scale);
    return {row_of_lane<ONE>(r.at, n), __int_as_float(ONE ? of_one_lane(scale, n) : of_lane(scale, n))};
}

template <class H>
__device__ inline f32x8 load8(CodeRow<H> r)
{
    const uint32_t *w = (const uint32_t *)r.at;
    const f32x4 a = wide<H>(w[0]) * r.scale, b = wide<H>(w[1]) * r.scale;
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A score's sum goes over the codes, as it does in the tiles.
template <class A, class H>
__device__ inline float dot_row(A a, CodeRow<H> b, int D)
{
    const float scale = b.scale;
    b.scale = 1.0f;
    float s = 0.0f;
    for (int d = 0; d < D; d += 8) {
        const auto x = load8(a + d);
        const auto y = load8(b + d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s = fmaf((float)x[e], y[e], s);
    }
    return s * scale;
}

// Scores or weights of a result's rows times the scales of their keys, four
// consecutive ones to a group of registers and eight apart; `scale`: of the
// lane's first.
template <int COUNT, class Acc>
__device__ inline void times_scales(Acc &x, const float *scale)
{
#pragma unroll
    for (int g = 0; g < COUNT / 4; ++g) {
        const f32x4 s = *(const f32x4 *)(scale + 8 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[4 * g + e] *= s[e];
    }
}

}  // namespace sdl
