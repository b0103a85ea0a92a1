// kv_pool8.hpp -- the 8-bit pool: e4m3 bytes, one scale for each block of
// tokens and head.
//
// A block is what one head has in one page, of K or of V: page_size rows of
// dim bytes.  Its scale is a power of two, s = 2^e with e the least integer
// for which every finite value x of the block has |x| <= 448 s, kept within
// 2^-100 .. 2^119 (the values then stay normal float32 and bf16 numbers, and
// 448 s is one); a byte is e4m3(x / s), ties to even, and stands for byte * s.
// What is not finite is held as NaN and has no part in the scale.
//
// A power of two costs at most one bit at the lower end of e4m3's 2^18 range,
// and buys three things: byte * s is exact in bf16, which is what the matrix
// cores take; it is formed by the conversion instruction itself; and a block
// that a later token outgrows is held anew by moving the bytes' exponents, which
// is exact but for what falls below 2^-6 s.  (With amax / 448 as the scale every
// such step rounds every byte again, and a 16-token page grows 2.4 times on
// average while it is filled token by token.)
#pragma once

#include "kv_step.hpp"

namespace kvmove {

constexpr int kLeastExponent = -100, kMostExponent = 119;
constexpr float kE4m3Max = 448.0f;

using gu32 = __attribute__((address_space(1))) uint32_t;

struct ScalesArg {
    uint64_t k_scales;       // uint64[L]: addresses of float32 [num_pages][heads]
    uint64_t v_scales;
};

// Addresses of a layer of either pool; the scales are 0 in a bf16 one.
struct LayerAt {
    uint64_t k, v, k_scales, v_scales;
};

__device__ __forceinline__ bool bad_scales(uint64_t p) { return p == 0 || (p & 3u) != 0; }

template <bool kByte>
__device__ __forceinline__ LayerAt layer_at(const PoolArg& p, const ScalesArg& s)
{
    LayerAt l{};
    l.k = wave_uniform(gptr<const gu64>(p.k_pages)[p.layer]);
    l.v = wave_uniform(gptr<const gu64>(p.v_pages)[p.layer]);
    if constexpr (kByte) {
        l.k_scales = wave_uniform(gptr<const gu64>(s.k_scales)[p.layer]);
        l.v_scales = wave_uniform(gptr<const gu64>(s.v_scales)[p.layer]);
    }
    return l;
}

template <bool kByte>
__device__ __forceinline__ bool bad_layer(const LayerAt& l)
{
    return bad_addr(l.k) || bad_addr(l.v) || (kByte && (bad_scales(l.k_scales) || bad_scales(l.v_scales)));
}

// Four e4m3 bytes times a scale as four bf16, exactly: the instruction takes
// the scale's exponent and nothing else of it.
__device__ __forceinline__ u32x2 bf16_of_bytes(uint32_t bytes, float scale)
{
    using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, scale, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, scale, true);
    return {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

__device__ __forceinline__ u32x4 bf16_of_bytes8(uint32_t b0, uint32_t b1, float scale)
{
    const u32x2 x = bf16_of_bytes(b0, scale), y = bf16_of_bytes(b1, scale);
    return {x[0], x[1], y[0], y[1]};
}

// e with 2^e the scale that a largest magnitude asks for: 448 = 1.75 * 2^8, so
// amax = m * 2^x (1 <= m < 2) needs 2^(x - 8) if m <= 1.75, else 2^(x - 7).
// Subnormal and zero amax are below the least scale either way.
__device__ __forceinline__ int scale_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    return clamp_i32(int32_t(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), kLeastExponent,
                     kMostExponent);
}

// Exponent of a scale that was stored; whatever is read, within the limits.
__device__ __forceinline__ int stored_exponent(float scale)
{
    return clamp_i32(int32_t((__float_as_uint(scale) >> 23) & 0xFFu) - 127, kLeastExponent, kMostExponent);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Magnitude of what counts for a scale: 0 where x is not finite.
__device__ __forceinline__ float finite_magnitude(float x)
{
    const float a = __builtin_fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}

// x times 1 / s as an e4m3 byte would hold it, before its rounding: saturated, NaN for what is not finite.
__device__ __forceinline__ float for_byte(float x, float inv)
{
    const float y = __builtin_fminf(__builtin_fmaxf(x * inv, -kE4m3Max), kE4m3Max);
    return __builtin_fabsf(x) < __builtin_inff() ? y : __builtin_nanf("");
}

// Four values already within +-448 (or NaN) to e4m3 bytes, ties to even.
__device__ __forceinline__ uint32_t bytes_of(float a, float b, float c, float d)
{
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// Four bytes held under a scale 2^shift times as large.
__device__ __forceinline__ uint32_t bytes_under(uint32_t bytes, float factor)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(bytes, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(bytes, true);
    return bytes_of(lo[0] * factor, lo[1] * factor, hi[0] * factor, hi[1] * factor);
}

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x = __builtin_fmaxf(x, __shfl_xor(x, d));
    return x;
}

}  // namespace kvmove
