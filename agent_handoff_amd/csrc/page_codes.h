// page_codes.h - how a paged cache holds bf16 vectors: 8 channels to codes and
// back, shared by the kernels that write and read pages (device side).
#pragma once

#include "attend.h"
#include "kernels_common.h"

namespace kvc {
namespace {

// Maximum over LPV (2, 4, 8 or 16) neighbouring lanes.
template <int LPV>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
    const auto step = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm xor 1
    if (LPV >= 4) v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad_perm xor 2
    if (LPV >= 8) v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // row_half_mirror
    if (LPV == 16) v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // row_mirror
    return v;
}

__device__ __forceinline__ void unpack8(const uint4& x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16_lo(w[i]);
        y[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Largest magnitude of 8 bf16 values as an integer: NaN above Inf above the rest.
__device__ __forceinline__ uint32_t magnitude8(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        const uint32_t y = lo > hi ? lo : hi;
        m = y > m ? y : m;
    }
    return m;
}

// 8 channels of a vector -> codes (8 bytes) and the vector's step, from its
// largest magnitude m (as an integer).
//
// code = round(x * M / m), m the vector's maximum. With m brought to A in
// [1/2, 1) by a power of two, x * (M * that power) is exact in binary32 (8 + 7
// bits), and q = x * M / m by a reciprocal is corrected by its exact remainder: a
// quotient that is a tie (representable) comes out exact; any other is at
// least 2^-13 of its size away from a tie, since it is a ratio of integers of few
// bits. So the codes are those of exact arithmetic. The step m / M is made the
// same way, correctly rounded (so for each of the 128 significands of m).
// Maxima below 2^-100 take the slow way: their factors leave binary32's range.
template <int FMT>
__device__ __forceinline__ uint2 quantise8(const uint4& x, uint32_t m, float& step) {
    const float most = FMT == kPageInt8 ? 127.0f : 448.0f, inv_most = 1.0f / most;
    const float big = __uint_as_float(m << 16);
    float y[8], q[8];
    unpack8(x, y);
    const int e = __builtin_amdgcn_frexp_expf(big);
    const float A = __builtin_amdgcn_ldexpf(big, -e);
    const float rA = __builtin_amdgcn_rcpf(A);
    const auto corrected = [](float r, float divisor, float reciprocal) {
        const float q0 = r * reciprocal;
        return fmaf(fmaf(-q0, divisor, r), reciprocal, q0);
    };
    if (m >= 0x0D80u) {  // 2^-100
        step = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __builtin_amdgcn_ldexpf(corrected(A, most, inv_most), e);
        if (m >= 0x7F80u) return make_uint2(0, 0);
        const float up = __builtin_amdgcn_ldexpf(most, -e);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = corrected(y[i] * up, A, rA);
    } else {
        step = big / most;
        if (m == 0) return make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = corrected(__builtin_amdgcn_ldexpf(y[i], -e) * most, A, rA);
    }
    if (FMT == kPageFp8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = copysignf(q[i], y[i]);  // the remainder of -0 is +0: e4m3 keeps the sign
    }
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (FMT == kPageInt8) {
            // adding 1.5 * 2^23 rounds to an integer (ties to even) held in the low bits
            uint32_t b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) b[u] = __float_as_uint(q[4 * i + u] + 12582912.0f);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
            o[i] = lo | hi;
        } else {
            int v = 0;
            v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], v, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], v, true);
            o[i] = (uint32_t)v;
        }
    }
    return make_uint2(o[0], o[1]);
}

template <int FMT>
__device__ __forceinline__ uint4 dequantise8(const uint2& c, float step) {
    float y[8];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (FMT == kPageInt8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) y[4 * i + u] = (float)(int32_t)(int8_t)(w[i] >> (8 * u) & 0xFF) * step;
        } else {
            y[4 * i] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 0) * step;
            y[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 1) * step;
            y[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 2) * step;
            y[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 3) * step;
        }
    }
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
}

// 8 channels of a block of 32 -> eight 4-bit codes, the first in the lowest bits,
// and the byte of the block's power of two, from the block's largest magnitude.
// The power 2^e puts the largest at 3.5 to 7 times 2^e. A code of 6 is then off by as
// much as any between 4 and 6 (1 * 2^e), where the next power up would leave the
// codes' two finest steps unused. e is held to -125 .. 125: every code is then a
// normal bf16 number or 0, and none passes bf16's range. The instruction divides
// by the scale exactly, rounds to nearest, ties to even, and cuts off at 6.
__device__ __forceinline__ uint32_t quantise8_fp4(const uint4& x, uint32_t m, uint32_t& power) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bool bad = m >= 0x7F80u;
    // + 31 carries into the exponent if the 7 bits behind the point are above 1.75's
    const int e = (int)((m + 31) >> 7) - 2;
    const uint32_t byte = e < 2 ? 2 : e > 252 ? 252 : e;
    power = bad ? 255 : byte;
    const float scale = __uint_as_float(byte << 23);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o = 0;
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
    return bad || m == 0 ? 0 : o;
}

// Two 4-bit codes, byte B of c, times the power of two whose byte is in bits 23 to 30
// of `scale` (the instruction looks at no others) as two bf16 numbers, exactly; a byte of 255 gives NaN.
template <int B>
__device__ __forceinline__ uint32_t widen_fp4(uint32_t c, uint32_t scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, __uint_as_float(scale), B));
}
__device__ __forceinline__ uint4 dequantise8_fp4(uint32_t c, uint32_t power) {
    const uint32_t s = power << 23;
    return make_uint4(widen_fp4<0>(c, s), widen_fp4<1>(c, s), widen_fp4<2>(c, s), widen_fp4<3>(c, s));
}

// ---- codes to the matrix cores' types, exactly

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    half2_t r;
    r.x = (_Float16)lo;
    r.y = (_Float16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// Bytes b0, b1 (or b2, b3) of w, int8 codes with their sign bit flipped, to
// two binary16 codes: 0x64bb is 1024 + b, exact, and so is the difference.
template <bool HI>
__device__ __forceinline__ uint32_t widen_int8(uint32_t w) {
    const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w, HI ? 0x04030402u : 0x04010400u);
    const half2_t bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, u) - bias);
}
template <bool HI>
__device__ __forceinline__ uint32_t widen_fp8(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HI));
}
}  // namespace
}  // namespace kvc
