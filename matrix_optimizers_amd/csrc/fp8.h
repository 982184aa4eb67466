// Shared by the 8-bit kernels: a block of 128 elements as e4m3 numbers q and one e8m0
// byte, x = q 2^(byte - 127).
//
// The byte is the least for which no element of the block exceeds e4m3's largest, 448
// = 1.75 2^8.  With the block's largest magnitude m 2^p, 1 <= m < 2, that is p - 8 + 127,
// one more where m > 1.75: an add and a compare on the bits.  The multiplication
// with 2^(127 - byte) is then exact (below 2^-126 it may not be), so the only
// rounding is the conversion's, to nearest even.  A scale that is a power of two is
// what the matrix instructions apply by themselves, and q 2^e is a bf16 number (down to 2^-130).
// Infinities and NaN do not count for the scale and become e4m3's NaN, each by
// itself; the byte 255 is NaN for its whole block, and is only ever read.
#pragma once

#include "op_common.h"

constexpr int F8_BLOCK = 128;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_e1 __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

MO_DEV uint32_t scale_byte(uint32_t amax_bits) {
    const int b = int(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return uint32_t(b > 0 ? b : 0);
}
// 2^(127 - byte) for a byte of scale_byte (at most 247)
MO_DEV float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
MO_DEV float scale_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte ? byte << 23 : 0x00400000u);
}

// The largest finite magnitude of 8 values, as bits.
MO_DEV uint32_t amax8(const f32x8& x) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t a = __float_as_uint(x.v[e]) & 0x7FFFFFFFu, f = a < 0x7F800000u ? a : 0u;
        m = f > m ? f : m;
    }
    return m;
}
// The maximum over 16 consecutive lanes, in each of them.
MO_DEV uint32_t max16(uint32_t x) {
#ifdef __HIP_DEVICE_COMPILE__
    auto most = [&](int y) __attribute__((always_inline)) { x = uint32_t(y) > x ? uint32_t(y) : x; };
    most(__builtin_amdgcn_mov_dpp(int(x), 0xB1, 0xF, 0xF, true));    // lanes 1 0 3 2
    most(__builtin_amdgcn_mov_dpp(int(x), 0x4E, 0xF, 0xF, true));    // lanes 2 3 0 1
    most(__builtin_amdgcn_mov_dpp(int(x), 0x141, 0xF, 0xF, true));   // mirrored in 8
    most(__builtin_amdgcn_mov_dpp(int(x), 0x140, 0xF, 0xF, true));   // mirrored in 16
#endif
    return x;
}

// x times `inverse` as eight e4m3 numbers.
MO_DEV u32x2 to_e4m3(const f32x8& x, float inverse) {
    u32x2 r = {0u, 0u};
#ifdef __HIP_DEVICE_COMPILE__
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(x.v[4 * h] * inverse, x.v[4 * h + 1] * inverse, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(x.v[4 * h + 2] * inverse, x.v[4 * h + 3] * inverse, w, true);
        r[h] = uint32_t(w);
    }
#endif
    return r;
}
// eight e4m3 numbers times `scale`
MO_DEV f32x8 from_e4m3(u32x2 q, float scale) {
    f32x8 o = {};
#ifdef __HIP_DEVICE_COMPILE__
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[h]), false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[h]), true);
        o.v[4 * h] = lo[0] * scale;
        o.v[4 * h + 1] = lo[1] * scale;
        o.v[4 * h + 2] = hi[0] * scale;
        o.v[4 * h + 3] = hi[1] * scale;
    }
#endif
    return o;
}

// The first n of 8 bytes (n may be 0, negative or more than 8); the others are zero.
MO_DEV u32x2 ldq8(const uint8_t* p, int n) {
    if (n >= 8) return *reinterpret_cast<const u32x2_e1*>(p);
    u32x2 r = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) r[e / 4] |= uint32_t(p[e]) << (8 * (e % 4));
    return r;
}
MO_DEV void stq8(uint8_t* p, u32x2 q, int n) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_e1*>(p) = q;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = uint8_t(q[e / 4] >> (8 * (e % 4)));
    }
}
