// Shared by the embedding, layer-norm and output-head kernels: 8-element loads
// and stores of caller tensors at any element alignment.
//
// A caller's row may start at any element (an odd row stride, a slice of a
// packed tail), so the vector types carry the element's own alignment: the
// 16-byte global accesses of gfx950 take any byte address, and an aligned row
// costs the same as with an aligned type.
#pragma once

#include "device_common.h"

typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef f32x4 f32x4_e4 __attribute__((aligned(4)));

// 8 elements, still in the storage type (4 or 8 registers)
template <typename T> struct raw8;
template <> struct raw8<bf16_t> { u32x4 q; };
template <> struct raw8<float> { f32x4 lo, hi; };

MO_DEV raw8<bf16_t> ld8(const bf16_t* p) { return {*reinterpret_cast<const u32x4_e2*>(p)}; }
MO_DEV raw8<float> ld8(const float* p) {
    return {*reinterpret_cast<const f32x4_e4*>(p), *reinterpret_cast<const f32x4_e4*>(p + 4)};
}
MO_DEV f32x8 widen(const raw8<bf16_t>& r) {
    f32x8 o;
    const bf16x8 b = __builtin_bit_cast(bf16x8, r.q);
#pragma unroll
    for (int e = 0; e < 8; ++e) o.v[e] = (float)b[e];
    return o;
}
MO_DEV f32x8 widen(const raw8<float>& r) {
    f32x8 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) { o.v[e] = r.lo[e]; o.v[4 + e] = r.hi[e]; }
    return o;
}
MO_DEV raw8<bf16_t> narrow(const f32x8& v, bf16_t) {
    bf16x8 b;
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = (bf16_t)v.v[e];
    return {__builtin_bit_cast(u32x4, b)};
}
MO_DEV raw8<float> narrow(const f32x8& v, float) {
    return {f32x4{v.v[0], v.v[1], v.v[2], v.v[3]}, f32x4{v.v[4], v.v[5], v.v[6], v.v[7]}};
}
MO_DEV void st8(bf16_t* p, const raw8<bf16_t>& r) { *reinterpret_cast<u32x4_e2*>(p) = r.q; }
MO_DEV void st8(float* p, const raw8<float>& r) {
    *reinterpret_cast<f32x4_e4*>(p) = r.lo;
    *reinterpret_cast<f32x4_e4*>(p + 4) = r.hi;
}
MO_DEV void st8(bf16_t* p, const f32x8& v) { st8(p, narrow(v, bf16_t())); }
MO_DEV void st8(float* p, const f32x8& v) { st8(p, narrow(v, float())); }

// The first `n` of 8 elements (n may be 0 or more than 8); the rest are zero.
template <typename T> MO_DEV raw8<T> ld8n(const T* p, int n) {
    if (n >= 8) return ld8(p);
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] = e < n ? to_f32(p[e]) : 0.f;
    return narrow(v, T());
}
template <typename T> MO_DEV void st8n(T* p, const f32x8& v, int n) {
    if (n >= 8) {
        st8(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = from_f32<T>(v.v[e]);
    }
}

// Chunk c .. c + 7 of a row of `cols` elements, zeros behind its end.  FULL (cols
// a multiple of 8): a chunk is whole or outside, and is loaded without a branch
// (from the row's start when it is outside), so that loads of several chunks and
// rows go out back to back.
template <bool FULL, typename T> MO_DEV raw8<T> row8(const T* row, int c, int cols) {
    if constexpr (FULL) {
        const bool in = c < cols;
        raw8<T> r = ld8(row + (in ? c : 0));
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) r.q[e] = in ? r.q[e] : 0u;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) { r.lo[e] = in ? r.lo[e] : 0.f; r.hi[e] = in ? r.hi[e] : 0.f; }
        }
        return r;
    } else {
        return ld8n(row + c, cols - c);
    }
}
template <bool FULL, typename T> MO_DEV void row8_out(T* row, int c, int cols, const f32x8& v) {
    if constexpr (FULL) {
        if (c < cols) st8(row + c, v);
    } else {
        st8n(row + c, v, cols - c);
    }
}
