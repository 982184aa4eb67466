// The output head's tiled NT GEMM on bf16 MFMA, C[i][j] = sum_k P[i][k] Q[j][k],
// for operands that are the caller's own tensors:
//   - P and Q have their own row strides, and rows past the end are read as the
//     last row (the epilogue drops their results), so a ragged matrix needs no
//     padded copy;
//   - tiles of 256 x 256, 256 x 128 and 256 x 64 (NB = 4, 2, 1): the narrow ones
//     are for few tokens, where the product streams the other operand;
//   - fp32 operands come as three bf16 planes whose sum is the value exactly
//     (split_f32 below).  The product then runs over six of the nine plane
//     pairs as one long K loop into the same fp32 accumulators; the three left
//     out come to at most 2^-23 of a term.  Six bf16 MFMAs cost 6/16 of the fp32
//     MFMAs they replace.
//
// Design, with the rate of a 16384 x 8192 x 4096 and a 16384 x 4096 x 8192 product
// (bf16 results written, normal random data) at each step; a library product
// of the same shapes runs at 1550 and 1590 TFLOP/s on the same card:
//   1370, 1390  the loop of gemm_core8.h: 32 x 32 x 16 MFMAs, stages of 64 bytes in a
//               ring of five, a barrier per stage
//   1430, 1460  16 x 16 x 32 MFMAs: half the accumulator traffic per flop
//   1420, 1450  stages of 128 bytes (whole lines) in two slots, one barrier per
//               64 of K instead of two
//   1440, 1460  loads through buffer descriptors: a scalar offset advances along K, no
//               address arithmetic on the vector unit
//   1453, 1490  five eighths of a stage's loads right behind the barrier
// Tried and not kept: the two wavefronts of a SIMD taking turns at MFMAs and
// loads with a barrier between (1220, 1235); four wavefronts of 128 x 128 each (1430,
// 1475); fragment reads sent out faster than one per two MFMAs (1300 to 1430).
#pragma once

#include "gemm_core.h"

namespace mo_head_gemm {

using namespace mo_gemm;

constexpr int H_THREADS = 512;
constexpr int HKB = 128;                              // bytes of K per stage and row: one line
constexpr int HP_BYTES = 256 * HKB;                   // 32 KB of P per stage
constexpr int head_lds(int NB) { return 2 * (HP_BYTES + 64 * NB * HKB); }

// x = hi + mid + lo exactly: each the nearest bf16 to what is left (24 bits of
// significand = 3 x 8), so |mid| <= 2^-8 |x| and |lo| <= 2^-16 |x| (below 2^-109, where
// lo runs out of exponent, to 2^-134).  A finite x that
// would round to infinity is truncated; infinities and NaN keep mid and lo at 0.
MO_DEV void split_f32(float x, bf16_t& hi, bf16_t& mid, bf16_t& lo) {
    const bool finite = __builtin_fabsf(x) < __builtin_inff();
    hi = (bf16_t)x;
    if (finite && !(__builtin_fabsf((float)hi) < __builtin_inff()))
        hi = (bf16_t)__uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float r = finite ? x - (float)hi : 0.f;
    mid = (bf16_t)r;
    lo = (bf16_t)(r - (float)mid);
}

// Wave layout of a 256 x TN tile (TN = 64 NB) on 8 wavefronts: WM x WN of them,
// each MB x NBW blocks of 16 x 16.
template <int NB> struct Layout;
template <> struct Layout<4> { static constexpr int WM = 2, WN = 4, MB = 8, NBW = 4; };
template <> struct Layout<2> { static constexpr int WM = 4, WN = 2, MB = 4, NBW = 4; };
template <> struct Layout<1> { static constexpr int WM = 8, WN = 1, MB = 2, NBW = 4; };

// One operand: bf16 rows at `base`, `ld` bytes apart (256 ld < 2^31), `rows` of
// them readable; plane p of an fp32 operand starts p * plane bytes further.
struct Operand {
    const uint8_t* base;
    int64_t ld, rows, plane;
};

// The plane pairs of a split product, largest last so that the small ones are
// summed first: lo hi, hi lo, mid mid, mid hi, hi mid, hi hi.
template <int PL> MO_DEV int seg_p(int s) { return PL == 1 ? 0 : s == 0 ? 2 : (s == 2 || s == 3) ? 1 : 0; }
template <int PL> MO_DEV int seg_q(int s) { return PL == 1 ? 0 : s == 1 ? 2 : (s == 2 || s == 4) ? 1 : 0; }
// Two planes of P (a value rounded to bf16, and what that left) and one of Q.
template <> MO_DEV int seg_p<2>(int s) { return s == 0 ? 1 : 0; }
template <> MO_DEV int seg_q<2>(int) { return 0; }

// 128-byte rows of eight 16-byte chunks; chunk c of row r sits at c ^ (r / 2 mod 8).
// A fragment read takes 16 rows at four consecutive chunks; any 16 lanes that
// the LDS serves together (consecutive ones, or four groups of four from two
// chunks) then fall on 16 distinct 16-byte bank groups.
MO_DEV int hswz(int row) { return (row >> 1) & 7; }

// Accumulates rows p0 .. p0 + 255 of P and q0 .. q0 + TN - 1 of Q over `nk1` K
// stages of 128 bytes (64 elements) from stage k0 on.  Acc is f32x4[MB][NBW];
// acc[a][b] of wave (wm, wn) holds, in lane l, rows wm 16 MB + 16 a + 4 (l / 16) ..
// + 3 and column wn 16 NBW + 16 b + l % 16.  Ends with a workgroup barrier: the
// LDS is the epilogue's.
//
// Stage s sits in slot s mod 2.  A stage is four quarters of MFMAs (first and
// second half of the row blocks, for each half of K).  While one runs, the
// next one's fragments are read, so all reads of a stage are done when its
// third quarter ends: there each wave waits for its reads and its loads of
// stage s + 1, and the barrier publishes s + 1 and frees the slot of s.  The loads of
// stage s + 2 into that slot go out during the fourth quarter (LH of them) and
// the first quarter of stage s + 1, and have the two quarters after that to land.
template <int NB, int PL, class Acc>
__device__ __forceinline__ void head_tile(uint8_t* smem, const Operand& P, const Operand& Q, int64_t p0,
                                          int64_t q0, int k0, int nk1, Acc& acc) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass cannot check the device builtins
    using L = Layout<NB>;
    constexpr int WN = L::WN, MB = L::MB, NBW = L::NBW, HA = MB / 2, MF = HA * NBW;
    constexpr int TN = 64 * NB, SBYTES = HP_BYTES + TN * HKB;
    constexpr int LS = 4 + NB;                   // load instructions per stage and wave
    constexpr int NSEG = PL == 3 ? 6 : PL;
    static_assert(PL >= 1 && PL <= 3, "planes");
    const int n = nk1 * NSEG;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r16 = lane & 15, kg = lane >> 4;

    // Loads, straight to LDS: 8 rows of 128 bytes (1 KB) per instruction; wave w fills P rows
    // [32 w, 32 w + 32) and Q rows [8 NB w, ..); lane l -> row + l / 8, physical
    // chunk l % 8, which holds chunk (l % 8) ^ swizzle of the row.
    const uint8_t* Pb = P.base + p0 * P.ld + int64_t(k0) * HKB;
    const uint8_t* Qb = Q.base + q0 * Q.ld + int64_t(k0) * HKB;
    const int plim = int(P.rows - p0 < 256 ? P.rows - p0 : 256) - 1;
    const int qlim = int(Q.rows - q0 < TN ? Q.rows - q0 : TN) - 1;
    uint32_t vo[LS];
#pragma unroll
    for (int i = 0; i < LS; ++i) {
        const int r = (i < 4 ? wave * 32 + i * 8 : wave * 8 * NB + (i - 4) * 8) + (lane >> 3);
        const int lim = i < 4 ? plim : qlim;
        vo[i] = uint32_t(r < lim ? r : lim) * uint32_t(i < 4 ? P.ld : Q.ld) + uint32_t(((lane & 7) ^ hswz(r)) << 4);
    }
    // cursor of the stage being loaded; slot of stage s: s mod 2
    auto rsrc = [&](const uint8_t* p) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, -1, 0x00027000);
    };
    auto rP = rsrc(Pb + (PL == 1 ? 0 : seg_p<PL>(0) * P.plane)), rQ = rsrc(Qb + (PL == 1 ? 0 : seg_q<PL>(0) * Q.plane));
    int ck = 0, cseg = 0, koff = 0;
    auto next_stage = [&]() __attribute__((always_inline)) {
        koff += HKB;
        if constexpr (PL != 1) {
            if (++ck == nk1) {
                ck = 0;
                ++cseg;
                koff = 0;
                rP = rsrc(Pb + seg_p<PL>(cseg) * P.plane);
                rQ = rsrc(Qb + seg_q<PL>(cseg) * Q.plane);
            }
        }
    };
    auto issue1 = [&](int slot, int i) __attribute__((always_inline)) {
        uint8_t* sp = smem + slot * SBYTES + (i < 4 ? (wave * 32 + i * 8) * HKB : HP_BYTES + (wave * 8 * NB + (i - 4) * 8) * HKB);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(i < 4 ? rP : rQ, (lds_void_t*)sp, 16, vo[i], koff, 0, 0);
    };

#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    // fragments: 16 rows x 32 K, lane -> row lane % 16, K chunk 4 sub + lane / 16
    const int x0 = ((kg ^ hswz(r16)) << 4), x1 = x0 ^ 64;
    const int pbase = (wm * (MB * 16) + r16) * HKB, qbase = HP_BYTES + (wn * (NBW * 16) + r16) * HKB;
    auto rdp = [&](int slot, int sub, int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4*>(smem + slot * SBYTES + pbase + (sub ? x1 : x0) + i * 16 * HKB);
    };
    auto rdq = [&](int slot, int sub, int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4*>(smem + slot * SBYTES + qbase + (sub ? x1 : x0) + i * 16 * HKB);
    };
    u32x4 a0[HA], a1[HA], b0[NBW], b1[NBW];
    // Quarter h of a stage: MF MFMAs (row blocks (h & 1) HA .., K half h / 2) with the
    // next quarter's reads and the loads l0 .. l1 - 1 of another stage between them.
    auto quarter = [&](int h, int slot, bool reads, int lslot, int l0, int l1) __attribute__((always_inline)) {
        const int nr = !reads ? 0 : (h & 1) ? HA + NBW : HA;
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const int a = i / NBW, b = i % NBW;
            const u32x4 fa = (h & 1) ? a1[a] : a0[a], fb = h < 2 ? b0[b] : b1[b];
            f32x4& c = acc[(h & 1) * HA + a][b];
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fa), __builtin_bit_cast(bf16x8, fb), c, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < HA + NBW; ++r)
                if (r < nr && (2 * r == i || (i == MF - 1 && 2 * r > i))) {
                    // after 0: a1 (sub 0); 1: b1, a0 (sub 1); 2: a1 (sub 1); 3: b0, a0 of the next stage
                    if (!(h & 1)) a1[r] = rdp(slot, h / 2, HA + r);
                    else {
                        const int sl = h == 1 ? slot : slot ^ 1, sub = h == 1;
                        if (r < NBW) (h == 1 ? b1 : b0)[r] = rdq(sl, sub, r);
                        else a0[r - NBW] = rdp(sl, sub, r - NBW);
                    }
                }
#pragma unroll
            for (int l = 0; l < LS; ++l)
                if (l >= l0 && l < l1) {
                    const int at = (l - l0) * MF / (l1 - l0) + 1;
                    if ((at < MF ? at : MF - 1) == i) issue1(lslot, l);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int LH = (LS * 5 + 7) / 8;
    // The stage in `slot`: in quarter 0 (ld0) the rest of the next stage's loads, in
    // quarter 3 (ld3) the first loads of the one after it.
    auto stage = [&](int slot, bool ld0, bool next, bool ld3) __attribute__((always_inline)) {
        quarter(0, slot, true, slot ^ 1, ld0 ? LH : 0, ld0 ? LS : 0);
        if (ld0) next_stage();
        quarter(1, slot, true, 0, 0, 0);
        quarter(2, slot, true, 0, 0, 0);
        if (next) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
        quarter(3, slot, next, slot, 0, ld3 ? LH : 0);
    };

#pragma unroll
    for (int l = 0; l < LS; ++l) issue1(0, l);
    next_stage();
    if (n > 1) {
#pragma unroll
        for (int l = 0; l < LS; ++l) issue1(1, l);
        next_stage();
    }
    if (n == 1) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else if constexpr (LS == 8) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else if constexpr (LS == 6) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(5)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < NBW; ++i) b0[i] = rdq(0, 0, i);
#pragma unroll
    for (int i = 0; i < HA; ++i) a0[i] = rdp(0, 0, i);
    __builtin_amdgcn_sched_barrier(0);
    int s = 0;
    if (n > 2) {
        stage(0, false, true, true);
        for (s = 1; s < n - 2; ++s) stage(s & 1, true, true, true);
        stage(s & 1, true, true, false);
        ++s;
    } else if (n == 2) {
        stage(0, false, true, false);
        s = 1;
    }
    stage(s & 1, false, false, false);
    __syncthreads();
#endif
}

// ---- P in fp32, as it lies in memory ---------------------------------------------------
//
// For few tokens the product is a read of the other operand, and splitting that
// one into planes first moves it five times more (4 bytes to read, 6 to write, and 12
// to read back for the six plane pairs).  Here P stays fp32 up to the registers,
// where each fragment is split; Q (tokens) still comes as planes.  Tiles of 64
// tokens only: there one wave needs a fragment of P, so it is split once.
//
// Stages of 32 K: 256 x 32 fp32 of P (32 KB) and three planes of 64 rows of 64 bytes
// of Q (12 KB), in a ring of three.  While a stage's 48 MFMAs run, the next one's
// fragments are read and split.  One product at 64 tokens x 32001 rows x 4096 (524 MB):
// 117 to 141 us; its loads alone take 99 to 110 and its MFMAs and splitting alone 95 to
// 105, of which six bf16 products at the rate of a large one are 70.  Without the
// pipeline over stages it was 129 to 155; tiles of 128 tokens, which do not have the
// registers for it, took 390 at 256 tokens against 413 with these.
// P is either
//   rows along K (NN false): as above, 128-byte rows, chunk c of row r at c ^ pswz(r);
//   K along the rows (NN true): 32 rows of 256 columns (1 KB); chunk c of row r at
//     c ^ 4 (r / 8 mod 4), so that the four K groups of a fragment's column fall on
//     four different quarters of the 64 banks.
// Q: chunk c of row r at c ^ qswz(r).
// The 16 lanes that the LDS serves together in a 16-byte read are consecutive ones,
// or rows 0-3 and 12-15 of one K group with rows 4-11 of the next, or the other way
// round.  A fragment of P takes chunks 2 kg and 2 kg + 1, so bit 1 of the chunk has
// to change as bit 0 of r / 2 does; with 64-byte rows the groups of four rows get
// 0, 2, 3, 1, which stay apart under an exchange of neighbours and ^ 1.
MO_DEV int pswz(int row) { const int x = row >> 1; return ((x << 1) & 6) | ((x >> 2) & 1); }
MO_DEV int qswz(int row) { const int g = (row >> 2) & 3; return ((g << 1) & 2) ^ ((g >> 1) * 3); }
constexpr int S32_SLOTS = 3, S32_BYTES = HP_BYTES + 3 * 64 * 64;
constexpr int head_lds32() { return S32_SLOTS * S32_BYTES; }

// Eight values as three planes, each the nearest bf16 (ties away from zero) to what is
// left; eight bits are left for the last one, which is exact.  In integer adds and
// masks (2 % faster here than conversions and shifts).  The high part stays finite;
// infinities and NaN leave NaN in the others (a product with the exact planes of
// split_f32 also ends in NaN: infinity times a zero low part).
MO_DEV void split_frag(const float (&x)[8], bf16x8 (&p)[3]) {
    constexpr float M = 3.3895313892515355e38f;   // the largest bf16
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = (__float_as_uint(__builtin_amdgcn_fmed3f(x[e], -M, M)) + 0x8000u) & 0xFFFF0000u;
        const float r = x[e] - __uint_as_float(h[e]);
        m[e] = (__float_as_uint(r) + 0x8000u) & 0xFFFF0000u;
        l[e] = __float_as_uint(r - __uint_as_float(m[e]));
    }
    u32x4 o[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // the upper halves of two
        o[0][e] = __builtin_amdgcn_perm(h[2 * e + 1], h[2 * e], 0x07060302u);
        o[1][e] = __builtin_amdgcn_perm(m[2 * e + 1], m[2 * e], 0x07060302u);
        o[2][e] = __builtin_amdgcn_perm(l[2 * e + 1], l[2 * e], 0x07060302u);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) p[i] = __builtin_bit_cast(bf16x8, o[i]);
}

// As head_tile, with P in fp32: `cols` of its columns are there (a multiple of 4).
// NN false: rows p0 .. of P, K along its columns; NN true: columns p0 .. of P,
// K along its rows.  K behind the end counts as zeros.  k0 and nk1 in stages of 64 K.
template <bool NN, class Acc>
__device__ __forceinline__ void head_tile32(uint8_t* smem, const Operand& P, int cols, const Operand& Q, int64_t p0,
                                            int64_t q0, int k0, int nk1, Acc& acc) {
#ifdef __HIP_DEVICE_COMPILE__
    using L = Layout<1>;
    constexpr int MB = L::MB, NBW = L::NBW, S = S32_SLOTS;
    static_assert(L::WN == 1 && MB == 2 && NBW == 4, "8 waves of 32 x 64");
    // Q: 12 instructions of 16 rows x 64 bytes over the 8 waves (the last one by five of them)
    constexpr int QI = 2;   // with the four of P: 6 loads per stage and wave
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int n = nk1 * 2, s0 = k0 * 2;   // stages of 32 K, an even number
    auto rsrc = [&](const uint8_t* p) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, -1, 0x00027000);
    };

    uint32_t prow[4], pch[4], vq[QI];
    const int plim = int(P.rows - p0 < 256 ? P.rows - p0 : 256) - 1;    // NN false
    const int qlim = int(Q.rows - q0 < 64 ? Q.rows - q0 : 64) - 1;
    auto qinst = [&](int i) __attribute__((always_inline)) { return wave + 8 * i < 12 ? wave + 8 * i : 11; };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (NN) {
            const int r = wave * 4 + i, c = lane ^ (((r >> 3) & 3) << 2), last = int(cols - p0) / 4 - 1;
            prow[i] = 0;
            pch[i] = uint32_t(c < last ? c : last) * 16;
        } else {
            const int r = wave * 32 + i * 8 + (lane >> 3);
            prow[i] = uint32_t(r < plim ? r : plim) * uint32_t(P.ld);
            pch[i] = uint32_t((lane & 7) ^ pswz(r)) * 16;
        }
    }
#pragma unroll
    for (int i = 0; i < QI; ++i) {
        const int r = qinst(i) % 4 * 16 + (lane >> 2);
        vq[i] = uint32_t(r < qlim ? r : qlim) * uint32_t(Q.ld) + uint32_t(((lane & 3) ^ qswz(r)) << 4);
    }
    const uint8_t* Pb = NN ? P.base + p0 * 4 : P.base + p0 * P.ld;
    const uint8_t* Qb = Q.base + q0 * Q.ld;
    const auto rP = rsrc(Pb);
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        uint8_t* sp = smem + slot * S32_BYTES;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lds_void_t* to = (lds_void_t*)(sp + (wave * 4 + i) * 1024);
            if constexpr (NN) {
                const int64_t k = int64_t(s0 + s) * 32 + wave * 4 + i;
                const auto row = rsrc(Pb + (k < P.rows ? k : P.rows - 1) * P.ld);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(row, to, 16, pch[i], 0, 0, 0);
            } else {
                const uint32_t at = uint32_t(s0 + s) * 128 + pch[i], last = uint32_t(cols) * 4 - 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rP, to, 16, prow[i] + (at < last ? at : last), 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < QI; ++i) {
            const int t = qinst(i);
            const auto q = rsrc(Qb + t / 4 * Q.plane);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(q, (lds_void_t*)(sp + HP_BYTES + t * 1024), 16, vq[i],
                                                     (s0 + s) * 64, 0, 0);
        }
    };

#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int64_t klim = NN ? P.rows : int64_t(cols);
    int pat[2];   // NN: K element 0 of column block a; else the two chunks of row block 0
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        if constexpr (NN) {
            const int c = wave * 32 + a * 16 + r16;
            pat[a] = kg * 8 * 1024 + (((c >> 2) ^ (kg << 2)) << 4) + (c & 3) * 4;
        } else {
            pat[a] = (wave * 32 + r16) * HKB + (((2 * kg + a) ^ pswz(r16)) << 4);
        }
    }
    const int qat = HP_BYTES + r16 * 64 + ((kg ^ qswz(r16)) << 4);

    struct Frag {
        bf16x8 p[MB][3];
        u32x4 q[3][NBW];
    } f0, f1;
    float x[MB][8];
    // the fragments of a stage: from LDS, and P's split
    auto read = [&](Frag& f, int slot) __attribute__((always_inline)) {
        const uint8_t* sp = smem + slot * S32_BYTES;
#pragma unroll
        for (int a = 0; a < MB; ++a) {
            if constexpr (NN) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[a][e] = *reinterpret_cast<const float*>(sp + pat[a] + e * 1024);
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(sp + pat[c] + a * (16 * HKB));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[a][c * 4 + e] = v[e];
                }
            }
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int b = 0; b < NBW; ++b)
                f.q[p][b] = *reinterpret_cast<const u32x4*>(sp + qat + p * (64 * 64) + b * (16 * 64));
    };
    auto split = [&](Frag& f, int s) __attribute__((always_inline)) {
        const int64_t left = klim - int64_t(s0 + s) * 32;
        if (left < 32)
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[a][e] = kg * 8 + e < left ? x[a][e] : 0.f;
#pragma unroll
        for (int a = 0; a < MB; ++a) split_frag(x[a], f.p[a]);
    };
    // the plane pairs, largest last
    auto mfma = [&](const Frag& f, int a) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 6; ++t)
#pragma unroll
            for (int b = 0; b < NBW; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    f.p[a][seg_p<3>(t)], __builtin_bit_cast(bf16x8, f.q[seg_q<3>(t)][b]), acc[a][b], 0, 0, 0);
    };
    // Stage s, its fragments in `f`.
    int slot = 0;   // of stage s
    auto stage = [&](int s, Frag& f, Frag& next) __attribute__((always_inline)) {
        // the loads of stage s + 1 have landed, and every wave has read the slot of stage s
        if (s + 2 < n) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (s + S < n) issue(s + S, slot);
        slot = slot == S - 1 ? 0 : slot + 1;
        // (behind the last stage: what the slot holds, read and not used)
        read(next, slot);
        mfma(f, 0);
        __builtin_amdgcn_sched_barrier(0);
        split(next, s + 1);
        mfma(f, 1);
#pragma unroll
        for (int t = 0; t < 24; ++t) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);   // an MFMA
            __builtin_amdgcn_sched_group_barrier(0x2, 6, 0);   // six of the splitting
        }
    };
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (i < n) issue(i, i);
    // stage 0 has landed
    if (n > 2) asm volatile("s_waitcnt vmcnt(12)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(f0, 0);
    split(f0, 0);
    for (int s = 0; s < n; s += 2) {
        stage(s, f0, f1);
        stage(s + 1, f1, f0);
    }
    __syncthreads();
#endif
}

// Tile of workgroup b among tm x tn: each XCD (b mod 8) takes one contiguous
// share of the tiles, ordered in bands of four tile rows, column by column, so
// the 32 tiles an XCD runs at once share 4 panels of P and 8 of Q in its L2.
// False past the end (the grid is a multiple of 8).
MO_DEV bool head_tile_of(uint32_t b, uint32_t tm, uint32_t tn, uint32_t& ti, uint32_t& tj) {
    const uint32_t nt = tm * tn, x = b & 7, j = b >> 3, share = nt >> 3, rem = nt & 7;
    if (j >= share + (x < rem ? 1u : 0u)) return false;
    const uint32_t t = x * share + (x < rem ? x : rem) + j;
    const uint32_t band = t / (4 * tn), r = t - band * 4 * tn;
    const uint32_t h = tm - band * 4 < 4 ? tm - band * 4 : 4;
    ti = band * 4 + r % h;
    tj = r / h;
    return true;
}
inline uint32_t head_grid(uint64_t tiles) { return uint32_t((tiles + 7) / 8 * 8); }

}  // namespace mo_head_gemm
