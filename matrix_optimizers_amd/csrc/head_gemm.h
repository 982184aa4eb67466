// The output head's tiled NT GEMM on bf16 MFMA, C[i][j] = sum_k P[i][k] Q[j][k]:
// the K pipeline of gemm_core8.h (512 threads, two wavefronts per SIMD, a ring
// of five LDS stages filled by direct-to-LDS loads) for operands that are the
// caller's own tensors:
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
#pragma once

#include "gemm_core.h"

namespace mo_head_gemm {

using namespace mo_gemm;

constexpr int H_THREADS = 512;

// x = hi + mid + lo exactly: each the nearest bf16 to what is left (24 bits of
// significand = 3 x 8), so |mid| <= 2^-8 |x| and |lo| <= 2^-16 |x|.  A finite x that
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

// Wave layout of a 256 x TN tile (TN = 64 NB) on 8 wavefronts.
template <int NB> struct Layout;
template <> struct Layout<4> { static constexpr int WM = 2, WN = 4, MB = 4, NBW = 2; };
template <> struct Layout<2> { static constexpr int WM = 4, WN = 2, MB = 2, NBW = 2; };
template <> struct Layout<1> { static constexpr int WM = 8, WN = 1, MB = 1, NBW = 2; };

// One operand: bf16 rows at `base`, `ld` bytes apart (256 ld < 2^32), `rows` of
// them readable; plane p of an fp32 operand starts p * plane bytes further.
struct Operand {
    const uint8_t* base;
    int64_t ld, rows, plane;
};

// The plane pairs of a split product, largest last so that the small ones are
// summed first: lo hi, hi lo, mid mid, mid hi, hi mid, hi hi.
template <int PL> MO_DEV int seg_p(int s) { return PL == 1 ? 0 : s == 0 ? 2 : (s == 2 || s == 3) ? 1 : 0; }
template <int PL> MO_DEV int seg_q(int s) { return PL == 1 ? 0 : s == 1 ? 2 : (s == 2 || s == 4) ? 1 : 0; }

constexpr int head_lds(int NB) { return NSTAGE * (OPND_BYTES + 64 * NB * KB); }

// Accumulates rows p0 .. p0 + 255 of P and q0 .. q0 + TN - 1 of Q over `nk1` K
// stages of 64 bytes from stage k0 on (nk1 even; 2, 4 or at least 8 with PL = 1,
// any even count with PL = 3).  Acc is f32x16[MB][NBW]; acc[a][b] of wave (wm, wn) holds rows
// wm MB 32 + 32 a and columns wn NBW 32 + 32 b in the MFMA layout of gemm_core.h.
// Ends with a workgroup barrier: the LDS is the epilogue's.
template <int NB, int PL, class Acc>
__device__ __forceinline__ void head_tile(uint8_t* smem, const Operand& P, const Operand& Q, int64_t p0,
                                          int64_t q0, int k0, int nk1, Acc& acc) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass cannot check the device builtins
    using L = Layout<NB>;
    constexpr int WN = L::WN, MB = L::MB, NBW = L::NBW;
    constexpr int TN = 64 * NB;
    constexpr int SBYTES = OPND_BYTES + TN * KB;
    constexpr int QI = NB == 4 ? 2 : 1;          // Q load instructions per stage and wave
    constexpr int LS = 2 + QI;
    constexpr int LP = 2 * LS;                   // loads per pair of stages
    constexpr int MF = MB * NBW;
    constexpr int NR = MB + NBW;
    constexpr int NSEG = PL == 1 ? 1 : 6;
    static_assert(PL == 1 || PL == 3, "planes");
    const int nk = nk1 * NSEG;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r32 = lane & 31, kg = lane >> 5;

    // Wave w fills P rows [32 w, 32 w + 32) and Q rows [16 QI w, ..), 16 rows
    // (1 KB) per instruction; lane l -> row + l / 4, physical chunk l % 4.  With
    // 64 Q rows four waves would do: waves 4 .. 7 repeat the loads of 0 .. 3 (same
    // bytes to the same place), so every wave counts the same loads.
    const int lrow = lane >> 2, pch = lane & 3;
    const uint32_t lch = uint32_t((pch ^ ((lrow >> 2) & 3)) << 4);
    const int qw = NB == 1 ? (wave & 3) : wave;
    const uint8_t* Pb = P.base + p0 * P.ld + int64_t(k0) * KB;
    const uint8_t* Qb = Q.base + q0 * Q.ld + int64_t(k0) * KB;
    const int plim = int(P.rows - p0 < 256 ? P.rows - p0 : 256) - 1;
    const int qlim = int(Q.rows - q0 < TN ? Q.rows - q0 : TN) - 1;
    uint32_t vo[LS];
#pragma unroll
    for (int i = 0; i < LS; ++i) {
        const int r = (i < 2 ? wave * 32 + i * 16 : qw * 16 * QI + (i - 2) * 16) + lrow;
        const int lim = i < 2 ? plim : qlim;
        vo[i] = uint32_t(r < lim ? r : lim) * uint32_t(i < 2 ? P.ld : Q.ld) + lch;
    }
    // cursor of the pair of stages being loaded
    const uint8_t *cP = Pb + (PL == 1 ? 0 : seg_p<PL>(0) * P.plane);
    const uint8_t *cQ = Qb + (PL == 1 ? 0 : seg_q<PL>(0) * Q.plane);
    int ck = 0, cseg = 0;
    auto next_pair = [&]() __attribute__((always_inline)) {
        cP += 2 * KB;
        cQ += 2 * KB;
        if constexpr (PL != 1) {
            ck += 2;
            if (ck == nk1) {
                ck = 0;
                ++cseg;
                cP = Pb + seg_p<PL>(cseg) * P.plane;
                cQ = Qb + seg_q<PL>(cseg) * Q.plane;
            }
        }
    };
    // instruction i of stage ks, the (ks & 1)-th of the cursor's pair
    auto issue1 = [&](int ks, int i) __attribute__((always_inline)) {
        uint8_t* sp = smem + (ks % NSTAGE) * SBYTES;
        if (i < 2) sp += (wave * 32 + i * 16) * KB;
        else sp += OPND_BYTES + (qw * 16 * QI + (i - 2) * 16) * KB;
        const uint8_t* g = (i < 2 ? cP : cQ) + (ks & 1) * KB;
        __builtin_amdgcn_global_load_lds(g + vo[i], (lds_void_t*)sp, 16, 0, 0);
    };

#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NBW; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.f;

    auto rd1 = [&](int ks, int sub, int i, u32x4 (&fa)[MB], u32x4 (&fb)[NBW]) __attribute__((always_inline)) {
        const uint8_t* sp = smem + (ks % NSTAGE) * SBYTES;
        const int chunk = 2 * sub + kg;
        if (i < MB) fa[i] = *reinterpret_cast<const u32x4*>(sp + swz(wm * (MB * 32) + i * 32 + r32, chunk));
        else fb[i - MB] = *reinterpret_cast<const u32x4*>(sp + OPND_BYTES + swz(wn * (NBW * 32) + (i - MB) * 32 + r32, chunk));
    };
    auto wait_loads = [&](int after) {
        if (after == 9) asm volatile("s_waitcnt vmcnt(9)" ::: "memory");
        else if (after == 8) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
        else if (after == 7) asm volatile("s_waitcnt vmcnt(7)" ::: "memory");
        else if (after == 6) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
        else if (after == 5) asm volatile("s_waitcnt vmcnt(5)" ::: "memory");
        else if (after == 4) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
        else if (after == 1) asm volatile("s_waitcnt vmcnt(1)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    };
    auto barrier = [&]() {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // MF MFMAs on (fa, fb), the reads of the next substep and quarter q of the
    // loads of the pair (ia, ia + 1) spread between them (gemm_core8's substep).
    auto substep = [&](const u32x4 (&fa)[MB], const u32x4 (&fb)[NBW], bool do_read, int rks, int rsub,
                       u32x4 (&na)[MB], u32x4 (&nb)[NBW], int ia, int q) __attribute__((always_inline)) {
        const int l0 = q * LP / 4, nl = (q + 1) * LP / 4 - l0;
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            Mfma<bf16_t>::run(fa[i / NBW], fb[i % NBW], acc[i / NBW][i % NBW]);
            __builtin_amdgcn_sched_barrier(0);
            if (do_read) {
                if (i < NR) rd1(rks, rsub, i, na, nb);
                if (i == MF - 1)
#pragma unroll
                    for (int r = MF; r < NR; ++r) rd1(rks, rsub, r, na, nb);
            }
            if (ia >= 0)
#pragma unroll
                for (int j = 0; j < nl; ++j)
                    if ((j + 1) * MF / nl - 1 == i) {
                        const int l = l0 + j;
                        issue1(ia + (l & 1), l >> 1);
                    }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    u32x4 f0a[MB], f0b[NBW], f1a[MB], f1b[NBW];
    if (nk >= 8) {
        // the schedule of gemm_core8: stage s in ring slot s % 5, pairs of
        // stages loaded four stages ahead in quarters over four substeps
        constexpr int W_EVEN = LP, W_ODD = 1 + LP / 2, W_FIRST = 1 + LP;
#pragma unroll
        for (int p = 0; p < 4; p += 2) {
#pragma unroll
            for (int l = 0; l < LP; ++l) issue1(p + (l & 1), l >> 1);
            next_pair();
        }
        wait_loads(W_FIRST);
        barrier();
#pragma unroll
        for (int i = 0; i < NR; ++i) rd1(0, 0, i, f0a, f0b);
        __builtin_amdgcn_sched_barrier(0);
        auto step = [&](int ks, int after, int pa, int qa, int pb, int qb) __attribute__((always_inline)) {
            substep(f0a, f0b, true, ks, 1, f1a, f1b, pa, qa);
            if (pa >= 0 && qa == 3) next_pair();
            wait_loads(after);
            barrier();     // stage ks + 1 visible everywhere; every read of stage ks done
            __builtin_amdgcn_sched_barrier(0);
            substep(f1a, f1b, true, ks + 1, 0, f0a, f0b, pb, qb);
        };
        step(0, W_EVEN, -1, 0, 4, 0);
        step(1, W_ODD, 4, 1, 4, 2);
        int ks = 2;
        for (; ks + 6 <= nk; ks += 2) {
            step(ks, W_EVEN, ks + 2, 3, ks + 4, 0);
            step(ks + 1, W_ODD, ks + 4, 1, ks + 4, 2);
        }
        step(ks, W_EVEN, ks + 2, 3, -1, 0);
        step(ks + 1, 1, -1, 0, -1, 0);
        step(ks + 2, 0, -1, 0, -1, 0);
        substep(f0a, f0b, true, nk - 1, 1, f1a, f1b, -1, 0);
        substep(f1a, f1b, false, 0, 0, f0a, f0b, -1, 0);
    } else {
        // two or four stages: all of them at once
        for (int p = 0; p < nk; p += 2) {
#pragma unroll
            for (int l = 0; l < LP; ++l) issue1(p + (l & 1), l >> 1);
            next_pair();
        }
        wait_loads(0);
        barrier();
        for (int ks = 0; ks < nk; ++ks) {
#pragma unroll
            for (int i = 0; i < NR; ++i) rd1(ks, 0, i, f0a, f0b);
            substep(f0a, f0b, true, ks, 1, f1a, f1b, -1, 0);
            substep(f1a, f1b, false, 0, 0, f0a, f0b, -1, 0);
        }
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
