// The tiled NT GEMM on 8-bit operands with a power-of-two scale for each block of 128
// along K: C[i][j] = sum over blocks kb of 2^(sp[i][kb] + sq[j][kb] - 254) sum_k P[i][k] Q[j][k].
//
// One instruction, 16 x 16 x 128 of e4m3 with e8m0 scales, takes a whole block, so the
// scales cost no arithmetic.  It holds its products to about 2^-17 of the largest of those
// it adds together before they go into the fp32 accumulator: measured against 64 bits,
// 1.5e-5 of the result's norm for normal data at any K, a hundredth of a bf16 rounding.
// A product whose result is fp32 is therefore not taken here.
//
// The tiles, the LDS rows of 128 bytes and their swizzle are those of the bf16 GEMM
// (head_gemm.h): a stage of 128 bytes per row is 128 elements of K here, one
// block, and the same bytes keep the matrix cores as long as 64 bf16 ones.  A lane's 32
// bytes of a fragment are chunks kg and kg + 4 of its row, in P and in Q alike: which
// element of a block meets which lane does not matter as both sides agree.
//
// Scales of rows: a workgroup's rows load four stages' bytes at once, one dword per row,
// straight to LDS; a wavefront keeps its 16-row blocks' dwords in registers and
// shifts them by a byte per stage.  Scales of P in blocks of 128 rows (a weight) are the
// same for all of a wavefront's rows: the workgroup's two blocks have theirs for all
// of K in LDS from the start.
#pragma once

#include "fp8.h"
#include "head_gemm.h"

namespace mo_f8 {

using namespace mo_head_gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

// One operand: `rows` rows of bytes at q, ld apart (ld < 2^23; 16-byte aligned, K a multiple of
// 128 bytes of them), and scales at s: row r's at s + (r >> shift) ld_s, inc apart.  Scales
// of rows are whole aligned dwords of four stages, inc 1.
struct Operand8 {
    const uint8_t *q, *s;
    int64_t ld, rows, ld_s, inc;
    int shift;
};

// Two slots of a stage, two of four stages' scales by rows, and P's in blocks (SQ).
constexpr int F8_MAX_STAGES = 8192;   // K up to 2^20
template <bool SQ> constexpr int f8_scale_rows(int NB) { return (SQ ? 0 : 256) + 64 * NB; }
template <bool SQ> constexpr int f8_lds(int NB) {
    return head_lds(NB) + 2 * f8_scale_rows<SQ>(NB) * 4 + (SQ ? 2 * F8_MAX_STAGES : 0);
}

// As head_tile: rows p0 .. of P and q0 .. of Q over nk stages from k0 on (a multiple of 4, as
// are the scales' row lengths), Layout and accumulators as there.
//
// A stage is MB row blocks of NBW MFMAs.  Up to the last two blocks, the fragments of the row
// blocks ahead are read; then every read of the stage is done, each wave waits for its loads
// of the next one and the barrier publishes it.  Beside the last two row blocks go the
// reads of the next stage's first fragments, each into registers that were just used, and
// the first loads of the stage after it.
template <int NB, bool SQ, class Acc>
__device__ __forceinline__ void f8_tile(uint8_t* smem, const Operand8& P, const Operand8& Q, int64_t p0, int64_t q0,
                                        int k0, int nk, Acc& acc) {
#ifdef __HIP_DEVICE_COMPILE__
    using L = Layout<NB>;
    constexpr int WN = L::WN, MB = L::MB, NBW = L::NBW;
    constexpr int TN = 64 * NB, SBYTES = HP_BYTES + TN * HKB, SROWS = f8_scale_rows<SQ>(NB);
    constexpr int LS = 4 + NB;                   // load instructions per stage and wave
    constexpr int RING = MB < 4 ? MB : 4, AHEAD = 2;        // fragments of P held
    static_assert(NBW == 4 && MB % RING == 0, "layout");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r16 = lane & 15, kg = lane >> 4;

    const int plim = int(P.rows - p0 < 256 ? P.rows - p0 : 256) - 1;
    const int qlim = int(Q.rows - q0 < TN ? Q.rows - q0 : TN) - 1;
    uint32_t vo[LS];
#pragma unroll
    for (int i = 0; i < LS; ++i) {
        const int r = (i < 4 ? wave * 32 + i * 8 : wave * 8 * NB + (i - 4) * 8) + (lane >> 3);
        const int lim = i < 4 ? plim : qlim;
        vo[i] = uint32_t(r < lim ? r : lim) * uint32_t(i < 4 ? P.ld : Q.ld) + uint32_t(((lane & 7) ^ hswz(r)) << 4);
    }
    const auto rP = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(P.q + p0 * P.ld + int64_t(k0) * HKB), 0, -1, 0x00027000);
    const auto rQ = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(Q.q + q0 * Q.ld + int64_t(k0) * HKB), 0, -1, 0x00027000);
    int koff = 0;   // of the stage being loaded
    auto issue1 = [&](int slot, int i) __attribute__((always_inline)) {
        uint8_t* sp = smem + slot * SBYTES + (i < 4 ? (wave * 32 + i * 8) * HKB : HP_BYTES + (wave * 8 * NB + (i - 4) * 8) * HKB);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(i < 4 ? rP : rQ, (lds_void_t*)sp, 16, vo[i], koff, 0, 0);
    };
    // Row 64 wave + lane of the 256 of P (not SQ) and TN of Q (the waves behind them load none): its
    // scales of four stages.
    const uint8_t* sg;
    {
        const int r = wave * 64 + lane - (SQ ? 0 : 256);
        if (r < 0) {
            sg = P.s + (p0 + (r + 256 < plim ? r + 256 : plim)) * P.ld_s;
        } else {
            const int64_t x = q0 + (r < qlim ? r : qlim);
            sg = Q.s + (x >> Q.shift) * Q.ld_s;
        }
        sg += k0;
    }
    uint8_t* const sl = smem + 2 * SBYTES;
    auto issue_scales = [&](int group) __attribute__((always_inline)) {
        if (wave * 64 < SROWS) {
            __builtin_amdgcn_global_load_lds(sg, (lds_void_t*)(sl + (group & 1) * (SROWS * 4) + wave * 256), 4, 0, 0);
            sg += 4;
        }
    };

#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    union Frag {
        i32x8 v;
        u32x4 h[2];
    };
    const int x0 = ((kg ^ hswz(r16)) << 4), x1 = x0 ^ 64;
    const int pbase = (wm * (MB * 16) + r16) * HKB, qbase = HP_BYTES + (wn * (NBW * 16) + r16) * HKB;
    Frag fa[RING], fb[NBW];
    auto rdp = [&](int slot, int a) __attribute__((always_inline)) {
        const uint8_t* p = smem + slot * SBYTES + pbase + a * 16 * HKB;
        fa[a % RING].h[0] = *reinterpret_cast<const u32x4*>(p + x0);
        fa[a % RING].h[1] = *reinterpret_cast<const u32x4*>(p + x1);
    };
    auto rdq = [&](int slot, int b) __attribute__((always_inline)) {
        const uint8_t* p = smem + slot * SBYTES + qbase + b * 16 * HKB;
        fb[b].h[0] = *reinterpret_cast<const u32x4*>(p + x0);
        fb[b].h[1] = *reinterpret_cast<const u32x4*>(p + x1);
    };
    constexpr int MS = SQ ? 1 : MB;
    uint32_t sp[MS], sq[NBW];   // the scales of this stage in the low byte, the next stages' above
    uint8_t* const st = sl + 2 * SROWS * 4;   // SQ: [block][stage]
    const int stl = (nk + 3) & ~3;
    auto rds = [&](int group) __attribute__((always_inline)) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(sl + (group & 1) * (SROWS * 4));
        if constexpr (SQ) {
            sp[0] = *reinterpret_cast<const uint32_t*>(st + (wm * (MB * 16) / F8_BLOCK) * stl + group * 4);
        } else {
#pragma unroll
            for (int a = 0; a < MB; ++a) sp[a] = p[wm * (MB * 16) + a * 16 + r16];
        }
#pragma unroll
        for (int b = 0; b < NBW; ++b) sq[b] = p[(SQ ? 0 : 256) + wn * (NBW * 16) + b * 16 + r16];
    };
    auto mfma = [&](int a, int b) __attribute__((always_inline)) {
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[a % RING].v, fb[b].v, acc[a][b], 0, 0, 0,
                                                                     int(sp[SQ ? 0 : a]), 0, int(sq[b]));
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int LH = MB == 2 ? LS : LS / 2;   // loads beside the last two row blocks
    const int kend = (nk - 1) * HKB;
    // One stage, in `slot`.  Behind the last stages the loads go on with the last stage's addresses,
    // into slots that nothing reads any more: one loop body, no ends peeled off it (the
    // compiler moved the accumulators between them through memory).
    auto stage = [&](int s, int slot) __attribute__((always_inline)) {
        if (s % 4 == 0) rds(s / 4);
#pragma unroll
        for (int a = 0; a < MB - 2; ++a)
#pragma unroll
            for (int b = 0; b < NBW; ++b) {
                mfma(a, b);
                if (a + AHEAD < MB && b == 0) rdp(slot, a + AHEAD);
                constexpr int N = (MB - 2) * NBW > 0 ? (MB - 2) * NBW : 1;
#pragma unroll
                for (int l = LH; l < LS; ++l)
                    if ((l - LH) * N / (LS - LH + (LS == LH)) + 1 == a * NBW + b) issue1(slot ^ 1, l);
                __builtin_amdgcn_sched_barrier(0);
            }
        if (MB != 2) koff = koff < kend ? koff + HKB : kend;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if ((s + 2) % 4 == 0 && s + 2 < nk) issue_scales((s + 2) / 4);
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
            mfma(MB - 2, b);
            if (RING > 2 && b < 2) rdp(slot ^ 1, b);
#pragma unroll
            for (int l = 0; l < LH; ++l)
                if (l * NBW / LH == b) issue1(slot, l);
            __builtin_amdgcn_sched_barrier(0);
            mfma(MB - 1, b);
            rdq(slot ^ 1, b);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (RING == 2) {
            rdp(slot ^ 1, 0);
            rdp(slot ^ 1, 1);
        }
        if (MB == 2) koff = koff < kend ? koff + HKB : kend;
#pragma unroll
        for (int a = 0; a < MS; ++a) sp[a] >>= 8;
#pragma unroll
        for (int b = 0; b < NBW; ++b) sq[b] >>= 8;
    };

    uint32_t s0 = 0;
    const int sblk = tid >> 8;   // P's block whose scales this thread fetches
    const bool swhole = p0 + sblk * F8_BLOCK < P.rows;
    const uint8_t* const sb = P.s + ((p0 >> 7) + (swhole ? sblk : 0)) * P.ld_s + int64_t(k0) * P.inc;
    if constexpr (SQ) {
        const int k = tid & 255;
        s0 = sb[(k < nk ? k : nk - 1) * P.inc];
    }
    issue_scales(0);
#pragma unroll
    for (int l = 0; l < LS; ++l) issue1(0, l);
    koff = koff < kend ? koff + HKB : kend;
#pragma unroll
    for (int l = 0; l < LH; ++l) issue1(1, l);   // the others in stage 0
    if (MB == 2) koff = koff < kend ? koff + HKB : kend;
    if constexpr (SQ) {
        for (int k = tid & 255; k < nk; k += 256) {
            st[sblk * stl + k] = uint8_t(s0);
            if (k + 256 < nk) s0 = sb[(k + 256) * P.inc];
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    }
    // stage 0 has landed
    if constexpr (LH == 4) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    else if constexpr (LH == 3) asm volatile("s_waitcnt vmcnt(3)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(5)" ::: "memory");
    static_assert(LH >= 3 && LH <= 5, "waits");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int b = 0; b < NBW; ++b) rdq(0, b);
    rdp(0, 0);
    rdp(0, 1);
    __builtin_amdgcn_sched_barrier(0);
    for (int s = 0; s < nk; ++s) stage(s, s & 1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#endif
}

}  // namespace mo_f8
