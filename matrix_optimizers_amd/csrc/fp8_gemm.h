// The tiled GEMM of the 8-bit operators, C[p][q] = sum_k P[p][k] Q[q][k], on MFMA with
// fp32 accumulators, for operands with K along their rows:
//   - both in 8 bits with a power-of-two scale for each block of 128 along K;
//   - both in 8 bits, multiplied as the bf16 numbers they stand for (VALUES8);
//   - both in bf16; or P in bf16 and Q as three bf16 planes whose sum is an fp32 value.
//
// 8 bits.  One instruction, 16 x 16 x 128 of e4m3 with e8m0 scales, takes a whole block, so
// the scales cost no arithmetic.  It holds its products to about 2^-17 of the largest of those
// it adds together before they go into the fp32 accumulator: measured against 64 bits,
// 1.5e-5 of the result's norm for normal data at any K, a hundredth of a bf16 rounding.
// A product whose result is fp32 is therefore not taken in 8 bits, but with the operands' values,
// whose products are exact in bf16 MFMA: VALUES8 brings 64 elements of K at a time through
// registers, where they are converted on their way to LDS.  It asks nothing of alignment, and takes
// the bf16 results of operands that cannot be loaded straight to LDS and are not worth a copy as well.
//
// Tiles, LDS rows of 128 bytes and their swizzle are those of the head's GEMM (head_gemm.h): a
// stage of 128 bytes per row is 64 elements of K in bf16, 128 in 8 bits, one block.  A lane's 32
// bytes of a row's stage are its chunks kg and kg + 4, in P and in Q alike: which element of K
// meets which lane does not matter as both sides agree.
//
// Weight gradients (TOKENS): K along both operands' columns, P in 8 bits, Q in bf16, read where
// they lie.  A stage is 64 rows (tokens) of 256 columns of P and 64 NB of Q, in bf16.  Both go
// through registers, two stages ahead: P for one conversion per two elements that applies
// the token's scale (q 2^e is a bf16 number, so exactly), Q because the compiler lets every
// transposing read wait for all loads to LDS under way (2258 us instead of 1705 for the case
// below).  The fragments come out of LDS through transposing reads: 16 lanes take 16 columns of four
// rows.  The granules of 16 columns (32 bytes) of a row are permuted so that the rows that 32
// lanes read together fall on different banks.  (With transposed copies made first, 16384
// tokens x 14336 x 4096 took 1705 us, 254 of them for the copies.)
//
// One workgroup per CU walks over its tiles and loads on across their ends: while a tile's last
// stages are multiplied, the next one's first are on their way, and its results are stored under the
// next tile's products.  16384 x 14336 x 4096 in 8 bits, one tile per workgroup: 845 us, of which 125
// were the stores that nothing hid.
//
// 16384 x 14336 x 4096 takes 735 to 796 us in 8 bits (2420 to 2620 TFLOP/s), where a library product of the same
// numbers with one scale each takes 630 to 690, and 1514 to 1625 as a weight gradient (the library's bf16 product along
// the tokens 1850 to 1960), by card: the clock is held at 1.76 and 2.0 GHz with MFMAs in 60 and 53 % of the cycles;
// fp32 results 1530 to 1580.  What lies beside the stages (1.4 us of 256 x 256 in 8 bits) is 8 us a tile, most of it
// 128 KB of results per CU at HBM's rate.  Workgroups started 2 to 4 us apart, so that they would not store together,
// took as long.
#pragma once

#include "fp8.h"
#include "head_gemm.h"

namespace mo_f8 {

using namespace mo_head_gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Kinds of operands: 8 bits with P's scales in blocks of 128 rows, or by rows; bf16; bf16 with Q
// in three planes; P in 8 bits and Q in bf16, both with K along their columns; 8 bits as values.
enum Kind { SQUARE8, ROWS8, BF16, BF16_3, TOKENS, VALUES8 };
constexpr bool is8(int kind) { return kind == SQUARE8 || kind == ROWS8; }

// One operand: `rows` rows of bytes at q, ld apart (16-byte aligned, K in whole stages, 256 ld
// < 2^31); plane p of three starts p * plane bytes further.  Scales at s: row r's at s +
// (r >> shift) ld_s, inc apart; those of rows are whole aligned dwords of four stages, inc 1.
// TOKENS: `rows` columns (of P a multiple of 16, of Q of 8) of `tokens` rows, 64 ld < 2^31.  VALUES8: `tokens`
// elements in a row, no alignment, 256 ld and 256 ld_s < 2^31.
struct Operand8 {
    const uint8_t *q, *s;
    int64_t ld, rows, plane, ld_s, inc;
    int shift;
    int64_t tokens;
};

// A product's tiles (tm x tn, 256 x 64 nb): the first `full` of them over all of K, the `rem` others
// in `splits` parts of `per` stages each, whose sums go to `part`: [tile - full][split][wave][MB x NBW][lane].
struct Tiles {
    uint32_t tm, tn, full, rem, splits, band;
    int nk, per;
    f32x4* part;
};

// Tile i in order: bands of `band` tile rows, column by column, so that the 32 tiles an XCD runs at
// once share the band's panels of P, and keep them, and few of Q.  Bands of 4, 8, 16 rows: 16384 x 14336 x
// 4096 in 8 bits 752, 742, 765 us; its weight gradient, where P's panels have half the bytes
// of Q's, 1605, 1565, 1548.
MO_DEV void tile_at(const Tiles& t, uint32_t i, uint32_t* ti, uint32_t* tj) {
    const uint32_t band = i / (t.band * t.tn), r = i - band * t.band * t.tn;
    const uint32_t h = t.tm - band * t.band < t.band ? t.tm - band * t.band : t.band;
    *ti = band * t.band + r % h;
    *tj = r / h;
}

// What a workgroup multiplies at a time.
struct Item {
    uint32_t ti, tj, slot;
    int k0, nk;
    bool split;
};

// Item n of this workgroup: its share of the full tiles (each XCD a contiguous share, its
// workgroups side by side), then of the parts.  False behind the last.
MO_DEV bool item_of(const Tiles& t, uint32_t n, Item* it) {
    const uint32_t grid = gridDim.x, rounds = (t.full + grid - 1) / grid;
    uint32_t tile;
    if (n < rounds) {
        const uint32_t b = blockIdx.x + n * grid, x = b & 7, j = b >> 3, share = t.full >> 3, rem = t.full & 7;
        if (j >= share + (x < rem ? 1u : 0u)) return false;   // (the last round, and then there are no parts)
        tile = x * share + (x < rem ? x : rem) + j;
        it->k0 = 0;
        it->nk = t.nk;
        it->split = false;
    } else {
        const uint32_t parts = t.rem * t.splits, b = blockIdx.x + (n - rounds) * grid;
        const uint32_t x = b & 7, j = b >> 3, share = parts >> 3, rem = parts & 7;
        if (j >= share + (x < rem ? 1u : 0u)) return false;
        const uint32_t i = x * share + (x < rem ? x : rem) + j, s = i / t.rem;
        tile = i - s * t.rem;
        it->slot = tile * t.splits + s;
        tile += t.full;
        it->k0 = int(s) * t.per;
        it->nk = t.nk - it->k0 < t.per ? t.nk - it->k0 : t.per;
        it->split = true;
    }
    tile_at(t, tile, &it->ti, &it->tj);
    return true;
}

template <int KIND> constexpr int scale_rows(int NB) { return is8(KIND) ? (KIND == SQUARE8 ? 0 : 256) + 64 * NB : 0; }
// Narrow tiles multiply a stage sooner than memory answers, and leave room for a third slot in LDS (us of 64
// stages of 64 x 4096, tiles of 64: bf16 46 with two, 35 with three; 112 stages of 512 x 4096 in 8 bits 87 and
// 65).  Kinds that go through registers wait for other things: a second set of registers changed nothing.
constexpr bool direct(int kind) { return kind != TOKENS && kind != VALUES8; }   // straight to LDS
template <int KIND> constexpr int slots(int NB) { return direct(KIND) && NB < 4 ? 3 : 2; }
// The slots of a stage, and four of four stages' scales by rows.
template <int KIND> constexpr int gemm_lds(int NB) { return head_lds(NB) / 2 * slots<KIND>(NB) + 4 * scale_rows<KIND>(NB) * 4; }

// Stores behind which a barrier's loads may be waited for without them.
template <int NB> constexpr int STORES = Layout<NB>::MB * Layout<NB>::NBW / 2;

// Runs over the workgroup's items and hands each one's accumulators to store(item, wave, lane,
// acc), acc f32x4[MB][NBW] as in head_tile; store returns whether it has issued STORES<NB> stores
// at least.  All operand checks are the host's.
//
// A stage is MB row blocks of NBW blocks of MFMAs, two rows at a time, column by column (a column's
// fragment of Q is then read in good time before its first use in the next stage: on one card 752
// us for the product of 16384 x 14336 x 4096 and 1605 for its weight gradient, row by row 795 and 1690).  Up to
// the last pair, the fragments of the next pair are read; then every read of the stage is done, each
// wave waits for its loads of the next one and the barrier publishes it.  Beside the last pair
// go the reads of the next stage's first fragments, each into registers that were just used, and the
// loads of the stage after it.  One loop body for all stages: with peeled ends the compiler moved
// the accumulators between them through memory.
template <int NB, int KIND, class Store>
__device__ __forceinline__ void run_tiles(uint8_t* smem, const Operand8& P, const Operand8& Q, const Tiles& t,
                                          const Store& store) {
#ifdef __HIP_DEVICE_COMPILE__
    using L = Layout<NB>;
    constexpr int WN = L::WN, MB = L::MB, NBW = L::NBW;
    constexpr int TN = 64 * NB, SBYTES = HP_BYTES + TN * HKB, SROWS = scale_rows<KIND>(NB);
    constexpr int LS = 4 + NB;                   // load instructions per stage and wave
    constexpr int SLOTS = slots<KIND>(NB);
    constexpr int RING = MB < 4 ? MB : 4;        // fragments of P held
    static_assert(MB % RING == 0, "layout");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r16 = lane & 15, kg = lane >> 4;

    auto rsrc = [&](const uint8_t* p) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, -1, 0x00027000);
    };

    // ---- the loads' own walk over the items: always as many stages ahead as there are slots ----
    Item li;
    uint32_t ln = 0;
    bool more = item_of(t, 0, &li);
    if (!more) return;
    constexpr bool TOK = KIND == TOKENS, VAL = KIND == VALUES8;
    constexpr int QROW = TN * 2, QCH = QROW / 16;   // TOKENS: bytes and 16-byte chunks of a row of Q in a stage
    // TOKENS: how row r's granules of 16 columns are permuted (Q's rows of 64 columns: two rows share the banks)
    auto pf = [&](int r) __attribute__((always_inline)) { return (r & 3) | (((r >> 1) ^ (r >> 2)) & 4); };
    auto qf = [&](int r) __attribute__((always_inline)) {
        return NB == 1 ? ((r >> 1) & 1) | (((r >> 2) ^ (r >> 3)) & 2) : pf(r);
    };
    int ls = 0, lseg = 0, koff = 0, lgroup = 0;   // stage of the item, plane, byte offset, group of scales
    uint32_t vo[LS];
    auto rP = rsrc(P.q), rQ = rsrc(Q.q);
    constexpr int SI = (SROWS / 64 + 7) / 8 > 0 ? (SROWS / 64 + 7) / 8 : 1;
    const uint8_t* sg[SI];
    // The lane, out of the compiler's sight: what is computed from it once per item is not kept in
    // registers over the stages.
    auto lane_here = [&]() __attribute__((always_inline)) {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    };
    // TOKENS: the operands from the first row of stage ls on.  What lies behind the last token reads as
    // zeros; columns behind the last (or the next row's in their place) are not stored.
    auto rS = rsrc(P.s);
    auto enter_rows = [&]() __attribute__((always_inline)) {
        const int64_t t0 = (int64_t(li.k0) + ls) * 64, left = (P.tokens - t0 < 64 ? P.tokens - t0 : 64) - 1;
        const int64_t p = int64_t(li.ti) * 256, q = int64_t(li.tj) * QROW;
        auto upto = [&](const uint8_t* from, int64_t bytes) __attribute__((always_inline)) {
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(from), 0, int(bytes), 0x00027000);
        };
        rP = upto(P.q + t0 * P.ld + p, left * P.ld + P.rows - p);
        rS = upto(P.s + t0 * P.ld_s + (p >> 7), left * P.ld_s + ((P.rows + 127) >> 7) - (p >> 7));
        rQ = upto(Q.q + t0 * Q.ld + q, left * Q.ld + Q.rows * 2 - q);
    };
    // VALUES8: a thread takes 16 bytes of VP rows of P and VQ of Q, 64 bytes of a row by four threads.
    constexpr int VP = 2, VQ = NB == 4 ? 2 : 1, VR = NB == 1 ? 64 : 128;
    uint32_t oP[VP], oQ[VQ], oSP[VP], oSQ[VQ];
    auto enter_values = [&]() __attribute__((always_inline)) {
        const int64_t p0 = int64_t(li.ti) * 256, q0 = int64_t(li.tj) * TN;
        const int plim = int(P.rows - p0 < 256 ? P.rows - p0 : 256) - 1;
        const int qlim = int(Q.rows - q0 < TN ? Q.rows - q0 : TN) - 1;
        const int r = (lane_here() + wave * 64) >> 2, c = (lane_here() & 3) * 16;
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const int x = r + 128 * i < plim ? r + 128 * i : plim;
            oP[i] = uint32_t(x) * uint32_t(P.ld) + c;
            oSP[i] = uint32_t(((p0 + x) >> P.shift) - (p0 >> P.shift)) * uint32_t(P.ld_s);
        }
#pragma unroll
        for (int i = 0; i < VQ; ++i) {
            const int y = (r & (VR - 1)) + 128 * i, x = y < qlim ? y : qlim;
            oQ[i] = uint32_t(x) * uint32_t(Q.ld) + c;
            oSQ[i] = uint32_t(((q0 + x) >> Q.shift) - (q0 >> Q.shift)) * uint32_t(Q.ld_s);
        }
    };
    // Sets the addresses to the start of item li.  Rows past an operand's end are its last row.
    auto enter = [&]() __attribute__((always_inline)) {
        const int lane = lane_here();
        const int64_t p0 = int64_t(li.ti) * 256, q0 = int64_t(li.tj) * TN;
        ls = lseg = koff = 0;
        if constexpr (TOK) {
            enter_rows();
            return;
        }
        if constexpr (VAL) {
            enter_values();
            return;
        }
        const int plim = int(P.rows - p0 < 256 ? P.rows - p0 : 256) - 1;
        const int qlim = int(Q.rows - q0 < TN ? Q.rows - q0 : TN) - 1;
#pragma unroll
        for (int i = 0; i < LS; ++i) {
            const int r = (i < 4 ? wave * 32 + i * 8 : wave * 8 * NB + (i - 4) * 8) + (lane >> 3);
            const int lim = i < 4 ? plim : qlim;
            vo[i] = uint32_t(r < lim ? r : lim) * uint32_t(i < 4 ? P.ld : Q.ld) + uint32_t(((lane & 7) ^ hswz(r)) << 4);
        }
        rP = rsrc(P.q + p0 * P.ld + int64_t(li.k0) * HKB);
        rQ = rsrc(Q.q + q0 * Q.ld + int64_t(li.k0) * HKB + (KIND == BF16_3 ? 2 * Q.plane : 0));
        if constexpr (SROWS > 0)
#pragma unroll
            for (int i = 0; i < SI; ++i) {
                const int r = (wave + 8 * i) * 64 + lane - (KIND == SQUARE8 ? 0 : 256);
                if (r < 0) {
                    sg[i] = P.s + (p0 + (r + 256 < plim ? r + 256 : plim)) * P.ld_s + li.k0;
                } else {
                    const int64_t x = q0 + (r < qlim ? r : qlim);
                    sg[i] = Q.s + (x >> Q.shift) * Q.ld_s + li.k0;
                }
            }
    };
    enter();
    auto issue1 = [&](int slot, int i) __attribute__((always_inline)) {
        uint8_t* sp = smem + slot * SBYTES + (i < 4 ? (wave * 32 + i * 8) * HKB : HP_BYTES + (wave * 8 * NB + (i - 4) * 8) * HKB);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(i < 4 ? rP : rQ, (lds_void_t*)sp, 16, vo[i], koff, 0, 0);
    };
    // Rows 64 (wave + 8 i) + lane of P's (by rows) and Q's scales: one dword, four stages.
    uint8_t* const sl = smem + SLOTS * SBYTES;
    auto issue_scales = [&]() __attribute__((always_inline)) {
        if constexpr (SROWS > 0) {
            if (ls % 4 != 0 || !more) return;
#pragma unroll
            for (int i = 0; i < SI; ++i)
                if ((wave + 8 * i) * 64 < SROWS) {
                    __builtin_amdgcn_global_load_lds(sg[i], (lds_void_t*)(sl + (lgroup & 3) * (SROWS * 4) + (wave + 8 * i) * 256),
                                                     4, 0, 0);
                    sg[i] += 4;
                }
            ++lgroup;
        }
    };
    // To the next stage.  Behind the last item the loads go on with its last stage, into slots that
    // nothing reads any more.
    auto advance = [&]() __attribute__((always_inline)) {
        if (++ls < li.nk) {
            koff += HKB;
            if constexpr (TOK) enter_rows();
        } else if (KIND == BF16_3 && lseg < 2 && more) {
            ++lseg;
            ls = koff = 0;
            rQ = rsrc(Q.q + int64_t(li.tj) * TN * Q.ld + int64_t(li.k0) * HKB + (2 - lseg) * Q.plane);
        } else if (more && (more = item_of(t, ++ln, &li))) {
            enter();
        }
    };

    // TOKENS: a thread takes 16 columns of two rows of P and eight of NB rows of Q.
    constexpr int QR = 512 / QCH;   // rows of Q that the workgroup loads at a time
    u32x4 xq[2], yq[NB];
    uint32_t xscale[2] = {0, 0};
    const uint32_t vP = uint32_t(tid >> 4) * uint32_t(P.ld) + (tid & 15) * 16;
    const uint32_t vS = uint32_t(tid >> 4) * uint32_t(P.ld_s) + ((tid >> 3) & 1);
    const uint32_t vQ = uint32_t(tid / QCH) * uint32_t(Q.ld) + uint32_t(tid % QCH) * 16;
    // (a row's whole offset is the vector one: the descriptor's range does not hold for a scalar offset)
    auto load_p = [&](int i) __attribute__((always_inline)) {
        xq[i] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rP, vP + uint32_t(32 * i) * uint32_t(P.ld), 0, 0));
        xscale[i] = __builtin_amdgcn_raw_buffer_load_b8(rS, vS + uint32_t(32 * i) * uint32_t(P.ld_s), 0, 0);
    };
    auto load_q = [&](int i) __attribute__((always_inline)) {
        yq[i] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rQ, vQ + uint32_t(QR * i) * uint32_t(Q.ld), 0, 0));
    };
    auto store_p = [&](int slot, int i) __attribute__((always_inline)) {
        const int r = (tid >> 4) + 32 * i, g = tid & 15;
        uint8_t* to = smem + slot * SBYTES + r * 512 + ((g ^ pf(r)) << 5);
        // (the conversion takes the exponent's field, with 0 and 255 as in e8m0)
        const float f = __uint_as_float(xscale[i] << 23);
        u32x4 w[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e / 2][e % 2 * 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(xq[i][e], f, false));
            w[e / 2][e % 2 * 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(xq[i][e], f, true));
        }
        // half the lanes write their second eight columns first: 16 lanes then fall on all banks
        const bool odd = (g & 8) != 0;
        u32x4 a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) { a[e] = odd ? w[1][e] : w[0][e]; b[e] = odd ? w[0][e] : w[1][e]; }
        *reinterpret_cast<u32x4*>(to + (odd ? 16 : 0)) = a;
        *reinterpret_cast<u32x4*>(to + (odd ? 0 : 16)) = b;
    };
    auto store_q = [&](int slot, int i) __attribute__((always_inline)) {
        const int r = tid / QCH + QR * i, c = tid % QCH;
        *reinterpret_cast<u32x4*>(smem + slot * SBYTES + HP_BYTES + r * QROW + ((c ^ (qf(r) << 1)) << 4)) = yq[i];
    };
    // Piece j of the stage in registers goes to LDS, and the one after it comes into its place.
    auto piece = [&](int slot, int j) __attribute__((always_inline)) {
        if (j < 2) {
            store_p(slot, j);
            load_p(j);
        } else {
            store_q(slot, j - 2);
            load_q(j - 2);
        }
    };

    // VALUES8: a stage into registers, and from there, as bf16, to its slot.
    u32x4 vp[VP], vq[VQ];
    uint32_t vsp[VP], vsq[VQ];
    auto load_values = [&]() __attribute__((always_inline)) {
        typedef u32x4 u32x4_e1 __attribute__((aligned(1)));
        const int st = li.k0 + (ls < li.nk ? ls : li.nk - 1);
        const int64_t p0 = int64_t(li.ti) * 256, q0 = int64_t(li.tj) * TN, k = int64_t(st) * 64;
        const uint8_t *p = P.q + p0 * P.ld + k, *q = Q.q + q0 * Q.ld + k;
        const uint8_t *ps = P.s + (p0 >> P.shift) * P.ld_s + (st >> 1) * P.inc;
        const uint8_t *qs = Q.s + (q0 >> Q.shift) * Q.ld_s + (st >> 1) * Q.inc;
        if (k + 64 <= P.tokens) {
#pragma unroll
            for (int i = 0; i < VP; ++i) vp[i] = *reinterpret_cast<const u32x4_e1*>(p + oP[i]);
#pragma unroll
            for (int i = 0; i < VQ; ++i) vq[i] = *reinterpret_cast<const u32x4_e1*>(q + oQ[i]);
        } else {
            const int n = int(P.tokens - k) - (tid & 3) * 16;
            auto part = [&](const uint8_t* x) __attribute__((always_inline)) {
                const u32x2 lo = ldq8(x, n), hi = ldq8(x + 8, n - 8);
                return u32x4{lo[0], lo[1], hi[0], hi[1]};
            };
#pragma unroll
            for (int i = 0; i < VP; ++i) vp[i] = part(p + oP[i]);
#pragma unroll
            for (int i = 0; i < VQ; ++i) vq[i] = part(q + oQ[i]);
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) vsp[i] = ps[oSP[i]];
#pragma unroll
        for (int i = 0; i < VQ; ++i) vsq[i] = qs[oSQ[i]];
    };
    auto store_values = [&](int slot) __attribute__((always_inline)) {
        auto put = [&](uint8_t* to, int r, u32x4 x, uint32_t scale) __attribute__((always_inline)) {
            const float f = __uint_as_float(scale << 23);   // (the conversion takes the exponent's field, as in e8m0)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * h + e], f, false));
                    w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * h + e], f, true));
                }
                *reinterpret_cast<u32x4*>(to + r * HKB + (((tid & 3) * 2 + h) ^ hswz(r)) * 16) = w;
            }
        };
        uint8_t* to = smem + slot * SBYTES;
#pragma unroll
        for (int i = 0; i < VP; ++i) put(to, (tid >> 2) + 128 * i, vp[i], vsp[i]);
#pragma unroll
        for (int i = 0; i < VQ; ++i) put(to + HP_BYTES, ((tid >> 2) & (VR - 1)) + 128 * i, vq[i], vsq[i]);
    };

    union Frag {
        i32x8 v;
        u32x4 h[2];
    };
    const int x0 = ((kg ^ hswz(r16)) << 4), x1 = x0 ^ 64;
    // TOKENS: row kg 8 + r16 / 4 (+ 4 and + 32), columns 4 (r16 % 4) .. of a granule
    const int trow = kg * 8 + (r16 >> 2);
    const int pbase = TOK ? trow * 512 + (((wm * MB) ^ pf(trow)) << 5) + (r16 & 3) * 8 : (wm * (MB * 16) + r16) * HKB;
    const int qbase = HP_BYTES + (TOK ? trow * QROW + (((wn * NBW) ^ qf(trow)) << 5) + (r16 & 3) * 8
                                      : (wn * (NBW * 16) + r16) * HKB);
    Frag fa[RING], fb[NBW];
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    // a fragment of 16 columns through four transposing reads
    auto tr = [&](Frag& f, const uint8_t* p, int row) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                              (lds_s16x4*)(p + (h * 32 + j * 4) * row)));
                f.h[h][2 * j] = x[0];
                f.h[h][2 * j + 1] = x[1];
            }
    };
    auto rdp = [&](int slot, int a) __attribute__((always_inline)) {
        if constexpr (TOK) {
            tr(fa[a % RING], smem + slot * SBYTES + (pbase ^ (a << 5)), 512);
            return;
        }
        const uint8_t* p = smem + slot * SBYTES + pbase + a * 16 * HKB;
        fa[a % RING].h[0] = *reinterpret_cast<const u32x4*>(p + x0);
        fa[a % RING].h[1] = *reinterpret_cast<const u32x4*>(p + x1);
    };
    auto rdq = [&](int slot, int b) __attribute__((always_inline)) {
        if constexpr (TOK) {
            tr(fb[b], smem + slot * SBYTES + (qbase ^ (b << 5)), QROW);
            return;
        }
        const uint8_t* p = smem + slot * SBYTES + qbase + b * 16 * HKB;
        fb[b].h[0] = *reinterpret_cast<const u32x4*>(p + x0);
        fb[b].h[1] = *reinterpret_cast<const u32x4*>(p + x1);
    };
    // This stage's scales.  P's in blocks of 128 rows are one for all rows of a wavefront: lane l of
    // pblock holds that of stage l of 64.
    constexpr int MS = KIND == ROWS8 ? MB : 1;
    uint32_t sp[MS], sq[NBW], pblock = 0, pnext = 0;
    auto rds = [&](int group, int k) __attribute__((always_inline)) {
        const uint8_t* p = sl + (group & 3) * (SROWS * 4) + r16 * 4 + k;
        if constexpr (KIND == ROWS8)
#pragma unroll
            for (int a = 0; a < MB; ++a) sp[a] = p[(wm * (MB * 16) + a * 16) * 4];
#pragma unroll
        for (int b = 0; b < NBW; ++b) sq[b] = p[((KIND == SQUARE8 ? 0 : 256) + wn * (NBW * 16) + b * 16) * 4];
    };
    auto load_block = [&](const Item& it, int s) __attribute__((always_inline)) {
        const int64_t row = int64_t(it.ti) * 256 + wm * (MB * 16), k = s + lane_here();
        const uint8_t* p = P.s + ((row < P.rows ? row : P.rows - 1) >> 7) * P.ld_s;
        pnext = p[(it.k0 + (k < it.nk ? k : it.nk - 1)) * P.inc];
    };
    f32x4 acc[MB][NBW];
    auto mfma = [&](int a, int b) __attribute__((always_inline)) {
        f32x4& c = acc[a][b];
        const Frag &x = fa[a % RING], &y = fb[b];
        if constexpr (is8(KIND)) {
            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, c, 0, 0, 0, int(sp[KIND == ROWS8 ? a : 0]), 0,
                                                                 int(sq[b]));
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.h[h]),
                                                            __builtin_bit_cast(bf16x8, y.h[h]), c, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    int stored = 0;   // 1: STORES stores or more are behind the loads that the next barrier waits for
    // Everything that branches is done first: the compiler moves MFMAs down across branches, and the
    // reads of their next operands then go to other registers.
    auto stage = [&](const Item& it, int s, int slot, int next, int group) __attribute__((always_inline)) {
        advance();
        issue_scales();
        if constexpr (VAL) {
            store_values(next);
            load_values();
        }
        if constexpr (KIND == SQUARE8) {
            if (s % 64 == 0) {
                if (s > 0) pblock = pnext;
                if (s + 64 < it.nk) load_block(it, s + 64);
            }
            sp[0] = uint32_t(__builtin_amdgcn_readlane(int(pblock), s & 63));
        }
        if constexpr (is8(KIND)) rds(group, s & 3);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int a = 0; a < MB - 2; a += 2)
#pragma unroll
            for (int b = 0; b < NBW; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mfma(a + i, b);
                    if (i == 0 && b < 2) rdp(slot, a + 2 + b);
                    if constexpr (TOK)
#pragma unroll
                        for (int j = 0; j < 2 + NB; ++j)
                            if (j * (MB - 2) * NBW / (2 + NB) + 1 == a * NBW + 2 * b + i) piece(next, j);
                    __builtin_amdgcn_sched_barrier(0);
                }
        if constexpr (TOK && MB == 2)
#pragma unroll
            for (int j = 0; j < 2 + NB; ++j) piece(next, j);
        if constexpr (direct(KIND))
            asm volatile("s_cmp_eq_u32 %0, 0\n"
                     "s_cbranch_scc1 .Lall%=\n"
                     "s_waitcnt vmcnt(%1)\n"
                     "s_branch .Lgo%=\n"
                     ".Lall%=: s_waitcnt vmcnt(%2)\n"
                     ".Lgo%=:" ::"s"(__builtin_amdgcn_readfirstlane(stored)), "n"((SLOTS - 2) * LS + STORES<NB>),
                     "n"((SLOTS - 2) * LS) : "memory", "scc");
        stored = 0;
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
            mfma(MB - 2, b);
            if (RING > 2 && b < 2) rdp(next, b);
            if constexpr (direct(KIND))
#pragma unroll
                for (int l = 0; l < LS; ++l)
                    if (l * NBW / LS == b) issue1(slot, l);
            __builtin_amdgcn_sched_barrier(0);
            mfma(MB - 1, b);
            rdq(next, b);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (RING == 2) {
            rdp(next, 0);
            rdp(next, 1);
        }
    };

    Item it = li;
    if constexpr (KIND == SQUARE8) load_block(it, 0);
    if constexpr (TOK) {
        load_p(0);
        load_p(1);
#pragma unroll
        for (int i = 0; i < NB; ++i) load_q(i);
        advance();
#pragma unroll
        for (int j = 0; j < 2 + NB; ++j) piece(0, j);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    } else if constexpr (VAL) {
        load_values();
        store_values(0);
        advance();
        load_values();
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    } else {
        for (int s = 0; s < SLOTS; ++s) {
            if (s) advance();
            issue_scales();
#pragma unroll
            for (int l = 0; l < LS; ++l) issue1(s, l);
        }
    }
    // stage 0 has landed (the others' LS loads each, and dwords of scales, came after it)
    if constexpr (direct(KIND)) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((SLOTS - 1) * LS) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int b = 0; b < NBW; ++b) rdq(0, b);
    rdp(0, 0);
    rdp(0, 1);
    __builtin_amdgcn_sched_barrier(0);
    int slot = 0, group = 0;
    for (uint32_t n = 0;;) {
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int b = 0; b < NBW; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (KIND == SQUARE8) pblock = pnext;
        Item next;
        const bool have = item_of(t, ++n, &next);
        if constexpr (KIND == SQUARE8)
            if (have && it.nk <= 64) load_block(next, 0);
        const int stages = it.nk * (KIND == BF16_3 ? 3 : 1);
#pragma clang loop unroll(disable)
        for (int s = 0; s < stages; ++s) {
            const int next = SLOTS == 2 ? slot ^ 1 : slot + 1 == SLOTS ? 0 : slot + 1;
            stage(it, s, slot, next, group);
            slot = next;
            if (is8(KIND) && s % 4 == 3) ++group;
        }
        if (is8(KIND) && stages % 4) ++group;
        if constexpr (KIND == SQUARE8)
            if (have && it.nk > 64) load_block(next, 0);
        stored = store(it, wave, lane_here(), acc) ? 1 : 0;
        if (!have) break;
        it = next;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (the loads behind the last stage write LDS)
#endif
}

}  // namespace mo_f8
