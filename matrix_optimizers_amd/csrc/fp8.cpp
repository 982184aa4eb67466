// Host side of the 8-bit operators: casts, the product of two matrices in 8 bits and the
// weight's gradient from an activation in 8 bits.  Argument checks, workspace plans and
// launches; the kernels are in fp8_cast.hip and fp8_gemm.hip.  As in operators.cpp every
// plan follows from sizes and alignments alone, and nothing is uploaded or allocated.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/mo.h"
#include "operator_host.h"
#include "operators.h"

using namespace mo_host;

namespace {

constexpr int64_t kBlock = 128;
constexpr int64_t kCastRows = int64_t(1) << 32, kCastCols = int64_t(1) << 24;
// Rows and K of a product and both sides of a weight: tile and block counts stay in 32 bits.
constexpr int64_t kMaxSide = int64_t(1) << 20;

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

mo_status cast_shape(int64_t rows, int64_t cols, int32_t dtype, int64_t max_rows, int64_t max_cols) {
    if (rows < 0 || cols < 0) return MO_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || rows > max_rows || cols > max_cols) return MO_ERR_UNSUPPORTED;
    return MO_OK;
}

int64_t scale_rows(const MoF8Operand& o) { return o.shift ? blocks_of(o.rows) : o.rows; }

// A matrix in 8 bits of `cols` columns; its pointers are checked where it has elements.
mo_status operand_of(const mo_fp8_matrix* m, int64_t cols, MoF8Operand* o) {
    if (!m || m->rows < 0) return MO_ERR_INVALID_ARG;
    if (m->block_rows != 1 && m->block_rows != int32_t(kBlock)) return MO_ERR_INVALID_ARG;
    if (m->rows > kMaxSide) return MO_ERR_UNSUPPORTED;
    *o = {};
    o->q = m->q;
    o->s = m->scales;
    o->rows = m->rows;
    o->shift = m->block_rows == 1 ? 0 : 7;
    MO_TRY(stride_of(m->ld_q, cols, &o->ld));
    // the scales by rows, or by columns (the transpose of others)
    o->inc = m->inc_scales ? m->inc_scales : 1;
    if (o->inc == 1) {
        MO_TRY(stride_of(m->ld_scales, blocks_of(cols), &o->ld_s));
    } else {
        if (m->ld_scales != 1) return MO_ERR_INVALID_ARG;
        o->ld_s = 1;
        MO_TRY(stride_of(m->inc_scales, scale_rows(*o), &o->inc));
    }
    return m->rows && cols && (!m->q || !m->scales) ? MO_ERR_INVALID_ARG : MO_OK;
}

void operand_ranges(const MoF8Operand& o, int64_t cols, Ranges* r) {
    const int64_t n = scale_rows(o), b = blocks_of(cols);
    r->add(matrix_range(o.q, o.rows, cols, o.ld, 1, 0));
    r->add(o.inc == 1 ? matrix_range(o.s, n, b, o.ld_s, 1, 0) : matrix_range(o.s, b, n, o.inc, 1, 0));
}

// us of a stage (128 bytes of K) of a tile of 256 x 256, 128 and 64, one tile per CU: in 8 bits, from 8 bits
// converted, in bf16, and a weight gradient's from the operands as they lie.
struct StageTimes { double t[3]; };
constexpr StageTimes kStage8 = {{1.5, 0.85, 0.6}}, kStageValues = {{1.5, 1.0, 0.8}}, kStageBf16 = {{1.35, 0.78, 0.55}},
                     kStageTokens = {{1.72, 1.15, 0.9}};

// Estimated us of a product in `tiles` tiles with `stages` stages of `stage` us on 256 CUs.  The rounds that
// fill them take a tile's K whole; the tiles left over are split into the parts (multiples of `unit` stages)
// that take the least.  The parts' fp32 sums are written, read and added by a second launch.  Of 15
// products from 40 x 28672 x 8192 to 4096 x 4096 x 4096 in both result types, the choice is within 5 % of the best of
// all widths and up to 16 parts in most, and within 12 % of it in all.
double product_us(int64_t tiles, int64_t stages, double stage, int nb, int unit, int64_t* full, int64_t* splits) {
    const int64_t rem = tiles % 256;
    const double whole = double(tiles / 256 * stages) * stage;
    double least = whole + (rem ? double(stages) * stage : 0);
    *full = tiles;
    *splits = 1;
    for (int64_t k = 2; rem && k <= std::min(256 / rem, (stages + unit - 1) / unit); ++k) {
        const double t = whole + double((stages + k - 1) / k) * stage + double(rem * k * nb) * 0.026 + double(k) * 0.1 + 4;
        if (t < least) {
            least = t;
            *full = tiles - rem;
            *splits = k;
        }
    }
    return least;
}

// Tiles and parts of a product with `p` rows along 256 and `q` along 64 nb; its estimated us.
double plan_tiles(MoF8Plan* plan, int64_t p, int64_t q, int64_t stages, const StageTimes& times, double planes, int unit,
                Carve* take) {
    double least = 0;
    int64_t splits = 1, full = 0;
    for (int i = 0; i < 3; ++i) {
        const int nb = 4 >> i;
        int64_t f, k;
        const double t = product_us((p + 255) / 256 * ((q + 64 * nb - 1) / (64 * nb)), stages, times.t[i] * planes, nb, unit,
                                    &f, &k);
        if (i == 0 || t < least) {
            least = t;
            plan->nb = nb;
            full = f;
            splits = k;
        }
    }
    plan->tm = uint32_t((p + 255) / 256);
    plan->tn = uint32_t((q + 64 * plan->nb - 1) / (64 * plan->nb));
    plan->full = uint32_t(full);
    plan->nk = int(stages);
    plan->stages = int(((stages + splits - 1) / splits + unit - 1) / unit * unit);
    plan->splits = int((stages + plan->stages - 1) / plan->stages);
    if (uint64_t rem = uint64_t(plan->tm) * plan->tn - full)
        plan->off_part = (*take)(rem * plan->splits * 256 * 64 * plan->nb * 4);
    return least;
}

// Whether the rows can be loaded straight to LDS: whole blocks, 16-byte aligned rows.
bool q_in_place(const MoF8Operand& o, int64_t dim) {
    return dim % kBlock == 0 && ((reinterpret_cast<uintptr_t>(o.q) | uintptr_t(o.ld)) & 15) == 0;
}
// Whether the scales can: four stages' at a time, so whole aligned dwords.
bool s_in_place(const MoF8Operand& o, int64_t dim) {
    return o.inc == 1 && blocks_of(dim) % 4 == 0 && ((reinterpret_cast<uintptr_t>(o.s) | uintptr_t(o.ld_s)) & 3) == 0;
}

// Estimated us of a product in small blocks, 16 rb rows of P (K along both) by 16 tb of Q per workgroup, `slots` of
// them on the card at a time: `start`, then a workgroup's own time for a share of K (every eighth block, so
// `turns` of them) or that of all workgroups, whichever is more; behind the fourth turn the L2 no longer holds what
// the workgroups read.  Of 4 x 4 a CU holds one, and rounds are whole.
struct SmallBlocks {
    int tb, rb, slots;
    double start, own, all0, all;
    double us(int64_t p, int64_t q, double turns) const {
        const int64_t n = ((p + 16 * rb - 1) / (16 * rb)) * ((q + 16 * tb - 1) / (16 * tb));
        if (n >= int64_t(1) << 20) return 1e30;
        const double rounds = slots == 256 ? double((n + 255) / 256) : double(n) / slots;
        const double longer = 1 + std::min(0.4, 0.1 * std::max(0.0, turns - 4)) * (slots == 256 ? 0.5 : 1);
        return start + std::max(own * turns, rounds * (all0 + all * turns * longer));
    }
};
constexpr SmallBlocks kSmall[] = {{1, 1, 512, 3.1, 0.36, 1.07, 0.53},
                                  {1, 2, 512, 3.1, 0.48, 1.1, 0.95},
                                  {2, 2, 512, 3.1, 0.69, 1.35, 1.25},
                                  {4, 4, 256, 1.5, 0, 2.7, 1.85}};

// A product in small blocks, without a workspace and in one launch, where that takes less than in tiles.
// The estimates come from these and others like them, us of the kernels in tiles and in the small blocks of the
// first to last kind above, bf16 results: 16 tokens x 4096 x 4096 16.1, 4.8 5.4 6.4 10.7; 64 x 4096 x 4096 16.1, 9.8
// 8.1 7.2 11.7; 64 x 14336 x 4096 19.9, 26.3 20.2 17.9 15.7; 18 x 1792 x 12672 19.4, 8.4 9.9 12.3 22.1; 512 x 2048
// x 2048 13.9, 19.5 13.5 10.4 8.1; 512 x 4096 x 4096 22.7, 54.8 41.5 31.3 23.2; 2048 x 2048 x 256 9.8, 42.0 25.7 17.6
// 14.1; 700 x 1500 x 8320 29.0, 61.2 46.0 38.0 35.9.  Of 15 products from 40 x 28672 x 8192 to 4096 x 4096 x 4096 in both
// types the choice is within 12 % of the best of all, of most the best; of 150 drawn ones it takes 1.03 of the best
// kind's time in the mean.  fp32 results take 1.15 of the time in either, and rows that are not 16-byte aligned 1.4
// in small blocks (1021 x 2001 x 1000 in tiles and in blocks of the last kind 22.6, 17.5; x 1024 18.7, 13.0).
bool plan_small(MoF8Plan* plan, const MoF8Operand& A, const MoF8Operand& B, int64_t dim, int32_t dtype, double tiles_us) {
    const uintptr_t rows_at = reinterpret_cast<uintptr_t>(A.q) | uintptr_t(A.ld) | reinterpret_cast<uintptr_t>(B.q) | uintptr_t(B.ld);
    const bool aligned = (rows_at & 15) == 0;
    const double turns = double(blocks_of(dim)) / 8, slower = (dtype == MO_F32 ? 1.15 : 1.0) * (aligned ? 1.0 : 1.4);
    const double read = double(A.rows + B.rows) * double(dim) / 5.2e6;
    double least = tiles_us;
    plan->tb = 0;
    for (const SmallBlocks& b : kSmall) {
        const double t = std::max(b.us(B.rows, A.rows, turns) * slower, read);
        if (t < least) {
            least = t;
            plan->tb = b.tb;
            plan->rb = b.rb;
        }
    }
    return plan->tb != 0;
}

// A product in tiles, in 8 bits where `bits8`; its estimated us.  In 8 bits rows that are not in place are copied first.
double plan_product(MoF8Plan* p, const MoF8Operand& A, const MoF8Operand& B, int64_t dim, bool bits8) {
    Carve take;
    const MoF8Operand* o[2] = {&A, &B};
    double us;
    *p = {};
    p->bf16 = !bits8;
    if (bits8) {
        double copied = 0;
        p->ks = (blocks_of(dim) + 3) / 4 * 4;
        // not a multiple of 4 KB, which would put a tile's rows on few memory channels
        p->ld_q = blocks_of(dim) * kBlock + (blocks_of(dim) % 32 == 0 ? kBlock : 0);
        for (int i = 0; i < 2; ++i) {
            p->pack_q[i] = !q_in_place(*o[i], dim);
            p->pack_s[i] = !(i == 1 && B.shift) && !s_in_place(*o[i], dim);   // (B's in blocks are read singly)
            if (p->pack_q[i]) p->off_q[i] = take(uint64_t(o[i]->rows) * p->ld_q);
            if (p->pack_s[i]) p->off_s[i] = take(uint64_t(scale_rows(*o[i])) * p->ks);
            if (p->pack_q[i]) copied += double(o[i]->rows) * double(p->ld_q);
        }
        us = plan_tiles(p, B.rows, A.rows, blocks_of(dim), kStage8, 1, 4, &take) + (copied > 0 ? 4 + 2 * copied / 4.5e6 : 0) +
             (p->pack_s[0] || p->pack_s[1] ? 3 : 0);
    } else {
        us = plan_tiles(p, B.rows, A.rows, (dim + 63) / 64, kStageValues, 1, 1, &take);
    }
    p->bytes = take.at;
    return us;
}

MoF8Plan matmul_plan(const MoF8Operand& A, const MoF8Operand& B, int64_t dim, int32_t dtype) {
    MoF8Plan p;
    double us = plan_product(&p, A, B, dim, dtype == MO_BF16);
    if (p.pack_q[0] || p.pack_q[1]) {
        MoF8Plan values;
        const double t = plan_product(&values, A, B, dim, false);
        if (t < us) us = t, p = values;
    }
    // a launch and a tile's ends; the results, which nothing hides in the last tile
    us += 4.3 + (p.splits == 1 ? double(A.rows) * double(B.rows) * double(elem_size(dtype)) / 5e6 : 0);
    if (plan_small(&p, A, B, dim, dtype, us)) p.bytes = 0;
    return p;
}

// Whether a weight gradient reads its operands as they lie: a bf16 dY, rows of both in whole aligned 16
// bytes, less than 2^25 bytes apart (a stage's offsets have 31 bits), scales by rows.
bool tokens_in_place(const MoF8Wgrad& a) {
    return a.dy_dtype == MO_BF16 && a.rows % 8 == 0 && a.dim % 16 == 0 && a.lddy < (int64_t(1) << 24) &&
           a.X.ld < (int64_t(1) << 25) && a.X.inc == 1 && a.X.ld_s < (int64_t(1) << 25) &&
           ((reinterpret_cast<uintptr_t>(a.dY) | uintptr_t(a.lddy * 2)) & 15) == 0 &&
           ((reinterpret_cast<uintptr_t>(a.X.q) | uintptr_t(a.X.ld)) & 15) == 0;
}

// A weight gradient in blocks of 64 x 64 straight from the operands, where that takes less than in tiles (`tiles_us`,
// with a launch, the results that nothing hides, and a launch that transposes): a workgroup alone on
// its CU has its own time for 64 tokens, each further one adds to it; few blocks share a long K's tokens among up to
// 32 workgroups each, whose fp32 sums a second launch adds.  (G's type is not known to the workspace's query: dY's
// stands for it.)  us of the kernels in blocks and in tiles: dY and G in bf16, 98 tokens x 281 x 9600 7.0, 13.0; 1021 x
// 1024 x 1024 13.7, 18.5; 64 x 4096 x 4096 14.2, 13.6; 512 x 4096 x 4096 40.8, 26.5; both in fp32, 206 x 5632 x 256
// 9.8, 21.8; 257 x 1000 x 2001 13.1, 19.8; 721 x 9344 x 16 18.2, 36.4; 512 x 4096 x 4096 79.7, 59.5.
void plan_small_wgrad(const MoF8Wgrad& a, double tiles_us, MoF8Plan* p) {
    const bool wide = a.dy_dtype == MO_F32;
    const double t = double(a.X.rows), n = double(a.rows), k = double(a.dim);
    const int64_t blocks = ((a.rows + 63) / 64) * ((a.dim + 63) / 64), chunks = (a.X.rows + 63) / 64;
    if (blocks >= int64_t(1) << 18) return;
    // rows of dY that are not 16-byte aligned touch more lines (bf16, 1627 x 5147 x 384 37.1, 29.9; 2766 x
    // 10607 x 411 128, 62)
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.dY) | uintptr_t(a.lddy * elem_size(a.dy_dtype))) & 15) == 0;
    const double slower = aligned ? 1 : wide ? 1.25 : 1.6;
    double least = tiles_us + 4.3 + (p->splits == 1 ? n * k * double(elem_size(a.dy_dtype)) / 5e6 : 0) +
                   (p->tokens ? 0
                              : 3.5 + (t * n * double(elem_size(a.dy_dtype)) + t * k + 2 * t * ((wide ? 3 : 1) * n + k)) / 4.5e6);
    for (int64_t splits = 1; splits <= std::min(chunks, int64_t(32)); ++splits) {
        const double per = double(blocks * splits) / 256;
        if (splits > 1 && per > 4) break;
        const double us = 4.2 + per * (wide ? 0.45 : 0.3) + double((chunks + splits - 1) / splits) * slower *
                          ((wide ? 1.0 : 0.56) + std::max(0.0, per - 1) * (wide ? 0.56 : 0.26)) +
                          (splits > 1 ? 3 + 0.08 * double(splits) + double(blocks * splits) * 0.008 : 0);
        if (us < least) {
            least = us;
            p->tb = 4;
            p->stages = int((chunks + splits - 1) / splits);
        }
    }
    if (!p->tb) return;
    p->splits = int((chunks + p->stages - 1) / p->stages);
    Carve take;
    if (p->splits > 1) p->off_part = take(uint64_t(blocks) * p->splits * 4096 * 4);
    p->bytes = take.at;
}

MoF8Plan wgrad_plan(const MoF8Wgrad& a) {
    MoF8Plan p = {};
    Carve take;
    p.bf16 = true;
    p.tokens = tokens_in_place(a);
    p.kd = (a.X.rows + 63) / 64 * 64;
    if (!p.tokens) {
        // not a multiple of 4 KB, which would put a tile's rows on few memory channels
        p.ld_t = p.kd * 2 % 4096 == 0 ? p.kd + 64 : p.kd;
        const int planes = a.dy_dtype == MO_BF16 ? 1 : 3;
        p.off_q[0] = take(uint64_t(planes) * a.rows * p.ld_t * 2);
        p.off_q[1] = take(uint64_t(a.dim) * p.ld_t * 2);
    }
    const double tiles_us = plan_tiles(&p, a.dim, a.rows, p.kd / 64, p.tokens ? kStageTokens : kStageBf16,
                                       a.dy_dtype == MO_BF16 ? 1 : 3, 1, &take);
    p.bytes = take.at;
    plan_small_wgrad(a, tiles_us, &p);
    return p;
}

}  // namespace

extern "C" {

mo_status fp8_quantize(const void* X, int64_t ld_x, int32_t dtype, int64_t rows, int64_t cols, uint8_t* q, int64_t ld_q,
                       uint8_t* scales, int64_t ld_scales, void* stream) {
    MO_TRY(cast_shape(rows, cols, dtype, kCastRows, kCastCols));
    MoF8Cast a = {};
    MO_TRY(stride_of(ld_x, cols, &a.ldx));
    MO_TRY(stride_of(ld_q, cols, &a.ldq));
    MO_TRY(stride_of(ld_scales, blocks_of(cols), &a.lds));
    if (rows == 0 || cols == 0) return MO_OK;
    if (!X || !q || !scales) return MO_ERR_INVALID_ARG;
    a.X = X;
    a.Q = q;
    a.S = scales;
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    Ranges r;
    r.add(matrix_range(X, rows, cols, a.ldx, elem_size(dtype), 0));
    r.add(matrix_range(q, rows, cols, a.ldq, 1, 1));
    r.add(matrix_range(scales, rows, blocks_of(cols), a.lds, 1, 1));
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    MO_RUN(MO_PHASE_F8_CAST, mo_launch_f8_quantize(a, s));
    return MO_OK;
}

mo_status fp8_dequantize(const uint8_t* q, int64_t ld_q, const uint8_t* scales, int64_t ld_scales, int64_t rows,
                         int64_t cols, void* X, int64_t ld_x, int32_t dtype, void* stream) {
    MO_TRY(cast_shape(rows, cols, dtype, kCastRows, kCastCols));
    MoF8Cast a = {};
    MO_TRY(stride_of(ld_x, cols, &a.ldx));
    MO_TRY(stride_of(ld_q, cols, &a.ldq));
    MO_TRY(stride_of(ld_scales, blocks_of(cols), &a.lds));
    if (rows == 0 || cols == 0) return MO_OK;
    if (!X || !q || !scales) return MO_ERR_INVALID_ARG;
    a.out = X;
    a.Q = const_cast<uint8_t*>(q);
    a.S = const_cast<uint8_t*>(scales);
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    Ranges r;
    r.add(matrix_range(X, rows, cols, a.ldx, elem_size(dtype), 1));
    r.add(matrix_range(q, rows, cols, a.ldq, 1, 0));
    r.add(matrix_range(scales, rows, blocks_of(cols), a.lds, 1, 0));
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    MO_RUN(MO_PHASE_F8_CAST, mo_launch_f8_dequantize(a, s));
    return MO_OK;
}

mo_status fp8_quantize_weight(const void* W, int64_t ld_w, int32_t dtype, int64_t rows, int64_t cols, uint8_t* q,
                              int64_t ld_q, uint8_t* scales, int64_t ld_scales, uint8_t* qt, int64_t ld_qt,
                              uint8_t* scales_t, int64_t ld_scales_t, void* stream) {
    MO_TRY(cast_shape(rows, cols, dtype, kMaxSide, kMaxSide));
    MoF8Cast a = {};
    MO_TRY(stride_of(ld_w, cols, &a.ldx));
    MO_TRY(stride_of(ld_q, cols, &a.ldq));
    MO_TRY(stride_of(ld_scales, blocks_of(cols), &a.lds));
    MO_TRY(stride_of(ld_qt, rows, &a.ldqt));
    MO_TRY(stride_of(ld_scales_t, blocks_of(rows), &a.ldst));
    if (!q != !scales || !qt != !scales_t) return MO_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MO_OK;
    if (!W || (!q && !qt)) return MO_ERR_INVALID_ARG;
    a.X = W;
    a.Q = q;
    a.S = scales;
    a.Qt = qt;
    a.St = scales_t;
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    Ranges r;
    r.add(matrix_range(W, rows, cols, a.ldx, elem_size(dtype), 0));
    if (q) {
        r.add(matrix_range(q, rows, cols, a.ldq, 1, 1));
        r.add(matrix_range(scales, blocks_of(rows), blocks_of(cols), a.lds, 1, 1));
    }
    if (qt) {
        r.add(matrix_range(qt, cols, rows, a.ldqt, 1, 1));
        r.add(matrix_range(scales_t, blocks_of(cols), blocks_of(rows), a.ldst, 1, 1));
    }
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    MO_RUN(MO_PHASE_F8_CAST, mo_launch_f8_weight(a, s));
    return MO_OK;
}

static mo_status matmul_args(const mo_fp8_matrix* A, const mo_fp8_matrix* B, int64_t dim, int32_t dtype, MoF8Operand* a,
                             MoF8Operand* b) {
    if (dim < 0) return MO_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || dim > kMaxSide) return MO_ERR_UNSUPPORTED;
    MO_TRY(operand_of(A, dim, a));
    MO_TRY(operand_of(B, dim, b));
    // the row offsets within a tile are 31 bits
    const int64_t most = int64_t(1) << 23;
    return std::max({a->ld, a->ld_s, b->ld, b->ld_s}) >= most ? MO_ERR_UNSUPPORTED : MO_OK;
}

mo_status fp8_matmul_workspace_bytes(const mo_fp8_matrix* A, const mo_fp8_matrix* B, int64_t dim, int32_t dtype,
                                     size_t* bytes) {
    if (!bytes) return MO_ERR_INVALID_ARG;
    *bytes = 0;
    MoF8Operand a, b;
    MO_TRY(matmul_args(A, B, dim, dtype, &a, &b));
    if (a.rows == 0 || b.rows == 0 || dim == 0) return MO_OK;
    const uint64_t need = matmul_plan(a, b, dim, dtype).bytes;
    *bytes = need ? size_t(need) + MO_WS_ALIGN : 0;
    return MO_OK;
}

mo_status fp8_matmul(const mo_fp8_matrix* A, const mo_fp8_matrix* B, int64_t dim, void* Y, int64_t ld_y, int32_t dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
    MoF8Operand a, b;
    MO_TRY(matmul_args(A, B, dim, dtype, &a, &b));
    int64_t ldy;
    MO_TRY(stride_of(ld_y, b.rows, &ldy));
    if (a.rows == 0 || b.rows == 0) return MO_OK;
    if (!Y) return MO_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (dim == 0) return zero_rows(Y, a.rows, b.rows, ldy, dtype, MO_PHASE_F8_GEMM, s);
    Ranges r;
    operand_ranges(a, dim, &r);
    operand_ranges(b, dim, &r);
    r.add(matrix_range(Y, a.rows, b.rows, ldy, elem_size(dtype), 1));
    const MoF8Plan p = matmul_plan(a, b, dim, dtype);
    uint8_t* ws;
    if (!take_workspace(workspace, workspace_bytes, p.bytes, &r, &ws)) return MO_ERR_WORKSPACE_TOO_SMALL;
    if (r.conflict()) return MO_ERR_ALIAS;
    if (p.tb) {
        MO_RUN(MO_PHASE_F8_GEMM, mo_launch_f8_small(a, b, p, dim, Y, ldy, dtype, s));
        return MO_OK;
    }
    if (p.pack_q[0] || p.pack_q[1]) MO_RUN(MO_PHASE_F8_PREP, mo_launch_f8_copy(a, b, p, dim, ws, s));
    for (int i = 0; i < 2; ++i)
        if (p.pack_s[i]) MO_RUN(MO_PHASE_F8_PREP, mo_launch_f8_pack(i ? b : a, p, i, dim, ws, s));
    MO_RUN(MO_PHASE_F8_GEMM, mo_launch_f8_matmul(a, b, p, dim, Y, ldy, dtype, ws, s));
    return MO_OK;
}

static mo_status wgrad_args(const void* dY, int64_t ld_dy, int32_t dy_dtype, const mo_fp8_matrix* X, int64_t dim,
                            int64_t rows, MoF8Wgrad* a) {
    if (dim < 0 || rows < 0) return MO_ERR_INVALID_ARG;
    if (!dtype_ok(dy_dtype) || dim > kMaxSide || rows > kMaxSide) return MO_ERR_UNSUPPORTED;
    *a = {};
    MO_TRY(operand_of(X, dim, &a->X));
    MO_TRY(stride_of(ld_dy, rows, &a->lddy));
    if (a->X.shift) return MO_ERR_INVALID_ARG;
    a->dY = dY;
    a->dim = dim;
    a->rows = rows;
    a->dy_dtype = dy_dtype;
    return MO_OK;
}

mo_status fp8_weight_grad_workspace_bytes(const void* dY, int64_t ld_dy, int32_t dy_dtype, const mo_fp8_matrix* X,
                                          int64_t dim, int64_t rows, size_t* bytes) {
    if (!bytes) return MO_ERR_INVALID_ARG;
    *bytes = 0;
    MoF8Wgrad a;
    MO_TRY(wgrad_args(dY, ld_dy, dy_dtype, X, dim, rows, &a));
    if (a.X.rows == 0 || dim == 0 || rows == 0) return MO_OK;
    const uint64_t need = wgrad_plan(a).bytes;
    *bytes = need ? size_t(need) + MO_WS_ALIGN : 0;
    return MO_OK;
}

mo_status fp8_weight_grad(const void* dY, int64_t ld_dy, int32_t dy_dtype, const mo_fp8_matrix* X, int64_t dim, void* G,
                          int64_t ld_g, int32_t g_dtype, int64_t rows, int32_t accumulate, void* workspace,
                          size_t workspace_bytes, void* stream) {
    MoF8Wgrad a;
    MO_TRY(wgrad_args(dY, ld_dy, dy_dtype, X, dim, rows, &a));
    if (!dtype_ok(g_dtype)) return MO_ERR_UNSUPPORTED;
    MO_TRY(stride_of(ld_g, dim, &a.ldg));
    if (rows == 0 || dim == 0 || (a.X.rows == 0 && accumulate)) return MO_OK;
    if (!G || (a.X.rows && !dY)) return MO_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (a.X.rows == 0) return zero_rows(G, rows, dim, a.ldg, g_dtype, MO_PHASE_F8_WGRAD, s);
    a.G = G;
    a.g_dtype = g_dtype;
    a.accumulate = accumulate;
    const MoF8Plan p = wgrad_plan(a);
    Ranges r;
    operand_ranges(a.X, dim, &r);
    r.add(matrix_range(dY, a.X.rows, rows, a.lddy, elem_size(dy_dtype), 0));
    r.add(matrix_range(G, rows, dim, a.ldg, elem_size(g_dtype), 1));
    uint8_t* ws;
    if (!take_workspace(workspace, workspace_bytes, p.bytes, &r, &ws)) return MO_ERR_WORKSPACE_TOO_SMALL;
    if (r.conflict()) return MO_ERR_ALIAS;
    if (p.tb) {
        MO_RUN(MO_PHASE_F8_WGRAD, mo_launch_f8_small_wgrad(a, p, ws, s));
        return MO_OK;
    }
    if (!p.tokens) MO_RUN(MO_PHASE_F8_PREP, mo_launch_f8_transpose(a, p, ws, s));
    MO_RUN(MO_PHASE_F8_WGRAD, mo_launch_f8_wgrad(a, p, ws, s));
    return MO_OK;
}

}  // extern "C"
