// Host side of the operators that write the gradients the owner steps read: the
// embedding, the layer norm and the output head's losses.  Argument checks,
// workspace plans and launches; the kernels are in embedding.hip, layer_norm.hip
// and head_loss.hip.  Every plan follows from sizes and alignments alone, no host
// memory is uploaded, and nothing is allocated, so each call can be captured.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/mo.h"
#include "host_common.h"
#include "mo_worklist.h"
#include "operators.h"

using namespace mo_host;

namespace {

#define MO_TRY(x)                          \
    do {                                   \
        const mo_status st_ = (x);         \
        if (st_ != MO_OK) return st_;      \
    } while (0)
#define MO_RUN(phase, launch)                                                              \
    do {                                                                                   \
        if (timed_launch(phase, s, [&] { return launch; }) != hipSuccess) return MO_ERR_HIP; \
    } while (0)

// Row strides up to 2^26 elements: byte ranges stay far inside 63 bits.
constexpr int64_t kMaxLd = int64_t(1) << 26;

// The stride in elements (0 means the row length).
mo_status stride_of(int64_t ld, int64_t cols, int64_t* out) {
    *out = ld ? ld : cols;
    if (*out < cols) return MO_ERR_INVALID_ARG;
    return *out > kMaxLd ? MO_ERR_UNSUPPORTED : MO_OK;
}

bool dtype_ok(int32_t d) { return d == MO_F32 || d == MO_BF16; }

Range vec_range(const void* p, int64_t n, int64_t es, int writable) { return matrix_range(p, 1, n, n, es, writable); }

// The ranges of one call, at most ten: no allocation, so no exception can reach the
// C entry points.
struct Ranges {
    Range r[12];
    int n = 0;
    void add(const Range& x) { r[n++] = x; }
    // Any overlap between a writable range and any other?
    bool conflict() const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((r[i].writable || r[j].writable) && r[i].lo < r[j].hi && r[j].lo < r[i].hi) return true;
        return false;
    }
};

// The workspace as a range and its aligned base; false when it is too small.
bool take_workspace(void* workspace, size_t have, uint64_t need, Ranges* ranges, uint8_t** base) {
    if (need == 0) {
        *base = nullptr;
        return true;
    }
    if (!workspace || have < need + MO_WS_ALIGN) return false;
    const uintptr_t w = reinterpret_cast<uintptr_t>(workspace);
    ranges->add(Range{w, w + have, 1});
    *base = reinterpret_cast<uint8_t*>(align_up(w, MO_WS_ALIGN));
    return true;
}

// Consecutive 256-byte aligned regions.
struct Carve {
    uint64_t at = 0;
    uint64_t operator()(uint64_t bytes) {
        const uint64_t o = at;
        at = align_up(at + bytes, MO_WS_ALIGN);
        return o;
    }
};

// ---- layer norm ------------------------------------------------------------------

constexpr int64_t kMaxRowLen = int64_t(1) << 24, kMaxRows = int64_t(1) << 32;

mo_status ln_shape(int64_t rows, int64_t cols, int32_t dtype) {
    if (rows < 0 || cols < 0) return MO_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || cols > kMaxRowLen || rows > kMaxRows) return MO_ERR_UNSUPPORTED;
    return MO_OK;
}

uint64_t ln_bwd_bytes(int64_t rows, int64_t cols) { return uint64_t(mo_ln_bwd_parts(rows, cols)) * 2 * cols * 4; }

// ---- embedding -------------------------------------------------------------------

constexpr int64_t kMaxVocab = int64_t(1) << 27, kMaxTokens = int64_t(1) << 30, kMaxDim = int64_t(1) << 20;

mo_status emb_shape(int64_t n, int64_t vocab, int64_t dim) {
    if (n < 0 || vocab < 0 || dim < 0) return MO_ERR_INVALID_ARG;
    if (n > kMaxTokens || vocab > kMaxVocab || dim > kMaxDim) return MO_ERR_UNSUPPORTED;
    return MO_OK;
}

MoEmbPlan emb_plan(int64_t n, int64_t vocab, int64_t dim) {
    MoEmbPlan p = {};
    if (n == 0 || dim == 0 || vocab == 0) return p;
    int bits = 1;
    while ((int64_t(1) << bits) <= vocab) ++bits;     // keys 0 .. vocab (the padded positions)
    p.passes = (bits + 8) / 9;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.tiles = uint32_t((n + MO_EMB_SORT_TILE - 1) / MO_EMB_SORT_TILE);
    p.C = int(std::max<int64_t>(4, (n + 511) / 512));
    p.chunks = uint32_t((n + p.C - 1) / p.C);
    Carve take;
    for (int b = 0; b < 2; ++b) {
        p.off_keys[b] = take(uint64_t(n) * 4);
        p.off_idx[b] = take(uint64_t(n) * 4);
    }
    // One workgroup sorts up to 2^15 positions (its LDS and registers) where the
    // key and the position share a 32-bit word, in one launch; otherwise three
    // launches per pass.
    int idx_bits = 1;
    while ((int64_t(1) << idx_bits) < n) ++idx_bits;
    p.idx_bits = n <= (1 << 15) && bits + idx_bits <= 32 ? idx_bits : 0;
    if (!p.idx_bits) p.off_hist = take((uint64_t(p.tiles) << p.bits) * 4);
    p.off_spans = take(uint64_t(p.chunks) * 12);
    p.off_count = take(4);
    p.off_head = take(uint64_t(p.chunks) * dim * 4);
    p.off_tail = take(uint64_t(p.chunks) * dim * 4);
    p.bytes = take.at;
    return p;
}

// ---- output head -----------------------------------------------------------------

constexpr int64_t kHeadMaxTokens = int64_t(1) << 20, kHeadMaxVocab = int64_t(1) << 26,
                  kHeadMaxDim = int64_t(1) << 16;
// Bytes of a piece's copies: more and smaller pieces add launches, partly filled last
// rounds and passes over dH's sums (backward 0.9 GB 2 % slower at 8192 x 128256 x
// 4096, 0.5 GB 4 %; larger ones gained nothing).  Forward the copies of a bf16 W take a
// quarter of it, fp32 planes all of it: 1078 tokens x 33926 x 6336 in four pieces 5.1
// ms, in one 3.6.
constexpr int64_t kHeadPieceBytes = int64_t(1600) << 20;

mo_status head_shape(const mo_head* h, int64_t* ldh, int64_t* ldw) {
    if (!h) return MO_ERR_INVALID_ARG;
    if (h->tokens < 0 || h->vocab < 1 || h->dim < 1) return MO_ERR_INVALID_ARG;
    if (!dtype_ok(h->dtype)) return MO_ERR_UNSUPPORTED;
    if (h->tokens > kHeadMaxTokens || h->vocab > kHeadMaxVocab || h->dim > kHeadMaxDim) return MO_ERR_UNSUPPORTED;
    MO_TRY(stride_of(h->ld_h, h->dim, ldh));
    return stride_of(h->ld_w, h->dim, ldw);
}

// A K extent of whole GEMM stages.
int64_t k_extent(int64_t k) { return (k + 63) / 64 * 64; }

// The row stride of a copy: not a multiple of 4 KB, which would put the 256 rows
// of a tile's stage on few memory channels.
int64_t copy_stride(int64_t k) { return k * 2 % 4096 == 0 ? k + 64 : k; }

// Whether bf16 rows can be loaded in place: 16-byte aligned rows of whole
// stages, less than 2^23 bytes apart (the GEMM's row offsets within a tile).
bool in_place(const void* p, int64_t ld, int64_t dim) {
    return k_extent(dim) == dim && ((reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * 2)) & 15) == 0 &&
           ld * 2 < (int64_t(1) << 23);
}

// Up to 512 tokens an fp32 W is read as fp32, in tiles of 64 tokens, in place or, where
// its rows are not whole 16 bytes, from a padded copy; more tokens pay for
// splitting it into planes once.  A step at 32001 rows x 4096 (us, in place and
// planes): 64 tokens 598 and 1790, 256 1654 and 2277, 512 3106 and 3342; at
// 32001 x 1000: 512 833 and 855, 1021 1611 and 1467.
constexpr int64_t kF32Tokens = 512;
bool f32_in_place(const void* p, int64_t ld, int64_t dim) {
    return dim % 4 == 0 && ((reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * 4)) & 15) == 0 &&
           ld * 4 < (int64_t(1) << 23);
}

// Up to 128 tokens a bf16 head's delta goes into dW's product in two planes: rounded, and
// what the rounding left.  A row of dW is then a term or two whose rounding nothing
// averages; with one plane dW's error was up to 1.6 times that of rounding the result
// (1 token x 32001 x 2048: 3.5e-3 of its norm against 2.3e-3; 8 x 128256 x 4096:
// 2.5e-3, 1.6e-3), with two it is that.  More tokens keep one plane: 1.2 times that in
// the middle of 60 batches of 129 to 1000 tokens, 1.46 times at most.  Backward at 32001 x 2048 (us, one plane and two):
// 64 tokens 195 and 201, 128 213 and 231, 512 318 and 363, 2048 800 and 1030.
constexpr int64_t kTwoPlaneTokens = 128;

// Estimated us of a product in `tiles` tiles of 256 x 64 nb with `stages`
// stages of 64 K, and the splits of K that it takes.  A stage takes 1.43, 0.8 and
// 0.6 us in a tile of 256, 128 and 64 tokens (256 CUs at 1.5 PFLOP/s; the narrow ones
// wait for their loads), six times that with three planes; splits write and read
// fp32 tiles at 5 TB/s, are added up one after the other, and are one launch more.
// In all, a step of 4405 rows x 34 tokens x 4672 went from 177 to 107 us in bf16
// with splits, 5168 x 40 x 256 (4 stages) stays without, at 50 to 60 us.
double product_us(int64_t tiles, int64_t stages, int nb, int planes, int64_t* splits) {
    const double stage = (nb == 4 ? 1.43 : nb == 2 ? 0.8 : 0.6) * (planes == 1 ? 1 : 6);
    double least = double((tiles + 255) / 256 * stages) * stage;
    *splits = 1;
    for (int64_t k = 2; k <= std::min(256 / tiles, stages); ++k) {
        const double t = double((stages + k - 1) / k) * stage + double(tiles * k * nb) * 0.026 + double(k) * 0.1 + 4;
        if (t < least) {
            least = t;
            *splits = k;
        }
    }
    return least;
}

// Tile width over the tokens: the one with the least time.
int token_tile(int64_t n, int64_t v_tiles, int64_t stages, int planes, int widest) {
    int best = widest;
    double least = 0;
    for (int nb = widest; nb >= 1; nb /= 2) {
        int64_t splits;
        const double t = product_us((n + 64 * nb - 1) / (64 * nb) * v_tiles, stages, nb, planes, &splits);
        if (nb == widest || t < least) {
            least = t;
            best = nb;
        }
    }
    return best;
}

MoHeadPlan head_plan(const MoHeadArgs& a, bool backward, bool need_dh, bool need_dw) {
    MoHeadPlan p = {};
    p.planes = a.dtype == MO_BF16 ? 1 : 3;
    p.dt_planes = p.planes == 1 && a.tokens <= kTwoPlaneTokens ? 2 : p.planes;
    p.v_tiles = (a.vocab + 255) / 256;
    p.kd = k_extent(a.dim);
    p.f32w = p.planes == 3 && a.tokens <= kF32Tokens;
    p.k4 = (a.dim + 3) / 4 * 4;
    p.nb = token_tile(a.tokens, p.v_tiles, p.kd / 64, p.planes, p.f32w ? 1 : 4);
    p.n_pad = (a.tokens + 64 * p.nb - 1) / (64 * p.nb) * (64 * p.nb);
    p.pack_h = p.planes != 1 || !in_place(a.H, a.ldh, a.dim);
    p.pack_w = p.f32w ? !f32_in_place(a.W, a.ldw, a.dim) : p.planes != 1 || !in_place(a.W, a.ldw, a.dim);
    p.nb_dw = a.dim <= 128 ? 1 : 4;
    const int64_t tn = p.n_pad / (64 * p.nb);
    // equal pieces bounded by the memory of their copies (and by the grid of one launch);
    // at least one tile
    const int64_t copy = !p.pack_w ? 0 : p.f32w ? 4 * p.k4 : 2 * p.planes * p.kd;   // bytes of a row
    int64_t row = copy;
    // (the same pieces whichever gradients are asked for, so that the size query holds for each)
    if (backward) row += 2 * 2 * (p.planes + p.dt_planes) * p.n_pad + (p.f32w ? copy : 4 * p.planes * a.dim);
    int64_t most = std::min<int64_t>((int64_t(1) << 22) / std::max<int64_t>(tn, (a.dim + 63) / 64), 1 << 13);
    if (row) most = std::min(most, (backward || p.planes == 3 ? kHeadPieceBytes : kHeadPieceBytes / 4) / row / 256);
    most = std::max<int64_t>(most, 1);
    const int64_t pieces = (p.v_tiles + most - 1) / most;
    p.piece = (p.v_tiles + pieces - 1) / pieces * 256;
    p.ld_t = copy_stride(p.n_pad);
    p.ld_p = copy_stride(p.piece);
    const int64_t z_tiles = p.piece / 256 * tn, nk = p.kd / 64;
    int64_t z_want;
    product_us(z_tiles, nk, p.nb, p.planes, &z_want);
    p.z_stages = int((nk + z_want - 1) / z_want);
    p.z_splits = int((nk + p.z_stages - 1) / p.z_stages);
    Carve take;
    if (p.z_splits > 1) p.off_z = take(uint64_t(4) * p.z_splits * z_tiles * 256 * 64 * p.nb);
    if (p.pack_h) p.off_hp = take(uint64_t(2) * p.planes * a.tokens * p.kd);
    if (p.pack_w && !p.f32w) p.off_wp = take(uint64_t(copy) * p.piece);
    if (p.pack_w && p.f32w)
        for (int i = 0; i < (backward && pieces > 1 ? 2 : 1); ++i) p.off_wt[i] = take(uint64_t(copy) * p.piece);
    if (!backward) {
        p.off_part = take(uint64_t(8) * p.v_tiles * (p.z_splits > 1 ? 8 : 1) * p.n_pad);
    } else {
        p.off_coef = take(uint64_t(4) * p.n_pad);
        p.off_nl2 = take(uint64_t(4) * p.n_pad);
        p.off_tval = take(uint64_t(4) * a.tokens * a.k);
        p.off_ref = take(4);
        if (p.planes == 1 && need_dh) {
            p.off_res = take(uint64_t(4) * a.tokens * a.k);
            p.off_corr = take(uint64_t(2) * a.tokens * a.dim);
        }
        const int sets = pieces > 1 ? 2 : 1;
        for (int i = 0; i < sets; ++i) {
            p.off_d[i] = take(uint64_t(2) * p.planes * p.n_pad * p.ld_p);
            p.off_dt[i] = take(uint64_t(2) * p.dt_planes * p.piece * p.ld_t);
            if (need_dh && !p.f32w) p.off_wt[i] = take(uint64_t(2) * p.planes * a.dim * p.ld_p);
        }
        if (need_dw) {
            p.off_ht = take(uint64_t(2) * p.planes * a.dim * p.ld_t);
            const int64_t tiles = p.piece / 256 * ((a.dim + 64 * p.nb_dw - 1) / (64 * p.nb_dw)), nk_dw = (a.tokens + 63) / 64;
            int64_t want;
            if (p.dt_planes == 2) want = 1;   // two stages of K at most
            else product_us(tiles, nk_dw, p.nb_dw, p.planes, &want);
            p.dw_stages = int((nk_dw + want - 1) / want);
            p.dw_splits = int((nk_dw + p.dw_stages - 1) / p.dw_stages);
            if (p.dw_splits > 1) p.off_dw = take(uint64_t(4) * p.dw_splits * tiles * 256 * 64 * p.nb_dw);
        }
        if (need_dh) {
            p.dh_tm = uint32_t((a.dim + 255) / 256);
            p.dh_tn = uint32_t(tn);
            // splits of K that fill the 256 CUs once, in whole tiles of 256 rows (4 stages)
            const int64_t tiles = int64_t(p.dh_tm) * p.dh_tn, groups = p.piece / 256;
            const int64_t want = std::max<int64_t>(1, std::min<int64_t>(256 / tiles, groups));
            p.dh_stages = int((groups + want - 1) / want * 4);
            p.dh_splits = int((groups * 4 + p.dh_stages - 1) / p.dh_stages);
            p.off_acc = take(uint64_t(4) * p.dh_splits * tiles * 256 * 64 * p.nb);
        }
    }
    p.bytes = take.at;
    return p;
}

struct Targets {
    const int64_t* ids;
    int64_t ld_ids;
    int32_t k;
    const void* teacher;
    int64_t ld_teacher;
    int32_t teacher_dtype;
    float temperature;
};

mo_status head_args(const mo_head* h, const Targets* t, MoHeadArgs* a) {
    int64_t ldh, ldw;
    MO_TRY(head_shape(h, &ldh, &ldw));
    *a = {};
    a->H = h->H;
    a->W = h->W;
    a->tokens = h->tokens;
    a->vocab = h->vocab;
    a->dim = h->dim;
    a->ldh = ldh;
    a->ldw = ldw;
    a->dtype = h->dtype;
    a->k = t->k;
    a->ids = t->ids;
    a->ld_ids = t->ld_ids;
    a->teacher = t->teacher;
    a->ld_teacher = t->ld_teacher;
    a->teacher_dtype = t->teacher_dtype;
    a->t = t->temperature;
    a->inv_t = 1.0f / t->temperature;
    return MO_OK;
}

mo_status topk_targets(const mo_topk* t, Targets* out) {
    if (!t || t->k < 1) return MO_ERR_INVALID_ARG;
    const float T = t->temperature;
    if (!(T > 0.f) || !finite(T * T) || !finite(1.0f / T)) return MO_ERR_INVALID_ARG;
    if (t->k > MO_TOPK_MAX || !dtype_ok(t->dtype)) return MO_ERR_UNSUPPORTED;
    *out = {t->ids, 0, t->k, t->logits, 0, t->dtype, T};
    MO_TRY(stride_of(t->ld_ids, t->k, &out->ld_ids));
    return stride_of(t->ld_logits, t->k, &out->ld_teacher);
}

// Ranges of what every head call reads.
void head_inputs(const MoHeadArgs& a, Ranges* r) {
    const int64_t es = elem_size(a.dtype);
    r->add(matrix_range(a.H, a.tokens, a.dim, a.ldh, es, 0));
    r->add(matrix_range(a.W, a.vocab, a.dim, a.ldw, es, 0));
    r->add(matrix_range(a.ids, a.tokens, a.k, a.ld_ids, 8, 0));
    if (a.teacher) r->add(matrix_range(a.teacher, a.tokens, a.k, a.ld_teacher, elem_size(a.teacher_dtype), 0));
}

mo_status head_forward(MoHeadArgs& a, void* workspace, size_t workspace_bytes, void* stream, bool distill) {
    if (a.tokens == 0) return MO_OK;
    if (!a.H || !a.W || !a.ids || !a.loss || !a.lse || (distill && (!a.teacher || !a.z))) return MO_ERR_INVALID_ARG;
    const MoHeadPlan p = head_plan(a, false, false, false);
    Ranges ranges;
    head_inputs(a, &ranges);
    ranges.add(vec_range(a.loss, a.tokens, 4, 1));
    ranges.add(vec_range(a.lse, a.tokens, 4, 1));
    if (distill) ranges.add(vec_range(a.z, a.tokens * a.k, 4, 1));
    uint8_t* ws;
    if (!take_workspace(workspace, workspace_bytes, p.bytes, &ranges, &ws)) return MO_ERR_WORKSPACE_TOO_SMALL;
    if (ranges.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (p.pack_h) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_pack(a, p, ws, true, 0, a.tokens, s));
    // from the planes of each piece, or from W itself at once
    const bool by_piece = p.planes == 3 && !p.f32w;
    if (distill && !by_piece) MO_RUN(MO_PHASE_HD_TARGET, mo_launch_head_targets(a, p, ws, 0, a.vocab, s));
    for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
        const int64_t rows = std::min(p.piece, a.vocab - v0);
        if (p.pack_w && p.f32w) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_copy(a, p, ws, 0, v0, rows, s));
        else if (p.pack_w) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_pack(a, p, ws, false, v0, rows, s));
        if (distill && by_piece) MO_RUN(MO_PHASE_HD_TARGET, mo_launch_head_targets(a, p, ws, v0, rows, s));
        MO_RUN(MO_PHASE_HD_LSE, mo_launch_head_lse(a, p, ws, v0, rows, s));
    }
    MO_RUN(MO_PHASE_HD_TARGET, mo_launch_head_loss(a, p, ws, s));
    return MO_OK;
}

// Zeros in a rows x cols matrix.
mo_status zero_rows(void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, int phase, hipStream_t s) {
    MoEmbArgs e = {};
    e.G = p;
    e.vocab = rows;
    e.dim = cols;
    e.ldg = ld;
    e.g_dtype = dtype;
    MO_RUN(phase, mo_launch_emb_fill(e, s));
    return MO_OK;
}

mo_status head_backward(MoHeadArgs& a, void* workspace, size_t workspace_bytes, void* stream, bool distill) {
    MO_TRY(stride_of(a.lddh, a.dim, &a.lddh));
    MO_TRY(stride_of(a.lddw, a.dim, &a.lddw));
    if (!a.dH && !a.dW) return MO_OK;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (a.tokens == 0) return a.dW ? zero_rows(a.dW, a.vocab, a.dim, a.lddw, a.dtype, MO_PHASE_HD_STEP, s) : MO_OK;
    if (!a.H || !a.W || !a.ids || !a.lse_in || !a.dloss) return MO_ERR_INVALID_ARG;
    if (distill ? (!a.teacher || !a.z_in) : !a.loss_in) return MO_ERR_INVALID_ARG;
    const MoHeadPlan p = head_plan(a, true, a.dH != nullptr, a.dW != nullptr);
    Ranges ranges;
    head_inputs(a, &ranges);
    const int64_t es = elem_size(a.dtype);
    ranges.add(vec_range(a.lse_in, a.tokens, 4, 0));
    ranges.add(vec_range(a.dloss, a.tokens, 4, 0));
    if (distill) ranges.add(vec_range(a.z_in, a.tokens * a.k, 4, 0));
    else ranges.add(vec_range(a.loss_in, a.tokens, 4, 0));
    if (a.dH) ranges.add(matrix_range(a.dH, a.tokens, a.dim, a.lddh, es, 1));
    if (a.dW) ranges.add(matrix_range(a.dW, a.vocab, a.dim, a.lddw, es, 1));
    uint8_t* ws;
    if (!take_workspace(workspace, workspace_bytes, p.bytes, &ranges, &ws)) return MO_ERR_WORKSPACE_TOO_SMALL;
    if (ranges.conflict()) return MO_ERR_ALIAS;
    MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_prep(a, p, ws, s));
    if (p.pack_h) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_pack(a, p, ws, true, 0, a.tokens, s));
    if (a.dW) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_ht(a, p, ws, s));
    // turn k: delta of piece k beside dH and dW of piece k - 1 (behind them if its logits are split)
    const int pieces = int((a.vocab + p.piece - 1) / p.piece);
    for (int k = 0; k <= pieces; ++k) {
        const int64_t v0 = k * p.piece, rows = k < pieces ? std::min(p.piece, a.vocab - v0) : 0;
        if (rows) {
            // the transpose for dH makes the copy as well
            if (p.pack_w && p.f32w) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_copy(a, p, ws, k, v0, rows, s));
            else if (a.dH && !p.f32w) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_wt(a, p, ws, k, v0, rows, s));
            else if (p.pack_w) MO_RUN(MO_PHASE_HD_PREP, mo_launch_head_pack(a, p, ws, false, v0, rows, s));
        }
        const int64_t last = k ? std::min(p.piece, a.vocab - (v0 - p.piece)) : 0, beside = p.z_splits > 1 ? 0 : rows;
        if (last || beside)
            MO_RUN(last ? MO_PHASE_HD_STEP : MO_PHASE_HD_DELTA,
                   mo_launch_head_step(a, p, ws, k - 1, v0 - p.piece, last, v0, beside, s));
        if (rows > beside) MO_RUN(MO_PHASE_HD_DELTA, mo_launch_head_delta_split(a, p, ws, k, v0, rows, s));
        if (rows) MO_RUN(MO_PHASE_HD_TARGET, mo_launch_head_patch(a, p, ws, k, v0, rows, s));
    }
    if (a.dH) MO_RUN(MO_PHASE_HD_DH, mo_launch_head_dh_out(a, p, ws, s));
    return MO_OK;
}

mo_status head_bytes(const MoHeadArgs& a, int32_t backward, size_t* bytes) {
    if (!bytes) return MO_ERR_INVALID_ARG;
    *bytes = 0;
    if (a.tokens == 0) return MO_OK;
    *bytes = size_t(head_plan(a, backward != 0, true, true).bytes) + MO_WS_ALIGN;
    return MO_OK;
}

Targets label_targets(const int64_t* labels) { return {labels, 1, 1, nullptr, 1, MO_F32, 1.0f}; }

}  // namespace

extern "C" {

mo_status layer_norm_forward(const void* X, int64_t ld_x, const float* weight, const float* bias, void* Y,
                             int64_t ld_y, float* mean, float* rstd, int64_t rows, int64_t cols, int32_t dtype,
                             float eps, void* stream) {
    MO_TRY(ln_shape(rows, cols, dtype));
    if (!finite(eps) || eps < 0.f) return MO_ERR_INVALID_ARG;
    MoLnArgs a = {};
    MO_TRY(stride_of(ld_x, cols, &a.ldx));
    MO_TRY(stride_of(ld_y, cols, &a.ldy));
    if (rows == 0 || cols == 0) return MO_OK;
    if (!X || !Y) return MO_ERR_INVALID_ARG;
    a.X = X;
    a.Y = Y;
    a.weight = weight;
    a.bias = bias;
    a.mean_out = mean;
    a.rstd_out = rstd;
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    a.eps = eps;
    const int64_t es = elem_size(dtype);
    Ranges r;
    r.add(matrix_range(X, rows, cols, a.ldx, es, 0));
    r.add(matrix_range(Y, rows, cols, a.ldy, es, 1));
    if (weight) r.add(vec_range(weight, cols, 4, 0));
    if (bias) r.add(vec_range(bias, cols, 4, 0));
    if (mean) r.add(vec_range(mean, rows, 4, 1));
    if (rstd) r.add(vec_range(rstd, rows, 4, 1));
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    MO_RUN(MO_PHASE_LN_FWD, mo_launch_ln_fwd(a, s));
    return MO_OK;
}

mo_status layer_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes) return MO_ERR_INVALID_ARG;
    MO_TRY(ln_shape(rows, cols, MO_F32));
    const uint64_t b = rows && cols ? ln_bwd_bytes(rows, cols) : 0;
    *bytes = b ? size_t(align_up(b, MO_WS_ALIGN)) + MO_WS_ALIGN : 0;
    return MO_OK;
}

mo_status layer_norm_backward(const void* dY, int64_t ld_dy, const void* X, int64_t ld_x, const float* weight,
                              const float* mean, const float* rstd, void* dX, int64_t ld_dx, float* dweight,
                              float* dbias, int64_t rows, int64_t cols, int32_t dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
    MO_TRY(ln_shape(rows, cols, dtype));
    MoLnArgs a = {};
    MO_TRY(stride_of(ld_x, cols, &a.ldx));
    MO_TRY(stride_of(ld_dy, cols, &a.lddy));
    MO_TRY(stride_of(ld_dx, cols, &a.lddx));
    if (cols == 0) return MO_OK;
    if (!dX && !dweight && !dbias) return MO_OK;
    a.X = X;
    a.dY = dY;
    a.weight = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.dX = dX;
    a.dweight = dweight;
    a.dbias = dbias;
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    const bool sums = dweight || dbias;
    const int64_t es = elem_size(dtype);
    Ranges r;
    if (rows) {
        if (!X || !dY || !mean || !rstd) return MO_ERR_INVALID_ARG;
        r.add(matrix_range(X, rows, cols, a.ldx, es, 0));
        r.add(matrix_range(dY, rows, cols, a.lddy, es, 0));
        r.add(vec_range(mean, rows, 4, 0));
        r.add(vec_range(rstd, rows, 4, 0));
        if (dX) r.add(matrix_range(dX, rows, cols, a.lddx, es, 1));
    }
    if (weight) r.add(vec_range(weight, cols, 4, 0));
    if (dweight) r.add(vec_range(dweight, cols, 4, 1));
    if (dbias) r.add(vec_range(dbias, cols, 4, 1));
    uint8_t* ws = nullptr;
    if (!take_workspace(workspace, workspace_bytes, sums ? align_up(ln_bwd_bytes(rows, cols), MO_WS_ALIGN) : 0, &r, &ws))
        return MO_ERR_WORKSPACE_TOO_SMALL;
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    float* part = reinterpret_cast<float*>(ws);
    if (rows) MO_RUN(MO_PHASE_LN_BWD, mo_launch_ln_bwd(a, part, s));
    if (sums) MO_RUN(MO_PHASE_LN_BWD, mo_launch_ln_reduce(a, part, s));
    return MO_OK;
}

mo_status embedding_forward(const int64_t* tokens, int64_t n, const void* W, int64_t ld_w, int64_t vocab,
                            int64_t dim, int32_t dtype, float scale, void* Y, int64_t ld_y, void* stream) {
    MO_TRY(emb_shape(n, vocab, dim));
    if (!dtype_ok(dtype)) return MO_ERR_UNSUPPORTED;
    if (!finite(scale)) return MO_ERR_INVALID_ARG;
    MoEmbArgs a = {};
    MO_TRY(stride_of(ld_w, dim, &a.ldw));
    MO_TRY(stride_of(ld_y, dim, &a.ldy));
    if (n == 0 || dim == 0) return MO_OK;
    if (!tokens || !Y || (vocab && !W)) return MO_ERR_INVALID_ARG;
    a.tokens = tokens;
    a.W = W;
    a.Y = Y;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.w_dtype = dtype;
    a.scale = scale;
    const int64_t es = elem_size(dtype);
    Ranges r;
    r.add(vec_range(tokens, n, 8, 0));
    r.add(matrix_range(Y, n, dim, a.ldy, es, 1));
    if (vocab) r.add(matrix_range(W, vocab, dim, a.ldw, es, 0));
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    MO_RUN(MO_PHASE_EMB_FWD, mo_launch_emb_fwd(a, s));
    return MO_OK;
}

mo_status embedding_workspace_bytes(int64_t n, int64_t vocab, int64_t dim, size_t* bytes) {
    if (!bytes) return MO_ERR_INVALID_ARG;
    MO_TRY(emb_shape(n, vocab, dim));
    const uint64_t b = emb_plan(n, vocab, dim).bytes;
    *bytes = b ? size_t(b) + MO_WS_ALIGN : 0;
    return MO_OK;
}

mo_status embedding_backward(const int64_t* tokens, int64_t n, const void* dY, int64_t ld_dy, int32_t dy_dtype,
                             void* G, int64_t ld_g, int32_t g_dtype, int64_t vocab, int64_t dim, float scale,
                             int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    MO_TRY(emb_shape(n, vocab, dim));
    if (!dtype_ok(dy_dtype) || !dtype_ok(g_dtype)) return MO_ERR_UNSUPPORTED;
    if (!finite(scale)) return MO_ERR_INVALID_ARG;
    MoEmbArgs a = {};
    MO_TRY(stride_of(ld_dy, dim, &a.lddy));
    MO_TRY(stride_of(ld_g, dim, &a.ldg));
    if (vocab == 0 || dim == 0 || (n == 0 && accumulate)) return MO_OK;
    if (!G || (n && (!tokens || !dY))) return MO_ERR_INVALID_ARG;
    a.tokens = tokens;
    a.dY = dY;
    a.G = G;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.dy_dtype = dy_dtype;
    a.g_dtype = g_dtype;
    a.accumulate = accumulate != 0;
    a.scale = scale;
    const MoEmbPlan p = emb_plan(n, vocab, dim);
    Ranges r;
    r.add(matrix_range(G, vocab, dim, a.ldg, elem_size(g_dtype), 1));
    if (n) {
        r.add(vec_range(tokens, n, 8, 0));
        r.add(matrix_range(dY, n, dim, a.lddy, elem_size(dy_dtype), 0));
    }
    uint8_t* ws;
    if (!take_workspace(workspace, workspace_bytes, p.bytes, &r, &ws)) return MO_ERR_WORKSPACE_TOO_SMALL;
    if (r.conflict()) return MO_ERR_ALIAS;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (n == 0) {
        MO_RUN(MO_PHASE_EMB_BWD, mo_launch_emb_fill(a, s));
        return MO_OK;
    }
    MO_RUN(MO_PHASE_EMB_SORT, mo_launch_emb_sort(a, p, ws, s));
    MO_RUN(MO_PHASE_EMB_BWD, mo_launch_emb_bwd(a, p, ws, s));
    return MO_OK;
}

mo_status softmax_xent_workspace_bytes(const mo_head* head, int32_t backward, size_t* bytes) {
    MoHeadArgs a;
    const Targets t = label_targets(nullptr);
    MO_TRY(head_args(head, &t, &a));
    return head_bytes(a, backward, bytes);
}

mo_status softmax_xent_forward(const mo_head* head, const int64_t* labels, float* loss, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
    MoHeadArgs a;
    const Targets t = label_targets(labels);
    MO_TRY(head_args(head, &t, &a));
    a.loss = loss;
    a.lse = lse;
    return head_forward(a, workspace, workspace_bytes, stream, false);
}

mo_status softmax_xent_backward(const mo_head* head, const int64_t* labels, const float* loss, const float* lse,
                                const float* dloss, void* dH, int64_t ld_dh, void* dW, int64_t ld_dw,
                                void* workspace, size_t workspace_bytes, void* stream) {
    MoHeadArgs a;
    const Targets t = label_targets(labels);
    MO_TRY(head_args(head, &t, &a));
    a.loss_in = loss;
    a.lse_in = lse;
    a.dloss = dloss;
    a.dH = dH;
    a.dW = dW;
    a.lddh = ld_dh;
    a.lddw = ld_dw;
    return head_backward(a, workspace, workspace_bytes, stream, false);
}

mo_status topk_distill_workspace_bytes(const mo_head* head, const mo_topk* top, int32_t backward, size_t* bytes) {
    MoHeadArgs a;
    Targets t;
    MO_TRY(topk_targets(top, &t));
    MO_TRY(head_args(head, &t, &a));
    return head_bytes(a, backward, bytes);
}

mo_status topk_distill_forward(const mo_head* head, const mo_topk* top, float* loss, float* lse, float* z,
                               void* workspace, size_t workspace_bytes, void* stream) {
    MoHeadArgs a;
    Targets t;
    MO_TRY(topk_targets(top, &t));
    MO_TRY(head_args(head, &t, &a));
    a.loss = loss;
    a.lse = lse;
    a.z = z;
    return head_forward(a, workspace, workspace_bytes, stream, true);
}

mo_status topk_distill_backward(const mo_head* head, const mo_topk* top, const float* lse, const float* z,
                                const float* dloss, void* dH, int64_t ld_dh, void* dW, int64_t ld_dw,
                                void* workspace, size_t workspace_bytes, void* stream) {
    MoHeadArgs a;
    Targets t;
    MO_TRY(topk_targets(top, &t));
    MO_TRY(head_args(head, &t, &a));
    a.lse_in = lse;
    a.z_in = z;
    a.dloss = dloss;
    a.dH = dH;
    a.dW = dW;
    a.lddh = ld_dh;
    a.lddw = ld_dw;
    return head_backward(a, workspace, workspace_bytes, stream, true);
}

}  // extern "C"
