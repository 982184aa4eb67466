// Argument records and launchers of the embedding, layer-norm and output-head
// operators (embedding.hip, layer_norm.hip, head_loss.hip); the entry points
// that check the arguments and plan the workspace are in operators.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mo.h"

// ---- layer norm ------------------------------------------------------------------
struct MoLnArgs {
    const void *X, *dY;
    const float *weight, *bias, *mean, *rstd;
    void *Y, *dX;
    float *mean_out, *rstd_out, *dweight, *dbias;
    int64_t ldx, lddy, ldy, lddx, rows, cols;
    int32_t dtype;
    float eps;
};
// Partial rows (each 2 x cols fp32) the backward pass leaves for the reduction.
int mo_ln_bwd_parts(int64_t rows, int64_t cols);
hipError_t mo_launch_ln_fwd(const MoLnArgs& a, hipStream_t s);
hipError_t mo_launch_ln_bwd(const MoLnArgs& a, float* part, hipStream_t s);
hipError_t mo_launch_ln_reduce(const MoLnArgs& a, const float* part, hipStream_t s);

// ---- embedding -------------------------------------------------------------------
constexpr int MO_EMB_SORT_TILE = 4096;   // positions per workgroup of the sort
struct MoEmbArgs {
    const int64_t* tokens;
    const void *W, *dY;
    void *Y, *G;
    int64_t n, vocab, dim, ldw, ldy, lddy, ldg;
    int32_t w_dtype, dy_dtype, g_dtype, accumulate;
    float scale;
};
// The sort (passes of `bits` bits; idx_bits > 0: in one workgroup, otherwise over
// `tiles` tiles) and the run sums (`chunks` chunks of C sorted positions), with
// their workspace offsets.
struct MoEmbPlan {
    int passes, bits, idx_bits, C;
    uint32_t tiles, chunks;
    uint64_t off_keys[2], off_idx[2], off_hist, off_spans, off_count, off_head, off_tail, bytes;
};
hipError_t mo_launch_emb_fill(const MoEmbArgs& a, hipStream_t s);
hipError_t mo_launch_emb_fwd(const MoEmbArgs& a, hipStream_t s);
hipError_t mo_launch_emb_sort(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s);
hipError_t mo_launch_emb_bwd(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s);

// ---- output head: softmax cross entropy and distillation ---------------------------
// H (tokens x dim) and W (vocab x dim) as bf16 planes (one for bf16 tensors, three
// for fp32 ones).  Every matrix below is read along K in stages of 64 elements.
struct MoHeadArgs {
    const void *H, *W;
    int64_t tokens, vocab, dim, ldh, ldw;
    int32_t dtype;
    // targets: k ids per token (cross entropy: k = 1, the label), the teacher's
    // logits (null for cross entropy), 1 / temperature and the temperature
    const int64_t* ids;
    const void* teacher;
    int64_t ld_ids, ld_teacher;
    int32_t teacher_dtype, k;
    float inv_t, t;
    // forward: loss, lse (tokens) and the target logits z (tokens x k);
    // backward: dloss and these as inputs
    float *loss, *lse, *z;
    const float *loss_in, *lse_in, *z_in, *dloss;
    void *dH, *dW;
    int64_t lddh, lddw;
};
struct MoHeadPlan {
    int planes;             // bf16 planes per operand: 1 or 3
    int dt_planes;          // of delta in dW's product: 1, 2 or 3
    int nb, nb_dw;          // tile width (64 nb): tokens side; dim side of dW
    int64_t n_pad;          // tokens rounded up to the tile width
    int64_t kd;             // dim as a K extent (rounded up, zeros behind)
    bool f32w;              // fp32 W read as fp32 (few tokens)
    int64_t k4;             // dim rounded up to 16 bytes of fp32
    bool pack_h, pack_w;    // operand copied (padded, split) before use
    int64_t piece;          // vocabulary rows per piece (a multiple of 256)
    int64_t ld_t, ld_p;     // row strides of the copies along the tokens and along the piece
    int64_t v_tiles;        // 256-row tiles of the vocabulary
    // dH: K stages per split, number of splits, tiles of 256 (dim) x 64 nb
    int dh_stages, dh_splits;
    uint32_t dh_tm, dh_tn;
    int z_stages, z_splits; // logits: K stages per split, splits (1: none)
    int dw_stages, dw_splits; // dW: the same
    uint64_t off_part, off_hp, off_wp, off_coef, off_nl2, off_tval, off_res, off_corr, off_ref, off_ht, off_wt[2],
        off_d[2], off_dt[2], off_acc, off_z, off_dw;
    uint64_t bytes;
};
hipError_t mo_launch_head_pack(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, bool h, int64_t v0,
                               int64_t rows, hipStream_t s);
hipError_t mo_launch_head_copy(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                               hipStream_t s);
hipError_t mo_launch_head_lse(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int64_t v0, int64_t rows,
                              hipStream_t s);
hipError_t mo_launch_head_targets(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int64_t v0, int64_t rows,
                                  hipStream_t s);
hipError_t mo_launch_head_loss(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s);
hipError_t mo_launch_head_prep(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s);
hipError_t mo_launch_head_ht(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s);
// k: the piece's number (two sets of piece buffers, used in turn)
hipError_t mo_launch_head_wt(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                             hipStream_t s);
hipError_t mo_launch_head_patch(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                                hipStream_t s);
hipError_t mo_launch_head_delta_split(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0,
                                      int64_t rows, hipStream_t s);
hipError_t mo_launch_head_step(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                               int64_t next_v0, int64_t next_rows, hipStream_t s);
hipError_t mo_launch_head_dh_out(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s);
