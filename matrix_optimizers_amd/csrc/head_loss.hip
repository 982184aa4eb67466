// The output head's losses without its logits: softmax cross entropy, and
// distillation from a teacher's top logits, with the gradients of the hidden
// states H (tokens x dim) and the head W (vocab x dim).
//
//   z = H W^T,  lse_n = log sum_v exp(z_nv / T)
//   cross entropy (T = 1)  loss_n = lse_n - z_ny
//   distillation           p = softmax(t / T) over the stored entries,
//                          loss_n = T^2 sum_k p_k (log p_k - (z_k / T - lse_n))
//   delta_nv = c_n (exp(z_nv / T - lse_n) - p_nv),  c_n = T dloss_n / r
//   dH = r delta W,  dW = r delta^T H
//
// r is the significand, in [1, 2), of one row's T |dloss| (ref_scale below): with
// the usual mean over rows every c_n is a power of two, and the label's delta,
// -(1 - p), the largest of its row, is rounded like that number.  Rounded as
// -(1 - p) / count it would carry nearly the same mantissa, and the same error of up
// to half a unit, in every row.  What rounding takes from delta at a row's targets is
// added to its dH (head_residual_kernel).  The error of dH at 8192 tokens x 128256 x
// 4096 bf16 was 3.0e-3 of its norm without the two, 2.0e-3 with the first; it is at
// most 1.8e-3, 1.7e-3 of which is the result's rounding.
//
// Forward: one product whose epilogue keeps, per tile and token, the maximum m of
// the logits and the sum s of exp((z - m) / T) over the tile's 256 vocabulary rows.
// A loss takes log q = (z_y - m) / T - log s, so z_y has to be the very number whose
// maximum m is: of a token the model is sure of, nothing but rounding would be left
// of a logit summed in another order (losses of +-1.5e-5 at logits of 60, and deltas
// like them).  The label's logit is taken from the product's accumulators, a
// teacher's k ids' from products of the same instructions in the same order.  With
// equal bits m - z_y >= 0 and s >= 1, so no cross entropy is negative.  Backward: pieces of the vocabulary, each
// computed again from H and W into delta (bf16, or the three planes of fp32),
// in both orientations, from which dW's rows are finished and dH accumulated
// in fp32; one launch does that for a piece and computes the next one's delta.
// 8 N V d flops in all, against 6 N V d when the logits are kept.
//
// Rounding: the logits are never rounded (fp32 accumulators); delta takes the
// tensors' own precision (bf16: half a unit in 2^8, the size of the rounding
// of the results themselves; fp32: exact); sums are fp32.
#include <type_traits>

#include "head_gemm.h"
#include "op_common.h"
#include "operators.h"

namespace {

using namespace mo_head_gemm;

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// How the products' operands come (PL): 1: bf16; 2: the same, with delta in two planes for
// dW; 3: fp32 as three planes each; F32W: W in fp32 as it lies in memory, the tokens'
// side as planes.
constexpr int F32W = 32;
constexpr int w_planes(int PL) { return PL == 2 ? 1 : PL; }      // of the products with W
constexpr int dw_planes(int PL) { return PL == F32W ? 3 : PL; }   // of delta in dW's
constexpr int lds_of(int NB, int PL) { return PL == F32W ? head_lds32() : head_lds(NB); }
// One tile of a product with W: NN: columns of W, K along its rows.
template <int NB, int PL, bool NN, class Acc>
__device__ __forceinline__ void w_tile(uint8_t* smem, const Operand& P, int dim, const Operand& Q, int64_t p0,
                                       int64_t q0, int k0, int n, Acc& acc) {
    if constexpr (PL == F32W) head_tile32<NN>(smem, P, dim, Q, p0, q0, k0, n, acc);
    else head_tile<NB, PL>(smem, P, Q, p0, q0, k0, n, acc);
}

MO_DEV float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- operand copies ---------------------------------------------------------------

// The three planes of 8 elements.
MO_DEV void split_planes(const f32x8& v, bf16x8 (&p)[3]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bf16_t a, b, c;
        split_f32(v.v[e], a, b, c);
        p[0][e] = a; p[1][e] = b; p[2][e] = c;
    }
}
// One 8-element chunk of a value's planes (16 bytes each).
template <int PL> MO_DEV void put_planes(bf16_t* dst, int64_t plane, const f32x8& v) {
    if constexpr (PL == 1) {
        st8(dst, v);
    } else {
        bf16x8 p[3];
        split_planes(v, p);
#pragma unroll
        for (int i = 0; i < dw_planes(PL); ++i) *reinterpret_cast<u32x4*>(dst + i * plane) = __builtin_bit_cast(u32x4, p[i]);
    }
}

// dst[plane][row][kd] <- src rows, zeros from dim to kd.
template <typename T, int PL>
__global__ __launch_bounds__(256) void head_pack_kernel(const T* src, int64_t ld, int64_t rows, int dim,
                                                        bf16_t* dst, int kd, int64_t plane) {
    const int64_t chunks = int64_t(kd / 8) * rows;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / (kd / 8);
        const int c = int(i - r * (kd / 8)) * 8;
        put_planes<PL>(dst + r * kd + c, plane, widen(ld8n(src + r * ld + c, dim - c)));
    }
}

// dst[r][c] <- src[r][c], c < k4: fp32 rows of whole 16 bytes, zeros behind dim.
__global__ __launch_bounds__(256) void head_copy_kernel(const float* src, int64_t ld, int64_t rows, int dim, float* dst,
                                                        int k4) {
    const int64_t chunks = int64_t(k4 / 4) * rows;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / (k4 / 4);
        const int c = int(i - r * (k4 / 4)) * 4;
        const float* p = src + r * ld + c;
        f32x4 v;
        if (c + 4 <= dim) v = *reinterpret_cast<const f32x4_e4*>(p);
        else
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = c + e < dim ? p[e] : 0.f;
        *reinterpret_cast<f32x4*>(dst + r * k4 + c) = v;
    }
}

// dst[plane][c][ldt] <- src[r][c] in 64 x 64 tiles; rows from `rows` up to 64 tr are
// zero, and so are the rows whose coefficient is 0 (they may hold anything).  With
// `packed` the rows as read go there too (head_pack_kernel's layout), so that a
// piece of fp32 W is read once for both.  The tiles are taken in blocks of 8 x 8:
// workgroups that run together then read whole 1 KB pieces of rows and write
// whole 1 KB pieces of columns (302 MB read and written in 63 us, 4.8 TB/s).
template <typename T, int PL>
__global__ __launch_bounds__(256) void head_transpose_kernel(const T* src, int64_t ld, int64_t rows, int dim,
                                                             const float* coef, bf16_t* dst, int64_t ldt,
                                                             int64_t plane, uint32_t tr, uint32_t tc,
                                                             bf16_t* packed, int kd, int64_t packed_plane) {
    __shared__ float tile[64][65];
    const uint32_t blocks_r = (tr + 7) / 8, units = blocks_r * ((tc + 7) / 8) * 64;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint32_t blk = u >> 6, ti = blk % blocks_r * 8 + (u & 7), tj = blk / blocks_r * 8 + (u >> 3 & 7);
        if (ti >= tr || tj >= tc) continue;
        const int64_t r0 = int64_t(ti) * 64;
        const int c0 = int(tj) * 64;
        f32x8 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = threadIdx.x + 256 * i, r = q >> 3, c = (q & 7) * 8;
            const bool on = r0 + r < rows && (!coef || coef[r0 + r] != 0.f);
            v[i] = widen(ld8n(src + (r0 + r) * ld + c0 + c, on ? dim - c0 - c : 0));
        }
        if (u != blockIdx.x) __syncthreads();   // the tile before has been read
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = threadIdx.x + 256 * i, r = q >> 3, c = (q & 7) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) tile[r][c + e] = v[i].v[e];
            if (packed && r0 + r < rows) put_planes<PL>(packed + (r0 + r) * kd + c0 + c, packed_plane, v[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = threadIdx.x + 256 * i, c = q >> 3, r = (q & 7) * 8;
            if (c0 + c >= dim) continue;
            f32x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] = tile[r + e][c];
            put_planes<PL>(dst + int64_t(c0 + c) * ldt + r0 + r, plane, o);
        }
    }
}

// A product with K in splits, one tile of one split per workgroup: the fp32 tile in
// accumulator order (lane by lane, 16 bytes each) is written, or added to what an
// earlier launch wrote there.  out[split][tile row][tile column][wave][block][lane].
struct SplitJob {
    Operand P, Q;
    int dim;
    int nk, stages;
    uint32_t tm, tn, splits, blocks;
    int first;
    f32x4* out;
};
template <int NB, int PL, bool NN>
__device__ __forceinline__ void split_tile(uint8_t* smem, const SplitJob& j, uint32_t block) {
    using L = Layout<NB>;
    uint32_t ti, tj;
    // the splits of a tile are rows of tiles: tile row ti of split s is s tm + ti
    if (!head_tile_of(block, j.tm * j.splits, j.tn, ti, tj)) return;
    const uint32_t sp = ti / j.tm;
    ti -= sp * j.tm;
    const int k0 = int(sp) * j.stages, n = j.nk - k0 < j.stages ? j.nk - k0 : j.stages;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    f32x4* o = j.out + (((int64_t(sp) * j.tm + ti) * j.tn + tj) * 8 + wave) * (L::MB * L::NBW * 64) + lane;
    if (n <= 0) {
        // a short last piece may leave a split without stages
        if (j.first)
#pragma unroll
            for (int i = 0; i < L::MB * L::NBW; ++i) o[i * 64] = f32x4{0.f, 0.f, 0.f, 0.f};
        return;
    }
    f32x4 acc[L::MB][L::NBW];
    w_tile<NB, PL, NN>(smem, j.P, j.dim, j.Q, int64_t(ti) * 256, int64_t(tj) * 64 * NB, k0, n, acc);
#pragma unroll
    for (int a = 0; a < L::MB; ++a)
#pragma unroll
        for (int b = 0; b < L::NBW; ++b) {
            f32x4* q = o + (a * L::NBW + b) * 64;
            f32x4 v = acc[a][b];
            if (!j.first) {
                const f32x4 old = *q;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += old[e];
            }
            *q = v;
        }
}

// The logits (and dW) of a piece with fewer than 128 tiles, which would leave more than half
// of the CUs idle: K is split over the others, and the forward's and the
// backward's epilogues add the splits up in order.  4405 rows x 34 tokens x 4672
// (18 tiles): the forward takes 36 us in bf16, 67 without splits.
template <int NB, int PL>
__global__ __launch_bounds__(H_THREADS) __attribute__((amdgpu_waves_per_eu(2))) void head_split_kernel(SplitJob j) {
    __shared__ __align__(16) uint8_t smem[lds_of(NB, PL)];
    split_tile<NB, PL, false>(smem, j, blockIdx.x);
}
// One wavefront's unit of those sums: 32 rows x 64 tokens of tile (ti, tj).
struct SplitSums {
    const f32x4* z;
    uint32_t tm, tn, splits;
};
template <int NB> struct Unit {
    uint32_t ti, tj;
    int row, col;   // of the unit inside its tile
    f32x4 acc[2][4];
    MO_DEV Unit(const SplitSums& s, uint32_t block) {
        using L = Layout<NB>;
        const uint32_t pair = block % NB, wave = block / NB % 8, tile = block / (8 * NB);
        ti = tile / s.tn;
        tj = tile - ti * s.tn;
        row = int(wave / L::WN * (L::MB * 16) + pair * 32);
        col = int(wave % L::WN * 64);
        const f32x4* q = s.z + (int64_t(tile) * 8 + wave) * (L::MB * L::NBW * 64) + pair * (8 * 64) + (threadIdx.x & 63);
        const int64_t stride = int64_t(s.tm) * s.tn * 8 * (L::MB * L::NBW * 64);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i / 4][i % 4] = q[i * 64];
#pragma unroll 4
        for (uint32_t t = 1; t < s.splits; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const f32x4 x = q[t * stride + i * 64];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i / 4][i % 4][e] += x[e];
            }
    }
};

// ---- forward ----------------------------------------------------------------------

// The labels of a cross entropy (null: none) and where their logits go; v0: vocabulary
// row of the piece's first.
struct Labels {
    const int64_t* ids;
    int64_t tokens, vocab, v0;
    float* z;
    // Row of token n's label below row `first` of the piece, or -1.
    MO_DEV int64_t row(int64_t n, int64_t first) const {
        const int64_t y = ids && n < tokens ? ids[n] : -1;
        return uint64_t(y) < uint64_t(vocab) ? y - v0 - first : -1;
    }
};

// Tile (ti, tj): vocabulary rows 256 ti .. of the piece, tokens TN tj ...  Each
// lane holds 4 MB vocabulary values of one token per column block, so the
// maximum and the sum are mostly in registers.
template <int NB, int PL>
__global__ __launch_bounds__(H_THREADS) __attribute__((amdgpu_waves_per_eu(2))) void head_lse_kernel(
    Operand W, int dim, Operand H, int nk, uint32_t tm, uint32_t tn, float zscale, float2* part, int64_t n_pad,
    Labels labels) {
    using L = Layout<NB>;
    __shared__ __align__(16) uint8_t smem[lds_of(NB, PL)];
    uint32_t ti, tj;
    if (!head_tile_of(blockIdx.x, tm, tn, ti, tj)) return;
    const int64_t v0 = int64_t(ti) * 256, n0 = int64_t(tj) * 64 * NB;
    f32x4 acc[L::MB][L::NBW];
    w_tile<NB, PL, false>(smem, W, dim, H, v0, n0, 0, nk, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / L::WN, wn = wave % L::WN, r16 = lane & 15, kg = lane >> 4;
    const int left = int(W.rows - v0 < 256 ? W.rows - v0 : 256) - wm * (L::MB * 16) - kg * 4;
    float2* st = reinterpret_cast<float2*>(smem);   // [WM][TN]
    const float k2 = zscale * LOG2E;
#pragma unroll
    for (int b = 0; b < L::NBW; ++b) {
        const int64_t n = n0 + wn * 64 + b * 16 + r16, y = labels.row(n, v0 + wm * (L::MB * 16) + kg * 4);
        float m = -__builtin_inff(), s = 0.f;
#pragma unroll
        for (int a = 0; a < L::MB; ++a)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float z = a * 16 + v < left ? acc[a][b][v] : -__builtin_inff();
                acc[a][b][v] = z;
                m = fmaxf(m, z);
            }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float mm = m == -__builtin_inff() ? 0.f : m;   // nothing but -inf: the sum is 0
#pragma unroll
        for (int a = 0; a < L::MB; ++a)
#pragma unroll
            for (int v = 0; v < 4; ++v) s += exp2_hw((acc[a][b][v] - mm) * k2);
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (kg == 0) st[wm * 64 * NB + wn * 64 + b * 16 + r16] = float2{m, s};
        if (uint64_t(y) < uint64_t(L::MB * 16) && (y & 15) < 4)
#pragma unroll
            for (int a = 0; a < L::MB; ++a)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (a * 16 + v == int(y)) labels.z[n] = acc[a][b][v];
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 64 * NB; t += H_THREADS) {
        float m = -__builtin_inff(), s = 0.f;
#pragma unroll
        for (int w = 0; w < L::WM; ++w) m = fmaxf(m, st[w * 64 * NB + t].x);
        const float mm = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
        for (int w = 0; w < L::WM; ++w) s += st[w * 64 * NB + t].y * exp2_hw((st[w * 64 * NB + t].x - mm) * k2);
        part[int64_t(ti) * n_pad + n0 + t] = float2{m, s};
    }
}

// The same from the sums of the splits, one partial per 32 vocabulary rows.
template <int NB>
__global__ __launch_bounds__(64) void head_lse_sum_kernel(SplitSums sums, int64_t rows, float zscale, float2* part,
                                                          int64_t n_pad, Labels labels) {
    const Unit<NB> u(sums, blockIdx.x);
    const int lane = threadIdx.x, r16 = lane & 15, kg = lane >> 4;
    const int64_t v0 = int64_t(u.ti) * 256 + u.row;
    const int left = int(rows - v0 < 32 ? rows - v0 : 32) - kg * 4;
    const float k2 = zscale * LOG2E;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int64_t n = int64_t(u.tj) * (64 * NB) + u.col + b * 16 + r16, y = labels.row(n, v0 + kg * 4);
        float z[8], m = -__builtin_inff(), s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] = i / 4 * 16 + i % 4 < left ? u.acc[i / 4][b][i % 4] : -__builtin_inff();
            m = fmaxf(m, z[i]);
        }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float mm = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += exp2_hw((z[i] - mm) * k2);
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (kg == 0) part[v0 / 32 * n_pad + n] = float2{m, s};
        if (uint64_t(y) < 32 && (y & 15) < 4)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i / 4 * 16 + i % 4 == int(y)) labels.z[n] = z[i];
    }
}

// z[n][j] = H_n . W_id (not yet divided by T), 0 where the id is outside the
// vocabulary: the bits that the logits' product has for it.  A wavefront takes 16
// pairs (n, j) as the rows and columns of one 16 x 16 tile and reads its diagonal: the
// same instructions over the same 32 elements of K, plane pairs and splits in the
// same order, where each output is a sum over its own row and column alone.  One in
// 16 products counts; the loads take longer.  W and H come as the product reads
// them: bf16 as it lies in memory or, PL = 3, the planes of the piece, whose ids alone
// are done then; F32W: W in fp32.  4096 tokens x 64 ids x 2048: 165 us (1.07 GB of W's
// rows; 135 as plain dot products, whose bits the product does not have).
struct TargetJob {
    const void *W, *H;
    int64_t ldw, plane_w, ldh, plane_h;   // elements
    const int64_t* ids;
    int64_t ld_ids, pairs, vocab;
    int64_t v0, rows;   // vocabulary rows behind W
    int k, dim, nk, stages;
    float* z;
};
// Chunk at element e of a row where `on`, else zeros.  FULL: whole chunks, loaded
// without a branch (from the row's start when off).
template <bool FULL, typename T> MO_DEV raw8<T> chunk_if(const T* row, int e, int dim, bool on) {
    if constexpr (FULL) return row8<true>(row, on ? e : 0, on ? dim : 0);
    else return ld8n(row + e, on ? dim - e : 0);
}
template <int PL, bool FULL>
__global__ __launch_bounds__(256) void head_target_kernel(TargetJob j) {
#ifdef __HIP_DEVICE_COMPILE__
    using TW = typename std::conditional<PL == F32W, float, bf16_t>::type;
    constexpr int DEPTH = PL == F32W ? 4 : 8, NSEG = PL == 3 ? 6 : 1, HP = PL == F32W ? 3 : 1;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int64_t items = (j.pairs + 15) / 16;
    for (int64_t it = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); it < items; it += int64_t(gridDim.x) * 4) {
        const int64_t i = it * 16 + r16, at = i < j.pairs ? i : j.pairs - 1, n = at / j.k;
        const int64_t id = i < j.pairs ? j.ids[n * j.ld_ids + (at - n * j.k)] : -1;
        const bool here = uint64_t(id) < uint64_t(j.vocab) && uint64_t(id - j.v0) < uint64_t(j.rows);
        const TW* w = static_cast<const TW*>(j.W) + (here ? id - j.v0 : 0) * j.ldw;
        const bf16_t* h = static_cast<const bf16_t*>(j.H) + n * j.ldh;
        float sum = 0.f;
        if (__ballot(here))
            for (int s0 = 0; s0 < j.nk; s0 += j.stages) {
                // steps of 32 elements of this split; those behind its end add zeros
                const int first = s0 * 2, end = (s0 + j.stages < j.nk ? s0 + j.stages : j.nk) * 2;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int seg = 0; seg < NSEG; ++seg) {
                    const TW* ws = PL == 3 ? w + seg_p<3>(seg) * j.plane_w : w;
                    const bf16_t* hs = PL == 3 ? h + seg_q<3>(seg) * j.plane_h : h;
                    for (int c = first; c < end; c += DEPTH) {
                        raw8<TW> wr[DEPTH];
                        raw8<bf16_t> hr[DEPTH][HP];
#pragma unroll
                        for (int d = 0; d < DEPTH; ++d) {
                            const int e = (c + d) * 32 + kg * 8;
                            const bool on = here && c + d < end;
                            wr[d] = chunk_if<FULL>(ws, e, j.dim, on);
#pragma unroll
                            for (int q = 0; q < HP; ++q) hr[d][q] = chunk_if<(FULL || PL == F32W)>(hs + q * j.plane_h, e, PL == F32W ? j.nk * 64 : j.dim, on);
                        }
#pragma unroll
                        for (int d = 0; d < DEPTH; ++d) {
                            if constexpr (PL == F32W) {
                                bf16x8 wp[3];
                                split_frag(widen(wr[d]).v, wp);
#pragma unroll
                                for (int t = 0; t < 6; ++t)
                                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wp[seg_p<3>(t)], __builtin_bit_cast(bf16x8, hr[d][seg_q<3>(t)].q), acc, 0, 0, 0);
                            } else {
                                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wr[d].q),
                                                                              __builtin_bit_cast(bf16x8, hr[d][0].q), acc, 0, 0, 0);
                            }
                        }
                    }
                }
                // lane l: rows 4 (l / 16) .. + 3, column l mod 16
                float own = acc[0];
#pragma unroll
                for (int v = 1; v < 4; ++v) own = (r16 & 3) == v ? acc[v] : own;
                sum = s0 == 0 ? own : sum + own;
            }
        // ids outside the vocabulary: with the first piece
        if (kg == r16 >> 2 && i < j.pairs && (here || (j.v0 == 0 && uint64_t(id) >= uint64_t(j.vocab)))) j.z[i] = here ? sum : 0.f;
    }
#endif
}

// Partial sums of 8 tokens -> lse, 64 strided shares of the vocabulary's partials per
// token, combined in order.  Cross entropy (labels): the loss, in place of the label's
// logit that the product left in it; otherwise (m, log s) over the token's first
// partial, for the distillation's loss.
__global__ __launch_bounds__(512) void head_combine_kernel(float2* part, int64_t n_pad, int64_t partials,
                                                           int64_t tokens, const int64_t* labels, int64_t vocab,
                                                           float zscale, float* loss, float* lse) {
    __shared__ float2 sh[8][65];
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = int64_t(blockIdx.x) * 8;
    const float k2 = zscale * LOG2E;
    float m = -__builtin_inff(), s = 0.f;
    if (n0 + tx < tokens)
#pragma unroll 4
        for (int64_t t = ty; t < partials; t += 64) {
            const float2 q = part[t * n_pad + n0 + tx];
            const float mn = fmaxf(m, q.x), mm = mn == -__builtin_inff() ? 0.f : mn;
            s = s * exp2_hw((m - mm) * k2) + q.y * exp2_hw((q.x - mm) * k2);
            m = mn;
        }
    sh[tx][ty] = float2{m, s};
    __syncthreads();
    const int64_t n = n0 + wave;
    if (n >= tokens) return;
    const float2 q = sh[wave][lane];
    m = q.x;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float mm = m == -__builtin_inff() ? 0.f : m;
    s = wave_sum(q.y * exp2_hw((q.x - mm) * k2));
    if (lane == 0) {
        const float ls = logf(s);
        const bool in = !labels || uint64_t(labels[n]) < uint64_t(vocab);
        if (labels) loss[n] = in ? ls + (m - loss[n]) * zscale : 0.f;
        else part[n] = float2{m, ls};
        lse[n] = in ? __builtin_fmaf(m, zscale, ls) : 0.f;
    }
}

// One row of the teacher, by one wavefront: the maximum of t over the entries whose id
// is inside the vocabulary, and the sum of exp((t - maximum) / T).  False for a row
// with no such entry, or only entries of -infinity.
MO_DEV bool teacher_row(const int64_t* ids, const void* teacher, bool bf16, int k, int64_t vocab, float inv_t,
                        float& maxt, float& sum) {
    const int lane = threadIdx.x & 63;
    float m = -__builtin_inff();
    for (int j = lane; j < k; j += 64)
        if (uint64_t(ids[j]) < uint64_t(vocab)) m = fmaxf(m, load_elem(teacher, j, bf16));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    float s = 0.f;
    const float mm = m == -__builtin_inff() ? 0.f : m;
    for (int j = lane; j < k; j += 64)
        if (uint64_t(ids[j]) < uint64_t(vocab)) s += expf((load_elem(teacher, j, bf16) - mm) * inv_t);
    sum = wave_sum(s);
    maxt = mm;
    return sum != 0.f;   // NaN counts as live and propagates
}

// loss_n = T^2 sum_j p_j (log p_j - log q_j), log q_j = (z_j - m) / T - log s from the
// combining launch's (m, log s); rows without entries: loss and lse 0.  One wavefront
// per row.
__global__ __launch_bounds__(256) void head_distill_loss_kernel(const int64_t* ids, int64_t ld_ids,
                                                                const void* teacher, int64_t ld_t, bool t_bf16,
                                                                int k, int64_t tokens, int64_t vocab,
                                                                float inv_t, float t, const float* z,
                                                                const float2* ms, float* loss, float* lse) {
    const int lane = threadIdx.x & 63;
    for (int64_t n = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); n < tokens; n += int64_t(gridDim.x) * 4) {
        const int64_t* id = ids + n * ld_ids;
        const uint8_t* te = static_cast<const uint8_t*>(teacher) + n * ld_t * (t_bf16 ? 2 : 4);
        float mt, st;
        const bool live = teacher_row(id, te, t_bf16, k, vocab, inv_t, mt, st);
        const float2 row = ms[n];
        const float lst = logf(st);
        float s = 0.f;
        if (live)
            for (int j = lane; j < k; j += 64) {
                if (uint64_t(id[j]) >= uint64_t(vocab)) continue;
                const float logp = (load_elem(te, j, t_bf16) - mt) * inv_t - lst, p = expf(logp);
                if (p != 0.f) s += p * (logp - ((z[n * k + j] - row.x) * inv_t - row.y));
            }
        s = wave_sum(s);
        if (lane == 0) {
            loss[n] = live ? t * t * s : 0.f;
            if (!live) lse[n] = 0.f;
        }
    }
}

// ---- backward: per-token coefficients ------------------------------------------------

// The scale r: the significand of T times the largest finite |dloss| in the first 64
// rows that hold one other than 0 (1 if none does).  Only the significand: c_n keeps
// the range of dloss.  Every wavefront computes the same.
MO_DEV float ref_scale(const float* dloss, int64_t tokens, float t) {
    for (int64_t n0 = 0; n0 < tokens; n0 += 64) {
        const int64_t n = n0 + (threadIdx.x & 63);
        float m = n < tokens ? __builtin_fabsf(dloss[n]) * t : 0.f;
        if (!(m < __builtin_inff())) m = 0.f;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
        if (m > 0.f) {
            int e;
            return 2.f * frexpf(m, &e);
        }
    }
    return 1.f;
}

// res (bf16): what rounding leaves of delta at a target, for head_residual_kernel.
// coef[n] = T dloss_n / r (0: the row takes no part), nl2[n] = -lse_n log2 e, delta at
// the label, c (exp(z_y - lse) - 1) = c expm1(-loss), and r itself.
__global__ __launch_bounds__(256) void head_xent_prep_kernel(const int64_t* labels, const float* loss,
                                                             const float* lse, const float* dloss,
                                                             int64_t tokens, int64_t n_pad, int64_t vocab,
                                                             float* coef, float* nl2, float* tval,
                                                             float* res, float* ref) {
    const float r = ref_scale(dloss, tokens, 1.f);
    const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (n == 0) *ref = r;
    if (n >= n_pad) return;
    float c = 0.f, l = 0.f;
    if (n < tokens && uint64_t(labels[n]) < uint64_t(vocab)) {
        c = dloss[n] / r;
        l = -lse[n] * LOG2E;
    }
    coef[n] = c;
    nl2[n] = l;
    if (n >= tokens) return;
    const float t = c != 0.f ? c * expm1f(-loss[n]) : 0.f;
    tval[n] = t;
    if (res) res[n] = t - (float)(bf16_t)t;
}

// The same for distillation, one wavefront per row; the entries of an id that a
// row names twice add up, and each of them gets the one value of that id.
__global__ __launch_bounds__(256) void head_distill_prep_kernel(const int64_t* ids, int64_t ld_ids,
                                                                const void* teacher, int64_t ld_t, bool t_bf16,
                                                                int k, int64_t tokens, int64_t n_pad,
                                                                int64_t vocab, float inv_t, float t,
                                                                const float* z, const float* lse,
                                                                const float* dloss, float* coef, float* nl2,
                                                                float* tval, float* res, float* ref) {
    const float r = ref_scale(dloss, tokens, t);
    const int lane = threadIdx.x & 63;
    const int64_t n = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (n == 0 && lane == 0) *ref = r;
    if (n >= n_pad) return;
    float c = 0.f, l = 0.f;
    if (n < tokens) {
        const int64_t* id = ids + n * ld_ids;
        const uint8_t* te = static_cast<const uint8_t*>(teacher) + n * ld_t * (t_bf16 ? 2 : 4);
        float mt, st;
        if (teacher_row(id, te, t_bf16, k, vocab, inv_t, mt, st)) {
            c = t * dloss[n] / r;
            l = lse[n];
        }
        for (int j = lane; j < k; j += 64) {
            const int64_t v = id[j];
            float o = 0.f;
            bool again = false;   // the id has come before
            if (c != 0.f && uint64_t(v) < uint64_t(vocab)) {
                float p = 0.f;
                for (int u = 0; u < k; ++u)
                    if (id[u] == v) {
                        p += expf((load_elem(te, u, t_bf16) - mt) * inv_t) / st;
                        again |= u < j;
                    }
                const float q = expf(__builtin_fmaf(z[n * k + j], inv_t, -l));   // at most 1, as in delta_rows
                o = c * ((q > 1.f ? 1.f : q) - p);
            }
            tval[n * k + j] = o;
            if (res) res[n * k + j] = again ? 0.f : o - (float)(bf16_t)o;
        }
    }
    if (lane == 0) {
        coef[n] = c;
        nl2[n] = -l * LOG2E;
    }
}

// ---- backward: delta of one piece ----------------------------------------------------

// One piece's delta: D[plane][token][piece] for dH and DT[plane][vocabulary row][token]
// for dW, both zero for tokens that take no part and rows behind the vocabulary.
struct DeltaJob {
    Operand W, H;
    int dim, nk;
    uint32_t tm, tn, blocks;
    float zscale;
    const float *coef, *nl2;
    bf16_t *D, *DT;
    int64_t ldd, plane_d, ldt, plane_t;
};
// c and -lse log2 e of the four columns that a lane holds of 64 tokens.
MO_DEV void delta_tokens(const DeltaJob& j, int64_t tok, float (&c)[4], float (&l)[4]) {
    const int r16 = threadIdx.x & 15;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        c[b] = j.coef[tok + b * 16 + r16];
        l[b] = j.nl2[tok + b * 16 + r16];
    }
}
// 32 vocabulary rows x 64 tokens of a wavefront, through its 8 KB of LDS into D
// and DT; `left`: the lane's rows inside the vocabulary.
template <int PL>
__device__ __forceinline__ void delta_rows(uint8_t* st, const DeltaJob& j, const f32x4 (*acc)[4], const float (&c)[4],
                                           const float (&l)[4], int left, int64_t vrow, int64_t tok) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const float k2 = j.zscale * LOG2E;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            f32x4 v4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // at most 1: lse is rounded, by more than a unit where logits pass 2^24
                const float q = exp2_hw(__builtin_fmaf(acc[g][b][e], k2, l[b])), d = c[b] * (q > 1.f ? 1.f : q);
                // rows behind the vocabulary and tokens that take no part
                v4[e] = g * 16 + e < left && c[b] != 0.f ? d : 0.f;
            }
            *reinterpret_cast<f32x4*>(st + st_off(b * 16 + r16, g * 16 + kg * 4)) = v4;
        }
    __builtin_amdgcn_wave_barrier();
    // a token of the block, 8 vocabulary rows
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int col = (lane >> 2) + 16 * t, ic = lane & 3;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(st + st_off(col, ic * 8));
        const f32x4 hi = *reinterpret_cast<const f32x4*>(st + st_off(col, ic * 8 + 4));
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) { v.v[e] = lo[e]; v.v[4 + e] = hi[e]; }
        put_planes<w_planes(PL)>(j.D + (tok + col) * j.ldd + vrow + ic * 8, j.plane_d, v);
    }
    // vocabulary row, 8 tokens
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int cc = lane & 7, row = (lane >> 3) + 8 * t;
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = *reinterpret_cast<const float*>(st + st_off(cc * 8 + e, row));
        put_planes<PL>(j.DT + (vrow + row) * j.ldt + tok + cc * 8, j.plane_t, v);
    }
    __builtin_amdgcn_wave_barrier();
}
template <int NB, int PL>
__device__ __forceinline__ void delta_tile(uint8_t* smem, const DeltaJob& j, uint32_t block) {
    using L = Layout<NB>;
    uint32_t ti, tj;
    if (!head_tile_of(block, j.tm, j.tn, ti, tj)) return;
    const int64_t v0 = int64_t(ti) * 256, n0 = int64_t(tj) * 64 * NB;
    f32x4 acc[L::MB][L::NBW];
    w_tile<NB, w_planes(PL), false>(smem, j.W, j.dim, j.H, v0, n0, 0, j.nk, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / L::WN, wn = wave % L::WN, kg = lane >> 4;
    const int left = int(j.W.rows - v0 < 256 ? j.W.rows - v0 : 256) - wm * (L::MB * 16) - kg * 4;
    uint8_t* st = smem + wave * (32 * 64 * 4);
    float c[4], l[4];
    delta_tokens(j, n0 + wn * 64, c, l);
#pragma unroll
    for (int a = 0; a < L::MB; a += 2)
        delta_rows<PL>(st, j, &acc[a], c, l, left - a * 16, v0 + wm * (L::MB * 16) + a * 16, n0 + wn * 64);
}

// The same from the sums of the splits.
template <int NB, int PL>
__global__ __launch_bounds__(64) void head_delta_sum_kernel(SplitSums sums, DeltaJob j) {
    __shared__ __align__(16) uint8_t st[32 * 64 * 4];
    const Unit<NB> u(sums, blockIdx.x);
    const int64_t v0 = int64_t(u.ti) * 256 + u.row, tok = int64_t(u.tj) * (64 * NB) + u.col;
    const int left = int(j.W.rows - v0 < 32 ? j.W.rows - v0 : 32) - (threadIdx.x >> 4) * 4;
    float c[4], l[4];
    delta_tokens(j, tok, c, l);
    delta_rows<PL>(st, j, u.acc, c, l, left, v0, tok);
}

// delta at the targets that fall into the piece, in both orientations.
template <int PL>
__global__ __launch_bounds__(256) void head_patch_kernel(const int64_t* ids, int64_t ld_ids, int k,
                                                         int64_t pairs, const float* tval, const float* coef,
                                                         int64_t v0, int64_t rows, bf16_t* D, int64_t ldd,
                                                         int64_t plane_d, bf16_t* DT, int64_t ldt,
                                                         int64_t plane_t) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < pairs; i += int64_t(gridDim.x) * 256) {
        const int64_t n = i / k, v = ids[n * ld_ids + (i - n * k)] - v0;
        if (uint64_t(v) >= uint64_t(rows) || coef[n] == 0.f) continue;
        const float x = tval[i];
        bf16_t p[3];
        if constexpr (PL == 1) p[0] = (bf16_t)x;
        else split_f32(x, p[0], p[1], p[2]);
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            if (q < w_planes(PL)) D[q * plane_d + n * ldd + v] = p[q];
            DT[q * plane_t + v * ldt + n] = p[q];
        }
    }
}

// bf16: what delta's rounding at a row's targets takes from its dH, corr[n] =
// sum_j res_nj W[id_nj] (rounded to bf16, a 2^-16th of dH), added before dH is rounded.
// The targets' deltas are the largest of a row, in a batch of few tokens the only
// ones that count.  One wavefront per token and 512 columns, eight rows of W
// requested together: 46 us at 8192
// tokens x 4096, 156 at 4096 x 2048 with 64 targets each (1.07 GB of W's rows, 6.9 TB/s
// with what the caches serve).
__global__ __launch_bounds__(256) void head_residual_kernel(const bf16_t* W, int64_t ldw, const int64_t* ids,
                                                            int64_t ld_ids, int k, const float* res,
                                                            int64_t tokens, int64_t vocab, int dim, bf16_t* corr) {
    const int lane = threadIdx.x & 63, slabs = (dim + 511) / 512;
    const int64_t items = tokens * slabs;
    for (int64_t it = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); it < items; it += int64_t(gridDim.x) * 4) {
        const int64_t n = it / slabs;
        const int c = (int(it - n * slabs) * 64 + lane) * 8;
        f32x8 sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] = 0.f;
        for (int j0 = 0; j0 < k; j0 += 8) {
            float r[8];
            raw8<bf16_t> x[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int64_t v = j0 + g < k ? ids[n * ld_ids + j0 + g] : -1;
                const bool in = uint64_t(v) < uint64_t(vocab);
                r[g] = in ? res[n * k + j0 + g] : 0.f;
                x[g] = ld8n(W + (in ? v : 0) * ldw + c, in ? dim - c : 0);
            }
#pragma unroll
            for (int g = 0; g < 8; ++g)
                if (r[g] != 0.f) {
                    const f32x8 w = widen(x[g]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum.v[e] = __builtin_fmaf(r[g], w.v[e], sum.v[e]);
                }
        }
        st8n(corr + n * dim + c, sum, dim - c);
    }
}

// ---- backward: the two products of a piece --------------------------------------------

// dW rows of the piece = r DT HT^T (K over the tokens), rounded to T.  bf16 with few
// tokens: delta in two planes.  Where that has
// few tiles (a small vocabulary and many tokens) K is split, in a launch of its own
// (head_split_kernel), and head_dw_sum_kernel adds the splits up.  A step of 8000
// tokens x 1000 rows x 256 (4 tiles of 125 stages) takes 88 us in bf16, 181 in
// fp32; 196 and 854 without.
struct DwJob {
    Operand DT, HT;
    int nk;
    uint32_t tm, tn, blocks;
    void* dW;
    int64_t ldw;
    int dim;
    const float* ref;
};
// 32 rows x 64 columns of a wavefront, through its 8 KB of LDS.
template <typename T>
__device__ __forceinline__ void dw_rows(uint8_t* st, const DwJob& j, const f32x4 (*acc)[4], float r, int64_t vrow,
                                        int64_t col) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    T* dW = static_cast<T*>(j.dW);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int g = 0; g < 2; ++g)
            *reinterpret_cast<f32x4*>(st + st_off(b * 16 + r16, g * 16 + kg * 4)) = acc[g][b];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int cc = lane & 7, row = (lane >> 3) + 8 * t;
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = r * *reinterpret_cast<const float*>(st + st_off(cc * 8 + e, row));
        const int64_t vr = vrow + row;
        const int c = int(col) + cc * 8;
        if (vr < j.DT.rows) st8n(dW + vr * j.ldw + c, v, j.dim - c);
    }
    __builtin_amdgcn_wave_barrier();
}
template <typename T, int NB, int PL>
__device__ __forceinline__ void dw_tile(uint8_t* smem, const DwJob& j, uint32_t block) {
    using L = Layout<NB>;
    uint32_t ti, tj;
    if (!head_tile_of(block, j.tm, j.tn, ti, tj)) return;
    const int64_t v0 = int64_t(ti) * 256, c0 = int64_t(tj) * 64 * NB;
    f32x4 acc[L::MB][L::NBW];
    head_tile<NB, dw_planes(PL)>(smem, j.DT, j.HT, v0, c0, 0, j.nk, acc);
    const int wave = threadIdx.x >> 6, wm = wave / L::WN, wn = wave % L::WN;
    const float r = *j.ref;
#pragma unroll
    for (int a = 0; a < L::MB; a += 2)
        dw_rows<T>(smem + wave * (32 * 64 * 4), j, &acc[a], r, v0 + wm * (L::MB * 16) + a * 16, c0 + wn * 64);
}
template <typename T, int NB>
__global__ __launch_bounds__(64) void head_dw_sum_kernel(SplitSums sums, DwJob j) {
    __shared__ __align__(16) uint8_t st[32 * 64 * 4];
    const Unit<NB> u(sums, blockIdx.x);
    dw_rows<T>(st, j, u.acc, *j.ref, int64_t(u.ti) * 256 + u.row, int64_t(u.tj) * (64 * NB) + u.col);
}

// One launch: dW and dH of a piece and delta of the next one.  The three do not
// depend on each other (two sets of D, DT and WT), and together they leave one
// partly filled last round per piece instead of three.  At 8192 tokens x 128256 x
// 4096 (seven pieces) the launches take 18.9 to 19.6 ms for 26 TFLOP, 0.5 more with dH
// before dW and 1.2 more as three launches per piece; without any store it would be
// 17.5 (delta's 4 bytes per logit 0.7, the fp32 sums of dH 0.7, dW 0.3).
template <typename T, int NB, int NBW, int PL>
__global__ __launch_bounds__(H_THREADS) __attribute__((amdgpu_waves_per_eu(2))) void head_step_kernel(
    SplitJob dh, DwJob dw, DeltaJob dl) {
    __shared__ __align__(16) uint8_t smem[lds_of(NB, PL) > head_lds(NBW) ? lds_of(NB, PL) : head_lds(NBW)];
    uint32_t b = blockIdx.x;
    if (b < dw.blocks) {
        dw_tile<T, NBW, PL>(smem, dw, b);
        return;
    }
    b -= dw.blocks;
    if (b < dh.blocks) {
        split_tile<NB, w_planes(PL), true>(smem, dh, b);
        return;
    }
    delta_tile<NB, PL>(smem, dl, b - dh.blocks);
}

// dH <- r times the sum of the splits in order (and corr, in bf16): one workgroup per 16 columns of dH and
// the 64 tokens of a wave's block, turned through LDS.  Tokens that take no part
// get zeros.
template <typename T, int NB>
__global__ __launch_bounds__(256) void head_dh_out_kernel(const f32x4* acc, uint32_t tm, uint32_t tn,
                                                          uint32_t splits, const float* coef, const float* ref,
                                                          const T* corr, T* dH,
                                                          int64_t ld, int64_t tokens, int dim) {
    using L = Layout<NB>;
    __shared__ float tile[64][20];
    const int lane = threadIdx.x & 63, b = threadIdx.x >> 6;
    const int64_t stride = int64_t(tm) * tn * 8 * (L::MB * L::NBW * 64);
    // u: tile, then wave, then row block of the wave
    for (uint32_t u = blockIdx.x; u < tm * tn * 8 * L::MB; u += gridDim.x) {
        const uint32_t a = u % L::MB, wave = u / L::MB % 8, tile_id = u / (L::MB * 8);
        const uint32_t ti = tile_id / tn, tj = tile_id - ti * tn;
        const f32x4* src = acc + (int64_t(tile_id) * 8 + wave) * (L::MB * L::NBW * 64) + (a * L::NBW + b) * 64 + lane;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (uint32_t s = 0; s < splits; ++s) {
            const f32x4 x = src[s * stride];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += x[e];
        }
        if (u != blockIdx.x) __syncthreads();   // the block before has been read
        *reinterpret_cast<f32x4*>(&tile[b * 16 + (lane & 15)][(lane >> 4) * 4]) = v;
        __syncthreads();
        const int64_t n0 = int64_t(tj) * 64 * NB + (wave % L::WN) * 64;
        const int c0 = int(ti) * 256 + int(wave / L::WN) * (16 * L::MB) + int(a) * 16;
        if (threadIdx.x < 128) {
            const int j = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
            if (n0 + j < tokens && c0 + c < dim) {
                const bool on = coef[n0 + j] != 0.f;
                const float r = *ref;
                f32x8 o;
#pragma unroll
                for (int e = 0; e < 8; ++e) o.v[e] = tile[j][c + e];
                if constexpr (sizeof(T) == 2) {
                    const f32x8 x = widen(ld8n(corr + (n0 + j) * dim + c0 + c, dim - c0 - c));
#pragma unroll
                    for (int e = 0; e < 8; ++e) o.v[e] += x.v[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) o.v[e] = on ? r * o.v[e] : 0.f;
                st8n(dH + (n0 + j) * ld + c0 + c, o, dim - c0 - c);
            }
        }
    }
}

// ---- operands ---------------------------------------------------------------------

Operand rows_of(const void* p, int64_t ld_elems, int64_t rows, int64_t plane_elems) {
    return {static_cast<const uint8_t*>(p), ld_elems * 2, rows, plane_elems * 2};
}
Operand h_operand(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws) {
    return p.pack_h ? rows_of(ws + p.off_hp, p.kd, a.tokens, a.tokens * p.kd) : rows_of(a.H, a.ldh, a.tokens, 0);
}
// W's rows of piece k.
Operand w_operand(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows) {
    if (p.f32w && p.pack_w) return {ws + p.off_wt[k & 1], p.k4 * 4, rows, 0};
    if (p.f32w) return {static_cast<const uint8_t*>(a.W) + v0 * a.ldw * 4, a.ldw * 4, rows, 0};
    return p.pack_w ? rows_of(ws + p.off_wp, p.kd, rows, p.piece * p.kd)
                    : rows_of(static_cast<const bf16_t*>(a.W) + v0 * a.ldw, a.ldw, rows, 0);
}

unsigned cap_grid(int64_t want, int64_t cap) { return unsigned(want < 1 ? 1 : want < cap ? want : cap); }

template <typename K, typename... A>
hipError_t go(K* kernel, dim3 grid, dim3 block, hipStream_t s, A... args) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, args...);
    return hipGetLastError();
}

}  // namespace

// Calls `f` with the plan's tile width and plane count as template arguments.
#define MO_HEAD_PICK(NBV, PLV, CALL)                                    \
    do {                                                                \
        if ((PLV) == 1) {                                               \
            if ((NBV) == 4) { CALL(4, 1); }                             \
            if ((NBV) == 2) { CALL(2, 1); }                             \
            CALL(1, 1);                                                 \
        }                                                               \
        if ((NBV) == 4) { CALL(4, 3); }                                 \
        if ((NBV) == 2) { CALL(2, 3); }                                 \
        CALL(1, 3);                                                     \
    } while (0)

hipError_t mo_launch_head_pack(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, bool h, int64_t v0,
                               int64_t rows, hipStream_t s) {
    const int64_t ld = h ? a.ldh : a.ldw;
    bf16_t* dst = reinterpret_cast<bf16_t*>(ws + (h ? p.off_hp : p.off_wp));
    const int64_t plane = (h ? a.tokens : p.piece) * p.kd;
    const dim3 grid(cap_grid((rows * (p.kd / 8) + 255) / 256, 1 << 16)), block(256);
    if (p.planes == 1)
        return go(head_pack_kernel<bf16_t, 1>, grid, block, s, static_cast<const bf16_t*>(h ? a.H : a.W) + v0 * ld, ld,
                  rows, int(a.dim), dst, int(p.kd), plane);
    return go(head_pack_kernel<float, 3>, grid, block, s, static_cast<const float*>(h ? a.H : a.W) + v0 * ld, ld, rows,
              int(a.dim), dst, int(p.kd), plane);
}

// Piece k of an fp32 W whose rows are not whole 16 bytes.
hipError_t mo_launch_head_copy(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                               hipStream_t s) {
    const dim3 grid(cap_grid((rows * (p.k4 / 4) + 255) / 256, 1 << 16)), block(256);
    return go(head_copy_kernel, grid, block, s, static_cast<const float*>(a.W) + v0 * a.ldw, a.ldw, rows, int(a.dim),
              reinterpret_cast<float*>(ws + p.off_wt[k & 1]), int(p.k4));
}

// The splits of a piece's logits, and where their sums are read.
static hipError_t split_logits(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, const Operand& W,
                               SplitSums* sums, hipStream_t s) {
    SplitJob j = {};
    j.P = W;
    j.Q = h_operand(a, p, ws);
    j.dim = int(p.k4);
    j.nk = int(p.kd / 64);
    j.stages = p.z_stages;
    j.tm = uint32_t((W.rows + 255) / 256);
    j.tn = uint32_t(p.n_pad / (64 * p.nb));
    j.splits = uint32_t(p.z_splits);
    j.first = 1;
    j.out = reinterpret_cast<f32x4*>(ws + p.off_z);
    *sums = {j.out, j.tm, j.tn, j.splits};
    const dim3 grid(head_grid(uint64_t(j.tm) * j.tn * j.splits)), block(H_THREADS);
    if (p.f32w) return go(head_split_kernel<1, F32W>, grid, block, s, j);
#define MO_CALL(NB, PL) return go(head_split_kernel<NB, PL>, grid, block, s, j)
    MO_HEAD_PICK(p.nb, p.planes, MO_CALL);
#undef MO_CALL
}

hipError_t mo_launch_head_lse(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int64_t v0, int64_t rows,
                              hipStream_t s) {
    const Operand H = h_operand(a, p, ws), W = w_operand(a, p, ws, 0, v0, rows);
    const uint32_t tm = uint32_t((rows + 255) / 256), tn = uint32_t(p.n_pad / (64 * p.nb));
    float2* part = reinterpret_cast<float2*>(ws + p.off_part) + v0 / 256 * p.n_pad * (p.z_splits > 1 ? 8 : 1);
    const Labels labels = {a.teacher ? nullptr : a.ids, a.tokens, a.vocab, v0, a.loss};
    if (p.z_splits > 1) {
        SplitSums sums;
        const hipError_t e = split_logits(a, p, ws, W, &sums, s);
        if (e != hipSuccess) return e;
        const dim3 units(tm * tn * 8 * uint32_t(p.nb)), wave(64);
        if (p.nb == 4) return go(head_lse_sum_kernel<4>, units, wave, s, sums, rows, a.inv_t, part, p.n_pad, labels);
        if (p.nb == 2) return go(head_lse_sum_kernel<2>, units, wave, s, sums, rows, a.inv_t, part, p.n_pad, labels);
        return go(head_lse_sum_kernel<1>, units, wave, s, sums, rows, a.inv_t, part, p.n_pad, labels);
    }
    const dim3 grid(head_grid(uint64_t(tm) * tn)), block(H_THREADS);
    if (p.f32w)
        return go(head_lse_kernel<1, F32W>, grid, block, s, W, int(p.k4), H, int(p.kd / 64), tm, tn, a.inv_t, part,
                  p.n_pad, labels);
#define MO_CALL(NB, PL)                                                                                              \
    return go(head_lse_kernel<NB, PL>, grid, block, s, W, int(a.dim), H, int(p.kd / 64), tm, tn, a.inv_t, part, p.n_pad, \
              labels)
    MO_HEAD_PICK(p.nb, p.planes, MO_CALL);
#undef MO_CALL
}

// The logits of the ids among `rows` vocabulary rows from v0 on.
hipError_t mo_launch_head_targets(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int64_t v0, int64_t rows,
                                  hipStream_t s) {
    TargetJob j = {};
    j.ids = a.ids;
    j.ld_ids = a.ld_ids;
    j.pairs = a.tokens * a.k;
    j.vocab = a.vocab;
    j.v0 = v0;
    j.rows = rows;
    j.k = a.k;
    j.nk = int(p.kd / 64);
    j.stages = p.z_stages;
    j.z = a.z;
    const bool planes = p.planes == 3 && !p.f32w;
    j.W = planes ? ws + p.off_wp : static_cast<const uint8_t*>(a.W) + v0 * a.ldw * (p.planes == 1 ? 2 : 4);
    j.ldw = planes ? p.kd : a.ldw;
    j.plane_w = p.piece * p.kd;
    j.H = p.planes == 3 ? ws + p.off_hp : a.H;
    j.ldh = p.planes == 3 ? p.kd : a.ldh;
    j.plane_h = a.tokens * p.kd;
    j.dim = int(planes ? p.kd : a.dim);
    const dim3 grid(cap_grid((j.pairs + 63) / 64, 1 << 20)), block(256);
    if (planes) return go(head_target_kernel<3, true>, grid, block, s, j);
    const bool full = a.dim % 8 == 0;
    if (p.f32w) return go(full ? head_target_kernel<F32W, true> : head_target_kernel<F32W, false>, grid, block, s, j);
    return go(full ? head_target_kernel<1, true> : head_target_kernel<1, false>, grid, block, s, j);
}

hipError_t mo_launch_head_loss(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s) {
    float2* part = reinterpret_cast<float2*>(ws + p.off_part);
    const int64_t partials = p.v_tiles * (p.z_splits > 1 ? 8 : 1);
    const hipError_t e = go(head_combine_kernel, dim3(unsigned((a.tokens + 7) / 8)), dim3(512), s, part, p.n_pad, partials,
                            a.tokens, a.teacher ? nullptr : a.ids, a.vocab, a.inv_t, a.loss, a.lse);
    if (e != hipSuccess || !a.teacher) return e;
    return go(head_distill_loss_kernel, dim3(cap_grid((a.tokens + 3) / 4, 1 << 20)), dim3(256), s, a.ids, a.ld_ids,
              a.teacher, a.ld_teacher, a.teacher_dtype == MO_BF16, a.k, a.tokens, a.vocab, a.inv_t, a.t,
              static_cast<const float*>(a.z), static_cast<const float2*>(part), a.loss, a.lse);
}

hipError_t mo_launch_head_prep(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s) {
    float *coef = reinterpret_cast<float*>(ws + p.off_coef), *nl2 = reinterpret_cast<float*>(ws + p.off_nl2);
    float *tval = reinterpret_cast<float*>(ws + p.off_tval), *ref = reinterpret_cast<float*>(ws + p.off_ref);
    float* res = p.planes == 1 && a.dH ? reinterpret_cast<float*>(ws + p.off_res) : nullptr;
    if (!a.teacher)
        return go(head_xent_prep_kernel, dim3(unsigned((p.n_pad + 255) / 256)), dim3(256), s, a.ids, a.loss_in,
                  a.lse_in, a.dloss, a.tokens, p.n_pad, a.vocab, coef, nl2, tval, res, ref);
    return go(head_distill_prep_kernel, dim3(unsigned((p.n_pad + 3) / 4)), dim3(256), s, a.ids, a.ld_ids, a.teacher,
              a.ld_teacher, a.teacher_dtype == MO_BF16, a.k, a.tokens, p.n_pad, a.vocab, a.inv_t, a.t, a.z_in,
              a.lse_in, a.dloss, coef, nl2, tval, res, ref);
}

// Transposes `rows` rows (and pads them to tr tiles of 64); with `packed` copies them too.
static hipError_t transpose(const MoHeadArgs& a, const MoHeadPlan& p, const void* src, int64_t ld, int64_t rows,
                            uint32_t tr, const float* coef, uint8_t* dst, int64_t ldt, uint8_t* packed,
                            int64_t packed_rows, hipStream_t s) {
    // whole stages of the copy: the columns behind dim are its zeros
    const uint32_t tc = uint32_t(((packed ? p.kd : a.dim) + 63) / 64);
    const dim3 grid(cap_grid(int64_t((tr + 7) / 8 * ((tc + 7) / 8)) * 64, 1 << 20)), block(256);
    bf16_t *d = reinterpret_cast<bf16_t*>(dst), *k = reinterpret_cast<bf16_t*>(packed);
    if (p.planes == 1)
        return go(head_transpose_kernel<bf16_t, 1>, grid, block, s, static_cast<const bf16_t*>(src), ld, rows,
                  int(a.dim), coef, d, ldt, a.dim * ldt, tr, tc, k, int(p.kd), packed_rows * p.kd);
    return go(head_transpose_kernel<float, 3>, grid, block, s, static_cast<const float*>(src), ld, rows, int(a.dim),
              coef, d, ldt, a.dim * ldt, tr, tc, k, int(p.kd), packed_rows * p.kd);
}

hipError_t mo_launch_head_ht(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s) {
    return transpose(a, p, a.H, a.ldh, a.tokens, uint32_t(p.n_pad / 64),
                     reinterpret_cast<const float*>(ws + p.off_coef), ws + p.off_ht, p.ld_t, nullptr, 0, s);
}

hipError_t mo_launch_head_wt(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                             hipStream_t s) {
    const uint8_t* w = static_cast<const uint8_t*>(a.W) + v0 * a.ldw * (p.planes == 1 ? 2 : 4);
    return transpose(a, p, w, a.ldw, rows, uint32_t((rows + 255) / 256 * 4), nullptr, ws + p.off_wt[k & 1], p.ld_p,
                     p.pack_w ? ws + p.off_wp : nullptr, p.piece, s);
}

hipError_t mo_launch_head_patch(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                                hipStream_t s) {
    const int64_t pairs = a.tokens * a.k;
    const float *coef = reinterpret_cast<const float*>(ws + p.off_coef),
                *tval = reinterpret_cast<const float*>(ws + p.off_tval);
    bf16_t *D = reinterpret_cast<bf16_t*>(ws + p.off_d[k & 1]), *DT = reinterpret_cast<bf16_t*>(ws + p.off_dt[k & 1]);
    const dim3 grid(cap_grid((pairs + 255) / 256, 1 << 16)), block(256);
    if (p.planes == 1)
        return go(p.dt_planes == 2 ? head_patch_kernel<2> : head_patch_kernel<1>, grid, block, s, a.ids, a.ld_ids, a.k, pairs, tval, coef, v0, rows, D, p.ld_p,
                  p.n_pad * p.ld_p, DT, p.ld_t, p.piece * p.ld_t);
    return go(head_patch_kernel<3>, grid, block, s, a.ids, a.ld_ids, a.k, pairs, tval, coef, v0, rows, D, p.ld_p,
              p.n_pad * p.ld_p, DT, p.ld_t, p.piece * p.ld_t);
}

static DeltaJob delta_job(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows) {
    DeltaJob dl = {};
    dl.W = w_operand(a, p, ws, k, v0, rows);
    dl.H = h_operand(a, p, ws);
    dl.dim = int(p.k4);
    dl.nk = int(p.kd / 64);
    dl.tm = uint32_t((rows + 255) / 256);
    dl.tn = uint32_t(p.n_pad / (64 * p.nb));
    dl.zscale = a.inv_t;
    dl.coef = reinterpret_cast<const float*>(ws + p.off_coef);
    dl.nl2 = reinterpret_cast<const float*>(ws + p.off_nl2);
    dl.D = reinterpret_cast<bf16_t*>(ws + p.off_d[k & 1]);
    dl.DT = reinterpret_cast<bf16_t*>(ws + p.off_dt[k & 1]);
    dl.ldd = p.ld_p;
    dl.plane_d = p.n_pad * p.ld_p;
    dl.ldt = p.ld_t;
    dl.plane_t = p.piece * p.ld_t;
    dl.blocks = head_grid(uint64_t(dl.tm) * dl.tn);
    return dl;
}

// delta of piece k from the splits of its logits.
hipError_t mo_launch_head_delta_split(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0,
                                      int64_t rows, hipStream_t s) {
    const DeltaJob dl = delta_job(a, p, ws, k, v0, rows);
    SplitSums sums;
    const hipError_t e = split_logits(a, p, ws, dl.W, &sums, s);
    if (e != hipSuccess) return e;
    const dim3 units(dl.tm * dl.tn * 8 * uint32_t(p.nb)), wave(64);
#define MO_CALL(NB, PL) return go(head_delta_sum_kernel<NB, PL>, units, wave, s, sums, dl)
    if (p.dt_planes == 2) {   // at most 128 tokens
        if (p.nb == 2) MO_CALL(2, 2);
        MO_CALL(1, 2);
    }
    MO_HEAD_PICK(p.nb, p.planes, MO_CALL);
#undef MO_CALL
}

// Piece k (rows from v0 on; rows 0: none) of dH and dW, and delta of piece k + 1
// (next_rows 0: none).
hipError_t mo_launch_head_step(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, int k, int64_t v0, int64_t rows,
                               int64_t next_v0, int64_t next_rows, hipStream_t s) {
    SplitJob dh = {};
    DwJob dw = {};
    DeltaJob dl = {};
    const uint32_t tn = uint32_t(p.n_pad / (64 * p.nb)), tm = uint32_t((rows + 255) / 256);
    if (rows && a.dH) {
        dh.P = p.f32w ? w_operand(a, p, ws, k, v0, rows) : rows_of(ws + p.off_wt[k & 1], p.ld_p, a.dim, a.dim * p.ld_p);
        dh.dim = int(p.k4);
        dh.Q = rows_of(ws + p.off_d[k & 1], p.ld_p, p.n_pad, p.n_pad * p.ld_p);
        dh.nk = int(tm * 4);   // the piece's rows, rounded up to whole tiles
        dh.stages = p.dh_stages;
        dh.tm = p.dh_tm;
        dh.tn = p.dh_tn;
        dh.splits = uint32_t(p.dh_splits);
        dh.first = k == 0;
        dh.out = reinterpret_cast<f32x4*>(ws + p.off_acc);
        dh.blocks = head_grid(uint64_t(dh.tm) * dh.tn * dh.splits);
    }
    if (rows && a.dW) {
        dw.DT = rows_of(ws + p.off_dt[k & 1], p.ld_t, rows, p.piece * p.ld_t);
        dw.HT = rows_of(ws + p.off_ht, p.ld_t, a.dim, a.dim * p.ld_t);
        dw.nk = int((a.tokens + 63) / 64);
        dw.tm = tm;
        dw.tn = uint32_t((a.dim + 64 * p.nb_dw - 1) / (64 * p.nb_dw));
        dw.dW = static_cast<uint8_t*>(a.dW) + v0 * a.lddw * (p.planes == 1 ? 2 : 4);
        dw.ldw = a.lddw;
        dw.dim = int(a.dim);
        dw.ref = reinterpret_cast<const float*>(ws + p.off_ref);
        dw.blocks = p.dw_splits > 1 ? 0 : head_grid(uint64_t(dw.tm) * dw.tn);
    }
    if (next_rows) dl = delta_job(a, p, ws, k + 1, next_v0, next_rows);
    const dim3 grid(dh.blocks + dw.blocks + dl.blocks), block(H_THREADS);
    hipError_t e = hipSuccess;
#define MO_STEP(T, NB, PL)                                                                             \
    e = p.nb_dw == 4 ? go(head_step_kernel<T, NB, 4, PL>, grid, block, s, dh, dw, dl)               \
                     : go(head_step_kernel<T, NB, 1, PL>, grid, block, s, dh, dw, dl)
    if (grid.x == 0) {
        // dW alone, in splits
    } else if (p.dt_planes == 2) {
        if (p.nb == 2) MO_STEP(bf16_t, 2, 2);
        else MO_STEP(bf16_t, 1, 2);
    } else if (p.planes == 1) {
        if (p.nb == 4) MO_STEP(bf16_t, 4, 1);
        else if (p.nb == 2) MO_STEP(bf16_t, 2, 1);
        else MO_STEP(bf16_t, 1, 1);
    } else if (p.f32w) MO_STEP(float, 1, F32W);
    else if (p.nb == 4) MO_STEP(float, 4, 3);
    else if (p.nb == 2) MO_STEP(float, 2, 3);
    else MO_STEP(float, 1, 3);
#undef MO_STEP
    if (e != hipSuccess || !dw.tm || p.dw_splits == 1) return e;
    SplitJob j = {};
    j.P = dw.DT;
    j.Q = dw.HT;
    j.nk = dw.nk;
    j.stages = p.dw_stages;
    j.tm = dw.tm;
    j.tn = dw.tn;
    j.splits = uint32_t(p.dw_splits);
    j.first = 1;
    j.out = reinterpret_cast<f32x4*>(ws + p.off_dw);
    const SplitSums sums = {j.out, j.tm, j.tn, j.splits};
    const dim3 sgrid(head_grid(uint64_t(j.tm) * j.tn * j.splits)), units(j.tm * j.tn * 8 * uint32_t(p.nb_dw)), wave(64);
    const bool wide = p.nb_dw == 4;
    if (p.planes == 1) {
        e = go(wide ? head_split_kernel<4, 1> : head_split_kernel<1, 1>, sgrid, block, s, j);
        if (e != hipSuccess) return e;
        return go(wide ? head_dw_sum_kernel<bf16_t, 4> : head_dw_sum_kernel<bf16_t, 1>, units, wave, s, sums, dw);
    }
    e = go(wide ? head_split_kernel<4, 3> : head_split_kernel<1, 3>, sgrid, block, s, j);
    if (e != hipSuccess) return e;
    return go(wide ? head_dw_sum_kernel<float, 4> : head_dw_sum_kernel<float, 1>, units, wave, s, sums, dw);
}

hipError_t mo_launch_head_dh_out(const MoHeadArgs& a, const MoHeadPlan& p, uint8_t* ws, hipStream_t s) {
    const f32x4* acc = reinterpret_cast<const f32x4*>(ws + p.off_acc);
    const float *coef = reinterpret_cast<const float*>(ws + p.off_coef),
                *ref = reinterpret_cast<const float*>(ws + p.off_ref);
    // 8 waves x MB row blocks, MB = 2 NB
    const dim3 grid(cap_grid(int64_t(p.dh_tm) * p.dh_tn * 16 * p.nb, 1 << 20)), block(256);
    void* corr = ws + p.off_corr;
    if (p.planes == 1) {
        const dim3 items(cap_grid((a.tokens * ((a.dim + 511) / 512) + 3) / 4, 1 << 20));
        const hipError_t e = go(head_residual_kernel, items, block, s, static_cast<const bf16_t*>(a.W), a.ldw, a.ids,
                                a.ld_ids, a.k, reinterpret_cast<const float*>(ws + p.off_res), a.tokens, a.vocab,
                                int(a.dim), static_cast<bf16_t*>(corr));
        if (e != hipSuccess) return e;
    }
#define MO_OUT(T, NB)                                                                                    \
    return go(head_dh_out_kernel<T, NB>, grid, block, s, acc, p.dh_tm, p.dh_tn, uint32_t(p.dh_splits), coef, ref, \
              static_cast<const T*>(corr), static_cast<T*>(a.dH), a.lddh, a.tokens, int(a.dim))
    if (p.planes == 1) {
        if (p.nb == 4) MO_OUT(bf16_t, 4);
        if (p.nb == 2) MO_OUT(bf16_t, 2);
        MO_OUT(bf16_t, 1);
    }
    if (p.nb == 4) MO_OUT(float, 4);
    if (p.nb == 2) MO_OUT(float, 2);
    MO_OUT(float, 1);
#undef MO_OUT
}
