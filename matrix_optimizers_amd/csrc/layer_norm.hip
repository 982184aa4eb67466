// Layer norm over the rows of a matrix, forward and backward.
//
//   mu = mean(x), r = (mean((x - mu)^2) + eps)^-1/2, y = (x - mu) r w + b
//   g = dy w, xh = (x - mu) r
//   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Every element is read once and written once: a row lives in the registers of
// its threads between the reductions and the result.  Statistics and sums are
// fp32; the variance is the mean of squared differences from the finished mean
// (no cancellation for rows with a large mean or a single large entry).  The
// means are quotients, not products with a rounded 1 / cols, so that a constant
// row whose sum is exact has variance 0.
#include "op_common.h"
#include "operators.h"
#include "row_team.h"

namespace {

constexpr int LN_MAX_THREADS = TEAM_MAX_THREADS;

// One row per team: W <= 64 threads (256 / W rows per workgroup) or, W = 1024,
// the whole workgroup of blockDim.x threads.  Thread t of a team holds the
// 8-element chunks t, t + team, .. (R of them); the next row is requested before
// this one's reductions.
template <typename T, int W, int R, bool FULL>
__global__ __launch_bounds__(W > 64 ? LN_MAX_THREADS : 256) void ln_fwd_kernel(
    const T* X, int64_t ldx, const float* weight, const float* bias, T* Y, int64_t ldy, float* mean,
    float* rstd, int64_t rows, int cols, float eps) {
    __shared__ float red[32];
    const int team = W > 64 ? blockDim.x : W, teams = W > 64 ? 1 : 256 / W;
    const int t = W > 64 ? threadIdx.x : threadIdx.x % W;
    const int sub = W > 64 ? 0 : threadIdx.x / W;
    const int64_t step = int64_t(gridDim.x) * teams;
    int turn = 0;
    raw8<T> next[R];
    auto request = [&](int64_t row) __attribute__((always_inline)) {
        const T* x = X + (row < rows ? row : rows - 1) * ldx;
#pragma unroll
        for (int i = 0; i < R; ++i) next[i] = row8<FULL>(x, (t + team * i) * 8, cols);
    };
    request(int64_t(blockIdx.x) * teams + sub);
    f32x8 w[R], b[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (t + team * i) * 8;
        if (weight) w[i] = widen(row8<FULL>(weight, c, cols));
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i].v[e] = 1.f;
        if (bias) b[i] = widen(row8<FULL>(bias, c, cols));
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) b[i].v[e] = 0.f;
    }
    const float n_cols = float(cols);
    for (int64_t base = int64_t(blockIdx.x) * teams; base < rows; base += step) {
        const int64_t row = base + sub;
        const bool live = row < rows;
        f32x8 x[R];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            x[i] = widen(next[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += x[i].v[e];
        }
        if (base + step < rows) request(row + step);
        team_sum<W>(s, red, turn);
        const float mu = s[0] / n_cols;
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (t + team * i) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[i].v[e] -= mu;
                if (c + (FULL ? 0 : e) < cols) q[0] += x[i].v[e] * x[i].v[e];
            }
        }
        team_sum<W>(q, red, turn);
        const float r = 1.0f / sqrtf(q[0] / n_cols + eps);
        if (live) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                f32x8 y;
#pragma unroll
                for (int e = 0; e < 8; ++e) y.v[e] = x[i].v[e] * r * w[i].v[e] + b[i].v[e];
                row8_out<FULL>(Y + row * ldy, (t + team * i) * 8, cols, y);
            }
            if (t == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = r;
            }
        }
    }
}

// Rows too long for registers: one workgroup per row, re-read per pass.
template <typename T>
__global__ __launch_bounds__(LN_MAX_THREADS) void ln_fwd_long_kernel(
    const T* X, int64_t ldx, const float* weight, const float* bias, T* Y, int64_t ldy, float* mean,
    float* rstd, int64_t rows, int cols, float eps) {
    __shared__ float red[32];
    int turn = 0;
    const float n_cols = float(cols);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* x = X + row * ldx;
        float s[1] = {0.f};
        for (int c = threadIdx.x * 8; c < cols; c += LN_MAX_THREADS * 8) {
            const f32x8 v = widen(ld8n(x + c, cols - c));
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v.v[e];
        }
        team_sum<LN_MAX_THREADS>(s, red, turn);
        const float mu = s[0] / n_cols;
        float q[1] = {0.f};
        for (int c = threadIdx.x * 8; c < cols; c += LN_MAX_THREADS * 8) {
            const f32x8 v = widen(ld8n(x + c, cols - c));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) q[0] += (v.v[e] - mu) * (v.v[e] - mu);
        }
        team_sum<LN_MAX_THREADS>(q, red, turn);
        const float r = 1.0f / sqrtf(q[0] / n_cols + eps);
        for (int c = threadIdx.x * 8; c < cols; c += LN_MAX_THREADS * 8) {
            f32x8 v = widen(ld8n(x + c, cols - c));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols)
                    v.v[e] = (v.v[e] - mu) * r * (weight ? weight[c + e] : 1.f) + (bias ? bias[c + e] : 0.f);
            st8n(Y + row * ldy + c, v, cols - c);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
        }
    }
}

// dx, and this workgroup's share of dw and db: a thread's columns stay the
// same over the rows it walks, so the two sums live in its registers and leave
// one fp32 partial row per workgroup (part[wg][0] = dw, part[wg][1] = db).
template <typename T, int W, int R, bool FULL>
__global__ __launch_bounds__(W > 64 ? LN_MAX_THREADS : 256) void ln_bwd_kernel(
    const T* dY, int64_t lddy, const T* X, int64_t ldx, const float* weight, const float* mean,
    const float* rstd, T* dX, int64_t lddx, float* part, int64_t rows, int cols) {
    __shared__ float red[64];
    __shared__ float comb[W > 64 ? 1 : 256 * 8];
    const int team = W > 64 ? blockDim.x : W, teams = W > 64 ? 1 : 256 / W;
    const int t = W > 64 ? threadIdx.x : threadIdx.x % W;
    const int sub = W > 64 ? 0 : threadIdx.x / W;
    const int64_t step = int64_t(gridDim.x) * teams;
    int turn = 0;
    f32x8 dw[R], db[R], w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) { dw[i].v[e] = 0.f; db[i].v[e] = 0.f; w[i].v[e] = 1.f; }
        if (weight) w[i] = widen(row8<FULL>(weight, (t + team * i) * 8, cols));
    }
    const float n_cols = float(cols);
    for (int64_t base = int64_t(blockIdx.x) * teams; base < rows; base += step) {
        const int64_t row = base + sub;
        const bool live = row < rows;
        const int64_t at = live ? row : rows - 1;
        const float mu = mean[at], r = rstd[at];
        raw8<T> x[R], dy[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            x[i] = row8<FULL>(X + at * ldx, (t + team * i) * 8, cols);
            dy[i] = row8<FULL>(dY + at * lddy, (t + team * i) * 8, cols);
        }
        float s[2] = {0.f, 0.f};
        if (live) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const f32x8 xv = widen(x[i]), gv = widen(dy[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = (xv.v[e] - mu) * r, g = gv.v[e] * w[i].v[e];
                    s[0] += g;
                    s[1] += g * xh;
                    dw[i].v[e] += gv.v[e] * xh;
                    db[i].v[e] += gv.v[e];
                }
            }
        }
        if (dX) {
            team_sum<W>(s, red, turn);
            const float m1 = s[0] / n_cols, m2 = s[1] / n_cols;
            if (live) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const f32x8 xv = widen(x[i]), gv = widen(dy[i]);
                    f32x8 o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float xh = (xv.v[e] - mu) * r, g = gv.v[e] * w[i].v[e];
                        o.v[e] = r * (g - m1 - xh * m2);
                    }
                    row8_out<FULL>(dX + row * lddx, (t + team * i) * 8, cols, o);
                }
            }
        }
    }
    if (!part) return;
    float* p = part + int64_t(blockIdx.x) * 2 * cols;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (W > 64) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = (t + team * i) * 8;
                st8n(p + int64_t(k) * cols + c, k ? db[i] : dw[i], cols - c);
            }
        } else {
            // R == 1: the workgroup's rows in row order
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) comb[threadIdx.x * 8 + e] = k ? db[0].v[e] : dw[0].v[e];
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += 256) {
                float a = 0.f;
                for (int u = 0; u < teams; ++u) a += comb[u * W * 8 + c];
                p[int64_t(k) * cols + c] = a;
            }
        }
    }
}

// Long rows, first the two sums and dx, one workgroup per row ..
template <typename T>
__global__ __launch_bounds__(LN_MAX_THREADS) void ln_bwd_long_kernel(
    const T* dY, int64_t lddy, const T* X, int64_t ldx, const float* weight, const float* mean,
    const float* rstd, T* dX, int64_t lddx, int64_t rows, int cols) {
    __shared__ float red[64];
    int turn = 0;
    const float n_cols = float(cols);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float mu = mean[row], r = rstd[row];
        const T *x = X + row * ldx, *dy = dY + row * lddy;
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x * 8; c < cols; c += LN_MAX_THREADS * 8) {
            const f32x8 xv = widen(ld8n(x + c, cols - c)), gv = widen(ld8n(dy + c, cols - c));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) {
                    const float g = gv.v[e] * (weight ? weight[c + e] : 1.f);
                    s[0] += g;
                    s[1] += g * ((xv.v[e] - mu) * r);
                }
        }
        team_sum<LN_MAX_THREADS>(s, red, turn);
        const float m1 = s[0] / n_cols, m2 = s[1] / n_cols;
        for (int c = threadIdx.x * 8; c < cols; c += LN_MAX_THREADS * 8) {
            const f32x8 xv = widen(ld8n(x + c, cols - c)), gv = widen(ld8n(dy + c, cols - c));
            f32x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) {
                    const float g = gv.v[e] * (weight ? weight[c + e] : 1.f);
                    o.v[e] = r * (g - m1 - (xv.v[e] - mu) * r * m2);
                }
            st8n(dX + row * lddx + c, o, cols - c);
        }
    }
}
// .. then partial dw and db of a strided share of the rows (blockIdx.y) for
// 2048 columns (blockIdx.x).
template <typename T>
__global__ __launch_bounds__(256) void ln_bwd_long_wb_kernel(const T* dY, int64_t lddy, const T* X,
                                                             int64_t ldx, const float* mean,
                                                             const float* rstd, float* part,
                                                             int64_t rows, int cols) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= cols) return;
    f32x8 dw, db;
#pragma unroll
    for (int e = 0; e < 8; ++e) { dw.v[e] = 0.f; db.v[e] = 0.f; }
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float mu = mean[row], r = rstd[row];
        const f32x8 xv = widen(ld8n(X + row * ldx + c, cols - c)), gv = widen(ld8n(dY + row * lddy + c, cols - c));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw.v[e] += gv.v[e] * ((xv.v[e] - mu) * r);
            db.v[e] += gv.v[e];
        }
    }
    float* p = part + int64_t(blockIdx.y) * 2 * cols + c;
    st8n(p, dw, cols - c);
    st8n(p + cols, db, cols - c);
}

// dw (blockIdx.y = 0) and db (1): the partial rows of each column in a fixed
// order, 32 columns by 32 strided shares per workgroup.
__global__ __launch_bounds__(1024) void ln_reduce_kernel(const float* part, int n_part, float* dweight,
                                                         float* dbias, int cols) {
    __shared__ float sum[32][33];
    float* out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    float a = 0.f;
    if (c < cols)
        for (int g = ty; g < n_part; g += 32) a += part[(int64_t(g) * 2 + blockIdx.y) * cols + c];
    sum[ty][tx] = a;
    __syncthreads();
    if (ty == 0 && c < cols) {
        for (int g = 1; g < 32; ++g) a += sum[g][tx];
        out[c] = a;
    }
}

// Columns up to which a row stays in registers (two chunks of 8 per thread).
constexpr int MAX_COLS = 2 * 8 * LN_MAX_THREADS;

// Rows of at most 512 columns share a workgroup (8 to 64 threads each); longer
// ones take a workgroup of their own, with one chunk per thread up to `one`
// chunks and two above.  Measured at 16384 x 8192 bf16 forward: two chunks 95 us,
// one 113, four 101; at 16384 x 4096: 47, 50, 49.  Backward at 16381 x 4096 one
// chunk 87 us, two 87, four 97; at 8192 x 8192 two 90, one 96 (16381 x 4096 takes 80
// now, 76 of them this kernel: 5.3 TB/s of its 403 MB).
Shape shape_of(int64_t cols, int one) {
    const int chunks = int((cols + 7) / 8);
    if (chunks <= 64) {
        int W = 8;
        while (W < chunks) W *= 2;
        return {W, 1, 256};
    }
    const int R = chunks <= one ? 1 : 2;
    return {LN_MAX_THREADS, R, ((chunks + R - 1) / R + 63) / 64 * 64};
}
Shape fwd_shape(int64_t cols) { return shape_of(cols, 64); }
Shape bwd_shape(int64_t cols) { return shape_of(cols, 512); }

template <typename T, bool FULL>
hipError_t fwd(const MoLnArgs& a, hipStream_t s) {
    const T* X = static_cast<const T*>(a.X);
    T* Y = static_cast<T*>(a.Y);
    const int cols = int(a.cols);
    if (cols > MAX_COLS) {
        hipLaunchKernelGGL(ln_fwd_long_kernel<T>, dim3(unsigned(a.rows < 512 ? a.rows : 512)),
                           dim3(LN_MAX_THREADS), 0, s, X, a.ldx, a.weight, a.bias, Y, a.ldy, a.mean_out,
                           a.rstd_out, a.rows, cols, a.eps);
        return hipGetLastError();
    }
    const Shape sh = fwd_shape(cols);
    const dim3 grid(wgs_for(a.rows, sh, sh.W > 64 ? 2048 / sh.threads : 16)), block(sh.threads);
#define MO_LN_FWD(W, R)                                                                               \
    hipLaunchKernelGGL((ln_fwd_kernel<T, W, R, FULL>), grid, block, 0, s, X, a.ldx, a.weight, a.bias, Y,   \
                       a.ldy, a.mean_out, a.rstd_out, a.rows, cols, a.eps)
    if (sh.W == 8) MO_LN_FWD(8, 1);
    else if (sh.W == 16) MO_LN_FWD(16, 1);
    else if (sh.W == 32) MO_LN_FWD(32, 1);
    else if (sh.W == 64) MO_LN_FWD(64, 1);
    else MO_LN_FWD(LN_MAX_THREADS, 2);
#undef MO_LN_FWD
    return hipGetLastError();
}

template <typename T, bool FULL>
hipError_t bwd(const MoLnArgs& a, float* part, int n_part, hipStream_t s) {
    const T *X = static_cast<const T*>(a.X), *dY = static_cast<const T*>(a.dY);
    T* dX = static_cast<T*>(a.dX);
    const int cols = int(a.cols);
    float* pp = a.dweight || a.dbias ? part : nullptr;
    if (cols > MAX_COLS) {
        if (dX)
            hipLaunchKernelGGL(ln_bwd_long_kernel<T>, dim3(unsigned(a.rows < 512 ? a.rows : 512)),
                               dim3(LN_MAX_THREADS), 0, s, dY, a.lddy, X, a.ldx, a.weight, a.mean, a.rstd, dX,
                               a.lddx, a.rows, cols);
        if (pp)
            hipLaunchKernelGGL(ln_bwd_long_wb_kernel<T>, dim3(unsigned((cols + 2047) / 2048), unsigned(n_part)),
                               dim3(256), 0, s, dY, a.lddy, X, a.ldx, a.mean, a.rstd, pp, a.rows, cols);
        return hipGetLastError();
    }
    const Shape sh = bwd_shape(cols);
    const dim3 grid{unsigned(n_part)}, block(sh.threads);
#define MO_LN_BWD(W, R)                                                                               \
    hipLaunchKernelGGL((ln_bwd_kernel<T, W, R, FULL>), grid, block, 0, s, dY, a.lddy, X, a.ldx, a.weight,   \
                       a.mean, a.rstd, dX, a.lddx, pp, a.rows, cols)
    if (sh.W == 8) MO_LN_BWD(8, 1);
    else if (sh.W == 16) MO_LN_BWD(16, 1);
    else if (sh.W == 32) MO_LN_BWD(32, 1);
    else if (sh.W == 64) MO_LN_BWD(64, 1);
    else if (sh.R == 1) MO_LN_BWD(LN_MAX_THREADS, 1);
    else MO_LN_BWD(LN_MAX_THREADS, 2);
#undef MO_LN_BWD
    return hipGetLastError();
}

}  // namespace

int mo_ln_bwd_parts(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    if (cols > MAX_COLS) return int(rows < 64 ? rows : 64);
    // two workgroups per CU (one of more than 512 threads): each leaves a partial
    // row of 8 bytes per column; at 16381 x 4096, four per CU measured 106 us
    // against 87, one 124
    const Shape sh = bwd_shape(cols);
    return int(wgs_for(rows, sh, sh.W > 64 ? (sh.threads > 512 ? 1 : 2) : 4));
}

hipError_t mo_launch_ln_fwd(const MoLnArgs& a, hipStream_t s) {
    if (a.cols % 8 == 0) return a.dtype == MO_BF16 ? fwd<bf16_t, true>(a, s) : fwd<float, true>(a, s);
    return a.dtype == MO_BF16 ? fwd<bf16_t, false>(a, s) : fwd<float, false>(a, s);
}
hipError_t mo_launch_ln_bwd(const MoLnArgs& a, float* part, hipStream_t s) {
    const int n = mo_ln_bwd_parts(a.rows, a.cols);
    if (a.cols % 8 == 0) return a.dtype == MO_BF16 ? bwd<bf16_t, true>(a, part, n, s) : bwd<float, true>(a, part, n, s);
    return a.dtype == MO_BF16 ? bwd<bf16_t, false>(a, part, n, s) : bwd<float, false>(a, part, n, s);
}
hipError_t mo_launch_ln_reduce(const MoLnArgs& a, const float* part, hipStream_t s) {
    hipLaunchKernelGGL(ln_reduce_kernel, dim3(unsigned((a.cols + 31) / 32), 2), dim3(1024), 0, s, part,
                       mo_ln_bwd_parts(a.rows, a.cols), a.dweight, a.dbias, int(a.cols));
    return hipGetLastError();
}
