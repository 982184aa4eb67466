// Root-mean-square norm over the rows of a matrix, with the residual's addition, and its
// gradients.
//
//   h = x + residual (rounded to the type: what is stored is what is normed)
//   r = (mean(h^2) + eps)^-1/2, y = h r w; y in the type or in 8 bits (fp8.h)
//   g = dy w, xh = h r
//   dx = r (g - xh mean(g xh)) + dh,  dw = sum_rows dy xh
//
// Every element is read once and written once, as in the layer norm: a row lives in
// its threads' registers between the sum and the result.  Sums are fp32.  The 8-bit
// result costs one maximum over 16 lanes more, which hold a block of 128.
#include "fp8.h"
#include "operators.h"
#include "row_team.h"

namespace {

// The row's team and chunks as in the layer norm: thread t holds the 8-element chunks
// t, t + team, .. (R of them), so 16 threads hold a block of 128.  The next row is
// requested before this one's reduction.
template <typename T, int W, int R, bool FULL, bool RES>
__global__ __launch_bounds__(W > 64 ? TEAM_MAX_THREADS : 256) void rms_fwd_kernel(MoRmsArgs a) {
    __shared__ float red[32];
    const T *X = static_cast<const T*>(a.X), *D = static_cast<const T*>(a.residual);
    T *Y = static_cast<T*>(a.Y), *H = static_cast<T*>(a.H_out);
    const int cols = int(a.cols);
    const int team = W > 64 ? blockDim.x : W, teams = W > 64 ? 1 : 256 / W;
    const int t = W > 64 ? threadIdx.x : threadIdx.x % W;
    const int sub = W > 64 ? 0 : threadIdx.x / W;
    const int64_t step = int64_t(gridDim.x) * teams;
    int turn = 0;
    raw8<T> nx[R], nd[R];
    auto request = [&](int64_t row) __attribute__((always_inline)) {
        row = row < a.rows ? row : a.rows - 1;
#pragma unroll
        for (int i = 0; i < R; ++i) nx[i] = row8<FULL>(X + row * a.ldx, (t + team * i) * 8, cols);
        if constexpr (RES)
#pragma unroll
            for (int i = 0; i < R; ++i) nd[i] = row8<FULL>(D + row * a.ldr, (t + team * i) * 8, cols);
    };
    request(int64_t(blockIdx.x) * teams + sub);
    f32x8 w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (a.weight) w[i] = widen(row8<FULL>(a.weight, (t + team * i) * 8, cols));
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i].v[e] = 1.f;
    }
    const float n_cols = float(cols);
    for (int64_t base = int64_t(blockIdx.x) * teams; base < a.rows; base += step) {
        const int64_t row = base + sub;
        const bool live = row < a.rows;
        f32x8 h[R];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            h[i] = widen(nx[i]);
            if constexpr (RES) {
                const f32x8 d = widen(nd[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i].v[e] = quantize<T>(h[i].v[e] + d.v[e]);
                if (H && live) row8_out<FULL>(H + row * a.ldh_out, (t + team * i) * 8, cols, h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += h[i].v[e] * h[i].v[e];
        }
        if (base + step < a.rows) request(row + step);
        team_sum<W>(s, red, turn);
        const float r = 1.0f / sqrtf(s[0] / n_cols + a.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (t + team * i) * 8;
            f32x8 y;
#pragma unroll
            for (int e = 0; e < 8; ++e) y.v[e] = h[i].v[e] * r * w[i].v[e];
            if (Y) row8_out<FULL>(Y + row * a.ldy, c, cols, y);
            if (a.Q) {
                const uint32_t b = scale_byte(max16(amax8(y)));
                if (c < cols) stq8(a.Q + row * a.ldq + c, to_e4m3(y, scale_inverse(b)), FULL ? 8 : cols - c);
                if ((t & 15) == 0 && c < cols) a.S[row * a.lds + c / F8_BLOCK] = uint8_t(b);
            }
        }
        if (t == 0 && a.rstd_out) a.rstd_out[row] = r;
    }
}

// Rows too long for registers: one workgroup per row, read again for the result.
template <typename T>
__global__ __launch_bounds__(TEAM_MAX_THREADS) void rms_fwd_long_kernel(MoRmsArgs a) {
    __shared__ float red[32];
    const int cols = int(a.cols);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T*>(a.X) + row * a.ldx;
        const T *d = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
        auto sum8 = [&](int c) __attribute__((always_inline)) {
            f32x8 h = widen(ld8n(x + c, cols - c));
            if (d) {
                const f32x8 v = widen(ld8n(d + c, cols - c));
#pragma unroll
                for (int e = 0; e < 8; ++e) h.v[e] = quantize<T>(h.v[e] + v.v[e]);
            }
            return h;
        };
        float s[1] = {0.f};
        for (int c = threadIdx.x * 8; c < cols; c += TEAM_MAX_THREADS * 8) {
            const f32x8 h = sum8(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += h.v[e] * h.v[e];
        }
        team_sum<TEAM_MAX_THREADS>(s, red, turn);
        const float r = 1.0f / sqrtf(s[0] / float(cols) + a.eps);
        // whole blocks of 16 threads stay together up to the row's last block
        for (int c0 = (threadIdx.x & ~15) * 8; c0 < cols; c0 += TEAM_MAX_THREADS * 8) {
            const int c = c0 + (threadIdx.x & 15) * 8, n = cols - c;
            const f32x8 h = sum8(n > 0 ? c : 0);
            f32x8 y;
#pragma unroll
            for (int e = 0; e < 8; ++e) y.v[e] = e < n ? h.v[e] * r * (a.weight ? a.weight[c + e] : 1.f) : 0.f;
            if (d && a.H_out) st8n(static_cast<T*>(a.H_out) + row * a.ldh_out + c, h, n);
            if (a.Y) st8n(static_cast<T*>(a.Y) + row * a.ldy + c, y, n);
            if (a.Q) {
                const uint32_t b = scale_byte(max16(amax8(y)));
                stq8(a.Q + row * a.ldq + c, to_e4m3(y, scale_inverse(b)), n);
                if (c == c0) a.S[row * a.lds + c / F8_BLOCK] = uint8_t(b);
            }
        }
        if (threadIdx.x == 0 && a.rstd_out) a.rstd_out[row] = r;
    }
}

// dx, and this workgroup's share of dw: a thread's columns stay the same over the
// rows it walks, so the sum lives in its registers and leaves one fp32 row per workgroup.
template <typename T, int W, int R, bool FULL>
__global__ __launch_bounds__(W > 64 ? TEAM_MAX_THREADS : 256) void rms_bwd_kernel(MoRmsArgs a, float* part) {
    __shared__ float red[32];
    __shared__ float comb[W > 64 ? 1 : 256 * 8];
    const T *H = static_cast<const T*>(a.H), *dY = static_cast<const T*>(a.dY), *dH = static_cast<const T*>(a.dH);
    T* dX = static_cast<T*>(a.dX);
    const int cols = int(a.cols);
    const int team = W > 64 ? blockDim.x : W, teams = W > 64 ? 1 : 256 / W;
    const int t = W > 64 ? threadIdx.x : threadIdx.x % W;
    const int sub = W > 64 ? 0 : threadIdx.x / W;
    const int64_t step = int64_t(gridDim.x) * teams;
    int turn = 0;
    f32x8 dw[R], w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) { dw[i].v[e] = 0.f; w[i].v[e] = 1.f; }
        if (a.weight) w[i] = widen(row8<FULL>(a.weight, (t + team * i) * 8, cols));
    }
    const float n_cols = float(cols);
    raw8<T> nh[R], ny[R], nd[R];
    float nr;
    auto request = [&](int64_t row) __attribute__((always_inline)) {
        row = row < a.rows ? row : a.rows - 1;
        nr = a.rstd[row];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            nh[i] = row8<FULL>(H + row * a.ldh, (t + team * i) * 8, cols);
            ny[i] = row8<FULL>(dY + row * a.lddy, (t + team * i) * 8, cols);
        }
        if (dX && dH)
#pragma unroll
            for (int i = 0; i < R; ++i) nd[i] = row8<FULL>(dH + row * a.lddh, (t + team * i) * 8, cols);
    };
    // The next row is requested before this one's reduction, except with two chunks of fp32, where 48 to 94 registers
    // were spilled for it (us at 16384 rows of 4100, 8192 and 16384 columns with dH: 204, 395 and 776; ahead 408, 834
    // and 1207).
    constexpr bool AHEAD = sizeof(T) == 2 || R == 1;
    if (AHEAD) request(int64_t(blockIdx.x) * teams + sub);
    for (int64_t base = int64_t(blockIdx.x) * teams; base < a.rows; base += step) {
        const int64_t row = base + sub;
        const bool live = row < a.rows;
        if (!AHEAD) request(row);
        const float r = nr;
        raw8<T> h[R], dy[R], dh[R];
#pragma unroll
        for (int i = 0; i < R; ++i) { h[i] = nh[i]; dy[i] = ny[i]; dh[i] = nd[i]; }
        if (AHEAD && base + step < a.rows) request(row + step);
        float s[1] = {0.f};
        if (live) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const f32x8 hv = widen(h[i]), gv = widen(dy[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = hv.v[e] * r, p = gv.v[e] * xh;
                    s[0] += p * w[i].v[e];
                    dw[i].v[e] += p;
                }
            }
        }
        if (dX) {
            team_sum<W>(s, red, turn);
            const float m = s[0] / n_cols;
            if (live) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const f32x8 hv = widen(h[i]), gv = widen(dy[i]);
                    f32x8 o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o.v[e] = r * (gv.v[e] * w[i].v[e] - hv.v[e] * r * m);
                    if (dH) {
                        const f32x8 dv = widen(dh[i]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o.v[e] += dv.v[e];
                    }
                    row8_out<FULL>(dX + row * a.lddx, (t + team * i) * 8, cols, o);
                }
            }
        }
    }
    if (!part) return;
    float* p = part + int64_t(blockIdx.x) * cols;
    if constexpr (W > 64) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (t + team * i) * 8;
            st8n(p + c, dw[i], cols - c);
        }
    } else {
        // R == 1: the workgroup's rows in row order
#pragma unroll
        for (int e = 0; e < 8; ++e) comb[threadIdx.x * 8 + e] = dw[0].v[e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += 256) {
            float x = 0.f;
            for (int u = 0; u < teams; ++u) x += comb[u * W * 8 + c];
            p[c] = x;
        }
    }
}

// Long rows, first the sum and dx, one workgroup per row ..
template <typename T>
__global__ __launch_bounds__(TEAM_MAX_THREADS) void rms_bwd_long_kernel(MoRmsArgs a) {
    __shared__ float red[32];
    const int cols = int(a.cols);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float r = a.rstd[row];
        const T *h = static_cast<const T*>(a.H) + row * a.ldh, *dy = static_cast<const T*>(a.dY) + row * a.lddy;
        const T* dh = a.dH ? static_cast<const T*>(a.dH) + row * a.lddh : nullptr;
        float s[1] = {0.f};
        for (int c = threadIdx.x * 8; c < cols; c += TEAM_MAX_THREADS * 8) {
            const f32x8 hv = widen(ld8n(h + c, cols - c)), gv = widen(ld8n(dy + c, cols - c));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) s[0] += gv.v[e] * (a.weight ? a.weight[c + e] : 1.f) * (hv.v[e] * r);
        }
        team_sum<TEAM_MAX_THREADS>(s, red, turn);
        const float m = s[0] / float(cols);
        for (int c = threadIdx.x * 8; c < cols; c += TEAM_MAX_THREADS * 8) {
            const int n = cols - c;
            const f32x8 hv = widen(ld8n(h + c, n)), gv = widen(ld8n(dy + c, n));
            f32x8 o, dv = {};
            if (dh) dv = widen(ld8n(dh + c, n));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o.v[e] = e < n ? r * (gv.v[e] * (a.weight ? a.weight[c + e] : 1.f) - hv.v[e] * r * m) + dv.v[e] : 0.f;
            st8n(static_cast<T*>(a.dX) + row * a.lddx + c, o, n);
        }
    }
}
// .. then partial dw of a strided share of the rows (blockIdx.y) for 2048 columns (blockIdx.x).
template <typename T>
__global__ __launch_bounds__(256) void rms_bwd_long_w_kernel(MoRmsArgs a, float* part) {
    const int cols = int(a.cols), c = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= cols) return;
    f32x8 dw = {};
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float r = a.rstd[row];
        const f32x8 hv = widen(ld8n(static_cast<const T*>(a.H) + row * a.ldh + c, cols - c));
        const f32x8 gv = widen(ld8n(static_cast<const T*>(a.dY) + row * a.lddy + c, cols - c));
#pragma unroll
        for (int e = 0; e < 8; ++e) dw.v[e] += gv.v[e] * (hv.v[e] * r);
    }
    st8n(part + int64_t(blockIdx.y) * cols + c, dw, cols - c);
}

// dw: the partial rows of each column in a fixed order, 32 columns by 32 strided shares
// per workgroup.
__global__ __launch_bounds__(1024) void rms_reduce_kernel(const float* part, int n_part, float* dweight, int cols) {
    __shared__ float sum[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    float x = 0.f;
    if (c < cols)
        for (int g = ty; g < n_part; g += 32) x += part[int64_t(g) * cols + c];
    sum[ty][tx] = x;
    __syncthreads();
    if (ty == 0 && c < cols) {
        for (int g = 1; g < 32; ++g) x += sum[g][tx];
        dweight[c] = x;
    }
}

// Columns up to which a row stays in registers (two chunks of 8 per thread).
constexpr int MAX_COLS = 2 * 8 * TEAM_MAX_THREADS;

// Rows of at most 512 columns share a workgroup (16 to 64 threads each: a block of 128 is
// 16 threads); longer ones take a workgroup of their own, with one chunk per thread up to
// 4096 columns and two above.
Shape shape_of(int64_t cols) {
    const int chunks = int((cols + 7) / 8);
    if (chunks <= 64) {
        int W = 16;
        while (W < chunks) W *= 2;
        return {W, 1, 256};
    }
    const int R = chunks <= 512 ? 1 : 2;
    return {TEAM_MAX_THREADS, R, ((chunks + R - 1) / R + 63) / 64 * 64};
}

// Forward, up to 8192 columns each row has a workgroup of its own (bf16 to 8 bits with a residual,
// 16384 x 8192 168 us, 5.6 TB/s; with as many workgroups as fit, walking over rows, 178; 16384 x 4096
// 83 and 92), wider ones walk (9362 x 14336 184 us, 208 with one row each).
unsigned fwd_wgs(int64_t rows, const Shape& sh) {
    return wgs_for(rows, sh, sh.W <= 64 ? 16 : sh.threads <= 512 ? 1 << 12 : 2048 / sh.threads);
}
// Backward, each workgroup leaves a partial row of 4 bytes per column: as few per CU as keep the loads
// going.  bf16, us at 16384 rows of 1024, 2048, 4096 and 8192 columns with dH: 41.6, 57.8, 105 and 198.5 (4.6 to 5.4
// TB/s), with half as many workgroups per CU 43 (three), 64.7, 117, -, with twice as many 69, 73, 120, 210.  Rows of two
// chunks leave a CU with five to seven wavefronts where they are short of 8192 columns: two of them in bf16
// (4104, 5000 and 7168 columns 111, 131 and 186, one alone 142, 160 and 189), one in fp32, which has twice the bytes
// under way (209, 257 and 363; 201, 244 and 337).
int bwd_per_cu(const Shape& sh, bool bf16) {
    if (sh.W <= 64) return 2;
    return sh.threads <= 128 ? 4 : sh.threads <= 256 ? 3 : sh.threads <= (sh.R == 1 ? 512 : bf16 ? 448 : 0) ? 2 : 1;
}

template <typename T, bool FULL, bool RES>
hipError_t fwd(const MoRmsArgs& a, hipStream_t s) {
    if (a.cols > MAX_COLS) {
        hipLaunchKernelGGL(rms_fwd_long_kernel<T>, dim3(unsigned(a.rows < 512 ? a.rows : 512)), dim3(TEAM_MAX_THREADS),
                           0, s, a);
        return hipGetLastError();
    }
    const Shape sh = shape_of(a.cols);
    const dim3 grid(fwd_wgs(a.rows, sh)), block(sh.threads);
#define MO_RMS_FWD(W, R) hipLaunchKernelGGL((rms_fwd_kernel<T, W, R, FULL, RES>), grid, block, 0, s, a)
    if (sh.W == 16) MO_RMS_FWD(16, 1);
    else if (sh.W == 32) MO_RMS_FWD(32, 1);
    else if (sh.W == 64) MO_RMS_FWD(64, 1);
    else if (sh.R == 1) MO_RMS_FWD(TEAM_MAX_THREADS, 1);
    else MO_RMS_FWD(TEAM_MAX_THREADS, 2);
#undef MO_RMS_FWD
    return hipGetLastError();
}

template <typename T, bool FULL>
hipError_t bwd(const MoRmsArgs& a, float* part, int n_part, hipStream_t s) {
    float* pp = a.dweight ? part : nullptr;
    if (a.cols > MAX_COLS) {
        if (a.dX)
            hipLaunchKernelGGL(rms_bwd_long_kernel<T>, dim3(unsigned(a.rows < 512 ? a.rows : 512)),
                               dim3(TEAM_MAX_THREADS), 0, s, a);
        if (pp)
            hipLaunchKernelGGL(rms_bwd_long_w_kernel<T>, dim3(unsigned((a.cols + 2047) / 2048), unsigned(n_part)),
                               dim3(256), 0, s, a, pp);
        return hipGetLastError();
    }
    const Shape sh = shape_of(a.cols);
    const dim3 grid{unsigned(n_part)}, block(sh.threads);
#define MO_RMS_BWD(W, R) hipLaunchKernelGGL((rms_bwd_kernel<T, W, R, FULL>), grid, block, 0, s, a, pp)
    if (sh.W == 16) MO_RMS_BWD(16, 1);
    else if (sh.W == 32) MO_RMS_BWD(32, 1);
    else if (sh.W == 64) MO_RMS_BWD(64, 1);
    else if (sh.R == 1) MO_RMS_BWD(TEAM_MAX_THREADS, 1);
    else MO_RMS_BWD(TEAM_MAX_THREADS, 2);
#undef MO_RMS_BWD
    return hipGetLastError();
}

}  // namespace

int mo_rms_bwd_parts(int64_t rows, int64_t cols, int32_t dtype) {
    if (rows == 0) return 0;
    if (cols > MAX_COLS) return int(rows < 64 ? rows : 64);
    const Shape sh = shape_of(cols);
    return int(wgs_for(rows, sh, bwd_per_cu(sh, dtype == MO_BF16)));
}

hipError_t mo_launch_rms_fwd(const MoRmsArgs& a, hipStream_t s) {
#define MO_RMS_T(T, F) (a.residual ? fwd<T, F, true>(a, s) : fwd<T, F, false>(a, s))
    if (a.cols % 8 == 0) return a.dtype == MO_BF16 ? MO_RMS_T(bf16_t, true) : MO_RMS_T(float, true);
    return a.dtype == MO_BF16 ? MO_RMS_T(bf16_t, false) : MO_RMS_T(float, false);
#undef MO_RMS_T
}
hipError_t mo_launch_rms_bwd(const MoRmsArgs& a, float* part, hipStream_t s) {
    const int n = mo_rms_bwd_parts(a.rows, a.cols, a.dtype);
    if (a.cols % 8 == 0) return a.dtype == MO_BF16 ? bwd<bf16_t, true>(a, part, n, s) : bwd<float, true>(a, part, n, s);
    return a.dtype == MO_BF16 ? bwd<bf16_t, false>(a, part, n, s) : bwd<float, false>(a, part, n, s);
}
hipError_t mo_launch_rms_reduce(const MoRmsArgs& a, const float* part, hipStream_t s) {
    hipLaunchKernelGGL(rms_reduce_kernel, dim3(unsigned((a.cols + 31) / 32)), dim3(1024), 0, s, part,
                       mo_rms_bwd_parts(a.rows, a.cols, a.dtype), a.dweight, int(a.cols));
    return hipGetLastError();
}
