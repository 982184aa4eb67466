// Matrices to 8 bits and back (fp8.h): activations in blocks of 128 along their rows,
// weights in blocks of 128 x 128 in both layouts.  One read and one write of
// each element; bound by memory.
#include "fp8.h"
#include "operators.h"

#include <algorithm>

namespace {

// 16 threads per block of 128, 8 elements each.  A workgroup takes CG blocks side by side of 16 / CG
// rows; one after the other only where the grid ends.  16384 x 14336 bf16 to 8 bits: 124 us (5.7 TB/s); in
// 8192 workgroups that walk over rows, four rows' loads under way, 136.

template <typename T>
__global__ __launch_bounds__(256) void f8_quantize_kernel(const T* X, int64_t ldx, int64_t rows, int cols, uint8_t* Q,
                                                          int64_t ldq, uint8_t* S, int64_t lds, int cg) {
    const int g = threadIdx.x >> 4, t = threadIdx.x & 15, rg = 16 / cg;
    const int blk = int(blockIdx.x) * cg + g % cg, c = blk * F8_BLOCK + t * 8, n = cols - c;
    if (blk * F8_BLOCK >= cols) return;
    for (int64_t r = int64_t(blockIdx.y) * rg + g / cg; r < rows; r += int64_t(gridDim.y) * rg) {
        const f32x8 v = widen(ld8n(X + r * ldx + c, n));
        const uint32_t b = scale_byte(max16(amax8(v)));
        stq8(Q + r * ldq + c, to_e4m3(v, scale_inverse(b)), n);
        if (t == 0) S[r * lds + blk] = uint8_t(b);
    }
}

// bf16 is stored past the caches: 16381 x 4096 31 us instead of 39; with the reading of the result behind it
// 73.5 instead of 72.3, at 16384 x 14336 233 instead of 246.  fp32, whose lanes store every other 16 bytes at a
// time, is not: 61 us through the caches and 96 past them, at 16384 x 14336 201 and 354.
template <typename T>
__global__ __launch_bounds__(256) void f8_dequantize_kernel(const uint8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds,
                                                            int64_t rows, int cols, T* X, int64_t ldx, int cg) {
    const int g = threadIdx.x >> 4, t = threadIdx.x & 15, rg = 16 / cg;
    const int blk = int(blockIdx.x) * cg + g % cg, c = blk * F8_BLOCK + t * 8, n = cols - c;
    if (c >= cols) return;
    for (int64_t r = int64_t(blockIdx.y) * rg + g / cg; r < rows; r += int64_t(gridDim.y) * rg) {
        const f32x8 v = from_e4m3(ldq8(Q + r * ldq + c, n), scale_value(S[r * lds + blk]));
        T* x = X + r * ldx + c;
        if (n < 8) {
            st8n(x, v, n);
        } else if constexpr (sizeof(T) == 2) {
            __builtin_nontemporal_store(narrow(v, T()).q, reinterpret_cast<u32x4_e2*>(x));
        } else {
            st8(x, v);
        }
    }
}

// One 128 x 128 block of a weight per workgroup and turn: thread t holds columns 8 (t % 16)
// .. and rows 8 (t / 16) .., so that the transposed copy goes through LDS in pieces
// of 8 bytes (one column, eight rows).  14336 x 4096 bf16 with both copies: 41 to 43 us, 5.5 TB/s.
constexpr int TSTRIDE = 136;   // bytes of LDS per column of the block

template <typename T>
__global__ __launch_bounds__(256) void f8_weight_kernel(const T* W, int64_t ldw, int64_t rows, int64_t cols, uint8_t* Q,
                                                        int64_t ldq, uint8_t* S, int64_t lds, uint8_t* Qt,
                                                        int64_t ldqt, uint8_t* St, int64_t ldst, uint32_t bc,
                                                        uint32_t blocks) {
    __shared__ __align__(16) uint8_t tile[F8_BLOCK * TSTRIDE];
    __shared__ uint32_t red[2][4];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    int turn = 0;
    for (uint32_t b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const uint32_t bi = b / bc, bj = b - bi * bc;
        const int64_t r0 = int64_t(bi) * F8_BLOCK + y * 8, c0 = int64_t(bj) * F8_BLOCK + x * 8;
        const int n = int(cols - c0 < 8 ? cols - c0 : 8), m = int(rows - r0 < 8 ? rows - r0 : 8);
        raw8<T> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ld8n(W + (r0 + (i < m ? i : 0)) * ldw + c0, i < m ? n : 0);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = amax8(widen(v[i]));
            top = a > top ? a : top;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint32_t o = uint32_t(__shfl_xor(int(top), off, 64));
            top = o > top ? o : top;
        }
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = top;
        __syncthreads();   // the tile of the turn before has been read as well
#pragma unroll
        for (int i = 0; i < 4; ++i) top = red[turn][i] > top ? red[turn][i] : top;
        const uint32_t sb = scale_byte(top);
        const float inv = scale_inverse(sb);
        u32x2 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[i] = to_e4m3(widen(v[i]), inv);
            if (Q && i < m) stq8(Q + (r0 + i) * ldq + c0, q[i], n);
        }
        if (threadIdx.x == 0) {
            if (Q) S[int64_t(bi) * lds + bj] = uint8_t(sb);
            if (Qt) St[int64_t(bj) * ldst + bi] = uint8_t(sb);
        }
        if (!Qt) continue;
        // column 8 x + e of rows 8 y ..: 8 bytes at piece y + 4 (x / 4) mod 16, which spreads the
        // 16 columns that a wave writes together over the banks
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            u32x2 p = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i / 4] |= ((q[i][e / 4] >> (8 * (e % 4))) & 255u) << (8 * (i % 4));
            *reinterpret_cast<u32x2*>(tile + (x * 8 + e) * TSTRIDE + ((y + (x >> 2) * 4) & 15) * 8) = p;
        }
        __syncthreads();
        const int64_t left = rows - int64_t(bi) * F8_BLOCK;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = i * 16 + y;   // column of the block; x: its piece
            const int64_t col = int64_t(bj) * F8_BLOCK + c;
            const int k = int(left - x * 8 < 8 ? left - x * 8 : 8);
            const u32x2 p = *reinterpret_cast<const u32x2*>(tile + c * TSTRIDE + ((x + (c >> 5) * 4) & 15) * 8);
            if (col < cols) stq8(Qt + col * ldqt + int64_t(bi) * F8_BLOCK + x * 8, p, k);
        }
    }
}

// Blocks side by side per workgroup, and its grid.
struct CastGrid {
    int cg;
    dim3 grid;
    CastGrid(int64_t rows, int64_t cols) {
        const int64_t kb = (cols + F8_BLOCK - 1) / F8_BLOCK;
        cg = 1;
        while (cg < 16 && cg < kb) cg *= 2;
        const int64_t gx = (kb + cg - 1) / cg, rg = 16 / cg, want = (rows + rg - 1) / rg;
        const int64_t most = int64_t(1) << 22, cap = gx >= most ? 1 : most / gx;
        grid = dim3(unsigned(gx), unsigned(std::min({want, cap, int64_t(65535)})));
    }
};

}  // namespace

hipError_t mo_launch_f8_quantize(const MoF8Cast& a, hipStream_t s) {
    const CastGrid g(a.rows, a.cols);
    if (a.dtype == MO_BF16)
        hipLaunchKernelGGL(f8_quantize_kernel<bf16_t>, g.grid, dim3(256), 0, s, static_cast<const bf16_t*>(a.X), a.ldx,
                           a.rows, int(a.cols), a.Q, a.ldq, a.S, a.lds, g.cg);
    else
        hipLaunchKernelGGL(f8_quantize_kernel<float>, g.grid, dim3(256), 0, s, static_cast<const float*>(a.X), a.ldx,
                           a.rows, int(a.cols), a.Q, a.ldq, a.S, a.lds, g.cg);
    return hipGetLastError();
}

hipError_t mo_launch_f8_dequantize(const MoF8Cast& a, hipStream_t s) {
    const CastGrid g(a.rows, a.cols);
    if (a.dtype == MO_BF16)
        hipLaunchKernelGGL(f8_dequantize_kernel<bf16_t>, g.grid, dim3(256), 0, s, a.Q, a.ldq, a.S, a.lds, a.rows,
                           int(a.cols), static_cast<bf16_t*>(a.out), a.ldx, g.cg);
    else
        hipLaunchKernelGGL(f8_dequantize_kernel<float>, g.grid, dim3(256), 0, s, a.Q, a.ldq, a.S, a.lds, a.rows,
                           int(a.cols), static_cast<float*>(a.out), a.ldx, g.cg);
    return hipGetLastError();
}

hipError_t mo_launch_f8_weight(const MoF8Cast& a, hipStream_t s) {
    const int64_t bc = (a.cols + F8_BLOCK - 1) / F8_BLOCK, blocks = bc * ((a.rows + F8_BLOCK - 1) / F8_BLOCK);
    const dim3 grid(unsigned(blocks < 4096 ? blocks : 4096));
#define MO_F8_WEIGHT(T)                                                                                          \
    hipLaunchKernelGGL(f8_weight_kernel<T>, grid, dim3(256), 0, s, static_cast<const T*>(a.X), a.ldx, a.rows, a.cols, \
                       a.Q, a.ldq, a.S, a.lds, a.Qt, a.ldqt, a.St, a.ldst, uint32_t(bc), uint32_t(blocks))
    if (a.dtype == MO_BF16) MO_F8_WEIGHT(bf16_t);
    else MO_F8_WEIGHT(float);
#undef MO_F8_WEIGHT
    return hipGetLastError();
}
