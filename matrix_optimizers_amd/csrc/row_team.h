// Shared by the norms: one row per team of threads, its elements in their registers
// in chunks of 8, and the sums over it.
#pragma once

#include "op_common.h"

constexpr int TEAM_MAX_THREADS = 1024;

// Sum over the team of threads that hold one row.  Rows in at most 64 threads
// are summed within a wavefront (width W); wider ones take the waves' sums
// through LDS in wave order.  `red` has two slots of 16 x N floats, used in
// turn, so one barrier per reduction is enough.
template <int W, int N>
MO_DEV void team_sum(float (&x)[N], float* red, int& turn) {
#pragma unroll
    for (int off = (W < 64 ? W : 64) / 2; off >= 1; off >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] += __shfl_xor(x[n], off, 64);
    if constexpr (W > 64) {
        float* slot = red + turn * 16 * N;
        turn ^= 1;
        const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) slot[wave * N + n] = x[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = 0.f;
        for (int w = 0; w < waves; ++w)
#pragma unroll
            for (int n = 0; n < N; ++n) x[n] += slot[w * N + n];
    }
}

// A row's team (W threads of a workgroup of `threads`, or all of them: W above 64) and
// its chunks per thread.
struct Shape { int W, R, threads; };

// Workgroups for `rows`, at most per_cu on each of 256 CUs.
inline unsigned wgs_for(int64_t rows, const Shape& s, int per_cu) {
    const int64_t per = s.W > 64 ? 1 : 256 / s.W;
    const int64_t want = (rows + per - 1) / per, cap = 256 * int64_t(per_cu);
    return unsigned(want < cap ? want : cap);
}
