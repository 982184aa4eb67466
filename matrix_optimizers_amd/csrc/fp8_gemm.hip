// Products with matrices in 8 bits:
//   Y = A B^T, both in 8 bits (bf16 results: fp8_gemm.h; fp32 results: the operands' values,
//       which are bf16 numbers, through the bf16 GEMM), and
//   G = dY^T X, X an activation kept in 8 bits, dY as it is: X's values are bf16 numbers, an
//       fp32 dY is three of them.
// P, the operand with tiles of 256 rows, is the one along the result's columns: a lane's
// four accumulators are then four neighbours of a row.
#include "fp8_gemm.h"
#include "operators.h"

namespace {

using namespace mo_f8;

constexpr int XT = 64;   // rows and columns of a transposing tile

// ---- the products ---------------------------------------------------------------------

// Where the results go: dst[q][p], element strides ld and 1.
template <typename T> struct Out {
    T* dst;
    int64_t ld, cols, rows;   // cols: along P, rows: along Q
    bool add;
};

// N neighbours of a row at d, n of them there.
template <int N, typename T> MO_DEV void put(T* d, const float (&v)[N], int n, bool add) {
    typedef T vec __attribute__((ext_vector_type(N)));
    typedef vec vec_e __attribute__((aligned(sizeof(T))));
    if (n >= N) {
        vec w;
        if (add) {
            const vec old = *reinterpret_cast<const vec_e*>(d);
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = from_f32<T>(v[e] + to_f32(T(old[e])));
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = from_f32<T>(v[e]);
        }
        *reinterpret_cast<vec_e*>(d) = w;
    } else {
#pragma unroll
        for (int e = 0; e < N - 1; ++e)
            if (e < n) d[e] = from_f32<T>(add ? v[e] + to_f32(d[e]) : v[e]);
    }
}
// Four neighbours of row q from column p on.
template <typename T> MO_DEV void put4(const Out<T>& o, int64_t q, int64_t p, f32x4 v) {
    const int64_t n = o.cols - p;
    if (q >= o.rows || n <= 0) return;
    const float x[4] = {v[0], v[1], v[2], v[3]};
    put<4>(o.dst + q * o.ld + p, x, int(n < 4 ? n : 4), o.add);
}
// A column block's results of two row blocks.  A lane has four neighbours of a row in each; the
// odd rows of 16 lanes change their first block's against their neighbours' second one, so that
// each lane stores eight neighbours (16 bytes of bf16, 64 in a line by four lanes).
MO_DEV void put8(const Out<bf16_t>& o, int64_t q, int64_t p, int kg, f32x4 v0, f32x4 v1) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#ifdef __HIP_DEVICE_COMPILE__
        const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v0[e]), __float_as_uint(v1[e]), false, false);
        x[e] = __uint_as_float(w[0]);
        x[4 + e] = __uint_as_float(w[1]);
#endif
    }
    p += (kg & 1) * 16 + (kg >> 1) * 8;
    const int64_t n = o.cols - p;
    if (q >= o.rows || n <= 0) return;
    put<8>(o.dst + q * o.ld + p, x, int(n < 8 ? n : 8), o.add);
}

template <int KIND, int NB, typename T>
__global__ __launch_bounds__(H_THREADS) __attribute__((amdgpu_waves_per_eu(2))) void f8_product_kernel(Operand8 P,
                                                                                                       Operand8 Q, Tiles t,
                                                                                                       Out<T> o) {
    using L = Layout<NB>;
    __shared__ __align__(16) uint8_t smem[gemm_lds<KIND>(NB)];
    auto store = [&](const Item& it, int wave, int lane, const f32x4 (&acc)[L::MB][L::NBW]) __attribute__((always_inline)) {
        if (it.split) {
            f32x4* z = t.part + (int64_t(it.slot) * 8 + wave) * (L::MB * L::NBW * 64) + lane;
#pragma unroll
            for (int i = 0; i < L::MB * L::NBW; ++i) z[i * 64] = acc[i / L::NBW][i % L::NBW];
            return true;
        }
        const int kg = lane >> 4;
        const int64_t p = int64_t(it.ti) * 256 + wave / L::WN * (L::MB * 16);
        const int64_t q = int64_t(it.tj) * 64 * NB + wave % L::WN * 64 + (lane & 15);
#pragma unroll
        for (int b = 0; b < L::NBW; ++b)
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int a = 0; a < L::MB; a += 2) put8(o, q + b * 16, p + a * 16, kg, acc[a][b], acc[a + 1][b]);
            } else {
#pragma unroll
                for (int a = 0; a < L::MB; ++a) put4(o, q + b * 16, p + a * 16 + kg * 4, acc[a][b]);
            }
        // (a wave whose rows or columns are not all there may have skipped some)
        return int64_t(it.ti) * 256 + 256 <= o.cols && int64_t(it.tj) * 64 * NB + 64 * NB <= o.rows;
    };
    run_tiles<NB, KIND>(smem, P, Q, t, store);
}

// The parts' sums in order: one wavefront per 16 x 64 of a wave's block.
template <int NB, typename T>
__global__ __launch_bounds__(256) void f8_sum_kernel(Tiles t, Out<T> o) {
    using L = Layout<NB>;
    const uint32_t unit = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t a = unit % L::MB, wave = unit / L::MB % 8, slot = unit / (L::MB * 8);
    if (slot >= t.rem) return;
    const int64_t stride = 8 * (L::MB * L::NBW * 64);
    const f32x4* z = t.part + int64_t(slot) * t.splits * stride + int64_t(wave) * (L::MB * L::NBW * 64) + a * (L::NBW * 64) + lane;
    f32x4 s[L::NBW];
#pragma unroll
    for (int b = 0; b < L::NBW; ++b) s[b] = z[b * 64];
#pragma unroll 4
    for (uint32_t k = 1; k < t.splits; ++k)
#pragma unroll
        for (int b = 0; b < L::NBW; ++b) {
            const f32x4 x = z[k * stride + b * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][e] += x[e];
        }
    uint32_t ti, tj;
    tile_at(t, t.full + slot, &ti, &tj);
    const int64_t p = int64_t(ti) * 256 + wave / L::WN * (L::MB * 16) + a * 16 + (lane >> 4) * 4;
    const int64_t q = int64_t(tj) * 64 * NB + wave % L::WN * 64 + (lane & 15);
#pragma unroll
    for (int b = 0; b < L::NBW; ++b) put4(o, q + b * 16, p, s[b]);
}

// ---- operands laid out for them ------------------------------------------------------

// q with rows of kd bytes (a multiple of 128, zeros behind dim), and its scales with rows of
// ks bytes (a multiple of 4, 127 behind the last block).
__global__ __launch_bounds__(256) void f8_copy_kernel(const uint8_t* q, int64_t ld, int64_t rows, int dim, uint8_t* dst,
                                                      int kd) {
    const int64_t chunks = int64_t(kd / 8) * rows;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / (kd / 8);
        const int c = int(i - r * (kd / 8)) * 8;
        *reinterpret_cast<u32x2*>(dst + r * kd + c) = ldq8(q + r * ld + c, dim - c);
    }
}
__global__ __launch_bounds__(256) void f8_copy_scales_kernel(const uint8_t* s, int64_t ld, int64_t inc, int64_t rows, int kb,
                                                             uint32_t* dst, int words) {
    const int64_t n = int64_t(words) * rows;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / words;
        const int c = int(i - r * words) * 4;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= uint32_t(c + e < kb ? s[r * ld + (c + e) * inc] : 127) << (8 * e);
        dst[i] = w;
    }
}

// The values of q in bf16, rows of kd elements (a multiple of 64, zeros behind dim).
__global__ __launch_bounds__(256) void f8_unpack_kernel(const uint8_t* q, int64_t ld, const uint8_t* s, int64_t ld_s,
                                                        int64_t inc, int shift, int64_t rows, int dim, bf16_t* dst, int kd) {
    const int64_t chunks = int64_t(kd / 8) * rows;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / (kd / 8);
        const int c = int(i - r * (kd / 8)) * 8;
        const float f = c < dim ? scale_value(s[(r >> shift) * ld_s + c / F8_BLOCK * inc]) : 0.f;
        store8(dst + r * kd + c, from_e4m3(ldq8(q + r * ld + c, dim - c), f));
    }
}

// Eight values of a row to transpose: of a matrix, or of one in 8 bits.
template <typename T> struct Source {
    const T* p;
    int64_t ld;
    MO_DEV f32x8 at(int64_t r, int64_t c, int n) const { return widen(ld8n(p + r * ld + c, n)); }
};
template <> struct Source<uint8_t> {
    const uint8_t* p;
    int64_t ld;
    const uint8_t* s;
    int64_t ld_s, inc;
    MO_DEV f32x8 at(int64_t r, int64_t c, int n) const {
        return from_e4m3(ldq8(p + r * ld + c, n), n > 0 ? scale_value(s[r * ld_s + c / F8_BLOCK * inc]) : 0.f);
    }
};

// dst[plane][c][ldt] <- src[r][c] in 64 x 64 tiles, zeros for rows from `rows` up to 64 tr;
// the tiles in blocks of 8 x 8 (whole 1 KB pieces of rows and columns by workgroups
// that run together).
template <typename T, int PL>
__global__ __launch_bounds__(256) void f8_transpose_kernel(Source<T> src, int64_t rows, int64_t cols, bf16_t* dst,
                                                           int64_t ldt, int64_t plane, uint32_t tr, uint32_t tc) {
    __shared__ float tile[XT][XT + 1];
    const uint32_t blocks_r = (tr + 7) / 8, units = blocks_r * ((tc + 7) / 8) * 64;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint32_t blk = u >> 6, ti = blk % blocks_r * 8 + (u & 7), tj = blk / blocks_r * 8 + (u >> 3 & 7);
        if (ti >= tr || tj >= tc) continue;
        const int64_t r0 = int64_t(ti) * XT, c0 = int64_t(tj) * XT;
        f32x8 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = threadIdx.x + 256 * i, r = w >> 3, c = (w & 7) * 8;
            const int64_t left = cols - c0 - c;
            const bool in = r0 + r < rows;
            v[i] = src.at(in ? r0 + r : 0, left > 0 ? c0 + c : 0, in ? int(left < 8 ? left : 8) : 0);
        }
        __syncthreads();   // the tile before has been read
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = threadIdx.x + 256 * i, r = w >> 3, c = (w & 7) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) tile[r][c + e] = v[i].v[e];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = threadIdx.x + 256 * i, c = w >> 3, r = (w & 7) * 8;
            if (c0 + c >= cols) continue;
            bf16x8 p[3];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = tile[r + e][c];
                if constexpr (PL == 1) {
                    p[0][e] = (bf16_t)x;
                } else {
                    bf16_t h, m, l;
                    split_f32(x, h, m, l);
                    p[0][e] = h;
                    p[1][e] = m;
                    p[2][e] = l;
                }
            }
#pragma unroll
            for (int k = 0; k < PL; ++k)
                *reinterpret_cast<u32x4*>(dst + k * plane + (c0 + c) * ldt + r0 + r) = __builtin_bit_cast(u32x4, p[k]);
        }
    }
}

unsigned grid_for(int64_t items) {
    const int64_t want = (items + 255) / 256;
    return unsigned(want < 4096 ? want : 4096);
}

// Workgroups of a product: one per CU at most, a multiple of the XCDs.
unsigned product_grid(const Tiles& t) {
    const uint64_t items = t.full ? t.full : uint64_t(t.rem) * t.splits;
    return items < 256 ? unsigned((items + 7) / 8 * 8) : 256u;
}
template <int KIND, int NB, typename T>
hipError_t product(const Operand8& P, const Operand8& Q, const Tiles& t, const Out<T>& o, hipStream_t s) {
    hipLaunchKernelGGL((f8_product_kernel<KIND, NB, T>), dim3(product_grid(t)), dim3(H_THREADS), 0, s, P, Q, t, o);
    if (t.rem) hipLaunchKernelGGL((f8_sum_kernel<NB, T>), dim3(t.rem * Layout<NB>::MB * 2), dim3(256), 0, s, t, o);
    return hipGetLastError();
}
template <int KIND, typename T>
hipError_t product_nb(const Operand8& P, const Operand8& Q, const MoF8Plan& p, const Out<T>& o, uint8_t* ws, hipStream_t s) {
    const Tiles t = {p.tm, p.tn, p.full, p.tm * p.tn - p.full, uint32_t(p.splits),
                     KIND == TOKENS ? 16u : 8u, p.nk, p.stages,
                     reinterpret_cast<f32x4*>(ws + p.off_part)};
    return p.nb == 4 ? product<KIND, 4>(P, Q, t, o, s) : p.nb == 2 ? product<KIND, 2>(P, Q, t, o, s)
                                                                   : product<KIND, 1>(P, Q, t, o, s);
}

}  // namespace

// Operand i (0: A, 1: B) of the product, copied or unpacked into the workspace.
hipError_t mo_launch_f8_pack(const MoF8Operand& a, const MoF8Plan& p, int i, int64_t dim, uint8_t* ws, hipStream_t s) {
    if (p.bf16) {
        hipLaunchKernelGGL(f8_unpack_kernel, dim3(grid_for(a.rows * (p.kd / 8))), dim3(256), 0, s, a.q, a.ld, a.s, a.ld_s,
                           a.inc, a.shift, a.rows, int(dim), reinterpret_cast<bf16_t*>(ws + p.off_q[i]), int(p.kd));
        return hipGetLastError();
    }
    if (p.pack_q[i])
        hipLaunchKernelGGL(f8_copy_kernel, dim3(grid_for(a.rows * (p.kd / 8))), dim3(256), 0, s, a.q, a.ld, a.rows, int(dim),
                           ws + p.off_q[i], int(p.kd));
    if (p.pack_s[i]) {
        const int64_t r = (a.rows + (int64_t(1) << a.shift) - 1) >> a.shift;
        hipLaunchKernelGGL(f8_copy_scales_kernel, dim3(grid_for(r * (p.ks / 4))), dim3(256), 0, s, a.s, a.ld_s, a.inc, r,
                           int((dim + F8_BLOCK - 1) / F8_BLOCK), reinterpret_cast<uint32_t*>(ws + p.off_s[i]), int(p.ks / 4));
    }
    return hipGetLastError();
}

hipError_t mo_launch_f8_matmul(const MoF8Operand& A, const MoF8Operand& B, const MoF8Plan& p, void* Y, int64_t ldy,
                               uint8_t* ws, hipStream_t s) {
    if (p.bf16) {
        const Operand8 Q = {ws + p.off_q[0], nullptr, p.kd * 2, A.rows}, P = {ws + p.off_q[1], nullptr, p.kd * 2, B.rows};
        return product_nb<BF16, float>(P, Q, p, {static_cast<float*>(Y), ldy, B.rows, A.rows, false}, ws, s);
    }
    auto operand = [&](const MoF8Operand& a, int i) {
        Operand8 o = {a.q, a.s, a.ld, a.rows, 0, a.ld_s, a.inc, a.shift};
        if (p.pack_q[i]) o.q = ws + p.off_q[i], o.ld = p.kd;
        if (p.pack_s[i]) o.s = ws + p.off_s[i], o.ld_s = p.ks, o.inc = 1;
        return o;
    };
    const Operand8 Q = operand(A, 0), P = operand(B, 1);
    const Out<bf16_t> o = {static_cast<bf16_t*>(Y), ldy, B.rows, A.rows, false};
    return B.shift ? product_nb<SQUARE8>(P, Q, p, o, ws, s) : product_nb<ROWS8>(P, Q, p, o, ws, s);
}

hipError_t mo_launch_f8_transpose(const MoF8Wgrad& a, const MoF8Plan& p, bool x, uint8_t* ws, hipStream_t s) {
    const int64_t cols = x ? a.dim : a.rows;
    const uint32_t tr = uint32_t(p.kd / XT), tc = uint32_t((cols + XT - 1) / XT);
    const uint64_t units = uint64_t((tr + 7) / 8) * ((tc + 7) / 8) * 64;
    const dim3 grid(unsigned(units < 8192 ? units : 8192));
    bf16_t* dst = reinterpret_cast<bf16_t*>(ws + p.off_q[x ? 1 : 0]);
    const int64_t plane = cols * p.ld_t;
    if (x)
        hipLaunchKernelGGL((f8_transpose_kernel<uint8_t, 1>), grid, dim3(256), 0, s,
                           Source<uint8_t>{a.X.q, a.X.ld, a.X.s, a.X.ld_s, a.X.inc}, a.X.rows, cols, dst, p.ld_t, plane, tr, tc);
    else if (a.dy_dtype == MO_BF16)
        hipLaunchKernelGGL((f8_transpose_kernel<bf16_t, 1>), grid, dim3(256), 0, s,
                           Source<bf16_t>{static_cast<const bf16_t*>(a.dY), a.lddy}, a.X.rows, cols, dst, p.ld_t, plane,
                           tr, tc);
    else
        hipLaunchKernelGGL((f8_transpose_kernel<float, 3>), grid, dim3(256), 0, s,
                           Source<float>{static_cast<const float*>(a.dY), a.lddy}, a.X.rows, cols, dst, p.ld_t, plane, tr,
                           tc);
    return hipGetLastError();
}

template <int KIND>
static hipError_t wgrad(const Operand8& P, const Operand8& Q, const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws,
                        hipStream_t s) {
    const bool add = a.accumulate != 0;
    if (a.g_dtype == MO_BF16)
        return product_nb<KIND, bf16_t>(P, Q, p, {static_cast<bf16_t*>(a.G), a.ldg, a.dim, a.rows, add}, ws, s);
    return product_nb<KIND, float>(P, Q, p, {static_cast<float*>(a.G), a.ldg, a.dim, a.rows, add}, ws, s);
}
hipError_t mo_launch_f8_wgrad(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    if (p.tokens) {
        const Operand8 P = {a.X.q, a.X.s, a.X.ld, a.dim, 0, a.X.ld_s, a.X.inc, 0, a.X.rows};
        const Operand8 Q = {static_cast<const uint8_t*>(a.dY), nullptr, a.lddy * 2, a.rows, 0, 0, 0, 0, a.X.rows};
        return wgrad<TOKENS>(P, Q, a, p, ws, s);
    }
    const Operand8 P = {ws + p.off_q[1], nullptr, p.ld_t * 2, a.dim};
    const Operand8 Q = {ws + p.off_q[0], nullptr, p.ld_t * 2, a.rows, a.rows * p.ld_t * 2};
    return a.dy_dtype == MO_BF16 ? wgrad<BF16>(P, Q, a, p, ws, s) : wgrad<BF16_3>(P, Q, a, p, ws, s);
}
