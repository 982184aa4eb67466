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

// ---- the products' tiles -------------------------------------------------------------

// Where a tile's results go: dst[q][p], element strides ld and 1.
template <typename T> struct Out {
    T* dst;
    int64_t ld, cols, rows;   // cols: along P, rows: along Q
    bool add;
};

// Four neighbours of row q from column p on.
template <typename T> MO_DEV void put4(const Out<T>& o, int64_t q, int64_t p, f32x4 v) {
    const int n = int(o.cols - p < 4 ? o.cols - p : 4);
    if (q >= o.rows || n <= 0) return;
    T* d = o.dst + q * o.ld + p;
    typedef T vec __attribute__((ext_vector_type(4)));
    typedef vec vec_e __attribute__((aligned(sizeof(T))));
    if (n == 4) {
        if (o.add) {
            const vec old = *reinterpret_cast<const vec_e*>(d);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += to_f32(T(old[e]));
        }
        vec w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = from_f32<T>(v[e]);
        *reinterpret_cast<vec_e*>(d) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) d[e] = from_f32<T>(o.add ? v[e] + to_f32(d[e]) : v[e]);
    }
}

// KIND 8: 8-bit operands, P's scales in blocks of 128 rows; 9: by rows; 1: bf16; 4: bf16, Q in
// three planes.
constexpr int KSQ = 8, KROW = 9;
template <int KIND> struct Operands { using type = Operand; };
template <> struct Operands<KSQ> { using type = Operand8; };
template <> struct Operands<KROW> { using type = Operand8; };
template <int KIND, int NB> constexpr int lds_of() {
    return KIND == KSQ ? f8_lds<true>(NB) : KIND == KROW ? f8_lds<false>(NB) : head_lds(NB);
}

template <int KIND> struct Job {
    typename Operands<KIND>::type P, Q;
    int nk, stages;           // K stages in all and per split
    uint32_t tm, tn, splits;
    f32x4* part;              // the splits' sums: [split][tile][wave][MB x NBW][lane]
};

template <int KIND, int NB, bool SPLIT, typename T>
__global__ __launch_bounds__(H_THREADS) __attribute__((amdgpu_waves_per_eu(2))) void f8_product_kernel(Job<KIND> j,
                                                                                                       Out<T> o) {
    using L = Layout<NB>;
    __shared__ __align__(16) uint8_t smem[lds_of<KIND, NB>()];
    uint32_t ti, tj, split = 0, b = blockIdx.x;
    if constexpr (SPLIT) {
        const uint32_t per = (j.tm * j.tn + 7) / 8 * 8;
        split = b / per;
        b -= split * per;
    }
    if (!head_tile_of(b, j.tm, j.tn, ti, tj)) return;
    const int k0 = int(split) * j.stages, nk = j.nk - k0 < j.stages ? j.nk - k0 : j.stages;
    const int64_t p0 = int64_t(ti) * 256, q0 = int64_t(tj) * 64 * NB;
    f32x4 acc[L::MB][L::NBW];
    if constexpr (KIND >= KSQ) f8_tile<NB, KIND == KSQ>(smem, j.P, j.Q, p0, q0, k0, nk, acc);
    else head_tile<NB, KIND>(smem, j.P, j.Q, p0, q0, k0, nk, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if constexpr (SPLIT) {
        f32x4* z = j.part + ((int64_t(split) * j.tm * j.tn + int64_t(ti) * j.tn + tj) * 8 + wave) * (L::MB * L::NBW * 64) + lane;
#pragma unroll
        for (int i = 0; i < L::MB * L::NBW; ++i) z[i * 64] = acc[i / L::NBW][i % L::NBW];
    } else {
        const int64_t p = p0 + wave / L::WN * (L::MB * 16) + (lane >> 4) * 4, q = q0 + wave % L::WN * 64 + (lane & 15);
#pragma unroll
        for (int b2 = 0; b2 < L::NBW; ++b2)
#pragma unroll
            for (int a = 0; a < L::MB; ++a) put4(o, q + b2 * 16, p + a * 16, acc[a][b2]);
    }
}

// The splits' sums in order: one wavefront per 16 x 64 of a wave's block.
template <int NB, typename T>
__global__ __launch_bounds__(256) void f8_sum_kernel(const f32x4* part, uint32_t tm, uint32_t tn, uint32_t splits, Out<T> o) {
    using L = Layout<NB>;
    const uint32_t unit = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t a = unit % L::MB, wave = unit / L::MB % 8, tile = unit / (L::MB * 8);
    if (tile >= tm * tn) return;
    const f32x4* z = part + (int64_t(tile) * 8 + wave) * (L::MB * L::NBW * 64) + a * (L::NBW * 64) + lane;
    const int64_t stride = int64_t(tm) * tn * 8 * (L::MB * L::NBW * 64);
    f32x4 s[L::NBW];
#pragma unroll
    for (int b = 0; b < L::NBW; ++b) s[b] = z[b * 64];
#pragma unroll 4
    for (uint32_t t = 1; t < splits; ++t)
#pragma unroll
        for (int b = 0; b < L::NBW; ++b) {
            const f32x4 x = z[t * stride + b * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][e] += x[e];
        }
    const uint32_t ti = tile / tn, tj = tile - ti * tn;
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

template <int KIND, int NB, typename T>
hipError_t product(const Job<KIND>& j, const Out<T>& o, hipStream_t s) {
    const uint32_t tiles = j.tm * j.tn, grid = head_grid(tiles);
    if (j.splits == 1) {
        hipLaunchKernelGGL((f8_product_kernel<KIND, NB, false, T>), dim3(grid), dim3(H_THREADS), 0, s, j, o);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((f8_product_kernel<KIND, NB, true, T>), dim3(grid * j.splits), dim3(H_THREADS), 0, s, j, o);
    hipLaunchKernelGGL((f8_sum_kernel<NB, T>), dim3(tiles * Layout<NB>::MB * 2), dim3(256), 0, s, j.part, j.tm, j.tn,
                       j.splits, o);
    return hipGetLastError();
}
template <int KIND, typename T>
hipError_t product_nb(const Job<KIND>& j, int nb, const Out<T>& o, hipStream_t s) {
    return nb == 4 ? product<KIND, 4>(j, o, s) : nb == 2 ? product<KIND, 2>(j, o, s) : product<KIND, 1>(j, o, s);
}
template <int KIND> Job<KIND> job_of(const MoF8Plan& p, uint8_t* ws) {
    Job<KIND> j = {};
    j.nk = p.nk;
    j.stages = p.stages;
    j.tm = p.tm;
    j.tn = p.tn;
    j.splits = uint32_t(p.splits);
    j.part = reinterpret_cast<f32x4*>(ws + p.off_part);
    return j;
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

template <int KIND>
static hipError_t matmul8(const MoF8Operand& A, const MoF8Operand& B, const MoF8Plan& p, void* Y, int64_t ldy,
                          uint8_t* ws, hipStream_t s) {
    Job<KIND> j = job_of<KIND>(p, ws);
    auto operand = [&](const MoF8Operand& a, int i) {
        Operand8 o = {a.q, a.s, a.ld, a.rows, a.ld_s, a.inc, a.shift};
        if (p.pack_q[i]) o.q = ws + p.off_q[i], o.ld = p.kd;
        if (p.pack_s[i]) o.s = ws + p.off_s[i], o.ld_s = p.ks, o.inc = 1;
        return o;
    };
    j.Q = operand(A, 0);
    j.P = operand(B, 1);
    return product_nb<KIND, bf16_t>(j, p.nb, {static_cast<bf16_t*>(Y), ldy, B.rows, A.rows, false}, s);
}
hipError_t mo_launch_f8_matmul(const MoF8Operand& A, const MoF8Operand& B, const MoF8Plan& p, void* Y, int64_t ldy,
                               uint8_t* ws, hipStream_t s) {
    if (p.bf16) {
        Job<1> j = job_of<1>(p, ws);
        j.Q = {ws + p.off_q[0], p.kd * 2, A.rows, 0};
        j.P = {ws + p.off_q[1], p.kd * 2, B.rows, 0};
        return product_nb<1, float>(j, p.nb, {static_cast<float*>(Y), ldy, B.rows, A.rows, false}, s);
    }
    return B.shift ? matmul8<KSQ>(A, B, p, Y, ldy, ws, s) : matmul8<KROW>(A, B, p, Y, ldy, ws, s);
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

template <int KIND> static hipError_t wgrad(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    Job<KIND> j = job_of<KIND>(p, ws);
    j.P = {ws + p.off_q[1], p.ld_t * 2, a.dim, 0};
    j.Q = {ws + p.off_q[0], p.ld_t * 2, a.rows, a.rows * p.ld_t * 2};
    if (a.g_dtype == MO_BF16)
        return product_nb<KIND, bf16_t>(j, p.nb, {static_cast<bf16_t*>(a.G), a.ldg, a.dim, a.rows, a.accumulate != 0}, s);
    return product_nb<KIND, float>(j, p.nb, {static_cast<float*>(a.G), a.ldg, a.dim, a.rows, a.accumulate != 0}, s);
}
hipError_t mo_launch_f8_wgrad(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    return a.dy_dtype == MO_BF16 ? wgrad<1>(a, p, ws, s) : wgrad<4>(a, p, ws, s);
}
