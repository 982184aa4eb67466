// Products with matrices in 8 bits:
//   Y = A B^T, both in 8 bits: in tiles (fp8_gemm.h; an fp32 result from the operands' values, which
//       are bf16 numbers) or, small ones, in blocks straight from registers; and
//   G = dY^T X, X an activation kept in 8 bits, dY as it is: X's values are bf16 numbers, an
//       fp32 dY is three of them.  In tiles, from the operands as they lie or from transposed
//       copies, or, small ones, in blocks.
// P, the operand with tiles of 256 rows, is the one along the result's columns: a lane's
// four accumulators are then four neighbours of a row.
#include "fp8_gemm.h"
#include "operators.h"

#include <cfloat>
#include <type_traits>

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
    const f32x4* z =
        t.part + int64_t(slot) * t.splits * stride + int64_t(wave) * (L::MB * L::NBW * 64) + a * (L::NBW * 64) + lane;
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

// ---- small products --------------------------------------------------------------------

// Few rows of Q, or little of everything: the product is a read of its operands, and the rest hides behind it.  A
// workgroup takes 16 RB rows of P and 16 TB of Q; its eight waves take every eighth block of K, D of them
// at a time, straight into registers, and add their sums up through LDS in order.  Workgroups start at
// different blocks, so that rows a power of two apart do not all ask the same memory channel at a time.
// Nothing is asked of the operands' alignment; what lies behind a row's end is not read.  T float: the
// values as bf16 numbers, with exact products.
//
// Four neighbouring lanes load 64 bytes of a row, 16 rows at once; the MFMA wants a row's four pieces in lanes
// 16 apart, so they change places through the wave's own part of LDS (which it uses in order:
// no barrier).  Loaded as the MFMA wants them, neighbouring lanes would read 16 different rows, and their lines
// are looked up one by one: 64 x 4096 x 4096 took 12.3 us and 8 x 14336 x 4096 12.6.
template <int TB, int RB, typename T>
__global__ __launch_bounds__(512) void f8_small_kernel(Operand8 P, Operand8 Q, int dim, uint32_t bp, uint32_t bq, Out<T> o) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int D = 4 / RB;
    __shared__ f32x4 sums[8][RB * TB < 4 ? 4 : RB * TB][64];
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // each XCD a contiguous share of the bp x bq blocks, the shorter side's side by side
    const uint32_t share = gridDim.x >> 3, rem = gridDim.x & 7, x = blockIdx.x & 7;
    const uint32_t block = x * share + (x < rem ? x : rem) + (blockIdx.x >> 3);
    const int64_t p0 = int64_t(bq < bp ? block / bq : block % bp) * (16 * RB);
    const int64_t q0 = int64_t(bq < bp ? block % bq : block / bp) * (16 * TB);
    const int full = dim / F8_BLOCK;
    union Frag {
        i32x8 v;
        u32x4 h[2];
    };
    const int lr = lane >> 2, lc = lane & 3;   // the row and the piece that a lane loads
    // Piece c of row r is piece 4 r + (c ^ r / 4) of 64: both sides of the turn use all banks.
    const int there = lr * 4 + (lc ^ (lr >> 2)), here = r16 * 4 + (kg ^ (r16 >> 2));
    auto turn = [&](u32x4 x, int i) __attribute__((always_inline)) {
        u32x4* z = reinterpret_cast<u32x4*>(sums[wave][i & 3]);
        z[there] = x;
        asm volatile("" ::: "memory");
        const u32x4 y = z[here];
        asm volatile("" ::: "memory");
        return y;
    };
    const uint8_t *pq[RB], *ps[RB], *qq[TB], *qs[TB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int64_t r = p0 + i * 16 + lr, row = r < P.rows ? r : P.rows - 1;
        pq[i] = P.q + row * P.ld + lc * 16;
        ps[i] = P.s + (row >> P.shift) * P.ld_s;
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int64_t r = q0 + i * 16 + lr, row = r < Q.rows ? r : Q.rows - 1;
        qq[i] = Q.q + row * Q.ld + lc * 16;
        qs[i] = Q.s + (row >> Q.shift) * Q.ld_s;
    }
    f32x4 acc[RB][TB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    typedef u32x4 u32x4_e1 __attribute__((aligned(1)));
    // A lane's two pieces of block k of a row (zeros behind its end; whole blocks without a branch)
    auto load = [&](Frag& f, const uint8_t* p, int k, bool whole) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* a = p + int64_t(k) * F8_BLOCK + h * 64;
            if (whole) {
                f.h[h] = *reinterpret_cast<const u32x4_e1*>(a);
            } else {
                const int n = dim - k * F8_BLOCK - h * 64 - lc * 16;
                const u32x2 lo = ldq8(a, n), hi = ldq8(a + 8, n - 8);
                f.h[h] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
        }
    };
    auto turn_all = [&](Frag& f, uint32_t& scale, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) f.h[h] = turn(f.h[h], 2 * i + h);
        scale = uint32_t(__builtin_amdgcn_ds_bpermute(r16 * 16, int(scale)));
    };
    // eight values of half e of piece h, as bf16
    auto wide = [&](const Frag& f, int h, int e, uint32_t scale) __attribute__((always_inline)) {
        const float s = __uint_as_float(scale << 23);   // (the conversion takes the exponent's field, as in e8m0)
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f.h[h][2 * e + i], s, false));
            w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f.h[h][2 * e + i], s, true));
        }
        return __builtin_bit_cast(bf16x8, w);
    };
    const int first = full ? int(block % uint32_t(full)) : 0;
    auto run = [&](int n, auto count, bool whole) __attribute__((always_inline)) {
        constexpr int N = decltype(count)::value;
        Frag a[N][RB], b[N][TB];
        uint32_t sa[N][RB], sb[N][TB];
#pragma unroll
        for (int d = 0; d < N; ++d) {
            int k = n + 8 * d;
            if (whole) {
                k += first;
                k = k < full ? k : k - full;
            }
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                load(a[d][i], pq[i], k, whole);
                sa[d][i] = ps[i][k * P.inc];
            }
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                load(b[d][i], qq[i], k, whole);
                sb[d][i] = qs[i][k * Q.inc];
            }
        }
#pragma unroll
        for (int d = 0; d < N; ++d) {
#pragma unroll
            for (int i = 0; i < RB; ++i) turn_all(a[d][i], sa[d][i], i);
#pragma unroll
            for (int i = 0; i < TB; ++i) turn_all(b[d][i], sb[d][i], RB + i);
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < TB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[d][i].v, b[d][j].v, acc[i][j], 0, 0, 0,
                                                                                     int(sa[d][i]), 0, int(sb[d][j]));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    bf16x8 y[TB];
#pragma unroll
                    for (int j = 0; j < TB; ++j) y[j] = wide(b[d][j], c / 2, c % 2, sb[d][j]);
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const bf16x8 x = wide(a[d][i], c / 2, c % 2, sa[d][i]);
#pragma unroll
                        for (int j = 0; j < TB; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y[j], acc[i][j], 0, 0, 0);
                    }
                }
            }
        }
    };
    int n = wave;
    for (; n + 8 * (D - 1) < full; n += 8 * D) run(n, std::integral_constant<int, D>(), true);
    for (; n < full; n += 8) run(n, std::integral_constant<int, 1>(), true);
    if (n == full && dim % F8_BLOCK) run(n, std::integral_constant<int, 1>(), false);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) sums[wave][i * TB + j][here] = acc[i][j];
    __syncthreads();
    // (turned back: four lanes store a row's 16 neighbours)
    for (int u = wave; u < RB * TB; u += 8) {
        f32x4 s = sums[0][u][there];
#pragma unroll
        for (int w = 1; w < 8; ++w) {
            const f32x4 x = sums[w][u][there];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += x[e];
        }
        put4(o, q0 + u % TB * 16 + lr, p0 + u / TB * 16 + lc * 4, s);
    }
#endif
}

// ---- operands laid out for them ------------------------------------------------------

// Scales with rows of ks bytes (a multiple of 4, 127 behind the last block).
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

// Rows to copy, 16-byte aligned and zeros behind their end: of either operand.  A wavefront per row; bound by memory.
struct CopyRows {
    const uint8_t* src;
    int64_t ld, rows;
    uint8_t* dst;
};
__global__ __launch_bounds__(256) void f8_copy_rows_kernel(CopyRows a, CopyRows b, int dim, int64_t ldd) {
    typedef u32x4 u32x4_e1 __attribute__((aligned(1)));
    const int lane = threadIdx.x & 63, chunks = int(ldd >> 4);
    for (int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); w < a.rows + b.rows; w += int64_t(gridDim.x) * 4) {
        const bool first = w < a.rows;
        const int64_t r = first ? w : w - a.rows;
        const uint8_t* src = first ? a.src + r * a.ld : b.src + r * b.ld;
        uint8_t* dst = (first ? a.dst : b.dst) + r * ldd;
#pragma unroll 4
        for (int c = lane; c < chunks; c += 64) {
            u32x4 x;
            const int n = dim - c * 16;
            if (n >= 16) {
                x = *reinterpret_cast<const u32x4_e1*>(src + c * 16);
            } else {
                const u32x2 lo = ldq8(src + c * 16, n), hi = ldq8(src + c * 16 + 8, n - 8);
                x = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
            *reinterpret_cast<u32x4*>(dst + c * 16) = x;
        }
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

// ---- small weight gradients ------------------------------------------------------------

// 64 rows of G (columns of dY) by 64 of its columns (of X) per workgroup, 64 tokens at a time: both operands
// come as they lie, eight neighbours of a row per thread and load, and go to LDS as bf16 (an fp32 dY as its three
// parts), from where transposing reads make fragments of them, as in TOKENS (fp8_gemm.h).  Nothing is asked of
// alignment, nothing is copied first, and several workgroups on a CU hide each other's waits; but every
// operand is read out of LDS for 64 columns of the other alone, so large gradients go faster in tiles.  The
// results turn in LDS, so that 16 lanes store 64 neighbours of a row.  A workgroup alone takes 0.56 us for 64 tokens in
// bf16 and 1.0 in fp32, bound by the wait from load to LDS to MFMA; several on a CU 0.26 and 0.56 each, bound by
// LDS (and by cutting fp32 in parts).  257 tokens x 1000 x 2001 in fp32: 13.1 us with the call, 20 in tiles.  Few
// blocks share a block's tokens among several workgroups (7803 x 16 x 16 in fp32: 15 us, 30 in tiles).
template <typename T, typename TG>
__global__ __launch_bounds__(256) void f8_small_wgrad_kernel(Source<uint8_t> x, Source<T> y, int64_t tokens, Out<TG> o,
                                                             uint32_t bx, uint32_t by, int64_t per, float* part) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int PL = sizeof(T) == 4 ? 3 : 1, PLANE = 64 * 128, ROW = 68;   // ROW: floats of a row of results
    constexpr int BYTES = PLANE * (1 + PL) > 64 * ROW * 4 ? PLANE * (1 + PL) : 64 * ROW * 4;
    __shared__ __align__(16) uint8_t smem[BYTES];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wp = wave & 1, wq = wave >> 1;
    // each XCD a contiguous share of the blocks, the shorter side's side by side; `per` tokens of a block at most
    const uint32_t share = gridDim.x >> 3, rem = gridDim.x & 7, xcd = blockIdx.x & 7;
    const uint32_t unit = xcd * share + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3), block = unit % (bx * by);
    const int64_t p0 = int64_t(by < bx ? block / by : block % bx) * 64, q0 = int64_t(by < bx ? block % by : block / bx) * 64;
    const int64_t from = int64_t(unit / (bx * by)) * per;
    if (tokens > from + per) tokens = from + per;
    // a thread's eight columns, of tokens row and row + 32 of a chunk
    const int row = tid >> 3, c = tid & 7;
    const int np = int(o.cols - p0 - c * 8 < 8 ? o.cols - p0 - c * 8 : 8);
    const int nq = int(o.rows - q0 - c * 8 < 8 ? o.rows - q0 - c * 8 : 8);
    const uint8_t* const xp = x.p + p0 + c * 8;
    const uint8_t* const xs = x.s + (p0 >> 7) * x.inc;
    const T* const yp = y.p + q0 + c * 8;
    u32x2 xq[2];
    uint32_t scale[2];
    raw8<T> yv[2];
    auto load = [&](int64_t t0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t t = t0 + row + 32 * i;
            const bool in = t < tokens;
            xq[i] = ldq8(xp + (in ? t : 0) * x.ld, in ? np : 0);
            scale[i] = in ? xs[t * x.ld_s] : 0u;
            yv[i] = ld8n(yp + (in ? t : 0) * y.ld, in ? nq : 0);
        }
    };
    // rows of 64 columns in granules of 16, permuted as TOKENS permutes Q's
    auto qf = [&](int r) __attribute__((always_inline)) { return ((r >> 1) & 1) | (((r >> 2) ^ (r >> 3)) & 2); };
    auto put_row = [&](uint8_t* plane, int r, u32x4 v) __attribute__((always_inline)) {
        *reinterpret_cast<u32x4*>(plane + r * 128 + ((c ^ (qf(r) << 1)) << 4)) = v;
    };
    auto store = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row + 32 * i;
            const float f = __uint_as_float(scale[i] << 23);   // (the conversion takes the exponent's field, as in e8m0)
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(xq[i][e], f, false));
                w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(xq[i][e], f, true));
            }
            put_row(smem, r, w);
            if constexpr (PL == 1) {
                put_row(smem + PLANE, r, __builtin_bit_cast(u32x4, yv[i]));
            } else {
                // its upper 8 bits, the next 8 and the rest, cut off and so exact; an infinity is one in the
                // first part alone, a NaN stays one
                const f32x8 v = widen(yv[i]);
                uint32_t z[3][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = __builtin_canonicalizef(v.v[e]), g = __builtin_amdgcn_fmed3f(f, -FLT_MAX, FLT_MAX);
                    const float r = g - __uint_as_float(__float_as_uint(g) & 0xFFFF0000u);
                    z[0][e] = __float_as_uint(f);
                    z[1][e] = __float_as_uint(r);
                    z[2][e] = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & 0xFFFF0000u));
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    u32x4 u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // the upper halves
                        u[e] = __builtin_amdgcn_perm(z[k][2 * e + 1], z[k][2 * e], 0x07060302);
                    put_row(smem + (1 + k) * PLANE, r, u);
                }
            }
        }
    };
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int trow = kg * 8 + (r16 >> 2);
    // tokens 32 h .. of granule g's 16 columns
    auto frag = [&](const uint8_t* plane, int g, int h) __attribute__((always_inline)) {
        const uint8_t* p = plane + trow * 128 + ((g ^ qf(trow)) << 5) + (r16 & 3) * 8 + h * 32 * 128;
        u32x4 f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + j * 4 * 128)));
            f[2 * j] = v[0];
            f[2 * j + 1] = v[1];
        }
        return __builtin_bit_cast(bf16x8, f);
    };
    f32x4 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    load(from);
    for (int64_t t0 = from; t0 < tokens; t0 += 64) {
        store();
        __syncthreads();
        if (t0 + 64 < tokens) load(t0 + 64);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 p[2];
#pragma unroll
            for (int a = 0; a < 2; ++a) p[a] = frag(smem, wp * 2 + a, h);
            // the smallest part first
#pragma unroll
            for (int k = PL; k >= 1; --k)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bf16x8 q = frag(smem + k * PLANE, wq * 2 + b, h);
#pragma unroll
                    for (int a = 0; a < 2; ++a) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[a], q, acc[a][b], 0, 0, 0);
                }
        }
        __syncthreads();
    }
    float* const z = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            *reinterpret_cast<f32x4*>(z + (wq * 32 + b * 16 + r16) * ROW + wp * 32 + a * 16 + kg * 4) = acc[a][b];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 16 + (tid >> 4), k = (tid & 15) * 4;
        const f32x4 v = *reinterpret_cast<const f32x4*>(z + r * ROW + k);
        if (part) *reinterpret_cast<f32x4*>(part + int64_t(unit) * 4096 + r * 64 + k) = v;
        else put4(o, q0 + r, p0 + k, v);
    }
#endif
}

// The sums of the parts of each block's tokens, in order.
template <typename TG>
__global__ __launch_bounds__(256) void f8_small_sum_kernel(const float* part, uint32_t splits, uint32_t bx, uint32_t by,
                                                           Out<TG> o) {
    const uint32_t block = blockIdx.x >> 2;
    const int at = (blockIdx.x & 3) * 1024 + threadIdx.x * 4;
    const f32x4* z = reinterpret_cast<const f32x4*>(part + int64_t(block) * 4096 + at);
    const int64_t stride = int64_t(bx * by) * 1024;
    f32x4 s = z[0];
#pragma unroll 8
    for (uint32_t k = 1; k < splits; ++k) {
        const f32x4 v = z[k * stride];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
    const int64_t p0 = int64_t(by < bx ? block / by : block % bx) * 64, q0 = int64_t(by < bx ? block % by : block / bx) * 64;
    put4(o, q0 + (at >> 6), p0 + (at & 63), s);
}

// dst[plane][c][ldt] <- src[r][c], zeros for rows from `rows` up to 64 tr.
template <typename T> struct Transpose {
    Source<T> src;
    int64_t cols;
    bf16_t* dst;
    int64_t plane;
    uint32_t tc, units;   // tiles of 64 columns; tiles in whole blocks of 8 x 8
};
// One 64 x 64 tile of it; the tiles in blocks of 8 x 8 (whole 1 KB pieces of rows and columns by
// workgroups that run together).
template <typename T, int PL>
MO_DEV void transpose_tile(float (&tile)[XT][XT + 1], const Transpose<T>& t, uint32_t u, int64_t rows, int64_t ldt, uint32_t tr) {
    const uint32_t blocks_r = (tr + 7) / 8;
    const uint32_t blk = u >> 6, ti = blk % blocks_r * 8 + (u & 7), tj = blk / blocks_r * 8 + (u >> 3 & 7);
    if (ti >= tr || tj >= t.tc) return;
    const int64_t r0 = int64_t(ti) * XT, c0 = int64_t(tj) * XT;
    f32x8 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int w = threadIdx.x + 256 * i, r = w >> 3, c = (w & 7) * 8;
        const int64_t left = t.cols - c0 - c;
        const bool in = r0 + r < rows;
        v[i] = t.src.at(in ? r0 + r : 0, left > 0 ? c0 + c : 0, in ? int(left < 8 ? left : 8) : 0);
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
        if (c0 + c >= t.cols) continue;
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
            *reinterpret_cast<u32x4*>(t.dst + k * t.plane + (c0 + c) * ldt + r0 + r) = __builtin_bit_cast(u32x4, p[k]);
    }
}
// Both operands of a weight gradient in one launch.
template <typename T, int PL>
__global__ __launch_bounds__(256) void f8_transpose_kernel(Transpose<uint8_t> x, Transpose<T> y, int64_t rows, int64_t ldt,
                                                           uint32_t tr) {
    __shared__ float tile[XT][XT + 1];
    for (uint32_t u = blockIdx.x; u < x.units + y.units; u += gridDim.x)
        if (u < x.units) transpose_tile<uint8_t, 1>(tile, x, u, rows, ldt, tr);
        else transpose_tile<T, PL>(tile, y, u - x.units, rows, ldt, tr);
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

// The rows of both operands of the product, or of the one that is not in place.
hipError_t mo_launch_f8_copy(const MoF8Operand& a, const MoF8Operand& b, const MoF8Plan& p, int64_t dim, uint8_t* ws,
                             hipStream_t s) {
    const CopyRows x = {a.q, a.ld, p.pack_q[0] ? a.rows : 0, ws + p.off_q[0]};
    const CopyRows y = {b.q, b.ld, p.pack_q[1] ? b.rows : 0, ws + p.off_q[1]};
    hipLaunchKernelGGL(f8_copy_rows_kernel, dim3(grid_for((x.rows + y.rows) * 64)), dim3(256), 0, s, x, y, int(dim), p.ld_q);
    return hipGetLastError();
}
// The scales of operand i (0: A, 1: B) of the product, copied into the workspace.
hipError_t mo_launch_f8_pack(const MoF8Operand& a, const MoF8Plan& p, int i, int64_t dim, uint8_t* ws, hipStream_t s) {
    const int64_t r = (a.rows + (int64_t(1) << a.shift) - 1) >> a.shift;
    hipLaunchKernelGGL(f8_copy_scales_kernel, dim3(grid_for(r * (p.ks / 4))), dim3(256), 0, s, a.s, a.ld_s, a.inc, r,
                       int((dim + F8_BLOCK - 1) / F8_BLOCK), reinterpret_cast<uint32_t*>(ws + p.off_s[i]), int(p.ks / 4));
    return hipGetLastError();
}

template <int TB, int RB, typename T>
static void small_tile(const Operand8& P, const Operand8& Q, int64_t dim, const Out<T>& o, hipStream_t s) {
    const uint32_t bp = uint32_t((P.rows + 16 * RB - 1) / (16 * RB)), bq = uint32_t((Q.rows + 16 * TB - 1) / (16 * TB));
    hipLaunchKernelGGL((f8_small_kernel<TB, RB, T>), dim3(bp * bq), dim3(512), 0, s, P, Q, int(dim), bp, bq, o);
}
template <typename T>
static hipError_t small(const Operand8& P, const Operand8& Q, int64_t dim, int tb, int rb, const Out<T>& o, hipStream_t s) {
    if (tb == 4) small_tile<4, 4>(P, Q, dim, o, s);
    else if (tb == 2) small_tile<2, 2>(P, Q, dim, o, s);
    else if (rb == 2) small_tile<1, 2>(P, Q, dim, o, s);
    else small_tile<1, 1>(P, Q, dim, o, s);
    return hipGetLastError();
}
hipError_t mo_launch_f8_small(const MoF8Operand& A, const MoF8Operand& B, const MoF8Plan& p, int64_t dim, void* Y, int64_t ldy,
                              int32_t dtype, hipStream_t s) {
    const Operand8 Q = {A.q, A.s, A.ld, A.rows, 0, A.ld_s, A.inc, A.shift};
    const Operand8 P = {B.q, B.s, B.ld, B.rows, 0, B.ld_s, B.inc, B.shift};
    if (dtype == MO_BF16) return small<bf16_t>(P, Q, dim, p.tb, p.rb, {static_cast<bf16_t*>(Y), ldy, B.rows, A.rows, false}, s);
    return small<float>(P, Q, dim, p.tb, p.rb, {static_cast<float*>(Y), ldy, B.rows, A.rows, false}, s);
}
hipError_t mo_launch_f8_matmul(const MoF8Operand& A, const MoF8Operand& B, const MoF8Plan& p, int64_t dim, void* Y,
                               int64_t ldy, int32_t dtype, uint8_t* ws, hipStream_t s) {
    auto operand = [&](const MoF8Operand& a, int i) {
        Operand8 o = {a.q, a.s, a.ld, a.rows, 0, a.ld_s, a.inc, a.shift, dim};
        if (p.pack_q[i]) o.q = ws + p.off_q[i], o.ld = p.ld_q;
        if (p.pack_s[i]) o.s = ws + p.off_s[i], o.ld_s = p.ks, o.inc = 1;
        return o;
    };
    const Operand8 Q = operand(A, 0), P = operand(B, 1);
    if (dtype == MO_F32) return product_nb<VALUES8, float>(P, Q, p, {static_cast<float*>(Y), ldy, B.rows, A.rows, false}, ws, s);
    const Out<bf16_t> o = {static_cast<bf16_t*>(Y), ldy, B.rows, A.rows, false};
    if (p.bf16) return product_nb<VALUES8>(P, Q, p, o, ws, s);
    return B.shift ? product_nb<SQUARE8>(P, Q, p, o, ws, s) : product_nb<ROWS8>(P, Q, p, o, ws, s);
}

template <typename T, int PL>
static hipError_t transpose(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    const uint32_t tr = uint32_t(p.kd / XT), br = (tr + 7) / 8;
    auto tiles = [](int64_t cols) { return uint32_t((cols + XT - 1) / XT); };
    const uint32_t tx = tiles(a.dim), ty = tiles(a.rows);
    const Transpose<uint8_t> x = {{a.X.q, a.X.ld, a.X.s, a.X.ld_s, a.X.inc}, a.dim, reinterpret_cast<bf16_t*>(ws + p.off_q[1]),
                                  0, tx, br * ((tx + 7) / 8) * 64};
    const Transpose<T> y = {{static_cast<const T*>(a.dY), a.lddy}, a.rows, reinterpret_cast<bf16_t*>(ws + p.off_q[0]),
                            a.rows * p.ld_t, ty, br * ((ty + 7) / 8) * 64};
    const uint32_t units = x.units + y.units;
    hipLaunchKernelGGL((f8_transpose_kernel<T, PL>), dim3(units < 8192 ? units : 8192), dim3(256), 0, s, x, y, a.X.rows,
                       p.ld_t, tr);
    return hipGetLastError();
}
hipError_t mo_launch_f8_transpose(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    return a.dy_dtype == MO_BF16 ? transpose<bf16_t, 1>(a, p, ws, s) : transpose<float, 3>(a, p, ws, s);
}

template <typename T, typename TG>
static hipError_t small_wgrad(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    const uint32_t bx = uint32_t((a.dim + 63) / 64), by = uint32_t((a.rows + 63) / 64), splits = uint32_t(p.splits);
    const Source<uint8_t> x = {a.X.q, a.X.ld, a.X.s, a.X.ld_s, a.X.inc};
    const Source<T> y = {static_cast<const T*>(a.dY), a.lddy};
    const Out<TG> o = {static_cast<TG*>(a.G), a.ldg, a.dim, a.rows, a.accumulate != 0};
    float* part = splits > 1 ? reinterpret_cast<float*>(ws + p.off_part) : nullptr;
    hipLaunchKernelGGL((f8_small_wgrad_kernel<T, TG>), dim3(bx * by * splits), dim3(256), 0, s, x, y, a.X.rows, o, bx, by,
                       int64_t(p.stages) * 64, part);
    if (part) hipLaunchKernelGGL(f8_small_sum_kernel<TG>, dim3(bx * by * 4), dim3(256), 0, s, part, splits, bx, by, o);
    return hipGetLastError();
}
hipError_t mo_launch_f8_small_wgrad(const MoF8Wgrad& a, const MoF8Plan& p, uint8_t* ws, hipStream_t s) {
    if (a.dy_dtype == MO_BF16)
        return a.g_dtype == MO_BF16 ? small_wgrad<bf16_t, bf16_t>(a, p, ws, s) : small_wgrad<bf16_t, float>(a, p, ws, s);
    return a.g_dtype == MO_BF16 ? small_wgrad<float, bf16_t>(a, p, ws, s) : small_wgrad<float, float>(a, p, ws, s);
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
