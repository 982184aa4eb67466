// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   Y[i] = s W[t_i],   G[v] = s sum_{i : t_i = v} dY[i]   (or G[v] += ..)
//
// A token outside 0 .. vocab - 1 marks a padded position: its Y row is zero and
// its dY row is not read.
//
// The gradient is the transpose of the lookup.  Adding rows with atomics would
// make the sum's order, hence its last bits, change from call to call; instead
// the positions are sorted by token (stable, so equal tokens stay in position
// order), and each run of equal tokens is summed in fp32 in that order and
// written once.
#include "op_common.h"
#include "operators.h"

namespace {

constexpr int EMB_THREADS = 256;

// `tpr` threads (a power of two, at most 256) per row, 16-byte chunks.
template <typename T>
__global__ __launch_bounds__(EMB_THREADS) void emb_fwd_kernel(const int64_t* tokens, int64_t n, const T* W,
                                                              int64_t ldw, int64_t vocab, T* Y, int64_t ldy,
                                                              int dim, float scale, int tpr) {
    const int per = EMB_THREADS / tpr, t = threadIdx.x & (tpr - 1), sub = threadIdx.x / tpr;
    for (int64_t i = int64_t(blockIdx.x) * per + sub; i < n; i += int64_t(gridDim.x) * per) {
        const int64_t v = tokens[i];
        const bool in = uint64_t(v) < uint64_t(vocab);
        const T* w = W + (in ? v : 0) * ldw;
        T* y = Y + i * ldy;
        for (int c = t * 8; c < dim; c += tpr * 8) {
            f32x8 x = widen(ld8n(w + c, in ? dim - c : 0));
#pragma unroll
            for (int e = 0; e < 8; ++e) x.v[e] = in ? x.v[e] * scale : 0.f;
            st8n(y + c, x, dim - c);
        }
    }
}

// Orders one wavefront's LDS accesses before and after it.
MO_DEV void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- stable sort of the positions by token --------------------------------------
// Least significant digit first, up to 9 bits per pass.  Per pass: digit counts
// per tile of SORT_TILE positions, one exclusive scan over (digit, tile), and a
// scatter in which each wavefront ranks its 64 positions at a time by ballots.

constexpr int SORT_TILE = MO_EMB_SORT_TILE, SORT_WAVES = EMB_THREADS / 64;
constexpr int MAX_DIGITS = 512;

MO_DEV uint32_t key_of(const int64_t* tokens, const uint32_t* keys, int64_t i, uint32_t vocab) {
    if (!tokens) return keys[i];
    const int64_t v = tokens[i];
    return uint64_t(v) < vocab ? uint32_t(v) : vocab;   // padded positions sort last
}

__global__ __launch_bounds__(EMB_THREADS) void emb_count_kernel(const int64_t* tokens, const uint32_t* keys,
                                                                int64_t n, uint32_t vocab, int shift, int bits,
                                                                uint32_t* hist) {
    __shared__ uint32_t h[MAX_DIGITS];
    const int nd = 1 << bits;
    for (int d = threadIdx.x; d < nd; d += EMB_THREADS) h[d] = 0;
    __syncthreads();
    const int64_t a = int64_t(blockIdx.x) * SORT_TILE;
    const int64_t b = a + SORT_TILE < n ? a + SORT_TILE : n;
    for (int64_t i = a + threadIdx.x; i < b; i += EMB_THREADS)
        atomicAdd(&h[(key_of(tokens, keys, i, vocab) >> shift) & (nd - 1)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < nd; d += EMB_THREADS) hist[int64_t(d) * gridDim.x + blockIdx.x] = h[d];
}

// Exclusive scan of `len` counts, in place, one workgroup.
__global__ __launch_bounds__(1024) void emb_scan_kernel(uint32_t* hist, int64_t len) {
    __shared__ uint32_t sums[16];
    uint32_t carry = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t base = 0; base < len; base += 4096) {
        const int64_t i = base + threadIdx.x * 4;
        uint32_t v[4], s = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = i + e < len ? hist[i + e] : 0; s += v[e]; }
        uint32_t inc = s;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63) sums[wave] = inc;
        __syncthreads();
        uint32_t before = carry, total = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) before += sums[w];
            total += sums[w];
        }
        uint32_t run = before + inc - s;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < len) { hist[i + e] = run; run += v[e]; }
        carry += total;
        __syncthreads();
    }
}

__global__ __launch_bounds__(EMB_THREADS) void emb_scatter_kernel(
    const int64_t* tokens, const uint32_t* keys, const uint32_t* idx, int64_t n, uint32_t vocab, int shift,
    int bits, const uint32_t* hist, uint32_t* out_keys, uint32_t* out_idx) {
    __shared__ uint32_t off[SORT_WAVES][MAX_DIGITS];
    const int nd = 1 << bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = threadIdx.x; d < SORT_WAVES * MAX_DIGITS; d += EMB_THREADS) (&off[0][0])[d] = 0;
    __syncthreads();
    constexpr int PER_WAVE = SORT_TILE / SORT_WAVES;
    const int64_t a = int64_t(blockIdx.x) * SORT_TILE + wave * PER_WAVE;
    const int64_t b = a + PER_WAVE < n ? a + PER_WAVE : n;
    for (int64_t i = a + lane; i < b; i += 64)
        atomicAdd(&off[wave][(key_of(tokens, keys, i, vocab) >> shift) & (nd - 1)], 1u);
    __syncthreads();
    // counts per wave -> where each wave's first key of a digit goes
    for (int d = threadIdx.x; d < nd; d += EMB_THREADS) {
        uint32_t run = hist[int64_t(d) * gridDim.x + blockIdx.x];
        for (int w = 0; w < SORT_WAVES; ++w) {
            const uint32_t c = off[w][d];
            off[w][d] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int64_t g = a; g < b; g += 64) {
        const int64_t i = g + lane;
        const bool on = i < b;
        const uint32_t key = on ? key_of(tokens, keys, i, vocab) : 0;
        const uint32_t d = (key >> shift) & (nd - 1);
        uint64_t same = __ballot(on);   // lanes with this lane's digit
        for (int k = 0; k < bits; ++k) {
            const uint64_t m = __ballot((d >> k) & 1);
            same &= (d >> k) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        uint32_t pos = 0;
        if (on) pos = off[wave][d] + rank;
        wave_sync();
        // the digit's last lane moves its offset on; every lane has read it
        if (on && (same >> lane) == 1) off[wave][d] = pos + 1;
        wave_sync();
        if (on) {
            out_keys[pos] = key;
            out_idx[pos] = tokens ? uint32_t(i) : idx[i];
        }
    }
}

// ---- sums over the runs -----------------------------------------------------------

// First position with key >= v.
MO_DEV int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t v) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Zeros in the rows no token names: 16 rows per workgroup.
constexpr int FILL_ROWS = 16;
template <typename T>
__global__ __launch_bounds__(EMB_THREADS) void emb_fill_kernel(const uint32_t* keys, int64_t n, T* G,
                                                               int64_t ldg, uint32_t vocab, int dim) {
    __shared__ int present[FILL_ROWS];
    const uint32_t v0 = blockIdx.x * FILL_ROWS;
    if (threadIdx.x < FILL_ROWS) {
        const uint32_t v = v0 + threadIdx.x;
        const int64_t p = lower_bound(keys, n, v);
        present[threadIdx.x] = v >= vocab || (p < n && keys[p] == v);
    }
    __syncthreads();
    f32x8 z;
#pragma unroll
    for (int e = 0; e < 8; ++e) z.v[e] = 0.f;
    for (int r = 0; r < FILL_ROWS; ++r) {
        if (present[r]) continue;
        T* g = G + int64_t(v0 + r) * ldg;
        for (int c = threadIdx.x * 8; c < dim; c += EMB_THREADS * 8) st8n(g + c, z, dim - c);
    }
}

template <typename T>
MO_DEV void put_row(T* g, const f32x8& sum, float scale, int accumulate, int n) {
    f32x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.v[e] = sum.v[e] * scale;
    if (accumulate) {
        const f32x8 old = widen(ld8n(g, n));
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] += old.v[e];
    }
    st8n(g, o, n);
}

// Chunk blockIdx.y of C sorted positions, 2048 columns.  A run inside the chunk
// is written; the part of a run that came in from the chunk before goes to
// head[chunk], the start of one that goes on to tail[chunk].
template <typename TY, typename TG>
__global__ __launch_bounds__(EMB_THREADS) void emb_sum_kernel(const uint32_t* keys, const uint32_t* idx,
                                                              int64_t n, int C, const TY* dY, int64_t lddy,
                                                              TG* G, int64_t ldg, uint32_t vocab, int dim,
                                                              float scale, int accumulate, float* head,
                                                              float* tail) {
    const int c = (blockIdx.x * EMB_THREADS + threadIdx.x) * 8;
    const int left = dim - c;
    const int64_t a = int64_t(blockIdx.y) * C, b = a + C < n ? a + C : n;
    if (left <= 0) return;
    const bool came_in = a > 0 && keys[a - 1] == keys[a];
    f32x8 sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum.v[e] = 0.f;
    bool first = true;
    for (int64_t p = a; p < b; ++p) {
        const uint32_t k = keys[p];
        if (k >= vocab) break;
        const f32x8 x = widen(ld8n(dY + int64_t(idx[p]) * lddy + c, left));
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] += x.v[e];
        const bool more = p + 1 < n && keys[p + 1] == k;
        if (more && p + 1 < b) continue;
        if (first && came_in) st8n(head + int64_t(blockIdx.y) * dim + c, sum, left);
        else if (more) st8n(tail + int64_t(blockIdx.y) * dim + c, sum, left);
        else put_row(G + int64_t(k) * ldg + c, sum, scale, accumulate, left);
        first = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] = 0.f;
    }
}

// Runs over several chunks: the chunk where one starts adds up its parts in order.
template <typename TG>
__global__ __launch_bounds__(EMB_THREADS) void emb_join_kernel(const uint32_t* keys, int64_t n, int C, TG* G,
                                                               int64_t ldg, uint32_t vocab, int dim, float scale,
                                                               int accumulate, const float* head,
                                                               const float* tail) {
    const int64_t a = int64_t(blockIdx.y) * C, b = a + C < n ? a + C : n;
    const uint32_t k = keys[b - 1];
    if (k >= vocab || b >= n || keys[b] != k) return;      // nothing goes on
    if (a > 0 && keys[a - 1] == k) return;                  // started before
    const int c = (blockIdx.x * EMB_THREADS + threadIdx.x) * 8;
    const int left = dim - c;
    if (left <= 0) return;
    const int64_t last = (lower_bound(keys, n, k + 1) - 1) / C;
    f32x8 sum = widen(ld8n(tail + int64_t(blockIdx.y) * dim + c, left));
#pragma unroll 4
    for (int64_t q = int64_t(blockIdx.y) + 1; q <= last; ++q) {
        const f32x8 x = widen(ld8n(head + q * dim + c, left));
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] += x.v[e];
    }
    put_row(G + int64_t(k) * ldg + c, sum, scale, accumulate, left);
}

template <typename T>
hipError_t fwd(const MoEmbArgs& a, hipStream_t s) {
    int tpr = 8;
    while (tpr < EMB_THREADS && tpr * 8 < a.dim) tpr *= 2;
    const int64_t per = EMB_THREADS / tpr, want = (a.n + per - 1) / per;
    hipLaunchKernelGGL(emb_fwd_kernel<T>, dim3(unsigned(want < (1 << 20) ? want : (1 << 20))),
                       dim3(EMB_THREADS), 0, s, a.tokens, a.n, static_cast<const T*>(a.W), a.ldw, a.vocab,
                       static_cast<T*>(a.Y), a.ldy, int(a.dim), a.scale, tpr);
    return hipGetLastError();
}

template <typename TY, typename TG>
hipError_t sums(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + p.off_keys[p.passes & 1]);
    const uint32_t* idx = reinterpret_cast<const uint32_t*>(ws + p.off_idx[p.passes & 1]);
    float *head = reinterpret_cast<float*>(ws + p.off_head), *tail = reinterpret_cast<float*>(ws + p.off_tail);
    TG* G = static_cast<TG*>(a.G);
    const uint32_t vocab = uint32_t(a.vocab);
    const int dim = int(a.dim);
    if (!a.accumulate)
        hipLaunchKernelGGL(emb_fill_kernel<TG>, dim3(unsigned((a.vocab + FILL_ROWS - 1) / FILL_ROWS)),
                           dim3(EMB_THREADS), 0, s, keys, a.n, G, a.ldg, vocab, dim);
    if (a.n == 0) return hipGetLastError();
    const dim3 grid(unsigned((dim + 2047) / 2048), unsigned(p.chunks));
    hipLaunchKernelGGL((emb_sum_kernel<TY, TG>), grid, dim3(EMB_THREADS), 0, s, keys, idx, a.n, p.C,
                       static_cast<const TY*>(a.dY), a.lddy, G, a.ldg, vocab, dim, a.scale, a.accumulate, head,
                       tail);
    hipLaunchKernelGGL(emb_join_kernel<TG>, grid, dim3(EMB_THREADS), 0, s, keys, a.n, p.C, G, a.ldg, vocab, dim,
                       a.scale, a.accumulate, head, tail);
    return hipGetLastError();
}

}  // namespace

hipError_t mo_launch_emb_fwd(const MoEmbArgs& a, hipStream_t s) {
    return a.w_dtype == MO_BF16 ? fwd<bf16_t>(a, s) : fwd<float>(a, s);
}

hipError_t mo_launch_emb_sort(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    uint32_t* hist = reinterpret_cast<uint32_t*>(ws + p.off_hist);
    const uint32_t vocab = uint32_t(a.vocab);
    for (int k = 0; k < p.passes; ++k) {
        // pass k reads buffer k & 1 (the first one the tokens) and writes the other
        const int64_t* tokens = k == 0 ? a.tokens : nullptr;
        const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + p.off_keys[k & 1]);
        const uint32_t* idx = reinterpret_cast<const uint32_t*>(ws + p.off_idx[k & 1]);
        uint32_t* ok = reinterpret_cast<uint32_t*>(ws + p.off_keys[~k & 1]);
        uint32_t* oi = reinterpret_cast<uint32_t*>(ws + p.off_idx[~k & 1]);
        hipLaunchKernelGGL(emb_count_kernel, dim3(p.tiles), dim3(EMB_THREADS), 0, s, tokens, keys, a.n, vocab,
                           k * p.bits, p.bits, hist);
        hipLaunchKernelGGL(emb_scan_kernel, dim3(1), dim3(1024), 0, s, hist, int64_t(p.tiles) << p.bits);
        hipLaunchKernelGGL(emb_scatter_kernel, dim3(p.tiles), dim3(EMB_THREADS), 0, s, tokens, keys, idx, a.n,
                           vocab, k * p.bits, p.bits, hist, ok, oi);
    }
    return hipGetLastError();
}

hipError_t mo_launch_emb_bwd(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    const bool yb = a.dy_dtype == MO_BF16, gb = a.g_dtype == MO_BF16;
    return yb ? (gb ? sums<bf16_t, bf16_t>(a, p, ws, s) : sums<bf16_t, float>(a, p, ws, s))
              : (gb ? sums<float, bf16_t>(a, p, ws, s) : sums<float, float>(a, p, ws, s));
}
