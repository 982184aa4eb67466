// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   Y[i] = s W[t_i],   G[v] = s sum_{i : t_i = v} dY[i]   (or G[v] += ..)
//
// A token outside 0 .. vocab - 1 marks a padded position: its Y row is zero and
// its dY row takes no part (it may be loaded ahead and is dropped).
//
// The gradient is the transpose of the lookup.  Adding rows with atomics would
// make the sum's order, hence its last bits, change from call to call; instead
// the positions are sorted by token (stable, so equal tokens stay in position
// order), and the runs of equal tokens are summed in fp32 in that order, in chunks
// of sorted positions whose size follows from n; a run inside one chunk is written
// once, the parts of one that crosses chunks are joined in a fixed strided order.
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

// The lanes among `of` whose digit equals this lane's: one ballot per bit, kept
// where the bits agree.
MO_DEV uint64_t same_digit(uint32_t d, int bits, uint64_t of) {
    uint32_t lo = uint32_t(of), hi = uint32_t(of >> 32);
    for (int k = 0; k < bits; ++k) {
        const uint32_t mine = uint32_t(__builtin_amdgcn_sbfe(int(d), k, 1));   // 0 or all ones
        const uint64_t m = __ballot(mine != 0);
        lo &= ~(uint32_t(m) ^ mine);
        hi &= ~(uint32_t(m >> 32) ^ mine);
    }
    return uint64_t(hi) << 32 | lo;
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
        const uint64_t same = same_digit(d, bits, __ballot(on));
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

// ---- runs that cross chunks ------------------------------------------------------------

// First position with key >= v.
MO_DEV int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t v) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// A run that starts in one chunk of C positions and goes on into others.
struct Span { uint32_t key, first, last; };

// Lists the spans, in any order, and their number: one workgroup.
MO_DEV void list_spans(const uint32_t* keys, int64_t n, int C, uint32_t chunks, uint32_t vocab, Span* spans,
                       uint32_t* count, uint32_t* lds_count) {
    if (threadIdx.x == 0) *lds_count = 0;
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < chunks; c += blockDim.x) {
        const int64_t a = int64_t(c) * C, b = a + C < n ? a + C : n;
        const uint32_t k = keys[b - 1];
        if (k >= vocab || b >= n || keys[b] != k) continue;      // nothing goes on
        if (a > 0 && keys[a - 1] == k) continue;                 // started before
        const uint32_t at = atomicAdd(lds_count, 1u);
        spans[at] = Span{k, c, uint32_t((lower_bound(keys, n, k + 1) - 1) / C)};
    }
    __syncthreads();
    if (threadIdx.x == 0) *count = *lds_count;
}

__global__ __launch_bounds__(1024) void emb_spans_kernel(const uint32_t* keys, int64_t n, int C, uint32_t chunks,
                                                         uint32_t vocab, Span* spans, uint32_t* count) {
    __shared__ uint32_t lds_count;
    list_spans(keys, n, C, chunks, vocab, spans, count, &lds_count);
}

// Zeros in all of G by the first 256 threads of the workgroups first ..: flat
// where the rows are contiguous, a wavefront per row otherwise.  Few stores in
// flight that advance together keep HBM's pages open: 128 workgroups of 256
// threads write a 1.05 GB G in 161 us (6.5 TB/s), 512 to 2048 of them in 200 to 230.
constexpr int FILL_WGS = 128, FILL_THREADS = 256;
template <typename T>
MO_DEV void fill_zeros(T* G, int64_t ldg, uint32_t vocab, int dim, int first) {
    if (threadIdx.x >= FILL_THREADS) return;
    const int64_t nt = int64_t(gridDim.x - first) * FILL_THREADS;
    const int64_t t = int64_t(blockIdx.x - first) * FILL_THREADS + threadIdx.x;
    f32x8 z;
#pragma unroll
    for (int e = 0; e < 8; ++e) z.v[e] = 0.f;
    if (ldg == dim) {
        constexpr int PER = 16 / sizeof(T);
        const int64_t len = int64_t(vocab) * dim, whole = len / PER;
        for (int64_t c = t; c < whole; c += nt) *reinterpret_cast<u32x4_e2*>(G + c * PER) = u32x4{0, 0, 0, 0};
        if (t == 0) st8n(G + whole * PER, z, int(len - whole * PER));
    } else {
        for (int64_t v = t >> 6; v < vocab; v += nt >> 6)
            for (int c = (threadIdx.x & 63) * 8; c < dim; c += 512) st8n(G + v * ldg + c, z, dim - c);
    }
}

template <typename T>
__global__ __launch_bounds__(FILL_THREADS) void emb_fill_kernel(T* G, int64_t ldg, uint32_t vocab, int dim) {
    fill_zeros(G, ldg, vocab, dim, 0);
}

// ---- short lists: the whole sort in one workgroup ---------------------------------------

constexpr int ONE_THREADS = 1024, ONE_WAVES = ONE_THREADS / 64;

// Up to 1024 R positions whose key and position fit 32 bits together
// (key << idx_bits | position): each thread keeps R words in registers, a
// pass ranks them by ballots, scans the waves' digit counts and exchanges the
// words through one LDS buffer.  The words are distinct, so the order is the one
// sorted order.  Workgroup 0 sorts while the others write G's zeros: the sort
// hides behind the fill, which costs the rows with tokens a second write (at
// most as many rows as the sums read).  Zeroing only the rows without tokens,
// between the sums and after the sort, measured 345 us against 285 for the whole call
// on 16384 tokens when the sort still took six launches (224 now).
template <typename T, int R>
__global__ __launch_bounds__(ONE_THREADS) void emb_sort_fill_kernel(
    const int64_t* tokens, int64_t n, uint32_t vocab, int passes, int bits, int idx_bits, uint32_t* out_keys,
    uint32_t* out_idx, int C, uint32_t chunks, Span* spans, uint32_t* count, T* G, int64_t ldg, int dim) {
    if (blockIdx.x != 0) {
        fill_zeros(G, ldg, vocab, dim, 1);
        return;
    }
    __shared__ uint32_t buf[ONE_THREADS * R];
    __shared__ uint16_t off[ONE_WAVES][MAX_DIGITS];
    __shared__ uint32_t wsum[ONE_WAVES];
    __shared__ uint32_t lds_count;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nd = 1 << bits;
    const int base = wave * 64 * R + lane;   // word r of this thread is position base + 64 r
    uint32_t w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = base + 64 * r;
        w[r] = i < n ? (key_of(tokens, nullptr, i, vocab) << idx_bits) | uint32_t(i) : 0xFFFFFFFFu;
    }
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = idx_bits + pass * bits;
        for (int d = threadIdx.x; d < ONE_WAVES * MAX_DIGITS / 2; d += ONE_THREADS)
            reinterpret_cast<uint32_t*>(&off[0][0])[d] = 0;
        __syncthreads();
        uint16_t rank[R];   // among the wave's words of the same digit
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t d = (w[r] >> shift) & (nd - 1);
            const uint64_t same = same_digit(d, bits, ~0ull);
            const uint32_t before = off[wave][d];
            rank[r] = uint16_t(before + __popcll(same & ((1ull << lane) - 1)));
            wave_sync();
            if ((same >> lane) == 1) off[wave][d] = uint16_t(rank[r] + 1);
            wave_sync();
        }
        __syncthreads();
        // exclusive scan over (digit, wave); threads 0 .. nd - 1 hold a digit each
        uint32_t total = 0;
        if (int(threadIdx.x) < nd)
            for (int v = 0; v < ONE_WAVES; ++v) total += off[v][threadIdx.x];
        uint32_t inc = total;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t x = __shfl_up(inc, o, 64);
            if (lane >= o) inc += x;
        }
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        uint32_t run = inc - total;
        for (int v = 0; v < wave; ++v) run += wsum[v];
        if (int(threadIdx.x) < nd)
            for (int v = 0; v < ONE_WAVES; ++v) {
                const uint32_t c = off[v][threadIdx.x];
                off[v][threadIdx.x] = uint16_t(run);
                run += c;
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) buf[uint32_t(off[wave][(w[r] >> shift) & (nd - 1)]) + rank[r]] = w[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = buf[base + 64 * r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = base + 64 * r;
        if (i < n) {
            out_keys[i] = w[r] >> idx_bits;
            out_idx[i] = w[r] & ((1u << idx_bits) - 1);
        }
    }
    __threadfence_block();
    __syncthreads();
    list_spans(out_keys, n, C, chunks, vocab, spans, count, &lds_count);
}

// ---- sums over the runs -----------------------------------------------------------

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

// Threads (a power of two) of a workgroup that share a row.
inline int row_threads(int dim) {
    int tpr = 8;
    while (tpr < EMB_THREADS && tpr * 8 < dim) tpr *= 2;
    return tpr;
}

// One chunk of C sorted positions, 2048 columns.  A run inside the chunk is
// written; the part of a run that came in from the chunk before goes to
// head[chunk], the start of one that goes on to tail[chunk].  A wavefront's lanes
// hold the chunk's keys and positions (one load each), and eight rows are
// requested before the first is added.
template <typename TY, typename TG, bool FULL>
__global__ __launch_bounds__(EMB_THREADS) void emb_sum_kernel(
    const uint32_t* keys, const uint32_t* idx, int64_t n, int C, const TY* dY, int64_t lddy, TG* G, int64_t ldg,
    uint32_t vocab, int dim, float scale, int accumulate, float* head, float* tail) {
    constexpr int DEPTH = 8, BATCH = 32;
    const int slabs = (dim + 2047) / 2048, lane = threadIdx.x & 63;
    const uint32_t chunk = blockIdx.x / slabs;
    const int c = (int(blockIdx.x % slabs) * EMB_THREADS + threadIdx.x) * 8;
    const int left = dim - c;
    const int64_t a = int64_t(chunk) * C, b = a + C < n ? a + C : n;
    f32x8 sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum.v[e] = 0.f;
    bool first = true, came_in = false;
    for (int64_t p0 = a; p0 < b; p0 += BATCH) {
        // lane l: the key of position p0 - 1 + l (a value no key has outside the list)
        // and the row of position p0 + l
        const int64_t kp = p0 - 1 + lane, ip = p0 + lane < b ? p0 + lane : b - 1;
        const uint32_t kv = kp >= 0 && kp < n ? keys[kp] : 0xFFFFFFFFu;
        const uint32_t iv = idx[ip];
        if (p0 == a) came_in = __builtin_amdgcn_readlane(kv, 0) == __builtin_amdgcn_readlane(kv, 1);
        const int m = b - p0 < BATCH ? int(b - p0) : BATCH;
        for (int i0 = 0; i0 < m; i0 += DEPTH) {
            raw8<TY> x[DEPTH];
#pragma unroll
            for (int i = 0; i < DEPTH; ++i)   // behind the end: the last row again, not used
                x[i] = row8<FULL>(dY + int64_t(uint32_t(__builtin_amdgcn_readlane(iv, i0 + i))) * lddy, c, dim);
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                if (i0 + i >= m) break;
                const uint32_t k = __builtin_amdgcn_readlane(kv, i0 + i + 1);
                if (k >= vocab) return;
                const f32x8 v = widen(x[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] += v.v[e];
                const bool more = uint32_t(__builtin_amdgcn_readlane(kv, i0 + i + 2)) == k;
                if (more && p0 + i0 + i + 1 < b) continue;
                if (first && came_in) st8n(head + int64_t(chunk) * dim + c, sum, left);
                else if (more) st8n(tail + int64_t(chunk) * dim + c, sum, left);
                else put_row(G + int64_t(k) * ldg + c, sum, scale, accumulate, left);
                first = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] = 0.f;
            }
        }
    }
}

// Runs over several chunks: their parts added up.  Eight wavefronts take every
// eighth head each, 512 columns per workgroup, and are added in order; the
// workgroups walk the list of spans.
constexpr int JOIN_WAVES = 8;
template <typename TG, bool FULL>
__global__ __launch_bounds__(JOIN_WAVES * 64) void emb_join_kernel(const Span* spans, const uint32_t* count, TG* G,
                                                               int64_t ldg, int dim, float scale, int accumulate,
                                                               const float* head, const float* tail) {
    __shared__ f32x4 part[JOIN_WAVES][64][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, slabs = (dim + 511) / 512;
    const int64_t items = int64_t(*count) * slabs;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const Span sp = spans[it / slabs];
        const int c = (int(it % slabs) * 64 + lane) * 8, left = dim - c;
        f32x8 sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] = 0.f;
        if (wave == 0) sum = widen(ld8n(tail + int64_t(sp.first) * dim + c, left));
#pragma unroll 8
        for (uint32_t q = sp.first + 1 + wave; q <= sp.last; q += JOIN_WAVES) {
            const f32x8 x = widen(row8<FULL>(head + int64_t(q) * dim, c, dim));
#pragma unroll
            for (int e = 0; e < 8; ++e) sum.v[e] += x.v[e];
        }
        const raw8<float> r = narrow(sum, float());
        part[wave][lane][0] = r.lo;
        part[wave][lane][1] = r.hi;
        __syncthreads();
        if (wave == 0) {
            for (int w = 1; w < JOIN_WAVES; ++w) {
                const f32x8 x = widen(raw8<float>{part[w][lane][0], part[w][lane][1]});
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] += x.v[e];
            }
            put_row(G + int64_t(sp.key) * ldg + c, sum, scale, accumulate, left);
        }
        __syncthreads();
    }
}

template <typename T>
hipError_t fwd(const MoEmbArgs& a, hipStream_t s) {
    const int tpr = row_threads(int(a.dim));
    const int64_t per = EMB_THREADS / tpr, want = (a.n + per - 1) / per;
    hipLaunchKernelGGL(emb_fwd_kernel<T>, dim3(unsigned(want < (1 << 20) ? want : (1 << 20))),
                       dim3(EMB_THREADS), 0, s, a.tokens, a.n, static_cast<const T*>(a.W), a.ldw, a.vocab,
                       static_cast<T*>(a.Y), a.ldy, int(a.dim), a.scale, tpr);
    return hipGetLastError();
}

template <typename T>
hipError_t fill(const MoEmbArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(emb_fill_kernel<T>, dim3(FILL_WGS), dim3(FILL_THREADS), 0, s, static_cast<T*>(a.G), a.ldg,
                       uint32_t(a.vocab), int(a.dim));
    return hipGetLastError();
}

// The one-workgroup sort, with the zeros unless they are not wanted.
template <typename T>
hipError_t sort_fill(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    uint32_t* keys = reinterpret_cast<uint32_t*>(ws + p.off_keys[p.passes & 1]);
    uint32_t* idx = reinterpret_cast<uint32_t*>(ws + p.off_idx[p.passes & 1]);
    const dim3 grid(a.accumulate ? 1 : 1 + FILL_WGS), block(ONE_THREADS);
#define MO_SORT(R)                                                                                            \
    hipLaunchKernelGGL((emb_sort_fill_kernel<T, R>), grid, block, 0, s, a.tokens, a.n, uint32_t(a.vocab),     \
                       p.passes, p.bits, p.idx_bits, keys, idx, p.C, p.chunks,                                \
                       reinterpret_cast<Span*>(ws + p.off_spans), reinterpret_cast<uint32_t*>(ws + p.off_count), \
                       static_cast<T*>(a.G), a.ldg, int(a.dim))
    if (a.n <= 1024) MO_SORT(1);
    else if (a.n <= 4096) MO_SORT(4);
    else if (a.n <= 16384) MO_SORT(16);
    else MO_SORT(32);
#undef MO_SORT
    return hipGetLastError();
}

template <typename TY, typename TG, bool FULL>
hipError_t sums(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + p.off_keys[p.passes & 1]);
    const uint32_t* idx = reinterpret_cast<const uint32_t*>(ws + p.off_idx[p.passes & 1]);
    float *head = reinterpret_cast<float*>(ws + p.off_head), *tail = reinterpret_cast<float*>(ws + p.off_tail);
    TG* G = static_cast<TG*>(a.G);
    const int dim = int(a.dim);
    hipLaunchKernelGGL((emb_sum_kernel<TY, TG, FULL>), dim3(p.chunks * uint32_t((dim + 2047) / 2048)),
                       dim3(EMB_THREADS), 0, s, keys, idx, a.n, p.C, static_cast<const TY*>(a.dY), a.lddy, G, a.ldg,
                       uint32_t(a.vocab), dim, a.scale, a.accumulate, head, tail);
    if (p.chunks == 1) return hipGetLastError();   // no run crosses a chunk
    const int64_t most = int64_t(p.chunks) * ((dim + 511) / 512);
    hipLaunchKernelGGL((emb_join_kernel<TG, FULL>), dim3(unsigned(most < 1024 ? most : 1024)), dim3(JOIN_WAVES * 64), 0, s,
                       reinterpret_cast<const Span*>(ws + p.off_spans),
                       reinterpret_cast<const uint32_t*>(ws + p.off_count), G, a.ldg, dim, a.scale, a.accumulate,
                       head, tail);
    return hipGetLastError();
}

}  // namespace

hipError_t mo_launch_emb_fwd(const MoEmbArgs& a, hipStream_t s) {
    return a.w_dtype == MO_BF16 ? fwd<bf16_t>(a, s) : fwd<float>(a, s);
}

hipError_t mo_launch_emb_fill(const MoEmbArgs& a, hipStream_t s) {
    return a.g_dtype == MO_BF16 ? fill<bf16_t>(a, s) : fill<float>(a, s);
}

hipError_t mo_launch_emb_sort(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    if (p.idx_bits) return a.g_dtype == MO_BF16 ? sort_fill<bf16_t>(a, p, ws, s) : sort_fill<float>(a, p, ws, s);
    const uint32_t vocab = uint32_t(a.vocab);
    uint32_t* hist = reinterpret_cast<uint32_t*>(ws + p.off_hist);
    for (int k = 0; k < p.passes; ++k) {
        // pass k reads buffer k & 1 (the first one the tokens) and writes the other
        const int64_t* tokens = k == 0 ? a.tokens : nullptr;
        const uint32_t* ik = reinterpret_cast<const uint32_t*>(ws + p.off_keys[k & 1]);
        const uint32_t* ii = reinterpret_cast<const uint32_t*>(ws + p.off_idx[k & 1]);
        uint32_t* ok = reinterpret_cast<uint32_t*>(ws + p.off_keys[~k & 1]);
        uint32_t* oi = reinterpret_cast<uint32_t*>(ws + p.off_idx[~k & 1]);
        hipLaunchKernelGGL(emb_count_kernel, dim3(p.tiles), dim3(EMB_THREADS), 0, s, tokens, ik, a.n, vocab,
                           k * p.bits, p.bits, hist);
        hipLaunchKernelGGL(emb_scan_kernel, dim3(1), dim3(1024), 0, s, hist, int64_t(p.tiles) << p.bits);
        hipLaunchKernelGGL(emb_scatter_kernel, dim3(p.tiles), dim3(EMB_THREADS), 0, s, tokens, ik, ii, a.n,
                           vocab, k * p.bits, p.bits, hist, ok, oi);
    }
    hipLaunchKernelGGL(emb_spans_kernel, dim3(1), dim3(1024), 0, s,
                       reinterpret_cast<const uint32_t*>(ws + p.off_keys[p.passes & 1]), a.n, p.C, p.chunks, vocab,
                       reinterpret_cast<Span*>(ws + p.off_spans), reinterpret_cast<uint32_t*>(ws + p.off_count));
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.accumulate ? e : mo_launch_emb_fill(a, s);
}

template <typename TY, typename TG>
static hipError_t sums_of(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    return a.dim % 8 == 0 ? sums<TY, TG, true>(a, p, ws, s) : sums<TY, TG, false>(a, p, ws, s);
}
hipError_t mo_launch_emb_bwd(const MoEmbArgs& a, const MoEmbPlan& p, uint8_t* ws, hipStream_t s) {
    const bool yb = a.dy_dtype == MO_BF16, gb = a.g_dtype == MO_BF16;
    return yb ? (gb ? sums_of<bf16_t, bf16_t>(a, p, ws, s) : sums_of<bf16_t, float>(a, p, ws, s))
              : (gb ? sums_of<float, bf16_t>(a, p, ws, s) : sums_of<float, float>(a, p, ws, s));
}
