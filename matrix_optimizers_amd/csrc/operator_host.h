// Shared by the entry points of the operators (operators.cpp, fp8.cpp): argument
// checks, the aliasing check of one call and the workspace's regions.
#pragma once

#include "../../include/mo.h"
#include "host_common.h"
#include "mo_worklist.h"
#include "operators.h"

#define MO_TRY(x)                          \
    do {                                   \
        const mo_status st_ = (x);         \
        if (st_ != MO_OK) return st_;      \
    } while (0)
#define MO_RUN(phase, launch)                                                              \
    do {                                                                                   \
        if (timed_launch(phase, s, [&] { return launch; }) != hipSuccess) return MO_ERR_HIP; \
    } while (0)

namespace mo_host {

// Row strides up to 2^26 elements: byte ranges stay far inside 63 bits.
constexpr int64_t kMaxLd = int64_t(1) << 26;

// The stride in elements (0 means the row length).
inline mo_status stride_of(int64_t ld, int64_t cols, int64_t* out) {
    *out = ld ? ld : cols;
    if (*out < cols) return MO_ERR_INVALID_ARG;
    return *out > kMaxLd ? MO_ERR_UNSUPPORTED : MO_OK;
}

inline bool dtype_ok(int32_t d) { return d == MO_F32 || d == MO_BF16; }

inline Range vec_range(const void* p, int64_t n, int64_t es, int writable) { return matrix_range(p, 1, n, n, es, writable); }

// The ranges of one call, at most ten: no allocation, so no exception can reach the
// C entry points.
struct Ranges {
    Range r[12];
    int n = 0;
    void add(const Range& x) { r[n++] = x; }
    // Any overlap between a writable range and any other?
    bool conflict() const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((r[i].writable || r[j].writable) && r[i].lo < r[j].hi && r[j].lo < r[i].hi) return true;
        return false;
    }
};

// The workspace as a range and its aligned base; false when it is too small.
inline bool take_workspace(void* workspace, size_t have, uint64_t need, Ranges* ranges, uint8_t** base) {
    if (need == 0) {
        *base = nullptr;
        return true;
    }
    if (!workspace || have < need + MO_WS_ALIGN) return false;
    const uintptr_t w = reinterpret_cast<uintptr_t>(workspace);
    ranges->add(Range{w, w + have, 1});
    *base = reinterpret_cast<uint8_t*>(align_up(w, MO_WS_ALIGN));
    return true;
}

// Consecutive 256-byte aligned regions.
struct Carve {
    uint64_t at = 0;
    uint64_t operator()(uint64_t bytes) {
        const uint64_t o = at;
        at = align_up(at + bytes, MO_WS_ALIGN);
        return o;
    }
};

// Zeros in a rows x cols matrix.
inline mo_status zero_rows(void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, int phase, hipStream_t s) {
    MoEmbArgs e = {};
    e.G = p;
    e.vocab = rows;
    e.dim = cols;
    e.ldg = ld;
    e.g_dtype = dtype;
    MO_RUN(phase, mo_launch_emb_fill(e, s));
    return MO_OK;
}

}  // namespace mo_host
