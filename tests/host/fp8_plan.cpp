// Prints the 8-bit products' plans (fp8.cpp, compiled here for the host), as key=value:
// one line per line of input
//   p m n k dtype block_rows_of_B offset_A offset_B pad_A scale_offset_A scales_by_columns_A
//   w tokens rows dim dy_dtype offset_dY offset_X pad_X scales_by_columns_X
// (offsets and pads in elements; everything else contiguous).  Nothing is launched.
#include <cinttypes>
#include <cstdio>

#include "fp8.cpp"

int main() {
    char what;
    while (std::scanf(" %c", &what) == 1) {
        auto at = [](int i, long long off) { return reinterpret_cast<uint8_t*>((uintptr_t(1) << 40) * i + off); };
        if (what == 'p') {
            long long m, n, k, oa, ob, pad, os;
            int dt, blk, inc;
            if (std::scanf("%lld %lld %lld %d %d %lld %lld %lld %lld %d", &m, &n, &k, &dt, &blk, &oa, &ob, &pad, &os, &inc) != 10) return 1;
            const mo_fp8_matrix A = {at(1, oa), at(2, os), m, k + pad, inc && m > 1 ? 1 : 0, inc && m > 1 ? m : 0, 1}, B = {at(3, ob), at(4, 0), n, 0, 0, 0, blk};
            MoF8Operand a, b;
            if (matmul_args(&A, &B, k, dt, &a, &b) != MO_OK) return 1;
            const MoF8Plan p = matmul_plan(a, b, k, dt);
            std::printf("small=%d values=%d nb=%d splits=%d rounds=%d copy_a=%d copy_b=%d scales_a=%d scales_b=%d bytes=%" PRIu64 "\n",
                        p.tb * 10 + p.rb, int(p.bf16), p.nb, p.splits, int(p.full / 256 + (p.full % 256 || p.splits > 1)), int(p.pack_q[0]),
                        int(p.pack_q[1]), int(p.pack_s[0]), int(p.pack_s[1]), p.bytes);
        } else {
            long long t, n, k, oy, ox, pad;
            int dt, inc;
            if (std::scanf("%lld %lld %lld %d %lld %lld %lld %d", &t, &n, &k, &dt, &oy, &ox, &pad, &inc) != 8) return 1;
            const mo_fp8_matrix X = {at(1, ox), at(2, 0), t, k + pad, inc ? 1 : 0, inc ? t : 0, 1};
            MoF8Wgrad a;
            if (wgrad_args(at(3, oy * elem_size(dt)), 0, dt, &X, k, n, &a) != MO_OK) return 1;
            const MoF8Plan p = wgrad_plan(a);
            std::printf("small=%d tokens=%d planes=%d nb=%d splits=%d rounds=%d bytes=%" PRIu64 "\n", p.tb, int(p.tokens), dt == MO_BF16 ? 1 : 3, p.nb, p.splits,
                        int(p.full / 256 + (p.full % 256 || p.splits > 1)), p.bytes);
        }
    }
    return 0;
}
