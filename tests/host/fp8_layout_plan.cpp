// Prints the 8-bit products' plans (fp8.cpp, compiled here for the host) for operands of any
// layout, as key=value: one line per line of input
//   p m n k dtype <A> <B>       (rows of A, rows of B, K)
//   w tokens rows dim dy_dtype offset_dY ld_dY <X>
// <matrix>: offset ld offset_scales ld_scales inc_scales block_rows; offsets in bytes, strides in
// elements.  Nothing is launched.
#include <cinttypes>
#include <cstdio>

#include "fp8.cpp"

static uint8_t* at(int i, long long off) { return reinterpret_cast<uint8_t*>((uintptr_t(1) << 40) * i + off); }

static bool matrix(int i, long long rows, mo_fp8_matrix* m) {
    long long off, ld, soff, lds, inc;
    int blk;
    if (std::scanf("%lld %lld %lld %lld %lld %d", &off, &ld, &soff, &lds, &inc, &blk) != 6) return false;
    *m = {at(i, off), at(i + 1, soff), rows, ld, lds, inc, blk};
    return true;
}

int main() {
    char what;
    while (std::scanf(" %c", &what) == 1) {
        int dt;
        MoF8Plan p;
        if (what == 'p') {
            long long m, n, k;
            mo_fp8_matrix A, B;
            if (std::scanf("%lld %lld %lld %d", &m, &n, &k, &dt) != 4 || !matrix(1, m, &A) || !matrix(3, n, &B)) return 1;
            MoF8Operand a, b;
            if (matmul_args(&A, &B, k, dt, &a, &b) != MO_OK) return 2;
            p = matmul_plan(a, b, k, dt);
            std::printf("values=%d copy_a=%d copy_b=%d scales_a=%d scales_b=%d ", int(p.bf16), int(p.pack_q[0]), int(p.pack_q[1]),
                        int(p.pack_s[0]), int(p.pack_s[1]));
        } else {
            long long t, n, k, oy, ldy;
            mo_fp8_matrix X;
            if (std::scanf("%lld %lld %lld %d %lld %lld", &t, &n, &k, &dt, &oy, &ldy) != 6 || !matrix(1, t, &X)) return 1;
            MoF8Wgrad a;
            if (wgrad_args(at(5, oy), ldy, dt, &X, k, n, &a) != MO_OK) return 2;
            p = wgrad_plan(a);
            std::printf("tokens=%d planes=%d ", int(p.tokens), dt == MO_BF16 ? 1 : 3);
        }
        std::printf("small=%d nb=%d split=%d many=%d\n", p.tb, p.nb, int(p.splits > 1),
                    int(p.full / 256 + (p.full % 256 || p.splits > 1)) > 1);
    }
    return 0;
}
