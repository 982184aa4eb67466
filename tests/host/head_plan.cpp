// Prints the output head's plans (head_plan of operators.cpp, compiled here for the
// host): one line per line of input
//   tokens vocab dim dtype backward k ld_h ld_w h_offset w_offset
// (strides and offsets in elements, 0 = contiguous and aligned), as key=value.
// Nothing is launched: the kernels' launchers stay unresolved.
#include <cinttypes>
#include <cstdio>

#include "operators.cpp"

int main() {
    long long n, v, d, ldh, ldw, oh, ow;
    int dt, back, k;
    while (std::scanf("%lld %lld %lld %d %d %d %lld %lld %lld %lld", &n, &v, &d, &dt, &back, &k, &ldh, &ldw, &oh, &ow) == 10) {
        const int es = dt == MO_BF16 ? 2 : 4;
        mo_head h = {};
        h.H = reinterpret_cast<const void*>((uintptr_t(1) << 44) + oh * es);
        h.W = reinterpret_cast<const void*>((uintptr_t(1) << 45) + ow * es);
        h.tokens = n;
        h.vocab = v;
        h.dim = d;
        h.ld_h = ldh;
        h.ld_w = ldw;
        h.dtype = dt;
        Targets t = label_targets(nullptr);
        t.k = k;
        MoHeadArgs a;
        const mo_status st = head_args(&h, &t, &a);
        if (st != MO_OK) {
            std::printf("status=%d\n", int(st));
            continue;
        }
        const MoHeadPlan p = head_plan(a, back != 0, true, true);
        std::printf("status=0 planes=%d dt_planes=%d f32w=%d nb=%d nb_dw=%d n_pad=%" PRId64 " kd=%" PRId64 " pack_h=%d pack_w=%d piece=%" PRId64
                    " pieces=%" PRId64 " z_stages=%d z_splits=%d dw_splits=%d dh_splits=%d dh_tm=%u dh_tn=%u bytes=%" PRIu64 "\n",
                    p.planes, p.dt_planes, int(p.f32w), p.nb, p.nb_dw, p.n_pad, p.kd, int(p.pack_h), int(p.pack_w), p.piece,
                    (a.vocab + p.piece - 1) / p.piece, p.z_stages, p.z_splits, p.dw_splits, p.dh_splits, p.dh_tm, p.dh_tn,
                    p.bytes);
    }
    return 0;
}
