"""Output-head sizes chosen for the plan that the library makes of them (tile width,
pieces of the vocabulary, splits of K, copies of the operands), for the tests on
the GPU; test_head_plans.py holds the plans to what is said here, so that a change
of the planning cannot leave a path without a case."""

BF16, F32 = "bf16", "f32"

# name: (dtype, tokens, vocab, dim, forward plan, backward plan); the plans' fields are
# those of MoHeadPlan, "split" whether K is split, "many" whether there are several pieces
CASES = {
    "bf16 64": (BF16, 40, 300, 192, dict(nb=1, split=0, many=0, pack_w=0), dict(nb=1, split=0, many=0, pack_w=0)),
    "bf16 64 copied": (BF16, 40, 300, 100, dict(nb=1, split=0, pack_w=1), dict(nb=1, split=0, pack_w=1)),
    "bf16 64 split": (BF16, 40, 300, 1024, dict(nb=1, split=1, pack_w=0), dict(nb=1, split=1, pack_w=0)),
    "bf16 64 copied split pieces": (BF16, 40, 60001, 5813, dict(nb=1, many=1, pack_w=1),
                                    dict(nb=1, split=1, many=1, pack_w=1)),
    "bf16 64 pieces": (BF16, 40, 100003, 4096, dict(nb=1, pack_w=0), dict(nb=1, split=0, many=1, pack_w=0)),
    "bf16 64 one plane": (BF16, 300, 1000, 192, dict(nb=1, split=0), dict(nb=1, dt_planes=1, split=0, many=0)),
    "bf16 64 one plane split": (BF16, 300, 1000, 1024, dict(nb=1, split=1), dict(nb=1, dt_planes=1, split=1, many=0)),
    "bf16 128 few": (BF16, 100, 60001, 256, dict(nb=2, split=0), dict(nb=2, dt_planes=2, split=0, many=0)),
    "bf16 128 few split": (BF16, 65, 10001, 7354, dict(nb=2, split=1), dict(nb=2, dt_planes=2, split=1, many=0)),
    "bf16 128 few pieces": (BF16, 65, 100003, 4096, dict(nb=2), dict(nb=2, dt_planes=2, split=0, many=1)),
    "bf16 128 few split pieces": (BF16, 65, 60001, 7354, dict(nb=2), dict(nb=2, dt_planes=2, split=1, many=1)),
    "bf16 128": (BF16, 2049, 1984, 192, dict(nb=2, split=0, pack_w=0), dict(nb=2, split=0, many=0, pack_w=0)),
    "bf16 128 copied": (BF16, 205, 29746, 233, dict(nb=2, split=0, pack_w=1), dict(nb=2, split=0, pack_w=1)),
    "bf16 128 copied pieces": (BF16, 257, 100003, 2500, dict(nb=2, many=1), dict(nb=2, split=0, many=1, pack_w=1)),
    "bf16 128 split": (BF16, 1345, 1000, 4096, dict(nb=2, split=1, pack_w=0), dict(nb=2, split=1, many=0, pack_w=0)),
    "bf16 256": (BF16, 257, 32001, 2048, dict(nb=4, split=0, pack_w=0), dict(nb=4, split=0, many=0, pack_w=0)),
    "bf16 256 pieces": (BF16, 2049, 100003, 192, dict(nb=4, split=0), dict(nb=4, split=0, many=1, pack_w=0)),
    "bf16 256 copied split": (BF16, 2049, 1984, 5813, dict(nb=4, split=1), dict(nb=4, split=1, many=0, pack_w=1)),
    "bf16 256 copied split pieces": (BF16, 129, 60001, 5813, dict(nb=4, split=1, many=1),
                                     dict(nb=4, split=1, many=1, pack_w=1)),
    "f32 64": (F32, 513, 300, 100, dict(f32w=0, nb=1, split=0), dict(f32w=0, nb=1, split=0)),
    "f32 64 split": (F32, 513, 300, 192, dict(f32w=0, nb=1, split=1), dict(f32w=0, nb=1, split=1)),
    "f32 128": (F32, 2049, 1984, 100, dict(f32w=0, nb=2, split=0), dict(f32w=0, nb=2, split=0)),
    "f32 128 pieces": (F32, 513, 100003, 100, dict(f32w=0, nb=2), dict(f32w=0, nb=2, split=0, many=1)),
    "f32 128 long pieces": (F32, 513, 32001, 4096, dict(f32w=0, nb=2), dict(f32w=0, nb=2, split=0, many=1)),
    "f32 128 split": (F32, 2049, 300, 1024, dict(f32w=0, nb=2, split=1), dict(f32w=0, nb=2, split=1)),
    "f32 256": (F32, 1021, 10001, 100, dict(f32w=0, nb=4, split=0), dict(f32w=0, nb=4, split=0, many=0)),
    "f32 256 pieces": (F32, 2049, 32001, 100, dict(f32w=0, nb=4, split=0), dict(f32w=0, nb=4, split=0, many=1)),
    "f32 256 split": (F32, 1345, 1984, 2560, dict(f32w=0, nb=4, split=1), dict(f32w=0, nb=4, split=1, many=0)),
    "f32 256 split pieces": (F32, 513, 20001, 4096, dict(f32w=0), dict(f32w=0, nb=4, split=1, many=1)),
    "f32 in place": (F32, 40, 300, 100, dict(f32w=1, split=0, pack_w=0), dict(f32w=1, split=0, pack_w=0)),
    "f32 in place split": (F32, 40, 300, 192, dict(f32w=1, split=1, pack_w=0), dict(f32w=1, split=1, pack_w=0)),
    "f32 padded copy": (F32, 40, 20001, 233, dict(f32w=1, split=0, pack_w=1), dict(f32w=1, split=0, many=0, pack_w=1)),
    "f32 padded copy pieces": (F32, 40, 100003, 5813, dict(f32w=1, many=1, pack_w=1),
                               dict(f32w=1, split=0, many=1, pack_w=1)),
    "f32 padded copy split pieces": (F32, 40, 32001, 7354, dict(f32w=1, pack_w=1),
                                     dict(f32w=1, split=1, many=1, pack_w=1)),
}
