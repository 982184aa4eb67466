"""Weight gradients read where they lie (fp8_gemm.h, TOKENS): which of a stage's loads the buffer
descriptors let through.  The offsets and the descriptors' sizes are the source's own text.

A load is held to its descriptor by its vector offset; whether a scalar offset takes part is not
the same in every description of it (left out, or taken from the size, which wraps below zero),
so a load has to be right by both."""
import os
import re

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = open(os.path.join(os.path.dirname(HERE), "matrix_optimizers_amd", "csrc", "fp8_gemm.h")).read()


def expression(text):
    """A C expression of whole numbers as Python's."""
    text = re.sub(r"u?int(?:32|64)_t\(", "(", text)
    text = re.sub(r"\b([PQ])\.(\w+)", r"\1_\2", text)
    text = re.sub(r"\bint\(|\bint64_t\(", "(", text)
    return text.replace("/", "//")


def arguments(text, at):
    """The top-level arguments of the call whose opening parenthesis is at `at`."""
    out, depth, start = [], 0, at + 1
    for i in range(at, len(text)):
        c = text[i]
        depth += {"(": 1, ")": -1}.get(c, 0)
        if (c == "," and depth == 1) or depth == 0:
            out.append(text[start:i].strip())
            start = i + 1
        if depth == 0:
            return out
    raise AssertionError("unbalanced")


def defined(name):
    return expression(re.search(r"const uint32_t " + name + r" = (.*);", SOURCE).group(1))


def loads():
    """(descriptor, vector offset, scalar offset, bytes) of every load of a stage."""
    found = []
    for m in re.finditer(r"__builtin_amdgcn_raw_buffer_load_b(\d+)\(", SOURCE):
        rsrc, v, s, _ = arguments(SOURCE, m.end() - 1)
        found.append((rsrc, expression(v), expression(s), int(m.group(1)) // 8))
    assert sorted(f[0] for f in found) == ["rP", "rQ", "rS"]
    return found


def size_of(rsrc):
    """A descriptor's bytes: the second argument of upto(from, bytes)."""
    at = SOURCE.index(f"{rsrc} = upto(")
    return expression(arguments(SOURCE, at + len(f"{rsrc} = upto"))[1])


def test_the_offsets_are_read_as_they_are():
    assert {f[3] for f in loads()} == {16, 1}
    assert all(defined(v) for v in ("vP", "vS", "vQ"))
    assert "left = (P.tokens - t0 < 64 ? P.tokens - t0 : 64) - 1" in SOURCE


@pytest.mark.parametrize("nb", [1, 2, 4])
@pytest.mark.parametrize("pad", [0, 16, 4096])
def test_rows_behind_the_last_token_are_not_read(nb, pad):
    names = {v: compile(defined(v), v, "eval") for v in ("vP", "vS", "vQ")}
    TN, p_rows, q_rows = 64 * nb, 272, 64 * nb + 8
    base = dict(P_ld=p_rows + pad, P_rows=p_rows, P_ld_s=3 + pad, Q_ld=2 * q_rows + pad, Q_rows=q_rows,
                QCH=TN * 2 // 16, QR=512 // (TN * 2 // 16))
    for rsrc, voffset, soffset, width in loads():
        v, s, size = (compile(x, rsrc, "eval") for x in (voffset, soffset, size_of(rsrc)))
        turns = nb if rsrc == "rQ" else 2
        for tokens in (1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64):
            left = tokens - 1
            for p, q in ((0, 0), (256, TN * 2)):
                env = dict(base, left=left, p=p, q=q)
                have = eval(size, {}, env)
                assert 0 < have < 1 << 31
                row_bytes = {"rP": base["P_ld"], "rS": base["P_ld_s"], "rQ": base["Q_ld"]}[rsrc]
                there = {"rP": p_rows - p, "rS": -(-p_rows // 128) - (p >> 7), "rQ": 2 * q_rows - q}[rsrc]
                for tid in range(512):
                    e = dict(env, tid=tid)
                    e.update({n: eval(c, {}, e) for n, c in names.items()})
                    for i in range(turns):
                        e["i"] = i
                        vo, so = eval(v, {}, e), eval(s, {}, e)
                        assert 0 <= vo < 1 << 31
                        row, col = divmod(vo + so, row_bytes)
                        # by either rule: the scalar offset left out, or taken from the size
                        through = vo < have, vo < (have - so) % (1 << 32)
                        if row > left:
                            assert not any(through), (rsrc, tokens, tid, i)
                        elif col + width <= there:
                            assert all(through) and vo + so + width <= have, (rsrc, tokens, tid, i)
                        # columns behind the last may be read (gaps, the next row), inside the matrix
                        elif any(through):
                            assert vo + so + width <= have, (rsrc, tokens, tid, i)
