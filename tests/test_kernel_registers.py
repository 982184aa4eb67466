"""What the compiler made of the RMS norm's and the casts' kernels: rows live in registers, so none may be spilled
to memory."""
import os
import re
import shutil
import subprocess

import pytest

from matrix_optimizers_amd import build as B


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """{source: AMD assembly}, with the library's own options."""
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    if shutil.which("c++") is None and shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    d, out, runs = tmp_path_factory.mktemp("asm"), {}, {}
    for src in ("rms_norm.hip", "fp8_cast.hip"):
        out[src] = str(d / (src + ".s"))
        runs[src] = subprocess.Popen([cc, "-x", "hip", *B.COMMON, *B.DEVICE_ONLY, "--offload-device-only", "-S",
                                      os.path.join(B.CSRC, src), "-o", out[src]], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    for src, run in runs.items():
        text = run.communicate()[0]
        assert run.returncode == 0, text[-2000:]
    return {src: open(path).read() for src, path in out.items()}


def kernels(text):
    """(name, spilled vector registers, bytes of scratch) of every kernel."""
    found = [(re.search(r"\.name:\s+(\S+)", b).group(1), int(re.search(r"\.vgpr_spill_count:\s+(\d+)", b).group(1)),
              int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", b).group(1))) for b in text.split("\n  - .agpr_count:")[1:]]
    assert found
    return found


@pytest.mark.parametrize("src", ["rms_norm.hip", "fp8_cast.hip"])
def test_nothing_is_spilled(assembly, src):
    bad = [k for k in kernels(assembly[src]) if k[1] or k[2]]
    assert not bad, bad


def test_stores_past_the_caches_leave_whole_lines(assembly):
    """Only bf16 results of the way back from 8 bits: a lane has two stores of fp32 and one of bf16, so that fp32's
    leave every other 16 bytes of a line to the next one."""
    bodies = re.findall(r"^(\w+):.*?\n(.*?)\n\s*s_endpgm", assembly["fp8_cast.hip"], re.M | re.S)
    past = {name for name, body in bodies if re.search(r"global_store_\w+ .*\bnt\b", body)}
    assert len(bodies) >= 6 and len(past) == 1 and all("dequantize" in n and "IDF16b" in n for n in past), past
