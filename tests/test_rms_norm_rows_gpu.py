"""The RMS norm where every workgroup walks over several rows, for each way of holding a row (16, 32 and 64
threads, one chunk and two chunks per thread, whole and ragged): the checks of test_rms_norm_gpu."""
import pytest
import torch

from test_rms_norm_gpu import test_backward as backward
from test_rms_norm_gpu import test_forward as forward

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(20011, 64), (18001, 100), (9001, 200), (9001, 256), (5003, 500), (5003, 512),             # 4 to 16 rows at a time
          (4301, 520), (3001, 1000), (2051, 2048), (1301, 4096),                                     # one chunk per thread
          (1100, 4097), (1103, 4104), (1101, 5000), (1030, 7168), (1030, 7171), (1027, 7176), (600, 8192),   # two
          (601, 10000), (1102, 12001), (1100, 16384), (700, 16385)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_over_many_rows(gpu, rows, cols, dtype):
    forward(rows, cols, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward_over_many_rows(gpu, rows, cols, dtype):
    backward(rows, cols, dtype)
