"""Layer norm of rows without elements: no output is left as the allocator gave it."""
import pytest
import torch

import matrix_optimizers_amd as mo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", [False, True])
def test_rows_of_no_columns_have_no_mean(gpu, stream):
    rows = 1000
    old = [torch.full((rows,), 7.0, device="cuda") for _ in range(4)]   # what the allocator hands out next
    torch.cuda.synchronize()
    del old
    x = torch.zeros(rows, 0, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream() if stream else None
    y, mean, rstd = mo.layer_norm_forward(x, stream=s)
    given = mo.layer_norm_forward(x, mean=torch.ones(rows, device="cuda"), rstd=torch.ones(rows, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == (rows, 0)
    for t in (mean, rstd, *given[1:]):
        assert t.shape == (rows,) and bool(torch.isnan(t).all())
    dx, dw, db = mo.layer_norm_backward(y, x, mean, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (rows, 0) and dw.shape == db.shape == (0,)
