"""The partial rows of the RMS norm's weight gradient, one per workgroup, by the workspace that holds them."""
import pytest

import matrix_optimizers_amd as mo


@pytest.mark.parametrize("cols,per_cu", [(1024, 4), (2048, 3), (4096, 2), (4104, 2), (5000, 2), (7168, 2), (7176, 1), (8192, 1), (16384, 1)])
def test_workgroups_per_cu(cols, per_cu):
    """Rows of two chunks that leave a CU with few wavefronts (4104 to 7168 columns) take two workgroups in bf16."""
    rows = 256 * per_cu * cols * 4
    assert rows <= mo.rms_norm_workspace_bytes(16384, cols) < rows + 1024
    assert mo.rms_norm_workspace_bytes(100, cols) < 100 * cols * 4 + 1024   # no more than there are rows
