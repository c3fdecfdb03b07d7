"""GPU tests of the layer norm where a warp takes a row: enough rows for that, and rows that end inside a lane's last
vector, one column count for each count of vectors per lane."""
import pytest
import torch

import test_norm_gpu as norm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# columns: 1, 33, 65, 97, 129, 193, 257, 321 and 385 vectors of 16 bytes (1, 2, 3, 4, 6, 8, 10, 12, 16 per lane)
VECS = (1, 33, 65, 97, 129, 193, 257, 321, 385)


@pytest.mark.parametrize("vecs", VECS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_that_end_inside_a_vector(vecs, dtype):
    norm.test_forward_and_backward(1300, vecs * (8 if dtype == BF else 4), dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_in_place_without_parameters_and_statistics(dtype):
    x, _, _, _ = norm.inputs(1300, 520, dtype, 7)
    y, _, _ = norm.ss.ss_norm_fwd(x)
    z = x.clone()
    out, mean, rstd = norm.ss.ss_norm_fwd(z, y=z, stats=False, sync_check=True)
    assert out is z and torch.equal(z, y) and mean is None and rstd is None
