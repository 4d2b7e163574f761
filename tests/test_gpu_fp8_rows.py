"""Products with a scale for each row of W (w_block_rows 1, the form of a weight's gradient) on the tile kernels, against float64."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import Weight, floats, held, product64
from tests._fused import check

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def tiles(M, n_out, n_in, y_dtype, experts=None):
    """How many tiles of 128 x 128 a call by rows has; the sizes' query speaks of blocks of 128 rows, whose one other tile is 256 x 256."""
    assert binding.linear_fp8_tile(M, n_out, n_in, bf, y_dtype, experts)[0] > 16
    return -(-M // 128) * -(-n_out // 128)


@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("M,n_in,n_out,steps", [(2001, 1056, 2003, 4), (2048, 1056, 4096, 2)])
def test_nothing_of_a_call_before_reaches_the_result(M, n_in, n_out, steps, y_dtype):
    """Scales of NaN and of infinity stay in LDS behind a call that was given them: the next call gives what it gave before."""
    assert (tiles(M, n_out, n_in, y_dtype) <= 256) == (steps == 4)   # steps in LDS
    w = Weight(n_out, n_in, 1, by_row=True)
    X, x64 = floats((M, n_in), bf, 2, outliers=2)
    want, bound = product64(held(x64), w.values, y_dtype, y_dtype is bf)
    for left in (float("nan"), float("inf")):
        bad = binding.linear_fp8(X, w.W, torch.full_like(w.s, left), y_dtype=y_dtype)
        Y = binding.linear_fp8(X, w.W, w.s, y_dtype=y_dtype)
        assert not torch.isfinite(bad).any()
        check(Y, want, bound, f"after {left}")
