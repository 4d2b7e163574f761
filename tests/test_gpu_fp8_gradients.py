"""The gradients of the product with 8-bit weights (products of the same kind) on the GPU, against float64: dX for every n_out."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import floats, from_code, held, product64, quantize64, spread
from tests._fused import check

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def narrow(M, n_out, n_in, dtype, y_dtype):
    """Whether these sizes run on the 8-bit matrix instructions."""
    return y_dtype is bf and binding.linear_fp8_tile(M, n_out, n_in, dtype, y_dtype)[0] > 16


@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("M,n_in,n_out", [(1, 64, 1), (77, 160, 203), (300, 256, 1003), (700, 2048, 1003), (2100, 4096, 515)])
def test_rows_gradient_of_any_width(M, n_in, n_out, dtype, y_dtype):
    """dX = dY W where n_out is no multiple of 32: with dY's rows padded by zeros to the transposed weight's length."""
    W, W64 = floats((n_out, n_in), f32, 1, std=0.02)
    Wt, wt_s = binding.fp8_quantize(W, 128, transposed=True)
    codes, scales = quantize64(W64, 128)
    w = from_code(codes) * spread(scales, n_out, n_in, False)
    dY, _ = floats((M, n_out), dtype, 2, std=1e-3)
    with pytest.raises(ValueError):                      # not of the weight's length
        binding.linear_fp8(dY, Wt, wt_s, y_dtype=y_dtype)
    with pytest.raises(binding.SplrError, match="SPLR_ERR_SHAPE"):
        binding.fp8_quantize(dY)
    padded = torch.nn.functional.pad(dY, (0, -n_out % 32))
    assert padded.shape[1] == Wt.shape[1]
    x = held(padded.double().cpu().numpy())
    want, bound = product64(x, np.pad(w, ((0, -n_out % 32), (0, 0))).T, y_dtype, narrow(M, n_in, padded.shape[1], dtype, y_dtype))
    check(binding.linear_fp8(padded, Wt, wt_s, y_dtype=y_dtype), want, bound, "dX")
    q, s = binding.fp8_quantize(padded)                  # quantised once, for several products
    check(binding.linear_fp8(q, Wt, wt_s, x_scales=s, y_dtype=y_dtype), want, bound, "dX of codes")
