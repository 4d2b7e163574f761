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


@pytest.mark.parametrize("n_in,n_out", [(64, 40), (96, 203)])
def test_expert_weight_gradients_from_host_offsets(n_in, n_out):
    """An expert's dW takes its rows by offsets that the host knows; rows whose start is not 16-byte aligned have to be copied."""
    ends, dtype = [0, 37, 37, 150, 301], bf
    dY, y64 = floats((301, n_out), dtype, 3, std=1e-3)
    X, x64 = floats((301, n_in), dtype, 4, outliers=2)
    for a, b in zip(ends, ends[1:]):
        if a == b:
            with pytest.raises(binding.SplrError, match="SPLR_ERR_(SHAPE|NULL)"):   # no rows, no product: this dW is 0
                binding.fp8_quantize(dY[a:b], transposed=True)
            continue
        part = dY[a:b]
        if part.data_ptr() % 16:
            with pytest.raises(binding.SplrError, match="SPLR_ERR_ALIGN"):
                binding.fp8_quantize(part, transposed=True)
            part = part.clone()
        dq, ds = binding.fp8_quantize(part, transposed=True)
        xq, xs = binding.fp8_quantize(X[a:b], transposed=True)
        want, bound = product64(held(y64[a:b].T), held(x64[a:b].T), f32, False)
        check(binding.linear_fp8(dq, xq, xs, x_scales=ds), want, bound, f"rows {a} .. {b}")


@pytest.mark.parametrize("M,n_in,n_out", [(777, 515, 2050), (400, 1600, 1003)])
def test_weight_gradient_on_tiles(M, n_in, n_out):
    """dW = dY^T X at sizes that the tile kernels take, with scales as far apart as tokens' gradients and outlier channels make them."""
    spread_of = torch.exp2(torch.arange(n_out, device="cuda") % 13 - 6.0)
    dY, _ = floats((M, n_out), f32, 5, std=1e-3)
    dY = (dY * spread_of).to(bf)
    X, x64 = floats((M, n_in), bf, 6, outliers=8)
    dq, ds = binding.fp8_quantize(dY, transposed=True)
    xq, xs = binding.fp8_quantize(X, transposed=True)
    for y_dtype in (f32, bf):
        assert binding.linear_fp8_tile(n_out, n_in, dq.shape[1], dq.dtype, y_dtype) == (128, 128)
        want, bound = product64(held(dY.double().cpu().numpy().T), held(x64.T), y_dtype, y_dtype is bf)
        check(binding.linear_fp8(dq, xq, xs, x_scales=ds, y_dtype=y_dtype), want, bound, f"dW {y_dtype}")
