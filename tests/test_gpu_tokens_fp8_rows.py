"""Rows in e4m3 on their way to the experts: codes by tokens_dispatch, their scales by a gather of their own."""
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import floats
from tests.test_gpu_tokens import routes, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,D", [(1, 2, 4, 96), (50, 3, 6, 1056), (400, 2, 5, 256)])
def test_codes_and_scales_move(T, k, E, D):
    """Blocks of one row: quantising before the dispatch and after it gives the same codes and scales."""
    ids = routes(T, k, E, 0.2, 1)
    X, _ = floats((T, D), torch.bfloat16, 2, outliers=2)
    Q, s = binding.fp8_quantize(X)
    offsets, positions, codes = binding.tokens_dispatch(ids, E, Q)
    scales = binding.tokens_gather(s.t().contiguous(), positions).t().contiguous()
    _, _, rows = binding.tokens_dispatch(ids, E, X)
    want, want_s = binding.fp8_quantize(rows)
    n = int(offsets[-1])
    assert same_bits(codes[:n], want[:n]) and torch.equal(scales[:, :n], want_s[:, :n])
