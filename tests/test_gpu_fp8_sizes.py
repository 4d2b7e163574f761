"""The largest sizes of the quantisation to e4m3, whose tiles pass a grid's second dimension."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import codes_of, floats, quantize64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,transposed", [(65535 * 128 + 129, 32, False), (1 << 24, 32, False), (33, 65535 * 128 + 129, True),
                                                  (32, 1 << 24, True)])
def test_more_blocks_than_65535(rows, cols, transposed):
    """Blocks of 128 x 128; entries repeat, so that every block's codes and scale are those of one of three."""
    few, _ = floats((384, 32) if not transposed else (33, 384), torch.bfloat16, 1)
    long = max(rows, cols)
    X = few.repeat(-(-long // 384), 1)[:rows] if not transposed else few[:rows].repeat(1, -(-long // 384))[:, :cols].contiguous()
    Q, s = binding.fp8_quantize(X, 128, transposed=transposed)
    x64 = X[:768].double().cpu().numpy() if not transposed else X[:, :768].double().cpu().numpy().T
    codes, scales = quantize64(x64, 128)
    K = x64.shape[1]
    assert np.array_equal(codes_of(Q[:768, :K]), codes) and np.array_equal(s[:6].cpu().numpy(), scales)
    assert not Q[:, K:].view(torch.uint8).any()
    whole = long // 384 * 384
    bits = Q.view(torch.uint8)
    assert (bits[:whole].view(-1, 384, bits.shape[1]) == bits[:384]).all() and (s[:whole // 128].view(-1, 3, 1) == s[:3]).all()
    # what is left of a third of a block has a scale of its own
    tail = X[whole:] if not transposed else X[:, whole:].T
    if len(tail):
        codes, scales = quantize64(tail.double().cpu().numpy(), 128)
        assert np.array_equal(codes_of(Q[whole:, :K]), codes) and np.array_equal(s[whole // 128:].cpu().numpy(), scales)
