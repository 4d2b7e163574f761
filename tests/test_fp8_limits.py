"""Sizes that splr_fp8_quantize documents pass its checks on the CPU: such a call ends at its launch, for want of a GPU."""
import os

import pytest

from tests.test_tokens_fp8_checks import HIP, SHAPE, quantize

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="the addresses are no device memory")


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols,transposed", [(1 << 24, 32, 0), (1 << 24, 1 << 12, 0), (1 << 16, 1 << 20, 0), (1, 1, 1), (1 << 20, 1 << 16, 1),
                                                  (1 << 12, 1 << 24, 1), (1, 1 << 24, 1)])
def test_documented_sizes_are_taken(rows, cols, transposed, block_rows):
    far = dict(X=1 << 40, Q=1 << 44, s=1 << 46)   # X and Q may have 2^36 entries each
    assert quantize(rows=rows, cols=cols, tr=transposed, br=block_rows, **far) == HIP
    assert quantize(rows=rows + (1 << 24), cols=cols, tr=transposed, br=block_rows, **far) == SHAPE
