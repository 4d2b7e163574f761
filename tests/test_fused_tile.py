"""splr_linear_fused_tile: the sizes that the GPU tests name for a kernel take that kernel."""
import ctypes

import pytest

from sparse_rank_linear_prune24_amd import binding
from tests._paths import BF16, F32, IDS, SIZES

OK, NULL, SHAPE = 0, 1, 2


@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_sizes_take_their_kernel(size):
    dtype, experts, tile, M, n_in, n_out, r = size
    assert binding.fused_tile(M, n_out, n_in, r, dtype, experts) == tile


def test_every_kernel_has_sizes():
    few = {(16, 16), (16, 32)}
    for dtype, tiles in ((F32, few | {(128, 64)}), (BF16, few | {(32, 16), (32, 32), (128, 64), (256, 128), (512, 128)})):
        for experts in (None, 4):
            assert {s[2] for s in SIZES if s[0] == dtype and s[1] == experts} == tiles


def test_refusals():
    f, a, b = binding.lib().splr_linear_fused_tile, ctypes.c_int32(), ctypes.c_int32()
    p, q = ctypes.byref(a), ctypes.byref(b)
    assert f(16, 0, 64, 64, 16, 1, p, q) == OK and f(16, 1, 64, 64, 16, 1, p, q) == OK
    assert f(16, 0, 64, 64, 16, 1, None, q) == NULL and f(16, 0, 64, 64, 16, 1, p, None) == NULL
    for bad in ((0, 0, 64, 64, 16, 1), (16, -1, 64, 64, 16, 1), (16, 1025, 64, 64, 16, 1), (16, 0, 0, 64, 16, 1),
                (16, 0, 64, 48, 16, 1), (16, 0, 64, 64, 8, 1), (16, 0, 64, 64, 16, 2), (16, 0, (1 << 21) + 1, 64, 16, 1)):
        assert f(*bad, p, q) == SHAPE, bad
    with pytest.raises(binding.SplrError, match="SPLR_ERR_SHAPE"):
        binding.fused_tile(0, 64, 64, 16, BF16)
