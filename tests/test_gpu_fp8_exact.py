"""The products with 8-bit weights on operands whose sums float32 holds exactly, so that every kernel has to give the result
itself: a lost, doubled or misplaced product, scale, row or column shows as such.

Entries are -2 .. 2 and scales 1, 2 or 4, drawn for every block of every row, so that sums are whole numbers below 4096 x 4 x 16
= 2^18. Products lie within a factor of four of each other, so the 8-bit matrix instructions drop none either. A bfloat16 Y is the
exact result rounded once.
"""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import E4M3
from tests.test_gpu_fp8 import offsets_of

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64

# M, n_in, n_out
SIZES = [(1, 4096, 520), (2, 32, 1), (16, 2048, 1024), (33, 512, 1003), (250, 1056, 4090), (700, 1056, 2003), (1300, 288, 4099),
         (2048, 1056, 4096), (3000, 512, 4500), (1025, 4096, 129)]
# rows, experts, n_in, n_out
EXPERTS = [(64, 32, 2048, 1024), (100, 60, 96, 203), (1000, 3, 1056, 1003), (2500, 4, 1056, 1003), (5000, 3, 1056, 2003), (4100, 1, 160, 2052)]


class Drawn:
    """Whole numbers, a scale for each block of `block_rows` x 128, and their codes. head: what the first columns of every block
    are; 448 in a row makes the scales that its quantisation finds the drawn ones, and meets zeros in the other operand."""

    def __init__(self, n, K, seed, block_rows=1, head=()):
        g = torch.Generator(device="cuda").manual_seed(seed)
        KB, NB = -(-K // 128), -(-n // block_rows)
        q = torch.randint(-2, 3, (n, K), generator=g, device="cuda").float()
        for i, value in enumerate(head):
            q[:, i::128] = value
        s = torch.exp2(torch.randint(0, 3, (NB, KB), generator=g, device="cuda").float())
        self.codes = q.to(E4M3)
        self.values = (q * s.repeat_interleave(block_rows, 0)[:n].repeat_interleave(128, 1)[:, :K]).double()
        self.scales = s.t().contiguous() if block_rows == 1 else s


def whole(shape, lo, hi, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)


def same(Y, want, tag):
    want = want.to(f32).to(Y.dtype)
    wrong = (Y != want).nonzero()
    assert not len(wrong), f"{tag}: {len(wrong)} entries, the first {wrong[0].tolist()}"


def test_sizes_take_every_kernel():
    for y_dtype in (bf, f32):
        want = {(16, 16), (16, 32), (128, 128)} | ({(256, 256)} if y_dtype is bf else set())
        assert {binding.linear_fp8_tile(M, n_out, n_in, E4M3, y_dtype) for M, n_in, n_out in SIZES} == want
        assert {binding.linear_fp8_tile(M, n_out, n_in, E4M3, y_dtype, E) for M, E, n_in, n_out in EXPERTS} >= want - {(16, 32)}


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("M,n_in,n_out", SIZES)
def test_linear(M, n_in, n_out, y_dtype, block_rows):
    w, x = Drawn(n_out, n_in, 1, block_rows), Drawn(M, n_in, 2)
    want = x.values @ w.values.T
    same(binding.linear_fp8(x.codes, w.codes, w.scales, x_scales=x.scales, y_dtype=y_dtype), want, "codes")
    bias, gate, residual = whole((n_out,), -9, 9, y_dtype, 3), whole((M, n_out), -2, 2, y_dtype, 4), whole((M, n_out), -200, 200, y_dtype, 5)
    Y = binding.linear_fp8(x.codes, w.codes, w.scales, x_scales=x.scales, y_dtype=y_dtype, bias=bias, activation="relu", gate=gate,
                           residual=residual)
    same(Y, (want + bias.double()).clamp(min=0) * gate.double() + residual.double(), "epilogue")
    # quantised by the call
    w, x = Drawn(n_out, n_in, 6, block_rows, head=(0.0,)), Drawn(M, n_in, 7, head=(448.0,))
    for dtype in (bf, f32):
        X = x.values.to(dtype)
        assert torch.equal(X.double(), x.values)
        same(binding.linear_fp8(X, w.codes, w.scales, y_dtype=y_dtype), x.values @ w.values.T, f"quantised from {dtype}")


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("rows,E,n_in,n_out", EXPERTS)
def test_experts(rows, E, n_in, n_out, y_dtype, block_rows):
    ws = [Drawn(n_out, n_in, 10 + e, block_rows, head=(0.0,)) for e in range(E)]
    W = torch.stack([w.codes.view(torch.uint8) for w in ws]).view(E4M3)
    s = torch.stack([w.scales for w in ws])
    ends = offsets_of(rows, E, 8, 3, 5)
    offsets = torch.from_numpy(ends).to(torch.int32).cuda()
    bias, gate = whole((E, n_out), -9, 9, y_dtype, 9), whole((rows, n_out), -2, 2, y_dtype, 10)
    x = Drawn(rows, n_in, 11, head=(448.0,))
    want = torch.full((rows, n_out), 55.0, dtype=f64, device="cuda")
    for e in range(E):
        r = slice(int(ends[e]), int(ends[e + 1]))
        want[r] = (x.values[r] @ ws[e].values.T + bias[e].double()) * gate[r].double()
    for X, xs in ((x.codes, x.scales), (x.values.to(bf), None)):
        out = torch.full((rows, n_out), 55.0, dtype=y_dtype, device="cuda")
        same(binding.linear_fp8_experts(X, offsets, W, s, x_scales=xs, bias=bias, gate=gate, y_dtype=y_dtype, out=out), want,
             "codes" if xs is not None else "quantised")


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,n_in,n_out,y_dtype", [(12600, 288, 4099, bf), (6301, 288, 4099, f32), (12601, 96, 4098, bf), (6300, 96, 4097, f32)])
def test_stores_past_the_caches_of_odd_rows(M, n_in, n_out, y_dtype, block_rows):
    """Y of more than 96 MiB goes past the caches, four entries at a time, here from any entry on."""
    assert M * n_out * (2 if y_dtype is bf else 4) > 96 << 20 and binding.linear_fp8_tile(M, n_out, n_in, E4M3, y_dtype)[0] >= 128
    w, x = Drawn(n_out, n_in, 20, block_rows), Drawn(M, n_in, 21)
    gate, residual = whole((M, n_out), -2, 2, y_dtype, 22), whole((M, n_out), -200, 200, y_dtype, 23)
    want = x.values @ w.values.T * gate.double() + residual.double()
    room = torch.full((M * n_out + 64,), 77.0, dtype=y_dtype, device="cuda")
    out = room[:M * n_out].view(M, n_out)
    same(binding.linear_fp8(x.codes, w.codes, w.scales, x_scales=x.scales, y_dtype=y_dtype, gate=gate, residual=residual, out=out), want, "Y")
    assert (room[M * n_out:] == 77.0).all()
    offsets = torch.tensor([0, 1000, M - 7], dtype=torch.int32, device="cuda")
    out.fill_(55.0)
    binding.linear_fp8_experts(x.codes, offsets, torch.stack([w.codes.view(torch.uint8)] * 2).view(E4M3), torch.stack([w.scales] * 2),
                               x_scales=x.scales, y_dtype=y_dtype, gate=gate, residual=residual, out=out)
    want[M - 7:] = 55.0
    same(out, want, "by expert")
    assert (room[M * n_out:] == 77.0).all()


@pytest.mark.parametrize("M,n_in,n_out", [(64, 1003, 40), (2100, 515, 2050), (700, 2048, 1056), (1500, 4096, 1003)])
@pytest.mark.parametrize("y_dtype", [bf, f32])
def test_weight_gradient(M, n_in, n_out, y_dtype):
    """dW = dY^T X, both sides quantised transposed. Every block of tokens has 448 in its first row of dY and in its second of X,
    which makes their scales the drawn ones, and zeros in the other's."""
    dy, x = Drawn(n_out, M, 30, head=(448.0, 0.0)), Drawn(n_in, M, 31, head=(0.0, 448.0))
    dY, X = dy.values.T.contiguous().to(bf), x.values.T.contiguous().to(bf)
    assert M % 128 > 1 and torch.equal(dY.double().T, dy.values) and torch.equal(X.double().T, x.values)
    dq, ds = binding.fp8_quantize(dY, transposed=True)
    xq, xs = binding.fp8_quantize(X, transposed=True)
    assert torch.equal(ds, dy.scales) and torch.equal(xs, x.scales)
    same(binding.linear_fp8(dq, xq, xs, x_scales=ds, y_dtype=y_dtype), dy.values @ x.values.T, "dW")
