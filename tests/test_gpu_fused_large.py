"""The fused and grouped products where an operand has more than 2^31 entries. Entries are -1, 0 or 1, so every sum
is exact in float32 and Y is the same bit for bit whichever kernel makes it and in whatever order it adds: rows
repeat, and every repetition equals the product of the first one alone."""
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def ternary(*shape, to, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(to)


def layer(n_in, n_out, r, dtype, seed):
    values, meta = binding.prune24_pack(ternary(n_out, n_in, to=dtype, seed=seed))
    return (values, meta, ternary(n_out, r, to=dtype, seed=seed + 1), ternary(r, n_in, to=dtype, seed=seed + 2),
            ternary(n_out, to=dtype, seed=seed + 3))


def repeated(block, times):
    return block.repeat(times, 1)


# Y, gate and residual past 2^31 entries; X past them in the tile kernels; X past them with few outputs, where
# the few-token kernels run; the largest n_in
@pytest.mark.parametrize("times,n_in,n_out", [(300, 64, 8200), (2100, 1056, 40), (1040, 2080, 8), (3, 2 ** 20, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_repeat(times, n_in, n_out, dtype):
    block, r = 1000, 16
    assert times * block * max(n_in, n_out) > 2 ** 31
    print(f"[large] {times} x {block} rows {n_in} -> {n_out} {dtype}", flush=True)
    values, meta, U, V, bias = layer(n_in, n_out, r, dtype, seed=n_in)
    X = ternary(block, n_in, to=dtype, seed=1)
    gate, residual = ternary(block, n_out, to=BF16, seed=2), ternary(block, n_out, to=BF16, seed=3)
    want = binding.linear_fused(X, values, meta, U, V, bias=bias, activation="relu", gate=gate, residual=residual,
                                y_dtype=BF16, n_out=n_out)
    assert int((want != 0).sum()) > want.numel() // 10
    out = repeated(residual, times)   # over the residual
    binding.linear_fused(repeated(X, times), values, meta, U, V, bias=bias, activation="relu",
                         gate=repeated(gate, times), residual=out, y_dtype=BF16, n_out=n_out, out=out)
    assert all(torch.equal(y, want) for y in out.view(times, block, n_out))


@pytest.mark.parametrize("rows", [1, 20, 60])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_experts_past_32_bits(rows, dtype):
    """1024 experts' S with more than 2^31 stored values, every expert with the same number of rows (few-token and
    tiled kernels); the experts repeat every 7."""
    E, n_in, n_out, r, period = 1024, 2048, 2112, 16, 7
    assert E * n_out * n_in // 2 > 2 ** 31
    print(f"[large] {E} experts of {rows} rows {n_in} -> {n_out} {dtype}", flush=True)
    layers = [layer(n_in, n_out, r, dtype, seed=10 * i) for i in range(period)]
    stacked = []
    for k in range(5):
        t = torch.empty((E, *layers[0][k].shape), dtype=layers[0][k].dtype, device="cuda")
        for i in range(period):
            t[i::period] = layers[i][k]
        stacked.append(t)
    values, meta, U, V, bias = stacked
    X, gate = ternary(rows, n_in, to=dtype, seed=1), ternary(rows, n_out, to=F32, seed=2)
    offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) * rows
    got = binding.linear_experts(repeated(X, E), offsets, values, meta, U, V, bias=bias, gate=repeated(gate, E),
                                 n_out=n_out).view(E, rows, n_out)
    for i, (v, m, u, w, b) in enumerate(layers):
        want = binding.linear_fused(X, v, m, u, w, bias=b, gate=gate, n_out=n_out)
        assert int((want != 0).sum()) > want.numel() // 3
        assert all(torch.equal(y, want) for y in got[i::period]), i


# the largest n_out there is, in rows of S that repeat; one row to a few tiles of them
@pytest.mark.parametrize("M", [1, 30, 140])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_outputs_repeat(M, dtype):
    n_out, n_in, r, times = 2 ** 21, 96, 16, 2 ** 13
    block = n_out // times
    print(f"[large] {M} rows {n_in} -> {n_out} {dtype}", flush=True)
    values, meta, U, V, bias = layer(n_in, block, r, dtype, seed=5)
    X, gate = ternary(M, n_in, to=dtype, seed=1), ternary(M, block, to=F32, seed=2)
    want = binding.linear_fused(X, values, meta, U, V, bias=bias, gate=gate)
    got = binding.linear_fused(X, values.repeat(times, 1, 1, 1), meta.repeat(times, 1, 1, 1), repeated(U, times), V,
                               bias=bias.repeat(times), gate=gate.repeat(1, times))
    assert int((want != 0).sum()) > want.numel() // 3
    assert torch.equal(got.view(M, times, block), want[:, None].expand(-1, times, -1))


def test_more_tiles_than_a_launch_takes():
    """512 experts of 2^21 outputs: the tile kernels' grids would pass the dispatch limits, so the few-token kernel runs.
    Every expert has the same S, and its rows repeat."""
    E, n_in, block, times, M = 512, 64, 256, 2 ** 13, 600
    print(f"[large] {E} experts {M} rows {n_in} -> {block * times}", flush=True)
    torch.cuda.empty_cache()
    v, m, _, _, bias = layer(n_in, block, 16, BF16, seed=5)
    values = torch.empty((E * times, *v.shape), dtype=v.dtype, device="cuda").copy_(v).view(E, times * v.shape[0], *v.shape[1:])
    meta = torch.empty((E * times, *m.shape), dtype=m.dtype, device="cuda").copy_(m).view(E, times * m.shape[0], *m.shape[1:])
    X = ternary(M, n_in, to=BF16, seed=1)
    ends = torch.linspace(0, M, E + 1).int().cuda()
    got = binding.linear_experts(X, ends, values, meta, None, None, bias=bias.repeat(E, times), y_dtype=BF16)
    want = binding.linear_fused(X, v, m, None, None, bias=bias, y_dtype=BF16)
    assert int((want != 0).sum()) > want.numel() // 3
    assert torch.equal(got.view(M, times, block), want[:, None].expand(-1, times, -1))
    del values, meta, got
    torch.cuda.empty_cache()
