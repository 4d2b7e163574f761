"""Quantisation to e4m3 and the products with 8-bit weights (splr_fp8_quantize, splr_linear_fp8, splr_linear_fp8_experts) on
the GPU, against float64."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests import _fp8
from tests._fp8 import E4M3, Weight, codes_of, dev_codes, floats, from_code, held, product64, quantize64, spread
from tests._fused import ACTS, check

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def special(shape, dtype, seed):
    """Entries with zeros, a block of zeros, infinities, NaN, and the smallest and largest magnitudes in places."""
    t, _ = floats(shape, f32, seed)
    t = t.cpu()
    n, K = shape
    g = torch.Generator().manual_seed(seed)
    for value in (0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e-42, -2e-38, 3e38, 448.0, 1e-30):
        for _ in range(max(1, n // 40)):
            t[int(torch.randint(n, (1,), generator=g)), int(torch.randint(K, (1,), generator=g))] = value
    t[n // 2] = 0.0
    t[n // 3] *= 1e-37
    t = t.to(dtype)
    return t.cuda(), t.double().numpy()


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (130, 160), (257, 1056), (64, 4096)])
def test_quantize(rows, cols, dtype):
    for X, x64 in (floats((rows, cols), dtype, 1, outliers=2), special((rows, cols), dtype, 2)):
        for block_rows in (1, 128):
            Q, s = binding.fp8_quantize(X, block_rows)
            codes, scales = quantize64(x64, block_rows)
            assert np.array_equal(s.cpu().numpy(), scales)
            assert np.array_equal(codes_of(Q), codes)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (31, 3), (33, 130), (128, 64), (257, 1003), (300, 256)])
def test_quantize_transposed(rows, cols, dtype):
    pitch = (rows + 31) // 32 * 32
    for X, x64 in (floats((rows, cols), dtype, 3, outliers=1), special((rows, cols), dtype, 4)):
        for block_rows in (1, 128):
            Q, s = binding.fp8_quantize(X, block_rows, transposed=True)
            codes, scales = quantize64(x64.T, block_rows)
            assert Q.shape == (cols, pitch)
            assert np.array_equal(s.cpu().numpy(), scales)
            assert np.array_equal(codes_of(Q)[:, :rows], codes) and not codes_of(Q)[:, rows:].any()


def test_every_rounding():
    """All float32 values next to the borders between e4m3 values, and the middles themselves, in a block whose scale is 1."""
    mid = _fp8.MIDDLES
    v = np.concatenate([mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)), np.nextafter(mid.astype(np.float32), np.float32(0)),
                        _fp8.VALUES]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = np.concatenate([v, np.zeros(-len(v) % 127, np.float32)]).reshape(-1, 127)
    v = np.concatenate([v, np.full((len(v), 1), 448.0, np.float32)], 1)
    Q, s = binding.fp8_quantize(torch.from_numpy(v).cuda())
    assert (s.cpu().numpy() == 1.0).all()
    assert np.array_equal(codes_of(Q), _fp8.to_code(v.astype(np.float64)))


# M, n_in, n_out
SIZES = [(1, 32, 1), (1, 4096, 4096), (2, 96, 203), (13, 1056, 203), (16, 2048, 1024), (17, 160, 130), (33, 512, 1003), (64, 1056, 520),
         (100, 2080, 1003), (250, 1056, 4090), (256, 4096, 1024), (333, 1056, 1003), (700, 992, 2050), (1000, 4096, 2048),
         (1100, 288, 4096), (2100, 544, 4096), (3000, 512, 4500)]


def narrow(M, n_out, n_in, dtype, y_dtype, experts=None):
    """Whether these sizes may run on the 8-bit matrix instructions."""
    return y_dtype is bf and binding.linear_fp8_tile(M, n_out, n_in, dtype, y_dtype, experts)[0] > 32


@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("dtype", [bf, f32, E4M3])
@pytest.mark.parametrize("M,n_in,n_out", SIZES)
def test_linear(M, n_in, n_out, dtype, y_dtype):
    w = Weight(n_out, n_in, 5)
    X, x64 = floats((M, n_in), bf if dtype is E4M3 else dtype, 6, outliers=2)
    scales = None
    if dtype is E4M3:
        X, scales = binding.fp8_quantize(X)
    want, bound = product64(held(x64), w.values, y_dtype, narrow(M, n_out, n_in, dtype, y_dtype))
    Y = binding.linear_fp8(X, w.W, w.s, x_scales=scales, y_dtype=y_dtype)
    check(Y, want, bound, f"{M} {n_in} {n_out}")
    assert torch.equal(Y, binding.linear_fp8(X, w.W, w.s, x_scales=scales, y_dtype=y_dtype))


@pytest.mark.parametrize("M,n_in,n_out", [(5, 160, 203), (48, 512, 516), (300, 1056, 1003), (600, 512, 2048), (2100, 544, 4098)])
@pytest.mark.parametrize("y_dtype", [bf, f32])
def test_epilogue(M, n_in, n_out, y_dtype):
    w = Weight(n_out, n_in, 7, std=0.2)
    X, x64 = floats((M, n_in), bf, 8)
    x64 = held(x64)
    bias, b64 = floats((n_out,), y_dtype, 9)
    gate, g64 = floats((M, n_out), y_dtype, 10)
    residual, r64 = floats((M, n_out), y_dtype, 11)
    thin = narrow(M, n_out, n_in, bf, y_dtype)
    for i, act in enumerate(ACTS):
        kw, kw64 = {}, {}
        for bit, name, t, t64 in ((1, "bias", bias, b64), (2, "gate", gate, g64), (4, "residual", residual, r64)):
            if (i + 3) & bit:
                kw[name], kw64[name] = t, t64
        want, bound = product64(x64, w.values, y_dtype, thin, act=act, **kw64)
        Y = binding.linear_fp8(X, w.W, w.s, activation=act, y_dtype=y_dtype, **kw)
        check(Y, want, bound, f"{act} {sorted(kw)}")
        for name in ("gate", "residual"):           # in place
            if name in kw:
                out = kw[name].clone()
                binding.linear_fp8(X, w.W, w.s, activation=act, y_dtype=y_dtype, out=out, **dict(kw, **{name: out}))
                assert torch.equal(out, Y), name


# rows, experts, n_in, n_out
EXPERTS = [(0, 3, 64, 40), (1, 5, 64, 40), (64, 32, 2048, 1024), (13, 4, 1056, 40), (100, 60, 96, 203), (500, 6, 512, 776), (700, 4, 1056, 1003),
           (3000, 7, 544, 1024), (2500, 4, 1056, 4090), (2000, 1, 512, 512), (600, 1000, 64, 50),
           (200, 4, 1056, 1003)]


def offsets_of(rows, E, seed, before=0, behind=0):
    g = np.random.Generator(np.random.PCG64(seed))
    p = np.exp(g.standard_normal(E)) * (g.random(E) < 0.8)
    p = p / p.sum() if p.sum() else np.full(E, 1.0 / E)
    counts = g.multinomial(rows - before - behind, p)
    return np.concatenate([[before], before + np.cumsum(counts)])


@pytest.mark.parametrize("dtype,y_dtype", [(bf, bf), (f32, f32), (E4M3, f32), (E4M3, bf), (bf, f32)])
@pytest.mark.parametrize("rows,E,n_in,n_out", EXPERTS)
def test_experts(rows, E, n_in, n_out, dtype, y_dtype):
    ws = [Weight(n_out, n_in, 100 + e % 4) for e in range(min(E, 4))]
    ws = [ws[e % 4] for e in range(E)]
    W, s = torch.stack([w.W.view(torch.uint8) for w in ws]).view(E4M3), torch.stack([w.s for w in ws])
    before, behind = (3, 5) if rows > 50 else (0, 0)
    ends = offsets_of(rows, E, 12, before, behind)
    X, x64 = floats((rows, n_in), bf if dtype is E4M3 else dtype, 13)
    bias, b64 = floats((E, n_out), y_dtype, 14)
    gate, g64 = floats((rows, n_out), y_dtype, 15)
    scales = None
    if dtype is E4M3:
        X, scales = (binding.fp8_quantize(X) if rows else (X.to(E4M3), torch.empty((n_in + 127) // 128, 0, device="cuda")))
    out = torch.full((rows, n_out), 55.0, dtype=y_dtype, device="cuda")
    offsets = torch.from_numpy(ends).to(torch.int32).cuda()
    Y = binding.linear_fp8_experts(X, offsets, W, s, x_scales=scales, bias=bias, activation="silu", gate=gate, y_dtype=y_dtype, out=out)
    if not rows:
        return
    x64 = held(x64)
    want, bound = np.full((rows, n_out), 55.0), np.zeros((rows, n_out))
    thin = narrow(rows, n_out, n_in, dtype, y_dtype, E)
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        if ends[e] < ends[e + 1]:
            want[r], bound[r] = product64(x64[r], ws[e].values, y_dtype, thin, bias=b64[e], act="silu", gate=g64[r])
    check(Y, want, bound, f"experts {rows} {E}")


def test_offsets_that_break_the_rules():
    """Unspecified rows, but nothing outside the buffers: guards before and behind Y stay."""
    rows, E, n_in, n_out = 300, 4, 256, 128
    ws = [Weight(n_out, n_in, 20 + e) for e in range(E)]
    W, s = torch.stack([w.W.view(torch.uint8) for w in ws]).view(E4M3), torch.stack([w.s for w in ws])
    X, _ = floats((rows, n_in), bf, 21)
    room = torch.full((rows + 200, n_out), 5.0, dtype=bf, device="cuda")
    for bad in ([0, 100, 50, 400, 300], [-5, -3, 10, 1 << 30, 1 << 30], [1 << 31 - 1, 0, 0, 0, 0], [300, 300, 200, 100, 0]):
        offsets = torch.tensor([min(b, (1 << 31) - 1) for b in bad], dtype=torch.int32, device="cuda")
        binding.linear_fp8_experts(X, offsets, W, s, y_dtype=bf, out=room[100:400])
        assert (room[:100] == 5.0).all() and (room[400:] == 5.0).all()


@pytest.mark.parametrize("M,n_in,n_out", [(1, 64, 32), (77, 130, 203), (300, 256, 1003), (1500, 512, 768)])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_gradients(M, n_in, n_out, dtype):
    """dX = dY W and dW = dY^T X as products of the same kind, against the formulas on the quantised operands, and dX against
    differences of the forward product (which is linear where X is quantised already)."""
    g = np.random.Generator(np.random.PCG64(22))
    dYt, dY = floats((M, n_out), dtype, 23, std=1e-3)
    Xt, X = floats((M, n_in), dtype, 24, outliers=2)
    # dW, rows of dY^T and X^T quantised along the tokens
    dy, dy_s = binding.fp8_quantize(dYt, transposed=True)
    x, x_s = binding.fp8_quantize(Xt, transposed=True)
    for y_dtype in (f32, bf):
        want, bound = product64(held(dY.T), held(X.T), y_dtype, y_dtype is bf)
        check(binding.linear_fp8(dy, x, x_s, x_scales=dy_s, y_dtype=y_dtype), want, bound, "dW")
    total, t64 = floats((n_out, n_in), f32, 25)
    want, bound = product64(held(dY.T), held(X.T), f32, False, residual=t64)
    binding.linear_fp8(dy, x, x_s, x_scales=dy_s, residual=total, out=total)   # added to a gradient that is there
    check(total, want, bound, "dW added")
    # dX: W^T in the same blocks
    if n_out % 32 or n_in % 32:
        return
    Wd, W64 = floats((n_out, n_in), f32, 26, std=0.02)
    Wt, wt_s = binding.fp8_quantize(Wd, 128, transposed=True)
    Wq, w_s = binding.fp8_quantize(Wd, 128)
    assert np.array_equal(codes_of(Wt)[:, :n_out], codes_of(Wq).T) and torch.equal(wt_s, w_s.T)
    codes, scales = quantize64(W64, 128)
    w = from_code(codes) * spread(scales, n_out, n_in, False)
    want, bound = product64(held(dY), w.T, f32, False)
    dX = binding.linear_fp8(dYt, Wt, wt_s)
    check(dX, want, bound, "dX")
    step, d64 = floats((M, n_in), f32, 27)
    q, q_s = binding.fp8_quantize(step)
    moved = binding.linear_fp8(q, Wq, w_s, x_scales=q_s).double().cpu().numpy()     # what a step in X moves Y by
    a, b = np.sum(held(dY) * moved), np.sum(dX.double().cpu().numpy() * held(d64))
    size = np.sum(np.abs(held(dY)) @ np.abs(w) * np.abs(held(d64)))
    assert abs(a - b) <= 2 * (128 + (max(n_in, n_out) + 127) // 128 + 16) * 2.0 ** -24 * size


def test_not_finite():
    """NaN and infinities in X make their rows NaN, in W (NaN codes) their columns, and nothing else; on every kernel."""
    for M, n_out in ((3, 64), (20, 200), (200, 1003), (600, 520), (1500, 2048), (2100, 4096)):
        n_in = 544
        w = Weight(n_out, n_in, 28)
        codes = w.codes.copy()
        codes[7, 530] = 0x7F
        X, _ = floats((M, n_in), bf, 29)
        X[1, 5], X[2, 543] = float("inf"), float("nan")
        for y_dtype in (bf, f32):
            Y = binding.linear_fp8(X, dev_codes(codes), w.s, y_dtype=y_dtype).float().cpu()
            bad = torch.zeros(M, n_out, dtype=torch.bool)
            bad[1:3], bad[:, 7] = True, True
            assert torch.equal(torch.isnan(Y), bad)


def test_scales_of_one_row():
    """w_block_rows 1 and 128 with the same scales give the same sums."""
    for M, n_in, n_out in ((9, 256, 300), (200, 544, 1003), (300, 544, 2048), (1100, 288, 4096), (3000, 512, 4500)):
        w = Weight(n_out, n_in, 30)
        X, x64 = floats((M, n_in), bf, 31)
        by_row = w.s.repeat_interleave(128, 0)[:n_out].T.contiguous()
        want, bound = product64(held(x64), w.values, f32, False)
        check(binding.linear_fp8(X, w.W, by_row), want, bound, "by row")
        want, bound = product64(held(x64), w.values, bf, True)
        check(binding.linear_fp8(X, w.W, by_row, y_dtype=bf), want, bound, "by row, bfloat16")


def test_graph_and_stream():
    M, n_in, n_out, E = 600, 544, 520, 3
    ws = [Weight(n_out, n_in, 40 + e) for e in range(E)]
    W, s = torch.stack([w.W.view(torch.uint8) for w in ws]).view(E4M3), torch.stack([w.s for w in ws])
    X, _ = floats((M, n_in), bf, 43)
    offsets = torch.tensor([0, 100, 450, 600], dtype=torch.int32, device="cuda")
    need = max(binding.linear_fp8_workspace_bytes(M, n_out, n_in, bf, bf), binding.linear_fp8_workspace_bytes(M, n_out, n_in, bf, bf, E), 16)
    wk = torch.full((2, need), 255, dtype=torch.uint8, device="cuda")
    Y, Z = torch.zeros(M, n_out, dtype=bf, device="cuda"), torch.zeros(M, n_out, dtype=bf, device="cuda")

    def run(stream=None):
        binding.linear_fp8(X, W[0], s[0], activation="silu", y_dtype=bf, out=Y, workspace=wk[0], stream=stream)
        binding.linear_fp8_experts(X, offsets, W, s, gate=Y, y_dtype=bf, out=Z, workspace=wk[1], stream=stream)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(4):
        X.copy_(floats((M, n_in), bf, 50 + seed)[0])
        offsets.copy_(torch.tensor([0, 100 * seed, 150 * seed + 5, 600 - seed], dtype=torch.int32))
        Z.zero_()
        run()
        want = [Y.clone(), Z.clone()]
        Y.zero_(), Z.zero_(), wk.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want[0]) and torch.equal(Z, want[1])
    side = torch.cuda.Stream()
    Y.zero_(), Z.zero_()
    torch.cuda.synchronize()
    run(side)
    side.synchronize()
    assert torch.equal(Y, want[0]) and torch.equal(Z, want[1])


@pytest.mark.parametrize("M,n_in,n_out", [(600_000, 64, 4100), (70_001, 32768, 24)])
def test_offsets_past_31_bits(M, n_in, n_out):
    """Y, and X with its quantised form, of more than 2^31 entries: rows of the start, the end and around 2^31 entries."""
    w = Weight(n_out, n_in, 70)
    few, x64 = floats((97, n_in), bf, 71)     # rows repeat, 97 of them
    X = few.repeat(-(-M // 97), 1)[:M].contiguous()
    assert max(M * n_in, M * n_out) > 1 << 31
    middle = (1 << 31) // max(n_in, n_out)
    at = np.unique(np.concatenate([np.arange(40), middle + np.arange(-20, 20), M - 1 - np.arange(300)]))
    thin = narrow(M, n_out, n_in, bf, bf)
    want, bound = product64(held(x64), w.values, bf, thin)
    offsets = torch.tensor([0, 5, M], dtype=torch.int32, device="cuda")
    pair = torch.stack([w.W.view(torch.uint8)] * 2).view(E4M3), torch.stack([w.s] * 2)
    for Y in (binding.linear_fp8(X, w.W, w.s, y_dtype=bf), binding.linear_fp8_experts(X, offsets, *pair, y_dtype=bf)):
        check(Y[torch.from_numpy(at).cuda()], want[at % 97], bound[at % 97], f"{M} {n_in} {n_out}")
        for lo in range(0, M, 97 * 1000):     # every row is the row of its kind, bit for bit
            part = Y[lo:lo + 97 * 1000]
            assert torch.equal(part, Y[:97].repeat(-(-len(part) // 97), 1)[:len(part)])
