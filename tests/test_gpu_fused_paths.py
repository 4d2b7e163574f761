"""The contracts of splr_linear_fused and splr_linear_experts on every one of their kernels (sizes in tests/_paths.py):
values against float64, Y over gate and over residual, graph replays with other inputs and other group sizes, two
streams at once, rows that are not finite, offsets that break the rules."""
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._paths import BF16, F32, IDS, SIZES

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
BUDGET_ROWS = 3   # rows behind the last expert, two before the first


class Call:
    """Weights, inputs and offsets of one size; `seed` decides the inputs, the weights are the size's."""

    def __init__(self, size, y_dtype, seed=0):
        self.dtype, self.experts, self.tile, self.M, self.n_in, self.n_out, self.r = size
        self.y_dtype, E = y_dtype, self.experts or 1
        assert binding.fused_tile(self.M, self.n_out, self.n_in, self.r, self.dtype, self.experts) == self.tile
        g = torch.Generator(device="cuda").manual_seed(self.M + self.r)

        def normal(*shape, std=1.0, to=self.dtype):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)
        packs = [binding.prune24_pack(normal(self.n_out, self.n_in, std=0.05)) for _ in range(E)]
        self.S = [binding.dense_reconstruct(*p, None, None, n_out=self.n_out, n_in=self.n_in) for p in packs]
        self.weights = dict(values=torch.stack([p[0] for p in packs]), meta=torch.stack([p[1] for p in packs]),
                            U=normal(E, self.n_out, self.r, std=0.2), V=normal(E, self.r, self.n_in, std=0.2),
                            bias=normal(E, self.n_out))
        g.manual_seed(1000 + seed)
        self.X = normal(self.M, self.n_in)
        self.gate, self.residual = normal(self.M, self.n_out, to=y_dtype), normal(self.M, self.n_out, to=y_dtype)
        self.offsets = None
        if self.experts:   # the second expert empty, rows at both ends to no expert, `seed` moves the boundary
            cut = 2 + (self.M - 5) * (2 + seed % 3) // 6
            third = cut + (self.M - 3 - cut) // (2 + seed % 2)
            self.ends = [2, cut, cut, third, self.M - BUDGET_ROWS]
            self.offsets = torch.tensor(self.ends, dtype=torch.int32, device="cuda")

    def run(self, act="silu", **kw):
        kw = dict(dict(gate=self.gate, residual=self.residual), **kw)
        w = self.weights
        common = dict(activation=act, y_dtype=self.y_dtype, n_out=self.n_out, **kw)
        if self.experts:
            if "out" not in kw:
                common["out"] = torch.full((self.M, self.n_out), 9.0, dtype=self.y_dtype, device="cuda")
            return binding.linear_experts(self.X, self.offsets, w["values"], w["meta"], w["U"], w["V"], bias=w["bias"],
                                          **common)
        return binding.linear_fused(self.X, w["values"][0], w["meta"][0], w["U"][0], w["V"][0], bias=w["bias"][0],
                                    **common)

    def spans(self):
        return [(0, 0, self.M)] if not self.experts else [(e, self.ends[e], self.ends[e + 1]) for e in range(4)]

    def workspace_bytes(self):
        if self.experts:
            return binding.experts_workspace_bytes(self.M, self.experts, self.n_out, self.n_in, self.r, self.dtype)
        return binding.fused_workspace_bytes(self.M, self.n_out, self.n_in, self.r, self.dtype)


each = pytest.mark.parametrize("size", SIZES, ids=IDS)
each_grouped = pytest.mark.parametrize("size", [s for s in SIZES if s[1]], ids=[i for i, s in zip(IDS, SIZES) if s[1]])


@each
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_against_float64(size, y_dtype):
    c = Call(size, y_dtype)
    got = c.run()
    if c.experts:
        assert bool((got[:2] == 9.0).all()) and bool((got[c.M - BUDGET_ROWS:] == 9.0).all())
    for e, lo, hi in c.spans():
        x, S, U, V, b, gate, residual = (t.double() for t in (c.X[lo:hi], c.S[e], c.weights["U"][e], c.weights["V"][e],
                                                              c.weights["bias"][e], c.gate[lo:hi], c.residual[lo:hi]))
        t = x @ V.t()
        z = x @ S.t() + t @ U.t() + b
        a = x.abs() @ S.abs().t() + t.abs() @ U.abs().t() + b.abs()
        d = (c.n_in * U32 * (x.abs() @ V.abs().t()) + 2.0 ** -17 * t.abs()) @ U.abs().t() + (c.n_in + 2 * c.r + 16) * U32 * a
        y, d = z * torch.sigmoid(z) * gate, (1.13 * d + 16 * U32 * z.abs()) * gate.abs()
        d = d + 4 * U32 * (y.abs() + residual.abs())
        y = y + residual
        d = d + (U32 if y_dtype == F32 else 2.0 ** -8) * (y.abs() + d)
        wrong = int((~((got[lo:hi].double() - y).abs() <= d)).sum())
        assert wrong == 0, (e, wrong)


@each
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_in_place_and_reproducible(size, y_dtype):
    """Y over gate, and over residual, is what a buffer of its own gets, every time."""
    c = Call(size, y_dtype)
    rows = slice(c.spans()[0][1], c.spans()[-1][2])
    want = c.run()
    for name in ("gate", "residual"):
        for _ in range(3):
            buffer = getattr(c, name).clone()
            got = c.run(**{name: buffer}, out=buffer)
            assert torch.equal(got[rows], want[rows]), name
            before = getattr(c, name)
            assert torch.equal(got[:rows.start], before[:rows.start]) and torch.equal(got[rows.stop:], before[rows.stop:])
    assert torch.equal(c.run(), want)
    lone = c.run(gate=None)   # residual without gate
    buffer = c.residual.clone()
    assert torch.equal(c.run(gate=None, residual=buffer, out=buffer)[rows], lone[rows])


@each
def test_graph_replays_follow_inputs_and_groups(size):
    """One captured call, replayed with other inputs and other group sizes between eager calls, from a workspace that holds
    other data each time: bitwise the eager result."""
    calls = [Call(size, BF16, seed=s) for s in range(3)]
    want = [c.run() for c in calls]
    live = Call(size, BF16, seed=0)
    ws = torch.empty(live.workspace_bytes(), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        live.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        live.run(out=out, workspace=ws)
    for i in (1, 2, 0, 2, 1):
        for name in ("X", "gate", "residual") + (("offsets",) if live.experts else ()):
            getattr(live, name).copy_(getattr(calls[i], name))
        out.fill_(9.0)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        assert torch.equal(calls[i].run(), want[i]), i


@each
def test_two_streams_at_once(size):
    a, b = Call(size, F32, seed=1), Call(size, F32, seed=2)
    want = a.run(), b.run()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.full_like(want[0], 9.0) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(out=outs[0], stream=s)
        b.run(out=outs[1], stream=t)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@each
def test_rows_that_are_not_finite_stay_apart(size):
    """A row of NaN or with infinities, a gate or residual entry that is not finite: every other row and entry as before."""
    c = Call(size, F32)
    clean = c.run()
    bad = sorted({3, 7, c.M // 2, c.M // 2 + 1, c.M - BUDGET_ROWS - 1})
    for i, m in enumerate(bad):
        c.X[m, (37 * i) % c.n_in if i % 2 else slice(None)] = float("inf") if i % 2 else float("nan")
    c.gate[4, 5] = float("nan")
    c.residual[5, 6] = float("inf")
    got = c.run()
    assert bool(torch.isnan(got[bad[::2]]).all()) and bool(torch.isnan(got[4, 5])) and float(got[5, 6]) == float("inf")
    same = torch.ones(c.M, c.n_out, dtype=torch.bool, device="cuda")
    same[bad] = False
    same[4, 5] = same[5, 6] = False
    assert torch.equal(got[same], clean[same])


@each_grouped
def test_offsets_that_break_the_rules_stay_in_bounds(size):
    """Y's rows may hold anything; what lies around Y, and behind the workspace's bytes, stays."""
    c = Call(size, F32)
    M, high = c.M, 2 ** 31 - 1
    size = M * c.n_out
    first = (size + 63) // 64 * 64   # Y starts aligned
    guard = torch.full((first + 2 * size,), 5.0, device="cuda")
    need = c.workspace_bytes()
    space = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    for bad in ([0, M, 0, M, M], [0, M, 0, M, 0], [-7, 5, M, M + 1000, M], [M, M - 1, 3, 1, 0], [-9, -5, -2, -1, -1], [high] * 5,
                [-high - 1, high, -high - 1, high, -high - 1], [M + 1, M + 2, M + 3, high, high], [0, 0, 0, 0, high]):
        c.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        c.run(out=guard[first:first + size].view(M, c.n_out), workspace=space[:need])
        torch.cuda.synchronize()
        assert bool((guard[:first] == 5.0).all()) and bool((guard[first + size:] == 5.0).all()), bad
        assert bool((space[need:] == 171).all()), bad
