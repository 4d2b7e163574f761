"""GPU parity of splr_linear_experts: rows grouped by expert, against the float64 evaluation of every
group by itself (bounds in tests/_fused.py), with empty groups, rows that belong to no group, sizes
across the tiles, offsets changed between graph replays and offsets that break the rules."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding, inputs
from tests._fused import Weights, check, fused64, rows64
from tests._helpers import meta_to_dev, to_dev

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def stacked(ws):
    d, r = ws[0].dtype, ws[0].r
    st = lambda name: np.stack([getattr(w, name) for w in ws])  # noqa: E731
    return dict(values=to_dev(st("values"), d), meta=meta_to_dev(st("meta")), U=to_dev(st("U"), d) if r else None,
                V=to_dev(st("V"), d) if r else None, bias=to_dev(st("bias"), d) if ws[0].bias is not None else None)


def case(offsets, M, n_in, n_out, r, dtype, y_dtype, act, bias, gate, residual, seed, integers=False, same=None):
    E = len(offsets) - 1
    if same:  # many experts: a few distinct ones, repeated
        base = [Weights(n_in, n_out, r, dtype, seed + e, bias, integers) for e in range(same)]
        ws = [base[e % same] for e in range(E)]
    else:
        ws = [Weights(n_in, n_out, r, dtype, seed + e, bias, integers) for e in range(E)]
    X = (inputs.small_integers((M, n_in), -2, 2, dtype, seed=seed, tensor_id=0) if integers
         else inputs.activations(M, n_in, dtype, 2, 20.0, seed=seed, config_id=1000, layer_id=0))
    g, g64 = rows64((M, n_out), y_dtype, seed, 6, integers) if gate else (None, None)
    s, s64 = rows64((M, n_out), y_dtype, seed, 7, integers) if residual else (None, None)
    d = dict(stacked(ws), X=to_dev(X, dtype), gate=g, residual=s, ws=ws, g64=g64, s64=s64,
             X64=inputs.to_f64(X, dtype))
    return d


def want_of(d, offsets, act, y_dtype, fill):
    M, n_out = d["X64"].shape[0], d["ws"][0].n_out
    want, bound = np.full((M, n_out), fill), np.zeros((M, n_out))
    for e, w in enumerate(d["ws"]):
        at = slice(offsets[e], offsets[e + 1])
        if offsets[e] < offsets[e + 1]:
            want[at], bound[at] = fused64(d["X64"][at], w, act, None if d["g64"] is None else d["g64"][at],
                                          None if d["s64"] is None else d["s64"][at], y_dtype)
    return want, bound


def run(d, offsets, act, y_dtype, n_out, fill=None, **kw):
    o = offsets if isinstance(offsets, torch.Tensor) else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    if fill is not None:
        kw["out"] = torch.full((d["X"].shape[0], n_out), fill, dtype=y_dtype, device="cuda")
    return binding.linear_experts(d["X"], o, d["values"], d["meta"], d["U"], d["V"], bias=d["bias"], activation=act,
                                  gate=d["gate"], residual=d["residual"], y_dtype=y_dtype, n_out=n_out, **kw)


# offsets, M: one row in all; two rows an expert; empty groups first, last and between; rows before,
# behind; one expert with everything; groups across the 16-, 64- and 128-row tiles
GROUPS = [
    ([0, 0, 1, 1], 1), ([0, 2, 4, 6, 8], 8), ([3, 3, 10, 10, 12, 12], 20), ([0, 70], 70),
    ([0, 0, 0, 90, 90], 90), ([5, 21, 38, 102, 103], 140), ([0, 130, 131, 259, 300, 300, 430], 431),
    ([0, 1, 200, 201, 460], 460),
]
SIZES = [(96, 40, 16), (288, 259, 0), (1056, 130, 80), (544, 530, 144)]  # n_in, n_out, r
EPILOGUES = [("none", False, False, False, F32), ("silu", False, True, False, BF16), ("gelu", True, True, True, F32),
             ("relu", True, False, True, BF16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group", range(len(GROUPS)))
def test_against_float64(group, dtype):
    offsets, M = GROUPS[group]
    for i, (n_in, n_out, r) in enumerate(SIZES):
        act, bias, gate, residual, y_dtype = EPILOGUES[(i + group) % len(EPILOGUES)]
        tag = f"{dtype} offsets {offsets} M={M} {n_in}->{n_out} r{r} {act} {y_dtype}"
        print(f"[experts] {tag}", flush=True)
        d = case(offsets, M, n_in, n_out, r, dtype, y_dtype, act, bias, gate, residual, seed=100 * group + i)
        want, bound = want_of(d, offsets, act, y_dtype, 7.0)
        check(run(d, offsets, act, y_dtype, n_out, fill=7.0), want, bound, tag)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,M", [(64, 100), (65, 100), (200, 900), (1024, 300), (1024, 3000)])
def test_many_experts(E, M, dtype):
    rng = np.random.default_rng(E + M)
    counts = np.bincount(rng.integers(0, E, size=M - 3), minlength=E)
    offsets = [int(v) for v in np.concatenate([[1], 1 + np.cumsum(counts)])]
    print(f"[experts] {dtype} E={E} M={M}", flush=True)
    d = case(offsets, M, 96, 50, 16, dtype, F32, "none", True, False, True, seed=E, same=5)
    want, bound = want_of(d, offsets, "none", F32, -3.0)
    check(run(d, offsets, "none", F32, 50, fill=-3.0), want, bound, f"{dtype} E={E} M={M}")


# rows of 5 experts together, n_in, n_out, r: sizes that take each kernel (few tokens, 128 x 64 tiles, 256
# and 512 x 128 tiles), quads and odd rows, more than one rank block
LARGE = [(64, 96, 4100, 16), (300, 2048, 1032, 48), (700, 1056, 1003, 80), (4000, 1024, 2048, 32), (4100, 1056, 1030, 144),
         (26000, 512, 1024, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,n_in,n_out,r", LARGE)
def test_every_entry_of_large_results(M, n_in, n_out, r, dtype):
    """Every entry of large grouped results against float64 products on the device, with the bound of
    tests/_fused.py."""
    dt = BF16 if dtype == "bf16" else F32
    E, u = 5, 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(M)

    def normal(*shape, std=1.0, to=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)
    counts = [M // 5, M // 9, 0, M // 3]
    offsets = [2]
    for n in counts + [M - 5 - sum(counts)]:
        offsets.append(offsets[-1] + n)
    X, R, U, V, bias = normal(M, n_in), normal(E, n_out, n_in, std=0.05), normal(E, n_out, r, std=0.2), normal(E, r, n_in, std=0.2), normal(E, n_out)
    packs = [binding.prune24_pack(R[e]) for e in range(E)]
    S = [binding.dense_reconstruct(v, m, None, None, n_out=n_out, n_in=n_in).double() for v, m in packs]
    values, meta = torch.stack([p[0] for p in packs]), torch.stack([p[1] for p in packs])
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for y_dtype in (F32, BF16):
        gate, residual = normal(M, n_out, to=y_dtype), normal(M, n_out, to=y_dtype)
        out = torch.full((M, n_out), 9.0, dtype=y_dtype, device="cuda")
        got = binding.linear_experts(X, off, values, meta, U, V, bias=bias, activation="silu", gate=gate,
                                     residual=residual, y_dtype=y_dtype, n_out=n_out, out=out)
        assert bool((got[:2] == 9.0).all()) and bool((got[M - 3:] == 9.0).all())
        for e in range(E):
            at = slice(offsets[e], offsets[e + 1])
            x, ue, ve = X[at].double(), U[e].double(), V[e].double()
            t = x @ ve.t()
            z = x @ S[e].t() + t @ ue.t() + bias[e].double()
            a = x.abs() @ S[e].abs().t() + t.abs() @ ue.abs().t() + bias[e].double().abs()
            d = (n_in * u * (x.abs() @ ve.abs().t()) + 2.0 ** -17 * t.abs()) @ ue.abs().t() + (n_in + 2 * r + 16) * u * a
            y, d = z * torch.sigmoid(z) * gate[at].double(), (1.13 * d + 16 * u * z.abs()) * gate[at].double().abs()
            d = d + 4 * u * (y.abs() + residual[at].double().abs())
            y = y + residual[at].double()
            d = d + (u if y_dtype == F32 else 2.0 ** -8) * (y.abs() + d)
            wrong = int(((got[at].double() - y).abs() > d).sum())
            assert wrong == 0, (dtype, y_dtype, e, wrong)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_small_integers_exactly(dtype):
    for offsets, M in GROUPS[2:]:
        d = case(offsets, M, 160, 70, 32, dtype, F32, "relu", True, True, True, seed=M, integers=True)
        want, _ = want_of(d, offsets, "relu", F32, 1.0)
        got = run(d, offsets, "relu", F32, 70, fill=1.0).cpu().double().numpy()
        assert np.array_equal(got, want), (dtype, offsets)


def test_no_rows():
    d = case([0, 0, 0], 1, 96, 40, 16, "bf16", F32, "none", True, False, False, seed=1)
    d["X"] = d["X"][:0]
    assert run(d, [0, 0, 0], "none", F32, 40).shape == (0, 40)
    d = case([0, 0, 0], 5, 96, 40, 16, "bf16", F32, "none", True, False, False, seed=1)
    got = run(d, [2, 2, 2], "none", F32, 40, fill=4.0)
    assert bool((got == 4.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [-7, 10, 20, 60], [0, 10, 500, 60], [60, 40, 20, 0], [-9, -5, -2, -1],
                                 [2**31 - 1] * 4, [-2**31, 2**31 - 1, -2**31, 2**31 - 1]])
def test_offsets_that_break_the_rules_stay_in_bounds(bad, dtype):
    """Y may hold anything, but only Y: the kernels clamp every row range. Guards lie on both sides."""
    M, n_out = 60, 48
    d = case([0, 20, 40, 60], M, 96, n_out, 16, dtype, F32, "none", True, False, False, seed=5)
    guard = torch.full((3 * M, n_out), 5.0, device="cuda")
    run(d, bad, "none", F32, n_out, out=guard[M:2 * M])
    torch.cuda.synchronize()
    assert bool((guard[:M] == 5.0).all()) and bool((guard[2 * M:] == 5.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_not_finite_rows_stay_apart(dtype):
    offsets, M = [0, 20, 45, 150], 150
    d = case(offsets, M, 288, 70, 16, dtype, F32, "none", False, False, False, seed=2)
    want, bound = want_of(d, offsets, "none", F32, 0.0)
    bad = [19, 20, 44, 60, 149]
    d["X"][bad] = float("nan")
    got = run(d, offsets, "none", F32, 70).cpu().double().numpy()
    rows = [m for m in range(M) if m not in bad]
    assert np.isnan(got[bad]).all()
    assert np.all(np.abs(got - want)[rows] <= bound[rows])


@pytest.mark.parametrize("dtype,M", [("bf16", 40), ("bf16", 300), ("fp32", 90)])
def test_graph_replayed_with_other_offsets(dtype, M):
    """The group sizes are read on the device, so a captured call follows new offsets and inputs."""
    E, n_in, n_out, r = 6, 544, 130, 32
    rng = np.random.default_rng(M)
    routes = [np.concatenate([[0], np.cumsum(np.bincount(rng.integers(0, E, M), minlength=E))]) for _ in range(2)]
    routes += [np.array([0, 0, 0, M, M, M, M])]
    d = case([0] * E + [M], M, n_in, n_out, r, dtype, BF16, "silu", True, True, True, seed=9)
    want = [run(d, [int(v) for v in o], "silu", BF16, n_out) for o in routes]
    dev = [torch.tensor(o, dtype=torch.int32, device="cuda") for o in routes]
    live, out = dev[0].clone(), torch.empty_like(want[0])
    ws = torch.empty(max(1, binding.experts_workspace_bytes(M, E, n_out, n_in, r, d["X"].dtype)), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run(d, live, "silu", BF16, n_out, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(d, live, "silu", BF16, n_out, out=out, workspace=ws)
    for i in (1, 0, 2, 1):
        live.copy_(dev[i])
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        assert torch.equal(run(d, dev[i], "silu", BF16, n_out), want[i])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_expert_mlp(dtype):
    """The operators as an expert MLP uses them: up, silu(gate) * up, down added to the residual, then a
    dense layer over all rows. Each step is held to float64 on the inputs it was given."""
    offsets, M, n, ff, r = [0, 33, 33, 100, 180], 180, 256, 352, 32
    t, y = ("bf16", BF16) if dtype == "bf16" else ("fp32", F32)
    E = len(offsets) - 1
    up, gate = ([Weights(n, ff, r, t, 10 * i + e) for e in range(E)] for i in (1, 2))
    down = [Weights(ff, n, r, t, 30 + e, bias=True) for e in range(E)]
    dense = Weights(n, 144, r, t, 50, bias=True)
    X = inputs.activations(M, n, t, 2, 20.0, seed=4, config_id=1000, layer_id=0)
    x = to_dev(X, t)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def step(ws, inp, act="none", g=None, res=None, out=None):
        d = stacked(ws)
        return binding.linear_experts(inp, off, d["values"], d["meta"], d["U"], d["V"], bias=d["bias"], activation=act,
                                      gate=g, residual=res, y_dtype=y, n_out=ws[0].n_out, out=out)

    u = step(up, x)
    h = step(gate, x, "silu", g=u, out=u.clone())
    z = step(down, h, res=x)
    dd = dict(values=to_dev(dense.values, t), meta=meta_to_dev(dense.meta), U=to_dev(dense.U, t), V=to_dev(dense.V, t))
    f = binding.linear_fused(z, dd["values"], dd["meta"], dd["U"], dd["V"], bias=to_dev(dense.bias, t),
                             activation="gelu", y_dtype=y)
    n64 = lambda v: v.cpu().double().numpy()  # noqa: E731
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        for got, ws, inp, act, g, res, tag in ((u, up, x, "none", None, None, "up"), (h, gate, x, "silu", u, None, "gate"),
                                               (z, down, h, "none", None, x, "down")):
            want, bound = fused64(n64(inp[at]), ws[e], act, None if g is None else n64(g[at]),
                                  None if res is None else n64(res[at]), y)
            check(got[at], want, bound, f"{dtype} {tag} {e}")
    want, bound = fused64(n64(z), dense, "gelu", None, None, y)
    check(f, want, bound, f"{dtype} dense")
