"""GPU parity of splr_linear_fused: the product, bias, activation, gate and residual against a plain
float64 evaluation, within the bound that counts the kernel's float32 roundings (tests/_fused.py)."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding, inputs
from tests._fused import ACTS, HALF_STEP, Weights, check, fused64, rows64
from tests._helpers import meta_to_dev, to_dev

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def device(w):
    d = w.dtype
    return dict(values=to_dev(w.values, d), meta=meta_to_dev(w.meta), U=to_dev(w.U, d) if w.r else None,
                V=to_dev(w.V, d) if w.r else None, bias=to_dev(w.bias, d))


def case(M, n_in, n_out, r, dtype, y_dtype, act, bias, gate, residual, seed, integers=False):
    w = Weights(n_in, n_out, r, dtype, seed, bias, integers)
    X = (inputs.small_integers((M, n_in), -2, 2, dtype, seed=seed, tensor_id=0) if integers
         else inputs.activations(M, n_in, dtype, 2, 20.0, seed=seed, config_id=1000, layer_id=0))
    g, g64 = rows64((M, n_out), y_dtype, seed, 6, integers) if gate else (None, None)
    s, s64 = rows64((M, n_out), y_dtype, seed, 7, integers) if residual else (None, None)
    d = dict(device(w), X=to_dev(X, dtype), gate=g, residual=s)
    want, bound = fused64(inputs.to_f64(X, dtype), w, act, g64, s64, y_dtype)
    return d, want, bound


def run(d, act, y_dtype, n_out, **kw):
    return binding.linear_fused(d["X"], d["values"], d["meta"], d["U"], d["V"], bias=d["bias"], activation=act,
                                gate=d["gate"], residual=d["residual"], y_dtype=y_dtype, n_out=n_out, **kw)


# (M, n_in, n_out, r): one token; the decode sizes' edges; ragged tiles in every dimension; tails of
# 32 columns; ranks below, at and past the blocks of 64; few and many K steps; odd row lengths
SHAPES = [
    (1, 32, 1, 0), (1, 4096, 96, 64), (2, 96, 17, 16), (16, 1056, 130, 48), (17, 512, 64, 128), (33, 2080, 48, 64),
    (64, 288, 1003, 32), (65, 64, 20, 16), (129, 544, 257, 80), (200, 1088, 515, 192), (300, 4096, 300, 64),
    (9, 64, 50, 1024), (130, 96, 40, 1024),
    (16, 96, 8200, 16), (20, 2080, 8195, 80),   # two row tiles a workgroup, an odd number of them
]
# act, bias, gate, residual, Y type
EPILOGUES = [
    ("none", False, False, False, F32), ("none", True, False, True, BF16), ("silu", False, True, False, BF16),
    ("gelu", True, True, True, F32), ("relu", False, False, True, F32), ("gelu_tanh", True, True, False, BF16),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_float64(shape, dtype):
    M, n_in, n_out, r = shape
    for i, (act, bias, gate, residual, y_dtype) in enumerate(EPILOGUES):
        tag = f"{dtype} {M}x{n_in}->{n_out} r{r} {act} bias={bias} gate={gate} residual={residual} {y_dtype}"
        print(f"[fused] {tag}", flush=True)
        d, want, bound = case(M, n_in, n_out, r, dtype, y_dtype, act, bias, gate, residual, seed=7 * M + n_in + i)
        check(run(d, act, y_dtype, n_out), want, bound, tag)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 140])
def test_every_activation_over_its_range(act, M):
    """X = 0, so Z is the bias: values from far below to far above where the activations bend."""
    n_in, n_out = 64, 512
    z = np.concatenate([np.linspace(-12, 12, 480), [0.0, -0.0, 1e-30, -1e-30, 30, -30, 88, -88, 120, -120, 1e4, -1e4],
                        np.linspace(-1e-3, 1e-3, 20)]).astype(np.float32)
    for dtype in ("bf16", "fp32"):
        w = Weights(n_in, n_out, 0, dtype, seed=1)
        w.bias = inputs.from_f64(z, dtype)
        w.b64 = inputs.to_f64(w.bias, dtype)
        X = inputs.from_f64(np.zeros((M, n_in)), dtype)
        d = dict(device(w), X=to_dev(X, dtype), gate=None, residual=None)
        with np.errstate(over="ignore"):
            want, bound = fused64(np.zeros((M, n_in)), w, act)
        check(run(d, act, F32, n_out), want, bound, f"{act} {dtype} M={M}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,n_in,n_out,r", [(1, 96, 40, 16), (33, 160, 100, 32), (70, 1056, 70, 80), (150, 224, 530, 16)])
def test_small_integers_exactly(M, n_in, n_out, r, dtype):
    """Integer inputs: every product and sum is exact, so Y is the exact value, bit for bit."""
    for act, y_dtype in (("none", F32), ("relu", F32)):
        d, want, _ = case(M, n_in, n_out, r, dtype, y_dtype, act, True, True, True, seed=M, integers=True)
        got = run(d, act, y_dtype, n_out).cpu().double().numpy()
        assert np.abs(want).max() < 2 ** 24
        assert np.array_equal(got, want), f"{dtype} {M}x{n_in}->{n_out} {act}"


@pytest.mark.parametrize("dtype,M", [("bf16", 5), ("bf16", 40), ("bf16", 130), ("fp32", 5), ("fp32", 130)])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_in_place(dtype, M, y_dtype):
    """Y written over residual, and over gate, gives what a buffer of its own gives."""
    d, _, _ = case(M, 320, 200, 16, dtype, y_dtype, "silu", True, True, True, seed=M)
    want = run(d, "silu", y_dtype, 200)
    for name in ("residual", "gate"):
        e = dict(d)
        e[name] = d[name].clone()
        got = run(e, "silu", y_dtype, 200, out=e[name])
        assert got is e[name] and torch.equal(got, want), name


def test_without_epilogue_is_linear_ex():
    """With nothing in the epilogue, and sizes that the same kernels take, the bfloat16 product is
    linear_ex's, bit for bit."""
    for M, n_out in ((7, 200), (50, 200), (2000, 4096)):
        d, _, _ = case(M, 544, n_out, 32, "bf16", F32, "none", False, False, False, seed=M)
        for y in (F32, BF16):
            a = run(d, "none", y, n_out)
            b = binding.linear_ex(d["X"], d["values"], d["meta"], d["U"], d["V"], y_dtype=y, n_out=n_out)
            assert torch.equal(a, b), (M, y)


def act64_on_device(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


@pytest.mark.parametrize("M,n_out", [(2000, 4096), (4000, 4096), (8192, 4096), (2500, 4098)])
@pytest.mark.parametrize("y_dtype", [F32, BF16])
def test_every_entry_of_a_large_result(M, n_out, y_dtype):
    """The epilogue on every entry of large results, several times over, against float64 arithmetic on the
    float32 sums (the plain product's, which the fused kernels share bit for bit)."""
    n_in, r = 1024, 16   # 256-row tiles, 512-row tiles, these with Y past the caches, rows that are no quads
    g = torch.Generator(device="cuda").manual_seed(M)
    def normal(*shape, std=1.0, to=BF16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)
    X, U, V, bias = normal(M, n_in), normal(n_out, r, std=0.3), normal(r, n_in, std=0.3), normal(n_out)
    values, meta = binding.prune24_pack(normal(n_out, n_in, std=0.2))
    gate, residual = normal(M, n_out, to=y_dtype), normal(M, n_out, to=y_dtype)
    sums = binding.linear_ex(X, values, meta, U, V, n_out=n_out).double()
    u = 2.0 ** -24
    for act in ACTS:
        for b, ga, re in ((bias, gate, residual), (bias, gate, None), (None, None, residual), (bias, None, None)):
            z = sums if b is None else sums + b.double()
            want, bound = act64_on_device(z, act), 17 * u * z.abs()   # 16 as in tests/_fused.py, 1 for the bias sum
            if ga is not None:
                want, bound = want * ga.double(), bound * ga.double().abs()
            if re is not None:
                want = want + re.double()
            bound = bound + 4 * u * (want.abs() + (0 if re is None else re.double().abs()))
            bound = bound + HALF_STEP[y_dtype] * (want.abs() + bound)
            for _ in range(3):
                got = binding.linear_fused(X, values, meta, U, V, bias=b, activation=act, gate=ga, residual=re,
                                           y_dtype=y_dtype, n_out=n_out)
                wrong = int(((got.double() - want).abs() > bound).sum())
                assert wrong == 0, (act, b is not None, ga is not None, re is not None, wrong)


@pytest.mark.parametrize("dtype,M", [("bf16", 5), ("bf16", 130), ("fp32", 130)])
def test_not_finite_rows_stay_apart(dtype, M):
    """A token row, a gate entry or a residual entry that is not finite changes no other row or entry;
    a bias of minus infinity gives relu 0."""
    d, want, bound = case(M, 288, 70, 16, dtype, F32, "relu", True, True, True, seed=3)
    d["X"][2] = float("nan")
    d["X"][4, 1] = float("inf")
    d["gate"][3, 5] = float("nan")
    d["residual"][1, 6] = float("inf")
    d["bias"][9] = float("-inf")
    got = run(d, "relu", F32, 70).cpu().double().numpy()
    assert np.isnan(got[2, :9]).all() and np.isnan(got[3, 5]) and np.isposinf(got[1, 6])
    rows = [m for m in range(M) if m not in (2, 4)]
    res = d["residual"].cpu().double().numpy()
    assert np.array_equal(got[rows, 9], res[rows, 9])
    keep = np.ones((M, 70), bool)
    keep[[2, 4]] = False
    keep[:, 9] = False
    keep[3, 5] = keep[1, 6] = False
    assert np.all(np.abs(got - want)[keep] <= bound[keep])


@pytest.mark.parametrize("dtype,M", [("bf16", 16), ("bf16", 300), ("fp32", 100)])
def test_graph_replays_and_streams(dtype, M):
    """Captured on another stream and replayed with new inputs between eager calls; two streams at once,
    each with its own workspace; bitwise the eager result every time."""
    cases = [case(M, 1056, 200, 64, dtype, BF16, "silu", True, True, True, seed=s)[0] for s in (1, 2, 3)]
    want = [run(c, "silu", BF16, 200) for c in cases]
    live = {k: v.clone() for k, v in cases[0].items()}
    ws = torch.empty(binding.fused_workspace_bytes(M, 200, 1056, 64, live["X"].dtype), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run(live, "silu", BF16, 200, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(live, "silu", BF16, 200, out=out, workspace=ws)
    for i in (1, 2, 0, 1):
        for k in live:
            live[k].copy_(cases[i][k])
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        assert torch.equal(run(cases[i], "silu", BF16, 200), want[i])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a = run(cases[0], "silu", BF16, 200, stream=s1)
        b = run(cases[1], "silu", BF16, 200, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_results_are_reproducible(dtype):
    d, _, _ = case(190, 1056, 333, 64, dtype, F32, "gelu", True, True, True, seed=8)
    first = run(d, "gelu", F32, 333)
    for _ in range(3):
        assert torch.equal(run(d, "gelu", F32, 333), first)
