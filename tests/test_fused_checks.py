"""Refusals of splr_linear_fused and splr_linear_experts on the CPU: the C ABI checks its arguments
before any HIP call, and the binding checks every tensor before the C ABI sees a pointer (host tensors
stand in for device tensors there, so those tests are skipped where a GPU is present)."""
import ctypes
import os

import pytest
import torch

from sparse_rank_linear_prune24_amd import binding

OK, NULL, SHAPE, DTYPE, ALIGN, HIP, WORKSPACE, SCRATCH = range(8)
OVERLAP = 8
A, MIS = 0x10000, 0x10008   # never dereferenced
BIG = 1 << 40
bf, f32 = torch.bfloat16, torch.float32


def ep(act=0, bias=None, gate=None, residual=None):
    return ctypes.byref(binding._Epilogue(act, bias, gate, residual))


def fused(X=A, M=16, K=64, v=A, m=A, N=32, U=A, V=A, r=16, dt=1, e=None, yd=1, Y=A, ws=A, wsb=BIG):
    return binding.lib().splr_linear_fused(X, M, K, v, m, N, U, V, r, dt, e, yd, Y, ws, wsb, None)


def experts(X=A, M=16, K=64, off=A, E=4, v=A, m=A, N=32, U=A, V=A, r=16, dt=1, e=None, yd=1, Y=A, ws=A, wsb=BIG):
    return binding.lib().splr_linear_experts(X, M, K, off, E, v, m, N, U, V, r, dt, e, yd, Y, ws, wsb, None)


@pytest.mark.parametrize("f", [fused, experts])
def test_shared_refusals(f):
    for name in ("X", "v", "m", "U", "V", "Y"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: MIS}) == ALIGN, name
    for kw in (dict(K=48), dict(K=0), dict(N=0), dict(M=-1), dict(r=8), dict(r=-16), dict(r=1040), dict(M=1 << 25),
               dict(N=1 << 25), dict(N=(1 << 21) + 1), dict(K=(1 << 20) + 32)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=2) == DTYPE and f(yd=2) == DTYPE and f(yd=-1) == DTYPE
    for act in (-1, 5):
        assert f(e=ep(act)) == SHAPE
    for kw in (dict(bias=MIS), dict(gate=MIS), dict(residual=MIS)):
        assert f(e=ep(**kw)) == ALIGN, kw
    assert f(ws=None) == WORKSPACE and f(wsb=0) == WORKSPACE and f(ws=MIS) == ALIGN


def test_experts_refusals():
    assert experts(off=None) == NULL
    assert experts(off=A + 2) == ALIGN
    assert experts(E=0) == SHAPE and experts(E=binding.EXPERTS_MAX + 1) == SHAPE
    assert experts(E=1024, N=1 << 20, K=1 << 12) == SHAPE       # weights above 2^36 entries
    assert fused(M=0) == SHAPE
    # no rows: nothing to do, row buffers may be missing, everything else is still checked
    assert experts(M=0, X=None, Y=None, ws=None, wsb=0) == OK
    assert experts(M=0, v=None) == NULL and experts(M=0, K=40) == SHAPE and experts(M=0, dt=7) == DTYPE


def test_workspace_sizes():
    f = binding.lib().splr_linear_experts_workspace_bytes
    assert f(64, 4, 32, 64, 0, 1) == 0 and f(0, 4, 32, 64, 16, 1) == 0
    assert f(64, 4, 32, 64, 16, 1) >= 64 * 16 * 4
    for bad in ((-1, 4, 32, 64, 16, 1), (64, 0, 32, 64, 16, 1), (64, 1025, 32, 64, 16, 1), (64, 4, 32, 48, 16, 1),
                (64, 4, 32, 64, 8, 1), (64, 4, 32, 64, 16, 3)):
        assert f(*bad) == 0
    need = f(64, 4, 32, 64, 16, 1)
    assert experts(M=64, wsb=need - 1) == WORKSPACE
    f = binding.lib().splr_linear_fused_workspace_bytes
    assert f(64, 32, 64, 0, 1) == 0
    for bad in ((0, 32, 64, 16, 1), (64, 32, 48, 16, 1), (64, 32, 64, 8, 1), (64, 32, 64, 16, 3)):
        assert f(*bad) == 0
    for dt in (0, 1):
        for M, K, r in ((64, 64, 16), (1, 4096, 64), (500, 14336, 128), (8192, 4096, 64)):
            need = f(M, 32, K, r, dt)
            assert need >= M * r * 4 and fused(M=M, K=K, r=r, dt=dt, wsb=need - 1) == WORKSPACE


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a call that got through would launch on made-up addresses")
@pytest.mark.parametrize("yd", [0, 1])
@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("grouped", [False, True])
def test_overlaps_are_refused(grouped, dt, yd):
    """Y and the workspace one entry or unit into the end of every operand, and every operand into theirs."""
    M, K, N, r, E, size, ysize = 50, 96, 40, 16, 3 if grouped else 1, (4, 2)[dt], (4, 2)[yd]
    L = binding.lib()
    need = (L.splr_linear_experts_workspace_bytes(M, E, N, K, r, dt) if grouped else
            L.splr_linear_fused_workspace_bytes(M, N, K, r, dt))
    TR, TK = binding.tiles(N, K)
    sizes = dict(X=M * K * size, off=4 * (E + 1), v=E * TR * TK * 512 * size, m=E * TR * 1024, U=E * N * r * size,
                 V=E * r * K * size, bias=E * N * size, gate=M * N * ysize, residual=M * N * ysize, Y=M * N * ysize, ws=need)
    place = {k: (i + 1) << 20 for i, k in enumerate(sizes)}

    def status(**moved):
        d = dict(place, **moved)
        e = ep(1, d.pop("bias"), d.pop("gate"), d.pop("residual"))
        if not grouped:
            d.pop("off")
        return (experts if grouped else fused)(M=M, K=K, N=N, r=r, dt=dt, yd=yd, e=e, wsb=need, **d,
                                               **(dict(E=E) if grouped else {}))
    for out in ("Y", "ws"):
        for other in sizes:
            if other == out or (other == "off" and not grouped):
                continue
            last = (sizes[other] - 1) // 16 * 16
            assert status(**{out: place[other] + last}) == OVERLAP, (out, other)
            last = (sizes[out] - 1) // 16 * 16
            assert status(**{other: place[out] + last}) == OVERLAP, (out, other)
            if not (out == "Y" and other in ("gate", "residual")):
                assert status(**{out: place[other]}) == OVERLAP, (out, other)
    assert status(Y=place["gate"], ws=place["gate"]) == OVERLAP


# experts, n_in, n_out, rows: inside every documented limit, with more tiles than a launch of the tile kernels takes
@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("E,K,N,M", [(1024, 64, 1 << 20, 1500), (1024, 64, 1 << 20, 8000), (1024, 32, (1 << 21) - 7, 1024), (512, 64, 1 << 21, 600),
                                     (512, 64, 1 << 21, 4000), (256, 128, 1 << 21, 32768), (700, 32, 3 << 19, 16000),
                                     (1000, 32, 1 << 21, 32768)])
def test_the_largest_sizes_find_a_kernel(E, K, N, M, dt):
    for r in (16, 64, 128):
        need = binding.lib().splr_linear_experts_workspace_bytes(M, E, N, K, r, dt)
        assert need >= M * r * 4
        assert experts(M=M, K=K, E=E, N=N, r=r, dt=dt, wsb=need - 1) == WORKSPACE


# ----------------------------------------------------------------------------- the binding
class _Stream:
    cuda_stream = 0


host = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="host tensors stand in for device tensors")


@pytest.fixture
def host_as_device(monkeypatch):
    monkeypatch.setattr(binding, "_is_device", lambda t: True)


def layer(E=None, M=32, n_in=128, n_out=48, r=16, dt=bf, y=f32):
    TR, TK = binding.tiles(n_out, n_in)
    e = () if E is None else (E,)
    d = dict(X=torch.zeros(M, n_in, dtype=dt), values=torch.zeros(*e, TR, TK, 64, 8, dtype=dt),
             meta=torch.zeros(*e, *binding.meta_shape(n_out, n_in), dtype=torch.int32),
             U=torch.zeros(*e, n_out, r, dtype=dt), V=torch.zeros(*e, r, n_in, dtype=dt),
             bias=torch.zeros(*e, n_out, dtype=dt), gate=torch.zeros(M, n_out, dtype=y),
             residual=torch.zeros(M, n_out, dtype=y), out=torch.zeros(M, n_out, dtype=y),
             workspace=torch.zeros(1 << 20, dtype=torch.uint8), n_out=n_out, y_dtype=y, stream=_Stream())
    if E is not None:
        d["offsets"] = torch.zeros(E + 1, dtype=torch.int32)
    return d


def call(E, **kw):
    d = dict(layer(E), **kw)
    X, v, m, U, V = (d.pop(k) for k in ("X", "values", "meta", "U", "V"))
    if E is None:
        return binding.linear_fused(X, v, m, U, V, **d)
    return binding.linear_experts(X, d.pop("offsets"), v, m, U, V, **d)


@host
@pytest.mark.parametrize("E", [None, 3])
def test_correct_shapes_reach_the_library(host_as_device, E):
    with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):   # no GPU: it fails at its launch
        call(E, activation="silu")
    with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):
        call(E, U=None, V=None, bias=None, gate=None, residual=None)


@host
@pytest.mark.parametrize("E", [None, 3])
@pytest.mark.parametrize("bad", [
    dict(activation="swish"), dict(activation=None), dict(y_dtype=torch.float16), dict(y_dtype=bf),
    dict(gate=torch.zeros(32, 48, dtype=bf)), dict(gate=torch.zeros(32, 47)), dict(gate=torch.zeros(48, 32).t()),
    dict(residual=torch.zeros(31, 48)), dict(residual=torch.zeros(32 * 48)), dict(out=torch.zeros(32, 40)),
    dict(out=torch.zeros(32, 48, dtype=bf)), dict(bias=torch.zeros(48)), dict(bias=torch.zeros(47, dtype=bf)),
    dict(bias=torch.zeros(2, 48, dtype=bf)), dict(U=None), dict(V=None), dict(U=torch.zeros(48, 8, dtype=bf)),
    dict(values=torch.zeros(1, 2, 64, 8, dtype=bf)), dict(meta=torch.zeros(1, 1, 64, 4, dtype=torch.int32)),
    dict(X=torch.zeros(32, 128, dtype=torch.float16)), dict(X=torch.zeros(32, 128, 1, dtype=bf)),
    dict(X=torch.zeros(32, 256, dtype=bf)[:, ::2]), dict(n_out=64),
])
def test_binding_rejects(host_as_device, E, bad):
    with pytest.raises((ValueError, TypeError)):
        call(E, **bad)


@host
@pytest.mark.parametrize("bad", [
    dict(offsets=torch.zeros(4, dtype=torch.int64)), dict(offsets=torch.zeros(3, dtype=torch.int32)),
    dict(offsets=torch.zeros(1, dtype=torch.int32)), dict(offsets=torch.zeros(2, 2, dtype=torch.int32)),
    dict(offsets=torch.zeros(8, dtype=torch.int32)[::2]), dict(offsets=[0, 1, 2, 3]),
    dict(offsets=torch.zeros(1026, dtype=torch.int32)), dict(U=torch.zeros(48, 16, dtype=bf)),
    dict(V=torch.zeros(3, 32, 128, dtype=bf)), dict(bias=torch.zeros(48, dtype=bf)),
])
def test_experts_binding_rejects(host_as_device, bad):
    with pytest.raises((ValueError, TypeError)):
        call(3, **bad)


@host
@pytest.mark.parametrize("E", [None, 3])
def test_n_out_is_asked_for_when_no_shape_tells_it(host_as_device, E):
    flat = dict(values=layer(E)["values"].flatten(), U=None, V=None, n_out=None)
    with pytest.raises(ValueError, match="n_out"):
        call(E, **flat)
    with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):
        call(E, **dict(flat, n_out=48))


@host
@pytest.mark.parametrize("E", [None, 3])
def test_out_over_other_operands(host_as_device, E):
    d = layer(E)
    for name in ("gate", "residual"):
        with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):   # in place: it reaches its launch
            call(E, **dict(d, out=d[name]))
    both = torch.zeros(33, 48)
    for bad in (dict(gate=both[:32], out=both[1:]), dict(residual=both[1:], out=both[:32]),
                dict(workspace=d["out"].view(-1).view(torch.uint8)),
                dict(y_dtype=bf, gate=None, residual=None, out=d["X"].view(-1)[:32 * 48].view(32, 48))):
        with pytest.raises(binding.SplrError, match="SPLR_ERR_OVERLAP"):
            call(E, **dict(d, **bad))
    # buffers that touch without overlapping
    halves = torch.zeros(64, 48)
    with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):
        call(E, **dict(d, gate=halves[:32], out=halves[32:]))
    with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):
        call(E, **dict(d, gate=halves[32:], out=halves[:32]))
