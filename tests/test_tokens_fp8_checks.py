"""Refusals of splr_tokens_*, splr_fp8_quantize and the products with 8-bit weights on the CPU: the C ABI checks its arguments
before any HIP call, and the binding checks every tensor before the C ABI sees a pointer (host tensors stand in for device
tensors there, so those tests are skipped where a GPU is present)."""
import ctypes
import os

import pytest
import torch

from sparse_rank_linear_prune24_amd import binding

OK, NULL, SHAPE, DTYPE, ALIGN, HIP, WORKSPACE, SCRATCH, OVERLAP = range(9)
BIG = 1 << 40
bf, f32, i32, i64, e4m3 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


def at(i):
    """Addresses far apart, never dereferenced."""
    return (i + 1) << 36


MIS16, MIS4 = at(60) + 8, at(61) + 2


def dispatch(ids=at(0), w=8, T=16, k=2, E=4, X=at(1), D=64, dt=1, off=at(2), pos=at(3), Xs=at(4), ws=at(5), wsb=BIG):
    return binding.lib().splr_tokens_dispatch(ids, w, T, k, E, X, D, dt, off, pos, Xs, ws, wsb, None)


def gather(X=at(1), T=16, D=64, dt=1, pos=at(3), k=2, Xs=at(4), rows=32):
    return binding.lib().splr_tokens_gather(X, T, D, dt, pos, k, Xs, rows, None)


def combine(Z=at(0), rows=32, D=64, dt=1, pos=at(1), T=16, k=2, w=at(2), res=at(3), Y=at(4)):
    return binding.lib().splr_tokens_combine(Z, rows, D, dt, pos, T, k, w, res, Y, None)


def backward(dY=at(0), Z=at(1), rows=32, D=64, dt=1, pos=at(2), T=16, k=2, w=at(3), dZ=at(4), dw=at(5)):
    return binding.lib().splr_tokens_combine_backward(dY, Z, rows, D, dt, pos, T, k, w, dZ, dw, None)


def test_dispatch_refusals():
    for name in ("ids", "off", "pos", "X", "Xs"):
        assert dispatch(**{name: None}) == NULL, name
    for kw in (dict(T=-1), dict(T=1 << 24), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(D=0), dict(D=(1 << 20) + 1),
               dict(T=1 << 23, k=64), dict(T=1 << 22, k=32, D=1 << 12)):
        assert dispatch(**kw) == SHAPE, kw
    assert dispatch(w=2) == DTYPE and dispatch(dt=3) == DTYPE and dispatch(dt=-1) == DTYPE
    assert dispatch(X=MIS16) == ALIGN and dispatch(Xs=MIS16) == ALIGN and dispatch(off=MIS4) == ALIGN and dispatch(pos=MIS4) == ALIGN
    assert dispatch(ids=at(0) + 4) == ALIGN and dispatch(ids=at(0) + 2, w=4) == ALIGN
    size = binding.lib().splr_tokens_dispatch_workspace_bytes
    assert size(16, 2, 4) == 0 and size(1 << 16, 2, 64) >= 4 * 64
    for bad in ((-1, 2, 4), (16, 0, 4), (16, 65, 4), (16, 2, 0), (16, 2, 1025), (1 << 24, 1, 4)):
        assert size(*bad) == 0
    need = size(1 << 16, 2, 64)
    assert dispatch(T=1 << 16, E=64, ws=None) == WORKSPACE and dispatch(T=1 << 16, E=64, wsb=need - 1) == WORKSPACE
    assert dispatch(T=1 << 16, E=64, ws=MIS16) == ALIGN
    assert dispatch(Xs=at(1)) == OVERLAP and dispatch(Xs=at(1) + 16 * 64 * 2 - 16) == OVERLAP
    assert dispatch(pos=at(0)) == OVERLAP and dispatch(off=at(3)) == OVERLAP and dispatch(off=at(4) + 16) == OVERLAP
    assert dispatch(T=1 << 16, E=64, ws=at(4)) == OVERLAP


def test_gather_refusals():
    for name in ("X", "pos", "Xs"):
        assert gather(**{name: None}) == NULL, name
    for kw in (dict(T=-1), dict(T=1 << 24), dict(k=0), dict(k=65), dict(D=0), dict(D=(1 << 20) + 1), dict(rows=-1),
               dict(rows=(1 << 28) + 1), dict(rows=1 << 20, D=1 << 17)):
        assert gather(**kw) == SHAPE, kw
    assert gather(dt=3) == DTYPE
    assert gather(X=MIS16) == ALIGN and gather(Xs=MIS16) == ALIGN and gather(pos=MIS4) == ALIGN
    assert gather(Xs=at(1)) == OVERLAP and gather(Xs=at(3)) == OVERLAP
    assert gather(T=0, X=None, pos=None, Xs=None) == OK and gather(rows=0, Xs=None) == OK


def test_combine_refusals():
    for name in ("Z", "pos", "Y"):
        assert combine(**{name: None}) == NULL, name
    for kw in (dict(T=-1), dict(T=1 << 24), dict(k=0), dict(k=65), dict(D=0), dict(D=(1 << 20) + 1), dict(rows=-1)):
        assert combine(**kw) == SHAPE, kw
    assert combine(dt=2) == DTYPE
    for kw in (dict(Z=MIS16), dict(res=MIS16), dict(Y=MIS16), dict(pos=MIS4), dict(w=MIS4)):
        assert combine(**kw) == ALIGN, kw
    for kw in (dict(Y=at(0)), dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(3) + 16), dict(Y=at(3) - 16)):
        assert combine(**kw) == OVERLAP, kw
    assert combine(T=0, Z=None, rows=0, pos=None, w=None, res=None, Y=None) == OK


def test_backward_refusals():
    for name in ("dY", "Z", "pos"):
        assert backward(**{name: None}) == NULL, name
    assert backward(dZ=None, dw=None) == NULL
    for kw in (dict(T=-1), dict(T=1 << 24), dict(k=0), dict(k=65), dict(D=0), dict(rows=-1)):
        assert backward(**kw) == SHAPE, kw
    assert backward(dt=2) == DTYPE
    for kw in (dict(dY=MIS16), dict(Z=MIS16), dict(dZ=MIS16), dict(pos=MIS4), dict(w=MIS4), dict(dw=MIS4)):
        assert backward(**kw) == ALIGN, kw
    for kw in (dict(dZ=at(0)), dict(dZ=at(2)), dict(dZ=at(3)), dict(dZ=at(1) + 16), dict(dw=at(0)), dict(dw=at(1)), dict(dw=at(2)),
               dict(dw=at(3)), dict(dw=at(4))):
        assert backward(**kw) == OVERLAP, kw
    assert backward(T=0) == OK


def quantize(X=at(0), rows=16, cols=64, dt=1, br=1, tr=0, Q=at(1), s=at(2)):
    return binding.lib().splr_fp8_quantize(X, rows, cols, dt, br, tr, Q, s, None)


def test_quantize_refusals():
    for name in ("X", "Q", "s"):
        assert quantize(**{name: None}) == NULL, name
    for kw in (dict(rows=0), dict(cols=0), dict(cols=48), dict(rows=(1 << 24) + 1), dict(cols=(1 << 20) + 32), dict(br=64), dict(br=0),
               dict(rows=1 << 21, cols=1 << 16), dict(tr=1, rows=(1 << 20) + 1)):
        assert quantize(**kw) == SHAPE, kw
    assert quantize(dt=2) == DTYPE
    assert quantize(X=MIS16) == ALIGN and quantize(Q=MIS16) == ALIGN and quantize(s=MIS4) == ALIGN
    assert quantize(Q=at(0)) == OVERLAP and quantize(s=at(0)) == OVERLAP and quantize(s=at(1)) == OVERLAP
    assert quantize(rows=17, tr=1, s=at(1) + 64 * 32 - 4) == OVERLAP   # Q's rows are padded to 32


def ep(act=0, bias=None, gate=None, residual=None):
    return ctypes.byref(binding._Epilogue(act, bias, gate, residual))


def linear(X=at(0), xs=at(1), M=16, K=64, dt=1, W=at(2), s=at(3), br=128, N=32, e=None, yd=1, Y=at(4), ws=at(5), wsb=BIG):
    return binding.lib().splr_linear_fp8(X, xs, M, K, dt, W, s, br, N, e, yd, Y, ws, wsb, None)


def experts(X=at(0), xs=at(1), M=16, K=64, dt=1, off=at(6), E=4, W=at(2), s=at(3), br=128, N=32, e=None, yd=1, Y=at(4), ws=at(5),
            wsb=BIG):
    return binding.lib().splr_linear_fp8_experts(X, xs, M, K, dt, off, E, W, s, br, N, e, yd, Y, ws, wsb, None)


@pytest.mark.parametrize("f", [linear, experts])
def test_product_refusals(f):
    for name in ("X", "W", "s", "Y"):
        assert f(**{name: None}) == NULL, name
    assert f(dt=2, xs=None) == NULL
    for name in ("X", "W", "Y"):
        assert f(**{name: MIS16}) == ALIGN, name
    for kw in (dict(xs=MIS4, dt=2), dict(s=MIS4), dict(e=ep(bias=MIS16)), dict(e=ep(gate=MIS16)), dict(e=ep(residual=MIS16))):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(K=48), dict(K=0), dict(N=0), dict(M=-1), dict(M=1 << 25), dict(N=(1 << 21) + 1), dict(K=(1 << 20) + 32), dict(br=0),
               dict(br=64), dict(e=ep(-1)), dict(e=ep(5))):
        assert f(**kw) == SHAPE, kw
    assert f(dt=3) == DTYPE and f(dt=-1) == DTYPE and f(yd=2) == DTYPE
    for dt in (0, 1, 2):   # Y over an operand; gate and residual only exactly
        for kw in (dict(Y=at(0)), dict(Y=at(2)), dict(Y=at(3)), dict(e=ep(bias=at(4))), dict(e=ep(gate=at(4) + 16)),
                   dict(e=ep(residual=at(4) - 16))):
            assert f(dt=dt, **kw) == OVERLAP, (dt, kw)
    assert f(dt=2, Y=at(1)) == OVERLAP


def test_experts_refusals():
    assert experts(off=None) == NULL and experts(off=MIS4) == ALIGN and experts(Y=at(6)) == OVERLAP
    assert experts(E=0) == SHAPE and experts(E=1025) == SHAPE and experts(E=1024, N=1 << 20, K=1 << 12) == SHAPE
    assert linear(M=0) == SHAPE
    assert experts(M=0, X=None, Y=None, ws=None, wsb=0) == OK
    assert experts(M=0, W=None) == NULL and experts(M=0, K=40) == SHAPE and experts(M=0, dt=7) == DTYPE


def test_product_workspace():
    size = binding.lib().splr_linear_fp8_workspace_bytes
    for bad in ((0, 0, 32, 64, 1, 1), (16, -1, 32, 64, 1, 1), (16, 1025, 32, 64, 1, 1), (16, 0, 0, 64, 1, 1), (16, 0, 32, 48, 1, 1),
                (16, 0, 32, 64, 3, 1), (16, 0, 32, 64, 1, 2)):
        assert size(*bad) == 0
    assert size(8192, 0, 4096, 4096, 2, 1) == 0            # quantised already
    need = size(8192, 0, 4096, 4096, 1, 1)
    if need:
        assert need >= 8192 * 4096
        for kw in (dict(ws=None), dict(wsb=need - 1)):
            assert linear(M=8192, N=4096, K=4096, **kw) == WORKSPACE
        assert linear(M=8192, N=4096, K=4096, ws=MIS16) == ALIGN
        for name in ("X", "W", "s", "Y"):
            assert linear(M=8192, N=4096, K=4096, ws=at({"X": 0, "W": 2, "s": 3, "Y": 4}[name])) == OVERLAP, name
        for e in (ep(bias=at(5)), ep(gate=at(5)), ep(residual=at(5))):
            assert linear(M=8192, N=4096, K=4096, e=e) == OVERLAP
    tile = binding.lib().splr_linear_fp8_tile
    a, b = ctypes.c_int32(), ctypes.c_int32()
    assert tile(16, 0, 32, 64, 1, 1, None, ctypes.byref(b)) == NULL
    assert tile(0, 0, 32, 64, 1, 1, ctypes.byref(a), ctypes.byref(b)) == SHAPE
    assert tile(16, 0, 32, 64, 1, 1, ctypes.byref(a), ctypes.byref(b)) == OK and a.value > 0 and b.value > 0


# ---------------------------------------------------------------------------------------------- the binding
cpu_only = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="host tensors stand in for device tensors")


class _Stream:
    cuda_stream = 0




@pytest.fixture
def host_as_device(monkeypatch):
    monkeypatch.setattr(binding, "_is_device", lambda t: True)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: __import__("contextlib").nullcontext())


def z(*shape, dtype=f32):
    return torch.zeros(shape, dtype=torch.uint8).view(e4m3) if dtype is e4m3 else torch.zeros(shape, dtype=dtype)


def expect(f, good, bad):
    """`good` passes every check and fails at its launch; each of `bad` raises before."""
    with pytest.raises(binding.SplrError, match="SPLR_ERR_HIP"):
        f(**good, stream=_Stream())
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            f(**dict(good, **kw), stream=_Stream())
            pytest.fail(f"accepted {list(kw)}: {[getattr(v, 'shape', v) for v in kw.values()]}")


@cpu_only
def test_binding_of_tokens(host_as_device):
    T, k, E, D = 6, 2, 4, 40
    pos = z(T, k, dtype=i32)
    expect(binding.tokens_dispatch, dict(ids=z(T, k, dtype=i64), n_experts=E, X=z(T, D)), [
        dict(ids=z(T, dtype=i64)), dict(ids=z(T, k)), dict(ids=z(T, 65, dtype=i64)), dict(ids=z(k, T, dtype=i64).t()), dict(n_experts=0),
        dict(n_experts=1025), dict(X=z(T + 1, D)), dict(X=z(T, D, dtype=torch.float16)), dict(X=z(D, T).t()), dict(X=z(T * D)),
        dict(offsets=z(E, dtype=i32)), dict(offsets=z(E + 1, dtype=i64)), dict(positions=z(T, k + 1, dtype=i32)),
        dict(positions=z(T, k, dtype=i64)), dict(out=z(T * k - 1, D)), dict(out=z(T * k, D, dtype=bf)), dict(X=None, out=z(T * k, D)),
        dict(workspace=z(4, 4).t()[1:])])
    expect(binding.tokens_gather, dict(X=z(T, D), positions=pos), [
        dict(positions=z(T - 1, k, dtype=i32)), dict(positions=z(T, k, dtype=i64)), dict(positions=z(T, dtype=i32)), dict(X=z(T, D, dtype=i32)),
        dict(out=z(9, D - 1)), dict(out=z(9, D, dtype=bf)), dict(rows=8, out=z(9, D)), dict(positions=None)])
    expect(binding.tokens_combine, dict(Z=z(T * k, D), positions=pos, weights=z(T, k), residual=z(T, D)), [
        dict(Z=z(T * k, D, dtype=e4m3)), dict(Z=z(T)), dict(positions=z(T, k, dtype=i64)), dict(weights=z(T, k, dtype=bf)),
        dict(weights=z(T, k + 1)), dict(weights=z(k, T).t()), dict(residual=z(T, D, dtype=bf)), dict(residual=z(T + 1, D)),
        dict(out=z(T, D, dtype=bf)), dict(out=z(T, D + 1)), dict(positions=None)])
    expect(binding.tokens_combine_backward, dict(dY=z(T, D), Z=z(T * k, D), positions=pos, weights=z(T, k)), [
        dict(dY=z(T, D, dtype=torch.float16)), dict(dY=z(T + 1, D)), dict(Z=z(T * k, D, dtype=bf)), dict(Z=z(T * k, D + 1)), dict(Z=None),
        dict(positions=z(T, k, dtype=i64)), dict(weights=z(T, k, dtype=bf)), dict(out=z(T * k + 1, D)), dict(out=z(T * k, D, dtype=bf)),
        dict(dweights=z(T, k, dtype=bf)), dict(dweights=z(T, k + 1))])


@cpu_only
def test_binding_of_products(host_as_device):
    M, K, N, E = 9, 160, 200, 3
    expect(binding.fp8_quantize, dict(X=z(M, K)), [
        dict(X=z(M, K, dtype=e4m3)), dict(X=z(K, M).t()), dict(X=z(M)), dict(block_rows=64), dict(out=z(M, K)), dict(out=z(M, K + 32, dtype=e4m3)),
        dict(scales=z(M, 2)), dict(scales=z(2, M, dtype=bf)), dict(transposed=True, out=z(K, M, dtype=e4m3)),
        dict(block_rows=128, scales=z(2, M))])
    W, s = z(N, K, dtype=e4m3), z(2, 2)
    shared = [dict(activation="tanh"), dict(y_dtype=torch.float16), dict(x_scales=z(2, M)), dict(bias=z(N + 1)), dict(gate=z(M, N + 1)),
              dict(residual=z(M, N, dtype=bf)), dict(out=z(M + 1, N)), dict(out=z(M, N, dtype=bf)), dict(workspace=z(4, 4).t()),
              dict(X=z(M, K, dtype=torch.float16)), dict(X=z(M, K, dtype=e4m3)), dict(X=z(K, M).t()), dict(W=None), dict(w_scales=None),
              dict(X=z(M, K, dtype=e4m3), x_scales=z(M, 2))]
    expect(binding.linear_fp8, dict(X=z(M, K), W=W, w_scales=s, bias=z(N), gate=z(M, N), residual=z(M, N)), shared + [
        dict(W=z(N, K)), dict(W=z(N, K - 32, dtype=e4m3)), dict(W=z(1, N, K, dtype=e4m3)), dict(w_scales=z(2, 3)), dict(w_scales=z(N, 2)),
        dict(w_scales=z(2, 2, dtype=bf))])
    expect(binding.linear_fp8, dict(X=z(M, K), W=W, w_scales=z(2, N)), [])
    expect(binding.linear_fp8, dict(X=z(M, K, dtype=e4m3), x_scales=z(2, M), W=W, w_scales=s), [])
    off = z(E + 1, dtype=i32)
    expect(binding.linear_fp8_experts,
           dict(X=z(M, K), offsets=off, W=z(E, N, K, dtype=e4m3), w_scales=z(E, 2, 2), bias=z(E, N), gate=z(M, N), residual=z(M, N)),
           shared + [dict(offsets=None), dict(offsets=z(E, dtype=i32)), dict(offsets=z(E + 1, dtype=i64)), dict(offsets=z(1, dtype=i32)),
                     dict(bias=z(N)), dict(W=W), dict(W=z(E + 1, N, K, dtype=e4m3)), dict(w_scales=s), dict(w_scales=z(E, N, 2))])


def test_every_kernel_has_a_size():
    """The sizes that the GPU tests run take every kernel of the products."""
    from tests.test_gpu_fp8 import EXPERTS, SIZES
    want = {(16, 16), (16, 32), (128, 128), (256, 256)}
    for E in (None, 1):
        for y_dtype in (bf, f32):
            sizes = [(M, n_out, n_in, None) for M, n_in, n_out in SIZES] if E is None else [(M, n_out, n_in, e) for M, e, n_in, n_out in EXPERTS if M]
            tiles = {binding.linear_fp8_tile(M, n_out, n_in, bf, y_dtype, e) for M, n_out, n_in, e in sizes}
            assert tiles == (want if y_dtype is bf else want - {(256, 256)}), (E, y_dtype, tiles)
    # tiles of 128 with two steps in LDS (more of them than CUs) and with four, for both types
    for y_dtype in (bf, f32):
        of = [-(-M // 128) * -(-n_out // 128) for M, n_in, n_out in SIZES if binding.linear_fp8_tile(M, n_out, n_in, bf, y_dtype) == (128, 128)]
        assert min(of) <= 256 < max(of)
    # X quantised by the workgroups (no workspace) and by a launch of its own, by the few-token kernels
    needs = {binding.linear_fp8_workspace_bytes(M, n_out, n_in, bf, bf) > 0 for M, n_in, n_out in SIZES
             if binding.linear_fp8_tile(M, n_out, n_in, bf, bf)[0] == 16}
    assert needs == {True, False}


def test_sizes_that_the_types_share():
    assert binding.SLOTS_MAX == 64 and binding.SPLR_E4M3 == 2
    assert binding.linear_fp8_workspace_bytes(16, 64, 64, e4m3, bf) == 0
