"""A mixture of experts as a user builds it: tokens_dispatch, the experts' gated products (compressed or in 8 bits),
tokens_combine, and its gradients. Every stage is held against float64 on what the stage before it gave."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import Weight, floats, held, product64
from tests._fused import HALF_STEP, U32, Weights, check, fused64
from tests.test_gpu_experts import stacked
from tests.test_gpu_fp8 import E4M3, narrow
from tests.test_gpu_tokens import routes, same_bits, sorted64

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32
D, H = 256, 416


def f64(t):
    return t.double().cpu().numpy()


def empty(n, width, dtype=bf):
    """Rows that no expert writes stay NaN: nothing may read them."""
    return torch.full((n, width), float("nan"), dtype=dtype, device="cuda")


class Layer8:
    """Three weights an expert in e4m3, and their transposes in the same blocks for the gradients."""

    def __init__(self, E, seed):
        for i, (name, n_out, n_in) in enumerate((("up", H, D), ("gate", H, D), ("down", D, H))):
            ws = [Weight(n_out, n_in, seed + 10 * e + i, std=0.1) for e in range(E)]
            W = torch.stack([w.W.view(torch.uint8) for w in ws])
            setattr(self, name, (W.view(E4M3), torch.stack([w.s for w in ws])))
            setattr(self, name + "_t", (W.transpose(1, 2).contiguous().view(E4M3),
                                        torch.stack([w.s for w in ws]).transpose(1, 2).contiguous()))
            setattr(self, name + "64", [w.values for w in ws])

    def forward(self, X, ids, weights, E):
        n = ids.numel()
        offsets, positions, rows = binding.tokens_dispatch(ids, E, X, out=empty(n, D))
        up = binding.linear_fp8_experts(rows, offsets, *self.up, y_dtype=bf, out=empty(n, H))
        h = binding.linear_fp8_experts(rows, offsets, *self.gate, activation="silu", gate=up, y_dtype=bf, out=empty(n, H))
        z = binding.linear_fp8_experts(h, offsets, *self.down, y_dtype=bf, out=empty(n, D))
        return offsets, positions, rows, up, h, z, binding.tokens_combine(z, positions, weights, residual=X)

    def backward(self, X, offsets, positions, rows, up, z, weights, dY):
        n = positions.numel()
        dz, dweights = binding.tokens_combine_backward(dY, z, positions, weights, out=empty(n, D))
        dh = binding.linear_fp8_experts(dz, offsets, *self.down_t, y_dtype=bf, out=empty(n, H))
        g = binding.linear_fp8_experts(rows, offsets, *self.gate, y_dtype=bf, out=empty(n, H)).float()
        s = torch.sigmoid(g)
        dup = (dh.float() * (g * s)).to(bf)
        dg = (dh.float() * up.float() * (s * (1 + g * (1 - s)))).to(bf)
        drows = binding.linear_fp8_experts(dup, offsets, *self.up_t, y_dtype=f32, out=empty(n, D, f32))
        binding.linear_fp8_experts(dg, offsets, *self.gate_t, residual=drows, y_dtype=f32, out=drows)
        return dz, dweights, dh, dup, dg, drows, binding.tokens_combine(drows, positions, residual=dY.float())


def by_expert(ends, n, width, of):
    """(want, bound) over the experts' rows, NaN and 0 for rows of no expert."""
    want, bound = np.full((n, width), np.nan), np.zeros((n, width))
    for e in range(len(ends) - 1):
        r = slice(ends[e], ends[e + 1])
        if ends[e] < ends[e + 1]:
            want[r], bound[r] = of(e, r)
    return want, bound


def check_rows(got, want, bound, end, tag):
    check(got[:end], want[:end], bound[:end], tag)
    assert bool(torch.isnan(got[end:].float()).all()), tag


def combine64(z64, positions, weights, residual, dtype):
    """k products and sums in float32, each off by half a step of what it adds to, then Y's type."""
    p = positions.clip(0)
    term = np.where((positions >= 0)[..., None], z64[p] * weights[..., None], 0.0)
    y, a = residual + term.sum(1), np.abs(residual) + np.abs(term).sum(1)
    d = (positions.shape[1] + 2) * U32 * a
    return y, d + HALF_STEP[dtype] * (np.abs(y) + d)


@pytest.mark.parametrize("T,k,E,away", [(1, 2, 4, 0.0), (5, 2, 3, 1.0), (16, 3, 5, 0.2), (333, 2, 6, 0.1), (3000, 2, 4, 0.05)])
def test_8_bit_layer_and_gradients(T, k, E, away):
    layer = Layer8(E, 40)
    ids = routes(T, k, E, away, 41)
    X, x64 = floats((T, D), bf, 42)
    weights, w64 = floats((T, k), f32, 43, std=0.5)
    dY, dy64 = floats((T, D), bf, 44, std=0.1)
    offsets, positions, rows, up, h, z, Y = layer.forward(X, ids, weights, E)
    ends, places = sorted64(ids, E)
    n, end = T * k, int(ends[-1])
    assert np.array_equal(offsets.cpu().numpy(), ends) and np.array_equal(positions.cpu().numpy(), places)
    of = np.zeros(end, np.int64)
    of[places[places >= 0]] = np.nonzero(places >= 0)[0]
    assert np.array_equal(f64(rows[:end]), x64[of])

    def product(x, ws, n_out, n_in, y_dtype, **kw):
        xq = np.zeros((n, n_in))
        xq[:end] = held(f64(x[:end])) if end else 0.0
        thin = narrow(n, n_out, n_in, bf, y_dtype, E)
        return by_expert(ends, n, n_out, lambda e, r: product64(xq[r], ws[e], y_dtype, thin,
                                                               **{a: (b if isinstance(b, str) else b[r]) for a, b in kw.items()}))
    check_rows(up, *product(rows, layer.up64, H, D, bf), end, "up")
    check_rows(h, *product(rows, layer.gate64, H, D, bf, act="silu", gate=f64(up)), end, "gated")
    check_rows(z, *product(h, layer.down64, D, H, bf), end, "down")
    check(Y, *combine64(f64(z), places, w64, x64, bf), "combined")

    dz, dweights, dh, dup, dg, drows, dX = layer.backward(X, offsets, positions, rows, up, z, weights, dY)
    want, bound = np.full((n, D), np.nan), np.zeros((n, D))
    t, j = np.nonzero(places >= 0)
    want[places[t, j]] = w64[t, j][:, None] * dy64[t]
    bound = np.abs(want) * (U32 + HALF_STEP[bf]) * (1 + U32)
    check_rows(dz, want, bound, end, "dz")
    z64 = f64(z)
    dot, size = np.zeros((T, k)), np.zeros((T, k))
    dot[t, j] = (dy64[t] * z64[places[t, j]]).sum(1)
    size[t, j] = np.abs(dy64[t] * z64[places[t, j]]).sum(1)
    check(dweights, dot, (D + 8) * U32 * size, "dweights")
    turned = lambda ws: [w.T for w in ws]  # noqa: E731
    check_rows(dh, *product(dz, turned(layer.down64), H, D, bf), end, "dh")
    first, b1 = product(dup, turned(layer.up64), D, H, f32)
    second, b2 = product(dg, turned(layer.gate64), D, H, f32)
    # the first product, rounded to float32, is added to the second: half a step more of the sum and 4 u of the first
    check_rows(drows, first + second, b1 + b2 + 5 * U32 * (np.abs(first) + np.abs(second)), end, "drows")
    check(dX, *combine64(f64(drows), places, np.ones((T, k)), dy64, f32), "dX")
    for e in range(E):   # the down projection's weight gradient, expert by expert
        a, b = int(ends[e]), int(ends[e + 1])
        if a == b:
            continue
        dq, ds = binding.fp8_quantize(dz[a:b], transposed=True)
        hq, hs = binding.fp8_quantize(h[a:b], transposed=True)
        want, bound = product64(held(f64(dz[a:b]).T), held(f64(h[a:b]).T), f32, False)
        check(binding.linear_fp8(dq, hq, hs, x_scales=ds), want, bound, f"weight gradient of expert {e}")


@pytest.mark.parametrize("T,k,E,away", [(1, 2, 4, 0.0), (40, 3, 5, 0.2), (700, 2, 6, 0.1)])
def test_compressed_layer(T, k, E, away):
    n, r = T * k, 16
    ids = routes(T, k, E, away, 51)
    X, x64 = floats((T, D), bf, 52)
    weights, w64 = floats((T, k), f32, 53, std=0.5)
    ups, gates, downs = ([Weights(a, b, r, "bf16", 54 + 100 * i + e, False) for e in range(E)]
                         for i, (a, b) in enumerate(((D, H), (D, H), (H, D))))
    offsets, positions, rows = binding.tokens_dispatch(ids, E, X, out=empty(n, D))

    def run(x, ws, n_out, **kw):
        d = stacked(ws)
        return binding.linear_experts(x, offsets, d["values"], d["meta"], d["U"], d["V"], y_dtype=bf, n_out=n_out,
                                      out=empty(n, n_out), **kw)
    up = run(rows, ups, H)
    h = run(rows, gates, H, activation="silu", gate=up)
    z = run(h, downs, D)
    Y = binding.tokens_combine(z, positions, weights, residual=X, out=X)   # in place of the layer's input
    ends, places = sorted64(ids, E)
    end = int(ends[-1])
    r64, u64, h64 = f64(rows), f64(up), f64(h)
    check_rows(up, *by_expert(ends, n, H, lambda e, s: fused64(r64[s], ups[e], y_dtype=bf)), end, "up")
    check_rows(h, *by_expert(ends, n, H, lambda e, s: fused64(r64[s], gates[e], "silu", u64[s], y_dtype=bf)), end, "gated")
    check_rows(z, *by_expert(ends, n, D, lambda e, s: fused64(h64[s], downs[e], y_dtype=bf)), end, "down")
    check(Y, *combine64(f64(z), places, w64, x64, bf), "combined")


def test_layer_in_a_graph():
    """One captured step, forward and backward, replayed with other tokens and routes: the bits of the eager step."""
    T, k, E = 96, 2, 5
    layer = Layer8(E, 60)

    def inputs_of(i):
        return (floats((T, D), bf, 61 + i)[0], routes(T, k, E, 0.1 * i, 71 + i), floats((T, k), f32, 81 + i)[0],
                floats((T, D), bf, 91 + i, std=0.1)[0])

    def step(X, ids, weights, dY):
        offsets, positions, rows, up, h, z, Y = layer.forward(X, ids, weights, E)
        return (offsets, positions, Y, *layer.backward(X, offsets, positions, rows, up, z, weights, dY))
    held_in = [t.clone() for t in inputs_of(0)]
    step(*held_in)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        outs = step(*held_in)
    for i in (0, 1, 2, 9, 0):
        new = inputs_of(i)
        for to, t in zip(held_in, new):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = step(*new)
        for a, b in zip(outs, want):
            assert same_bits(a, b), i
