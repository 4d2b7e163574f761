"""The way of tokens to their experts and back (splr_tokens_*) on the GPU, against plain loops and float64 sums."""
import numpy as np
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._fp8 import E4M3
from tests._fused import HALF_STEP, U32

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32

# tokens, slots, experts, columns, type, ids' type, share of slots without an expert
SIZES = [
    (1, 8, 32, 2048, bf, torch.int64, 0.0), (1, 1, 1, 1, f32, torch.int32, 0.0), (3, 1, 2, 7, bf, torch.int32, 1.0),
    (16, 8, 32, 2048, bf, torch.int64, 0.0), (333, 3, 60, 1003, f32, torch.int32, 0.1), (100, 5, 7, 1411, bf, torch.int64, 0.9),
    (341, 3, 5, 40, f32, torch.int32, 0.0), (342, 3, 5, 40, f32, torch.int32, 0.0),        # 1023 and 1026 slots: one workgroup, two
    (32, 8, 1024, 128, bf, torch.int32, 0.1), (33, 8, 9, 128, bf, torch.int32, 0.0), (37, 2, 12, 5000, f32, torch.int64, 0.1),
    (8193, 2, 8, 24, bf, torch.int32, 0.0),                                                # the most slots of one launch are 16384
    (2048, 2, 1024, 72, bf, torch.int64, 0.3), (4097, 1, 256, 100, bf, torch.int32, 0.0), (700, 64, 300, 33, bf, torch.int32, 0.2),
    (8192, 2, 8, 512, bf, torch.int64, 0.0), (20011, 3, 1024, 8, f32, torch.int64, 0.05),
]
IDS = ["-".join(str(x).replace("torch.", "") for x in s) for s in SIZES]


def routes(T, k, E, away, seed, dtype=torch.int64):
    """ids [T][k], with ids past the experts and repeated ones among them."""
    g = np.random.Generator(np.random.PCG64(seed))
    ids = np.minimum((g.random((T, k)) ** 1.5 * E).astype(np.int64), E - 1)
    gone = g.random((T, k)) < away
    bad = np.array([-1, E, E + 5, -(1 << 31), (1 << 31) - 1])
    ids = np.where(gone, bad[g.integers(0, len(bad), (T, k))], ids)
    return torch.from_numpy(ids).to(dtype).cuda()


def sorted64(ids, E):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    here = (flat >= 0) & (flat < E)
    offsets = np.array([np.sum(here & (flat < e)) for e in range(E + 1)])
    positions, at = np.full(flat.size, -1), offsets.copy()
    for i in np.nonzero(here)[0]:
        positions[i] = at[flat[i]]
        at[flat[i]] += 1
    return offsets, positions.reshape(ids.shape)


def rows(n, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, D, generator=g).to(dtype).cuda()


def same_bits(a, b):
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(kind), b.view(kind))


@pytest.mark.parametrize("T,k,E,D,dtype,id_type,away", SIZES, ids=IDS)
def test_dispatch(T, k, E, D, dtype, id_type, away):
    ids, X = routes(T, k, E, away, 1, id_type), rows(T, D, dtype, 2)
    out = torch.full((T * k, D), -7.0, dtype=dtype, device="cuda")
    offsets, positions, Xs = binding.tokens_dispatch(ids, E, X, out=out)
    assert Xs is out
    want_o, want_p = sorted64(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), want_o)
    assert np.array_equal(positions.cpu().numpy(), want_p)
    want = torch.full((T * k, D), -7.0, dtype=dtype)   # rows behind the last expert's stay
    here = want_p.reshape(-1) >= 0
    want[want_p.reshape(-1)[here]] = X.cpu()[np.nonzero(here)[0] // k]
    assert torch.equal(out.cpu(), want)
    # the routing alone, and the rows alone
    o2, p2, none = binding.tokens_dispatch(ids, E)
    assert none is None and torch.equal(o2, offsets) and torch.equal(p2, positions)
    out2 = torch.full_like(out, -7.0)
    binding.tokens_gather(X, positions, out=out2)
    assert torch.equal(out2, out)


@pytest.mark.parametrize("D", [1, 16, 100, 4096])
def test_rows_of_8_bits(D):
    T, k, E = 50, 3, 6
    ids = routes(T, k, E, 0.2, 3)
    X = torch.randint(0, 256, (T, D), dtype=torch.uint8).view(E4M3).cuda()
    out = torch.zeros(T * k, D, dtype=torch.uint8, device="cuda").view(E4M3)
    _, positions, _ = binding.tokens_dispatch(ids, E, X, out=out)
    p = positions.cpu().numpy().reshape(-1)
    want = torch.zeros(T * k, D, dtype=torch.uint8)
    want[p[p >= 0]] = X.cpu().view(torch.uint8)[np.nonzero(p >= 0)[0] // k]
    assert torch.equal(out.cpu().view(torch.uint8), want)


def combined64(Z, positions, weights, residual):
    """(Y, bound): at most one rounding for each of the slots' products and sums, and the store's."""
    p, T, k = positions.cpu().numpy(), *positions.shape
    Z = Z.double().cpu().numpy()
    w = np.ones((T, k)) if weights is None else weights.double().cpu().numpy()
    y = np.zeros((T, Z.shape[1])) if residual is None else residual.double().cpu().numpy()
    a = np.abs(y)
    for j in range(k):
        here = (p[:, j] >= 0) & (p[:, j] < Z.shape[0])
        t = np.nonzero(here)[0]
        y[t] += w[t, j, None] * Z[p[t, j]]
        a[t] += np.abs(w[t, j, None] * Z[p[t, j]])
    return y, (k + 2) * U32 * a


def near(got, want, bound, tag):
    got, dtype = got.double().cpu().numpy(), got.dtype
    bound = bound + HALF_STEP[dtype] * (np.abs(want) + bound)
    worst = float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300))) if got.size else 0.0
    assert np.all(np.isfinite(got)) and worst <= 1.0, f"{tag}: {worst:.3f} of the bound"


@pytest.mark.parametrize("T,k,E,D,dtype,id_type,away", SIZES, ids=IDS)
def test_combine_and_its_gradient(T, k, E, D, dtype, id_type, away):
    _, positions, _ = binding.tokens_dispatch(routes(T, k, E, away, 4, id_type), E)
    Z, weights, residual, dY = rows(T * k, D, dtype, 5), torch.rand(T, k).cuda(), rows(T, D, dtype, 6), rows(T, D, dtype, 7)
    for w, r in ((weights, residual), (weights, None), (None, None)):
        want, bound = combined64(Z, positions, w, r)
        near(binding.tokens_combine(Z, positions, w, residual=r), want, bound, f"combine {w is None} {r is None}")
    out = residual.clone()
    binding.tokens_combine(Z, positions, weights, residual=out, out=out)   # in place
    assert torch.equal(out, binding.tokens_combine(Z, positions, weights, residual=residual))

    dZ0 = torch.full((T * k, D), -3.0, dtype=dtype, device="cuda")
    dZ, dw = binding.tokens_combine_backward(dY, Z, positions, weights, out=dZ0)
    p, y64, z64, w64 = positions.cpu().numpy(), dY.double().cpu().numpy(), Z.double().cpu().numpy(), weights.double().cpu().numpy()
    want, want_w, bound_w = np.full((T * k, D), -3.0), np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        t = np.nonzero(p[:, j] >= 0)[0]
        want[p[t, j]] = w64[t, j, None] * y64[t]
        want_w[t, j] = np.sum(y64[t] * z64[p[t, j]], axis=1)
        bound_w[t, j] = (D + 2) * U32 * np.sum(np.abs(y64[t] * z64[p[t, j]]), axis=1)
    near(dZ, want, U32 * np.abs(want), "dZ")
    near(dw, want_w, bound_w, "dw")
    inplace = Z.clone()
    dZ2, dw2 = binding.tokens_combine_backward(dY, inplace, positions, weights, out=inplace)   # over Z itself
    assert torch.equal(dw2, dw)
    named = torch.from_numpy(np.isin(np.arange(T * k), p)).cuda()
    assert torch.equal(dZ2[named], dZ[named]) and torch.equal(dZ2[~named], Z[~named])
    zeros, _ = binding.tokens_combine_backward(dY, Z, positions, weights)   # a new one starts as zeros
    assert torch.equal(zeros[named], dZ[named]) and not zeros[~named].any()


@pytest.mark.parametrize("D", [96, 1003])
def test_gradients_against_differences(D):
    """combine and gather are linear in each operand, so a difference is the operator of the difference itself:
    <dY, combine(Z + E) - combine(Z)> = <dY, combine(E)> has to be <dZ, E>, and so for the weights and for gather."""
    T, k, E = 37, 4, 9
    _, positions, _ = binding.tokens_dispatch(routes(T, k, E, 0.2, 8), E)
    Z, dY, dXs, X = rows(T * k, D, f32, 9), rows(T, D, f32, 10), rows(T * k, D, f32, 11), rows(T, D, f32, 12)
    weights, step_w, step = torch.rand(T, k).cuda(), torch.randn(T, k).cuda(), rows(T * k, D, f32, 13)

    def dot(a, b):
        return float((a.double() * b.double()).sum()), float((a.double() * b.double()).abs().sum())

    dZ, dw = binding.tokens_combine_backward(dY, Z, positions, weights)
    pairs = [(dot(dZ, step), dot(dY, binding.tokens_combine(step, positions, weights))),
             (dot(dw, step_w), dot(dY, binding.tokens_combine(Z, positions, step_w)))]
    Xs = torch.zeros(T * k, D, device="cuda")
    binding.tokens_gather(X, positions, out=Xs)
    pairs.append((dot(binding.tokens_combine(dXs, positions), X), dot(dXs, Xs)))
    for (a, size), (b, _) in pairs:
        assert abs(a - b) <= (D + 16) * U32 * size   # each side a float32 sum of D or k terms, then float64


def test_infinite_rows_reach_their_own_token_only():
    T, k, D = 6, 2, 72
    _, positions, _ = binding.tokens_dispatch(torch.tensor([[0, 1], [1, -1], [0, 2], [-1, -1], [2, 2], [1, 0]]).cuda(), 3)
    Z, weights = rows(T * k, D, bf, 14), torch.rand(T, k).cuda()
    total = int((positions >= 0).sum())
    Z[total:] = float("nan")                       # behind the last expert's rows
    Z[positions[2, 1]] = float("inf")
    weights[3] = float("nan")                      # of slots without a row
    Y = binding.tokens_combine(Z, positions, weights)
    assert torch.isinf(Y[2]).all() and torch.isfinite(Y[[0, 1, 3, 4, 5]]).all()
    assert not Y[3].any()                          # no slot has a row
    dZ, dw = binding.tokens_combine_backward(rows(T, D, bf, 15), Z, positions, weights)
    assert not dw[3].any() and torch.isfinite(dw[[0, 1, 3, 4, 5]]).all() and not dZ[total:].any()
    # positions that lie outside the rows count as none
    wild = positions.clone()
    wild[0, 0], wild[1, 0] = T * k, -(1 << 31)
    Y = binding.tokens_combine(Z, wild, weights)
    want = weights[0, 1] * Z[positions[0, 1]].float()
    assert torch.equal(Y[0], want.to(bf)) and not Y[1].any()
    out = torch.zeros(total, D, dtype=bf, device="cuda")
    wild[5, 0] = total                              # one past a shorter buffer
    binding.tokens_gather(rows(T, D, bf, 16), wild, out=out)
    binding.tokens_combine_backward(rows(T, D, bf, 17), out, wild, weights)


def test_no_tokens_and_no_rows():
    ids = torch.empty(0, 4, dtype=torch.int64, device="cuda")
    offsets = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    _, positions, Xs = binding.tokens_dispatch(ids, 5, torch.empty(0, 64, device="cuda"), offsets=offsets)
    assert not offsets.any() and positions.shape == (0, 4) and Xs.shape == (0, 64)
    assert binding.tokens_combine(Xs, positions).shape == (0, 64)
    # tokens whose slots are all elsewhere, and no rows at all
    positions = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    residual = rows(3, 64, f32, 18)
    assert torch.equal(binding.tokens_combine(Xs, positions, torch.rand(3, 4).cuda(), residual=residual), residual)
    dZ, dw = binding.tokens_combine_backward(residual, Xs, positions)
    assert dZ.shape == (0, 64) and not dw.any()


def test_offsets_past_31_bits():
    """Rows of 2^20 columns: the last ones lie past 2^31 entries."""
    T, k, D = 1100, 2, 1 << 20
    ids = torch.stack((torch.arange(T) % 2, torch.full((T,), -1)), 1).cuda()
    X = torch.zeros(T, D, dtype=bf, device="cuda")
    X[:, ::4099] = torch.arange(T, device="cuda")[:, None] % 251 - 125.0
    offsets, positions, Xs = binding.tokens_dispatch(ids, 2, X)
    assert offsets.tolist() == [0, T // 2, T]
    at = positions[:, 0].long()
    for t in (0, 1, 549, 1098, 1099):
        assert torch.equal(Xs[at[t]], X[t])
    Xs[T] = 1.0                                    # rows T .. 2 T - 1 lie past 2^30 entries, the last past 2^31
    positions[5, 1], positions[6, 1] = T, 2 * T - 1
    Xs[2 * T - 1] = 2.0
    weights = torch.ones(T, k, device="cuda")
    Y = binding.tokens_combine(Xs, positions, weights)
    assert torch.equal(Y[5], (X[5].float() + 1).to(bf)) and torch.equal(Y[6], (X[6].float() + 2).to(bf)) and torch.equal(Y[9], X[9])
    _, dw = binding.tokens_combine_backward(Y, Xs, positions, weights, out=Xs)
    assert torch.equal(Xs[2 * T - 1], Y[6])
    assert float(dw[6, 1]) == pytest.approx(float(2 * Y[6].double().sum()), rel=1e-4)


def test_streams_graphs_and_replays():
    T, k, E, D = 9000, 2, 12, 256
    ids, X, weights = routes(T, k, E, 0.1, 20), rows(T, D, bf, 21), torch.rand(T, k).cuda()
    out, Y = torch.zeros(T * k, D, dtype=bf, device="cuda"), torch.zeros(T, D, dtype=bf, device="cuda")
    offsets, positions = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    need = binding.lib().splr_tokens_dispatch_workspace_bytes(T, k, E)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    dZ, dw = torch.zeros_like(out), torch.zeros(T, k, device="cuda")

    def run(stream=None):
        binding.tokens_dispatch(ids, E, X, offsets=offsets, positions=positions, out=out, workspace=ws, stream=stream)
        binding.tokens_combine(out, positions, weights, out=Y, stream=stream)
        binding.tokens_combine_backward(Y, out, positions, weights, out=dZ, dweights=dw, stream=stream)
        return [t.clone() for t in (offsets, positions, out, Y, dZ, dw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.tokens_dispatch(ids, E, X, offsets=offsets, positions=positions, out=out, workspace=ws)
        binding.tokens_combine(out, positions, weights, out=Y)
        binding.tokens_combine_backward(Y, out, positions, weights, out=dZ, dweights=dw)
    for seed in range(4):
        ids.copy_(routes(T, k, E, 0.1 * seed, 30 + seed))
        X.copy_(rows(T, D, bf, 40 + seed))
        for t in (out, dZ):
            t.zero_()
        want = run()
        for t in (offsets, positions, out, Y, dZ, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((offsets, positions, out, Y, dZ, dw), want):
            assert torch.equal(a, b)
    # a stream given as an argument
    torch.cuda.synchronize()
    for t in (out, dZ):
        t.zero_()
    torch.cuda.synchronize()
    binding.tokens_dispatch(ids, E, X, offsets=offsets, positions=positions, out=out, workspace=ws, stream=side)
    binding.tokens_combine(out, positions, weights, out=Y, stream=side)
    side.synchronize()
    assert torch.equal(out, want[2]) and torch.equal(Y, want[3])
