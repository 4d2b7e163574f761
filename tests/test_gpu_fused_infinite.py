"""Infinite and not-a-number entries of X in the fused and grouped products without a rank-r part. Y's sums run
over the entries that S keeps, so such an entry of X reaches the outputs whose row of S keeps its column, with the
sign of what is kept there, and no other output: not through the zeros that fill S's last tile or the steps past the
last one. The same in every kernel, whatever the number of rows selects. In float32 too, where the kernels multiply
bfloat16 parts: there finite entries above bfloat16's range, and S's own infinities, give what float32 gives."""
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding
from tests._paths import BF16, F32, SIZES

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
LARGE = 3.4e38   # finite in float32, infinite in bfloat16


def weights(n_in, n_out, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    values, meta = binding.prune24_pack((torch.randn(n_out, n_in, generator=g, device="cuda") * 0.05).to(dtype))
    return values, meta, binding.dense_reconstruct(values, meta, None, None, n_out=n_out, n_in=n_in).double()


def rows(M, n_in, dtype, seed):
    """X with one special entry a row in most rows: its first columns, its last 64 in turn, and a middle one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(M, n_in, generator=g, device="cuda").to(dtype)
    columns = [n_in - 32, n_in - 4, 0, n_in - 1, n_in // 2] + list(range(max(0, n_in - 64), n_in))
    special = []
    for m in range(M):
        if m % 7 == 6:
            continue   # a row without one
        special.append((m, columns[m % len(columns)], (INF, -INF, INF, NAN)[m % 4]))
        if dtype == F32 and m % 5 == 4:
            special[-1] = (*special[-1][:2], LARGE if m % 2 else -LARGE)
    return X, special


def want_of(X, S, special):
    """(Y, bound of a float32 sum's error) in float64; special entries where S keeps their column."""
    X = X.double()
    for m, k, v in special:
        if abs(v) == LARGE:
            X[m, k] = v
    want, bound = X @ S.t(), (X.shape[1] + 16) * 2.0 ** -24 * (X.abs() @ S.abs().t())
    for m, k, v in special:
        s = S[:, k]
        assert bool((s != 0).any()) and bool((s == 0).any())
        if abs(v) == LARGE:
            continue
        want[m] = torch.where(s == 0, want[m] - X[m, k] * s, v * torch.sign(s))
    return want, bound


def check(got, want, bound, tag):
    got = got.double()
    finite = torch.isfinite(want)
    wrong = int(((got - want).abs() > bound)[finite].sum()) + int((~torch.isfinite(got))[finite].sum())
    other = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    wrong_special = int(other[~finite].sum())
    print(f"[infinite] {tag}: {wrong} finite and {wrong_special} other entries wrong", flush=True)
    assert wrong == 0 and wrong_special == 0, tag


# M, n_in, n_out: the few-token kernels (16 and 32 tokens, one and two row tiles), 128 x 64 tiles, 256- and 512-row
# tiles; n_in that is 0 and 32 mod 64, and steps that leave the waves' rings part-filled
SINGLE = [(1, 96, 40), (5, 64, 40), (16, 4128, 50), (12, 2112, 130), (16, 96, 8200), (9, 160, 8195), (40, 1056, 1003), (64, 544, 70),
          (20, 2080, 8195), (32, 2112, 8200), (256, 4096, 4096), (250, 4128, 4090), (2000, 1056, 4096),
          (2000, 1024, 4096), (4000, 1056, 4096), (4000, 960, 4098)]
SINGLE += [s[3:6] for s in SIZES if s[1] is None and s[3:6] not in SINGLE]   # every kernel's
TYPES = [BF16, F32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,n_in,n_out", SINGLE)
def test_one_layer(M, n_in, n_out, dtype):
    print(f"[infinite] {M} x {n_in} -> {n_out} {dtype}", flush=True)
    values, meta, S = weights(n_in, n_out, dtype, seed=M)
    for turn in range(4 if M == 1 else 1):
        X, special = rows(M, n_in, dtype, seed=M + turn)
        if M == 1:
            special = [(0, [n_in - 32, n_in - 4, 0, n_in - 1][turn], INF)]
        want, bound = want_of(X, S, special)
        for m, k, v in special:
            X[m, k] = v
        check(binding.linear_fused(X, values, meta, None, None, n_out=n_out), want, bound, f"{M} {n_in} {n_out} {dtype}")


# rows of 4 experts together, n_in, n_out
GROUPED = [(8, 96, 40), (30, 2080, 1000), (64, 96, 4100), (300, 2080, 1032), (700, 1056, 1003), (4000, 1056, 2048),
           (26000, 544, 1024)]
GROUPED += [s[3:6] for s in SIZES if s[1] and s[3:6] not in GROUPED]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,n_in,n_out", GROUPED)
def test_experts(M, n_in, n_out, dtype):
    print(f"[infinite] experts {M} x {n_in} -> {n_out} {dtype}", flush=True)
    ends = [0, M // 3, M // 3, M // 2, M]
    layers = [weights(n_in, n_out, dtype, seed=M + e) for e in range(4)]
    X, special = rows(M, n_in, dtype, seed=M)
    want, bound = torch.empty(M, n_out, dtype=torch.float64, device="cuda"), torch.empty(M, n_out, dtype=torch.float64, device="cuda")
    for e in range(4):
        lo, hi = ends[e], ends[e + 1]
        want[lo:hi], bound[lo:hi] = want_of(X[lo:hi], layers[e][2], [(m - lo, k, v) for m, k, v in special if lo <= m < hi])
    for m, k, v in special:
        X[m, k] = v
    got = binding.linear_experts(X, torch.tensor(ends, dtype=torch.int32, device="cuda"), torch.stack([l[0] for l in layers]),
                                 torch.stack([l[1] for l in layers]), None, None, n_out=n_out)
    check(got, want, bound, f"experts {M} {n_in} {n_out} {dtype}")


# n_in, n_out, rows of X: few tokens, tiles, and in bfloat16 the prefill kernels
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,n_in,n_out", [(3, 96, 40), (40, 1056, 500), (256, 2080, 4100), (2000, 1056, 4096)])
def test_infinite_weights(M, n_in, n_out, dtype):
    """An infinite entry of S makes its output infinite with the sign of X there, and no other output."""
    g = torch.Generator(device="cuda").manual_seed(M)
    R = (torch.randn(n_out, n_in, generator=g, device="cuda") * 0.05).to(dtype)
    at = [(n, (7 * n) % n_in, INF if n % 2 else -INF) for n in range(1, n_out, 9)] + [(n_out - 1, n_in - 1, INF)]
    for n, k, v in at:
        R[n, k] = v   # the largest of its group: kept
    values, meta = binding.prune24_pack(R)
    for n, k, v in at:
        R[n, k] = 0.0
    others = torch.ones(n_out, dtype=torch.bool, device="cuda")
    others[[n for n, _, _ in at]] = False
    S = binding.dense_reconstruct(*binding.prune24_pack(R), None, None, n_out=n_out, n_in=n_in).double()
    X = torch.randn(M, n_in, generator=g, device="cuda").to(dtype)
    X = torch.where(X == 0, torch.ones_like(X), X)
    got = binding.linear_fused(X, values, meta, None, None, n_out=n_out).double()
    for n, k, v in at:
        assert bool((got[:, n] == v * torch.sign(X[:, k].double())).all()), n
    want, bound = X.double() @ S.t(), (n_in + 16) * 2.0 ** -24 * (X.double().abs() @ S.abs().t())
    assert bool(((got - want).abs() <= bound)[:, others].all())


@pytest.mark.parametrize("M,n_in,n_out", [(3, 96, 40), (40, 1056, 500), (300, 2080, 1030)])
def test_infinity_through_the_factors(M, n_in, n_out):
    """float32 with ranks: positive weights and factors carry a positive infinity to the whole row, and only there."""
    g = torch.Generator(device="cuda").manual_seed(M)

    def positive(*shape):
        return torch.rand(*shape, generator=g, device="cuda") + 0.1
    values, meta = binding.prune24_pack(positive(n_out, n_in))
    U, V, X = positive(n_out, 48), positive(48, n_in), positive(M, n_in)
    clean = binding.linear_fused(X, values, meta, U, V, n_out=n_out)
    bad = list(range(0, M, 2))
    for m in bad:
        X[m, (5 * m + n_in - 1) % n_in] = INF
    got = binding.linear_fused(X, values, meta, U, V, n_out=n_out)
    assert bool((got[bad] == INF).all())
    assert torch.equal(got[1::2], clean[1::2])


@pytest.mark.parametrize("scale", [-126, -120, -112, -104])
@pytest.mark.parametrize("M,n_in,n_out", [(3, 96, 40), (300, 2080, 1030)])
def test_tiny_entries(M, n_in, n_out, scale):
    """float32 entries so small that their low parts leave bfloat16's range: its subnormal numbers are 2^-133 apart, so
    an entry is off by 2^-134 at most (2^-133 counted here) and its product by that times the other factor; a product's
    own rounding among float32's subnormal numbers is 2^-150."""
    values, meta, S = weights(n_in, n_out, F32, seed=M)
    values, S = values * 2.0 ** 20, S * 2.0 ** 20
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn(M, n_in, generator=g, device="cuda", dtype=torch.float64).mul(2.0 ** scale).float()
    got = binding.linear_fused(X, values, meta, None, None, n_out=n_out).double()
    x = X.double()
    want, s = x @ S.t(), S.abs().sum(1)[None]
    bound = (n_in + 16) * 2.0 ** -24 * (x.abs() @ S.abs().t()) + 2.0 ** -133 * (s + x.abs().sum(1)[:, None]) + 6 * n_in * 2.0 ** -150
    print(f"[infinite] 2^{scale}: error / bound {float(((got - want).abs() / bound).max()):.3g}", flush=True)
    assert bool(((got - want).abs() <= bound).all())
