"""The fused and grouped products with more than two blocks of 64 ranks and T in more than four K slices, in tiles of
256 and of 512 rows: every entry against float64 products on the device, with the bound of tests/_fused.py."""
import pytest
import torch

from sparse_rank_linear_prune24_amd import binding

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32 = 2.0 ** -24


def normal(g, *shape, std=1.0, to=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)


def want_of(x, S, U, V, bias, gate, residual, y_dtype):
    """silu(z) * gate + residual in float64 and its bound."""
    n_in, r = x.shape[1], V.shape[0]
    x, U, V, bias, gate, residual = (t.double() for t in (x, U, V, bias, gate, residual))
    t = x @ V.t()
    z = x @ S.t() + t @ U.t() + bias
    a = x.abs() @ S.abs().t() + t.abs() @ U.abs().t() + bias.abs()
    d = (n_in * U32 * (x.abs() @ V.abs().t()) + 2.0 ** -17 * t.abs()) @ U.abs().t() + (n_in + 2 * r + 16) * U32 * a
    y, d = z * torch.sigmoid(z) * gate, (1.13 * d + 16 * U32 * z.abs()) * gate.abs()
    d = d + 4 * U32 * (y.abs() + residual.abs())
    y = y + residual
    return y, d + (U32 if y_dtype == F32 else 2.0 ** -8) * (y.abs() + d)


# rows, n_in, n_out, r, experts (0: one layer)
SIZES = [(496, 960, 32768, 144, 0), (300, 960, 43520, 192, 0), (490, 928, 32770, 144, 0), (500, 960, 26112, 144, 2), (500, 960, 26112, 208, 2),
         (500, 1024, 4096, 144, 0), (600, 1024, 4100, 192, 3)]


@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("M,n_in,n_out,r,experts", SIZES)
def test_against_float64(M, n_in, n_out, r, experts, y_dtype):
    print(f"[ranks] {M} x {n_in} -> {n_out} r{r} {experts} experts {y_dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + r)
    E = max(1, experts)
    X, R, bias = normal(g, M, n_in), normal(g, E, n_out, n_in, std=0.05), normal(g, E, n_out)
    U, V = normal(g, E, n_out, r, std=0.2), normal(g, E, r, n_in, std=0.2)
    gate, residual = normal(g, M, n_out, to=y_dtype), normal(g, M, n_out, to=y_dtype)
    packs = [binding.prune24_pack(R[e]) for e in range(E)]
    ends = [0] + [M * (2 * e + 1) // (2 * E) for e in range(1, E)] + [M]
    kw = dict(activation="silu", gate=gate, residual=residual, y_dtype=y_dtype, n_out=n_out)
    for _ in range(3):
        if experts:
            got = binding.linear_experts(X, torch.tensor(ends, dtype=torch.int32, device="cuda"),
                                         torch.stack([p[0] for p in packs]), torch.stack([p[1] for p in packs]), U, V,
                                         bias=bias, **kw)
        else:
            got = binding.linear_fused(X, *packs[0], U[0], V[0], bias=bias[0], **kw)
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            S = binding.dense_reconstruct(*packs[e], None, None, n_out=n_out, n_in=n_in).double()
            y, d = want_of(X[at], S, U[e], V[e], bias[e], gate[at], residual[at], y_dtype)
            wrong = int((~((got[at].double() - y).abs() <= d)).sum())
            assert wrong == 0, (e, wrong)
