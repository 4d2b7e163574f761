"""Cases that measure the way of tokens to their experts and back, and the products with weights held in
8-bit floating point (e4m3) with a scale for each block of 128.

    tokens_dispatch          rows of X sorted by the expert that each token's slots chose, group offsets on the device
    tokens_combine           Y[t] = residual[t] + sum_j w[t][j] Z[positions[t][j]]
    tokens_combine_backward  dZ[positions[t][j]] = w[t][j] dY[t],  dw[t][j] = <dY[t], Z[positions[t][j]]>
    linear_fp8               Y = act(X W^T + bias) * gate + residual, W in e4m3 with a scale for each 128 x 128
                             block, X quantised in the call with a scale for each row and 128 columns
    linear_fp8_experts       the same for rows grouped by expert
    fp8_weight_gradient      dW = dY^T X, both quantised with a scale for each column and 128 rows

A block's scale is s = max(largest finite magnitude / 448, 2^-126), its entries are held as e4m3(x (1 / s)), every step
rounded to float32. Slots whose id is outside 0 .. experts - 1 chose no expert here: position -1, no row. Where `own` is false,
run() computes the operators with elementary torch operations in float32; where it is true, it calls the framework.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "i32": torch.int32, "i64": torch.int64}
E4M3 = torch.float8_e4m3fn


def _tokens(name, op, tokens, slots, experts, dim, dtype, ids="i64", away=0.0, residual=False, skew=0.0):
    case = dict(op=op, tokens=tokens, slots=slots, experts=experts, dim=dim, dtype=dtype, ids=ids, away=away, residual=residual,
                skew=skew)
    return dict(case, name=name) if name else case


def _product(name, op, rows, n_in, n_out, x, y, act="none", bias=False, gate=False, residual=False, experts=1, skew=0.0):
    case = dict(op=op, rows=rows, n_in=n_in, n_out=n_out, x=x, y=y, act=act, bias=bias, gate=gate, residual=residual,
                experts=experts, skew=skew)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token's way to 8 of 32 small experts in decoding: pure latency
        _tokens("dispatch one token", "tokens_dispatch", 1, 8, 32, 2048, "bf16"),
        # a prefill's tokens, each to 2 of 8 large experts
        _tokens("dispatch 8192 tokens", "tokens_dispatch", 8192, 2, 8, 4096, "bf16"),
        # a decode batch back onto the residual stream
        _tokens("combine 16 tokens", "tokens_combine", 16, 8, 32, 2048, "bf16", residual=True),
        # a prefill over 60 uneven experts of which some are on another card, odd row length, float32
        _tokens("combine uneven float32", "tokens_combine", 2500, 4, 60, 1411, "fp32", ids="i32", away=0.25, skew=0.5),
        # the gradient of a small fine-tuning batch, odd sizes
        _tokens("combine backward 333 tokens", "tokens_combine_backward", 333, 3, 60, 1003, "fp32", ids="i32", away=0.1, skew=0.5),
        # the gradient of a full training sequence
        _tokens("combine backward 8192 tokens", "tokens_combine_backward", 8192, 2, 8, 4096, "bf16"),
        # one token's attention output projection added to the residual stream: pure latency
        _product("8-bit one token", "linear_fp8", 1, 4096, 4096, "bf16", "bf16", bias=True, residual=True),
        # the block's gate projection at its full prefill length, times the up projection's output: the largest case
        _product("8-bit gated 8192 tokens", "linear_fp8", 8192, 4096, 14336, "bf16", "bf16", act="silu", gate=True),
        # no size a multiple of a tile, a tail of 32 columns, an odd row length, float32 on both sides
        _product("8-bit odd sizes", "linear_fp8", 333, 1056, 1003, "fp32", "fp32", act="gelu", bias=True),
        # the weight gradient of an attention projection over a calibration segment
        _product("8-bit weight gradient", "fp8_weight_gradient", 2048, 4096, 4096, "bf16", "fp32"),
        # a decode batch of 8 tokens, each to 8 of 32 small experts: two rows an expert, some with none
        _product("8-bit experts 64 rows", "linear_fp8_experts", 64, 2048, 1024, "bf16", "bf16", act="silu", gate=True, experts=32),
        # a prefill over few large experts, unevenly loaded
        _product("8-bit experts 8192 rows", "linear_fp8_experts", 8192, 4096, 4096, "bf16", "bf16", act="silu", gate=True, experts=8,
                 skew=0.5),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.45:
        op = rng.choice(("tokens_dispatch", "tokens_combine", "tokens_combine_backward"))
        experts = log(2, 256)
        while True:
            tokens, slots, dim = log(1, 16384), rng.randint(1, min(8, experts)), log(200, 8192)
            dim -= 0 if rng.random() < 0.3 else dim % 32
            if tokens * slots * dim <= 1 << 27:
                break
        return _tokens(None, op, tokens, slots, experts, dim, rng.choice(("bf16", "bf16", "fp32")), rng.choice(("i32", "i64")),
                       round(rng.choice((0.0, 0.0, 0.25, 0.9)), 2), rng.random() < 0.5, round(rng.choice((0.0, 0.5, 1.0)), 1))
    op = rng.choice(("linear_fp8", "linear_fp8", "linear_fp8_experts", "linear_fp8_experts", "fp8_weight_gradient"))
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    x, y = rng.choice(("bf16", "bf16", "fp32")), rng.choice(("bf16", "fp32"))
    bias, gate, residual = (rng.random() < 0.5 for _ in range(3))
    while True:
        n_in, n_out = 32 * log(8, 448), log(200, 14336)
        n_out -= 0 if rng.random() < 0.3 else n_out % 16
        e = log(2, 64) if op == "linear_fp8_experts" else 1
        rows = log(1, 16384 if e > 1 else 8192)
        if e * n_in * n_out <= 1 << 28 and rows * n_in * n_out <= 1 << 38:
            break
    if op == "fp8_weight_gradient":
        return _product(None, op, rows, n_in, n_out, x, y)
    return _product(None, op, rows, n_in, n_out, x, y, act, bias, gate, residual, e, round(rng.choice((0.0, 0.5, 1.0)), 1) if e > 1 else 0.0)


def _blocks(n):
    return (n + 127) // 128


def _quantised(x):
    """e4m3 entries and scales of x [..., n] with a scale for each 128 entries of the last dimension, as float32 values."""
    n = x.shape[-1]
    f = torch.nn.functional.pad(x.float(), (0, -n % 128)).unflatten(-1, (-1, 128))
    s = (f.abs().amax(-1).double() / 448.0).float().clamp(min=2.0 ** -126)
    q = (f * (1.0 / s.double()).float()[..., None]).to(E4M3)
    return q.flatten(-2)[..., :n], s


def _token_inputs(case, seed):
    """A router's choices: the best `slots` of random scores with a spread of popularity over the experts, some of them on another card."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, k, E, D, dt = case["tokens"], case["slots"], case["experts"], case["dim"], TYPES[case["dtype"]]

    def normal(*shape, to=dt):
        return torch.randn(*shape, generator=g, device="cuda").to(to)

    score = normal(T, E, to=torch.float32) + case["skew"] * normal(E, to=torch.float32)
    best = score.topk(k, dim=1)
    gone = torch.rand(T, k, generator=g, device="cuda") < case["away"]
    ids = torch.where(gone, -1, best.indices).to(TYPES[case["ids"]])
    d = dict(ids=ids, weights=torch.softmax(best.values, 1), experts=E)
    if case["op"] == "tokens_dispatch":
        d["X"] = normal(T, D)
        return d
    _, d["positions"] = _sorted(ids, E)
    d["Z"] = normal(T * k, D)
    if case["op"] == "tokens_combine":
        d["residual"] = normal(T, D) if case["residual"] else None
    else:
        d["dY"] = normal(T, D)
    return d


def _sorted(ids, experts):
    """(offsets [experts + 1], positions [T][k]) int32 of the stable sort by expert."""
    flat = ids.reshape(-1).long()
    here = (flat >= 0) & (flat < experts)
    by, order = torch.sort(torch.where(here, flat, experts), stable=True)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device="cuda"))
    at = torch.empty_like(order)
    at[order] = torch.arange(flat.numel(), device="cuda")
    return offsets.to(torch.int32), torch.where(here, at, -1).to(torch.int32).view(ids.shape)


def _weight(g, n_experts, n_out, n_in):
    """e4m3 weights [E, n_out, n_in] and the scales of their 128 x 128 blocks."""
    W = torch.randn(n_experts, n_out, n_in, generator=g, device="cuda") * 0.02
    W[:, :, torch.randperm(n_in, generator=g, device="cuda")[:4]] *= 8.0   # a few channels of larger weights
    nb, kb = _blocks(n_out), _blocks(n_in)
    f = torch.nn.functional.pad(W, (0, kb * 128 - n_in, 0, nb * 128 - n_out)).view(n_experts, nb, 128, kb, 128)
    s = (f.abs().amax((2, 4)).double() / 448.0).float().clamp(min=2.0 ** -126)
    q = (f * (1.0 / s.double()).float()[:, :, None, :, None]).to(E4M3)
    return q.view(n_experts, nb * 128, kb * 128)[:, :n_out, :n_in].contiguous(), s


def _product_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    xt, yt = TYPES[case["x"]], TYPES[case["y"]]
    rows, n_in, n_out, E = case["rows"], case["n_in"], case["n_out"], case["experts"]

    def normal(*shape, std=1.0, to=yt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)

    X = torch.randn(rows, n_in, generator=g, device="cuda")
    X[:, torch.randperm(n_in, generator=g, device="cuda")[:8]] *= 20.0   # activations have outlier channels
    d = dict(X=X.to(xt))
    if case["op"] == "fp8_weight_gradient":
        d["dY"] = normal(rows, n_out, std=1e-3, to=xt)
        return d
    d["W"], d["scales"] = _weight(g, E, n_out, n_in)
    d["bias"] = normal(E, n_out, std=0.2) if case["bias"] else None
    d["gate"] = normal(rows, n_out) if case["gate"] else None
    d["residual"] = normal(rows, n_out) if case["residual"] else None
    if case["op"] == "linear_fp8_experts":
        # a router's choices: every row picks an expert by weights of the given spread, rows sorted by expert
        w = torch.exp(case["skew"] * torch.randn(E, generator=g, device="cuda"))
        chosen = torch.multinomial(w, rows, replacement=True, generator=g)
        counts = torch.bincount(chosen, minlength=E)
        d["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0))).to(torch.int32)
        d["capacity"] = max(1, int(counts.max()))
    return d


def prepare(case, seed):
    """Inputs, and the buffers that a program which calls in a loop keeps."""
    if case["op"].startswith("tokens"):
        s = dict(_token_inputs(case, seed), op=case["op"])
        T, k, D, dt = case["tokens"], case["slots"], case["dim"], TYPES[case["dtype"]]
        if case["op"] == "tokens_combine":
            s["out"] = torch.zeros(T, D, dtype=dt, device="cuda")
        else:
            s["out"] = torch.zeros(T * k, D, dtype=dt, device="cuda")
        if case["op"] == "tokens_dispatch":
            s["offsets"] = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
            s["positions"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
            s["workspace"] = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
        return s
    s = dict(_product_inputs(case, seed), op=case["op"], act=case["act"], y=TYPES[case["y"]], experts=case["experts"])
    rows, n_in, n_out = case["rows"], case["n_in"], case["n_out"]
    if case["op"] == "fp8_weight_gradient":
        s["out"] = torch.empty(n_out, n_in, dtype=s["y"], device="cuda")
        return s
    s["out"] = torch.empty(rows, n_out, dtype=s["y"], device="cuda")
    s["workspace"] = torch.empty(rows * n_in * 2 + (1 << 20), dtype=torch.uint8, device="cuda")
    if case["op"] == "linear_fp8":
        s.update(W=s["W"][0], scales=s["scales"][0], bias=None if s["bias"] is None else s["bias"][0])
    else:
        s["Wt"] = s["W"].transpose(1, 2).contiguous()   # the plain product's order
    return s


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _spread(s, n, dim):
    """Block scales over the n entries of `dim` that they hold for."""
    return s.repeat_interleave(128, dim).narrow(dim, 0, n)


def _values(x):
    """x as its quantisation holds it, float32."""
    q, s = _quantised(x)
    return q.float() * _spread(s, x.shape[-1], x.dim() - 1)


def _plain_dispatch(s):
    offsets, positions = _sorted(s["ids"], s["experts"])
    N, k = positions.numel(), positions.shape[1]
    at = positions.reshape(-1).long()
    token = torch.zeros(N + 1, dtype=torch.long, device="cuda")
    token[torch.where(at < 0, N, at)] = torch.arange(N, device="cuda") // k
    filled = torch.arange(N, device="cuda") < offsets[-1]
    return offsets, positions, torch.where(filled[:, None], s["X"][token[:N]], s["out"])


def _plain_combine(s):
    at = s["positions"].long()
    z = s["Z"].float()[at.clamp(min=0)] * s["weights"][..., None]
    y = torch.where((at >= 0)[..., None], z, torch.zeros((), device="cuda")).sum(1)
    return y if s["residual"] is None else y + s["residual"].float()


def _plain_combine_backward(s):
    at, P = s["positions"].long(), s["Z"].shape[0]
    dy = s["dY"].float()[:, None, :]
    dw = torch.where(at >= 0, (dy * s["Z"].float()[at.clamp(min=0)]).sum(-1), 0.0)
    dz = torch.cat((s["out"], s["out"][:1]))
    dz[torch.where(at < 0, P, at)] = (s["weights"][..., None] * dy).to(dz.dtype)
    return dz[:P], dw


def _plain_linear(s):
    n_out, n_in = s["W"].shape
    w = s["W"].float() * _spread(_spread(s["scales"], n_out, 0), n_in, 1)
    z = _values(s["X"]) @ w.t()
    return z if s["bias"] is None else z + s["bias"].float()


def _plain_experts(s):
    (rows, n_in), E, cap = s["X"].shape, s["experts"], s["capacity"]
    n_out = s["Wt"].shape[2]
    row = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True)
    at = expert * cap + row - s["offsets"].long()[expert]
    x = torch.zeros(E * cap, n_in, device="cuda")
    x[at] = _values(s["X"])
    w = s["Wt"].float() * _spread(_spread(s["scales"].transpose(1, 2).contiguous(), n_in, 1), n_out, 2)
    z = torch.bmm(x.view(E, cap, -1), w).view(E * cap, -1)[at]
    return z if s["bias"] is None else z + s["bias"].float()[expert]


def _own(s):
    from sparse_rank_linear_prune24_amd import binding

    op = s["op"]
    if op == "tokens_dispatch":
        return binding.tokens_dispatch(s["ids"], s["experts"], s["X"], offsets=s["offsets"], positions=s["positions"], out=s["out"],
                                       workspace=s["workspace"])
    if op == "tokens_combine":
        return binding.tokens_combine(s["Z"], s["positions"], s["weights"], residual=s["residual"], out=s["out"])
    if op == "tokens_combine_backward":
        return binding.tokens_combine_backward(s["dY"], s["Z"], s["positions"], s["weights"], out=s["out"])
    if op == "fp8_weight_gradient":
        dy, dy_scales = binding.fp8_quantize(s["dY"], transposed=True)
        x, x_scales = binding.fp8_quantize(s["X"], transposed=True)
        return binding.linear_fp8(dy, x, x_scales, x_scales=dy_scales, y_dtype=s["y"], out=s["out"])
    kw = dict(bias=s["bias"], activation=s["act"], gate=s["gate"], residual=s["residual"], y_dtype=s["y"], out=s["out"],
              workspace=s["workspace"])
    if op == "linear_fp8":
        return binding.linear_fp8(s["X"], s["W"], s["scales"], **kw)
    return binding.linear_fp8_experts(s["X"], s["offsets"], s["W"], s["scales"], **kw)


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "tokens_dispatch":
        return _plain_dispatch(s)
    if op == "tokens_combine":
        return _plain_combine(s).to(s["out"].dtype)
    if op == "tokens_combine_backward":
        return _plain_combine_backward(s)
    if op == "fp8_weight_gradient":
        return (_values(s["dY"].t().contiguous()) @ _values(s["X"].t().contiguous()).t()).to(s["y"])
    y = _act(_plain_linear(s) if op == "linear_fp8" else _plain_experts(s), s["act"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["y"])


def work(case):
    if case["op"].startswith("tokens"):
        T, E, b = case["tokens"], case["experts"], 2 if case["dtype"] == "bf16" else 4
        N, row = T * case["slots"], case["dim"] * b
        kept = N * (1.0 - case["away"])
        if case["op"] == "tokens_dispatch":
            return {"bytes": T * row + kept * row + N * (4 if case["ids"] == "i32" else 8) + 4 * N + 4 * (E + 1), "flops": 0}
        if case["op"] == "tokens_combine":
            return {"bytes": kept * row + T * row * (1 + case["residual"]) + 8 * N, "flops": 2 * kept * case["dim"]}
        return {"bytes": T * row + 2 * kept * row + 12 * N, "flops": 3 * kept * case["dim"]}
    rows, n_in, n_out, E = case["rows"], case["n_in"], case["n_out"], case["experts"]
    bx, by = (2 if case[k] == "bf16" else 4 for k in ("x", "y"))
    flops = 2 * rows * n_in * n_out
    if case["op"] == "fp8_weight_gradient":
        return {"bytes": rows * (n_in + n_out) * bx + n_in * n_out * by, "flops": flops}
    # experts that rows reach on average: those without rows are not read
    reached = E * (1.0 - (1.0 - 1.0 / E) ** rows) if E > 1 else 1.0
    weights = n_out * n_in + 4 * _blocks(n_out) * _blocks(n_in) + (n_out * by if case["bias"] else 0)
    return {"bytes": reached * weights + rows * (n_in * bx + n_out * by * (1 + case["gate"] + case["residual"])), "flops": flops}


def _held64(x):
    """x [..., n] as its quantisation along the last dimension holds it, in float64: the rounding to e4m3 (3 bits after the
    point, smallest exponent -6, ties to even) is written out."""
    n = x.shape[-1]
    f = x.double()
    f = torch.cat((f, f.new_zeros(*f.shape[:-1], -n % 128)), -1).view(*f.shape[:-1], -1, 128)
    s = torch.maximum((f.abs().max(-1, keepdim=True).values / 448.0).float(), torch.tensor(2.0 ** -126, device="cuda"))
    v = (f * (1.0 / s.double()).float().double()).float().double()
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6.0)
    step = torch.exp2(exponent - 3.0)
    q = torch.round(v / step) * step
    return (q * s.double()).view(*x.shape[:-1], -1)[..., :n]


def exact(case, seed):
    if case["op"] == "tokens_dispatch":
        return None   # indexes and copies
    if case["op"].startswith("tokens"):
        d = _token_inputs(case, seed)
        at, w = d["positions"].long(), d["weights"].double()
        here = at >= 0
        w = w * here
        if case["op"] == "tokens_combine":
            y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
            if d["residual"] is not None:
                y += d["residual"].double()
            for j in range(case["slots"]):
                y += w[:, j, None] * d["Z"].double()[at[:, j].clamp(min=0)]
            return y
        dz = torch.zeros(d["Z"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(at.shape, dtype=torch.float64, device="cuda")
        dy = d["dY"].double()
        for j in range(case["slots"]):
            m = here[:, j]
            dz[at[m, j]] = w[m, j, None] * dy[m]
            dw[m, j] = (dy[m] * d["Z"].double()[at[m, j]]).sum(-1)
        return dz, dw
    d = _product_inputs(case, seed)
    if case["op"] == "fp8_weight_gradient":
        return torch.matmul(_held64(d["dY"].t()), _held64(d["X"].t()).T)
    rows, E = case["rows"], case["experts"]
    out = torch.empty(rows, case["n_out"], dtype=torch.float64, device="cuda")
    ends = d["offsets"].tolist() if case["op"] == "linear_fp8_experts" else [0, rows]
    x = _held64(d["X"])
    col = torch.arange(case["n_in"], device="cuda") // 128
    row = torch.arange(case["n_out"], device="cuda") // 128
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        y = torch.matmul(x[lo:hi], (d["W"][e].double() * d["scales"][e].double()[row][:, col]).T)
        if d["bias"] is not None:
            y += d["bias"][e].double()
        if case["act"] == "relu":
            y = y.clamp(min=0)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        if d["gate"] is not None:
            y *= d["gate"][lo:hi].double()
        if d["residual"] is not None:
            y += d["residual"][lo:hi].double()
        out[lo:hi] = y
    return out
