"""Cases that measure the layer product with a fused epilogue and the layer product grouped by expert.

    linear_fused     Y = act(X S^T + (X V^T) U^T + bias) * gate + residual
    linear_experts   the same with rows sorted by expert: rows offsets[e] .. offsets[e+1]-1 of X, gate,
                     residual and Y belong to expert e and go through its S_e, U_e, V_e and bias_e

S is 2:4 along n_in. Where `own` is false, run() computes them from the dense S with elementary torch
operations in float32; where it is true, it calls the framework, on the packed S. Both have every
form of the weights in hand in the state, so nothing is laid out in a call but what the call casts.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, rows, n_in, n_out, r, dtype, y, act="none", bias=False, gate=False, residual=False, experts=1, skew=0.0):
    case = dict(op=op, rows=rows, n_in=n_in, n_out=n_out, r=r, dtype=dtype, y=y, act=act, bias=bias, gate=gate,
                residual=residual, experts=experts, skew=skew)
    return dict(case, name=name) if name else case


def listed():
    fused, experts = "linear_fused", "linear_experts"
    return [
        # one token's attention output projection added to the residual stream: pure latency
        _case("project one token", fused, 1, 4096, 4096, 64, "bf16", "bf16", bias=True, residual=True),
        # a decode batch through the gate projection, times the up projection's output
        _case("gated 16 tokens", fused, 16, 4096, 14336, 64, "bf16", "bf16", act="silu", gate=True),
        # one calibration segment through an attention projection, float32 residual stream
        _case("project 2048 tokens", fused, 2048, 4096, 4096, 64, "bf16", "fp32", residual=True),
        # the block's gate projection at its full prefill length: the largest case
        _case("gated 8192 tokens", fused, 8192, 4096, 14336, 128, "bf16", "bf16", act="silu", gate=True),
        # the MLP's down projection back onto the residual stream: the longest sums
        _case("down 4096 tokens", fused, 4096, 14336, 4096, 64, "bf16", "bf16", residual=True),
        # no size a multiple of a tile, a tail of 32 columns, an odd row length, a rank of three quarters of a block
        _case("odd sizes gelu", fused, 333, 1056, 1003, 48, "bf16", "fp32", act="gelu", bias=True),
        # the small float32 layer, with every part of the epilogue
        _case("float32 32 tokens", fused, 32, 512, 512, 16, "fp32", "fp32", act="gelu_tanh", bias=True, gate=True, residual=True),
        # a float32 layer of ordinary size, rows not a multiple of four
        _case("float32 1000 tokens", fused, 1000, 2048, 2050, 32, "fp32", "fp32", act="relu", bias=True),
        # a decode batch of 8 tokens, each to 8 of 32 small experts: two rows an expert, some with none
        _case("experts 64 rows", experts, 64, 2048, 1024, 32, "bf16", "bf16", act="silu", gate=True, experts=32),
        # a prefill over few large experts
        _case("experts 8192 rows", experts, 8192, 4096, 4096, 64, "bf16", "bf16", act="silu", gate=True, experts=8),
        # many small experts, unevenly loaded, with biases and a float32 result
        _case("experts uneven", experts, 6000, 2048, 1408, 16, "bf16", "fp32", act="gelu", bias=True, experts=60, skew=0.5),
        # float32 experts
        _case("experts float32", experts, 500, 512, 776, 16, "fp32", "fp32", act="relu", bias=True, residual=True, experts=6, skew=0.5),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("linear_fused", "linear_experts"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    small = dtype == "fp32"
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    y = "fp32" if small else rng.choice(("bf16", "fp32"))
    bias, gate, residual = (rng.random() < 0.5 for _ in range(3))
    while True:
        n_in, n_out = 32 * log(8, 64 if small else 448), log(200, 2500 if small else 14336)
        n_out -= 0 if rng.random() < 0.3 else n_out % 16
        r = 16 * rng.randint(0, 4 if small else 8)
        if op == "linear_fused":
            rows, e = log(1, 2048 if small else 8192), 1
        else:
            e = log(2, 64)
            rows = log(1, 2048 if small else 16384)
        if e * n_in * n_out <= 1 << 28 and rows * n_in * n_out <= (1 << 33 if small else 1 << 38):
            break
    return _case(None, op, rows, n_in, n_out, r, dtype, y, act, bias, gate, residual, e,
                 round(rng.choice((0.0, 0.5, 1.0)), 1) if e > 1 else 0.0)


def _keep(R):
    """The 2:4 projection of R [..., n_in]: kept positions a < b of every group of four (the two of
    largest magnitude, equal ones to the lower column)."""
    k = [R[..., i::4].abs() for i in range(4)]
    one = torch.int8
    rank = [sum((((k[i] >= k[j]) if j > i else (k[i] > k[j])).to(one)) for j in range(4) if j != i) for i in range(4)]
    keep = [x >= 2 for x in rank]
    first = torch.where(keep[0], 0, torch.where(keep[1], 1, 2))
    second = torch.where(keep[3], 3, torch.where(keep[2], 2, 1))
    return first, second


def _pack(R, first, second):
    """The packed layout (include/splr.h) of R's projection: values (E, TR, TK, 64, 8) and metadata
    (E, TR, TKB, 64, 4) int32."""
    E, N, K = R.shape
    TR, TK = (N + 15) // 16, (K + 63) // 64
    TKB = (TK + 7) // 8
    kept = torch.gather(R.view(E, N, K // 4, 4), 3, torch.stack((first, second), -1))
    v = torch.zeros(E, TR * 16, TK * 16, 2, dtype=R.dtype, device=R.device)
    v[:, :N, : K // 4] = kept
    v = v.view(E, TR, 16, TK, 4, 4, 2).permute(0, 1, 3, 4, 2, 5, 6).reshape(E, TR, TK, 64, 8).contiguous()
    m = torch.zeros(E, TR * 16, TKB * 8 * 16, dtype=torch.int32, device=R.device)
    m[:, :N, : K // 4] = (first | (second << 2)).to(torch.int32)
    m = m.view(E, TR, 16, TKB, 8, 4, 4)
    m = m[..., 0] | (m[..., 1] << 4) | (m[..., 2] << 8) | (m[..., 3] << 12)   # E, TR, row, TKB, column, quarter
    m = m.permute(0, 1, 3, 5, 2, 4).reshape(E, TR, TKB, 64, 4, 2)             # two 16-bit units a word
    return v, (m[..., 0] | (m[..., 1] << 16)).contiguous()


def _inputs(case, seed):
    """What both forms start from: activations with eight outlier columns, a pruned residual weight,
    thin factors whose product is about a third of it, and the epilogue's operands."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, yt = TYPES[case["dtype"]], TYPES[case["y"]]
    rows, n_in, n_out, r, E = case["rows"], case["n_in"], case["n_out"], case["r"], case["experts"]

    def normal(*shape, std=1.0, to=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)

    X = torch.randn(rows, n_in, generator=g, device="cuda")
    X[:, torch.randperm(n_in, generator=g, device="cuda")[:8]] *= 20.0
    R = normal(E, n_out, n_in, std=0.02)
    d = dict(X=X.to(dt), R=R)
    d["first"], d["second"] = _keep(R)
    at = torch.arange(4, device="cuda")
    kept = (d["first"][..., None] == at) | (d["second"][..., None] == at)
    d["S"] = torch.where(kept.view(R.shape), R, torch.zeros((), dtype=dt, device="cuda"))
    if r:
        s = math.sqrt(0.006 / math.sqrt(r))
        d["U"], d["V"] = normal(E, n_out, r, std=s), normal(E, r, n_in, std=s)
    else:
        d["U"] = d["V"] = None
    d["bias"] = normal(E, n_out, std=0.2) if case["bias"] else None
    d["gate"] = normal(rows, n_out, to=yt) if case["gate"] else None
    d["residual"] = normal(rows, n_out, to=yt) if case["residual"] else None
    if case["op"] == "linear_experts":
        # a router's choices: every row picks an expert by weights of the given spread, rows sorted by expert
        w = torch.exp(case["skew"] * torch.randn(E, generator=g, device="cuda"))
        chosen = torch.multinomial(w, rows, replacement=True, generator=g)
        counts = torch.bincount(chosen, minlength=E)
        d["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0))).to(torch.int32)
        d["capacity"] = max(1, int(counts.max()))
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    values, meta = _pack(d["R"], d["first"], d["second"])
    E, rows, n_out, r = case["experts"], case["rows"], case["n_out"], case["r"]
    s = {k: d[k] for k in ("X", "U", "V", "bias", "gate", "residual")}
    s.update(op=case["op"], act=case["act"], y=TYPES[case["y"]], n_out=n_out, values=values, meta=meta)
    # what a program that calls in a loop keeps: its result's buffer and the first stage's workspace
    s["out"] = torch.empty(rows, n_out, dtype=s["y"], device="cuda")
    s["workspace"] = torch.empty(16 * rows * r * 4, dtype=torch.uint8, device="cuda") if r else None
    if case["op"] == "linear_fused":
        for k in ("U", "V", "bias", "values", "meta"):
            s[k] = None if s[k] is None else s[k][0]
        s["S"] = d["S"][0]
    else:
        s.update(offsets=d["offsets"], capacity=d["capacity"], experts=E)
        s["St"] = d["S"].transpose(1, 2).contiguous()               # (E, n_in, n_out): the plain product's order
        s["Ut"] = d["U"].transpose(1, 2).contiguous() if r else None
        s["Vt"] = d["V"].transpose(1, 2).contiguous() if r else None
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


def _plain_fused(s):
    x = s["X"].float()
    z = x @ s["S"].float().t()
    if s["U"] is not None:
        z = z + (x @ s["V"].float().t()) @ s["U"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    return z


def _plain_experts(s):
    rows, E, cap = s["X"].shape[0], s["experts"], s["capacity"]
    row = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True)
    at = expert * cap + row - s["offsets"].long()[expert]
    x = torch.zeros(E * cap, s["X"].shape[1], device="cuda")
    x[at] = s["X"].float()
    x = x.view(E, cap, -1)
    z = torch.bmm(x, s["St"].float())
    if s["Ut"] is not None:
        z = z + torch.bmm(torch.bmm(x, s["Vt"].float()), s["Ut"].float())
    z = z.view(E * cap, -1)[at]
    if s["bias"] is not None:
        z = z + s["bias"].float()[expert]
    return z


def run(s):
    if own:
        from sparse_rank_linear_prune24_amd import binding

        kw = dict(bias=s["bias"], activation=s["act"], gate=s["gate"], residual=s["residual"], y_dtype=s["y"],
                  n_out=s["n_out"], out=s["out"], workspace=s["workspace"])
        if s["op"] == "linear_fused":
            return binding.linear_fused(s["X"], s["values"], s["meta"], s["U"], s["V"], **kw)
        return binding.linear_experts(s["X"], s["offsets"], s["values"], s["meta"], s["U"], s["V"], **kw)
    y = _act(_plain_fused(s) if s["op"] == "linear_fused" else _plain_experts(s), s["act"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["y"])


def work(case):
    rows, n_in, n_out, r, E = case["rows"], case["n_in"], case["n_out"], case["r"], case["experts"]
    b, by = (2 if case[k] == "bf16" else 4 for k in ("dtype", "y"))
    # experts that rows reach on average: those without rows are not read
    reached = E * (1.0 - (1.0 - 1.0 / E) ** rows) if E > 1 else 1.0
    weights = n_out * n_in // 2 * b + n_out * n_in // 8 + r * (n_out + n_in) * b + (n_out * b if case["bias"] else 0)
    per_row = n_in * b + n_out * by * (1 + case["gate"] + case["residual"])
    # the kept products only, and the two thin ones
    return {"bytes": reached * weights + rows * per_row, "flops": rows * (n_out * n_in + 2 * r * (n_in + n_out))}


def exact(case, seed):
    d = _inputs(case, seed)
    rows, E = case["rows"], case["experts"]
    out = torch.empty(rows, case["n_out"], dtype=torch.float64, device="cuda")
    ends = d["offsets"].tolist() if case["op"] == "linear_experts" else [0, rows]
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        W = d["S"][e].double()
        if d["U"] is not None:
            W += d["U"][e].double() @ d["V"][e].double()
        y = torch.matmul(d["X"][lo:hi].double(), W.T)
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
