"""Plain float64 forms of the fused-epilogue products, and how far a float32 kernel may be from them.

The bound is per entry and counts roundings. With u = 2^-24 (half a step of float32) and absolute
values in every factor,
  T = X V^T           |dT| <= K u A_T,                  A_T = |X| |V|^T    (K products and sums)
  T U^T               |d|  <= (|dT| + 2^-17 |T|) |U|^T                     (T may pass as two bfloat16 numbers)
  Z                   |dZ| <= that + (K + 2 r + 16) u (|X| |S|^T + |T| |U|^T + |bias|)
  act(Z)              |dA| <= 1.13 |dZ| + 16 u |Z|      (no activation is steeper than 1.13)
  A gate + residual   |dY| <= |dA| |gate| + 4 u (|A gate| + |residual|)
  stored              + half a step of Y's type.
Float32 sums of n terms in any order are off by at most n u times the sum of the absolute values.
"""
import math

import numpy as np
import torch

import oracle
from sparse_rank_linear_prune24_amd import inputs

U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act64(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    return z


class Weights:
    """One layer: dense S, factors and bias in float64, and their storage arrays."""

    def __init__(self, n_in, n_out, r, dtype, seed, bias=False, integers=False):
        self.dtype, self.n_in, self.n_out, self.r = dtype, n_in, n_out, r
        if integers:  # every sum below 2^24, so float32 arithmetic is exact
            def draw(shape, t):
                return inputs.small_integers(shape, -2, 2, dtype, seed=seed, tensor_id=t)
            R, self.U, self.V = draw((n_out, n_in), 1), draw((n_out, r), 2), draw((r, n_in), 3)
            b = draw((n_out,), 5)
        else:
            L = inputs.random_case(1, n_in, n_out, r, dtype, seed=seed, uv_std=math.sqrt(0.006 / math.sqrt(max(r, 1))))
            R, self.U, self.V = L.R, L.U, L.V
            b = inputs.gaussian((n_out,), 0.2, dtype, seed=seed, config_id=1000, tensor_id=5)
        self.values, self.meta = oracle.prune24_pack(R, dtype)
        self.bias = b if bias else None
        self.S = oracle.dense_reconstruct(self.values, self.meta, n_out, n_in, None, None, dtype)
        f = lambda a: inputs.to_f64(a, dtype)  # noqa: E731
        self.U64, self.V64 = f(self.U), f(self.V)
        self.b64 = f(self.bias) if bias else np.zeros(n_out)


def product64(X64, w):
    """(Z without bias, bound of its error without the bias term's, sum of absolute values)."""
    K, r = w.n_in, w.r
    T = X64 @ w.V64.T
    z = X64 @ w.S.T + T @ w.U64.T
    a_t = np.abs(X64) @ np.abs(w.V64).T
    a = np.abs(X64) @ np.abs(w.S).T + np.abs(T) @ np.abs(w.U64).T + np.abs(w.b64)
    d = (K * U32 * a_t + 2.0 ** -17 * np.abs(T)) @ np.abs(w.U64).T + (K + 2 * r + 16) * U32 * a
    return z + w.b64, d


def fused64(X64, w, act="none", gate=None, residual=None, y_dtype=torch.float32):
    """(Y, bound) in float64; gate and residual as float64 arrays."""
    z, d = product64(X64, w)
    y = act64(z, act)
    d = 1.13 * d + 16 * U32 * np.abs(z)
    if gate is not None:
        y, d = y * gate, d * np.abs(gate)
    d = d + 4 * U32 * np.abs(y)
    if residual is not None:
        y = y + residual
        d = d + 4 * U32 * np.abs(residual)
    return y, d + HALF_STEP[y_dtype] * (np.abs(y) + d)


def check(got, want, bound, tag):
    got = got.detach().cpu().double().numpy()
    assert np.all(np.isfinite(got)), f"{tag}: not finite"
    worst = float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300))) if got.size else 0.0
    print(f"[fused] {tag}: worst error / bound = {worst:.3f}", flush=True)
    assert worst <= 1.0, f"{tag}: {worst:.3f} of the bound"


def rows64(shape, y_dtype, seed, tensor_id, integers=False):
    """A gate or residual: (storage tensor on the device, float64 values)."""
    t = "bf16" if y_dtype == torch.bfloat16 else "fp32"
    a = (inputs.small_integers(shape, -2, 2, t, seed=seed, tensor_id=tensor_id) if integers
         else inputs.gaussian(shape, 1.0, t, seed=seed, config_id=1000, tensor_id=tensor_id))
    from tests._helpers import to_dev
    return to_dev(a, t), inputs.to_f64(a, t)
