"""The quantisation to e4m3 and the products with 8-bit weights in plain float64, and how far a kernel may be from them.

With u = 2^-24 (half a step of float32) and A = sum over k of |x_k w_k| of the quantised values:
  sums       a block's 128 products are exact in float32 (4 x 4 bits); their sum in any order, its product with sx sw (itself
             rounded) and the sum over the blocks and waves are off by at most (128 + KB + 16) u A
  8-bit matrix instructions (bfloat16 Y, tile kernels): each of eight products is cut at 2^-13 of the largest one's power of two, so
             a group loses less than 8 2^-13 of its largest product, and all of them less than 2^-10 A
  epilogue   as in _fused: 1.13 (no activation is steeper) and 16 u |z|, 4 u of what is added, half a step of Y's type
"""
import numpy as np
import torch

from tests._fused import HALF_STEP, U32, act64

E4M3 = torch.float8_e4m3fn


def _codes():
    """The 127 non-negative finite codes' values, in order."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append((1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6)
    return np.array(v)


VALUES = _codes()
MIDDLES = (VALUES[1:] + VALUES[:-1]) / 2


def to_code(v):
    """e4m3 codes (uint8) of float64 values of magnitude 464 at most: to nearest, ties to the even code; NaN is 0x7F."""
    a = np.abs(np.nan_to_num(v, nan=0.0))
    low = np.searchsorted(MIDDLES, a, side="left")     # ties: the lower code
    tie = (low < 126) & (MIDDLES[np.minimum(low, 125)] == a)
    code = low + (tie & (low % 2 == 1))
    code = (code | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def from_code(c):
    c = c.astype(np.int64)
    v = np.where((c & 127) == 127, np.nan, VALUES[np.minimum(c & 127, 126)])
    return np.where(c & 128, -v, v)


def scale_of(amax):
    return np.maximum((amax.astype(np.float64) / 448.0).astype(np.float32), np.float32(2.0 ** -126))


def quantize64(x, block_rows=1):
    """(codes [n][K], scales) of float64-held float32 values x [n][K]: scales [KB][n] for block_rows 1, [NB][KB] for 128."""
    n, K = x.shape
    KB, NB = (K + 127) // 128, (n + block_rows - 1) // block_rows
    codes, scales = np.zeros((n, K), np.uint8), np.zeros((NB, KB), np.float32)
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    for b in range(NB):
        r = slice(b * block_rows, min(n, (b + 1) * block_rows))
        for kb in range(KB):
            c = slice(kb * 128, min(K, kb * 128 + 128))
            s = scale_of(finite[r, c].max())
            inv = (1.0 / s.astype(np.float64)).astype(np.float32).astype(np.float64)
            v = np.where(np.isfinite(x[r, c]), x[r, c], np.nan)
            codes[r, c] = to_code((v * inv).astype(np.float32).astype(np.float64))
            scales[b, kb] = s
    return codes, scales.T.copy() if block_rows == 1 else scales


def spread(scales, n, K, by_row):
    """Scales over the entries [n][K] that they hold for, float64."""
    s = scales.astype(np.float64)
    if by_row:
        return np.repeat(s.T, 128, axis=1)[:, :K]
    return np.repeat(np.repeat(s, 128, axis=0)[:n], 128, axis=1)[:, :K]


def product64(x, w, y_dtype, narrow, bias=None, act="none", gate=None, residual=None):
    """(Y, bound) of dequantised x [M][K] and w [N][K]; narrow: on the 8-bit matrix instructions."""
    K = x.shape[1]
    z, a = x @ w.T, np.abs(x) @ np.abs(w).T
    d = ((128 + (K + 127) // 128 + 16) * U32 + (2.0 ** -10 if narrow else 0.0)) * a
    if bias is not None:
        z, d = z + bias, d + U32 * (np.abs(z) + np.abs(bias))
    y, d = act64(z, act), 1.13 * d + 16 * U32 * np.abs(z)
    if gate is not None:
        y, d = y * gate, d * np.abs(gate)
    d = d + 4 * U32 * np.abs(y)
    if residual is not None:
        y, d = y + residual, d + 4 * U32 * np.abs(residual)
    return y, d + HALF_STEP[y_dtype] * (np.abs(y) + d)


def dev_codes(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(E4M3).cuda()


def codes_of(t):
    """The codes of a device tensor, its NaN (0x7F and 0xFF, the contract asks for either) as 0x7F."""
    c = t.detach().cpu().view(torch.uint8).numpy()
    return np.where(c == 0xFF, np.uint8(0x7F), c)


def floats(shape, dtype, seed, std=1.0, outliers=0):
    """(device tensor, its values in float64) of random normal entries with whole outlier columns."""
    g = np.random.Generator(np.random.PCG64(seed))
    a = g.standard_normal(shape) * std
    if outliers:
        a[..., g.permutation(shape[-1])[:outliers]] *= 20.0
    t = torch.from_numpy(a).to(torch.float32).to(dtype)
    return t.cuda(), t.double().numpy()


class Weight:
    """e4m3 weights in blocks of 128 x 128 (by_row: 1 x 128): codes and scales on the device, the values in float64."""

    def __init__(self, n_out, n_in, seed, by_row=False, std=0.02):
        g = np.random.Generator(np.random.PCG64(seed))
        w = (g.standard_normal((n_out, n_in)) * std).astype(np.float32).astype(np.float64)
        codes, scales = quantize64(w, 1 if by_row else 128)
        self.values = from_code(codes) * spread(scales, n_out, n_in, by_row)
        self.codes, self.scales = codes, scales
        self.W, self.s = dev_codes(codes), torch.from_numpy(scales).cuda()


def held(x64):
    """x as the call's own quantisation holds it."""
    codes, scales = quantize64(x64)
    return from_code(codes) * spread(scales, *x64.shape, True)
