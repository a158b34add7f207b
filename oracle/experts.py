"""fp64 definitions of the expert training operators (numpy, CPU; shares no code with the library)."""
from __future__ import annotations

import numpy as np

_M = np.uint64(0xFFFFFFFF)


def philox(counter, key, rounds=10):
    """Philox4x32 (Salmon, Moraes, Dror and Shaw 2011): counter [..., 4] and key [2] of 32-bit words."""
    c = np.asarray(counter, dtype=np.uint64)
    x = [c[..., j] for j in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), q & _M, (p >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), p & _M]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(x, -1)


def keep_mask(index, p, seed, offset):
    """Whether the elements `index` (non-negative integers) are kept."""
    i = np.asarray(index, dtype=np.uint64)
    b = i >> np.uint64(2)
    c = np.stack([b & _M, b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)], -1)
    words = philox(c, (seed & 0xFFFFFFFF, seed >> 32))
    w = np.take_along_axis(words, (i & np.uint64(3)).astype(np.int64)[..., None], -1)[..., 0]
    return w >= np.uint64(int(np.floor(p * 2.0 ** 32)))


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, dtype=np.float64)
    m = keep_mask(np.arange(x.size).reshape(x.shape), p, seed, offset)
    out = np.where(m, x / (1.0 - p), 0.0)
    return out if residual is None else out + residual


def _branches(g, u, act, beta, linear_beta):
    """s, 1 - s, f(g), f'(g), h(u), h'(u) of a = s f h, without differences that cancel."""
    with np.errstate(over="ignore"):
        s, rest = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
        if act == "silu":
            return s, rest, g, np.ones_like(g), u, np.ones_like(u)
        slope = lambda x: 1.0 / np.square(np.cosh(x))  # noqa: E731
        return (s, rest, beta * np.tanh(g / beta), slope(g / beta), linear_beta * np.tanh(u / linear_beta),
                slope(u / linear_beta))


def glu_dropout(gu, p, seed, offset, act="silu", beta=4.0, linear_beta=25.0):
    g, u = np.split(np.asarray(gu, dtype=np.float64), 2, axis=1)
    s, _, f, _, h, _ = _branches(g, u, act, beta, linear_beta)
    return dropout(s * f * h, p, seed, offset)


def glu_dropout_grad(da, gu, p, seed, offset, act="silu", beta=4.0, linear_beta=25.0):
    g, u = np.split(np.asarray(gu, dtype=np.float64), 2, axis=1)
    s, rest, f, df, h, dh = _branches(g, u, act, beta, linear_beta)
    d = dropout(da, p, seed, offset)
    return np.concatenate([d * h * s * (rest * f + df), d * s * f * dh], 1)


def plan_rows(idx, n_experts, first=0):
    idx = np.asarray(idx)
    pos = np.full(idx.shape, -1, dtype=np.int32)
    offsets = np.zeros(n_experts + 1, dtype=np.int32)
    row = 0
    for e in range(n_experts):
        offsets[e] = row
        hit = np.flatnonzero(idx.reshape(-1) == e + first)
        pos.reshape(-1)[hit] = row + np.arange(hit.size)
        row += hit.size
    offsets[n_experts] = row
    return offsets, pos


def combine_rows(y, pos, w=None):
    y = np.asarray(y, dtype=np.float64)
    z = np.zeros((pos.shape[0], y.shape[1]))
    for t, k in zip(*np.nonzero(pos >= 0)):
        z[t] += (1.0 if w is None else float(w[t, k])) * y[pos[t, k]]
    return z


def combine_rows_grad(dz, y, pos, w):
    dy, dw = np.zeros(np.shape(y)), np.zeros(pos.shape)
    dz, y = np.asarray(dz, dtype=np.float64), np.asarray(y, dtype=np.float64)
    for t, k in zip(*np.nonzero(pos >= 0)):
        dy[pos[t, k]] = float(w[t, k]) * dz[t]
        dw[t, k] = dz[t] @ y[pos[t, k]]
    return dy, dw


def group_mm(x, w, offsets):
    """Rows of no expert give zeros."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        y[offsets[e]:offsets[e + 1]] = x[offsets[e]:offsets[e + 1]] @ w[e].T
    return y


def group_mm_grad_x(dy, w, offsets):
    return group_mm(dy, np.swapaxes(np.asarray(w, dtype=np.float64), 1, 2), offsets)


def group_mm_grad_w(dy, x, offsets):
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    return np.stack([dy[a:b].T @ x[a:b] for a, b in zip(offsets[:-1], offsets[1:])])


# ------------------------------------------------------------------------------------------ gated block
def group_glu(x, w, offsets, act="silu", beta=4.0, linear_beta=25.0):
    """Rows of no expert give zeros, as in group_mm."""
    return glu_dropout(group_mm(x, w, offsets), 0.0, 0, 0, act, beta, linear_beta)


def group_glu_grad(da, x, w, offsets, act="silu", beta=4.0, linear_beta=25.0):
    return glu_dropout_grad(da, group_mm(x, w, offsets), 0.0, 0, 0, act, beta, linear_beta)


# ------------------------------------------------------------------------------------------ 8-bit operands
F8 = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}      # mantissa bits, least normal exponent, largest value


def round8(v, kind):
    """To the format's nearest value, ties to even; |v| is at most the largest value, or not finite."""
    mantissa, least, _ = F8[kind]
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        e = np.maximum(np.frexp(np.where(np.isfinite(v), v, 1.0))[1] - 1, least)
        out = np.ldexp(np.rint(np.ldexp(v, mantissa - e)), e - mantissa)
    if kind == "e4m3":
        out = np.where(np.isinf(v), np.nan, out)
    return out


def scale_exponent(amax, kind):
    """The smallest k >= -127 with amax <= 2^k largest."""
    k = -127
    while amax > F8[kind][2] * 2.0 ** k:
        k += 1
    return k


def quant8(x, kind, rows=1, cols=128):
    """x [..., n, m] -> (codes' values, scale bytes k + 127) with a scale for each block of rows x cols."""
    x = np.asarray(x, dtype=np.float64)
    n, m = x.shape[-2:]
    codes = np.empty_like(x)
    scales = np.empty(x.shape[:-2] + (-(-n // rows), -(-m // cols)), dtype=np.uint8)
    for i in np.ndindex(*scales.shape):
        at = i[:-2] + (slice(i[-2] * rows, (i[-2] + 1) * rows), slice(i[-1] * cols, (i[-1] + 1) * cols))
        v = x[at]
        k = scale_exponent(np.max(np.abs(v[np.isfinite(v)]), initial=0.0), kind)
        scales[i] = k + 127
        codes[at] = round8(np.ldexp(v, -k), kind)
    return codes, scales


def dequant8(codes, scales, rows=1, cols=128):
    k = np.repeat(np.repeat(np.asarray(scales, dtype=np.int64) - 127, rows, -2), cols, -1)
    codes = np.asarray(codes, dtype=np.float64)
    return np.ldexp(codes, k[..., :codes.shape[-2], :codes.shape[-1]])


def group_mm8(x, x_scales, w, w_scales, offsets):
    return group_mm(dequant8(x, x_scales), dequant8(w, w_scales, 128), offsets)


# ------------------------------------------------------------------------------------------ norms
def rms_norm(x, gain=None, eps=1e-6):
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, 1, keepdims=True) + eps)
    return n if gain is None else n * gain


def rms_norm_grad(dy, x, gain=None, eps=1e-6, add=None):
    """(dx, dgain): dgain also without a gain."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, 1, keepdims=True) + eps)
    v = dy if gain is None else dy * gain
    dx = r * v - x * r ** 3 * np.mean(v * x, 1, keepdims=True)
    return dx if add is None else dx + add, (dy * x * r).sum(0)


def _gate(gate):
    return 1.0 if gate is None else np.asarray(gate, dtype=np.float64).reshape(len(gate), -1)


def norm_residual(y, residual, gain=None, gate=None, residual_scale=1.0, next_gain=None, eps=1e-6):
    h = residual_scale * np.asarray(residual, dtype=np.float64) + _gate(gate) * rms_norm(y, gain, eps)
    return h, rms_norm(h, next_gain, eps)


def norm_residual_grad(dh, dn, y, h, gain=None, gate=None, residual_scale=1.0, next_gain=None, eps=1e-6):
    """(dy, dresidual, dgain, dgate, dnext_gain); dgate for each element and (rows) summed where the gate is by row."""
    t = 0.0 if dh is None else np.asarray(dh, dtype=np.float64)
    dnext = None
    if dn is not None:
        t, dnext = rms_norm_grad(dn, h, next_gain, eps, add=t)
    b = rms_norm(y, gain, eps)
    dgate = None if gate is None else (t * b if np.ndim(gate) == 2 else (t * b).sum(1))
    dy, dgain = rms_norm_grad(t * _gate(gate), y, gain, eps)
    return dy, residual_scale * t, dgain, dgate, dnext
