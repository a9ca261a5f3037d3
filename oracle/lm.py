"""Float64 oracle of the language-model operators: RMSNorm of the residual stream with its gradients,
E4M3 codes with block scales, the linear layer on such codes with its gradients, rotary positions.

Each function is the operator's formula, written without regard to speed.  The casts are defined in
float32 (the scale is a float32 number that the codes and every product depend on), so they are
reproduced bit for bit; everything else is float64.
"""
from __future__ import annotations

import math
from decimal import Decimal, localcontext

import numpy as np

from . import e4m3 as E

TILE = 128
_DECODE = np.array([E.e4m3_decode(c) for c in range(256)])


def _f64(x):
    return np.asarray(x, np.float64)


# ------------------------------------------------------------------------------------- RMSNorm
def rmsnorm(h, gain, eps):
    """y = h gain / sqrt(mean(h^2) + eps) per row, and the reciprocal root r."""
    h = _f64(h)
    r = 1.0 / np.sqrt((h * h).mean(axis=-1) + eps)
    return h * r[:, None] * _f64(gain), r


def rmsnorm_bwd(dy, h, gain, eps, dh_in=None):
    """(dh, dgain) by the quotient rule: y_i = g_i h_i r, dr/dh_k = -r^3 h_k / D."""
    dy, h, g = _f64(dy), _f64(h), _f64(gain)
    _, r = rmsnorm(h, g, eps)
    dot = (dy * g * h).sum(axis=-1)
    dh = dy * g * r[:, None] - h * (r ** 3 * dot / h.shape[1])[:, None]
    if dh_in is not None:
        dh = dh + _f64(dh_in)
    return dh, (dy * h * r[:, None]).sum(axis=0)


# ------------------------------------------------------------------------------------- block scales
def block_scale(amax):
    """min(448 (1 / amax), 2^100) in float32 steps; 1 for an amax of zero."""
    amax = np.asarray(amax, np.float32)
    with np.errstate(divide="ignore", over="ignore"):
        s = np.minimum((np.float32(1) / amax) * np.float32(448), np.float32(2.0 ** 100))
    return np.where(amax > 0, s, np.float32(1)).astype(np.float32)


def _amax(x, axis):
    return np.nanmax(np.abs(np.where(np.isnan(x), 0, x)), axis=axis)


def encode(v):
    """E4M3 codes of float32 values (nearest, ties to even, saturating; NaN -> NaN)."""
    return E.e4m3_encode(np.asarray(v, np.float64))


def decode(q):
    return _DECODE[np.asarray(q)]


def cast_rows(x):
    """Codes [R, C] and scales [ceil(C/128), R] of 1 x 128 tiles."""
    x = np.asarray(x, np.float32)
    q, s = np.zeros(x.shape, np.uint8), []
    for c in range(0, x.shape[1], TILE):
        t = x[:, c:c + TILE]
        sc = block_scale(_amax(t, 1))
        q[:, c:c + TILE] = encode(t * sc[:, None])
        s.append(sc)
    return q, np.array(s, np.float32)


def cast_square(x):
    """Codes [R, C] and scales [ceil(R/128), ceil(C/128)] of 128 x 128 tiles."""
    x = np.asarray(x, np.float32)
    q = np.zeros(x.shape, np.uint8)
    s = np.zeros((-(-x.shape[0] // TILE), -(-x.shape[1] // TILE)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            sl = (slice(i * TILE, (i + 1) * TILE), slice(j * TILE, (j + 1) * TILE))
            s[i, j] = block_scale(_amax(x[sl], (0, 1)))
            q[sl] = encode(x[sl] * s[i, j])
    return q, s


def values_rows(q, s):
    """What codes [R, C] under scales [ceil(C/128), R] stand for."""
    return decode(q) / np.repeat(_f64(s).T, TILE, axis=1)[:, :q.shape[1]]


def values_square(q, s):
    w = np.repeat(np.repeat(_f64(s), TILE, axis=0), TILE, axis=1)
    return decode(q) / w[:q.shape[0], :q.shape[1]]


def block_linear(x_q, s_x, w_q, s_w, b=None):
    """y = x W^T + b of the represented values."""
    y = values_rows(x_q, s_x) @ values_square(w_q, s_w).T
    return y if b is None else y + _f64(b)


def block_linear_bwd(dy, w_q, s_w, x_t, s_xt):
    """(dx, dw, db): dy cast per direction, the products of the represented values.  w_q [N, K]; x_t
    [K, M] the codes of x's columns."""
    g, sg = cast_rows(dy)
    gt, sgt = cast_rows(np.asarray(dy).T)
    dx = values_rows(g, sg) @ values_square(w_q, s_w)
    dw = values_rows(gt, sgt) @ values_rows(x_t, s_xt).T
    return dx, dw, _f64(dy).sum(axis=0)


# ------------------------------------------------------------------------------------- rotary positions
def rope_frequencies(rot, theta=10000.0, scaling="none", factor=1.0, orig_len=0.0, low=1.0, high=4.0):
    """f_j = theta^(-2j / rot), interpolated as `scaling` says."""
    f = np.array([theta ** (-2.0 * j / rot) for j in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        turns = orig_len * f / (2.0 * math.pi)
        g = np.clip((turns - low) / (high - low), 0.0, 1.0)
        return f * g + f / factor * (1.0 - g)
    return f


def rope_cos_sin(positions, freqs):
    """cos and sin [..., pairs] of position x frequency, each angle reduced modulo a turn in long
    integers (2^-200 of a turn), so that far positions keep their fraction."""
    two_pi = 2.0 * math.pi
    one = 1 << 200
    turns = [int(math.ldexp(f / two_pi, 100)) << 100 for f in freqs]
    pos = np.asarray(positions)
    ang = np.empty(pos.shape + (len(turns),))
    for idx in np.ndindex(pos.shape):
        p = int(pos[idx])
        for j, t in enumerate(turns):
            ang[idx + (j,)] = ((p * t) % one) / one * two_pi
    return np.cos(ang), np.sin(ang)


def _two_pi(digits):
    """2 pi as a Decimal of so many digits: 4 (4 arctan(1/5) - arctan(1/239)) 2, the series in whole numbers."""
    one = 10 ** (digits + 10)

    def arctan_inv(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    with localcontext() as ctx:
        ctx.prec = digits
        return Decimal(8 * (4 * arctan_inv(5) - arctan_inv(239))) / one


def rope_turns_exact(rot, theta=10000.0, scaling="none", factor=1.0, orig_len=0.0, low=1.0, high=4.0):
    """f_j / 2 pi as Decimals of 80 digits: the frequencies without a double's rounding."""
    with localcontext() as ctx:
        ctx.prec = 80
        theta, factor, orig, lo, hi = (Decimal(v) for v in (theta, factor, orig_len, low, high))
        two_pi, out = _two_pi(80), []
        for j in range(rot // 2):
            f = theta ** (Decimal(-2 * j) / rot)
            if scaling == "linear":
                f = f / factor
            elif scaling == "by_parts":
                g = min(max((orig * f / two_pi - lo) / (hi - lo), Decimal(0)), Decimal(1))
                f = f * g + f / factor * (1 - g)
            out.append(f / two_pi)
        return out


def rope_cos_sin_exact(positions, turns):
    """cos and sin [..., pairs] of position x exact frequency (rope_turns_exact), reduced in 80 digits."""
    pos = np.asarray(positions)
    ang = np.empty(pos.shape + (len(turns),))
    with localcontext() as ctx:
        ctx.prec = 80
        for idx in np.ndindex(pos.shape):
            for j, t in enumerate(turns):
                ang[idx + (j,)] = float(int(pos[idx]) * t % 1) * 2.0 * math.pi
    return np.cos(ang), np.sin(ang)


def rope(x, cos, sin, rot, interleaved, mscale=1.0, transposed=False):
    """x [B, S, H, d] rotated by cos, sin [B, S, rot/2] (the transposed rotation for gradients)."""
    x = _f64(x)
    y = x.copy()
    c, s = mscale * cos[:, :, None, :], (-mscale if transposed else mscale) * sin[:, :, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y
