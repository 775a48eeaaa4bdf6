"""Plain NumPy gated activation, residual norms and their gradients, in 64 bits.

act(g) = g * sigmoid(g), or the tanh form of GELU; h = act(g) * u.
z = v * x / rms(x) (or x); s = r + scale * gate * z; y = w * s / rms(s); rms(a) = sqrt(mean(a^2) + eps) over a row.
"""

import numpy as np


def _arg(g, act):
    """(z, dz/dg) with act(g) = g * sigmoid(z)."""
    if act == "silu":
        return g, np.ones_like(g)
    c = 2.0 * np.sqrt(2.0 / np.pi)   # 0.5 (1 + tanh(y)) = sigmoid(2 y)
    return c * (g + 0.044715 * g ** 3), c * (1.0 + 3.0 * 0.044715 * g ** 2)


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act_value(g, act):
    return g * _sigmoid(_arg(g, act)[0])


def act_slope_terms(g, act):
    """The two terms whose sum is the slope."""
    z, dz = _arg(g, act)
    return _sigmoid(z), g * _sigmoid(z) * _sigmoid(-z) * dz


def gated(pre, act):
    pre = np.asarray(pre, dtype=np.float64)
    n = pre.shape[-1] // 2
    return act_value(pre[..., :n], act) * pre[..., n:]


def gated_grad(dh, pre, act):
    pre, dh = np.asarray(pre, dtype=np.float64), np.asarray(dh, dtype=np.float64)
    n = pre.shape[-1] // 2
    g, u = pre[..., :n], pre[..., n:]
    p, q = act_slope_terms(g, act)
    return np.concatenate((dh * u * (p + q), dh * act_value(g, act)), axis=-1)


def _inv_rms(a, eps):
    return 1.0 / np.sqrt(np.mean(a * a, axis=1, keepdims=True) + eps)


def _per_row(gate, rows):
    """The gate of each row: (hidden,), or (gate_rows, hidden) for rows / gate_rows consecutive rows each."""
    if gate is None:
        return None
    gate = np.atleast_2d(np.asarray(gate, dtype=np.float64))
    return np.repeat(gate, rows // gate.shape[0], axis=0) if rows else gate[:0]


def residual_norm(x, residual, weight, gate=None, post_norm=False, post_weight=None, scale=1.0, eps=1e-6):
    """(sum, y)."""
    s = np.asarray(residual, dtype=np.float64)
    one = np.ones(s.shape[1])
    if x is not None:
        z = np.asarray(x, dtype=np.float64)
        if post_norm:
            z = z * _inv_rms(z, eps) * (one if post_weight is None else post_weight)
        s = s + scale * z * (1.0 if gate is None else _per_row(gate, s.shape[0]))
    return s, s * _inv_rms(s, eps) * (one if weight is None else weight)


def residual_norm_grad(dy, dsum, x, s, weight, gate=None, post_norm=False, post_weight=None, scale=1.0, eps=1e-6):
    """dict of dx, dresidual, dweight, dgate, dpost_weight (None where there is nothing to have one) and, for each, the sum of
    the magnitudes that its terms have ("size_..."), to which rounding errors are proportional."""
    dy, s = np.asarray(dy, dtype=np.float64), np.asarray(s, dtype=np.float64)
    rows, hidden = s.shape
    w = np.ones(hidden) if weight is None else np.asarray(weight, dtype=np.float64)
    ds = np.zeros_like(s) if dsum is None else np.asarray(dsum, dtype=np.float64)
    rho = _inv_rms(s, eps)

    def back(t, a, inv):
        """Gradient of a / rms(a) from t, and the magnitudes of its terms."""
        inner = np.mean(t * a, axis=1, keepdims=True)
        size = np.mean(np.abs(t * a), axis=1, keepdims=True)
        return inv * (t - a * inv ** 2 * inner), inv * (np.abs(t) + np.abs(a) * inv ** 2 * size)

    du, size = back(dy * w, s, rho)
    du, size = du + ds, size + np.abs(ds)
    out = dict(dresidual=du, size_dresidual=size, dx=None, dgate=None, dpost_weight=None,
               dweight=None if weight is None else (dy * s * rho).sum(0), size_dweight=np.abs(dy * s * rho).sum(0))
    if x is None:
        return out
    x = np.asarray(x, dtype=np.float64)
    sigma = _inv_rms(x, eps) if post_norm else np.ones((rows, 1))
    v = np.ones(hidden) if post_weight is None else np.asarray(post_weight, dtype=np.float64)
    z = x * sigma * v
    if gate is not None:
        groups = np.atleast_2d(gate).shape[0]
        dg = (scale * du * z).reshape(groups, rows // groups, hidden)
        out["dgate"] = dg.sum(1).reshape(np.shape(gate))
        out["size_dgate"] = (np.abs(scale * z) * size).reshape(dg.shape).sum(1).reshape(np.shape(gate))
    g = scale * (np.ones((1, 1)) if gate is None else _per_row(gate, rows))
    dz, size = g * du, np.abs(g) * size
    if post_norm:
        if post_weight is not None:
            out["dpost_weight"] = (dz * x * sigma).sum(0)
            out["size_dpost_weight"] = (size * np.abs(x * sigma)).sum(0)
        wide = np.mean(size * np.abs(v * x), axis=1, keepdims=True)
        dz, size = back(dz * v, x, sigma)[0], sigma * (size * np.abs(v) + np.abs(x) * sigma ** 2 * wide)
    out["dx"], out["size_dx"] = dz, size
    return out
