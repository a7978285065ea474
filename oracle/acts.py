"""fp64 oracle of the 8-bit activation checkpoints, the weight gradients from them
and the block seams (numpy; the formulas at muon_act8, muon_act8_grad_item, muon_seam
and muon_seam_grad in include/muon.h, written out plainly).

Shares no code with the library.  A checkpoint is a pair (q, e): whole numbers
and, per block of 32 columns, the exponent byte e + 127 (255: the block stands for NaNs).
"""
import numpy as np

BLOCK, E_MIN, E_MAX, BAD = 32, -120, 119, 255


def encode(x):
    x = np.asarray(x, dtype=np.float64)
    T, C = x.shape
    nb = -(-C // BLOCK)
    q = np.zeros((T, C), dtype=np.int64)
    e = np.zeros((T, nb), dtype=np.int64)
    for b in range(nb):
        cols = slice(b * BLOCK, min(C, (b + 1) * BLOCK))
        top = np.max(np.abs(x[:, cols]), axis=1)          # NaN propagates
        for t in range(T):
            if not np.isfinite(top[t]):
                e[t, b] = BAD
                continue
            k = E_MIN
            if top[t] > 0:
                k = max(E_MIN, int(np.floor(np.log2(top[t]))) - 8)
                while 127.0 * 2.0 ** k < top[t]:
                    k += 1
            if k > E_MAX:
                e[t, b] = BAD
                continue
            e[t, b] = k + 127
            q[t, cols] = np.rint(x[t, cols] / 2.0 ** k).astype(np.int64)   # halves to even
    return q, e


def decode(q, e):
    q = np.asarray(q, dtype=np.float64)
    e = np.repeat(np.asarray(e, dtype=np.float64), BLOCK, axis=1)[:, :q.shape[1]]
    return np.where(e == BAD, np.nan, q * 2.0 ** np.where(e == BAD, 0.0, e - 127))


def grad(dY, X, *, gain=None, shift=None, dy_sum=None, beta=0.0, G=None):
    """G of one layer; X: the checkpoint's values."""
    out = np.asarray(dY, dtype=np.float64).T @ X
    if gain is not None:
        out = out * gain[None, :]
    if shift is not None:
        out = out + np.outer(dy_sum, shift)
    return out if beta == 0 else out + beta * G


def normalise(v, kind, eps):
    """(normalised rows, reciprocal deviations)."""
    v = np.asarray(v, dtype=np.float64)
    if kind == "none":
        return v, np.ones(v.shape[0])
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(axis=1) + eps)
    return v * r[:, None], r


def _affine(n, gain, bias):
    n = n if gain is None else n * gain[None, :]
    return n if bias is None else n + bias[None, :]


def gate_of(gate, rows, gate_rows):
    return 1.0 if gate is None else np.asarray(gate, np.float64)[np.arange(rows) // gate_rows]


def seam_forward(x, f=None, *, post="none", pre="none", eps=1e-5, skip=1.0, scale=1.0, gate=None, gate_rows=1,
                 post_gain=None, post_bias=None, pre_gain=None, pre_bias=None, round_out=lambda v: v):
    """dict with out, y, n_f, n, post_rstd, pre_rstd (unrounded but for round_out, x's type)."""
    x = np.asarray(x, dtype=np.float64)
    res = dict(out=None, y=None, n_f=None, n=None)
    if f is not None:
        res["n_f"], res["post_rstd"] = normalise(f, post, eps)
        u = _affine(res["n_f"], post_gain, post_bias)
        x = skip * x + scale * gate_of(gate, x.shape[0], gate_rows) * u
        res["out"] = x
        x = round_out(x)
    if pre != "none":
        res["n"], res["pre_rstd"] = normalise(x, pre, eps)
        res["y"] = _affine(res["n"], pre_gain, pre_bias)
    return res


def _norm_back(g, n, r, kind):
    if kind == "none":
        return g
    g0 = g.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    return r[:, None] * (g - g0 - n * (g * n).mean(axis=1, keepdims=True))


def seam_backward(*, dy=None, dout=None, n=None, n_f=None, pre_rstd=None, post_rstd=None, post="none", pre="none",
                  skip=1.0, scale=1.0, gate=None, gate_rows=1, post_gain=None, post_bias=None, pre_gain=None,
                  has_f=True):
    """dict with dx, df, dgate, d_post_gain, d_post_bias, d_pre_gain, d_pre_bias; n, n_f: the checkpoints' values."""
    d = 0.0 if dout is None else np.asarray(dout, np.float64)
    res = {}
    if pre != "none":
        dy = np.asarray(dy, np.float64)
        g = dy if pre_gain is None else dy * pre_gain[None, :]
        d = d + _norm_back(g, n, pre_rstd, pre)
        res["d_pre_gain"], res["d_pre_bias"] = (dy * n).sum(axis=0), dy.sum(axis=0)
    res["dx"] = skip * d
    if not has_f:
        return res
    rows = d.shape[0]
    du = scale * gate_of(gate, rows, gate_rows) * d
    h = du if post_gain is None else du * post_gain[None, :]
    res["df"] = _norm_back(h, n_f, post_rstd, post)
    res["d_post_bias"] = du.sum(axis=0)
    if n_f is not None:
        res["d_post_gain"] = (du * n_f).sum(axis=0)
        if gate is not None:
            each = scale * d * _affine(n_f, post_gain, post_bias)
            res["dgate"] = np.stack([each[i:i + gate_rows].sum(axis=0) for i in range(0, rows, gate_rows)])
    return res
