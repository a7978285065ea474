"""Pins of the fp64 oracle of the activation checkpoints and block seams: values
worked by hand, the format's defining inequalities, and gradients against central
differences of the forward formulas."""
import numpy as np
import pytest

from oracle import acts


def test_encode_by_hand():
    # one row of 40 columns: block 0 has largest magnitude 3 (127 2^-5 = 3.97 holds it, 127 2^-6 = 1.98 does not),
    # block 1 exactly 127 2^-3
    x = np.zeros((1, 40))
    x[0, :4] = [3.0, -1.0, 2.0 ** -6, 3 * 2.0 ** -6]
    x[0, 32:35] = [127 / 8, -127 / 8, 0.3]
    q, e = acts.encode(x)
    assert list(e[0]) == [127 - 5, 127 - 3]
    # 2^-6 and 3 2^-6 are 0.5 and 1.5 steps: halves go to the even neighbour
    assert list(q[0, :4]) == [96, -32, 0, 2]
    assert list(q[0, 32:35]) == [127, -127, 2]
    v = acts.decode(q, e)
    assert v[0, 0] == 3.0 and v[0, 34] == 0.25 and not v[0, 4:32].any()


def test_encode_limits():
    x = np.zeros((6, 32))
    x[0, 0] = 127 * 2.0 ** 119
    x[1, 0] = 127 * 2.0 ** 119 * (1 + 2.0 ** -20)     # beyond the largest block
    x[2, 3] = np.inf
    x[3, 3] = np.nan
    x[4, 0] = 2.0 ** -121                              # half a step of the smallest exponent: to even, 0
    x[5, 0] = 1.5 * 2.0 ** -120
    q, e = acts.encode(x)
    assert list(e[:, 0]) == [119 + 127, 255, 255, 255, 7, 7]
    assert q[0, 0] == 127 and q[4, 0] == 0 and q[5, 0] == 2
    assert np.isnan(acts.decode(q, e)[1:4]).all()


@pytest.mark.parametrize("seed", range(4))
def test_encode_error_is_half_a_step(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((9, 75)) * 10.0 ** rng.integers(-30, 30, (9, 1))
    q, e = acts.encode(x)
    step = 2.0 ** (np.repeat(e, 32, axis=1)[:, :75] - 127.0)
    assert np.all(np.abs(acts.decode(q, e) - x) <= step / 2)
    top = np.array([[np.max(np.abs(x[t, b * 32:b * 32 + 32])) for b in range(3)] for t in range(9)])
    assert np.all(127 * 2.0 ** (e - 127.0) >= top) and np.all(127 * 2.0 ** (e - 128.0) < top)


def test_grad_is_the_gradient_of_the_layer():
    # loss = <dY, X W^T> with X = X^ diag(gain) + 1 shift^T; central differences are exact for a linear function
    rng = np.random.default_rng(0)
    dY, X = rng.standard_normal((5, 3)), rng.standard_normal((5, 4))
    gain, shift = rng.standard_normal(4), rng.standard_normal(4)
    G = acts.grad(dY, X, gain=gain, shift=shift, dy_sum=dY.sum(axis=0))

    def loss(W):
        return np.sum(dY * ((X * gain + shift) @ W.T))
    for o in range(3):
        for c in range(4):
            E = np.zeros((3, 4))
            E[o, c] = 1.0
            assert abs((loss(E) - loss(-E)) / 2 - G[o, c]) <= 1e-12
    H = rng.standard_normal((3, 4))
    assert np.allclose(acts.grad(dY, X, beta=0.25, G=H), dY.T @ X + 0.25 * H, rtol=0, atol=1e-14)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 7])
def test_seam_backward_against_differences(post, pre, gate_rows):
    # checkpoints held exactly, so the backward formulas are the forward's derivatives up to eps-free rounding
    rng = np.random.default_rng(7)
    T, C = 7, 5
    gr = max(1, gate_rows)
    v = dict(x=rng.standard_normal((T, C)), f=rng.standard_normal((T, C)))
    if gate_rows:
        v["gate"] = rng.standard_normal((-(-T // gr), C))
    for k in ("post_gain", "post_bias") + (("pre_gain", "pre_bias") if pre != "none" else ()):
        v[k] = rng.standard_normal(C)
    kw = dict(post=post, pre=pre, skip=0.9, scale=0.7, gate_rows=gr, eps=1e-3)
    dout = rng.standard_normal((T, C))
    dy = rng.standard_normal((T, C)) if pre != "none" else None

    def loss(w):
        r = acts.seam_forward(**w, **kw)
        return np.sum(dout * r["out"]) + (np.sum(dy * r["y"]) if dy is not None else 0.0)
    fwd = acts.seam_forward(**v, **kw)
    got = acts.seam_backward(dy=dy, dout=dout, n=fwd["n"], n_f=fwd["n_f"], pre_rstd=fwd.get("pre_rstd"),
                             post_rstd=fwd["post_rstd"], post=post, pre=pre, skip=0.9, scale=0.7,
                             gate=v.get("gate"), gate_rows=gr, post_gain=v["post_gain"], post_bias=v["post_bias"],
                             pre_gain=v.get("pre_gain"))
    names = {"x": "dx", "f": "df", "gate": "dgate", "post_gain": "d_post_gain", "post_bias": "d_post_bias",
             "pre_gain": "d_pre_gain", "pre_bias": "d_pre_bias"}
    h = 1e-5
    for k in v:
        num = np.zeros_like(v[k])
        for i in np.ndindex(*v[k].shape):
            w = {n: a.copy() for n, a in v.items()}
            w[k][i] += h
            up = loss(w)
            w[k][i] -= 2 * h
            num[i] = (up - loss(w)) / (2 * h)
        # differences: h^2 times third derivatives (below 100 at these sizes) and 2^-52 |loss| / h
        assert np.max(np.abs(num - got[names[k]])) <= 1e-7, k


def test_normalise_by_hand():
    n, r = acts.normalise([[3.0, 4.0]], "rms", 0.0)
    assert np.allclose(n, [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5)]]) and np.allclose(r, [1 / np.sqrt(12.5)])
    n, r = acts.normalise([[1.0, 3.0]], "layer", 0.0)
    assert np.allclose(n, [[-1.0, 1.0]]) and np.allclose(r, [1.0])
