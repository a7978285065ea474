"""GPU parity of seam_forward and seam_backward against the fp64 oracle (oracle/acts.py).

Tolerances, from the arithmetic (u = 2^-24, fp32's half unit; H = half a unit of the
stored type, eps / 2):
  sums over a row: a thread adds at most 16 values one after another (at most 32 where a warp holds the
    row), then 5 + 5 shuffles: at most 42 roundings, each at most u times the sum of magnitudes.
  r      of a mean square (all terms positive): (42 + 3) u / 2 + 2 u < 2^-19 relative
  n      |dn| <= 2^-18 (|n| + r (mean|v| + |v|)): r's error and, behind a mean, the mean's
  codes  |q 2^e - n| <= 2^(e-1) + dn, e the smallest that holds the block up to dn
  x', y  the error carried through (at most 6 more roundings, inside the same 2^-18 of the magnitudes
         that enter) and one rounding H.  y is checked from the x' that was stored.
  backward: with A the magnitudes that enter an element (formulas below), 2^-18 A and one rounding H;
  sums over T tokens add T roundings: (2^-18 + T u) sum A, and H.
"""
import threading

import numpy as np
import pytest
import torch

import muon_family_optimizer_b200 as mo
from oracle import acts

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
R = 2.0 ** -18


def _np(t):
    return t.detach().double().cpu().numpy()


def _half(dt):
    return torch.finfo(dt).eps / 2


def _tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def _mat(T, C, dt, g, scale=1.0, mean=0.0, pad=0, base=0):
    buf = torch.zeros(base + T * (C + pad) + 8, dtype=dt, device="cuda")
    v = buf.as_strided((T, C), (C + pad, 1), base)
    v.copy_((torch.randn(T, C, generator=g) * scale + mean).to(dt))
    return v


def _build(T, C, dt, wt, post, pre, gate_rows, *, f=True, bias=None, seed=0, pad=0, base=0, mean=0.0, keep=True,
           skip=0.75, scale=0.5, gain=True):
    g = torch.Generator().manual_seed(seed)
    bias = ("layer" in (post, pre)) if bias is None else bias
    s = dict(post=post, pre=pre, eps=1e-5, x=_mat(T, C, dt, g, mean=mean, pad=pad, base=base))
    w = lambda: (1 + 0.3 * torch.randn(C, generator=g)).to(wt).cuda()  # noqa: E731
    if f:
        s.update(skip=skip, scale=scale, f=_mat(T, C, dt, g, 2.0, mean, pad, base), out=_mat(T, C, dt, g, pad=pad, base=base))
        if gain:
            s["post_gain"] = w()
        if bias:
            s["post_bias"] = w()
        if gate_rows:
            s.update(gate=_mat(-(-T // gate_rows), C, dt, g, pad=pad, base=base), gate_rows=gate_rows)
        if post != "none":
            s["post_rstd"] = torch.empty(T, device="cuda")
        if keep:
            s["post_c"] = mo.act8_empty(T, C)
    if pre != "none":
        s["y"] = _mat(T, C, dt, g, pad=pad, base=base)
        if gain:
            s["pre_gain"] = w()
        if bias:
            s["pre_bias"] = w()
        s["pre_rstd"] = torch.empty(T, device="cuda")
        if keep:
            s["pre_c"] = mo.act8_empty(T, C)
    return s


def _vecs(s, *names):
    return {k: _np(s[k]) for k in names if s.get(k) is not None}


def _check_ckpt(c, n, dn):
    q, e = c["q"].cpu().numpy().astype(np.float64), c["e"].cpu().numpy().astype(np.int64)
    assert np.all((e >= 7) & (e <= 246))
    step = 2.0 ** (np.repeat(e, 32, axis=1)[:, :n.shape[1]] - 127.0)
    assert np.all(np.abs(q) <= 127) and np.all(np.abs(q * step - n) <= step / 2 + dn)
    pad = -n.shape[1] % 32
    blocks = lambda a: np.pad(a, ((0, 0), (0, pad))).reshape(n.shape[0], -1, 32).max(axis=2)  # noqa: E731
    top, slack = blocks(np.abs(n)), blocks(dn)
    assert np.all(127 * 2.0 ** (e - 127.0) >= top - slack)
    assert np.all((e == 7) | (127 * 2.0 ** (e - 128.0) < top + slack))


def _dn(v, kind, n, r):
    v = np.abs(v)
    return 0.0 * v if kind == "none" else R * (np.abs(n) + r[:, None] * (v.mean(axis=1, keepdims=True) + v))


def _check_forward(s):
    dt = s["x"].dtype
    args = dict(post=s["post"], pre=s["pre"], eps=float(np.float32(s["eps"])), skip=s.get("skip", 1.0),
                scale=s.get("scale", 1.0), gate_rows=s.get("gate_rows") or 1,
                **_vecs(s, "gate", "post_gain", "post_bias", "pre_gain", "pre_bias"))
    x, f = _np(s["x0"] if "x0" in s else s["x"]), _np(s["f0"] if "f0" in s else s["f"]) if "f" in s else None
    stored = _np(s["out"]) if f is not None else None
    ref = acts.seam_forward(x, f, round_out=lambda v: stored, **args)
    if f is not None:
        dn = _dn(f, s["post"], ref["n_f"], ref["post_rstd"])
        if s.get("post_rstd") is not None:
            assert np.all(np.abs(_np(s["post_rstd"]) - ref["post_rstd"]) <= R * ref["post_rstd"] * (
                1 if s["post"] == "rms" else 1 + np.abs(f).mean(axis=1) * ref["post_rstd"]))
        if s.get("post_c") is not None:
            _check_ckpt(s["post_c"], ref["n_f"], dn)
        g = np.abs(acts.gate_of(args.get("gate"), x.shape[0], args["gate_rows"])) * abs(args["scale"])
        pg, pb = np.abs(args.get("post_gain", np.ones(1))), np.abs(args.get("post_bias", np.zeros(1)))
        err = g * pg * dn + R * (g * (np.abs(ref["n_f"]) * pg + pb) + np.abs(args["skip"] * x))
        err = err + _half(dt) * (np.abs(ref["out"]) + err) + _tiny(dt)
        assert np.all(np.abs(stored - ref["out"]) <= err)
        x = stored
    if s["pre"] != "none":
        dn = _dn(x, s["pre"], ref["n"], ref["pre_rstd"])
        if s.get("pre_rstd") is not None:
            assert np.all(np.abs(_np(s["pre_rstd"]) - ref["pre_rstd"]) <= R * ref["pre_rstd"] * (
                1 if s["pre"] == "rms" else 1 + np.abs(x).mean(axis=1) * ref["pre_rstd"]))
        if s.get("pre_c") is not None:
            _check_ckpt(s["pre_c"], ref["n"], dn)
        g, b = np.abs(args.get("pre_gain", np.ones(1))), np.abs(args.get("pre_bias", np.zeros(1)))
        err = g * dn + R * (np.abs(ref["n"]) * g + b)
        err = err + _half(dt) * (np.abs(ref["y"]) + err) + _tiny(dt)
        assert np.all(np.abs(_np(s["y"]) - ref["y"]) <= err)


def _back_of(s, *, seed=1, dout=True, pad=0, base=0, wt=FP, beta=0.0, vectors=True):
    """The gradient call of a seam that has run forward."""
    T, C = s["x"].shape
    dt = s["x"].dtype
    g = torch.Generator().manual_seed(seed)
    b = {k: s[k] for k in ("post", "pre", "skip", "scale", "gate", "gate_rows", "post_gain", "post_bias", "pre_gain",
                           "post_c", "pre_c", "post_rstd", "pre_rstd") if k in s}
    b["dx"] = _mat(T, C, dt, g, pad=pad, base=base)
    if s["pre"] != "none":
        b["dy"] = _mat(T, C, dt, g, pad=pad, base=base)
    if dout or s["pre"] == "none":
        b["dout"] = _mat(T, C, dt, g, pad=pad, base=base)
    if "f" in s:
        b["df"] = _mat(T, C, dt, g, pad=pad, base=base)
        if s.get("gate") is not None:
            b["dgate"] = _mat(*s["gate"].shape, dt, g, pad=pad, base=base)
    if vectors:
        for side in ("post", "pre"):
            for k in ("gain", "bias"):
                if s.get(f"{side}_{k}") is not None:
                    b[f"d_{side}_{k}"] = torch.randn(C, generator=g).to(s[f"{side}_{k}"].dtype).cuda()
        b["beta"] = beta
    return b


def _run_back(b, stream=None):
    n = mo.seam_backward_workspace_size(b)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    mo.seam_backward(b, ws, stream=stream)
    return ws


def _values(c):
    return None if c is None else acts.decode(c["q"].cpu().numpy(), c["e"].cpu().numpy())


def _back_inputs(b):
    got = _vecs(b, "dy", "dout", "gate", "post_gain", "post_bias", "pre_gain", "pre_rstd", "post_rstd", "d_post_gain",
                "d_post_bias", "d_pre_gain", "d_pre_bias")
    got["n"], got["n_f"] = _values(b.get("pre_c")), _values(b.get("post_c"))
    return got


def _check_back(b, v):
    """b after the call; v: _back_inputs(b) taken before it."""
    dt = b["dx"].dtype
    T, C = b["dx"].shape
    kw = dict(post=b["post"], pre=b["pre"], skip=b.get("skip", 1.0), scale=b.get("scale", 1.0),
              gate_rows=b.get("gate_rows") or 1, has_f="df" in b)
    ref = acts.seam_backward(**{k: v.get(k) for k in ("dy", "dout", "n", "n_f", "pre_rstd", "post_rstd", "gate", "post_gain",
                                                      "post_bias", "pre_gain")}, **kw)
    A = np.abs(v["dout"]) if "dout" in v else np.zeros((T, C))
    m = lambda a: a.mean(axis=1, keepdims=True)  # noqa: E731
    if b["pre"] != "none":
        g = np.abs(v["dy"]) * np.abs(v.get("pre_gain", np.ones(1)))
        n = np.abs(v["n"])
        A = A + v["pre_rstd"][:, None] * (g + (m(g) if b["pre"] == "layer" else 0) + n * m(g * n))

    def close(name, got, want, mag):
        err = mag + _half(got.dtype) * (np.abs(want) + mag) + _tiny(got.dtype)
        assert np.all(np.abs(_np(got) - want) <= err), (name, float(np.max(np.abs(_np(got) - want) - err)))
    close("dx", b["dx"], ref["dx"], R * abs(kw["skip"]) * A)
    tok = R + T * 2.0 ** -24
    beta = b.get("beta", 0.0)

    def vector(name, mag):
        if b.get(name) is not None:
            want = ref[name] + (beta * v[name] if beta else 0.0)
            close(name, b[name], want, tok * (mag.sum(axis=0) + (np.abs(beta * v[name]) if beta else 0.0)))
    if b["pre"] != "none":
        vector("d_pre_gain", np.abs(v["dy"]) * np.abs(v["n"]))
        vector("d_pre_bias", np.abs(v["dy"]))
    if "df" not in b:
        return
    gate = np.abs(acts.gate_of(v.get("gate"), T, kw["gate_rows"])) * abs(kw["scale"])
    gain = np.abs(v.get("post_gain", np.ones(1)))
    du = gate * A * np.ones((T, C))
    h = du * gain
    nf = np.abs(v["n_f"]) if v["n_f"] is not None else np.zeros((T, C))
    mag = h if b["post"] == "none" else v["post_rstd"][:, None] * (h + (m(h) if b["post"] == "layer" else 0) + nf * m(h * nf))
    close("df", b["df"], ref["df"], R * mag)
    vector("d_post_bias", du)
    vector("d_post_gain", du * nf)
    if b.get("dgate") is not None:
        each = abs(kw["scale"]) * A * (nf * gain + np.abs(v.get("post_bias", np.zeros(1))))
        gr = kw["gate_rows"]
        sums = np.stack([each[i:i + gr].sum(axis=0) for i in range(0, T, gr)])
        close("dgate", b["dgate"], ref["dgate"], tok * sums)


def _both(s, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mo.seam_forward(s, d_status=status)
    _check_forward(s)
    b = _back_of(s, **kw)
    v = _back_inputs(b)
    _run_back(b)
    _check_back(b, v)
    assert int(status.item()) == 0


KINDS = ["none", "rms", "layer"]


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("pre", KINDS)
@pytest.mark.parametrize("dt,wt", [(BF, BF), (HF, FP), (FP, FP)])
def test_every_pair_of_norms(post, pre, dt, wt):
    for gate_rows in (0, 1, 4, 19):
        _both(_build(19, 136, dt, wt, post, pre, gate_rows, seed=gate_rows))


@pytest.mark.parametrize("T,C", [(1, 1), (1, 7), (2, 8), (3, 31), (5, 32), (9, 33), (2, 255), (6, 257), (5, 511), (3, 513),
                                 (5, 768), (4, 1000), (3, 1025), (2, 2048), (3, 2056), (2, 4096), (3, 4104), (2, 8192),
                                 (2, 8200), (2, 16383), (3, 16384)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_row_lengths(T, C, dt):
    _both(_build(T, C, dt, dt, "rms", "layer", 1, seed=C))
    _both(_build(T, C, dt, FP, "layer", "rms", 2, seed=C + 1))
    _both(_build(T, C, dt, dt, "rms", "rms", 0, seed=C + 2))


@pytest.mark.parametrize("T", [1, 2, 147, 1000, 2999])
@pytest.mark.parametrize("gate_rows", [0, 1, 2, 3, 7, 64, 1000, 5000])
def test_many_tokens(T, gate_rows):
    # runs of rows in every relation to the gate rows: whole groups in a run, runs inside a group, a short last group
    _both(_build(T, 72, BF, FP, "rms", "rms", gate_rows, seed=T + gate_rows))


def test_many_tokens_long_rows():
    for gate_rows in (0, 50, 700):
        _both(_build(1500, 1536, BF, BF, "rms", "layer", gate_rows, seed=gate_rows))


@pytest.mark.parametrize("pad,base", [(8, 0), (1, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_strided_and_unaligned(pad, base, dt):
    for C in (40, 264, 1100):
        _both(_build(11, C, dt, dt, "rms", "layer", 3, seed=C, pad=pad, base=base), pad=pad, base=base)


@pytest.mark.parametrize("pad,base", [(0, 0), (0, 4), (4, 0), (8, 8)])
@pytest.mark.parametrize("C", [1032, 8200])
def test_fp32_rows_on_16_and_on_32_byte_boundaries(pad, base, C):
    _both(_build(5, C, FP, FP, "rms", "layer", 1, seed=C, pad=pad, base=base), pad=pad, base=base)


def test_without_f():
    for pre in ("rms", "layer"):
        s = _build(13, 300, BF, BF, "none", pre, 0, f=False)
        _both(s)
        s2 = _build(13, 300, BF, BF, "none", pre, 0, f=False)
        mo.seam_forward(s2)
        b = _back_of(s2, dout=False)
        v = _back_inputs(b)
        _run_back(b)
        _check_back(b, v)


def test_without_gains_and_vectors():
    s = _build(17, 520, BF, FP, "rms", "rms", 1, gain=False, bias=False)
    mo.seam_forward(s)
    _check_forward(s)
    b = _back_of(s, vectors=False)
    assert mo.seam_backward_workspace_size(b) == 0
    v = _back_inputs(b)
    mo.seam_backward(b)
    _check_back(b, v)


@pytest.mark.parametrize("C", [40, 136, 203, 1003, 4104])
def test_layer_norms_without_gains(C):
    # no gain to hide what a thread without columns adds to the row's sums
    s = _build(7, C, FP, FP, "layer", "layer", 0, gain=False, bias=False)
    mo.seam_forward(s)
    _check_forward(s)
    b = _back_of(s, vectors=False)
    v = _back_inputs(b)
    _run_back(b)
    _check_back(b, v)


def test_without_checkpoints_or_deviations():
    s = _build(9, 264, BF, FP, "rms", "layer", 1, keep=False)
    full = _build(9, 264, BF, FP, "rms", "layer", 1)
    for k in ("post_rstd", "pre_rstd"):
        s.pop(k)
    mo.seam_forward(s)
    mo.seam_forward(full)
    assert torch.equal(s["out"], full["out"]) and torch.equal(s["y"], full["y"])


def test_joined_seam_equals_two_calls():
    # x' is normalised as it was stored, so one call equals the residual sum and the norm made apart
    s = _build(23, 1032, BF, BF, "rms", "rms", 4)
    mo.seam_forward(s)
    a = {k: v for k, v in s.items() if not k.startswith("pre") and k != "y"}
    a.update(pre="none", out=torch.empty_like(s["out"]))
    mo.seam_forward(a)
    n = dict(post="none", pre="rms", eps=s["eps"], x=a["out"], y=torch.empty_like(s["y"]), pre_gain=s["pre_gain"],
             pre_c=mo.act8_empty(23, 1032))
    mo.seam_forward(n)
    assert torch.equal(a["out"], s["out"]) and torch.equal(n["y"], s["y"])
    assert torch.equal(n["pre_c"]["q"], s["pre_c"]["q"]) and torch.equal(n["pre_c"]["e"], s["pre_c"]["e"])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_of_zeros_large_means_and_large_values(kind):
    s = _build(6, 256, FP, FP, kind, kind, 0, seed=2, bias=True)
    s["f"][0] = 0
    s["f"][1] = 5.0                                  # no deviation at all
    s["f"][2] += 300.0                               # a mean far above the deviation
    s["f"][3] *= 1e-20
    if kind == "rms":
        s["f"][4] *= 1e25                            # squares beyond fp32
    mo.seam_forward(s)
    _check_forward(s)
    b = _back_of(s)
    v = _back_inputs(b)
    _run_back(b)
    _check_back(b, v)


def test_values_that_are_not_finite_are_flagged():
    s = _build(5, 96, FP, FP, "none", "rms", 0, f=False)
    s["x"][3, 50] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mo.seam_forward(s, d_status=status)
    assert int(status.item()) == mo.FLAG_NONFINITE
    e = s["pre_c"]["e"].cpu()
    assert int(e[3, 1]) == 255 and int((e == 255).sum()) == 1
    assert bool(torch.isfinite(s["y"][[0, 1, 2, 4]]).all())


def test_in_place():
    # out on x or on f; dx and df on dout and dy
    for pre, gate_rows in (("rms", 1), ("layer", 3)):
        ref = _build(21, 520, BF, FP, "rms", pre, gate_rows, seed=5)
        mo.seam_forward(ref)
        for k in ("x", "f"):
            s = _build(21, 520, BF, FP, "rms", pre, gate_rows, seed=5)
            s["out"] = s[k]
            mo.seam_forward(s)
            assert torch.equal(s["out"], ref["out"]) and torch.equal(s["y"], ref["y"])
        b = _back_of(ref)
        _run_back(b)
        for dx, df in (("dout", "dy"), ("dy", "dout")):
            i = _back_of(ref)
            i["dx"], i["df"] = i[dx], i[df]
            _run_back(i)
            for k in ("dx", "df", "dgate", "d_pre_gain", "d_post_gain"):
                assert torch.equal(i[k], b[k]), (dx, k)


@pytest.mark.parametrize("beta", [1.0, 0.5])
def test_vector_gradients_accumulate(beta):
    for wt in (FP, BF):
        _both(_build(300, 136, BF, wt, "layer", "layer", 0, seed=9), beta=beta)


def test_beta_zero_does_not_read():
    s = _build(30, 136, BF, FP, "rms", "rms", 5)
    mo.seam_forward(s)
    b = _back_of(s)
    b["d_pre_gain"].fill_(float("nan"))
    b["dgate"].fill_(float("nan"))
    v = _back_inputs(b)
    _run_back(b)
    _check_back(b, v)


def test_no_rows():
    s = _build(0, 64, BF, FP, "rms", "rms", 1)
    mo.seam_forward(s)
    b = _back_of(s, beta=0.5)
    before = b["d_pre_gain"].clone()
    _run_back(b)
    assert torch.equal(b["d_pre_gain"], before * 0.5)


def test_equal_inputs_give_equal_bits():
    s = _build(2000, 264, BF, FP, "rms", "rms", 300)
    mo.seam_forward(s)
    first = None
    for _ in range(4):
        b = _back_of(s)
        _run_back(b)
        got = [b[k].clone() for k in ("dx", "df", "dgate", "d_post_gain", "d_pre_gain")]
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_rows_behind_the_last_are_left():
    s = _build(9, 72, BF, FP, "rms", "rms", 2)
    big = {k: torch.full((12, 72), 3.0, dtype=BF, device="cuda") for k in ("out", "y")}
    for k in big:
        s[k] = big[k][:9]
    mo.seam_forward(s)
    b = _back_of(s)
    for k in ("dx", "df"):
        big[k] = torch.full((12, 72), 3.0, dtype=BF, device="cuda")
        b[k] = big[k][:9]
    _run_back(b)
    for t in big.values():
        assert bool((t[9:] == 3.0).all())


def test_captured_graph_on_its_own_stream():
    s = _build(600, 264, BF, FP, "rms", "rms", 100)
    mo.seam_forward(s)
    b = _back_of(s)
    ws = torch.empty(mo.seam_backward_workspace_size(b), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        mo.seam_backward(b, ws)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        mo.seam_forward(s)
        mo.seam_backward(b, ws)
    for k in range(2):
        s["x"].mul_(0.5 + k)
        s["f"].neg_()
        b["dy"].mul_(-2.0)
        g.replay()
        torch.cuda.synchronize()
        _check_forward(s)
        _check_back(b, _back_inputs(b))


def test_workspace_is_required():
    s = _build(9, 72, BF, FP, "rms", "rms", 0)
    mo.seam_forward(s)
    b = _back_of(s)
    need = mo.seam_backward_workspace_size(b)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(mo.MuonError) as err:
            mo.seam_backward(b, ws)
        assert err.value.status == mo.ERR_WORKSPACE


def test_offsets_beyond_32_bits():
    # rows 2^31 + 64 elements apart: row 2 starts past 2^32
    ld, T, C = 2 ** 31 + 64, 3, 72
    s = _build(T, C, BF, FP, "rms", "rms", 0)
    buf = torch.empty(2 * ld + C, dtype=BF, device="cuda")
    x = buf.as_strided((T, C), (ld, 1))
    x.copy_(s["x"])
    s["x"] = x
    _both(s)


def test_a_block_trained_end_to_end():
    """Two blocks, each pre-norm -> linear -> tanh -> linear -> post-norm, gate and residual sum: forward with the
    seams, backward from the 8-bit checkpoints alone, gradients into one muon_model_step.  The matrix gradients are
    checked against the oracle's from the same checkpoints (as above), the whole against fp64 autograd of the same
    network: the checkpoints' error, at most 2^(e-1) <= max / 127 an element, moves a gradient far less than the 5%
    allowed here (it enters G linearly and nothing else)."""
    T, C, D, L = 192, 128, 256, 2
    g = torch.Generator().manual_seed(0)
    dt = FP
    W = [[(torch.randn(D, C, generator=g) / C ** 0.5).cuda(), (torch.randn(C, D, generator=g) / D ** 0.5).cuda()]
         for _ in range(L)]
    gains = [[torch.ones(C, device="cuda"), (1 + 0.1 * torch.randn(C, generator=g)).cuda()] for _ in range(L)]
    gate = [(1 + 0.2 * torch.randn(1, C, generator=g)).cuda() for _ in range(L)]
    x0, target = torch.randn(T, C, generator=g).cuda(), torch.randn(T, C, generator=g).cuda()

    # forward: seam 0 is the first pre-norm alone, seam l joins block l - 1 and makes block l's input
    seams, saved, x = [], [], x0
    f = None
    for l in range(L + 1):
        s = dict(post="rms" if l else "none", pre="rms" if l < L else "none", eps=1e-5, x=x)
        if l:
            s.update(f=f, out=torch.empty(T, C, device="cuda"), scale=0.5, gate=gate[l - 1], gate_rows=T,
                     post_gain=gains[l - 1][1], post_c=mo.act8_empty(T, C), post_rstd=torch.empty(T, device="cuda"))
        if l < L:
            s.update(y=torch.empty(T, C, device="cuda"), pre_gain=gains[l][0], pre_c=mo.act8_empty(T, C),
                     pre_rstd=torch.empty(T, device="cuda"))
        mo.seam_forward(s)
        seams.append(s)
        x = s["out"] if l else x0
        if l < L:
            a = torch.tanh(s["y"] @ W[l][0].T)
            c = mo.act8_empty(T, D)
            mo.act8_encode_batched([dict(x=a, **c)])
            saved.append((c, a))
            f = a @ W[l][1].T
    d = (x - target) / T

    # backward
    G = [[torch.empty_like(w) for w in pair] for pair in W]
    dgains, dgate = [[torch.empty(C, device="cuda") for _ in range(2)] for _ in range(L)], [torch.empty_like(v) for v in gate]
    dy, items = None, []
    for l in range(L, -1, -1):
        s = seams[l]
        b = {k: s[k] for k in ("post", "pre", "scale", "gate", "gate_rows", "post_gain", "pre_gain", "post_c", "pre_c",
                               "post_rstd", "pre_rstd") if k in s}
        b.update(dout=d, dx=torch.empty_like(d))
        if l < L:
            b.update(dy=dy, d_pre_gain=dgains[l][0])
        if l:
            b.update(df=torch.empty_like(d), dgate=dgate[l - 1], d_post_gain=dgains[l - 1][1])
        _run_back(b)
        d = b["dx"]
        if l:
            c, a = saved[l - 1]
            p = seams[l - 1]
            da = (b["df"] @ W[l - 1][1]) * (1 - a * a)
            items += [dict(dY=b["df"], G=G[l - 1][1], **c),
                      dict(dY=da, G=G[l - 1][0], gain=p["pre_gain"], **p["pre_c"])]
            dy = da @ W[l - 1][0]
    n = mo.act8_grad_workspace_size(items)
    mo.act8_grad_batched(items, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    for it in items:
        X = _values(it)
        ref = acts.grad(_np(it["dY"]), X, gain=None if it.get("gain") is None else _np(it["gain"]))
        S = np.abs(_np(it["dY"])).T @ np.abs(X) * (1 if it.get("gain") is None else np.abs(_np(it["gain"])))
        assert np.all(np.abs(_np(it["G"]) - ref) <= (3 * T + 4) * 2.0 ** -23 * S + 2.0 ** -24 * np.abs(ref))

    # the same network in fp64
    leaf = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    W64, g64, t64 = [[leaf(w) for w in p] for p in W], [[leaf(w) for w in p] for p in gains], [leaf(v) for v in gate]
    x64 = x0.double().cpu()
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5)  # noqa: E731
    for l in range(L):
        h = torch.tanh((rms(x64) * g64[l][0]) @ W64[l][0].T) @ W64[l][1].T
        x64 = x64 + 0.5 * t64[l] * (rms(h) * g64[l][1])
    (((x64 - target.double().cpu()) ** 2).sum() / (2 * T)).backward()
    for got, want in [(G[l][i], W64[l][i].grad) for l in range(L) for i in range(2)] + \
            [(dgains[l][i], g64[l][i].grad) for l in range(L) for i in range(2)] + \
            [(dgate[l], t64[l].grad) for l in range(L)]:
        assert float((got.double().cpu() - want).norm() / want.norm()) <= 0.05

    # one optimizer step on them
    mats = [dict(W=w, G=gr, G_prev=torch.zeros_like(w), A=torch.zeros_like(w), M=torch.zeros_like(w))
            for pw, pg in zip(W, G) for w, gr in zip(pw, pg)]
    vecs = [dict(W=w, G=gr, m=torch.zeros_like(w), v=torch.zeros_like(w))
            for pw, pg in list(zip(gains, dgains)) + [(gate, dgate)] for w, gr in zip(pw, pg)]
    before = [p["W"].clone() for p in mats + vecs]
    sched = mo.quintic_schedule(5)
    ws = torch.empty(mo.muon_workspace_size(mats, mo.BF16, sched), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mo.muon_model_step(mats, vecs, mo.FP32, mo.BF16, dict(mu=0.95, eta=0.01, gamma=1.0, beta_a=0.9, alpha=0.5,
                                                          **{"lambda": 0.0}),
                       dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0), 1, sched, ws, d_status=status)
    assert int(status.item()) == 0
    for p, w in zip(mats + vecs, before):
        assert bool(torch.isfinite(p["W"]).all()) and not torch.equal(p["W"], w)


def test_calls_of_two_threads():
    # seams of different widths that share a kernel, and their gradients, called from two threads at once
    jobs = []
    for C, pre in ((4096, "layer"), (1032, "rms")):
        s = _build(3, C, BF, BF, "rms", pre, 1, seed=C)
        mo.seam_forward(s)
        b = _back_of(s)
        ws = _run_back(b)
        outs = [s["out"], s["y"], b["dx"], b["df"], b["dgate"]]
        jobs.append((mo.make_seam(s), mo.make_seam_grad(b), ws, outs, [t.clone() for t in outs], (s, b)))   # (s, b): alive
    torch.cuda.synchronize()
    errors = []
    start = threading.Barrier(2)

    def run(fwd, back, ws):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(2000):
                mo.seam_forward(fwd, stream=stream)
                mo.seam_backward(back, ws, stream=stream)
        except Exception as e:          # noqa: BLE001 - reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=job[:3]) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for _, _, _, outs, ref, _ in jobs:
        assert all(torch.equal(a, r) for a, r in zip(outs, ref))


@pytest.mark.parametrize("C", [72, 768, 1003, 4096, 16384])
@pytest.mark.parametrize("mean", [1e4, -300.0])
def test_layer_norm_of_rows_far_from_zero(C, mean):
    # The bound that the header states: with b = 42 u r mean|v| (u = 2^-24), the mean's error times r, n is off by b, and r, whose
    # mean square grows by the error's own square, by b^2 / 2; its sums' and the root's roundings 2^-19, two more of n u each.
    v = (torch.randn(5, C, generator=torch.Generator().manual_seed(C)) + mean).cuda()
    s = dict(post="layer", x=torch.zeros_like(v), f=v, out=torch.empty_like(v), post_rstd=torch.empty(5, device="cuda"))
    mo.seam_forward(s)
    n, r = acts.normalise(_np(v), "layer", float(np.float32(1e-5)))
    b = 42 * 2.0 ** -24 * r * np.abs(_np(v)).mean(axis=1)
    assert np.all(np.abs(_np(s["post_rstd"]) - r) <= r * (b * b / 2 + 2.0 ** -19))
    b = b[:, None]
    assert np.all(np.abs(_np(s["out"]) - n) <= b + (np.abs(n) + b) * (b * b / 2 + 2.0 ** -19 + 2.0 ** -23))
