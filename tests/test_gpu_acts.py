"""GPU parity of the 8-bit activation checkpoints and the weight gradients made from
them, against the fp64 oracle (oracle/acts.py).

Tolerances, from the arithmetic:
  codes and exponents   equal: x 2^-e is exact and rounded once, in both
  values                equal: q 2^e is exact in bfloat16 and fp32; fp16 one rounding, the same in both
  G     a product of a dY and a checkpoint value is exact in fp32 (at most 11 + 11 significant
        bits; fp32 dY: three bfloat16 parts that sum to it), so an element's error is that of the
        fp32 sum of T (fp32 dY: 3 T) terms, at most 2^-23 each times S = sum |dY| |X^| (a sum that
        truncates loses a whole unit in the last place per addition), of the three operations of the
        epilogue, and the rounding to G's type: half a unit, eps / 2 of the result.
"""
import threading

import numpy as np
import pytest
import torch

import muon_family_optimizer_b200 as mo
from oracle import acts

pytestmark = pytest.mark.gpu

DTS = [torch.bfloat16, torch.float16, torch.float32]
GUARD = 77          # what memory outside a result holds, before and after


def _np(t):
    return t.detach().double().cpu().numpy()


def _x(T, C, dt, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g) * torch.exp(spread * torch.randn(T, 1, generator=g))
    if T and C > 40:
        x[0, :32] = 0                               # an empty block
    if T > 2:
        x[2] = 0                                    # an empty row
    return x.to(dt).cuda()


def _padded(T, C, pad, dtype, fill=GUARD, base=0):
    """A T x C view with row stride C + pad, `base` elements into its buffer, and the buffer."""
    buf = torch.full((base + T * (C + pad) + 64,), fill, dtype=dtype, device="cuda")
    return buf.as_strided((T, C), (C + pad, 1), base), buf


def _ckpt_of(x):
    c = mo.act8_empty(*x.shape)
    mo.act8_encode_batched([dict(x=x, **c)])
    return c


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,C", [(1, 1), (1, 31), (3, 32), (5, 33), (4, 40), (7, 255), (2, 256), (9, 1000), (130, 768),
                                 (33, 4097)])
@pytest.mark.parametrize("layout", ["dense", "strided", "unaligned"])
def test_encode_and_decode(dt, T, C, layout):
    x = _x(T, C, dt, seed=T + C)
    if layout != "dense":
        v, _ = _padded(T, C, 24 if layout == "strided" else 3, dt, 0, 0 if layout == "strided" else 1)
        v.copy_(x)
        x = v
    ld = (C + 15) // 16 * 16 + 32
    qb = torch.full((T * ld,), GUARD, dtype=torch.int8, device="cuda")
    q = qb.view(T, ld)[:, :C]
    nb = -(-C // 32)
    e, eb = _padded(T, nb, 5, torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mo.act8_encode_batched([dict(x=x, q=q, e=e)], d_status=status)
    q_ref, e_ref = acts.encode(_np(x))
    assert int(status.item()) == 0
    assert np.array_equal(q.cpu().numpy(), q_ref) and np.array_equal(e.cpu().numpy(), e_ref)
    assert bool((qb.view(T, ld)[:, C:] == GUARD).all())            # the rest of the buffers is untouched
    assert int((eb == GUARD).sum()) >= eb.numel() - T * nb
    for to in DTS:
        out, ob = _padded(T, C, 8, to)
        mo.act8_decode_batched([dict(x=out, q=q, e=e)])
        ref = torch.from_numpy(acts.decode(q_ref, e_ref)).to(to)
        assert torch.equal(out.cpu(), ref)
        assert bool((ob.as_strided((T, 8), (C + 8, 1), C) == GUARD).all())


def test_encode_marks_blocks_it_cannot_hold():
    x = torch.ones(4, 100, device="cuda")
    x[0, 40] = float("nan")
    x[1, 99] = float("inf")
    x[2, 0] = 3e38
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = mo.act8_empty(4, 100)
    mo.act8_encode_batched([dict(x=x, **c)], d_status=status)
    assert int(status.item()) == mo.FLAG_NONFINITE
    out = torch.empty_like(x)
    mo.act8_decode_batched([dict(x=out, **c)])
    nan = torch.isnan(out).cpu()
    expect = torch.zeros(4, 100, dtype=torch.bool)
    expect[0, 32:64] = True
    expect[1, 96:] = True
    expect[2, :32] = True
    assert torch.equal(nan, expect)
    q_ref, e_ref = acts.encode(_np(x))
    assert np.array_equal(c["q"].cpu().numpy(), q_ref) and np.array_equal(c["e"].cpu().numpy(), e_ref)


def test_many_items_of_ragged_length_one_of_them_empty():
    # more items than one launch takes; an item without rows changes nothing
    sizes = [(0, 64)] + [(1 + 7 * i % 23, 1 + 37 * i % 300) for i in range(130)] + [(0, 5)]
    xs = [_x(t, c, torch.bfloat16, seed=i) for i, (t, c) in enumerate(sizes)]
    cs = [mo.act8_empty(t, c) for t, c in sizes]
    mo.act8_encode_batched([dict(x=x, **c) for x, c in zip(xs, cs)])
    outs = [torch.empty_like(x) for x in xs]
    mo.act8_decode_batched([dict(x=x, **c) for x, c in zip(outs, cs)])
    for x, c, o in zip(xs, cs, outs):
        q_ref, e_ref = acts.encode(_np(x))
        assert np.array_equal(c["q"].cpu().numpy(), q_ref) and np.array_equal(c["e"].cpu().numpy(), e_ref)
        assert torch.equal(o.double().cpu(), torch.from_numpy(acts.decode(q_ref, e_ref)))


def test_offsets_beyond_32_bits():
    # rows 2^31 + 16 bytes apart: row 2 starts past 2^32
    ld, T, C = 2 ** 31 + 16, 3, 72
    buf = torch.empty(2 * ld + C + 16, dtype=torch.int8, device="cuda")
    q = buf.as_strided((T, C), (ld, 1))
    c = dict(q=q, e=torch.empty(T, 3, dtype=torch.uint8, device="cuda"))
    x = _x(T, C, torch.bfloat16, seed=5, spread=0.5)
    x[2] = 1.5
    mo.act8_encode_batched([dict(x=x, **c)])
    q_ref, e_ref = acts.encode(_np(x))
    assert np.array_equal(q.cpu().numpy(), q_ref)
    dY = torch.randn(T, 40, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    G = torch.empty(40, C, device="cuda")
    items = [dict(dY=dY, G=G, **c)]
    mo.act8_grad_batched(items, _ws(items))
    _check_G(G, dY, acts.decode(q_ref, e_ref))
    out = torch.empty_like(x)
    mo.act8_decode_batched([dict(x=out, **c)])
    assert torch.equal(out.double().cpu(), torch.from_numpy(acts.decode(q_ref, e_ref)))


# ---------------------------------------------------------------- gradients
def _ws(items):
    n = mo.act8_grad_workspace_size(items)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None      # no state: any contents


def _check_G(G, dY, X, gain=None, shift=None, dy_sum=None, beta=0.0, G0=None):
    if dY.dtype == torch.float16:
        X = torch.from_numpy(X).to(torch.float16).double().numpy()
    d = _np(dY)
    ref = acts.grad(d, X, gain=gain, shift=shift, dy_sum=dy_sum, beta=beta, G=G0)
    terms = d.shape[0] * (3 if dY.dtype == torch.float32 else 1)
    S = np.abs(d).T @ np.abs(X)
    if gain is not None:
        S = S * np.abs(gain)[None, :]
    own = np.abs(S)
    if shift is not None:
        own = own + np.abs(np.outer(dy_sum, shift))
    if beta:
        own = own + np.abs(beta * G0)
    half = torch.finfo(G.dtype).eps / 2
    tiny = torch.finfo(G.dtype).smallest_normal * torch.finfo(G.dtype).eps      # a step of the subnormals
    tol = terms * 2.0 ** -23 * S + 3 * 2.0 ** -23 * own
    tol = tol + half * (np.abs(ref) + tol) + tiny
    got = _np(G)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (float(np.max(np.abs(got - ref) - tol)), np.argwhere(bad)[:5].tolist())


def _case(T, O, C, dt, wt, seed=0, gain=False, shift=False, beta=0.0, pad=0, base=0):
    g = torch.Generator().manual_seed(seed)
    x = _x(T, C, torch.float32, seed=seed + 1, spread=0.3)
    c = _ckpt_of(x) if T else mo.act8_empty(0, C)
    dY, _ = _padded(T, O, pad, dt, 0, base)
    dY.copy_((torch.randn(T, O, generator=g) * 0.1).to(dt))
    G, buf = _padded(O, C, 0, wt, GUARD)
    it = dict(dY=dY, G=G, beta=beta, **c)
    if gain:
        it["gain"] = (1 + torch.randn(C, generator=g)).to(wt).cuda()
    if shift:
        it["shift"] = torch.randn(C, generator=g).to(wt).cuda()
        it["dy_sum"] = dY.float().sum(0)
    if beta:
        G.copy_(torch.randn(O, C, generator=g).to(wt))
    return it, buf


def _run_and_check(items, status=None):
    before = [_np(it["G"]) if it["beta"] else None for it in items]
    mo.act8_grad_batched(items, _ws(items), d_status=status)
    for it, G0 in zip(items, before):
        X = acts.decode(it["q"].cpu().numpy(), it["e"].cpu().numpy())
        opt = {k: _np(it[k]) for k in ("gain", "shift", "dy_sum") if it.get(k) is not None}
        _check_G(it["G"], it["dY"], X, beta=it["beta"], G0=G0, **opt)


SHAPES = [(1, 1, 1), (1, 64, 32), (2, 5, 3), (15, 33, 65), (16, 128, 128), (63, 130, 64), (64, 256, 256),
          (65, 257, 129), (100, 96, 520), (200, 300, 264), (333, 200, 768), (1000, 520, 72), (1025, 768, 256)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,O,C", SHAPES)
def test_grad(dt, T, O, C):
    items = []
    for k, wt in enumerate([torch.float32, dt]):
        it, buf = _case(T, O, C, dt, wt, seed=T + O + C + k, gain=k == 1)
        _run_and_check([it])
        assert bool((buf[O * C:] == GUARD).all())
        items.append(it)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("gain,shift,beta", [(True, True, 0.0), (False, True, 1.0), (True, False, 0.5), (False, False, -1.0)])
def test_grad_epilogue(dt, gain, shift, beta):
    for T, O, C in [(70, 72, 104), (0, 40, 64), (3, 300, 33)]:
        for wt in (torch.float32, torch.bfloat16):
            it, _ = _case(T, O, C, dt, wt, seed=3, gain=gain, shift=shift, beta=beta)
            _run_and_check([it])


@pytest.mark.parametrize("pad,base", [(8, 0), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("dt", DTS)
def test_grad_strided_and_unaligned_dY(dt, pad, base):
    it, _ = _case(77, 136, 96, dt, torch.float32, seed=4, pad=pad, base=base)
    _run_and_check([it])


@pytest.mark.parametrize("O,C", [(130, 308), (512, 308), (70, 4), (300, 1284)])
def test_grad_rows_that_end_inside_a_group_of_eight(O, C):
    # fp32 rows of 8 k + 4 columns are 16-byte aligned; over many tokens they go through the join, over few not
    for T in (40, 1984):
        for beta in (0.0, 1.0):
            it, buf = _case(T, O, C, torch.float16, torch.float32, seed=C, gain=True, shift=beta != 0, beta=beta)
            _run_and_check([it])
            assert bool((buf[O * C:] == GUARD).all())


def test_grad_without_tokens_writes_zeros():
    it, buf = _case(0, 130, 70, torch.bfloat16, torch.bfloat16)
    it["G"].fill_(float("nan"))
    mo.act8_grad_batched([it], _ws([it]))
    assert not it["G"].any()
    assert bool((buf[130 * 70:] == GUARD).all())


def test_grad_beta_zero_does_not_read_G():
    it, _ = _case(40, 64, 64, torch.bfloat16, torch.float32, seed=6)
    it["G"].fill_(float("nan"))
    _run_and_check([it])


def test_grad_ragged_experts_in_one_call():
    # experts with 0, 1, few and many tokens, of several shapes, a checkpoint and a dY used twice, more than one launch
    items = [_case(t, o, c, torch.bfloat16, torch.float32, seed=i, gain=i % 2 == 0)[0]
             for i, (t, o, c) in enumerate([(0, 72, 64), (1, 72, 64), (37, 72, 64), (300, 72, 64), (64, 40, 520)] * 30)]
    items.append(dict(items[3], G=torch.empty_like(items[3]["G"])))
    _run_and_check(items)
    assert torch.equal(items[3]["G"], items[-1]["G"])


def test_grad_equal_inputs_give_equal_bits():
    it, _ = _case(5000, 200, 264, torch.bfloat16, torch.float32, seed=8)
    _run_and_check([it])
    first = it["G"].clone()
    for _ in range(5):
        mo.act8_grad_batched([it], _ws([it]))
        assert torch.equal(it["G"], first)


def test_grad_long_sum():
    it, _ = _case(20001, 96, 64, torch.bfloat16, torch.float32, seed=9)
    _run_and_check([it])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_grad_long_sums_of_many_tiles_do_not_shrink(dt):
    # Whole tiles over 24576 tokens, with an fp32 G (81 tiles, so their tokens are not split).  The tensor cores truncate
    # the running sum at every 16 tokens, on average by half of at most 2^-23: over n steps of a sum that grows like a
    # random walk n 2^-24 2/3 of the result.  Segments hold at most 96 x 4 steps (a third of them in the hi parts of an fp32
    # dY): 1.6e-5; one sum over all 1536 steps measured 2.6e-5.
    T, O, C = 24576, 4608, 2304
    g = torch.Generator(device="cuda").manual_seed(3)
    c = _ckpt_of(torch.randn(T, C, generator=g, device="cuda"))
    dY = torch.randn(T, O, generator=g, device="cuda").to(dt)
    G = torch.empty(O, C, device="cuda")
    items = [dict(dY=dY, G=G, **c)]
    mo.act8_grad_batched(items, _ws(items))
    X = torch.empty(T, C, device="cuda")
    mo.act8_decode_batched([dict(x=X, **c)])
    ref = dY.double().T @ X.double()
    assert float((G.double() - ref).norm() / ref.norm()) <= 1.6e-5


@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("gain,shift,beta", [(False, False, 1.0), (True, True, 0.5)])
def test_grad_added_to_G_over_many_tiles(wt, gain, shift, beta):
    # more tiles than pairs of SMs, the last row of tiles and the last column of tiles partly outside of G
    it, buf = _case(130, 4648, 2296, torch.bfloat16, wt, seed=11, gain=gain, shift=shift, beta=beta)
    _run_and_check([it])
    assert bool((buf[4648 * 2296:] == GUARD).all())


@pytest.mark.parametrize("C,base,beta", [(2304, 0, 1.0), (2304, 4, 1.0), (2300, 0, 1.0), (2304, 0, 0.5), (2304, 4, 0.0)])
def test_grad_fp32_segments_are_added_to_G(C, base, beta):
    # 81 whole tiles over 98 k-blocks of 64 tokens, so two segments of 49 x 4 steps at the most; the error of the product as in
    # the test above, 196 x 2^-24 x 2/3, and three roundings.  Rows that can be written in 32-byte pieces, in 16-byte pieces,
    # and whose last group of eight columns is half there.
    T, O = 6272, 4608
    g = torch.Generator(device="cuda").manual_seed(4)
    c = _ckpt_of(torch.randn(T, C, generator=g, device="cuda"))
    dY = torch.randn(T, O, generator=g, device="cuda").to(torch.bfloat16)
    buf = torch.randn(base + O * C + 8, generator=g, device="cuda") * 50
    G, before = buf[base:base + O * C].view(O, C), buf.clone()
    G0, gain = before[base:base + O * C].view(O, C), torch.randn(C, generator=g, device="cuda")
    items = [dict(dY=dY, G=G, gain=gain, beta=beta, **c)]
    mo.act8_grad_batched(items, _ws(items))
    X = torch.empty(T, C, device="cuda")
    mo.act8_decode_batched([dict(x=X, **c)])
    product = (dY.double().T @ X.double()) * gain.double()
    err = G.double() - (product + beta * G0.double())
    assert float(err.norm()) <= 196 * 2.0 ** -24 * 2 / 3 * float(product.norm()) + 3 * 2.0 ** -24 * float((product.abs() + beta * G0.abs()).norm())
    assert torch.equal(buf[:base], before[:base]) and torch.equal(buf[base + O * C:], before[base + O * C:])


def test_grad_extreme_exponents():
    # blocks at the ends of the exponent range times a dY that brings the sum back into range
    for s, d in ((2.0 ** 118, 2.0 ** -100), (2.0 ** -116, 2.0 ** 100)):
        x = torch.randn(40, 64, generator=torch.Generator().manual_seed(2)).cuda() * s
        c = _ckpt_of(x)
        dY = (torch.randn(40, 48, generator=torch.Generator().manual_seed(3)) * d).to(torch.bfloat16).cuda()
        it = dict(dY=dY, G=torch.empty(48, 64, device="cuda"), beta=0.0, **c)
        _run_and_check([it])


def test_grad_fp16_small_and_subnormal_values():
    # values below fp16's normal range are rounded to its subnormals, as the oracle's are
    x = torch.randn(33, 64, generator=torch.Generator().manual_seed(2)).cuda() * torch.exp2(
        torch.arange(33, device="cuda") - 34.0)[:, None]
    it = dict(dY=torch.ones(33, 8, dtype=torch.float16, device="cuda"), G=torch.empty(8, 64, device="cuda"), beta=0.0,
              **_ckpt_of(x))
    it["dY"] *= torch.linspace(1, 8, 33, device="cuda").half()[:, None]
    _run_and_check([it])


def test_grad_nan_blocks_reach_only_their_columns():
    x = torch.randn(50, 96, generator=torch.Generator().manual_seed(2)).cuda()
    x[17, 40] = float("inf")
    for dt in DTS:
        it = dict(dY=torch.randn(50, 70, generator=torch.Generator().manual_seed(3)).to(dt).cuda(),
                  G=torch.empty(70, 96, device="cuda"), **_ckpt_of(x))
        mo.act8_grad_batched([it], _ws([it]))
        nan = torch.isnan(it["G"])
        assert bool(nan[:, 32:64].all()) and not bool(nan[:, :32].any()) and not bool(nan[:, 64:].any())


def test_grad_infinite_dY_reaches_only_its_rows():
    it, _ = _case(50, 70, 96, torch.bfloat16, torch.float32, seed=10)
    it["dY"][3, 5] = float("nan")
    mo.act8_grad_batched([it], _ws([it]))
    nan = torch.isnan(it["G"])
    assert bool(nan[5].all()) and int(nan.sum()) == 96


def test_grad_workspace_is_required():
    it, _ = _case(20000, 64, 64, torch.bfloat16, torch.float32, seed=9, pad=1)
    need = mo.act8_grad_workspace_size([it])
    if need:
        for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
                   torch.empty(need + 256, dtype=torch.uint8, device="cuda")[1:]):
            with pytest.raises(mo.MuonError) as err:
                mo.act8_grad_batched([it], ws)
            assert err.value.status == mo.ERR_WORKSPACE


def test_other_stream_and_captured_graph():
    # encode and gradient captured once and replayed on new inputs, on a stream of its own
    x = _x(700, 264, torch.bfloat16, seed=1, spread=0.3)
    it, _ = _case(700, 200, 264, torch.bfloat16, torch.float32, seed=11)
    ws = _ws([it])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mo.act8_encode_batched([dict(x=x, q=it["q"], e=it["e"])])
        mo.act8_grad_batched([it], ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mo.act8_encode_batched([dict(x=x, q=it["q"], e=it["e"])])
        mo.act8_grad_batched([it], ws)
    for seed in (20, 21):
        x.copy_(_x(700, 264, torch.bfloat16, seed=seed, spread=0.3))
        it["dY"].mul_(-0.5)
        g.replay()
        torch.cuda.synchronize()
        q_ref, e_ref = acts.encode(_np(x))
        assert np.array_equal(it["q"].cpu().numpy(), q_ref)
        _check_G(it["G"], it["dY"], acts.decode(q_ref, e_ref))


@pytest.mark.parametrize("C", [40, 41, 256])
def test_fp16_values_at_the_end_of_the_range_stay_finite(C):
    # fp16 values from 65024 on are held as 64 2^10 = 65536 (half a step: 512), which fp16 does not have; it takes 65504 for it
    top = torch.tensor([65504.0, -65504.0, 65056.0, 65024.0, -65024.0, 64992.0, 32768.0, 1.0], dtype=torch.float16)
    x = torch.zeros(9, C, dtype=torch.float16)
    x[:, :8] = top.roll(1)
    x[1, :8] = top
    x[4, C - 1] = 65504.0
    x = x.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = mo.act8_empty(9, C)
    mo.act8_encode_batched([dict(x=x, **c)], d_status=status)
    q_ref, e_ref = acts.encode(_np(x))
    assert int(status.item()) == 0 and int(q_ref.max()) == 64
    assert np.array_equal(c["q"].cpu().numpy(), q_ref) and np.array_equal(c["e"].cpu().numpy(), e_ref)
    out = torch.empty_like(x)
    mo.act8_decode_batched([dict(x=out, **c)])
    assert float((out.double() - x.double()).abs().max()) <= 512         # also: no infinity and no NaN
    X = acts.decode(q_ref, e_ref)
    X = np.where(np.abs(X) == 65536, np.copysign(65504.0, X), X)
    for wt in (torch.float32, torch.float16):
        dY = (torch.randn(9, 72, generator=torch.Generator().manual_seed(C)) * 1e-2).half().cuda()
        G = torch.empty(72, C, dtype=wt, device="cuda")
        items = [dict(dY=dY, G=G, **c)]
        mo.act8_grad_batched(items, _ws(items))
        _check_G(G, dY, X)


def test_fp16_takes_larger_values_as_infinite():
    # a checkpoint of another type: 2^16 is 65504 in fp16, the next values up are beyond it
    x = torch.tensor([[65536.0, -65536.0, 66560.0, 131072.0, -131072.0, 3e38, 1.0, 0.0] + [0.0] * 8 for _ in range(2)])
    x[1, 5] = float("nan")                                              # a bad block
    for C in (16, 15):                                                  # vector and single accesses
        v = x[:, :C].contiguous().cuda()
        c = mo.act8_empty(2, C)
        v[0, 5] = 0.0
        mo.act8_encode_batched([dict(x=v, **c)])
        out = torch.empty(2, C, dtype=torch.float16, device="cuda")
        mo.act8_decode_batched([dict(x=out, **c)])
        inf = float("inf")
        assert out[0, :5].tolist() == [65504.0, -65504.0, 65504.0, inf, -inf]
        assert bool(torch.isnan(out[1]).all())


def test_grad_fp32_dY_of_every_magnitude():
    # the three parts of an fp32 dY sum to it up to its largest value (3.396e38 and more round to infinity in
    # bfloat16), and down to 2^-133, bfloat16's smallest step: what lies below is lost, half a step an element
    g = torch.Generator().manual_seed(12)
    big = torch.tensor([3.4028234e38, -3.4028234e38, 3.4e38, 3.396e38, -3.39e38, 3.2e38, 3.0123456e38, -1.2345678e38])
    x = _x(24, 72, torch.float32, seed=12, spread=0.0) * 2.0 ** -8
    c = _ckpt_of(x)
    X = acts.decode(c["q"].cpu().numpy(), c["e"].cpu().numpy())
    dY = big[torch.randint(0, 8, (24, 40), generator=g)] * (torch.rand(24, 40, generator=g) < 0.2)
    G = torch.empty(40, 72, device="cuda")
    items = [dict(dY=dY.cuda(), G=G, **c)]
    mo.act8_grad_batched(items, _ws(items))
    _check_G(G, items[0]["dY"], X)

    dY = torch.randn(24, 40, generator=g) * torch.exp2(torch.randint(-135, -90, (24, 40), generator=g).float())
    c = _ckpt_of(x * 2.0 ** 100)
    X = acts.decode(c["q"].cpu().numpy(), c["e"].cpu().numpy())
    items = [dict(dY=dY.cuda(), G=G, **c)]
    mo.act8_grad_batched(items, _ws(items))
    d = dY.double().numpy()
    S = np.abs(d).T @ np.abs(X)
    lost = 2.0 ** -134 * np.abs(X).sum(axis=0)[None, :]
    assert np.all(np.abs(_np(G) - d.T @ X) <= lost + (3 * 24 + 4) * 2.0 ** -23 * (S + lost) + 2.0 ** -149)


def test_descriptors_keep_their_tensors_device():
    it, _ = _case(5, 24, 40, torch.bfloat16, torch.float32)
    x = torch.zeros(5, 40, dtype=torch.bfloat16, device="cuda")
    seam = dict(pre="rms", x=x, y=torch.empty_like(x))
    back = dict(dx=torch.empty_like(x), dout=x)
    made = [(mo.make_act8_grads([it]), lambda d: mo.act8_grad_batched(d, _ws(d))),
            (mo.make_act8_items([dict(x=x, q=it["q"], e=it["e"])]), mo.act8_decode_batched),
            (mo.make_seam(seam), mo.seam_forward), (mo.make_seam_grad(back), mo.seam_backward)]
    for d, call in made:
        assert d.device == torch.cuda.current_device()
        call(d)
        d.device += 1
        with pytest.raises(ValueError, match="current one"):
            call(d)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,O,C,wt", [(700, 9216, 2304, torch.bfloat16), (6300, 4608, 2304, torch.float32),
                                      (1900, 1536, 1024, torch.float32), (130, 9000, 2296, torch.float16)])
def test_grad_many_tiles_per_pair_of_SMs_give_equal_bits(T, O, C, wt):
    # several tiles and segments one after another through the same stages and accumulators, tall tiles and low ones: every
    # run gives the first one's bits, and that is the product.  The sum's error as in the tests above: up to 4 T / 64 steps of
    # 2^-24 2/3 of the result on average (segments hold fewer), and a rounding to G's type.
    g = torch.Generator(device="cuda").manual_seed(T)
    dt = torch.float16 if wt == torch.float16 else torch.bfloat16
    c = _ckpt_of(torch.randn(T, C, generator=g, device="cuda"))
    dY = (torch.randn(T, O, generator=g, device="cuda") * 0.1).to(dt)
    G = torch.empty(O, C, dtype=wt, device="cuda")
    items = mo.make_act8_grads([dict(dY=dY, G=G, **c)])
    ws = _ws(items)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mo.act8_grad_batched(items, ws, d_status=status)
    first = G.clone()
    X = torch.empty(T, C, device="cuda")
    mo.act8_decode_batched([dict(x=X, **c)])
    ref = dY.double().T @ X.double()
    tol = min(4 * -(-T // 64), 384) * 2.0 ** -24 * 2 / 3 + torch.finfo(wt).eps / 2
    assert float((first.double() - ref).norm() / ref.norm()) <= tol
    for _ in range(20):
        G.fill_(GUARD)
        mo.act8_grad_batched(items, ws, d_status=status)
        assert torch.equal(G, first)
    assert int(status.item()) == 0


def test_grad_added_to_subnormal_G():
    # beta = 1 on an fp32 G of whole tiles: additions in memory, where what lies below 2^-126 counts as zero; each of the
    # sum's parts (G, the product) may lose that much, the sum is rounded once.
    T, O, C = 64, 4608, 2304
    g = torch.Generator(device="cuda").manual_seed(6)
    c = _ckpt_of(torch.randint(-2, 3, (T, C), generator=g, device="cuda").float() * 2.0 ** -100)
    dY = (torch.randint(-2, 3, (T, O), generator=g, device="cuda").float() * 2.0 ** -20).to(torch.bfloat16)
    G0 = torch.randn(O, C, generator=g, device="cuda") * torch.exp2(torch.randint(-140, -110, (O, C), generator=g, device="cuda").float())
    G = G0.clone()
    items = [dict(dY=dY, G=G, beta=1.0, **c)]
    mo.act8_grad_batched(items, _ws(items))
    X = torch.empty(T, C, device="cuda")
    mo.act8_decode_batched([dict(x=X, **c)])
    ref = dY.double().T @ X.double() + G0.double()
    assert bool(((G.double() - ref).abs() <= 2 * 2.0 ** -126 + 2.0 ** -24 * ref.abs()).all())


def _norm_error(it):
    """|G - the product in 64 bits| / |the product|, Frobenius."""
    X = torch.empty(it["dY"].shape[0], it["G"].shape[1], device="cuda")
    mo.act8_decode_batched([dict(x=X, q=it["q"], e=it["e"])])
    ref = it["dY"].double().T @ X.double()
    return float((it["G"].double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("T", [16381, 4999, 333])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_grad_long_sums_over_few_tiles(T, dt):
    # Nine tiles or fewer, so their tokens are split into ranges, the last k-block partly filled.  On average a step of 16 tokens
    # costs at most 2^-24 of the running sum, which grows like a random walk (2/3 of the result): with at most 96 x 4
    # steps in a range 1.6e-5, and 2^-24 for each of up to 74 ranges added.
    it, buf = _case(T, 768, 768, dt, torch.float32, seed=T)
    mo.act8_grad_batched([it], _ws([it]))
    assert _norm_error(it) <= 1.6e-5 + 74 * 2.0 ** -24
    assert bool((buf[768 * 768:] == GUARD).all())


@pytest.mark.parametrize("T", [16381, 20001, 6209])
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("O,C", [(96, 64), (768, 520)])
def test_grad_sees_every_token_of_a_long_sum(T, dt, O, C):
    # One token at a time: first, last, around the ends of k-blocks and ranges.  dY of the rest is zero, so the gradient is this
    # token's outer product, exactly (at most 14 significant bits, added to zeros).
    x = torch.randn(T, C, generator=torch.Generator().manual_seed(T)).cuda()
    c = _ckpt_of(x)
    X = torch.empty(T, C, device="cuda")
    mo.act8_decode_batched([dict(x=X, **c)])
    dY, G = torch.zeros(T, O, dtype=dt, device="cuda"), torch.empty(O, C, device="cuda")
    items = [dict(dY=dY, G=G, **c)]
    ws = _ws(items)
    d = (1 + torch.arange(O, device="cuda") % 7).to(dt)
    tokens = {0, 1, 63, 64, T // 2, 6143, 6144, T - 65, T - 64, T - 2, T - 1} | set(range(1023, T, 1024))
    for t in sorted(t for t in tokens if t < T):
        dY[t] = d
        mo.act8_grad_batched(items, ws)
        values = X[t].half().double() if dt == torch.float16 else X[t].double()
        assert torch.equal(G.double(), d.double()[:, None] * values[None, :]), t
        dY[t] = 0


@pytest.mark.parametrize("dt,wt,T", [(torch.float32, torch.bfloat16, 22001), (torch.float32, torch.float16, 22001),
                                     (torch.bfloat16, torch.bfloat16, 65601), (torch.float16, torch.float16, 65601)])
def test_grad_16_bit_G_beyond_one_segment(dt, wt, T):
    # More than 1024 k-blocks (over the parts of an fp32 dY): a 16-bit G goes through ranges of at most as many.  Truncation as
    # above over at most 4096 steps, a third of them in an fp32 dY's hi part, and the rounding to G's type.
    for O, C in ((72, 136), (40, 77)):
        it, buf = _case(T, O, C, dt, wt, seed=O, gain=False)
        mo.act8_grad_batched([it], _ws([it]))
        assert _norm_error(it) <= 4096 * 2.0 ** -24 * 2 / 3 + torch.finfo(wt).eps / 2
        assert bool((buf[O * C:] == GUARD).all())
        it["dY"].zero_()
        it["dY"][T - 1] = 1.0                      # the last token alone
        mo.act8_grad_batched([it], _ws([it]))
        X = torch.empty(T, C, device="cuda")
        mo.act8_decode_batched([dict(x=X, q=it["q"], e=it["e"])])
        last = (X[T - 1].half() if dt == torch.float16 else X[T - 1]).to(wt)
        assert torch.equal(it["G"], last[None, :].expand(O, C))


def test_gradients_of_two_threads_on_two_streams():
    # calls that overlap on the GPU, each with a workspace of its own: tall tiles, low ones, ranges of tokens, an fp32 dY
    jobs = []
    for T, O, C, dt, wt in ((900, 4608, 2304, torch.bfloat16, torch.bfloat16), (5000, 520, 264, torch.float32, torch.float32)):
        it, _ = _case(T, O, C, dt, wt, seed=O)
        arr, ws = mo.make_act8_grads([it]), _ws([it])
        mo.act8_grad_batched(arr, ws)
        x = torch.empty(T, C, dtype=dt, device="cuda")
        jobs.append((arr, ws, mo.make_act8_items([dict(x=x, q=it["q"], e=it["e"])]), it, it["G"].clone(), x))
    torch.cuda.synchronize()
    errors, start, status = [], threading.Barrier(2), torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(arr, ws, items):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(200):
                mo.act8_decode_batched(items, stream=stream)
                mo.act8_grad_batched(arr, ws, d_status=status, stream=stream)
        except Exception as e:          # noqa: BLE001 - reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=job[:3]) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and int(status.item()) == 0
    for _, _, _, it, first, x in jobs:
        assert torch.equal(it["G"], first)
        X = torch.from_numpy(acts.decode(it["q"].cpu().numpy(), it["e"].cpu().numpy()))
        assert torch.equal(x.cpu(), X.to(x.dtype))
