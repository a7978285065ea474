"""Host-side checks of the checkpoint, gradient and seam entry points (CPU): the
descriptors' layout against the header, refusals before any launch (the pointers below
are never read), workspace queries, and the binding's own checks."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import muon_family_optimizer_b200 as mo
from muon_family_optimizer_b200 import build as mbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an address that is never read


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return mo.lib()


STRUCTS = {"muon_act8": mo.Act8, "muon_act8_item": mo.Act8Item, "muon_act8_grad_item": mo.Act8GradItem,
           "muon_seam": mo.Seam, "muon_seam_grad": mo.SeamGrad}


def test_struct_layouts_match_header(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines.append('printf("MUON_SEAM_MAX_COLS %d\\n", MUON_SEAM_MAX_COLS);')
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){%s return 0;}' % "\n".join(lines))
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    got = dict(line.rsplit(" ", 1) for line in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got.pop("MUON_SEAM_MAX_COLS")) == mo.SEAM_MAX_COLS
    for key, val in got.items():
        if "." in key:
            name, field = key.split(".")
            assert getattr(STRUCTS[name], field).offset == int(val), key
        else:
            assert ctypes.sizeof(STRUCTS[key]) == int(val), key


@pytest.mark.parametrize("pack,cls", [(mo._PACK_ITEM, mo.Act8Item), (mo._PACK_GRAD, mo.Act8GradItem),
                                      (mo._PACK_SEAM, mo.Seam), (mo._PACK_SEAM_GRAD, mo.SeamGrad)])
def test_packed_descriptors_match_the_structures(pack, cls):
    # distinct values through the binding's one-call layouts come back out of the right fields
    flat = []

    def fields(c, prefix=""):
        for n, t in c._fields_:
            if t is mo.Act8:
                yield from fields(t, prefix + n + ".")
            else:
                yield prefix + n, t
    names = list(fields(cls))
    flat = [float(i) + 0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(names)]
    obj = cls()
    pack.pack_into(obj, 0, *flat)
    assert ctypes.sizeof(cls) - pack.size < 8
    for (name, _), want in zip(names, flat):
        got = obj
        for part in name.split("."):
            got = getattr(got, part)
        assert got == want, name


def _ckpt(**kw):
    d = dict(rows=4, cols=40, q=P, ldq=48, e=P, lde=2)
    d.update(kw)
    return mo.Act8(*[d[k] for k in ("rows", "cols", "q", "ldq", "e", "lde")])


BAD_CKPT = [dict(rows=-1), dict(cols=0), dict(q=None), dict(e=None), dict(q=P + 8), dict(ldq=40), dict(ldq=32),
            dict(lde=1)]


@pytest.mark.parametrize("bad", BAD_CKPT + [dict(x=None), dict(ldx=39), dict(n=0), dict(dt=3), dict(dt=-1)])
@pytest.mark.parametrize("fn", ["act8_encode_batched", "act8_decode_batched"])
def test_encode_decode_refusals(L, fn, bad):
    bad = dict(bad)
    n, dt = bad.pop("n", 1), bad.pop("dt", mo.BF16)
    x, ldx = bad.pop("x", P), bad.pop("ldx", 40)
    arr = (mo.Act8Item * 1)(mo.Act8Item(_ckpt(**bad), x, ldx))
    args = (arr, n, dt) + ((None,) if fn == "act8_encode_batched" else ()) + (None,)
    assert getattr(L, fn)(*args) == mo.ERR_INVALID_ARG
    if not bad:
        args = (None,) + args[1:]
        assert getattr(L, fn)(*args) == mo.ERR_INVALID_ARG


def _grad(**kw):
    c = _ckpt(**{k: kw.pop(k) for k in list(kw) if k in ("rows", "cols", "q", "ldq", "e", "lde")})
    d = dict(dY=P, lddy=24, out=24, G=P, gain=None, shift=None, dy_sum=None, beta=0.0)
    d.update(kw)
    return mo.Act8GradItem(c, *[d[k] for k in ("dY", "lddy", "out", "G", "gain", "shift", "dy_sum", "beta")])


@pytest.mark.parametrize("bad", BAD_CKPT + [dict(dY=None), dict(lddy=23), dict(out=0), dict(G=None), dict(shift=P),
                                            dict(dy_sum=P), dict(beta=math.nan), dict(beta=math.inf)])
def test_grad_refusals(L, bad):
    arr = (mo.Act8GradItem * 2)(_grad(), _grad(**bad))
    out = ctypes.c_size_t(7)
    assert L.act8_grad_workspace_size(arr, 2, mo.BF16, mo.BF16, ctypes.byref(out)) == mo.ERR_INVALID_ARG
    assert L.act8_grad_batched(arr, 2, mo.BF16, mo.BF16, P, 1 << 40, None, None) == mo.ERR_INVALID_ARG


@pytest.mark.parametrize("n", [2, 64, 65, 300])
def test_grad_refuses_gradients_that_overlap(L, n):
    # G of 24 x 40 bfloat16: 1920 bytes
    def call(ats):
        arr = (mo.Act8GradItem * n)(*[_grad(G=at) for at in ats])
        return L.act8_grad_batched(arr, n, mo.BF16, mo.BF16, None, 0, None, None)
    apart = [P + 1920 * ((7 * i) % n if n % 7 else i) for i in range(n)]
    assert len(set(apart)) == n and call(apart) != mo.ERR_INVALID_ARG          # no workspace, or no device
    for at in (apart[0], apart[0] + 1904, apart[0] + 16):
        assert call(apart[:-1] + [at]) == mo.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(rows=(1 << 30) + 1), dict(cols=(1 << 30) + 16, ldq=1 << 31, lde=1 << 26),
                                 dict(out=(1 << 30) + 1, lddy=1 << 31)])
def test_dimensions_beyond_the_limit_are_refused(L, bad):
    out = ctypes.c_size_t(0)
    arr = (mo.Act8GradItem * 1)(_grad(**bad))
    assert L.act8_grad_workspace_size(arr, 1, mo.BF16, mo.BF16, ctypes.byref(out)) == mo.ERR_INVALID_ARG
    if "out" not in bad:
        item = (mo.Act8Item * 1)(mo.Act8Item(_ckpt(**bad), P, 1 << 31))
        assert L.act8_encode_batched(item, 1, mo.BF16, None, None) == mo.ERR_INVALID_ARG
    if "rows" in bad:
        seam = _seam(rows=bad["rows"], post_c=mo.Act8(), pre_c=mo.Act8())
        assert L.seam_forward(ctypes.byref(seam), mo.BF16, mo.BF16, None, None) == mo.ERR_INVALID_ARG
        assert L.seam_backward_workspace_size(ctypes.byref(_back(rows=bad["rows"])), ctypes.byref(out)) == mo.ERR_INVALID_ARG


def test_grad_refusals_of_the_call(L):
    arr = (mo.Act8GradItem * 1)(_grad())
    out = ctypes.c_size_t(0)
    assert L.act8_grad_workspace_size(arr, 1, 3, mo.BF16, ctypes.byref(out)) == mo.ERR_INVALID_ARG
    assert L.act8_grad_workspace_size(arr, 1, mo.BF16, 3, ctypes.byref(out)) == mo.ERR_INVALID_ARG
    assert L.act8_grad_workspace_size(arr, 1, mo.BF16, mo.BF16, None) == mo.ERR_INVALID_ARG
    assert L.act8_grad_workspace_size(arr, 0, mo.BF16, mo.BF16, ctypes.byref(out)) == mo.ERR_INVALID_ARG
    assert L.act8_grad_workspace_size(None, 1, mo.BF16, mo.BF16, ctypes.byref(out)) == mo.ERR_INVALID_ARG
    assert L.act8_grad_batched(arr, 1, 3, mo.BF16, None, 0, None, None) == mo.ERR_INVALID_ARG
    assert L.act8_grad_batched(arr, 1, mo.BF16, 5, None, 0, None, None) == mo.ERR_INVALID_ARG


def _seam(**kw):
    d = dict(rows=4, cols=40, post=1, pre=1, eps=1e-5, skip=1.0, scale=1.0, x=P, ldx=40, f=P, ldf=40, gate=P, ldgate=40,
             gate_rows=3, post_gain=P, post_bias=None, pre_gain=P, pre_bias=None, out=P, ldout=40, y=P, ldy=40,
             post_c=_ckpt(), pre_c=_ckpt(), post_rstd=P, pre_rstd=P)
    d.update(kw)
    return mo.Seam(*[d[f] for f, _ in mo.Seam._fields_])


NOTHING = mo.Act8(0, 0, None, 0, None, 0)
BAD_SEAM = [dict(rows=-1), dict(cols=0), dict(post=3), dict(pre=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan),
            dict(eps=math.inf), dict(skip=math.inf), dict(scale=math.nan), dict(x=None), dict(ldx=39), dict(ldf=39),
            dict(out=None), dict(ldout=39), dict(y=None), dict(ldy=39), dict(ldgate=39), dict(gate_rows=0),
            dict(f=None), dict(pre=0), dict(post_c=_ckpt(rows=3)), dict(pre_c=_ckpt(cols=41)),
            dict(pre_c=_ckpt(ldq=40)), dict(f=None, post=0, gate=None, post_gain=None, post_c=NOTHING, post_rstd=None)]


@pytest.mark.parametrize("bad", BAD_SEAM)
def test_seam_refusals(L, bad):
    assert L.seam_forward(ctypes.byref(_seam(**bad)), mo.BF16, mo.BF16, None, None) == mo.ERR_INVALID_ARG


def test_seam_refusals_of_the_call(L):
    s = _seam()
    assert L.seam_forward(None, mo.BF16, mo.BF16, None, None) == mo.ERR_INVALID_ARG
    assert L.seam_forward(ctypes.byref(s), 3, mo.BF16, None, None) == mo.ERR_INVALID_ARG
    assert L.seam_forward(ctypes.byref(s), mo.BF16, -1, None, None) == mo.ERR_INVALID_ARG
    wide = dict(cols=16385, ldx=16385, ldf=16385, ldgate=16385, ldout=16385, ldy=16385, post_c=NOTHING, pre_c=NOTHING)
    assert L.seam_forward(ctypes.byref(_seam(**wide)), mo.BF16, mo.BF16, None, None) == mo.ERR_UNSUPPORTED
    # a residual sum without f, and no output at all
    lone = dict(f=None, post=0, gate=None, post_gain=None, post_c=NOTHING, post_rstd=None, out=None)
    assert L.seam_forward(ctypes.byref(_seam(**lone, skip=0.5)), mo.BF16, mo.BF16, None, None) == mo.ERR_INVALID_ARG
    none = dict(lone, pre=0, y=None, pre_gain=None, pre_c=NOTHING, pre_rstd=None)
    assert L.seam_forward(ctypes.byref(_seam(**none)), mo.BF16, mo.BF16, None, None) == mo.ERR_INVALID_ARG


def _back(**kw):
    d = dict(rows=4, cols=40, post=1, pre=1, skip=1.0, scale=1.0, gate=P, ldgate=40, gate_rows=3, post_gain=P,
             post_bias=None, pre_gain=P, post_c=_ckpt(), pre_c=_ckpt(), post_rstd=P, pre_rstd=P, dy=P, lddy=40, dout=P,
             lddout=40, dx=P, lddx=40, df=2 * P, lddf=40, dgate=P, lddgate=40, d_post_gain=P, d_post_bias=None,
             d_pre_gain=P, d_pre_bias=None, beta=0.0)
    d.update(kw)
    return mo.SeamGrad(*[d[f] for f, _ in mo.SeamGrad._fields_])


BAD_BACK = [dict(rows=-1), dict(cols=0), dict(post=3), dict(pre=7), dict(skip=math.nan), dict(scale=math.inf),
            dict(beta=math.nan), dict(gate_rows=0), dict(ldgate=39), dict(lddgate=39), dict(gate=None), dict(dy=None),
            dict(lddy=39), dict(lddout=39), dict(dx=None), dict(lddx=39), dict(lddf=39), dict(df=P), dict(df=None),
            dict(post_c=NOTHING), dict(pre_c=NOTHING), dict(post_rstd=None), dict(pre_rstd=None),
            dict(post_c=_ckpt(rows=5)), dict(pre_c=_ckpt(q=P + 1)), dict(pre=0), dict(pre=0, dy=None),
            dict(post=0, post_c=NOTHING)]


@pytest.mark.parametrize("bad", BAD_BACK)
def test_seam_backward_refusals(L, bad):
    s, out = _back(**bad), ctypes.c_size_t(0)
    assert L.seam_backward_workspace_size(ctypes.byref(s), ctypes.byref(out)) == mo.ERR_INVALID_ARG
    assert L.seam_backward(ctypes.byref(s), mo.BF16, mo.BF16, P, 1 << 40, None, None) == mo.ERR_INVALID_ARG


def test_seam_backward_workspace(L):
    s, out = _back(), ctypes.c_size_t(0)
    assert L.seam_backward_workspace_size(ctypes.byref(s), ctypes.byref(out)) == mo.OK and out.value > 0
    need = out.value
    for ws, size in ((None, need), (P, need - 1), (P + 128, need)):
        assert L.seam_backward(ctypes.byref(s), mo.BF16, mo.BF16, ws, size, None, None) == mo.ERR_WORKSPACE
    assert L.seam_backward_workspace_size(ctypes.byref(s), None) == mo.ERR_INVALID_ARG
    # nothing to sum over tokens: no workspace
    s = _back(d_post_gain=None, d_pre_gain=None, gate_rows=1)
    assert L.seam_backward_workspace_size(ctypes.byref(s), ctypes.byref(out)) == mo.OK and out.value == 0
    wide = _back(cols=20000, ldgate=20000, lddy=20000, lddout=20000, lddx=20000, lddf=20000, lddgate=20000,
                 post_c=_ckpt(cols=20000, ldq=20000, lde=625), pre_c=_ckpt(cols=20000, ldq=20000, lde=625))
    assert L.seam_backward_workspace_size(ctypes.byref(wide), ctypes.byref(out)) == mo.ERR_UNSUPPORTED


def test_act8_empty_rows_are_aligned():
    c = mo.act8_empty(5, 70, device="cpu")
    assert c["q"].shape == (5, 70) and c["q"].stride(0) == 80 and c["e"].shape == (5, 3)
    assert c["q"].dtype == torch.int8 and c["e"].dtype == torch.uint8
    assert mo.act8_empty(0, 70, device="cpu")["q"].shape == (0, 70)


def test_binding_refuses_host_workspaces_and_status_words(L):
    ws, status = torch.empty(1 << 20, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    grads = (mo.Act8GradItem * 1)(_grad())
    grads.dy_dtype = grads.w_dtype = mo.BF16
    items = (mo.Act8Item * 1)(mo.Act8Item(_ckpt(), P, 40))
    items.x_dtype = mo.BF16
    seam, back = _seam(), _back()
    for d in (seam, back):
        d.x_dtype = d.w_dtype = mo.BF16
    for call in (lambda: mo.act8_grad_batched(grads, ws), lambda: mo.act8_grad_batched(grads, None, status),
                 lambda: mo.act8_encode_batched(items, status), lambda: mo.seam_forward(seam, status),
                 lambda: mo.seam_backward(back, ws), lambda: mo.seam_backward(back, None, status)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_binding_refuses_other_devices_and_shapes():
    # host tensors never reach the library
    c = mo.act8_empty(4, 40, device="cpu")
    x = torch.zeros(4, 40)
    for call in (lambda: mo.act8_encode_batched([dict(x=x, **c)]), lambda: mo.act8_decode_batched([dict(x=x, **c)]),
                 lambda: mo.act8_grad_batched([dict(dY=torch.zeros(4, 8), G=torch.zeros(8, 40), **c)]),
                 lambda: mo.seam_forward(dict(x=x, y=x, pre="rms")),
                 lambda: mo.seam_backward(dict(dx=x, dout=x))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        mo.seam_forward(dict(x=x, y=x, pre="batch"))
    with pytest.raises(ValueError):
        mo.seam_forward(dict(x=x[0], y=x, pre="rms"))


@pytest.mark.parametrize("make,lead", [(mo.make_seam, "x"), (mo.make_seam_grad, "dx")])
def test_binding_refuses_gate_rows_below_one(make, lead):
    t = torch.zeros(4, 40)
    for gr in (0, -1):
        with pytest.raises(ValueError, match="gate_rows"):
            make({lead: t, "gate": t, "gate_rows": gr})
    with pytest.raises(ValueError, match="gate_rows"):
        make({lead: t, "gate_rows": -1})
    # without a gate 0 is what there is; the next check refuses the host tensor
    for more in (dict(gate_rows=0), dict(gate_rows=0, gate=None), dict(gate=t), dict(gate=t, gate_rows=None),
                 dict(gate=t, gate_rows=4)):
        with pytest.raises(ValueError, match="current CUDA device"):
            make({lead: t, **more})


@pytest.mark.parametrize("make,lead", [(mo.make_seam, "x"), (mo.make_seam_grad, "dx")])
def test_binding_refuses_unknown_norms_and_other_ranks(make, lead):
    t = torch.zeros(4, 40)
    for side in ("post", "pre"):
        for kind in ("batch", None, 1):
            with pytest.raises(ValueError, match=f"{side}: must be one of"):
                make({lead: t, side: kind})
    for bad in (t[0], t[None]):
        with pytest.raises(ValueError, match="2-D"):
            make({lead: bad, "pre": "rms"})
    for kind in mo.NORMS:           # the known kinds come as far as the host tensor's own refusal
        with pytest.raises(ValueError, match="current CUDA device"):
            make({lead: t, "post": kind, "pre": kind})


def test_binding_refuses_descriptors_of_another_device(monkeypatch):
    # the tensors' device is kept when a descriptor is made; a call launches on the current one
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mo, "lib", lambda: pytest.fail("reached the library"))
    grads, items, seam, back = (mo.Act8GradItem * 1)(_grad()), (mo.Act8Item * 1)(mo.Act8Item(_ckpt(), P, 40)), _seam(), _back()
    for d in (grads, items, seam, back):
        d.x_dtype = d.dy_dtype = d.w_dtype = mo.BF16
        d.device = 1
    for call in (lambda: mo.act8_encode_batched(items), lambda: mo.act8_decode_batched(items),
                 lambda: mo.act8_grad_batched(grads), lambda: mo.seam_forward(seam), lambda: mo.seam_backward(back)):
        with pytest.raises(ValueError, match="made for CUDA device 1, the current one is 0"):
            call()


def test_arrivals_on_another_cta_release_at_cluster_scope():
    # An arrival on an mbarrier of another CTA has to name cluster scope: without a scope it releases to its own CTA only.
    # tcgen05 commits and the completions of copies, the other signals between CTAs, have that scope by definition.
    src = os.path.join(ROOT, "muon_family_optimizer_b200", "csrc")
    found = 0
    for name in sorted(os.listdir(src)):
        with open(os.path.join(src, name)) as fh:
            for line in fh:
                if "mbarrier.arrive" in line and "shared::cluster" in line and "asm" in line and "tcgen05" not in line:
                    found += 1
                    assert ".release.cluster." in line, (name, line)
    assert found


def test_seam_refuses_a_deviation_without_its_norm(L):
    # it would be left unwritten
    bare = dict(post=0, post_gain=None)
    assert L.seam_forward(ctypes.byref(_seam(**bare)), mo.BF16, mo.BF16, None, None) == mo.ERR_INVALID_ARG
    assert L.seam_forward(ctypes.byref(_seam(**bare, rows=0)), mo.BF16, mo.BF16, None, None) != mo.ERR_INVALID_ARG
    ok = _seam(**bare, post_rstd=None)
    if not torch.cuda.is_available():           # the addresses are never read: there is no device
        assert L.seam_forward(ctypes.byref(ok), mo.BF16, mo.BF16, None, None) not in (mo.OK, mo.ERR_INVALID_ARG)
