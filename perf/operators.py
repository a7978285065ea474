"""Measured cases of the 8-bit activation checkpoints and the block seams.

Three families of calls, all on the way from a block's activations to the gradients an optimizer step reads:

checkpoint  activations -> int8 codes with one power-of-two scale per 32 columns, and back to values;
grad        weight gradients dY^T X of linear layers whose input X is held as such a checkpoint;
seam        the joint between two blocks: x' = skip x + scale gate norm(f), y = norm(x'), the normalised rows
            kept as checkpoints (forward), and the gradients of all of it from those checkpoints (backward).

`run` computes them in elementary torch operations, or, where `own` is true, with this library's entry points;
`exact` computes them from the definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # a short sequence of the smallest model's width: launches and latency
        {"name": "checkpoint short", "op": "checkpoint", "tokens": 512, "cols": 768, "dtype": "bf16"},
        # the hidden activations of the widest feed-forward layer over one micro-batch
        {"name": "checkpoint hidden", "op": "checkpoint", "tokens": 8192, "cols": 14336, "dtype": "bf16"},
        # one token through a key projection: the gradient is an outer product, only G is written
        {"name": "grad one token", "op": "grad", "items": 1, "tokens": 1, "out": 1024, "cols": 4096, "dtype": "bf16",
         "wdtype": "bf16", "gain": True},
        # a small model's projection over a long micro-batch: few tiles, a long sum
        {"name": "grad long sum", "op": "grad", "items": 1, "tokens": 16384, "out": 768, "cols": 768, "dtype": "bf16",
         "wdtype": "fp32", "gain": True},
        # experts that hold an odd number of tokens each
        {"name": "grad experts", "op": "grad", "items": 16, "tokens": 333, "out": 2048, "cols": 768, "dtype": "fp16",
         "wdtype": "fp16", "gain": False},
        # the widest layer of the largest model
        {"name": "grad wide", "op": "grad", "items": 1, "tokens": 8192, "out": 14336, "cols": 4096, "dtype": "bf16",
         "wdtype": "bf16", "gain": True},
        # a few tokens between two blocks of the largest model: latency
        {"name": "seam few tokens", "op": "seam", "tokens": 7, "cols": 4096, "dtype": "bf16", "wdtype": "bf16",
         "post": "rms", "pre": "rms", "gate_rows": 0},
        # layer norms with biases, no norm behind the block: the smallest model's own seam
        {"name": "seam layer norm", "op": "seam", "tokens": 16384, "cols": 768, "dtype": "bf16", "wdtype": "fp32",
         "post": "none", "pre": "layer", "gate_rows": 0},
        # norms on both sides of the block, a gate row for each sequence of 2048 tokens
        {"name": "seam both norms", "op": "seam", "tokens": 16384, "cols": 4096, "dtype": "bf16", "wdtype": "bf16",
         "post": "rms", "pre": "rms", "gate_rows": 2048},
        # the same seams on the way back
        {"name": "seam back few tokens", "op": "seam_back", "tokens": 7, "cols": 4096, "dtype": "bf16",
         "wdtype": "bf16", "post": "rms", "pre": "rms", "gate_rows": 0},
        {"name": "seam back layer norm", "op": "seam_back", "tokens": 16384, "cols": 768, "dtype": "bf16",
         "wdtype": "fp32", "post": "none", "pre": "layer", "gate_rows": 0},
        # a gate value for every token and column
        {"name": "seam back both norms", "op": "seam_back", "tokens": 16384, "cols": 4096, "dtype": "bf16",
         "wdtype": "bf16", "post": "rms", "pre": "rms", "gate_rows": 1},
    ]


def _size(rng, lo, hi):
    """A size from lo to hi, spread over its logarithm; every second one as it falls, the others on a multiple of 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if rng.random() < 0.5 or n < 64 else min(hi, (n + 32) // 64 * 64)


def draw(rng):
    op = rng.choice(["checkpoint", "grad", "grad", "seam", "seam_back"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "checkpoint":
        return {"op": op, "tokens": _size(rng, 1, 16384), "cols": _size(rng, 64, 14336), "dtype": dtype}
    wdtype = rng.choice([dtype, "fp32"])
    if op == "grad":
        items = rng.choice([1, 1, 2, 3, 16])
        tokens = _size(rng, 1, 16384 if items < 16 else 1024)
        out, cols = _size(rng, 64, 14336 if items == 1 else 4096), _size(rng, 64, 4096)
        while items * tokens * out * cols > 8192 * 14336 * 4096:
            tokens //= 2
        return {"op": op, "items": items, "tokens": tokens, "out": out, "cols": cols, "dtype": dtype,
                "wdtype": wdtype, "gain": rng.random() < 0.5}
    tokens = _size(rng, 1, 16384)
    return {"op": op, "tokens": tokens, "cols": _size(rng, 64, 8192), "dtype": dtype, "wdtype": wdtype,
            "post": rng.choice(["none", "rms", "layer"]), "pre": rng.choice(["rms", "layer"]),
            "gate_rows": rng.choice([0, 1, _size(rng, 1, tokens), tokens])}


# ------------------------------------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, tokens, cols, dtype):
    """Activations of a trained layer: channels of different strength, tokens of different strength."""
    x = _randn(gen, tokens, cols)
    x *= torch.exp(0.25 * _randn(gen, 1, cols))
    x *= torch.exp(0.25 * _randn(gen, tokens, 1))
    return x.to(dtype)


def _blocks(x):
    """The columns in blocks of 32, the last one filled up with zeros."""
    pad = -x.shape[-1] % BLOCK
    return torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, BLOCK))


def _quantise(x):
    """Codes (as whole numbers in x's type) in blocks, and the exponent of each block's scale."""
    b = _blocks(x)
    mant, ex = torch.frexp(b.abs().amax(-1, keepdim=True))           # max = (2 mant) 2^(ex - 1), 1 <= 2 mant < 2
    e = (ex - 7 + (mant > 127 / 128)).clamp_min(-120)
    return torch.round(torch.ldexp(b, -e)), e


def _pack(x):
    """A checkpoint as the library stores it: codes (rows 16-byte aligned) and exponents with a bias of 127."""
    codes, e = _quantise(x.float())
    codes = codes.flatten(-2).to(torch.int8)
    width = -(-x.shape[-1] // 16) * 16
    q = torch.zeros(*x.shape[:-1], width, dtype=torch.int8, device=x.device)
    q[..., :x.shape[-1]] = codes[..., :x.shape[-1]]
    return {"q": q[..., :x.shape[-1]], "e": (e.squeeze(-1) + 127).to(torch.uint8)}


def _values(c, to=torch.float32):
    """What a checkpoint stands for."""
    scale = torch.exp2(c["e"].to(to) - 127).repeat_interleave(BLOCK, -1)
    return c["q"].to(to) * scale[..., :c["q"].shape[-1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, T, C = DTYPES[case["dtype"]], case["tokens"], case["cols"]
    s = {"case": case}
    if case["op"] == "checkpoint":
        s["x"] = _activations(gen, T, C, dt)
        return s
    wt = DTYPES[case["wdtype"]]
    if case["op"] == "grad":
        n, O = case["items"], case["out"]
        x = _activations(gen, n * T, C, torch.float32)
        s["c"] = {k: v.unflatten(0, (n, T)) for k, v in _pack(x).items()}
        s["dY"] = (_randn(gen, n, T, O) * 1e-2 * torch.exp(0.5 * _randn(gen, n, T, 1))).to(dt)
        s["gain"] = (1 + 0.1 * _randn(gen, C)).to(wt) if case["gain"] else None
        return s
    for side in ("post", "pre"):
        kind = case[side]
        s[side + "_gain"] = (1 + 0.1 * _randn(gen, C)).to(wt) if kind != "none" else None
        s[side + "_bias"] = (0.1 * _randn(gen, C)).to(wt) if kind == "layer" else None
    gr = case["gate_rows"]
    s["gate"] = (1 + 0.3 * _randn(gen, -(-T // gr), C)).to(dt) if gr else None
    s["skip"], s["scale"] = 1.0, 0.5
    if case["op"] == "seam":
        s["x"], s["f"] = _activations(gen, T, C, dt), _activations(gen, T, C, dt)
        return s
    for side in ("post", "pre"):
        kept = case[side] != "none" or (side == "post" and gr)
        s[side + "_c"], s[side + "_rstd"] = None, None
        if kept:
            n = _activations(gen, T, C, torch.float32)
            rms = n.square().mean(-1, keepdim=True).sqrt()
            s[side + "_c"] = _pack(n / rms)
            s[side + "_rstd"] = (1 / rms.squeeze(-1)) if case[side] != "none" else None
    s["dy"], s["dout"] = (1e-2 * _randn(gen, T, C)).to(dt), (1e-2 * _randn(gen, T, C)).to(dt)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _checkpointed(n):
    """The values that a checkpoint of n stands for."""
    codes, e = _quantise(n)
    return torch.ldexp(codes, e).flatten(-2)[..., :n.shape[-1]].to(torch.bfloat16)


def _norm(x, kind):
    """(normalised rows, reciprocal deviation or None)."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r.squeeze(-1)


def _affine(n, gain, bias):
    n = n if gain is None else n * gain.float()
    return n if bias is None else n + bias.float()


def _gate(s):
    """The gate of every token, or 1."""
    g, T = s["gate"], s["case"]["tokens"]
    return 1.0 if g is None else g.float().repeat_interleave(s["case"]["gate_rows"], 0)[:T]


def _norm_back(g, n, r, kind):
    """Gradient of the rows that were normalised, from g, the gradient of the normalised rows."""
    if kind == "none":
        return g
    back = g - n * (g * n).mean(-1, keepdim=True)
    if kind == "layer":
        back = back - g.mean(-1, keepdim=True)
    return back * r[:, None]


def _gate_sums(d, gr):
    """Sums over the tokens that share a gate row."""
    pad = -d.shape[0] % gr
    return torch.nn.functional.pad(d, (0, 0, 0, pad)).unflatten(0, (-1, gr)).sum(1)


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "checkpoint":
        return {"values": _checkpointed(s["x"].float()).to(dt)}
    wt = DTYPES[case["wdtype"]]
    if case["op"] == "grad":
        G = s["dY"].float().mT @ _values(s["c"])
        return {"G": (G if s["gain"] is None else G * s["gain"].float()).to(wt)}
    if case["op"] == "seam":
        n, r = _norm(s["f"].float(), case["post"])
        u = _affine(n, s["post_gain"], s["post_bias"])
        out = (s["skip"] * s["x"].float() + s["scale"] * _gate(s) * u).to(dt)
        m, t = _norm(out.float(), case["pre"])
        y = _affine(m, s["pre_gain"], s["pre_bias"]).to(dt)
        kept = case["post"] != "none" or s["gate"] is not None
        return {"out": out, "y": y, "post": _checkpointed(n) if kept else None, "pre": _checkpointed(m),
                "post_rstd": r, "pre_rstd": t}
    m = _values(s["pre_c"])
    dy = s["dy"].float()
    g = dy if s["pre_gain"] is None else dy * s["pre_gain"].float()
    d = s["dout"].float() + _norm_back(g, m, s["pre_rstd"], case["pre"])
    n = _values(s["post_c"]) if s["post_c"] is not None else None
    du = s["scale"] * _gate(s) * d
    h = du if s["post_gain"] is None else du * s["post_gain"].float()
    res = {"dx": (s["skip"] * d).to(dt), "df": _norm_back(h, n, s["post_rstd"], case["post"]).to(dt),
           "pre_gain": (dy * m).sum(0).to(wt)}
    if s["pre_bias"] is not None:
        res["pre_bias"] = dy.sum(0).to(wt)
    if s["post_gain"] is not None:
        res["post_gain"] = (du * n).sum(0).to(wt)
    if s["post_bias"] is not None:
        res["post_bias"] = du.sum(0).to(wt)
    if s["gate"] is not None:
        u = _affine(n, s["post_gain"], s["post_bias"])
        res["gate"] = _gate_sums(s["scale"] * d * u, case["gate_rows"]).to(dt)
    return res


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    import muon_family_optimizer_b200 as mo
    case = s["case"]
    dt, T, C = DTYPES[case["dtype"]], case["tokens"], case["cols"]

    def like(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if case["op"] == "checkpoint":
        c, x = mo.act8_empty(T, C), s["x"]
        values = torch.empty_like(x)
        mo.act8_encode_batched([dict(x=x, **c)])
        mo.act8_decode_batched([dict(x=values, **c)])
        return {"values": values}
    wt = DTYPES[case["wdtype"]]
    if case["op"] == "grad":
        n, O = case["items"], case["out"]
        G, c, dY = like(n, O, C, dtype=wt), s["c"], s["dY"]
        items = [dict(dY=dY[i], q=c["q"][i], e=c["e"][i], G=G[i], gain=s["gain"]) for i in range(n)]
        if "ws" not in s:   # a program keeps its workspace from step to step
            s["ws"] = torch.empty(mo.act8_grad_workspace_size(items), dtype=torch.uint8, device="cuda")
        mo.act8_grad_batched(items, s["ws"])
        return {"G": G}
    seam = dict(post=case["post"], pre=case["pre"], eps=EPS, skip=s["skip"], scale=s["scale"], gate=s["gate"],
                gate_rows=case["gate_rows"], post_gain=s["post_gain"], post_bias=s["post_bias"],
                pre_gain=s["pre_gain"], pre_bias=s["pre_bias"])
    if case["op"] == "seam":
        res = {"out": like(T, C), "y": like(T, C), "post": None, "pre": like(T, C, dtype=torch.bfloat16),
               "post_rstd": None, "pre_rstd": like(T, dtype=torch.float32)}
        kept = {"pre": mo.act8_empty(T, C)}
        if case["post"] != "none" or s["gate"] is not None:
            kept["post"], res["post"] = mo.act8_empty(T, C), like(T, C, dtype=torch.bfloat16)
        if case["post"] != "none":
            res["post_rstd"] = like(T, dtype=torch.float32)
        mo.seam_forward(dict(seam, x=s["x"], f=s["f"], out=res["out"], y=res["y"], post_c=kept.get("post"),
                             pre_c=kept["pre"], post_rstd=res["post_rstd"], pre_rstd=res["pre_rstd"]))
        mo.act8_decode_batched([dict(x=res[k], **c) for k, c in kept.items()])
        return res
    res = {"dx": like(T, C), "df": like(T, C), "pre_gain": like(C, dtype=wt)}
    for k in ("pre_bias", "post_gain", "post_bias"):
        if s[k] is not None:
            res[k] = like(C, dtype=wt)
    if s["gate"] is not None:
        res["gate"] = torch.empty_like(s["gate"])
    back = dict(seam, dy=s["dy"], dout=s["dout"], post_c=s["post_c"], pre_c=s["pre_c"], post_rstd=s["post_rstd"],
                pre_rstd=s["pre_rstd"], dx=res["dx"], df=res["df"], dgate=res.get("gate"),
                d_post_gain=res.get("post_gain"), d_post_bias=res.get("post_bias"), d_pre_gain=res["pre_gain"],
                d_pre_bias=res.get("pre_bias"))
    if "ws" not in s:
        s["ws"] = torch.empty(mo.seam_backward_workspace_size(back), dtype=torch.uint8, device="cuda")
    mo.seam_backward(back, s["ws"])
    return res


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ bytes and operations
def work(case):
    T, C, b = case["tokens"], case["cols"], BYTES[case["dtype"]]
    ckpt = T * C + T * -(-C // BLOCK)
    if case["op"] == "checkpoint":      # x read, codes written, values written
        return {"bytes": 2 * T * C * b + ckpt, "flops": 0}
    w = BYTES[case["wdtype"]]
    if case["op"] == "grad":
        n, O = case["items"], case["out"]
        return {"bytes": n * (T * O * b + ckpt + O * C * w), "flops": 2 * n * T * O * C}
    gr = case["gate_rows"]
    gate = -(-T // gr) * C * b if gr else 0
    vectors = sum({"none": 0, "rms": 1, "layer": 2}[case[k]] * C * w for k in ("post", "pre"))
    norms = sum(case[k] != "none" for k in ("post", "pre"))
    kept = 1 + (case["post"] != "none" or gr > 0)
    if case["op"] == "seam":            # x, f, gate read; out, y, the checkpoints and their values written
        return {"bytes": 4 * T * C * b + gate + vectors + kept * (ckpt + 2 * T * C) + 4 * norms * T, "flops": 0}
    return {"bytes": 4 * T * C * b + kept * ckpt + 2 * gate + 2 * vectors + 4 * norms * T, "flops": 0}


# ------------------------------------------------------------------------------------------------ the definition, in 64 bits
def _exact_checkpoint(n, dtype):
    """Every block of 32 columns on the grid of the smallest power of two that holds its largest value in 127 steps."""
    T, C = n.shape
    wide = torch.zeros(T, -(-C // 32) * 32, dtype=torch.float64, device=n.device)
    wide[:, :C] = n
    top = wide.view(T, -1, 32).abs().max(2).values
    step = torch.full_like(top, 2.0 ** -120)
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -200))) - 6
    for shift in (-1, 0, 1):            # the smallest of the neighbouring exponents that holds the block
        cand = torch.exp2(e - shift)
        step = torch.where((127 * cand >= top) & (e - shift >= -120), cand, step)
    grid = step[:, :, None]
    return (torch.round(wide.view(T, -1, 32) / grid) * grid).view(T, -1)[:, :C].to(dtype)


def _exact_values(c):
    T, C = c["q"].shape
    blocks = torch.arange(C, device=c["q"].device) // 32
    return c["q"].double() * torch.pow(2.0, c["e"].double()[:, blocks] - 127)


def exact(case, seed):
    s = prepare(case, seed)
    dt, T, C = DTYPES[case["dtype"]], case["tokens"], case["cols"]
    if case["op"] == "checkpoint":
        return {"values": _exact_checkpoint(s["x"].double(), torch.float64)}
    if case["op"] == "grad":
        G = torch.empty(case["items"], case["out"], C, dtype=torch.float64, device="cuda")
        for i in range(case["items"]):
            torch.mm(s["dY"][i].double().t(), _exact_values({k: v[i] for k, v in s["c"].items()}), out=G[i])
        return {"G": G if s["gain"] is None else G * s["gain"].double()}
    one, zero = torch.ones(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    gain = {k: one if s[k + "_gain"] is None else s[k + "_gain"].double() for k in ("post", "pre")}
    bias = {k: zero if s[k + "_bias"] is None else s[k + "_bias"].double() for k in ("post", "pre")}
    gr = case["gate_rows"]
    row = torch.arange(T, device="cuda") // max(1, gr)
    gate = s["gate"].double()[row] if gr else torch.ones(T, 1, dtype=torch.float64, device="cuda")
    if case["op"] == "seam":
        def normalised(v, kind):
            mean = v.sum(1, keepdim=True) / C if kind == "layer" else 0.0
            r = 1 / torch.sqrt(((v - mean) ** 2).sum(1, keepdim=True) / C + EPS)
            return (v, None) if kind == "none" else ((v - mean) * r, r[:, 0])
        n, r = normalised(s["f"].double(), case["post"])
        out = s["skip"] * s["x"].double() + s["scale"] * gate * (n * gain["post"] + bias["post"])
        m, t = normalised(out.to(dt).double(), case["pre"])
        kept = case["post"] != "none" or gr
        return {"out": out, "y": m * gain["pre"] + bias["pre"],
                "post": _exact_checkpoint(n, torch.float64) if kept else None,
                "pre": _exact_checkpoint(m, torch.float64), "post_rstd": r, "pre_rstd": t}

    def through(g, n, r, kind):
        if kind == "none":
            return g
        inner = (g * n).sum(1, keepdim=True) / C
        mean = g.sum(1, keepdim=True) / C if kind == "layer" else 0.0
        return r.double()[:, None] * (g - mean - n * inner)
    m, dy = _exact_values(s["pre_c"]), s["dy"].double()
    d = s["dout"].double() + through(dy * gain["pre"], m, s["pre_rstd"], case["pre"])
    n = _exact_values(s["post_c"]) if s["post_c"] is not None else None
    du = s["scale"] * gate * d
    res = {"dx": s["skip"] * d, "df": through(du * gain["post"], n, s["post_rstd"], case["post"]),
           "pre_gain": torch.einsum("tc,tc->c", dy, m)}
    if s["pre_bias"] is not None:
        res["pre_bias"] = dy.sum(0)
    if s["post_gain"] is not None:
        res["post_gain"] = torch.einsum("tc,tc->c", du, n)
    if s["post_bias"] is not None:
        res["post_bias"] = du.sum(0)
    if gr:
        each = s["scale"] * d * (n * gain["post"] + bias["post"])
        res["gate"] = torch.zeros(-(-T // gr), C, dtype=torch.float64, device="cuda").index_add_(0, row, each)
    return res
