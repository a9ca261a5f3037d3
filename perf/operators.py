"""The language-model operators of the framework as measured cases: residual + RMSNorm with an E4M3
output (and its gradients), the linear layer on E4M3 codes with a scale for each block of 128 (and
its gradients and casts), and rotary positions for long contexts (and their gradients).

Each case has a plain form in elementary torch operations (float32 arithmetic, float64 angles) and
the framework's own calls; ``own`` selects which of the two ``run`` takes.  ``exact`` is the same
result from the operator's definition in float64.

Scales follow the framework's blockwise recipe: a tile with largest magnitude amax is stored as
E4M3(v s) with s = min(448 / amax, 2^100) (1 for a tile of zeros), and a code c stands for c / s.
"""
import math

import torch

own = False

TILE = 128
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a layer's norm while answering: the residual stream is updated in place of
        # a separate addition and the normalised row feeds an FP8 linear
        dict(name="norm_token", op="norm", rows=1, dim=4096, act="bf16", res="bf16", fp8=True, train=False),
        # a prompt (4096 + 512 tokens, the benchmark's sequence) with the fp32 residual stream the blocks keep
        dict(name="norm_prompt", op="norm", rows=4608, dim=4096, act="bf16", res="f32", fp8=True, train=False),
        # the gradient of a norm in a training step on an odd number of packed tokens
        dict(name="norm_grad", op="norm_bwd", rows=4095, dim=5120, act="bf16", res="bf16"),
        # one token through a fused q|k|v projection: the weights' bytes are the whole cost
        dict(name="linear_token", op="linear", m=1, n=6144, k=4096, bias=False),
        # a batch of sequences answering together, through the long-K second linear of an MLP
        dict(name="linear_batch", op="linear", m=48, n=4096, k=14336, bias=True),
        # a chunk of a prompt on ragged widths (a tile that ends inside a block in every direction)
        dict(name="linear_ragged", op="linear", m=1000, n=2568, k=1360, bias=True),
        # a whole prompt through the first linear of an MLP: the tensor cores' case
        dict(name="linear_prompt", op="linear", m=4608, n=12288, k=4096, bias=True),
        # the gradients of a linear in a training step: the gradient's casts, dx, dW and db
        dict(name="linear_grad", op="linear_bwd", m=4095, n=4096, k=4096),
        # a training step's activations cast for the forward product and, transposed, for dW
        dict(name="cast_both", op="cast", rows=4095, cols=4096, square=False, src="bf16"),
        # one new token for each of 32 sequences far into their context, grouped heads
        dict(name="rope_token", op="rope", batch=32, seq=1, hq=32, hk=8, d=128, rot=128, inter=False,
             scaling="by_parts", start=120000, head_major=False, grad=False, act="bf16"),
        # a prompt rotated straight into the head-major layout the attention reads
        dict(name="rope_prompt", op="rope", batch=2, seq=4608, hq=32, hk=8, d=128, rot=128, inter=True,
             scaling="linear", start=0, head_major=True, grad=False, act="bf16"),
        # the gradient of a partial rotation (half of each head) with odd lengths and head counts
        dict(name="rope_grad", op="rope", batch=3, seq=1537, hq=25, hk=5, d=96, rot=48, inter=False,
             scaling="none", start=7, head_major=False, grad=True, act="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "linear", "linear", "linear_bwd", "cast", "rope", "rope"])
    if op == "norm":
        fp8 = rng.random() < 0.7
        dim = _log_int(rng, 256, 8192, 16 if fp8 else 8)
        rows = _log_int(rng, 1, min(16384, 20_000_000 // dim))
        return dict(op=op, rows=rows, dim=dim, act=rng.choice(["bf16", "bf16", "f32"]),
                    res=rng.choice(["none", "bf16", "f32"]), fp8=fp8, train=rng.random() < 0.5)
    if op == "norm_bwd":
        dim = _log_int(rng, 256, 8192, 8)
        rows = _log_int(rng, 1, min(16384, 20_000_000 // dim))
        return dict(op=op, rows=rows, dim=dim, act=rng.choice(["bf16", "bf16", "f32"]), res=rng.choice(["bf16", "f32"]))
    if op == "linear":
        n, k = _log_int(rng, 128, 12288, 8), _log_int(rng, 128, 14336, 16)
        m = _log_int(rng, 1, max(2, min(6000, 180_000_000_000 // (n * k))))
        return dict(op=op, m=m, n=n, k=k, bias=rng.random() < 0.5)
    if op == "linear_bwd":
        n, k = _log_int(rng, 128, 6144, 8), _log_int(rng, 128, 6144, 16)
        m = _log_int(rng, 16, max(32, min(6000, 60_000_000_000 // (n * k))))
        return dict(op=op, m=m, n=n, k=k)
    if op == "cast":
        cols = _log_int(rng, 128, 8192, 16)
        return dict(op=op, rows=_log_int(rng, 1, max(2, min(8192, 16_000_000 // cols))), cols=cols,
                    square=rng.random() < 0.4, src=rng.choice(["bf16", "bf16", "f32"]))
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 4, 5, 8, 12])
    hq = hk * rng.choice([1, 2, 4, 5, 7])
    batch = rng.choice([1, 1, 2, 3, 8, 32])
    seq = _log_int(rng, 1, max(2, min(16384, 40_000_000 // (batch * (hq + hk) * d))))
    return dict(op="rope", batch=batch, seq=seq, hq=hq, hk=hk, d=d, rot=rng.choice([d, d, d // 2, 32, 20]),
                inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "by_parts"]),
                start=rng.choice([0, 3, 4095, 131072, 1000000]), head_major=rng.random() < 0.5,
                grad=rng.random() < 0.3, act=rng.choice(["bf16", "bf16", "f32"]))


# ---------------------------------------------------------------------------------------- inputs
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tiles(n):
    return (n + TILE - 1) // TILE


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, dim):
    """Rows as a layer sees them: unit values, a few channels and a few tokens far larger, and padding rows."""
    x = _normal(g, rows, dim)
    x[:, torch.randint(0, dim, (max(1, dim // 512),), generator=g, device="cuda")] *= 12.0
    x *= torch.exp(0.5 * _normal(g, rows, 1))
    if rows >= 64:
        x[rows // 2] = 0.0
    return x


def _padded(t, rows_to, cols_to):
    out = torch.zeros(rows_to, cols_to, dtype=t.dtype, device=t.device)
    out[: t.shape[0], : t.shape[1]] = t
    return out


def _row_cast(x):
    """Codes [R, C] and scales [ceil(C/128), R] of 1 x 128 tiles."""
    rows, cols = x.shape
    t = _padded(x.float(), rows, _tiles(cols) * TILE).view(rows, -1, TILE)
    amax = t.abs().amax(-1)
    s = torch.where(amax > 0, (448.0 / amax).clamp(max=2.0**100), torch.ones_like(amax))
    q = (t * s[:, :, None]).clamp(-448.0, 448.0).to(F8).view(rows, -1)[:, :cols]
    return q.contiguous(), s.t().contiguous()


def _square_cast(x):
    """Codes [R, C] and scales [ceil(R/128), ceil(C/128)] of 128 x 128 tiles."""
    rows, cols = x.shape
    tr, tc = _tiles(rows), _tiles(cols)
    t = _padded(x.float(), tr * TILE, tc * TILE).view(tr, TILE, tc, TILE)
    amax = t.abs().amax(dim=(1, 3))
    s = torch.where(amax > 0, (448.0 / amax).clamp(max=2.0**100), torch.ones_like(amax))
    q = (t * s[:, None, :, None]).clamp(-448.0, 448.0).to(F8).view(tr * TILE, tc * TILE)[:rows, :cols]
    return q.contiguous(), s.contiguous()


def _wide(t):
    """[R, C] codes with their rows padded to a multiple of 16 bytes, zeros behind the last column."""
    return _padded(t.view(torch.uint8), t.shape[0], (t.shape[1] + 15) // 16 * 16)


def _rope_cfg(c):
    """(theta, factor, orig_len, low, high, mscale) of a case."""
    if c["scaling"] == "none":
        return 10000.0, 1.0, 0, 1.0, 4.0, 1.0
    if c["scaling"] == "linear":
        return 10000.0, 4.0, 0, 1.0, 4.0, 1.0
    return 500000.0, 16.0, 8192, 1.0, 32.0, 0.1 * math.log(16.0) + 1.0


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    s = {"case": c}
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        r, d, act = c["rows"], c["dim"], DT[c["act"]]
        res = None if c["res"] == "none" else DT[c["res"]] if c["act"] == "bf16" else torch.float32
        s["x"] = _activations(g, r, d).to(act)
        s["res"] = None if res is None else (3.0 * _activations(g, r, d)).to(res)
        s["gain"] = (1.0 + 0.2 * _normal(g, d)).to(act)
        s["h"] = None if res is None else new(r, d, dtype=res)
        s["y"] = None if c["fp8"] and not c["train"] else new(r, d, dtype=act)
        s["yq"], s["sy"] = (new(r, d, dtype=torch.uint8), new(_tiles(d), r)) if c["fp8"] else (None, None)
        s["rstd"] = new(r) if c["train"] else None
    elif c["op"] == "norm_bwd":
        r, d, act = c["rows"], c["dim"], DT[c["act"]]
        res = DT[c["res"]] if c["act"] == "bf16" else torch.float32
        s["h"] = (3.0 * _activations(g, r, d)).to(res)
        s["dy"] = (0.01 * _normal(g, r, d)).to(act)
        s["gain"] = (1.0 + 0.2 * _normal(g, d)).to(act)
        s["rstd"] = (s["h"].double().square().mean(-1) + 1e-6).rsqrt().float()
        s["dh_in"] = (0.01 * _normal(g, r, d)).to(res)
        s["dh"], s["dgain"] = new(r, d, dtype=res), new(d)
    elif c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        xq, s["sx"] = _row_cast(_activations(g, m, k).to(torch.bfloat16))
        wq, s["sw"] = _square_cast((_normal(g, n, k) * k**-0.5).to(torch.bfloat16))
        s["xq"], s["wq"] = xq.view(torch.uint8), wq.view(torch.uint8)
        s["b"] = (0.1 * _normal(g, n)).to(torch.bfloat16) if c["bias"] else None
        s["y"] = new(m, n, dtype=torch.bfloat16)
    elif c["op"] == "linear_bwd":
        m, n, k = c["m"], c["n"], c["k"]
        s["dy"] = (0.001 * _activations(g, m, n)).to(torch.bfloat16)
        wq, s["sw"] = _square_cast((_normal(g, n, k) * k**-0.5).to(torch.bfloat16))
        xt, s["sxt"] = _row_cast(_activations(g, m, k).to(torch.bfloat16).t())
        s["wt"], s["xt"] = _wide(wq.t()), _wide(xt)
        s["dx"], s["dw"], s["db"] = new(m, k, dtype=torch.bfloat16), new(n, k), new(n)
    elif c["op"] == "cast":
        r, k = c["rows"], c["cols"]
        s["x"] = (_activations(g, r, k) * (0.02 if c["square"] else 1.0)).to(DT[c["src"]])
        ld = (r + 15) // 16 * 16
        s["q"], s["qt"] = new(r, k, dtype=torch.uint8), new(k, ld, dtype=torch.uint8)
        s["s"] = new(_tiles(r), _tiles(k)) if c["square"] else new(_tiles(k), r)
        s["st"] = None if c["square"] else new(_tiles(r), k)
    else:
        b, n, hq, hk, d, act = c["batch"], c["seq"], c["hq"], c["hk"], c["d"], DT[c["act"]]
        # q and k lie in one packed projection, v behind them
        packed = _normal(g, b, n, (hq + 2 * hk) * d).to(act)
        s["q"] = packed[..., : hq * d].unflatten(-1, (hq, d))
        s["k"] = packed[..., hq * d : (hq + hk) * d].unflatten(-1, (hk, d))
        s["pos"] = (c["start"] + torch.arange(n, device="cuda"))[None, :] + torch.randint(0, 64, (b, 1), generator=g, device="cuda")
        for name, h in (("q_out", hq), ("k_out", hk)):
            s[name] = new(b, h, n, d, dtype=act).transpose(1, 2) if c["head_major"] else new(b, n, h, d, dtype=act)
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    h = x if s["res"] is None else (x + s["res"].float()).to(s["res"].dtype)
    v = h.float()
    rstd = 1.0 / torch.sqrt(v.square().mean(-1) + 1e-6)
    y = v * rstd[:, None] * s["gain"].float()
    out = {}
    if s["res"] is not None:
        out["h"] = h
    if s["y"] is not None:
        out["y"] = y.to(s["x"].dtype)
    if c["fp8"]:
        out["yq"], out["sy"] = _row_cast(y)
    if c["train"]:
        out["rstd"] = rstd
    return out


def _plain_norm_bwd(s):
    v, g, rstd = s["h"].float(), s["gain"].float(), s["rstd"][:, None]
    n = v * rstd
    dy = s["dy"].float()
    a = dy * g
    dh = rstd * (a - n * (a * n).mean(-1, keepdim=True)) + s["dh_in"].float()
    return {"dh": dh.to(s["h"].dtype), "dgain": (dy * n).sum(0)}


def _values_rows(q, s, cols):
    """The values of codes [R, >= C] under scales [ceil(C/128), R]."""
    return q.view(F8).float()[:, :cols] / s.t().repeat_interleave(TILE, 1)[:, :cols]


def _values_square(q, s, rows, cols):
    return q.view(F8).float()[:rows, :cols] / s.repeat_interleave(TILE, 0)[:rows].repeat_interleave(TILE, 1)[:, :cols]


def _plain_linear(s):
    c = s["case"]
    x, w = _values_rows(s["xq"], s["sx"], c["k"]), _values_square(s["wq"], s["sw"], c["n"], c["k"])
    y = x @ w.t()
    if s["b"] is not None:
        y = y + s["b"].float()
    return {"y": y.to(torch.bfloat16)}


def _plain_linear_bwd(s):
    c = s["case"]
    m, n, k = c["m"], c["n"], c["k"]
    gq, gs = _row_cast(s["dy"])
    tq, ts = _row_cast(s["dy"].t())
    w = _values_square(s["wt"], s["sw"].t(), k, n)
    dx = _values_rows(gq, gs, n) @ w.t()
    dw = _values_rows(tq, ts, m) @ _values_rows(s["xt"], s["sxt"], m).t()
    return {"dx": dx.to(torch.bfloat16), "dw": dw, "db": s["dy"].float().sum(0)}


def _plain_cast(s):
    if s["case"]["square"]:
        q, sc = _square_cast(s["x"])
        return {"q": q, "s": sc, "qt": _wide(q.t()).view(F8)}
    q, sc = _row_cast(s["x"])
    qt, st = _row_cast(s["x"].t())
    return {"q": q, "s": sc, "qt": _wide(qt).view(F8), "st": st}


def _frequencies(c, dtype=torch.float64):
    theta, factor, orig, low, high, mscale = _rope_cfg(c)
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=dtype)
    f = theta ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "by_parts":
        ramp = ((orig * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * ramp + (1.0 - ramp) * f / factor
    return f, mscale


def _plain_rope(s):
    c = s["case"]
    f, mscale = _frequencies(c)
    angle = s["pos"].double()[..., None] * f
    cos, sin = (mscale * angle.cos()).float()[:, :, None, :], (mscale * angle.sin()).float()[:, :, None, :]
    if c["grad"]:
        sin = -sin
    half = c["rot"] // 2

    def turn(x):
        v = x.float()
        a, b = (v[..., 0 : c["rot"] : 2], v[..., 1 : c["rot"] : 2]) if c["inter"] else (v[..., :half], v[..., half : c["rot"]])
        a, b = a * cos - b * sin, a * sin + b * cos
        y = v.clone()
        if c["inter"]:
            y[..., 0 : c["rot"] : 2], y[..., 1 : c["rot"] : 2] = a, b
        else:
            y[..., :half], y[..., half : c["rot"]] = a, b
        return y.to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "linear": _plain_linear, "linear_bwd": _plain_linear_bwd,
         "cast": _plain_cast, "rope": _plain_rope}


# ---------------------------------------------------------------------------------------- the framework's calls
def _own(s):
    from diffusion_transformer_flux_gb300 import _lib as L

    c = s["case"]
    if c["op"] == "norm":
        L.mmdit_add_rmsnorm_fwd(s["x"], s["gain"], residual=s["res"], h=s["h"], y=s["y"], y_q=s["yq"], s_y=s["sy"],
                                rstd=s["rstd"], eps=1e-6)
        out = {k: s[k] for k in ("h", "y", "sy", "rstd") if s[k] is not None}
        if s["yq"] is not None:
            out["yq"] = s["yq"].view(F8)
        return out
    if c["op"] == "norm_bwd":
        if "ws" not in s:
            s["ws"] = L.workspace(L.mmdit_add_rmsnorm_bwd_workspace_size(c["rows"], c["dim"]))
        L.mmdit_add_rmsnorm_bwd(s["dy"], s["h"], s["gain"], s["rstd"], s["dh"], dh_in=s["dh_in"], dgain=s["dgain"],
                                ws=s["ws"])
        return {"dh": s["dh"], "dgain": s["dgain"]}
    if c["op"] == "linear":
        if "ws" not in s:
            s["ws"] = L.workspace(L.mmdit_fp8_block_linear_workspace_size(c["m"], c["n"], c["k"]))
        L.mmdit_fp8_block_linear_fwd(s["xq"], s["sx"], s["wq"], s["sw"], s["b"], s["y"], ws=s["ws"])
        return {"y": s["y"]}
    if c["op"] == "linear_bwd":
        if "ws" not in s:
            s["ws"] = L.workspace(L.mmdit_fp8_block_linear_bwd_workspace_size(c["m"], c["n"], c["k"]))
        L.mmdit_fp8_block_linear_bwd(s["dy"], s["wt"], s["sw"], s["xt"], s["sxt"], dx=s["dx"], dw=s["dw"], db=s["db"],
                                     ws=s["ws"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if c["op"] == "cast":
        L.mmdit_fp8_block_cast(s["x"], s["q"], s["s"], q_t=s["qt"], s_t=s["st"], square=c["square"])
        out = {"q": s["q"].view(F8), "s": s["s"], "qt": s["qt"].view(F8)}
        if s["st"] is not None:
            out["st"] = s["st"]
        return out
    if "cfg" not in s:
        theta, factor, orig, low, high, mscale = _rope_cfg(c)
        s["cfg"] = L.make_rope_cfg(c["rot"], theta=theta, interleaved=c["inter"], scaling=c["scaling"], factor=factor,
                                   orig_len=orig, low=low, high=high, mscale=mscale)
    turn = L.mmdit_rope_bwd if c["grad"] else L.mmdit_rope_fwd
    turn(s["cfg"], s["q"], s["q_out"], k=s["k"], k_out=s["k_out"], positions=s["pos"])
    return {"q": s["q_out"], "k": s["k_out"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------- float64 definitions
def _split64(t, axis):
    """Largest magnitude of each group of 128 along `axis`, spread back over the group."""
    parts = [p.abs().amax(axis, keepdim=True).expand_as(p) for p in t.split(TILE, axis)]
    return torch.cat(parts, axis)


def _scale64(amax):
    return torch.where(amax > 0, (448.0 / amax).clamp(max=2.0**100), torch.ones_like(amax))


def _first(t, axis):
    """One value of each group of 128 along `axis`."""
    return t.index_select(axis, torch.arange(0, t.shape[axis], TILE, device=t.device))


def _round_e4m3(t, s):
    """The values that E4M3 codes of float32 inputs `t` under float32 scales stand for."""
    s32 = s.float()
    return (t.float() * s32).clamp(-448, 448).to(F8).double() / s32.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        h = s["x"].double() if s["res"] is None else (s["x"].double() + s["res"].double()).to(s["res"].dtype).double()
        ms = torch.einsum("rd,rd->r", h, h) / c["dim"]
        y = h * (ms + 1e-6)[:, None].pow(-0.5) * s["gain"].double()
        out = {}
        if s["res"] is not None:
            out["h"] = h
        if s["y"] is not None:
            out["y"] = y
        if c["fp8"]:
            sc = _scale64(_split64(y, 1))
            # the codes' unrounded value: both sides sit half an E4M3 step around it
            out["yq"], out["sy"] = y * sc, _first(sc, 1).t().contiguous()
        if c["train"]:
            out["rstd"] = (ms + 1e-6).pow(-0.5)
        return out
    if c["op"] == "norm_bwd":
        # y_j = g_j h_j r, r the stored reciprocal: dL/dh_i = r g_i dy_i - r^3 h_i / D sum_j dy_j g_j h_j
        h, r = s["h"].double(), s["rstd"].double()
        dot = torch.einsum("rd,rd,d->r", s["dy"].double(), h, s["gain"].double())
        dh = r[:, None] * s["dy"].double() * s["gain"].double() - (r.pow(3) * dot / c["dim"])[:, None] * h
        return {"dh": dh + s["dh_in"].double(), "dgain": torch.einsum("rd,rd,r->d", s["dy"].double(), h, r)}
    if c["op"] == "linear":
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        x, w = s["xq"].view(F8).double(), s["wq"].view(F8).double()
        for j in range(_tiles(c["k"])):
            part = slice(j * TILE, min((j + 1) * TILE, c["k"]))
            sw = s["sw"][:, j].double().repeat_interleave(TILE)[: c["n"]]
            y += (x[:, part] @ w[:, part].t()) / s["sx"][j].double()[:, None] / sw[None, :]
        return {"y": y if s["b"] is None else y + s["b"].double()}
    if c["op"] == "linear_bwd":
        dy = s["dy"].double()
        g_rows, g_cols = _round_e4m3(dy, _scale64(_split64(s["dy"].float(), 1))), _round_e4m3(dy, _scale64(_split64(s["dy"].float(), 0)))
        w = s["wt"].view(F8).double()[:, : c["n"]].t()
        w = w / s["sw"].double().repeat_interleave(TILE, 0)[: c["n"]].repeat_interleave(TILE, 1)[:, : c["k"]]
        x = s["xt"].view(F8).double()[:, : c["m"]].t() / s["sxt"].double().repeat_interleave(TILE, 0)[: c["m"]]
        return {"dx": g_rows @ w, "dw": g_cols.t() @ x, "db": dy.sum(0)}
    if c["op"] == "cast":
        x = s["x"].double()
        if c["square"]:
            sc = _scale64(_split64(_split64(x, 0), 1))
            q, first = x * sc, _first(_first(sc, 0), 1)
            qt = torch.zeros(c["cols"], s["qt"].shape[1], dtype=torch.float64, device="cuda")
            qt[:, : c["rows"]] = q.t()
            return {"q": q, "s": first, "qt": qt}
        sr, sk = _scale64(_split64(x, 1)), _scale64(_split64(x, 0))
        qt = torch.zeros(c["cols"], s["qt"].shape[1], dtype=torch.float64, device="cuda")
        qt[:, : c["rows"]] = (x * sk).t()
        return {"q": x * sr, "s": _first(sr, 1).t().contiguous(), "qt": qt, "st": _first(sk, 0)}
    # rotary positions as a complex product: (a + ib) times m exp(i p f), or its conjugate for the gradient
    theta, factor, orig, low, high, mscale = _rope_cfg(c)
    f = torch.tensor([theta ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)], dtype=torch.float64, device="cuda")
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "by_parts":
        turns = orig * f / (2.0 * math.pi)
        keep = torch.where(turns >= high, torch.ones_like(f), torch.where(turns <= low, torch.zeros_like(f), (turns - low) / (high - low)))
        f = keep * f + (1 - keep) * (f / factor)
    z = torch.polar(torch.full_like(f, mscale).expand(*s["pos"].shape, -1).contiguous(), s["pos"].double()[..., None] * f)
    z = (z.conj() if c["grad"] else z)[:, :, None, :]
    out = {}
    for name in ("q", "k"):
        v = s[name].double()
        r = v[..., : c["rot"]]
        pairs = r.unflatten(-1, (-1, 2)) if c["inter"] else torch.stack((r[..., : c["rot"] // 2], r[..., c["rot"] // 2 :]), -1)
        t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        t = t.flatten(-2) if c["inter"] else torch.cat((t[..., 0], t[..., 1]), -1)
        out[name] = torch.cat((t, v[..., c["rot"] :]), -1)
    return out


# ---------------------------------------------------------------------------------------- floors
def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] == "norm":
        n, a = c["rows"] * c["dim"], size[c["act"]]
        r = size[c["res"]] if c["act"] == "bf16" or c["res"] == "none" else 4
        out = 2 * r + (a if c["train"] or not c["fp8"] else 0) + (1 if c["fp8"] else 0)
        small = c["dim"] * a + (4 * _tiles(c["dim"]) * c["rows"] if c["fp8"] else 0) + (4 * c["rows"] if c["train"] else 0)
        return {"bytes": n * (a + out) + small, "flops": 6 * n}
    if c["op"] == "norm_bwd":
        n, a = c["rows"] * c["dim"], size[c["act"]]
        r = size[c["res"]] if c["act"] == "bf16" else 4
        return {"bytes": n * (a + 3 * r) + c["dim"] * (a + 4) + 4 * c["rows"], "flops": 10 * n}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k + n * k + 2 * m * n + 4 * m * _tiles(k) + 4 * _tiles(n) * _tiles(k), "flops": 2 * m * n * k}
    if c["op"] == "linear_bwd":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * n + n * k + m * k + 4 * k * _tiles(m) + 2 * m * k + 4 * n * k + 4 * n, "flops": 4 * m * n * k}
    if c["op"] == "cast":
        n = c["rows"] * c["cols"]
        scales = 4 * _tiles(c["rows"]) * _tiles(c["cols"]) if c["square"] else 4 * (_tiles(c["cols"]) * c["rows"] + _tiles(c["rows"]) * c["cols"])
        return {"bytes": n * (size[c["src"]] + 2) + scales, "flops": 4 * n}
    n = c["batch"] * c["seq"] * (c["hq"] + c["hk"]) * c["d"]
    return {"bytes": 2 * n * size[c["act"]] + 8 * c["batch"] * c["seq"], "flops": 3 * n}
