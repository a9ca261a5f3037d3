"""GPU parity of the language-model operators against the float64 oracle (oracle.lm).

Tolerances count roundings.  u = 2^-24 is half a float32 step; a stored bf16 value is off by 2^-8 of
itself, an E4M3 code by 2^-4 of itself (2^-10 below its normal range).  Sums of n float32 terms in any
order are off by at most n u times the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from diffusion_transformer_flux_gb300 import _lib as L
from oracle import lm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(rng, shape, dtype=torch.bfloat16, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(dtype)


def check(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref) - tol
    assert err.max() <= 0, f"{what}: {np.abs(got - ref).max():.3e} off at {np.unravel_index(err.argmax(), err.shape)}"


def tiles(n):
    return (n + 127) // 128


def nans(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), device="cuda", dtype=dtype)


def bytes_(*shape):
    return torch.full(shape, 0xAA, device="cuda", dtype=torch.uint8)


# ------------------------------------------------------------------------------------- RMSNorm
NORM_SHAPES = [(1, 8), (3, 24), (5, 128), (130, 272), (7, 2048), (33, 4096), (2, 4104), (3, 8200), (2, 16384)]


@pytest.mark.parametrize("rows,dim", NORM_SHAPES)
@pytest.mark.parametrize("act,res", [("bf16", None), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", None)])
def test_norm(rows, dim, act, res):
    rng = np.random.default_rng(rows * 7 + dim)
    dt = DT[act]
    x, gain = make(rng, (rows, dim), dt), (1 + 0.2 * make(rng, (dim,), torch.float32)).to(dt)
    x[:, dim // 3] *= 16
    if rows > 2:
        x[1] = 0
    r = None if res is None else make(rng, (rows, dim), DT[res], 3.0)
    if r is not None and rows > 2:
        r[1] = 0
    h = None if res is None else nans(rows, dim, dtype=DT[res])
    y, rstd = nans(rows, dim, dtype=dt), nans(rows)
    q, s = (bytes_(rows, dim), nans(tiles(dim), rows)) if dim % 16 == 0 else (None, None)
    L.mmdit_add_rmsnorm_fwd(x, gain, residual=r, h=h, y=y, y_q=q, s_y=s, rstd=rstd, eps=1e-6)
    if r is None:
        hv = f64(x)
    else:
        # one float32 addition, one rounding to the residual's type: reproduced exactly
        assert torch.equal(h, (x.float() + r.float()).to(h.dtype))
        hv = f64(h)
    yo, ro = lm.rmsnorm(hv, f64(gain), 1e-6)
    # the mean of squares: dim additions and products, then a division, an addition and a root
    stat = (dim + 8) * U
    check(f64(rstd), ro, stat * ro, "rstd")
    check(f64(y), yo, (HALF[dt] + stat + 4 * U) * np.abs(yo), "y")
    if q is not None:
        amax = np.stack([np.abs(yo[:, 128 * j:128 * (j + 1)]).max(1) for j in range(tiles(dim))])
        so = np.where(amax > 0, 448.0 / np.where(amax > 0, amax, 1), 1.0)
        check(f64(s), so, (stat + 8 * U) * so, "s_y")
        v = yo * np.repeat(f64(s).T, 128, 1)[:, :dim]
        check(lm.decode(q.cpu().numpy()), v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + (stat + 8 * U) * np.abs(v), "codes")


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("outputs", ["y", "q", "yq", "h", "hq", "hyq"])
def test_norm_output_sets(res, outputs):
    """Every set of outputs that may be asked for gives what the full set gives."""
    if res is None and "h" in outputs:
        pytest.skip("h needs a residual")
    rng = np.random.default_rng(8)
    x, gain = make(rng, (5, 272)), make(rng, (272,))
    r = None if res is None else make(rng, (5, 272), DT[res])
    full = dict(h=None if r is None else nans(5, 272, dtype=r.dtype), y=nans(5, 272, dtype=torch.bfloat16), y_q=bytes_(5, 272),
                s_y=nans(3, 5), rstd=nans(5))
    L.mmdit_add_rmsnorm_fwd(x, gain, residual=r, **full)
    names = ["y"] if outputs == "h" else []  # h beside y
    names += [n for c, ns in (("h", ["h"]), ("y", ["y"]), ("q", ["y_q", "s_y"])) if c in outputs for n in ns]
    some = {n: torch.full_like(full[n], 0xAA if n == "y_q" else float("nan")) for n in names}
    L.mmdit_add_rmsnorm_fwd(x, gain, residual=r, **some)
    assert all(torch.equal(some[n], full[n]) for n in names)


def test_norm_strided_rows_in_place_residual():
    rng = np.random.default_rng(3)
    wide = make(rng, (9, 3 * 256))
    x, res, gain = wide[:, 256:512], make(rng, (9, 256), torch.float32), make(rng, (256,))
    h0 = x.float() + res
    y = nans(9, 256, dtype=torch.bfloat16)
    L.mmdit_add_rmsnorm_fwd(x, gain, residual=res, h=res, y=y)
    assert torch.equal(res, h0)
    yo, _ = lm.rmsnorm(f64(h0), f64(gain), 1e-6)
    check(f64(y), yo, (2.0 ** -8 + 270 * U) * np.abs(yo), "y")


def test_norm_extreme_rows():
    """Infinities and NaN stay in their rows; denormal rows keep a finite scale; a NaN element leaves its
    tile's other codes alone only where the row's mean stays finite, so it makes its own row NaN."""
    x = torch.ones(6, 256, device="cuda")
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1e-42
    x[4] = 0
    gain = torch.ones(256, device="cuda")
    y, q, s = nans(6, 256), bytes_(6, 256), nans(2, 6)
    L.mmdit_add_rmsnorm_fwd(x, gain, y=y, y_q=q, s_y=s, eps=0.5)
    v = lm.decode(q.cpu().numpy())
    assert torch.isnan(y[2]).all() and np.isnan(v[2]).all()
    assert torch.isnan(y[1, 3]) and (y[1, 4:] == 0).all()
    for r in (0, 5):
        check(f64(y[r]), np.full(256, 1.5 ** -0.5), 300 * U, "ones")
        assert (v[r] == 448).all()
    assert (v[4] == 0).all() and (s[:, 4] == 1).all()
    assert torch.isfinite(s[:, 3]).all() and (s[:, 3] == 2.0 ** 100).all() and np.isfinite(v[3]).all()


@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 24), (129, 272), (1500, 512), (33, 4096), (3, 8200), (2, 16384)])
@pytest.mark.parametrize("act,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_norm_gradients(rows, dim, act, res):
    rng = np.random.default_rng(rows + dim)
    dt, rt = DT[act], DT[res]
    h, dy = make(rng, (rows, dim), rt, 3.0), make(rng, (rows, dim), dt)
    gain, dh_in = (1 + 0.2 * make(rng, (dim,), torch.float32)).to(dt), make(rng, (rows, dim), rt)
    if rows > 2:
        h[1] = 0
    y, r32 = nans(rows, dim, dtype=dt), nans(rows)
    if act == res:
        L.mmdit_add_rmsnorm_fwd(h, gain, y=y, rstd=r32)
    else:
        L.mmdit_add_rmsnorm_fwd(torch.zeros(rows, dim, device="cuda", dtype=dt), gain, residual=h, y=y, rstd=r32)
    dho, dgo = lm.rmsnorm_bwd(f64(dy), f64(h), f64(gain), 1e-6, f64(dh_in))
    r = f64(r32)[:, None]
    n, a = f64(h) * r, f64(dy) * f64(gain)
    # r carries the forward's error (dim + 8) u; the row sum dim u of its magnitudes; ten roundings beside
    big = r * (np.abs(a) + np.abs(n) * (np.abs(a * n)).mean(1, keepdims=True))
    tol = (3 * (dim + 8) + dim + 16) * U * big + (HALF[rt] + 2 * U) * np.abs(dho)
    ws = None
    for given in (dh_in, None):
        dh, dg = nans(rows, dim, dtype=rt), nans(dim)
        dx = nans(rows, dim, dtype=dt) if act != res else None
        ws = L.mmdit_add_rmsnorm_bwd(dy, h, gain, r32, dh, dh_in=given, dx=dx, dgain=dg, ws=ws)
        ref = dho if given is not None else dho - f64(dh_in)
        t = tol if given is not None else tol + (HALF[rt] + 2 * U) * np.abs(ref)
        check(f64(dh), ref, t, "dh")
        if dx is not None:
            check(f64(dx), ref, t + 2.0 ** -8 * np.abs(ref), "dx")
        check(f64(dg), dgo, (rows + dim + 16) * U * np.abs(f64(dy) * n).sum(0) + U * np.abs(dgo), "dgain")
    again = nans(dim)
    L.mmdit_add_rmsnorm_bwd(dy, h, gain, r32, dh, dgain=again, ws=ws)
    assert torch.equal(again, dg)
    assert L.mmdit_workspace_status(ws) == 0


def test_norm_gradient_in_place_and_empty():
    rng = np.random.default_rng(1)
    h, dy, gain = make(rng, (5, 64)), make(rng, (5, 64)), make(rng, (64,))
    r, y = nans(5), nans(5, 64, dtype=torch.bfloat16)
    L.mmdit_add_rmsnorm_fwd(h, gain, y=y, rstd=r)
    d = make(rng, (5, 64))
    out = nans(5, 64, dtype=torch.bfloat16)
    L.mmdit_add_rmsnorm_bwd(dy, h, gain, r, out, dh_in=d)
    L.mmdit_add_rmsnorm_bwd(dy, h, gain, r, d, dh_in=d)
    assert torch.equal(out, d)
    dg = nans(64)
    e = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    L.mmdit_add_rmsnorm_bwd(e, e, gain, torch.empty(0, device="cuda"), e, dgain=dg)
    assert (dg == 0).all()
    L.mmdit_add_rmsnorm_fwd(e, gain, y=e)


# ------------------------------------------------------------------------------------- casts
def cast_source(rng, rows, cols, dtype):
    x = make(rng, (rows, cols), dtype)
    x[rows // 2, cols // 2] = 300.0
    if rows > 3:
        x[3] = 0
    x[:, 1] = 0
    if cols > 128 and rows > 5:
        x[5, 128:] *= 1e-34  # below 448 2^-100: the scale's limit
    return x


@pytest.mark.parametrize("rows,cols", [(1, 16), (2, 128), (16, 144), (100, 64), (128, 128), (129, 272), (300, 400)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_cast_rows(rows, cols, act):
    x = cast_source(np.random.default_rng(rows + cols), rows, cols, DT[act])
    ld = (rows + 15) // 16 * 16
    xv = x.float().cpu().numpy()
    qo, so = lm.cast_rows(xv)
    qto, sto = lm.cast_rows(xv.T)
    for both in (3, 1, 2):
        q, s, qt, st = bytes_(rows, cols), nans(tiles(cols), rows), bytes_(cols, ld), nans(tiles(rows), cols)
        L.mmdit_fp8_block_cast(x, q if both & 1 else None, s if both & 1 else None, q_t=qt if both & 2 else None,
                               s_t=st if both & 2 else None)
        if both & 1:
            assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo)
        if both & 2:
            got = qt.cpu().numpy()
            assert np.array_equal(st.cpu().numpy(), sto) and np.array_equal(got[:, :rows], qto)
            assert not got[:, rows:].any()


@pytest.mark.parametrize("rows,cols", [(1, 16), (24, 128), (128, 144), (200, 64), (257, 272)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_cast_square(rows, cols, act):
    x = cast_source(np.random.default_rng(rows * cols), rows, cols, DT[act])
    qo, so = lm.cast_square(x.float().cpu().numpy())
    q, s, qt = bytes_(rows, cols), nans(tiles(rows), tiles(cols)), bytes_(cols, (rows + 15) // 16 * 16)
    L.mmdit_fp8_block_cast(x, q, s, q_t=qt, square=True)
    assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo)
    got = qt.cpu().numpy()
    assert np.array_equal(got[:, :rows], qo.T) and not got[:, rows:].any()
    s2, qt2 = nans(tiles(rows), tiles(cols)), bytes_(*qt.shape)
    L.mmdit_fp8_block_cast(x, s=s2, q_t=qt2, square=True)
    assert torch.equal(s, s2) and torch.equal(qt, qt2)


def test_cast_nan_and_infinity_stay_in_their_tiles():
    x = torch.ones(130, 256, device="cuda")
    x[0, 7], x[1, 200] = float("nan"), float("inf")
    q, s, qt, st = bytes_(130, 256), nans(2, 130), bytes_(256, 144), nans(2, 256)
    L.mmdit_fp8_block_cast(x, q, s, q_t=qt, s_t=st)
    v, vt = lm.decode(q.cpu().numpy()), lm.decode(qt.cpu().numpy())
    assert np.isnan(v[0, 7]) and (np.delete(v[0], 7) == 448).all() and s[1, 1] == 0 and np.isnan(v[1, 200])
    assert (np.delete(v[1, 128:], 72) == 0).all() and (v[1, :128] == 448).all() and (v[2:] == 448).all()
    assert np.isnan(vt[7, 0]) and (vt[7, 1:130] == 448).all() and np.isnan(vt[200, 1]) and vt[200, 0] == 0
    assert (np.delete(vt, (7, 200), 0)[:, :130] == 448).all()


# ------------------------------------------------------------------------------------- linear
def linear_operands(seed, M, N, K):
    rng = np.random.default_rng(seed)
    x, w = make(rng, (M, K)), make(rng, (N, K), scale=K ** -0.5)
    x[0, K // 2] = 50.0  # an outlier owns its tile's scale
    if M > 2:
        x[2] = 0
    xq, sx, wq, sw = bytes_(M, K), nans(tiles(K), M), bytes_(N, K), nans(tiles(N), tiles(K))
    L.mmdit_fp8_block_cast(x, xq, sx)
    L.mmdit_fp8_block_cast(w, wq, sw, square=True)
    return rng, x, w, xq, sx, wq, sw


def sum_tol(a, b, slices):
    """A slice's four accumulations on the tensor cores (each within 2^-23 of the slice's magnitudes, which
    their sum bounds), the two reciprocals and two products of its factor, and one addition per slice."""
    return (8 + 8 + slices) * 2 * U * (np.abs(a) @ np.abs(b).T)


LINEAR_SHAPES = [(1, 8, 16), (1, 128, 128), (2, 136, 144), (4, 264, 1040), (5, 256, 128), (16, 120, 272), (17, 384, 2064),
                 (33, 136, 400), (64, 256, 4096), (65, 128, 528), (100, 520, 144), (128, 256, 256), (129, 264, 272),
                 (255, 8, 1024), (256, 256, 128), (300, 776, 656), (513, 1024, 384), (3, 24, 33024), (9, 8, 160),
                 (12, 1040, 2000), (2100, 1288, 272), (513, 2600, 2064), (300, 2056, 2176),
                 (10, 136, 8208), (64, 7816, 272),
                 (2100, 2568, 272), (5000, 1288, 16), (2100, 2568, 640)]  # more tiles than pairs, of 3, 1 and 5 slices


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_linear(M, N, K):
    rng, x, w, xq, sx, wq, sw = linear_operands(M * 3 + N + K, M, N, K)
    b = make(rng, (N,))
    xv = lm.values_rows(xq.cpu().numpy(), sx.cpu().numpy())
    wv = lm.values_square(wq.cpu().numpy(), sw.cpu().numpy())
    ref, tol = xv @ wv.T, sum_tol(xv, wv, tiles(K))
    ws = L.workspace(256)
    for bias in (None, b):
        r = ref if bias is None else ref + f64(bias)
        t = tol + 2 * U * np.abs(r)
        y32, y16 = nans(M, N), nans(M, N, dtype=torch.bfloat16)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, bias, y32, ws=ws)
        check(f64(y32), r, t, "y fp32")
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, bias, y16, ws=ws)
        assert torch.equal(y16, y32.to(torch.bfloat16))
        again = nans(M, N)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, bias, again, ws=ws)
        assert torch.equal(again, y32)
    assert L.mmdit_workspace_status(ws) == 0


def test_linear_writes_its_rows_alone():
    _, _, _, xq, sx, wq, sw = linear_operands(5, 37, 200, 304)
    pad = torch.full((40, 200), 7.0, device="cuda", dtype=torch.bfloat16)
    L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, pad[:37])
    assert (pad[37:] == 7).all() and torch.isfinite(pad).all()
    one = torch.full((3, 200), 7.0, device="cuda", dtype=torch.bfloat16)
    L.mmdit_fp8_block_linear_fwd(xq[:1], sx[:, :1].contiguous(), wq, sw, None, one[1:2])
    assert (one[0] == 7).all() and (one[2] == 7).all()
    rows = torch.stack([one[1], pad[0]]).float()  # a row's sums do not depend on its batch beyond rounding
    assert (rows[0] - rows[1]).abs().max() <= 2.0 ** -7 * rows.abs().max()
    empty = torch.empty(0, 304, device="cuda", dtype=torch.uint8)
    L.mmdit_fp8_block_linear_fwd(empty, torch.empty(3, 0, device="cuda"), wq, sw, None,
                                 torch.empty(0, 200, device="cuda", dtype=torch.bfloat16))


def test_linear_tiles_write_inside_the_output():
    """Tiles that reach over the last row and column leave what lies behind them."""
    M, N, K = 2090, 2568, 272
    _, _, _, xq, sx, wq, sw = linear_operands(6, M, N, K)
    for dtype in (torch.bfloat16, torch.float32):
        pad = torch.full((M + 30, N), 7.0, device="cuda", dtype=dtype)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, pad[10:M + 10])
        assert (pad[:10] == 7).all() and (pad[M + 10:] == 7).all()
        row = nans(1, N, dtype=dtype)
        L.mmdit_fp8_block_linear_fwd(xq[-1:], sx[:, -1:].contiguous(), wq, sw, None, row)
        diff = (row[0].float() - pad[M + 9].float()).abs()
        assert diff.max() <= 2.0 ** -7 * row.float().abs().max()


def test_linear_extreme_scales():
    """Tiles at the scale's limit and near float32's top: the factor 1 / (s_x s_w) stays in range."""
    M, N, K = 20, 128, 256
    x, w = torch.ones(M, K, device="cuda"), torch.ones(N, K, device="cuda")
    x[:, 128:] = 1e-37  # scale 2^100: contributes nothing beside the ones
    x[1] = 1e30
    x[2] = 0
    w[:, 128:] = 1e-35
    xq, sx, wq, sw = bytes_(M, K), nans(2, M), bytes_(N, K), nans(1, 2)
    L.mmdit_fp8_block_cast(x, xq, sx)
    L.mmdit_fp8_block_cast(w, wq, sw, square=True)
    y = nans(M, N)
    L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, y)
    ref = np.full((M, N), 128.0)
    ref[1], ref[2] = 128e30, 0
    check(f64(y), ref, 2.0 ** -3 * 2.0 ** -15 * ref + 1e-30, "y")


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (16, 128, 128), (100, 136, 272), (129, 264, 400), (300, 776, 656),
                                   (520, 128, 1040), (40, 600, 128), (2100, 1288, 1360), (300, 2568, 2576), (16, 2568, 2576)])
def test_linear_gradients(M, N, K):
    rng, x, w, _, _, wq, sw = linear_operands(M + N * 5 + K, M, N, K)
    ldm, ldn = (M + 15) // 16 * 16, (N + 15) // 16 * 16
    dy = make(rng, (M, N), scale=1e-3)
    if M > 4:
        dy[4] = 0
    wt, xt, sxt = bytes_(K, ldn), bytes_(K, ldm), nans(tiles(M), K)
    L.mmdit_fp8_block_cast(w, s=sw, q_t=wt, square=True)
    L.mmdit_fp8_block_cast(x, q_t=xt, s_t=sxt)
    wqc, swc, xtc, sxtc = (t.cpu().numpy() for t in (wq, sw, xt, sxt))
    dxo, dwo, dbo = lm.block_linear_bwd(dy.float().cpu().numpy(), wqc, swc, xtc[:, :M], sxtc)
    g, gt = lm.values_rows(*lm.cast_rows(f64(dy))), lm.values_rows(*lm.cast_rows(f64(dy).T))
    wv, xv = lm.values_square(wqc, swc), lm.values_rows(xtc[:, :M], sxtc)
    dx, dw, db = nans(M, K, dtype=torch.bfloat16), nans(N, K), nans(N)
    ws = L.mmdit_fp8_block_linear_bwd(dy, wt, sw, xt, sxt, dx=dx, dw=dw, db=db)
    check(f64(dx), dxo, sum_tol(g, wv.T, tiles(N)) + 2.0 ** -8 * np.abs(dxo), "dx")
    check(f64(dw), dwo, sum_tol(gt, xv, tiles(M)), "dw")
    check(f64(db), dbo, (M + 8) * U * np.abs(f64(dy)).sum(0), "db")
    for keep in ("dx", "dw", "db"):  # each alone, without the others' operands
        out = {"dx": nans(M, K, dtype=torch.bfloat16), "dw": nans(N, K), "db": nans(N)}[keep]
        ops = {"dx": dict(w_t=wt, s_w=sw), "dw": dict(x_t=xt, s_xt=sxt), "db": {}}[keep]
        L.mmdit_fp8_block_linear_bwd(dy, **ops, **{keep: out}, ws=L.workspace(ws.numel()))
        assert torch.equal(out, {"dx": dx, "dw": dw, "db": db}[keep])
    assert L.mmdit_workspace_status(ws) == 0


def test_linear_gradients_of_no_rows():
    e = torch.empty(0, 128, device="cuda", dtype=torch.bfloat16)
    dw, db = nans(128, 64), nans(128)
    L.mmdit_fp8_block_linear_bwd(e, x_t=torch.empty(64, 0, device="cuda", dtype=torch.uint8),
                                 s_xt=torch.empty(0, 64, device="cuda"), dw=dw, db=db)
    assert (dw == 0).all() and (db == 0).all()


def test_linear_gradient_against_differences():
    """Along a direction of W, the loss <y, dy> of the exact product moves by <dW, direction>: dW from the
    codes agrees to the casts (each factor off by at most 2^-4 of itself, so the sum by 2^-3 of its
    magnitudes; errors of either sign leave far less)."""
    rng, x, w, _, _, _, _ = linear_operands(9, 256, 128, 128)
    dy = make(rng, (256, 128))
    xt, sxt, dw = bytes_(128, 256), nans(2, 128), nans(128, 128)
    L.mmdit_fp8_block_cast(x, q_t=xt, s_t=sxt)
    L.mmdit_fp8_block_linear_bwd(dy, x_t=xt, s_xt=sxt, dw=dw)
    X, D, e = f64(x), f64(dy), 1e-3
    for _ in range(4):
        d = rng.standard_normal((128, 128))
        loss = lambda t: float(((X @ (f64(w) + t * d).T) * D).sum())  # noqa: E731
        slope = (loss(e) - loss(-e)) / (2 * e)
        size = np.sqrt(((np.abs(D).T @ np.abs(X)) ** 2 * d ** 2).sum())
        assert abs(float((f64(dw) * d).sum()) - slope) <= 2.0 ** -3 * size


# ------------------------------------------------------------------------------------- rotary positions
def rope_case(seed, B, S, Hq, Hk, d, rot, inter, act, scaling="none", start=0, head_major=False, mscale=1.0):
    rng = np.random.default_rng(seed)
    kw = dict(theta=10000.0, scaling=scaling, factor=8.0, orig_len=4096.0, low=1.0, high=32.0)
    cfg = L.make_rope_cfg(rot, interleaved=inter, mscale=mscale, **kw)
    packed = make(rng, (B, S, (Hq + 2 * Hk) * d), DT[act])
    q = packed[..., :Hq * d].unflatten(-1, (Hq, d))
    k = packed[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    pos = start + torch.arange(S)[None] + torch.from_numpy(rng.integers(0, 50, (B, 1)))
    out = [nans(B, h, S, d, dtype=DT[act]).transpose(1, 2) if head_major else nans(B, S, h, d, dtype=DT[act])
           for h in (Hq, Hk)]
    cos, sin = lm.rope_cos_sin(pos.numpy(), lm.rope_frequencies(rot, **kw))
    return cfg, q, k, pos.cuda(), out, cos, sin


def rope_check(got, x, cos, sin, rot, inter, mscale, transposed, act):
    ref = lm.rope(f64(x), cos, sin, rot, inter, mscale, transposed)
    # cos and sin: a 24-bit phase of half turns (2^-25 pi) and the function's two steps; three products,
    # one addition; the magnitudes of both terms
    size = lm.rope(np.abs(f64(x)), np.ones_like(cos), np.ones_like(sin), rot, inter, mscale)
    both = np.abs(size)
    if inter:
        pair = np.abs(f64(x))[..., 0:rot:2] + np.abs(f64(x))[..., 1:rot:2]
        both[..., 0:rot:2], both[..., 1:rot:2] = mscale * pair, mscale * pair
    else:
        pair = np.abs(f64(x))[..., :rot // 2] + np.abs(f64(x))[..., rot // 2:rot]
        both[..., :rot // 2], both[..., rot // 2:rot] = mscale * pair, mscale * pair
    check(f64(got)[..., :rot], ref[..., :rot], (HALF[DT[act]] * np.abs(ref) + 16 * U * both)[..., :rot], "rotated")
    assert np.array_equal(f64(got)[..., rot:], f64(x)[..., rot:])


@pytest.mark.parametrize("B,S,Hq,Hk,d,rot,inter,act,scaling,start,head_major", [
    (1, 1, 1, 1, 8, 2, True, "bf16", "none", 0, False),
    (1, 1, 1, 1, 8, 2, False, "f32", "none", 5, False),
    (2, 3, 4, 2, 64, 64, True, "bf16", "none", 0, True),
    (2, 3, 4, 2, 64, 64, False, "bf16", "linear", 9, False),
    (1, 17, 3, 1, 64, 20, False, "bf16", "none", 100, False),   # V = 2
    (1, 17, 3, 1, 64, 20, True, "f32", "none", 100, True),
    (3, 5, 2, 1, 96, 48, False, "bf16", "none", 7, True),
    (1, 4, 2, 2, 80, 40, False, "f32", "none", 1, False),       # V = 4
    (1, 4, 2, 2, 40, 38, False, "bf16", "none", 1, False),      # V = 1
    (32, 1, 8, 2, 128, 128, False, "bf16", "by_parts", 1 << 20, False),
    (1, 9, 2, 1, 256, 256, True, "bf16", "by_parts", 10 ** 9, False),
    (1, 3, 1, 1, 512, 512, False, "f32", "linear", (1 << 40) + 7, True),
    (1, 6, 2, 1, 128, 64, True, "bf16", "none", -20, False),
    (1, 5, 9, 3, 512, 510, False, "bf16", "none", 3, False),    # the most pieces to a head
    (2, 3, 1, 1, 512, 2, False, "f32", "none", 3, True),
    (1, 2, 70, 10, 64, 64, True, "bf16", "none", 11, True),
    (5, 1000, 2, 1, 64, 64, False, "bf16", "none", 0, True),    # four tokens to a CTA
])
def test_rope(B, S, Hq, Hk, d, rot, inter, act, scaling, start, head_major):
    cfg, q, k, pos, (qo, ko), cos, sin = rope_case(B + S + d, B, S, Hq, Hk, d, rot, inter, act, scaling, start, head_major,
                                                   1.25)
    L.mmdit_rope_fwd(cfg, q, qo, k=k, k_out=ko, positions=pos)
    rope_check(qo, q, cos, sin, rot, inter, 1.25, False, act)
    rope_check(ko, k, cos, sin, rot, inter, 1.25, False, act)
    L.mmdit_rope_bwd(cfg, q, qo, k=k, k_out=ko, positions=pos)
    rope_check(qo, q, cos, sin, rot, inter, 1.25, True, act)
    rope_check(ko, k, cos, sin, rot, inter, 1.25, True, act)
    # q alone, in place, on shared positions
    alone = nans(*q.shape, dtype=q.dtype)
    L.mmdit_rope_fwd(cfg, q, alone, positions=pos[0])
    here = q.clone()
    L.mmdit_rope_fwd(cfg, here, here, positions=pos[0])
    assert torch.equal(here, alone)


def test_rope_tables_of_the_image_axes():
    """The tables of rope3d_freqs, applied to q and k outside a block."""
    B, S, H, d = 2, 12, 3, 128
    rng = np.random.default_rng(0)
    ids = torch.from_numpy(rng.integers(0, 20, (B, S, 3)).astype(np.float32)).cuda()
    cos, sin = nans(B, S, 64), nans(B, S, 64)
    L.rope3d_freqs(ids, (16, 56, 56), 10000.0, cos, sin)
    q = make(rng, (B, S, H, d))
    out = nans(B, S, H, d, dtype=torch.bfloat16)
    L.mmdit_rope_fwd(L.make_rope_cfg(128), q, out, cos=cos, sin=sin)
    rope_check(out, q, f64(cos), f64(sin), 128, True, 1.0, False, "bf16")


def test_rope_special_values_pass():
    """Infinities and NaN behind rot_dim pass unchanged; those of one head stay in it."""
    q = torch.zeros(1, 2, 2, 64, device="cuda")
    q[..., 32:] = float("inf")
    q[0, 0, 0, 40] = float("nan")
    q[0, 1, 1, 3] = float("nan")
    out = nans(1, 2, 2, 64)
    for inter in (True, False):
        L.mmdit_rope_fwd(L.make_rope_cfg(32, interleaved=inter), q, out, positions=torch.tensor([3, 4], device="cuda"))
        assert torch.equal(out[..., 32:].isinf(), q[..., 32:].isinf()) and torch.isnan(out[0, 0, 0, 40])
        bad = torch.isnan(out[..., :32])
        assert bad.sum() == 2 and bad[0, 1, 1].sum() == 2


def test_rope_broadcast_input():
    """An input whose heads share an address (one key rotated into every head's place)."""
    one = make(np.random.default_rng(8), (2, 5, 1, 64))
    out, alone = nans(2, 5, 4, 64, dtype=torch.bfloat16), nans(2, 5, 1, 64, dtype=torch.bfloat16)
    cfg, pos = L.make_rope_cfg(64), torch.arange(5, device="cuda")
    L.mmdit_rope_fwd(cfg, one.expand(2, 5, 4, 64), out, positions=pos)
    L.mmdit_rope_fwd(cfg, one, alone, positions=pos)
    assert torch.equal(out, alone.expand(2, 5, 4, 64))


def test_rope_empty():
    e = torch.empty(1, 0, 2, 64, device="cuda")
    L.mmdit_rope_fwd(L.make_rope_cfg(64), e, e, positions=torch.empty(0, dtype=torch.int64, device="cuda"))


# ------------------------------------------------------------------------------------- how they are called
def test_other_stream_and_two_graphs_on_one_workspace():
    """Calls on a side stream, and two captured graphs that share a workspace, replayed with new inputs."""
    _, x, w, xq, sx, wq, sw = linear_operands(21, 40, 256, 384)
    ws = L.workspace(1 << 20)
    side = torch.cuda.Stream()
    want, got = nans(40, 256), nans(40, 256)
    L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, want, ws=ws)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, got, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, got.zero_(), ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    dy, xt, sxt = make(np.random.default_rng(1), (40, 256)), bytes_(384, 48), nans(1, 384)
    wt = bytes_(384, 256)
    L.mmdit_fp8_block_cast(w, s=sw, q_t=wt, square=True)
    y, dx, dw = nans(40, 256), nans(40, 384, dtype=torch.bfloat16), nans(256, 384)

    def forward():
        L.mmdit_fp8_block_cast(x, xq, sx, q_t=xt, s_t=sxt)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, y, ws=ws)

    def backward():
        L.mmdit_fp8_block_linear_bwd(dy, wt, sw, xt, sxt, dx=dx, dw=dw, ws=ws)

    graphs = []
    for f in (forward, backward):
        f()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(1))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    r = [t.clone() for t in (y, dx, dw)]
    for t in (y, dx, dw):
        t.fill_(float("nan"))
    forward()
    backward()
    assert all(torch.equal(a, b) for a, b in zip(r, (y, dx, dw)))
    assert L.mmdit_workspace_status(ws) == 0


def test_workspace_of_a_call_on_another_stream():
    """A workspace that the binding makes belongs to the call's stream: its zeros are written before the call,
    not whenever the current stream comes to them."""
    dy = make(np.random.default_rng(5), (200, 256))
    side, db = torch.cuda.Stream(), nans(256)
    for stream in (side, side.cuda_stream, 0):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        ws = L.mmdit_fp8_block_linear_bwd(dy, db=db, stream=stream)
        torch.cuda.synchronize()
        assert ws.count_nonzero() > 256  # the partial sums of db
        check(f64(db), f64(dy).sum(0), 208 * U * np.abs(f64(dy)).sum(0), "db")


def test_binding_refusals():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    g = x[0].clone()
    with pytest.raises(ValueError, match="shape"):
        L.mmdit_add_rmsnorm_fwd(x, g[:32].clone(), y=x.clone())
    with pytest.raises(TypeError, match="residual"):
        L.mmdit_add_rmsnorm_fwd(x, g, residual=x.half(), y=x.clone())
    with pytest.raises(TypeError, match="dtype"):
        L.mmdit_add_rmsnorm_fwd(x.half(), g, y=x.clone())
    with pytest.raises(ValueError, match="cpu"):
        L.mmdit_add_rmsnorm_fwd(x, g.cpu(), y=x.clone())
    with pytest.raises(L.MMDitError, match="alias"):
        L.mmdit_add_rmsnorm_fwd(x, g, y=x)
    with pytest.raises(ValueError, match="contiguous"):
        L.mmdit_fp8_block_cast(x.t().contiguous().t(), bytes_(4, 64), nans(1, 4))
    with pytest.raises(ValueError, match="shape"):
        L.mmdit_fp8_block_cast(x, bytes_(4, 64), nans(4, 1))
    q = torch.zeros(1, 4, 2, 64, device="cuda")
    with pytest.raises(TypeError, match="int64"):
        L.mmdit_rope_fwd(L.make_rope_cfg(64), q, q, positions=torch.arange(4, device="cuda", dtype=torch.int32))
    with pytest.raises(ValueError, match="positions"):
        L.mmdit_rope_fwd(L.make_rope_cfg(64), q, q, positions=torch.arange(5, device="cuda"))
    with pytest.raises(ValueError, match="adjacent"):
        L.mmdit_rope_fwd(L.make_rope_cfg(64), q.transpose(2, 3).contiguous().transpose(2, 3), q, positions=torch.arange(4, device="cuda"))
    with pytest.raises(L.MMDitError, match="strides"):
        L.mmdit_rope_fwd(L.make_rope_cfg(64), q, q.view(1, 2, 4, 64).transpose(1, 2), positions=torch.arange(4, device="cuda"))


def test_layer_of_a_text_model():
    """The operators as a layer uses them: residual + norm to codes, the q|k|v linear on them, rotary
    positions straight into the attention's head-major layout, the attention, its output cast and
    projected, and the next norm; each stage checked from what the GPU handed to it."""
    B, S, H, d = 1, 160, 2, 128
    D, rng = H * d, np.random.default_rng(77)
    x, res, gain = make(rng, (B * S, D)), make(rng, (B * S, D), torch.float32, 2.0), make(rng, (D,), scale=0.1) + 1
    w_qkv, w_o = make(rng, (3 * D, D), scale=D ** -0.5), make(rng, (D, D), scale=D ** -0.5)
    codes = {}
    for name, w in (("qkv", w_qkv), ("o", w_o)):
        codes[name] = bytes_(*w.shape), nans(tiles(w.shape[0]), tiles(D))
        L.mmdit_fp8_block_cast(w, *codes[name], square=True)
    h, q8, s8 = nans(B * S, D), bytes_(B * S, D), nans(tiles(D), B * S)
    L.mmdit_add_rmsnorm_fwd(x, gain, residual=res, h=h, y_q=q8, s_y=s8)
    qkv = nans(B * S, 3 * D, dtype=torch.bfloat16)
    ws = L.mmdit_fp8_block_linear_fwd(q8, s8, *codes["qkv"], None, qkv)
    q, k, v = (t.unflatten(-1, (H, d)).unflatten(0, (B, S)) for t in qkv.split(D, dim=-1))
    qh, kh = nans(B, H, S, d, dtype=torch.bfloat16), nans(B, H, S, d, dtype=torch.bfloat16)
    cfg = L.make_rope_cfg(d, theta=10000.0, interleaved=False)
    L.mmdit_rope_fwd(cfg, q, qh.transpose(1, 2), k=k, k_out=kh.transpose(1, 2), positions=torch.arange(S, device="cuda"))
    vh = v.transpose(1, 2).contiguous()
    o = nans(B, S, D, dtype=torch.bfloat16)
    L.mmdit_attention_fwd(qh, kh, vh, o)
    o2 = o.view(B * S, D)
    oq, so = bytes_(B * S, D), nans(tiles(D), B * S)
    L.mmdit_fp8_block_cast(o2, oq, so)
    proj = nans(B * S, D, dtype=torch.bfloat16)
    L.mmdit_fp8_block_linear_fwd(oq, so, *codes["o"], None, proj, ws=ws)
    h2, y2 = nans(B * S, D), nans(B * S, D, dtype=torch.bfloat16)
    L.mmdit_add_rmsnorm_fwd(proj, gain, residual=h, h=h2, y=y2)
    assert L.mmdit_workspace_status(ws) == 0
    # stage by stage
    n = lambda t: t.cpu().numpy()  # noqa: E731
    assert torch.equal(h, x.float() + res)
    yo, _ = lm.rmsnorm(f64(h), f64(gain), 1e-6)
    y8 = lm.values_rows(n(q8), n(s8))
    check(y8, yo, np.maximum(2.0 ** -4 * np.abs(yo), 2.0 ** -10 / np.repeat(f64(s8).T, 128, 1)) + 300 * U * np.abs(yo), "norm")
    wv = lm.values_square(*map(n, codes["qkv"]))
    ref = y8 @ wv.T
    check(f64(qkv), ref, sum_tol(y8, wv, tiles(D)) + 2.0 ** -8 * np.abs(ref), "qkv")
    cos, sin = lm.rope_cos_sin(np.arange(S)[None], lm.rope_frequencies(d))
    rope_check(qh.transpose(1, 2), q, cos, sin, d, False, 1.0, False, "bf16")
    rope_check(kh.transpose(1, 2), k, cos, sin, d, False, 1.0, False, "bf16")
    sc = f64(qh) @ f64(kh).swapaxes(-1, -2) / np.sqrt(d)
    p = np.exp(sc - sc.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ao = (p @ f64(vh)).transpose(0, 2, 1, 3).reshape(B * S, D)
    # the attention's own bar: 2e-2 of the output's root mean square beyond the bf16 rounding
    check(f64(o2), ao, 2e-2 * np.sqrt((ao ** 2).mean()) + 2.0 ** -8 * np.abs(ao), "attention")
    ov, wo = lm.values_rows(n(oq), n(so)), lm.values_square(*map(n, codes["o"]))
    ref = ov @ wo.T
    check(f64(proj), ref, sum_tol(ov, wo, tiles(D)) + 2.0 ** -8 * np.abs(ref), "projection")
    assert torch.equal(h2, proj.float() + h)
    yo, _ = lm.rmsnorm(f64(h2), f64(gain), 1e-6)
    check(f64(y2), yo, (2.0 ** -8 + 300 * U) * np.abs(yo), "second norm")


@pytest.mark.parametrize("scaling", ["none", "linear", "by_parts"])
@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 24) + 1, 1 << 31, (1 << 40) + 7, -(1 << 40) - 7])
def test_rope_against_exact_frequencies(scaling, start):
    """Far positions against angles without a double's rounding: the bound that the header states, in radians, on
    top of the rotation's own."""
    kw = dict(theta=500000.0, scaling=scaling, factor=16.0, orig_len=8192.0, low=1.0, high=32.0)
    rot, S = 64, 5
    pos = start + torch.arange(S)
    x = make(np.random.default_rng(4), (1, S, 2, rot), torch.float32)
    out = nans(1, S, 2, rot)
    L.mmdit_rope_fwd(L.make_rope_cfg(rot, interleaved=False, **kw), x, out, positions=pos.cuda())
    turns = lm.rope_turns_exact(rot, **kw)
    cos, sin = lm.rope_cos_sin_exact(pos.numpy()[None], turns)
    ref = lm.rope(f64(x), cos, sin, rot, False)
    steps = 16.0 * (5 * 32 / 31 + 3) + 8 if scaling == "by_parts" else 5.0
    f = np.array([float(t) for t in turns])
    angle = 2 * np.pi * np.abs(pos.numpy())[:, None] * (f * steps * 2.0 ** -53 + 2.0 ** -64)
    pair = np.abs(f64(x))[..., :rot // 2] + np.abs(f64(x))[..., rot // 2:]
    tol = (16 * U + angle)[None, :, None, :] * pair
    check(f64(out), ref, U * np.abs(ref) + np.concatenate([tol, tol], -1), "rotated")


@pytest.mark.parametrize("rows,dim", [(5003, 512), (5003, 264), (2500, 2048), (1300, 4096), (700, 5120), (700, 6152),
                                      (701, 8192), (650, 8200)])
@pytest.mark.parametrize("act,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_norm_gradients_over_many_rows(rows, dim, act, res):
    """More rows than the launch has places: a CTA walks several (short ones in groups, the last group partly past the
    end), with the next row's operands on their way, and in place."""
    rng = np.random.default_rng(rows + dim)
    dt, rt = DT[act], DT[res]
    h, dy = make(rng, (rows, dim), rt, 3.0), make(rng, (rows, dim), dt)
    gain, dh_in = (1 + 0.2 * make(rng, (dim,), torch.float32)).to(dt), make(rng, (rows, dim), rt)
    h[1] = 0
    r32 = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dho, dgo = lm.rmsnorm_bwd(f64(dy), f64(h), f64(gain), 1e-6, f64(dh_in))
    r = f64(r32)[:, None]
    n, a = f64(h) * r, f64(dy) * f64(gain)
    # r is half a step off; the row's sum dim u of its magnitudes; ten roundings beside, and the stored type's
    big = r * (np.abs(a) + np.abs(n) * (np.abs(a * n)).mean(1, keepdims=True))
    tol = (dim + 16) * U * big + (HALF[rt] + 2 * U) * np.abs(dho)
    dh, dg, dx = nans(rows, dim, dtype=rt), nans(dim), nans(rows, dim, dtype=dt)
    ws = L.mmdit_add_rmsnorm_bwd(dy, h, gain, r32, dh, dh_in=dh_in, dx=dx, dgain=dg)
    check(f64(dh), dho, tol, "dh")
    check(f64(dx), dho, tol + HALF[dt] * np.abs(dho), "dx")
    check(f64(dg), dgo, (rows + 16) * U * np.abs(f64(dy) * n).sum(0) + U * np.abs(dgo), "dgain")
    here, again = dh_in.clone(), nans(dim)
    L.mmdit_add_rmsnorm_bwd(dy, h, gain, r32, here, dh_in=here, dgain=again, ws=ws)
    assert torch.equal(here, dh) and torch.equal(again, dg)
    assert L.mmdit_workspace_status(ws) == 0


def test_norm_repeats_itself_and_codes_part_at_borders_alone():
    """A prompt's norm gives the same bits again after other calls; a code is the nearest one of the float64 value, or
    its neighbour where that value lies within the row sum's error of the border between them."""
    rng = np.random.default_rng(12)
    rows, dim = 4608, 4096
    x, res, gain = make(rng, (rows, dim)), make(rng, (rows, dim), torch.float32, 3.0), (1 + 0.2 * make(rng, (dim,), torch.float32)).bfloat16()
    first = None
    for _ in range(4):
        h, q, s, r = nans(rows, dim), bytes_(rows, dim), nans(tiles(dim), rows), nans(rows)
        L.mmdit_add_rmsnorm_fwd(x, gain, residual=res, h=h, y_q=q, s_y=s, rstd=r)
        L.mmdit_add_rmsnorm_fwd(x.flip(0), gain, residual=res, h=nans(rows, dim), y_q=bytes_(rows, dim), s_y=nans(tiles(dim), rows))
        first = first or (h, q, s, r)
        assert all(torch.equal(a, b) for a, b in zip(first, (h, q, s, r)))
    some = slice(0, rows, 97)
    yo, _ = lm.rmsnorm(f64(first[0][some]), f64(gain), 1e-6)
    v = yo * np.repeat(f64(first[2][:, some]).T, 128, 1)
    got, off = lm.decode(first[1][some].cpu().numpy()), (dim + 8 + 8) * U
    assert (np.abs(got) >= np.abs(lm.decode(lm.encode(v * (1 - off))))).all()
    assert (np.abs(got) <= np.abs(lm.decode(lm.encode(v * (1 + off))))).all()
    assert (np.signbit(got) == np.signbit(v)).all()  # negative values below half a step become -0


@pytest.mark.parametrize("M,N,K", [
    (48, 136, 14336), (64, 264, 20496),                # 64 columns, K on eight CTAs: 14 and 21 slices each
    (40, 5000, 4112), (64, 9800, 2576), (33, 19600, 1040),   # on four, two and one: 9, 11 and 9 slices
    (24, 5000, 8208), (17, 9800, 5136), (20, 19600, 2064),   # the same with 32 columns
    (7700, 8, 272), (7700, 24, 272), (7700, 56, 144), (7700, 40, 16),  # outputs narrower than a stored box
    (7700, 24, 2064), (7940, 264, 2064), (2090, 2568, 1040),  # two pairs to a narrow tile; 9 slices to each of many tiles
])
def test_linear_walks_and_narrow_outputs(M, N, K):
    """Shapes whose rings, product buffers and factor windows come round inside a tile, and outputs of fewer columns
    than the kernel stores at once, with guard rows around them."""
    rng, x, w, xq, sx, wq, sw = linear_operands(M + N * 3 + K, M, N, K)
    b = make(rng, (N,))
    xv = lm.values_rows(xq.cpu().numpy(), sx.cpu().numpy())
    wv = lm.values_square(wq.cpu().numpy(), sw.cpu().numpy())
    r = xv @ wv.T + f64(b)
    t = sum_tol(xv, wv, tiles(K)) + 2 * U * np.abs(r)
    ws = L.workspace(256)
    for dtype in (torch.float32, torch.bfloat16):
        pad = torch.full((M + 16, N), 7.0, device="cuda", dtype=dtype)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, b, pad[8:M + 8], ws=ws)
        check(f64(pad[8:M + 8]), r, t + (HALF[dtype] * np.abs(r) + 2.0 ** -8 * t if dtype is torch.bfloat16 else 0), str(dtype))
        assert (pad[:8] == 7).all() and (pad[M + 8:] == 7).all()
        again = torch.empty_like(pad)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, b, again[8:M + 8], ws=ws)
        assert torch.equal(again[8:M + 8], pad[8:M + 8])
    assert L.mmdit_workspace_status(ws) == 0


@pytest.mark.parametrize("M,N,K", [(9000, 136, 128), (20000, 40, 144), (9000, 24, 272),  # dW on few tiles: 9 to 20 slices a CTA
                                   (1000, 2568, 2576)])                                   # more tiles than pairs, of 8 slices
def test_linear_gradients_of_many_rows(M, N, K):
    rng, x, w, _, _, wq, sw = linear_operands(M + N * 5 + K, M, N, K)
    ldm, ldn = (M + 15) // 16 * 16, (N + 15) // 16 * 16
    dy = make(rng, (M, N), scale=1e-3)
    wt, xt, sxt = bytes_(K, ldn), bytes_(K, ldm), nans(tiles(M), K)
    L.mmdit_fp8_block_cast(w, s=sw, q_t=wt, square=True)
    L.mmdit_fp8_block_cast(x, q_t=xt, s_t=sxt)
    wqc, swc, xtc, sxtc = (t.cpu().numpy() for t in (wq, sw, xt, sxt))
    g, gt = lm.values_rows(*lm.cast_rows(f64(dy))), lm.values_rows(*lm.cast_rows(f64(dy).T))
    wv, xv = lm.values_square(wqc, swc), lm.values_rows(xtc[:, :M], sxtc)
    dxo, dwo, dbo = g @ wv, gt @ xv.T, f64(dy).sum(0)
    dx, dw, db = nans(M, K, dtype=torch.bfloat16), nans(N, K), nans(N)
    ws = L.mmdit_fp8_block_linear_bwd(dy, wt, sw, xt, sxt, dx=dx, dw=dw, db=db)
    check(f64(dx), dxo, sum_tol(g, wv.T, tiles(N)) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(dxo), "dx")
    check(f64(dw), dwo, sum_tol(gt, xv, tiles(M)), "dw")
    check(f64(db), dbo, (M + 8) * U * np.abs(f64(dy)).sum(0), "db")
    again = nans(N, K)
    L.mmdit_fp8_block_linear_bwd(dy, x_t=xt, s_xt=sxt, dw=again, ws=ws)
    assert torch.equal(again, dw)
    assert L.mmdit_workspace_status(ws) == 0


def test_linear_gradient_against_differences_within_the_casts_roundings():
    """The slope of <y, dy> along directions in which it is large: the whole gradient's, and those of single quarters
    of the rows, which a dW that leaves rows out would miss.  The casts' errors e are independent roundings, each at
    most 2^-4 of its value (2^-10 of the code's unit below the normal range), that enter as
    sum e_x (dy d) + sum e_dy (x d^T) + sum e_dy d e_x: sums of independent terms of bounds c stay below
    6 sqrt(sum c^2) but for one time in 10^7."""
    M, N, K = 256, 128, 128
    rng, x, w, _, _, _, _ = linear_operands(9, M, N, K)
    dy = make(rng, (M, N))
    xt, sxt, dw = bytes_(K, M), nans(2, K), nans(N, K)
    L.mmdit_fp8_block_cast(x, q_t=xt, s_t=sxt)
    L.mmdit_fp8_block_linear_bwd(dy, x_t=xt, s_xt=sxt, dw=dw)
    X, D, W, e = f64(x), f64(dy), f64(w), 1e-3

    def error(v):  # of the codes of v's columns in tiles of 128 rows
        amax = np.abs(v).reshape(2, 128, -1).max(1)
        return np.maximum(2.0 ** -4 * np.abs(v), np.repeat(2.0 ** -10 * amax / 448, 128, 0))

    ex, ed = error(X), error(D)
    parts = [slice(0, M)] + [slice(64 * i, 64 * i + 64) for i in range(4)]
    for p in parts:
        d = D[p].T @ X[p] / 16 + 0.1 * rng.standard_normal((N, K))
        loss = lambda t: float(((X @ (W + t * d).T) * D).sum())  # noqa: E731
        slope = (loss(e) - loss(-e)) / (2 * e)
        bar = 6 * np.sqrt((ex ** 2 * (D @ d) ** 2).sum() + (ed ** 2 * (X @ d.T) ** 2).sum() + ((ed ** 2 @ d ** 2) * ex ** 2).sum())
        assert abs(slope) > 8 * bar
        assert abs(float((f64(dw) * d).sum()) - slope) <= bar


@pytest.mark.parametrize("B,S,Hq,Hk,d,rot,inter,act", [
    (5, 1003, 2, 1, 64, 64, False, "bf16"),   # eight tokens to a CTA, the last one's partly behind the sequence
    (5, 1003, 2, 1, 64, 64, True, "bf16"),
    (3, 1537, 1, 1, 96, 20, True, "f32"),
    (3, 1537, 1, 1, 96, 20, False, "f32"),
    (2, 1001, 1, 1, 80, 38, False, "bf16"),
    (1, 3, 70, 10, 256, 256, True, "bf16"),   # more heads than a CTA holds at a time
    (1, 3, 70, 10, 256, 256, False, "bf16"),
    (1, 2, 300, 30, 128, 64, True, "f32"),
])
def test_rope_of_token_groups_and_many_heads(B, S, Hq, Hk, d, rot, inter, act):
    cfg, q, k, pos, (qo, ko), cos, sin = rope_case(B + S + d, B, S, Hq, Hk, d, rot, inter, act, start=3)
    guard = torch.full((B * S * Hq * d + 64,), 7.0, device="cuda", dtype=DT[act])
    qo = guard[:-64].view(B, S, Hq, d)
    L.mmdit_rope_fwd(cfg, q, qo, k=k, k_out=ko, positions=pos)
    rope_check(qo, q, cos, sin, rot, inter, 1.0, False, act)
    rope_check(ko, k, cos, sin, rot, inter, 1.0, False, act)
    assert (guard[-64:] == 7).all()


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("act,d,rot", [("bf16", 128, 128), ("bf16", 80, 20), ("f32", 96, 48), ("f32", 40, 38)])
def test_rope_in_place_on_a_packed_projection(inter, act, d, rot):
    """q and k rotated where they lie between each other and v, forward and by tables, then turned back."""
    B, S, Hq, Hk = 2, 130, 6, 2
    cfg, q, k, pos, (qo, ko), cos, sin = rope_case(d, B, S, Hq, Hk, d, rot, inter, act, start=70)
    L.mmdit_rope_fwd(cfg, q, qo, k=k, k_out=ko, positions=pos)
    packed = q._base if q._base is not None else q
    packed = packed.view(B, S, (Hq + 2 * Hk) * d)
    before = packed.clone()
    L.mmdit_rope_fwd(cfg, q, q, k=k, k_out=k, positions=pos)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(packed[..., (Hq + Hk) * d:], before[..., (Hq + Hk) * d:])
    packed.copy_(before)
    c32, s32 = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (cos, sin))
    L.mmdit_rope_fwd(cfg, q, q, k=k, k_out=k, cos=c32, sin=s32)
    x = before[..., :Hq * d].unflatten(-1, (Hq, d))
    rope_check(q, x, f64(c32), f64(s32), rot, inter, 1.0, False, act)
    turned, kt = q.clone(), k.clone()
    L.mmdit_rope_bwd(cfg, q, q, k=k, k_out=k, cos=c32, sin=s32)
    rope_check(q, turned, f64(c32), f64(s32), rot, inter, 1.0, True, act)
    rope_check(k, kt, f64(c32), f64(s32), rot, inter, 1.0, True, act)


def test_rope_of_k_alone():
    cfg, q, k, pos, (_, ko), cos, sin = rope_case(3, 2, 9, 3, 2, 64, 64, True, "bf16")
    none = q[:, :, :0]
    L.mmdit_rope_fwd(cfg, none, none, k=k, k_out=ko, positions=pos)
    rope_check(ko, k, cos, sin, 64, True, 1.0, False, "bf16")


def test_two_streams_at_once():
    """Every operator on two streams side by side, each with its own workspace and outputs: the bits of the calls one
    after another."""
    M, N, K = 2100, 2568, 1360
    rng, x, w, xq, sx, wq, sw = linear_operands(31, M, N, K)
    dy, gain = make(rng, (M, N), scale=1e-3), make(rng, (K,))
    wt, xt, sxt = bytes_(K, (N + 15) // 16 * 16), bytes_(K, (M + 15) // 16 * 16), nans(tiles(M), K)
    L.mmdit_fp8_block_cast(w, s=sw, q_t=wt, square=True)
    L.mmdit_fp8_block_cast(x, q_t=xt, s_t=sxt)
    heads, pos = x[:, :1344].reshape(1, M, 21, 64), torch.arange(M, device="cuda")
    cfg, nbytes = L.make_rope_cfg(64), L.mmdit_fp8_block_linear_bwd_workspace_size(M, N, K)

    def buffers():
        b16 = lambda *s: nans(*s, dtype=torch.bfloat16)  # noqa: E731
        return dict(y=b16(M, N), y48=b16(48, N), y1=b16(1, N), dx=b16(M, K), dw=nans(N, K), db=nans(N), n=b16(M, K), r=nans(M),
                    dh=b16(M, K), dg=nans(K), q=bytes_(M, K), s=nans(tiles(K), M), turned=b16(1, M, 21, 64)), L.workspace(nbytes)

    s48, s1 = sx[:, :48].contiguous(), sx[:, :1].contiguous()

    def calls(o, ws):
        L.mmdit_add_rmsnorm_fwd(x, gain, y=o["n"], rstd=o["r"])
        L.mmdit_fp8_block_cast(x, o["q"], o["s"])
        L.mmdit_fp8_block_linear_fwd(xq[:48], s48, wq, sw, None, o["y48"], ws=ws)
        L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, None, o["y"], ws=ws)
        L.mmdit_fp8_block_linear_fwd(xq[:1], s1, wq, sw, None, o["y1"], ws=ws)
        L.mmdit_rope_fwd(cfg, heads, o["turned"], positions=pos)
        L.mmdit_fp8_block_linear_bwd(dy, wt, sw, xt, sxt, dx=o["dx"], dw=o["dw"], db=o["db"], ws=ws)
        L.mmdit_add_rmsnorm_bwd(x, x, gain, o["r"], o["dh"], dgain=o["dg"], ws=ws)

    want, ws = buffers()
    calls(want, ws)
    torch.cuda.synchronize()
    sides = [(torch.cuda.Stream(), *buffers()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(6):
        for stream, o, w_ in sides:
            with torch.cuda.stream(stream):
                calls(o, w_)
    torch.cuda.synchronize()
    for _, o, w_ in sides:
        assert all(torch.equal(o[n], want[n]) for n in want)
        assert L.mmdit_workspace_status(w_) == 0


def linear_times(M, K, widths):
    """GPU time of one call for each N: the shortest of 60 replays of 20 captured calls, so that nothing else on the
    machine counts."""
    xq, sx = torch.randint(0, 120, (M, K), device="cuda", dtype=torch.uint8), torch.ones(tiles(K), M, device="cuda")
    times = []
    for N in widths:
        w, sw = torch.randint(0, 120, (N, K), device="cuda", dtype=torch.uint8), torch.ones(tiles(N), tiles(K), device="cuda")
        y, ws = nans(M, N, dtype=torch.bfloat16), L.workspace(256)
        call = lambda: L.mmdit_fp8_block_linear_fwd(xq, sx, w, sw, None, y, ws=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        g, took = torch.cuda.CUDAGraph(), []
        with torch.cuda.graph(g):
            for _ in range(20):
                call()
        for _ in range(60):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            took.append(a.elapsed_time(b) / 20)
        times.append(min(took))
    return times


def test_two_pairs_to_a_tile_only_where_all_have_a_place():
    """Past the clusters of two pairs that fit at once, a tile more would wait for a second turn of the whole launch
    (1.8 times the time); one pair to a tile takes 1.1 times the time of the split tiles."""
    times = linear_times(256, 2048, range(256 * 32, 256 * 41, 256))
    assert max(b / a for a, b in zip(times, times[1:])) < 1.5, times


def test_k_on_eight_ctas_only_where_all_clusters_have_a_place():
    """Few rows: K goes to clusters of eight CTAs while all of them fit at once; one more would cost a second turn of
    the launch (1.4 times the time), clusters of four take no longer."""
    times = linear_times(64, 2048, range(128 * 32, 128 * 42, 128))
    assert max(b / a for a, b in zip(times, times[1:])) < 1.2, times


FIRST_CALLS = """
import torch
from diffusion_transformer_flux_gb300 import _lib as L
t = lambda n: (n + 127) // 128
codes = lambda *s: torch.randint(0, 120, s, device="cuda", dtype=torch.uint8)
ones, ws = lambda *s: torch.ones(*s, device="cuda"), L.workspace(64 << 20)
todo = []
for M, N, K in ((1, 1024, 1024), (48, 4096, 4096), (1024, 4096, 1024), (512, 4096, 4096)):
    x, sx, w, sw, y = codes(M, K), ones(t(K), M), codes(N, K), ones(t(N), t(K)), torch.zeros(M, N, device="cuda")
    todo.append((y, lambda x=x, sx=sx, w=w, sw=sw, y=y: L.mmdit_fp8_block_linear_fwd(x, sx, w, sw, None, y, ws=ws)))
M, N, K = 1000, 1024, 2048
dy, wt, sw, xt, sxt = torch.randn(M, N, device="cuda").bfloat16(), codes(K, N), ones(t(N), t(K)), codes(K, 1008), ones(t(M), K)
dw, dx = torch.zeros(N, K, device="cuda"), torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
todo.append((dw, lambda: L.mmdit_fp8_block_linear_bwd(dy, wt, sw, xt, sxt, dx=dx, dw=dw, ws=ws)))
h, gain = torch.randn(100, 4096, device="cuda").bfloat16(), torch.ones(4096, device="cuda", dtype=torch.bfloat16)
n, r, dh = torch.zeros_like(h), torch.ones(100, device="cuda"), torch.zeros_like(h)
todo.append((n, lambda: L.mmdit_add_rmsnorm_fwd(h, gain, y=n)))
todo.append((dh, lambda: L.mmdit_add_rmsnorm_bwd(h, h, gain, r, dh, ws=ws)))
q, pos, cfg = torch.randn(2, 100, 4, 64, device="cuda"), torch.arange(100, device="cuda"), L.make_rope_cfg(64)
o = torch.zeros_like(q)
todo.append((o, lambda: L.mmdit_rope_fwd(cfg, q, o, positions=pos)))
torch.cuda.synchronize()
for i, (out, call) in enumerate(todo):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    first = out.clone()
    out.zero_()
    call()
    assert first.count_nonzero() and torch.equal(first, out), i
assert L.mmdit_workspace_status(ws) == 0
"""


def test_first_call_of_a_process_inside_a_capture():
    """What a call asks of the device once (kernel sizes, places of clusters) may be asked while a graph is captured."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
