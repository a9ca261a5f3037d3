"""GPU parity of the attention of a text model against the float64 oracle (oracle.lm): packed sequences, paged caches,
their block tables and writes.

Tolerances count roundings.  u = 2^-24 is half a float32 step; a value rounded to bf16 is off by 2^-8 of itself.  A score
z = scale q . k is a float32 sum of d exact products, off by at most 2 d u scale |q| . |k| (2: a tensor core may cut instead
of rounding), its exponential by 2^-21 beside that and 4 u |z - max| of its argument.
"""
import numpy as np
import pytest
import torch

from diffusion_transformer_flux_gb300 import _lib as L
from oracle import lm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
B16 = torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def sums(n):
    return np.concatenate(([0], np.cumsum(n))).tolist()


def rand(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(B16)


def check(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = np.isneginf(got) & np.isneginf(ref)
    odd = np.argwhere(~(np.isfinite(got) | same))[:4].tolist()
    assert not odd, f"{what}: not finite at {odd}"
    with np.errstate(invalid="ignore"):
        err = np.where(same, 0.0, np.abs(got - ref) - tol)
    if err.size:
        assert err.max() <= 0, f"{what}: {err.max():.3e} over its bound at {np.unravel_index(err.argmax(), err.shape)}"


def weight_error(q, k, scale, causal):
    """A bound on the relative error of any weight of each row, [n, Hq]: its score's and that of the row's maximum."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    see = lm.seen(n, k.shape[0], causal)
    z = np.einsum("ihd,jhd->ihj", np.abs(q), np.repeat(np.abs(k), group, 1)) * scale
    z = np.where(see[:, None, :], z, 0.0).max(-1, initial=0.0)
    return 2 * ((2 * d + 8) * U * z + 2.0 ** -21)


def attention_reference(q, k, v, causal, scale=None):
    """(out, lse, bound of out, bound of lse) of one sequence in float64."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse = lm.attention(q, k, v, scale, causal)
    mean, _ = lm.attention(q, k, np.abs(v), scale, causal)
    w, m = weight_error(q, k, scale, causal), k.shape[0]
    # each weight is rounded to bf16 for the second product; sums of m terms; the result is rounded to bf16
    tol = (2.0 ** -8 + 2 * w[:, :, None] + (2 * m + 16) * U) * mean * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out)
    return out, lse, tol, w + (m + 16) * U + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def packed(rng, nq, nk, hq, hk, d, layout="packed", pad=0, spread=2.0):
    """q, k, v of sequences with `pad` rows of NaN behind the last one, and cu_q, cu_k."""
    tq, tk = sum(nq) + pad, sum(nk) + pad

    def heads(rows, h, scale=1.0):
        return rand(rng, rows, h, d, scale=scale)

    q, k, v = heads(tq, hq, spread), heads(tk, hk), heads(tk, hk)
    if pad:
        for t in (q, k, v):
            t[-pad:] = float("nan")
    if layout == "head_major":
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    elif layout == "packed":  # views of wider rows
        q, k, v = (torch.cat((t, torch.full_like(t, float("nan"))), 1)[:, : t.shape[1]] for t in (q, k, v))
    return q, k, v, ints(sums(nq)), ints(sums(nk))


def run_varlen(q, k, v, cu_q, cu_k, causal, scale=None, lse=True, out=None, ws=None):
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format) if out is None else out
    sums_ = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    ws = L.mmdit_varlen_attention_fwd(q, k, v, out, cu_q, cu_k=cu_k, lse=sums_, causal=causal, scale=scale, ws=ws)
    torch.cuda.synchronize()
    assert L.mmdit_workspace_status(ws) == 0
    return out, sums_


def compare_varlen(q, k, v, cu_q, cu_k, causal, scale=None):
    out, lse = run_varlen(q, k, v, cu_q, cu_k, causal, scale)
    a, b = cu_q.tolist(), cu_k.tolist()
    for i in range(len(a) - 1):
        x, y = slice(a[i], a[i + 1]), slice(b[i], b[i + 1])
        ref, rl, tol, tl = attention_reference(f64(q[x]), f64(k[y]), f64(v[y]), causal, scale)
        check(f64(out[x]), ref, tol, f"out of sequence {i}")
        check(f64(lse[x]), rl, tl, f"lse of sequence {i}")
    # rows of no sequence are left as they were
    assert (out[a[-1]:] == 7).all() and (lse[a[-1]:] == 7).all()
    return out, lse


LENGTHS = {
    "one": ([1], [1]), "one_far": ([1], [130]), "tile": ([128], [128]), "odd": ([129], [129]), "three_tiles": ([257], [300]),
    "ragged": ([5, 0, 70, 1, 131, 33], [5, 9, 70, 200, 131, 33]), "no_keys": ([3, 40, 2], [0, 40, 0]), "all_empty": ([0, 0], [0, 0]),
    "more_queries": ([70, 140], [3, 130]),  # rows before the first key see nothing
    "many": ([7] * 40, [7] * 40),
}


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (2, 2, 64), (5, 1, 96)])
def test_varlen(lengths, causal, hq, hk, d):
    nq, nk = LENGTHS[lengths]
    rng = np.random.default_rng(len(lengths) + 31 * d + causal)
    compare_varlen(*packed(rng, nq, nk, hq, hk, d, pad=3), causal)


@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 3), (7, 1), (16, 1), (48, 1), (128, 1), (14, 2)])
def test_varlen_groups(hq, hk):
    rng = np.random.default_rng(hq)
    compare_varlen(*packed(rng, [9, 37], [40, 37], hq, hk, 64, pad=1), True)


@pytest.mark.parametrize("d", [8, 16, 40, 56, 64, 72, 80, 120, 128])
@pytest.mark.parametrize("layout", ["dense", "packed", "head_major"])
def test_varlen_head_dims_and_layouts(d, layout):
    rng = np.random.default_rng(d)
    compare_varlen(*packed(rng, [131], [131], 4, 2, d, layout=layout, pad=2), True)


def test_varlen_output_view():
    """A strided output: rows of a wider tensor, heads first."""
    rng = np.random.default_rng(5)
    q, k, v, cu, _ = packed(rng, [50, 90], [50, 90], 4, 2, 96)
    whole = torch.full((6, 140, 104), 7.0, device="cuda", dtype=B16)
    out = whole[1:5, :, :96].transpose(0, 1)
    run_varlen(q, k, v, cu, cu, True, out=out)
    ref, _ = run_varlen(q, k, v, cu, cu, True)
    assert torch.equal(out, ref)
    assert (whole[0] == 7).all() and (whole[5] == 7).all() and (whole[:, :, 96:] == 7).all()


def test_varlen_long_rows_and_maxima_that_move():
    """Scores that rise along the keys make every tile's maximum larger than the last one's."""
    rng = np.random.default_rng(11)
    q, k, v, cu, _ = packed(rng, [900], [900], 2, 1, 128, layout="dense")
    q[:] = 1.0
    k *= 0.1
    k += (torch.arange(900, device="cuda") / 90).to(B16)[:, None, None]
    compare_varlen(q, k, v, cu, cu, True)
    compare_varlen(q, -k, v, cu, cu, False)


@pytest.mark.parametrize("scale", [1e-6, 0.25, 4.0])
def test_varlen_scales(scale):
    rng = np.random.default_rng(12)
    compare_varlen(*packed(rng, [140], [140], 2, 2, 64), True, scale=scale)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_varlen_masked_places_hold_anything(bad, d):
    """Keys and values of later tokens, of other sequences and behind the last one do not reach a row."""
    rng = np.random.default_rng(13)
    q, k, v, cu, _ = packed(rng, [100, 200], [100, 200], 4, 2, d, layout="dense")
    ref, ref_lse = run_varlen(q, k, v, cu, cu, True)
    for at in (0, 57, 99, 100, 170, 299):
        k2, v2 = k.clone(), v.clone()
        k2[at], v2[at] = bad, bad
        out, lse = run_varlen(q, k2, v2, cu, cu, True)
        rows = torch.arange(300, device="cuda")
        clean = (rows < at) | ((rows >= 100) if at < 100 else (rows < 100))
        assert torch.equal(out[clean], ref[clean]) and torch.equal(lse[clean], ref_lse[clean])
    # a value alone: the rows that see it are not finite in its column, the other columns are as they were
    v2 = v.clone()
    v2[150, 1, 5] = bad
    out, lse = run_varlen(q, k, v2, cu, cu, True)
    assert torch.equal(lse, ref_lse)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[150:, 2:, 5] = True
    assert torch.equal(out[~hit], ref[~hit]) and not torch.isfinite(out[hit]).any()


def test_varlen_rows_that_are_not_finite_stay_alone():
    rng = np.random.default_rng(14)
    q, k, v, cu, _ = packed(rng, [150], [150], 4, 1, 128, layout="dense")
    ref, _ = run_varlen(q, k, v, cu, cu, True)
    q[40, 2] = float("nan")
    out, lse = run_varlen(q, k, v, cu, cu, True)
    assert torch.isnan(out[40, 2]).all() and torch.isnan(lse[40, 2])
    out[40, 2] = ref[40, 2]
    assert torch.equal(out, ref)


def test_varlen_lengths_outside_the_tensors_stay_inside():
    """Prefix sums that leave the tensors or fall are cut to them: nothing outside is read or written."""
    rng = np.random.default_rng(15)
    q, k, v, _, _ = packed(rng, [64], [64], 2, 1, 64, layout="dense")
    room = torch.full((128, 2, 64), 7.0, device="cuda", dtype=B16)
    for cu in ([0, 1000], [-5, 64], [0, 2 ** 30], [64, 0], [70, 90]):
        run_varlen(q, k, v, ints(cu), ints(cu), True, out=room[32:96])
        assert (room[:32] == 7).all() and (room[96:] == 7).all()


def test_varlen_repeats_itself():
    rng = np.random.default_rng(16)
    q, k, v, cu, _ = packed(rng, [700, 33, 260], [700, 33, 260], 8, 2, 128)
    a, la = run_varlen(q, k, v, cu, cu, True)
    for _ in range(5):
        b, lb = run_varlen(q, k, v, cu, cu, True)
        assert torch.equal(a, b) and torch.equal(la, lb)


def gradient_tolerances(dout, q, k, v, out, scale, causal):
    """Bounds of dq, dk, dv: every weight is off by w of itself (weight_error, with an lse that is off as much again), p and dz
    are rounded to bf16, g = dout . v - dout . out is a float32 difference of sums of d products, sums of n (m) terms follow and
    the result is rounded to bf16."""
    n, hq, d = q.shape
    group, m = hq // k.shape[1], k.shape[0]
    see = lm.seen(n, m, causal)
    kk, vv = np.repeat(k, group, 1), np.repeat(v, group, 1)
    z = np.where(see[:, None, :], np.einsum("ihd,jhd->ihj", q, kk) * scale, -np.inf)
    top = np.maximum(z.max(-1, keepdims=True, initial=-1e300), -1e300)
    e = np.where(see[:, None, :], np.exp(z - top), 0.0)
    p = e / np.maximum(e.sum(-1, keepdims=True), 1e-300)
    w = 2 * weight_error(q, k, scale, causal)[:, :, None] + (m + 16) * U
    g = np.abs(np.einsum("ihd,jhd->ihj", dout, vv) - np.einsum("ihd,ihd->ih", dout, out)[:, :, None])
    size = np.einsum("ihd,jhd->ihj", np.abs(dout), np.abs(vv)) + np.einsum("ihd,ihd->ih", np.abs(dout), np.abs(out))[:, :, None]
    off = p * (g * (2.0 ** -8 + w + 8 * U) + 2 * (d + 4) * U * size)  # of one dz
    sums = 2 * (n * group + m + 16) * U
    dq = scale * np.einsum("ihj,jhd->ihd", off + sums * p * g, np.abs(kk))
    dk = scale * np.einsum("ihj,ihd->jhd", off + sums * p * g, np.abs(q))
    dv = np.einsum("ihj,ihd->jhd", p * (2.0 ** -8 + w + sums), np.abs(dout))
    return dq, *(x.reshape(m, hq // group, group, d).sum(2) for x in (dk, dv))


def run_gradients(dout, q, k, v, cu_q, cu_k, causal, scale=None, out=None, lse=None, ws=None):
    if out is None:
        out, lse = run_varlen(q, k, v, cu_q, cu_k, causal, scale)
    dq, dk, dv = (torch.full_like(t, 7.0, memory_format=torch.contiguous_format) for t in (q, k, v))
    ws = L.mmdit_varlen_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, cu_q, cu_k=cu_k, causal=causal, scale=scale, ws=ws)
    torch.cuda.synchronize()
    assert L.mmdit_workspace_status(ws) == 0
    return dq, dk, dv, out, lse


def compare_gradients(q, k, v, cu_q, cu_k, causal, scale=None, seed=0):
    dout = rand(np.random.default_rng(seed), *q.shape)
    a, b = cu_q.tolist(), cu_k.tolist()
    dout[a[-1]:] = float("nan")
    dq, dk, dv, out, lse = run_gradients(dout, q, k, v, cu_q, cu_k, causal, scale)
    s = q.shape[2] ** -0.5 if scale is None else scale
    for i in range(len(a) - 1):
        x, y = slice(a[i], a[i + 1]), slice(b[i], b[i + 1])
        args = f64(dout[x]), f64(q[x]), f64(k[y]), f64(v[y]), f64(out[x])
        refs = lm.attention_bwd(*args, f64(lse[x]), s, causal)
        for name, got, ref, tol in zip(("dq", "dk", "dv"), (dq[x], dk[y], dv[y]), refs, gradient_tolerances(*args, s, causal)):
            check(f64(got), ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 1e-30, f"{name} of sequence {i}")
    assert (dq[a[-1]:] == 7).all() and (dk[b[-1]:] == 7).all() and (dv[b[-1]:] == 7).all()


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (2, 2, 64), (5, 1, 96)])
def test_gradients(lengths, causal, hq, hk, d):
    nq, nk = LENGTHS[lengths]
    rng = np.random.default_rng(len(lengths) + 17 * d + causal)
    compare_gradients(*packed(rng, nq, nk, hq, hk, d, pad=3), causal)


@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 3), (7, 1), (16, 1), (48, 1), (64, 1), (14, 2)])
def test_gradients_groups(hq, hk):
    rng = np.random.default_rng(hq + 1)
    compare_gradients(*packed(rng, [9, 37], [40, 37], hq, hk, 64, pad=1), True)


@pytest.mark.parametrize("d", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("layout", ["dense", "packed", "head_major"])
def test_gradients_head_dims_and_layouts(d, layout):
    rng = np.random.default_rng(d + 1)
    compare_gradients(*packed(rng, [131], [131], 4, 2, d, layout=layout, pad=2), True)


@pytest.mark.parametrize("scale", [1e-3, 1.0])
def test_gradients_scales(scale):
    rng = np.random.default_rng(22)
    compare_gradients(*packed(rng, [140], [140], 2, 2, 64), True, scale=scale)


def test_gradients_into_views_of_a_packed_projection():
    rng = np.random.default_rng(23)
    q, k, v, cu, _ = packed(rng, [90, 150], [90, 150], 8, 2, 96)
    dout = rand(rng, *q.shape)
    dq, dk, dv, out, lse = run_gradients(dout, q, k, v, cu, cu, True)
    whole = torch.full((240, 14, 96), 7.0, device="cuda", dtype=B16)
    L.mmdit_varlen_attention_bwd(dout, q, k, v, out, lse, whole[:, 1:9], whole[:, 9:11], whole[:, 11:13], cu)
    assert torch.equal(whole[:, 1:9], dq) and torch.equal(whole[:, 9:11], dk) and torch.equal(whole[:, 11:13], dv)
    assert (whole[:, 0] == 7).all() and (whole[:, 13] == 7).all()


def test_gradients_repeat_themselves():
    rng = np.random.default_rng(24)
    q, k, v, cu, _ = packed(rng, [600, 33, 260], [600, 33, 260], 8, 2, 128)
    dout = rand(rng, *q.shape)
    first = run_gradients(dout, q, k, v, cu, cu, True)
    for _ in range(4):
        again = run_gradients(dout, q, k, v, cu, cu, True, out=first[3], lse=first[4])
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_masked_places(d):
    """A query row that is not finite reaches the keys that it sees, a key row the queries that see it, nothing else."""
    rng = np.random.default_rng(25)
    q, k, v, cu, _ = packed(rng, [100, 200], [100, 200], 2, 1, d, layout="dense")
    dout = rand(rng, *q.shape)
    dq, dk, dv, out, lse = run_gradients(dout, q, k, v, cu, cu, True)
    rows = torch.arange(300, device="cuda")
    for at in (0, 57, 99, 100, 170, 299):
        mine = rows < 100 if at < 100 else rows >= 100
        for which in ("q", "dout"):
            q2, g2 = q.clone(), dout.clone()
            (q2 if which == "q" else g2)[at] = float("nan")
            eq, ek, ev, _, _ = run_gradients(g2, q2, k, v, cu, cu, True, out=out, lse=lse)
            clean = ~mine | (rows > at)
            assert torch.equal(ek[clean], dk[clean]) and torch.equal(ev[clean], dv[clean])
            assert torch.isnan(ek[~clean]).all() and torch.isnan(ev[~clean]).all()
            assert torch.equal(eq[rows != at], dq[rows != at]) and torch.isnan(eq[at]).all()
        k2 = k.clone()
        k2[at] = float("nan")
        eq, ek, ev, _, _ = run_gradients(dout, q, k2, v, cu, cu, True, out=out, lse=lse)
        clean = ~mine | (rows < at)
        assert torch.equal(eq[clean], dq[clean]) and torch.isnan(eq[~clean]).all()
        assert torch.equal(ek[rows != at], dk[rows != at]) and torch.equal(ev[rows != at], dv[rows != at])


def test_gradients_against_differences():
    """d loss / d x of loss = sum(dout out) by central differences of the float64 forward, within the gradients' bounds."""
    rng = np.random.default_rng(26)
    q, k, v, cu, _ = packed(rng, [40], [40], 4, 2, 64, layout="dense", spread=1.0)
    dout = rand(rng, *q.shape)
    dq, dk, dv, out, _ = run_gradients(dout, q, k, v, cu, cu, True)
    host, g, scale, h = [f64(t) for t in (q, k, v)], f64(dout), 0.125, 1e-5
    # out's own rounding to bf16 enters dz through dout . out: 2^-8 of each term
    args = g, *host, f64(out)
    tols = gradient_tolerances(*args, scale, True)
    slack = np.einsum("ihd,ihd->ih", np.abs(g), np.abs(f64(out))).max() * 2.0 ** -8 * scale
    for name, got, tol, i in (("dq", dq, tols[0], 0), ("dk", dk, tols[1], 1), ("dv", dv, tols[2], 2)):
        for _ in range(12):
            at = tuple(int(rng.integers(0, n)) for n in host[i].shape)
            d = []
            for sign in (1, -1):
                moved = [x.copy() for x in host]
                moved[i][at] += sign * h
                d.append((g * lm.attention(*moved, scale, True)[0]).sum())
            ref = (d[0] - d[1]) / (2 * h)
            # the sum of a row's weights is one, of a column's at most the rows times the group
            extra = 0.0 if i == 2 else slack * (np.abs(host[1]).max() if i == 0 else np.abs(host[0]).max() * 2 * 40)
            assert abs(float(got[at]) - ref) <= tol[at] * 1.01 + 2.0 ** -8 * abs(ref) + extra + 1e-6, (name, at)


# ------------------------------------------------------------------------------------- paged cache
def paged(rng, new, total, hq, hk, d, page, width=None, pad=0, spread=2.0, layout="pages", dead=()):
    """A cache whose unused slots are NaN, with shuffled pages; `dead`: (request, page) pairs without a page."""
    count = [-(-t // page) for t in total]
    width = max(max(count), 1) if width is None else width
    pages = sum(count) + 2
    order = rng.permutation(pages)
    shape = (pages, page, hk, d) if layout == "pages" else (pages, hk, page, d)
    kc, vc = (torch.full(shape, float("nan"), device="cuda", dtype=B16) for _ in range(2))
    if layout != "pages":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    tables = torch.full((len(new), width), 123456, dtype=torch.int32)
    keys, values, at = [], [], 0
    for b, t in enumerate(total):
        k, v = rand(rng, t, hk, d), rand(rng, t, hk, d)
        for p in range(count[b]):
            part = slice(p * page, min((p + 1) * page, t))
            tables[b, p] = int(order[at])
            kc[order[at], : part.stop - part.start], vc[order[at], : part.stop - part.start] = k[part], v[part]
            if (b, p) in dead:
                tables[b, p] = [-1, pages, 2 ** 30][(b + p) % 3]
            at += 1
        keys.append(k)
        values.append(v)
    q = rand(rng, sum(new) + pad, hq, d, scale=spread)
    if pad:
        q[-pad:] = float("nan")
    return q, kc, vc, tables.cuda(), ints(total), ints(sums(new)), keys, values


def run_paged(case, max_q=None, max_kv=None, lse=True, ws=None):
    q, kc, vc, tables, lens, cu, _, _ = case
    out = torch.full_like(q, 7.0)
    sums_ = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    ws = L.mmdit_paged_attention_fwd(q, kc, vc, out, tables, lens, cu, lse=sums_, max_q=max_q, max_kv=max_kv, ws=ws)
    torch.cuda.synchronize()
    assert L.mmdit_workspace_status(ws) == 0
    return out, sums_


def compare_paged(case, max_q=None, max_kv=None, dead=(), page=None):
    q, _, _, _, _, cu, keys, values = case
    out, lse = run_paged(case, max_q, max_kv)
    a = cu.tolist()
    for b in range(len(a) - 1):
        x = slice(a[b], a[b + 1])
        if a[b] == a[b + 1]:
            continue
        k, v, n = f64(keys[b]), f64(values[b]), a[b + 1] - a[b]
        there = np.ones(len(k), bool)
        for r, p in dead:
            if r == b:
                there[p * page:(p + 1) * page] = False
        # rows in order see prefixes of the request; pages that are not there hold no keys
        ref, rl, tol, tl = (np.zeros((n, q.shape[1], q.shape[2])), np.zeros((n, q.shape[1])), None, None)
        if there.all():
            ref, rl, tol, tl = attention_reference(f64(q[x]), k, v, True)
        else:
            parts = []
            for i in range(n):
                keep = np.flatnonzero(there[: len(k) - n + i + 1])
                parts.append(attention_reference(f64(q[a[b] + i:a[b] + i + 1]), k[keep], v[keep], False))
            ref, rl, tol, tl = (np.concatenate(t) for t in zip(*parts))
        # a split row's parts are joined in float32: two more roundings of each and the exponential of their weights
        check(f64(out[x]), ref, tol + 2.0 ** -20 * np.abs(tol) / 2.0 ** -8, f"out of request {b}")
        check(f64(lse[x]), rl, tl + 2.0 ** -20, f"lse of request {b}")
    assert (out[a[-1]:] == 7).all() and (lse[a[-1]:] == 7).all()


PAGED = {
    "one": ([1], [1]), "page_end": ([1, 1, 1], [16, 17, 15]), "none_cached": ([1, 1], [0, 1]), "batch": ([1] * 9, [1, 300, 77, 512, 16, 1030, 8, 9, 255]),
    "speculative": ([3, 4, 1, 2], [3, 700, 90, 33]), "idle": ([1, 0, 2, 0], [40, 50, 60, 0]), "chunk": ([150], [400]),
    "whole": ([200], [200]), "mixed": ([1, 140, 1, 37, 0, 5], [500, 140, 33, 600, 12, 70]), "cut": ([20], [12]),
}


@pytest.mark.parametrize("name", list(PAGED))
@pytest.mark.parametrize("hq,hk,d,page", [(4, 1, 128, 16), (2, 2, 64, 8), (10, 2, 96, 64), (7, 1, 80, 256)])
def test_paged(name, hq, hk, d, page):
    new, total = PAGED[name]
    rng = np.random.default_rng(len(name) + d)
    compare_paged(paged(rng, new, total, hq, hk, d, page, pad=2))
    compare_paged(paged(rng, new, total, hq, hk, d, page), max_q=max(new), max_kv=max(total))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 512])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_paged_page_sizes_and_layouts(page, new):
    rng = np.random.default_rng(page + new)
    compare_paged(paged(rng, [new, new], [new + 333, new], 4, 2, 64, page, layout="heads", width=70))


@pytest.mark.parametrize("new,hq,hk,d", [(1, 8, 2, 128), (4, 4, 1, 64), (2, 16, 2, 128), (9, 8, 2, 128), (130, 4, 2, 64)])
def test_paged_long_contexts_are_split(new, hq, hk, d):
    """Few rows over long contexts: several CTAs to a request, joined afterwards."""
    rng = np.random.default_rng(new + d)
    case = paged(rng, [new], [9000], hq, hk, d, 64)
    compare_paged(case)
    compare_paged(paged(rng, [new, 1, new], [5000, 300, 2600], hq, hk, d, 16))
    a, la = run_paged(case)
    for _ in range(4):
        b, lb = run_paged(case)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("new", [1, 3, 30])
@pytest.mark.parametrize("page", [8, 32, 128, 256])
def test_paged_entries_without_a_page_hold_no_keys(new, page):
    rng = np.random.default_rng(page + 2 * new)
    dead = {(0, 0), (0, 3), (1, 1)} | ({(2, 0)} if page >= 128 else {(2, p) for p in range(0, 200 // page)})
    total = [max(new + 500, 4 * page), new + page + 5, 150 if page < 128 else 90]
    case = paged(rng, [new] * 3, total, 4, 1, 128, page, dead=dead, width=max(-(-t // page) for t in total) + 3)
    compare_paged(case, dead=dead, page=page)


def test_paged_lengths_beyond_the_tables_stop_there():
    rng = np.random.default_rng(3)
    q, kc, vc, tables, lens, cu, keys, values = paged(rng, [1, 40], [64, 64], 4, 1, 128, 16)
    for n in (1, 2):
        part = (q[:n] if n == 1 else q, kc, vc, tables, lens, cu, keys, values)
        ref, _ = run_paged((q, kc, vc, tables, lens, cu, keys, values))
        out, _ = run_paged((q, kc, vc, tables, ints([2 ** 30, 64]), cu, keys, values))
        assert torch.equal(out, ref) and part is not None


@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_paged_later_tokens_do_not_reach_a_row(new, bad):
    rng = np.random.default_rng(new)
    q, kc, vc, tables, lens, cu, keys, values = paged(rng, [new], [new + 70], 4, 1, 64, 16)
    ref, _ = run_paged((q, kc, vc, tables, lens, cu, keys, values))
    for i in range(0, new, 3):
        pos = 70 + i
        kc2, vc2 = kc.clone(), vc.clone()
        at = (int(tables[0, pos // 16]), pos % 16)
        kc2[at], vc2[at] = bad, bad
        out, _ = run_paged((q, kc2, vc2, tables, lens, cu, keys, values))
        assert torch.equal(out[:i], ref[:i])
        vc2 = vc.clone()
        vc2[at[0], at[1], 0, 9] = bad
        out, _ = run_paged((q, kc, vc2, tables, lens, cu, keys, values))
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[i:, :, 9] = True
        assert torch.equal(out[~hit], ref[~hit]) and not torch.isfinite(out[hit]).any()


# ------------------------------------------------------------------------------------- tables and writes
def tables_case(rng, batch, page, width, n_pages, ctx, new, done=0.2, dead=0.0):
    before = rng.integers(0, ctx + 1, batch)
    after = np.where(rng.random(batch) < done, rng.integers(0, before + 1), before + rng.integers(0, new + 1, batch))
    held = -(-np.clip(before, 0, width * page) // page)
    order = rng.permutation(n_pages)
    tables = np.full((batch, width), -7, np.int64)
    at = 0
    for b, h in enumerate(held):
        tables[b, :h] = order[at:at + h]
        at += h
    assert at <= n_pages
    tables[(rng.random(tables.shape) < dead) & (np.arange(width)[None, :] < held[:, None])] = -1
    free = np.full(n_pages, -9, np.int64)
    free[: n_pages - at] = order[at:]
    return before, after, tables, free, n_pages - at


def run_tables(before, after, tables, free, n_free, page, capacity, in_place=False):
    t = {n: ints(np.asarray(x, np.int64).tolist()).reshape(np.shape(x)) for n, x in (("before", before), ("after", after), ("tables", tables), ("free", free),
                                                     ("n_free", [n_free]))}
    out = t["n_free"] if in_place else ints([-1])
    cu, missing = ints([-1] * (len(before) + 1)), ints([-1, -1])
    pos, slots = (torch.full((capacity,), -5, dtype=torch.int64, device="cuda") for _ in range(2))
    for _ in range(1 if in_place else 2):  # the same call again gives the same result
        L.mmdit_block_tables(t["before"], t["after"], t["tables"], t["free"], t["n_free"], page, out, cu, pos, slots, missing)
    return [x.cpu().numpy() for x in (t["tables"], t["free"], out, cu, pos, slots, missing)]


def compare_tables(before, after, tables, free, n_free, page, capacity, in_place=False):
    got = run_tables(before, after, tables, free, n_free, page, capacity, in_place)
    ref = lm.block_tables(before, after, tables, free, n_free, page, capacity)
    for name, x, y in zip(("tables", "free_pages", "n_free", "cu", "positions", "slots", "missing"), got, ref):
        assert np.array_equal(np.ravel(x), np.ravel(y)), name


@pytest.mark.parametrize("batch,page,width,ctx,new", [(1, 16, 8, 100, 20), (3, 8, 40, 0, 300), (256, 16, 70, 1000, 1), (70, 64, 30, 900, 600),
                                                      (1025, 8, 12, 60, 30), (3000, 32, 5, 100, 40)])
def test_block_tables(batch, page, width, ctx, new):
    rng = np.random.default_rng(batch)
    case = tables_case(rng, batch, page, width, batch * width + 5, ctx, new)
    total = int(np.maximum(case[1] - case[0], 0).sum())
    compare_tables(*case, page, total)
    compare_tables(*case, page, total + 77, in_place=True)
    compare_tables(*case, page, max(total - 10, 0))


def test_block_tables_of_few_pages():
    """More pages wanted than free, entries without a page given back, lengths beyond the tables."""
    rng = np.random.default_rng(9)
    for dead in (0.0, 0.3):
        before, after, tables, free, n_free = tables_case(rng, 60, 8, 20, 700, 80, 60, dead=dead)
        compare_tables(before, after, tables, free, min(n_free, 5), 8, 4000)
        after[3], before[5], after[7] = 10000, -3, -1
        compare_tables(before, after, tables, free, n_free, 8, 5000)
    compare_tables([], [], np.zeros((0, 4)), np.arange(5), 5, 8, 3)


def test_cache_write():
    rng = np.random.default_rng(4)
    for tokens, h, d, page, layout in ((1, 1, 8, 8, "pages"), (33, 8, 128, 16, "pages"), (500, 3, 80, 64, "heads"), (70, 40, 512, 32, "pages"),
                                       (2500, 2, 64, 256, "heads")):
        pages = tokens // page + 9
        shape = (pages, page, h, d) if layout == "pages" else (pages, h, page, d)
        kc, vc = rand(rng, *shape), rand(rng, *shape)
        if layout == "heads":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        wide = rand(rng, tokens, 3 * h, d)
        k, v = wide[:, h:2 * h], wide[:, 2 * h:]
        slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int64)).cuda()
        slots[::7] = -1
        slots[3::11] = pages * page + 5
        rk, rv = kc.clone(), vc.clone()
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page:
                rk[s // page, s % page], rv[s // page, s % page] = k[t], v[t]
        L.mmdit_kv_cache_write(k, v, kc, vc, slots)
        assert torch.equal(kc, rk) and torch.equal(vc, rv)
