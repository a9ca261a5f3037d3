"""Rows of the text model's attention whose scores are infinite, and calls at the ends of the documented ranges."""
import numpy as np
import pytest
import torch

import test_gpu_attention as base
from diffusion_transformer_flux_gb300 import _lib as L

pytestmark = pytest.mark.gpu
B16 = torch.bfloat16
INF = float("inf")


def row_reference(q, k, v, keys):
    """(out, lse, bounds) [1, 1, d] of one row of one head over the keys in `keys`."""
    return base.attention_reference(base.f64(q)[None, None], base.f64(k)[keys][:, None], base.f64(v)[keys][:, None], False)


def check_row(out, lse, q, k, v, keys, seen, what):
    """A row that sees no key: 0 and -inf.  Scores that are all -inf have no weights (0 / 0): NaN.  Else the -inf ones weigh 0."""
    if not seen:
        assert (out == 0).all() and lse == -INF, what
    elif not len(keys):
        assert torch.isnan(out).all() and torch.isnan(lse), what
    else:
        ref, rl, tol, tl = row_reference(q, k, v, keys)
        # parts of a split row are joined in float32, as in base.compare_paged
        base.check(base.f64(out)[None, None], ref, tol * (1 + 2.0 ** -12), what)
        base.check(base.f64(lse)[None, None], rl, tl + 2.0 ** -20, what)


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 128), (3, 1, 96), (2, 2, 64)])
def test_packed_rows_whose_scores_are_all_minus_infinity(hq, hk, d, causal, sign):
    """One infinite element of q against keys of the opposite sign: the row is NaN, all others keep their bits."""
    rng = np.random.default_rng(d + causal)
    q, k, v, cu, _ = base.packed(rng, [5, 300, 1], [5, 300, 1], hq, hk, d, layout="dense")
    k[:, :, 0] = -sign * (k[:, :, 0].abs() + 0.125)
    clean, sums = base.run_varlen(q, k, v, cu, cu, causal)
    rows = [0, 3, 5, 5 + 140, 304, 305]  # first tokens, with one key each where the mask is causal; rows of one tile and of three
    bad = q.clone()
    bad[rows, 1, 0] = sign * INF
    out, lse = base.run_varlen(bad, k, v, cu, cu, causal)
    assert torch.isnan(out[rows, 1]).all() and torch.isnan(lse[rows, 1]).all()
    out[rows, 1], lse[rows, 1] = clean[rows, 1], sums[rows, 1]
    assert torch.equal(out, clean) and torch.equal(lse, sums)


def test_packed_keys_of_minus_infinity():
    """Keys whose score is -inf weigh nothing; a row that sees only such keys is NaN, one that sees none at all is 0."""
    rng = np.random.default_rng(7)
    n, m, dead = 300, 290, 150  # the first ten rows see no key
    q, k, v, cq, ck = base.packed(rng, [n], [m], 2, 1, 64, layout="dense")
    q[:, :, 0] = q[:, :, 0].abs() + 0.125
    k[:dead, :, 0] = -INF
    out, lse = base.run_varlen(q, k, v, cq, ck, True)
    for i in (0, 9, 10, 11, 100, 137, 138, 139, 159, 160, 161, 200, 299):
        see = m - n + i + 1
        for h in range(2):
            check_row(out[i, h], lse[i, h], q[i, h], k[:, 0], v[:, 0], np.arange(dead, max(see, dead)), see > 0, (i, h))


# new tokens and cached ones: few rows in one CTA, over several; a tile, a tile whose keys are split, and both kernels at once
PAGED = {"few": ([1, 3], [40, 9]), "few_runs": ([1, 4], [20000, 700]), "tile": ([30], [300]), "tile_parts": ([130], [20000]),
         "mixed": ([1, 40, 2], [6000, 5000, 33])}


@pytest.mark.parametrize("name", list(PAGED))
@pytest.mark.parametrize("d", [64, 128])
def test_paged_rows_whose_scores_are_all_minus_infinity(name, d):
    new, total = PAGED[name]
    rng = np.random.default_rng(len(name) + d)
    case = base.paged(rng, new, total, 4, 2, d, 16)
    q, kc = case[0], case[1]
    kc[..., 0] = kc[..., 0].abs() + 0.125
    clean, sums = base.run_paged(case)
    starts = base.sums(new)
    rows = sorted({r for b in range(len(new)) for r in (starts[b], starts[b + 1] - 1)})
    bad = q.clone()
    bad[rows, 2, 0] = -INF
    out, lse = base.run_paged((bad, *case[1:]))
    assert torch.isnan(out[rows, 2]).all() and torch.isnan(lse[rows, 2]).all()
    out[rows, 2], lse[rows, 2] = clean[rows, 2], sums[rows, 2]
    assert torch.equal(out, clean) and torch.equal(lse, sums)


@pytest.mark.parametrize("name", list(PAGED))
@pytest.mark.parametrize("share", [0.4, 1.0])
def test_paged_keys_of_minus_infinity(name, share):
    """The first `share` of each request's keys have a score of -inf: parts of nothing else weigh nothing beside others; where
    all keys are such, rows are NaN."""
    new, total = PAGED[name]
    rng = np.random.default_rng(len(name))
    q, kc, vc, tables, lens, cu, keys, values = base.paged(rng, new, total, 4, 2, 64, 16)
    q[..., 0] = q[..., 0].abs() + 0.125
    dead = [round(share * t) for t in total]
    for b, n in enumerate(dead):
        at = torch.arange(n, device="cuda")
        kc[tables[b, at // 16].long(), at % 16, :, 0] = -INF
    out, lse = base.run_paged((q, kc, vc, tables, lens, cu, keys, values))
    starts = base.sums(new)
    for b, (n, t) in enumerate(zip(new, total)):
        for i in sorted({0, n // 2, n - 1}):
            see = t - n + i + 1
            for h in (0, 3):
                r, g = starts[b] + i, h // 2
                check_row(out[r, h], lse[r, h], q[r, h], keys[b][:, g], values[b][:, g], np.arange(dead[b], max(see, dead[b])), True,
                          (b, i, h))


@pytest.mark.parametrize("new,total", [([1], [64]), ([1], [9000]), ([40], [300]), ([130], [9000])])
def test_paged_rows_without_a_page_stay_zero(new, total):
    """Without any page a row sees no key; with one, whose scores are -inf, it is NaN."""
    rng = np.random.default_rng(new[0])
    page, count = 16, -(-total[0] // 16)
    case = base.paged(rng, new, total, 4, 2, 64, page, dead=[(0, p) for p in range(count)])
    out, lse = base.run_paged(case)
    assert (out == 0).all() and (lse == -INF).all()
    q, kc, _, tables = case[:4]
    q[..., 0] = -INF
    kc[0, :, :, 0] = 1.0
    tables[0, 1] = 0
    case[2][0] = 1.0
    kc[0, :, :, 1:] = 1.0
    out, lse = base.run_paged(case)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_items_that_take_seconds():
    """One query over 4 x 10^8 keys: the warps that clean the last tile, and those of the item's absent second tile, wait longer for it
    than a wait may stand still."""
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("needs 50 GB")
    m, d, half = (3 << 27) - 5, 8, 3 << 26
    kv = torch.ones(m, 1, d, dtype=B16, device="cuda")
    kv[half:] = -1
    q, dout, one = torch.zeros(1, 1, d, dtype=B16, device="cuda"), *(torch.ones(1, 1, d, dtype=B16, device="cuda") for _ in range(2))
    cu_q, cu_k = base.ints([0, 1]), base.ints([0, m])
    out, lse = base.run_varlen(q, kv, kv, cu_q, cu_k, True)
    mean = (half - (m - half)) / m
    # all weights are 1.  A product adds a few keys' terms at a time to a float32 sum, which takes none of them any more once they are
    # below its last place (of terms of 8, at 2^27): a sum of m terms is off by up to m 2^-23 of the sum of their magnitudes
    assert (out.double() - mean).abs().max() <= 2.0 ** -8 * mean + m * 2.0 ** -23
    assert abs(lse.item() - np.log(m)) <= 2.0 ** -22 * np.log(m)
    v = torch.zeros_like(kv)
    v[-1000:] = 3
    out, _ = base.run_varlen(q, kv, v, cu_q, cu_k, True)
    assert (out.double() * m / 3000 - 1).abs().max() <= 2.0 ** -8 + 2.0 ** -16
    # gradients: with out = 1 and v = 1, dz = p (dout . v - dout . out) is 0 but for the last 1000 keys, where it is 16 p
    v = torch.ones_like(kv)
    v[-1000:] = 3
    dk, dv, dq = torch.full_like(kv, 7), torch.full_like(kv, 7), torch.full_like(q, 7)
    ws = L.mmdit_varlen_attention_bwd(dout, q, kv, v, one, lse, dq, dk, dv, cu_q, cu_k)
    torch.cuda.synchronize()
    assert L.mmdit_workspace_status(ws) == 0
    # p is off by 2^-16 (its exponent is 29, in float32), and dz or p and the result are rounded to bf16
    tol = 2.0 ** -7 + 2.0 ** -15
    assert (dq.double() * m / (-16000 * d ** -0.5) - 1).abs().max() <= tol
    assert not dk.any() and all((x.double() * m - 1).abs() <= tol for x in (dv.amax(), dv.amin()))


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_of_more_rows_than_31_bits_count(causal):
    """One sequence whose queries by the heads of a group pass 2^31.  All rows but the last tokens' have dout = 0 and add nothing;
    q, dout and out are read through views that overlap, dq needs its 34 GB."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    rng = np.random.default_rng(causal)
    group, d, m, n, last = 64, 8, 100, (1 << 25) + 1024, 128
    k, v = base.rand(rng, m, 1, d), base.rand(rng, m, 1, d)
    q, dout = (torch.zeros(n + group, d, dtype=B16, device="cuda") for _ in range(2))
    # element (token, head) is row token + head: the last 64 and the group's rows behind them are of the last 127 tokens
    q[n - 64:], dout[n - 64:] = base.rand(rng, 64 + group, d), base.rand(rng, 64 + group, d)
    view = [t.as_strided((n, group, d), (d, d, 1)) for t in (q, dout, torch.zeros_like(q))]
    lse = torch.zeros(n, group, device="cuda")
    end = slice(n - last, n)
    see = base.lm.seen(last, m, causal)
    ql, gl = (base.f64(t[end]) for t in view[:2])
    kl, vl, scale = base.f64(k), base.f64(v), d ** -0.5
    # rows of the last tokens may have any out and lse: the formula takes them as they are
    lse[end] = torch.logsumexp(torch.einsum("ihd,jd->ihj", view[0][end].float(), k[:, 0].float()) * scale, -1)
    cu_q, cu_k = base.ints([0, n]), base.ints([0, m])
    dq = torch.empty(n, group, d, dtype=B16, device="cuda")
    dq.fill_(7)
    dk, dv = torch.full_like(k, 7), torch.full_like(v, 7)
    ws = L.mmdit_varlen_attention_bwd(view[1], view[0], k, v, view[2], lse, dq, dk, dv, cu_q, cu_k, causal=causal)
    torch.cuda.synchronize()
    assert L.mmdit_workspace_status(ws) == 0
    ll = base.f64(lse[end])
    p = np.where(see[:, None, :], np.exp(scale * np.einsum("ihd,jd->ihj", ql, kl[:, 0]) - ll[:, :, None]), 0)
    z = p * np.einsum("ihd,jd->ihj", gl, vl[:, 0])
    refs = scale * np.einsum("ihj,jd->ihd", z, kl[:, 0]), scale * np.einsum("ihj,ihd->jd", z, ql), np.einsum("ihj,ihd->jd", p, gl)
    # each weight is off by its score's and the lse's error and two roundings to bf16 (of p or dz and of the result); zeros add nothing
    w = 4 * ((2 * d + 8) * base.U * np.abs(scale * np.einsum("ihd,jd->ihj", np.abs(ql), np.abs(kl[:, 0]))).max() + 2.0 ** -21)
    size = p * np.einsum("ihd,jd->ihj", np.abs(gl), np.abs(vl[:, 0]))
    each = 2.0 ** -8 + w + 2 * (last * group + m + d + 32) * base.U
    tols = (scale * np.einsum("ihj,jd->ihd", size, np.abs(kl[:, 0])) * each, scale * np.einsum("ihj,ihd->jd", size, np.abs(ql)) * each,
            np.einsum("ihj,ihd->jd", p, np.abs(gl)) * each)
    for name, got, ref, tol in zip(("dq", "dk", "dv"), (dq[end], dk[:, 0], dv[:, 0]), refs, tols):
        base.check(base.f64(got), ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 1e-30, name)
    for i in range(0, n - last, 1 << 22):
        assert not dq[i:min(i + (1 << 22), n - last)].any()


def test_gradients_of_many_queries_over_few_keys():
    """More than 16384 queries: their key tiles are worked on in parts as those of fewer are."""
    rng = np.random.default_rng(5)
    base.compare_gradients(*base.packed(rng, [17000, 40], [200, 40], 2, 1, 64, layout="dense"), False)


@pytest.mark.parametrize("new,total,large", [([130], [9000], (1500, 1, 9000)), ([1, 40, 2], [6000, 5000, 33], (6000, 3, 6000)),
                                             ([130], [9000], None), ([1, 4], [20000, 700], (300, 2, 20000))])
def test_paged_workspaces_of_other_calls(new, total, large):
    """One made for a larger call, or with no room for parts of the tiles (large: None), serves: no byte behind it is touched, and
    with its own or more the bits are the same."""
    rng = np.random.default_rng(len(new))
    hq, hk, d = 16, 4, 64
    case = base.paged(rng, new, total, hq, hk, d, 16)
    tables = torch.cat((case[3], torch.full((len(new), 2000 - case[3].shape[1]), -1, dtype=torch.int32, device="cuda")), 1)
    case = (*case[:3], tables, *case[4:])
    kv = max(total)
    own = L.mmdit_paged_attention_workspace_size(sum(new), len(new), hq, hk, d, max(new), kv)
    other = 256 if large is None else L.mmdit_paged_attention_workspace_size(large[0], large[1], hq, hk, d, large[0], large[2])

    def run(size):
        ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out = base.run_paged(case, max_q=max(new), max_kv=kv, ws=ws[:size])
        assert (ws[size:] == 0xA5).all()
        return out

    ref = run(own)
    again = run(own + (1 << 20))
    assert torch.equal(ref[0], again[0]) and torch.equal(ref[1], again[1])
    out, lse = run(other)
    # both are within the bounds that base.compare_paged checks; here one against the other: roundings of the weights and of the result
    assert ((out.double() - ref[0].double()).abs() <= 2.0 ** -6 * ref[0].double().abs() + 2.0 ** -6).all()
    assert ((lse - ref[1]).abs() <= 2.0 ** -8).all()  # twice the sums of up to 20000 terms, 2^-24 each
    base.compare_paged(case, max_q=max(new), max_kv=kv)


def test_block_tables_whose_places_nobody_asks_for():
    """The entry point without positions and slots, of a capacity that counts: prefix sums and pages, and no walk over the tokens."""
    batch, page, capacity = 64, 1 << 14, 1 << 24
    width = capacity // batch // page
    before, after = base.ints([0] * batch), base.ints([capacity // batch - 3] * batch)
    tables, free = torch.full((batch, width), -1, dtype=torch.int32, device="cuda"), torch.arange(batch * width, dtype=torch.int32, device="cuda")
    n_free, after_n, cu, missing = base.ints([batch * width]), base.ints([7]), base.ints([7] * (batch + 1)), base.ints([7, 7])
    best = float("inf")
    for _ in range(4):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        L._launch("mmdit_block_tables", before.device, None, batch, page, width, batch * width, before.data_ptr(), after.data_ptr(),
                  tables.data_ptr(), free.data_ptr(), n_free.data_ptr(), after_n.data_ptr(), cu.data_ptr(), capacity, None, None,
                  missing.data_ptr())
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end))
    assert cu.tolist() == [i * (capacity // batch - 3) for i in range(batch + 1)] and missing.tolist() == [0, 0] and after_n.tolist() == [0]
    assert tables.flatten().tolist() == list(range(batch * width - 1, -1, -1))
    assert best < 2.0, f"{best} ms"  # one CTA's few reads; the walk over the tokens took 13
