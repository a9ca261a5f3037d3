"""The attention of a text model and its paged cache as they are used: a server's steps, training steps, captured graphs,
several streams and more items than the GPU has SMs.  Tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest
import torch

import test_gpu_attention as base
from diffusion_transformer_flux_gb300 import _lib as L
from oracle import lm

pytestmark = pytest.mark.gpu
B16 = torch.bfloat16


# ------------------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("causal", [True, False])
def test_more_items_than_sms(causal):
    """40 heads of 3 sequences: 240 items of two tiles, so that a counter hands out the last ones."""
    rng = np.random.default_rng(1)
    base.compare_varlen(*base.packed(rng, [520, 40, 300], [520, 40, 300], 40, 40, 64, pad=2), causal)


def test_gradients_of_more_items_than_sms():
    rng = np.random.default_rng(2)
    base.compare_gradients(*base.packed(rng, [390, 40, 260], [390, 40, 260], 40, 40, 64, pad=2), True)


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (8, 1, 128), (3, 3, 128)])
def test_gradients_whose_queries_come_in_parts(hq, hk, d):
    """Few key tiles of many rows: several CTAs share one and their sums are joined."""
    rng = np.random.default_rng(hq)
    base.compare_gradients(*base.packed(rng, [700, 3], [200, 3], hq, hk, d, pad=1), False)
    base.compare_gradients(*base.packed(rng, [500], [500], hq, hk, d), True)


@pytest.mark.parametrize("batch", [33, 70, 200])
@pytest.mark.parametrize("hq,hk,d,page", [(8, 2, 128, 16), (7, 1, 64, 8)])
def test_paged_batches(batch, hq, hk, d, page):
    """Most requests get a token, some none, some a draft's few, some a chunk; contexts from none to hundreds."""
    rng = np.random.default_rng(batch + d)
    new = rng.choice([1, 1, 1, 1, 1, 1, 0, 2, 5, 40], batch).tolist()
    total = [int(n + rng.integers(0, 300)) for n in new]
    new[batch // 2], total[batch // 2] = 150, 170
    base.compare_paged(base.paged(rng, new, total, hq, hk, d, page, pad=2))


@pytest.mark.parametrize("width", [1, 200])
def test_paged_tables_wider_than_the_requests(width):
    """max_kv is the tables' reach by default: most of the work that is planned for has no keys."""
    rng = np.random.default_rng(width)
    base.compare_paged(base.paged(rng, [1, 1, 1], [64, 3, 40], 8, 2, 128, 64, width=width))
    base.compare_paged(base.paged(rng, [40, 1, 0], [64, 3, 40], 8, 2, 128, 64, width=width))


@pytest.mark.parametrize("d", [8, 24, 40, 72, 104, 120])
@pytest.mark.parametrize("new,hq,hk", [([1, 1], 4, 2), ([3, 1], 5, 1), ([70, 1], 6, 3)])
def test_paged_head_dims(d, new, hq, hk):
    rng = np.random.default_rng(d + hq)
    base.compare_paged(base.paged(rng, new, [900, 77], hq, hk, d, 32, pad=1))


@pytest.mark.parametrize("new,group", [(1, 8), (1, 9), (1, 16), (1, 17), (2, 8), (3, 5), (4, 4), (16, 1), (17, 1), (1, 128)])
def test_paged_rows_around_the_kernels_border(new, group):
    """Sequences of up to 16 rows are one kernel's, of more another's; up to 8 rows are one column of the first's products."""
    rng = np.random.default_rng(new + group)
    base.compare_paged(base.paged(rng, [new, 1], [1400, 40], 2 * group, 2, 64, 16, pad=1))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,total", [([1, 1, 1], [40, 300, 9]), ([3, 1, 4], [2000, 600, 4]), ([30, 1, 50], [2500, 600, 50])])
def test_paged_queries_that_are_not_finite_stay_alone(new, total, bad):
    """Their rows are NaN, whichever kernel they are of and however their keys are split; all others keep their bits."""
    rng = np.random.default_rng(sum(total))
    case = base.paged(rng, new, total, 4, 2, 64, 16)
    clean, sums = base.run_paged(case)
    for at in {0, new[0] - 1, new[0], sum(new) - 1}:
        q = case[0].clone()
        q[at, 1] = bad
        out, lse = base.run_paged((q, *case[1:]))
        assert torch.isnan(out[at, 1]).all() and torch.isnan(lse[at, 1])
        out[at, 1], lse[at, 1] = clean[at, 1], sums[at, 1]
        assert torch.equal(out, clean) and torch.equal(lse, sums)


def far_apart(small, stride, offset=0):
    """The values of `small` in a view whose first extent has stride `stride` (elements)."""
    room = torch.empty((small.shape[0] - 1) * stride + small[0].numel() + offset, dtype=small.dtype, device="cuda")
    view = room[offset:].as_strided(small.shape, (stride, *small.stride()[1:]))
    view.copy_(small)
    return view


@pytest.mark.parametrize("new", [1, 40])
def test_paged_offsets_beyond_32_bits(new):
    rng = np.random.default_rng(new)
    q, kc, vc, tables, lens, cu, keys, values = base.paged(rng, [new, 1], [100, 60], 4, 2, 64, 16)
    kc, vc = far_apart(kc, 1 << 28), far_apart(vc, 1 << 28)  # 12 pages: 6 GB
    assert (kc.shape[0] - 1) << 28 > 2 ** 31
    base.compare_paged((q, kc, vc, tables, lens, cu, keys, values))
    slots = base.ints([16 * (kc.shape[0] - 1) + 5], torch.int64)
    x = base.rand(rng, 1, 2, 64)
    L.mmdit_kv_cache_write(x, x, kc, vc, slots)
    assert torch.equal(kc[-1, 5], x[0]) and torch.equal(vc[-1, 5], x[0])


def test_packed_offsets_beyond_32_bits():
    rng = np.random.default_rng(3)
    q, k, v, cu, _ = base.packed(rng, [30, 12], [30, 12], 2, 1, 64, layout="dense")
    q, k, v = (far_apart(t, 1 << 26) for t in (q, k, v))
    assert (q.shape[0] - 1) << 26 > 2 ** 31
    base.compare_varlen(q, k, v, cu, cu, True)
    base.compare_gradients(q, k, v, cu, cu, True)
    out = far_apart(torch.zeros(42, 2, 64, device="cuda", dtype=B16), 1 << 26)
    ref, _ = base.run_varlen(q, k, v, cu, cu, True)
    base.run_varlen(q, k, v, cu, cu, True, out=out)
    assert torch.equal(out, ref)


# ------------------------------------------------------------------------------------- a server
class Server:
    """Requests over a paged cache; `history` keeps what a contiguous cache would hold."""

    def __init__(self, rng, batch=5, page=16, width=20, pages=90, hq=6, hk=2, d=64):
        self.rng, self.batch, self.page, self.hq, self.hk, self.d = rng, batch, page, hq, hk, d
        self.k_cache, self.v_cache = (torch.full((pages, page, hk, d), float("nan"), device="cuda", dtype=B16) for _ in range(2))
        self.tables = torch.full((batch, width), -1, device="cuda", dtype=torch.int32)
        self.free, self.n_free = base.ints(rng.permutation(pages).tolist()), base.ints([pages])
        self.lens = [0] * batch
        self.history = [(torch.zeros(0, hk, d, dtype=B16, device="cuda"),) * 2 for _ in range(batch)]
        self.rope = L.make_rope_cfg(d)

    def step(self, lens, capacity=None):
        new = [max(a - b, 0) for a, b in zip(lens, self.lens)]
        total = sum(new)
        cap = total if capacity is None else capacity
        before, after = base.ints(self.lens), base.ints(lens)
        cu, missing = torch.zeros(self.batch + 1, device="cuda", dtype=torch.int32), base.ints([9, 9])
        pos, slots = (torch.full((cap,), 99, device="cuda", dtype=torch.int64) for _ in range(2))
        L.mmdit_block_tables(before, after, self.tables, self.free, self.n_free, self.page, self.n_free, cu, pos, slots, missing)
        # one projection's rows: queries, keys and values side by side
        qkv = base.rand(self.rng, cap, self.hq + 2 * self.hk, self.d)
        q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
        L.mmdit_rope_fwd(self.rope, q[None], q[None], k[None], k[None], positions=pos)
        L.mmdit_kv_cache_write(k, v, self.k_cache, self.v_cache, slots)
        out = torch.full((cap, self.hq, self.d), 7.0, device="cuda", dtype=B16)
        ws = L.mmdit_paged_attention_fwd(q, self.k_cache, self.v_cache, out, self.tables, after, cu, max_q=max(new + [1]))
        torch.cuda.synchronize()
        assert L.mmdit_workspace_status(ws) == 0 and missing.tolist() == [0, 0]
        assert cu.tolist() == base.sums(new)
        at = 0
        for b, n in enumerate(new):
            kept = min(self.lens[b], lens[b])
            assert pos[at:at + n].tolist() == list(range(kept, kept + n))
            old_k, old_v = (t[:kept] for t in self.history[b])
            x = slice(at, at + n)
            self.history[b] = torch.cat((old_k, k[x])), torch.cat((old_v, v[x]))
            at += n
            if n:
                ref, _, tol, _ = base.attention_reference(base.f64(q[x]), *(base.f64(t) for t in self.history[b]), True)
                base.check(base.f64(out[x]), ref, tol + 2.0 ** -20 * np.abs(tol) / 2.0 ** -8, f"request {b}")
        assert (out[total:] == 7).all() and (slots[total:] == -1).all()
        self.lens = list(lens)
        return qkv, out, new


def test_server():
    """Prompts, single tokens, a chunk beside them, requests that end, new ones on their pages, drafts that are taken back."""
    s = Server(np.random.default_rng(10))
    s.step([37, 200, 0, 5, 16])
    for _ in range(3):
        s.step([n + 1 if n else 0 for n in s.lens])
    s.step([41, 0, 120, 9, 20], capacity=140)  # the second is done; a third arrives
    s.step([42, 150, 121, 10, 21])             # and one on the second's pages
    s.step([46, 154, 125, 14, 25])             # four tokens drafted each
    s.step([44, 152, 126, 12, 22])             # some taken back; shrinking requests get no tokens
    s.step([45, 153, 127, 13, 23])
    assert s.n_free.tolist() == [90 - sum(-(-n // 16) for n in s.lens)]


def test_paged_chunks_are_the_whole_prompt():
    """A prompt in chunks over a paged cache and the packed one agree to their roundings, and with the oracle."""
    s = Server(np.random.default_rng(11), batch=1, hq=8, hk=1, d=128)
    parts = []
    for n in (100, 101, 164, 300):
        qkv, out, _ = s.step([n])
        parts.append((qkv, out))
    qkv, out = (torch.cat(t) for t in zip(*parts))
    q, k, v = qkv.split([8, 1, 1], 1)
    whole, _ = base.run_varlen(q, k, v, base.ints([0, 300]), base.ints([0, 300]), True)
    _, _, tol, _ = base.attention_reference(base.f64(q), base.f64(k), base.f64(v), True)
    base.check(base.f64(out), base.f64(whole), 2 * tol * (1 + 2.0 ** -12), "chunks and whole")


# ------------------------------------------------------------------------------------- graphs and streams
def paged_call(case, out, lse, ws, max_q, **kw):
    q, kc, vc, tables, lens, cu, _, _ = case
    return L.mmdit_paged_attention_fwd(q, kc, vc, out, tables, lens, cu, lse=lse, max_q=max_q, ws=ws, **kw)


def captured(fn):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


def test_captured_steps_follow_the_lengths():
    """A decode step captured once: block tables, rotation, cache write and attention follow the device's lengths."""
    hq, hk, d, page, batch, width = 8, 2, 128, 16, 6, 40
    rng = np.random.default_rng(20)
    start = [1, 100, 333, 600, 15, 16]
    new, total = [1] * batch, [n + 1 for n in start]
    pages = 130

    def fresh():
        gen = np.random.default_rng(21)
        kc, vc = (base.rand(gen, pages, page, hk, d) for _ in range(2))
        tables = torch.full((batch, width), -1, dtype=torch.int32)
        order, at = gen.permutation(pages).tolist(), 0
        for b, n in enumerate(start):
            for p in range(-(-n // page)):
                tables[b, p] = order[at]
                at += 1
        return dict(kc=kc, vc=vc, tables=tables.cuda(), free=base.ints(order[at:] + [0] * at), n_free=base.ints([pages - at]),
                    before=base.ints(start), after=base.ints(total), qkv=base.rand(gen, batch, hq + 2 * hk, d),
                    cu=base.ints([0] * (batch + 1)), pos=base.ints([0] * batch, torch.int64), slots=base.ints([0] * batch, torch.int64),
                    missing=base.ints([0, 0]), rot=torch.zeros(batch, hq + hk, d, dtype=B16, device="cuda"),
                    out=torch.zeros(batch, hq, d, dtype=B16, device="cuda"),
                    ws=torch.zeros(L.mmdit_paged_attention_workspace_size(batch, batch, hq, hk, d, 1, width * page),
                                   dtype=torch.uint8, device="cuda"))

    cfg = L.make_rope_cfg(d)

    def step(s):
        L.mmdit_block_tables(s["before"], s["after"], s["tables"], s["free"], s["n_free"], page, s["n_free"], s["cu"], s["pos"],
                             s["slots"], s["missing"])
        q, k, v = s["qkv"].split([hq, hk, hk], 1)
        q_out, k_out = s["rot"].split([hq, hk], 1)
        L.mmdit_rope_fwd(cfg, q[None], q_out[None], k[None], k_out[None], positions=s["pos"])
        L.mmdit_kv_cache_write(k_out, v, s["kc"], s["vc"], s["slots"])
        L.mmdit_paged_attention_fwd(q_out, s["kc"], s["vc"], s["out"], s["tables"], s["after"], s["cu"], max_q=1, ws=s["ws"])

    def grow(s):
        s["before"].copy_(s["after"])
        s["after"].add_(1)
        s["qkv"].mul_(-0.875)

    eager, graphed = fresh(), fresh()
    g = captured(lambda: step(graphed))
    for _ in range(20):
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        for name in ("tables", "n_free", "cu", "pos", "slots", "missing", "out", "kc", "vc"):
            assert torch.equal(eager[name], graphed[name]), name
        assert eager["missing"].tolist() == [0, 0]
        grow(eager), grow(graphed)


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream: neither finds what the other left there."""
    rng = np.random.default_rng(22)
    cases = [(base.paged(rng, [1, 3, 1], [900, 40, 2000], 8, 2, 128, 16), 3), (base.paged(rng, [200, 1], [1500, 700], 8, 2, 128, 16), 200)]
    plain, graphs, outs = [], [], []
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    for case, max_q in cases:
        out, lse = base.run_paged(case, max_q=max_q)
        plain.append((out, lse))
        o, s = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        outs.append((o, s))
        graphs.append(captured(lambda: paged_call(case, o, s, ws, max_q)))
    for turn in (0, 1, 1, 0, 1, 0, 0, 1):
        outs[turn][0].fill_(7.0), outs[turn][1].fill_(7.0)
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[turn][0], plain[turn][0]) and torch.equal(outs[turn][1], plain[turn][1])
        assert L.mmdit_workspace_status(ws) == 0


def test_captured_training_step_with_an_eager_one_beside_it():
    """Forward and backward of packed sequences, captured; eager calls on the same tensors before, between and after."""
    rng = np.random.default_rng(23)
    q, k, v, cu, _ = base.packed(rng, [300, 41, 513], [300, 41, 513], 8, 2, 64)
    dout = base.rand(rng, *q.shape)
    first = base.run_gradients(dout, q, k, v, cu, cu, True)
    out, lse = torch.zeros_like(first[3]), torch.zeros_like(first[4])
    grads = [torch.zeros_like(t) for t in first[:3]]
    ws = torch.zeros(max(L.mmdit_varlen_attention_bwd_workspace_size(q.shape[0], 8, 64), 256), dtype=torch.uint8, device="cuda")

    def step():
        L.mmdit_varlen_attention_fwd(q, k, v, out, cu, lse=lse, ws=ws)
        L.mmdit_varlen_attention_bwd(dout, q, k, v, out, lse, *grads, cu, ws=ws)

    g = captured(step)
    for _ in range(3):
        for t in (out, lse, *grads):
            t.fill_(7.0)
        g.replay()
        again = base.run_gradients(dout, q, k, v, cu, cu, True)
        torch.cuda.synchronize()
        for a, b, c in zip(first, (*grads, out, lse), again):
            assert torch.equal(a, b) and torch.equal(a, c)
    # other sequences of the same tensors through the same graph
    cu.copy_(base.ints([0, 100, 600, 854]))
    g.replay()
    other = base.run_gradients(dout, q, k, v, cu, cu, True)
    for a, b in zip(other, (*grads, out, lse)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    rng = np.random.default_rng(24)
    packed_case = base.packed(rng, [700, 33, 1500], [700, 33, 1500], 16, 4, 128)
    q, k, v, cu, _ = packed_case
    paged_case = base.paged(rng, [1, 90, 4], [3000, 500, 900], 16, 4, 128, 16)
    dout = base.rand(rng, *q.shape)
    plain = base.run_gradients(dout, q, k, v, cu, cu, True)
    plain_paged = base.run_paged(paged_case, max_q=90)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros(1 << 27, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out, lse = torch.zeros_like(plain[3]), torch.zeros_like(plain[4])
    grads = [torch.zeros_like(t) for t in plain[:3]]
    o, s = torch.zeros_like(plain_paged[0]), torch.zeros_like(plain_paged[1])
    torch.cuda.synchronize()
    for _ in range(10):
        L.mmdit_varlen_attention_fwd(q, k, v, out, cu, lse=lse, ws=ws[0], stream=streams[0])
        paged_call(paged_case, o, s, ws[1], 90, stream=streams[1])
        L.mmdit_varlen_attention_bwd(dout, q, k, v, out, lse, *grads, cu, ws=ws[0], stream=streams[0])
        paged_call(paged_case, o, s, ws[1], 90, stream=streams[1])
    torch.cuda.synchronize()
    for a, b in zip(plain, (*grads, out, lse)):
        assert torch.equal(a, b)
    assert torch.equal(o, plain_paged[0]) and torch.equal(s, plain_paged[1])


def test_current_stream_is_the_calls():
    """On a side stream the calls come after that stream's work and before what follows there."""
    rng = np.random.default_rng(25)
    q, k, v, cu, _ = base.packed(rng, [300], [300], 4, 2, 64, layout="dense")
    ref, _ = base.run_varlen(q, k, v, cu, cu, True)
    side = torch.cuda.Stream()
    late, out = torch.zeros_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            late.copy_(q)
        L.mmdit_varlen_attention_fwd(late, k, v, out, cu)
        copy = out.clone()
    side.synchronize()
    assert torch.equal(copy, ref)


# ------------------------------------------------------------------------------------- empty calls
def test_empty_calls_touch_nothing():
    q = torch.zeros(0, 4, 64, dtype=B16, device="cuda")
    k = torch.zeros(3, 2, 64, dtype=B16, device="cuda")
    cu = base.ints([0, 0])
    L.mmdit_varlen_attention_fwd(q, k, k, q.clone(), cu, cu_k=base.ints([0, 3]))
    x = torch.zeros(3, 4, 64, dtype=B16, device="cuda")
    out = torch.full_like(x, 7.0)
    L.mmdit_varlen_attention_fwd(x, k, k, out, base.ints([0]), cu_k=base.ints([0]))
    cache = torch.full((2, 16, 2, 64), 7.0, dtype=B16, device="cuda")
    none = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    L.mmdit_paged_attention_fwd(x, cache, cache, out, none, base.ints([]), base.ints([0]))
    L.mmdit_kv_cache_write(k[:0], k[:0].clone(), cache, torch.full_like(cache, 7.0), base.ints([], torch.int64))
    # keys without queries have gradients of zero; queries without keys too
    dk, dv = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    lse = torch.zeros(0, 4, device="cuda")
    L.mmdit_varlen_attention_bwd(q, q, k, k, q, lse, q.clone(), dk, dv, cu, cu_k=base.ints([0, 3]))
    torch.cuda.synchronize()
    assert (out == 7).all() and (cache == 7).all() and (dk == 0).all() and (dv == 0).all()


def test_block_tables_without_places_or_requests():
    free, n = base.ints([3, 1, 2]), base.ints([3])
    tables = base.ints([[-1, -1]])
    cu, missing, after_n = base.ints([5, 5]), base.ints([5, 5]), base.ints([5])
    L.mmdit_block_tables(base.ints([0]), base.ints([17]), tables, free, n, 16, after_n, cu, None, None, missing)
    # without places the capacity is none: all tokens are left out of the map, the pages are theirs
    assert tables.tolist() == [[2, 1]] and after_n.tolist() == [1] and cu.tolist() == [0, 0] and missing.tolist() == [0, 17]
    pos = torch.full((4,), 9, dtype=torch.int64, device="cuda")
    L.mmdit_block_tables(base.ints([]), base.ints([]), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), free, n, 16, after_n,
                         cu[:1], pos, None, missing)
    assert pos.tolist() == [0] * 4 and after_n.tolist() == [3] and cu.tolist() == [0, 0] and missing.tolist() == [0, 0]


@pytest.mark.parametrize("batch", [64, 2049, 3000])
def test_block_tables_of_many_requests(batch):
    """Many that move many pages at once, and more than shared memory holds the sums of."""
    rng = np.random.default_rng(batch)
    page, width, pages = 8, 12, 6 * batch
    before = rng.integers(0, page * width + 1, batch)
    after = np.where(rng.random(batch) < 0.3, 0, rng.integers(0, page * width + 1, batch))
    tables, order, at = np.full((batch, width), -1, np.int32), rng.permutation(pages), 0
    for b in range(batch):
        for p in range(-(-int(before[b]) // page)):
            if at < pages:
                tables[b, p] = order[at]
                at += 1
    free = np.concatenate((order[at:], np.zeros(at, int))).astype(np.int32)
    fresh = int(np.maximum(after - before, 0).sum())
    for cap in (fresh + 3, 4096):
        ref = lm.block_tables(before, after, tables, free, pages - at, page, cap)
        t, f, n = base.ints(tables.tolist()), base.ints(free.tolist()), base.ints([0])
        cu, missing = base.ints([0] * (batch + 1)), base.ints([0, 0])
        pos, slots = (torch.zeros(cap, dtype=torch.int64, device="cuda") for _ in range(2))
        L.mmdit_block_tables(base.ints(before.tolist()), base.ints(after.tolist()), t, f, base.ints([pages - at]), page, n, cu, pos,
                             slots, missing)
        assert t.cpu().numpy().tolist() == ref[0].tolist() and n.tolist() == [ref[2]]
        assert f.cpu().numpy()[:ref[2]].tolist() == ref[1][:ref[2]].tolist()
        assert cu.tolist() == ref[3].tolist() and missing.tolist() == list(ref[6])
        assert pos.tolist() == ref[4].tolist() and slots.tolist() == ref[5].tolist()
