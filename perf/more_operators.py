"""The attention operators of a text model as measured cases: causal or bidirectional attention over packed
sequences with grouped heads (and its gradients), attention of new tokens over a paged cache of keys and
values, the block tables and slot maps of such a cache, and the write of new keys and values into it.

Each case has a plain form in elementary torch operations (float32 arithmetic) and the framework's own
calls; ``own`` selects which of the two ``run`` takes.  ``exact`` is the same result from the operator's
definition in float64.

Packed sequences lie one behind the other, sequence b at rows cu[b] .. cu[b + 1].  Query i of a sequence of n
queries and m keys stands at position m - n + i; with ``causal`` it sees the keys up to its own position.
Query head h reads key head h // (Hq / Hk).  A cache holds token p of request b in slot p % page of page
tables[b, p // page].
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a batch of two prompts of the benchmark's sequence (4096 + 512 tokens) through a causal layer
        dict(name="prompt", op="attn", n_seq=2, longest=4608, mix=0, prefix=0, hq=32, hk=8, d=128, causal=True, train=False),
        # a text encoder's batch, packed: sequences of 1 to 3000 tokens that see all of themselves, 5 heads to a group
        dict(name="packed_encoder", op="attn", n_seq=23, longest=3000, mix=5, prefix=0, hq=25, hk=5, d=96, causal=False, train=True),
        # a training step on packed documents of odd lengths
        dict(name="grad_packed", op="grad", n_seq=9, longest=2041, mix=3, prefix=0, hq=32, hk=8, d=128, causal=True),
        # a training step on whole sequences, as many key as query heads, narrow heads
        dict(name="grad_long", op="grad", n_seq=2, longest=4608, mix=0, prefix=0, hq=24, hk=24, d=64, causal=True),
        # one new token for each of 32 requests far into their contexts
        dict(name="paged_batch", op="paged", batch=32, chunks=0, longest=1, ctx=16384, mix=1, page=16, hq=32, hk=8, d=128),
        # one new token of one request behind a very long context: the time to the next word
        dict(name="paged_far", op="paged", batch=1, chunks=0, longest=1, ctx=120000, mix=0, page=64, hq=32, hk=8, d=128),
        # a chunk of a long prompt over what is cached of it
        dict(name="paged_chunk", op="paged", batch=1, chunks=1, longest=1000, ctx=31000, mix=0, page=64, hq=32, hk=8, d=128),
        # a step of a server: two prompts' chunks beside requests that answer, 7 heads to a group
        dict(name="paged_mixed", op="paged", batch=40, chunks=2, longest=333, ctx=5000, mix=2, page=32, hq=28, hk=4, d=64),
        # the tables of a step in which 256 requests get one token each and some are done
        dict(name="tables_step", op="tables", batch=256, ctx=8192, new=1, done=0.03, mix=1, page=16, width=640),
        # the tables of new prompts, and of requests that go on
        dict(name="tables_prompts", op="tables", batch=64, ctx=4608, new=2000, done=0.1, mix=2, page=64, width=128),
        # the new tokens of 32 answering requests into the cache
        dict(name="write_batch", op="write", tokens=32, hk=8, d=128, page=16, pages=4096),
        # a prompt's keys and values into the cache
        dict(name="write_prompt", op="write", tokens=9216, hk=8, d=128, page=64, pages=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    d = rng.choice([64, 64, 80, 96, 128, 128, 128])
    hk = rng.choice([1, 2, 4, 5, 8])
    return d, hk * rng.choice([1, 2, 4, 5, 7, 8]), hk


def draw(rng):
    op = rng.choice(["attn", "attn", "grad", "paged", "paged", "paged", "tables", "write"])
    mix = rng.randrange(1, 1 << 20)
    if op in ("attn", "grad"):
        d, hq, hk = _heads(rng)
        n_seq = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, max(2, min(6000, int((8e9 / (n_seq * hq * d)) ** 0.5))))
        c = dict(op=op, n_seq=n_seq, longest=longest, mix=mix, prefix=rng.choice([0, 0, 100, 777]), hq=hq, hk=hk, d=d,
                 causal=rng.random() < 0.7)
        return dict(c, train=rng.random() < 0.5) if op == "attn" else c
    if op == "paged":
        d, hq, hk = _heads(rng)
        batch = _log_int(rng, 1, 64)
        chunks = rng.choice([0, 0, 1, batch])
        ctx = _log_int(rng, 1, max(2, min(60000, int(4e8 / (batch * hk * d)))))
        longest = _log_int(rng, 1, max(2, min(1500, int(6e9 / (max(1, chunks) * hq * d * (ctx + 700)))))) if chunks else 1
        return dict(op=op, batch=batch, chunks=chunks, longest=longest, ctx=ctx, mix=mix, page=rng.choice([8, 16, 32, 64, 128, 256]),
                    hq=hq, hk=hk, d=d)
    if op == "tables":
        page = rng.choice([8, 16, 32, 64, 128])
        batch, ctx = _log_int(rng, 1, 1000), _log_int(rng, 1, 20000)
        new = _log_int(rng, 1, max(2, min(4000, 100000 // batch)))
        return dict(op=op, batch=batch, ctx=ctx, new=new, done=rng.choice([0.0, 0.05, 0.3]), mix=mix, page=page,
                    width=(ctx + new) // page + rng.randrange(1, 9))
    d, _, hk = _heads(rng)
    page = rng.choice([8, 16, 32, 64])
    tokens = _log_int(rng, 1, 16384)
    return dict(op=op, tokens=tokens, hk=hk, d=d, page=page, pages=tokens // page + rng.randrange(2, 300))


# ---------------------------------------------------------------------------------------- inputs
def _lengths(c):
    """(queries, keys) of each packed sequence: the longest first, the others between 1 and it, now and then none."""
    r = random.Random(c["mix"])
    n = [c["longest"]] * c["n_seq"]
    if c["mix"]:
        n = n[:1] + [0 if r.random() < 0.03 else _log_int(r, 1, c["longest"]) for _ in n[1:]]
    return n, [i + (r.randrange(c["prefix"] + 1) if c["prefix"] else 0) for i in n]


def _requests(c):
    """(new tokens, tokens with them) of each request of a cache."""
    r = random.Random(c["mix"])
    n = [_log_int(r, max(1, c["longest"] // 2), c["longest"]) if b < c["chunks"] else 1 for b in range(c["batch"])]
    if c["chunks"] == 1:
        n[0] = c["longest"]
    ctx = [r.randrange(c["ctx"] // 4, c["ctx"] + 1) if c["mix"] else c["ctx"] for _ in n]
    return n, [i + j for i, j in zip(n, ctx)]


def _growth(c):
    """(tokens before, tokens after) a step of each request: most grow, some are done and give their pages back."""
    r = random.Random(c["mix"])
    before = [r.randrange(c["ctx"] + 1) for _ in range(c["batch"])]
    return before, [0 if r.random() < c["done"] else b + (1 if c["new"] == 1 else r.randrange(c["new"] + 1)) for b in before]


def _sums(n):
    out = [0]
    for i in n:
        out.append(out[-1] + i)
    return out


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 31)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _projection(g, rows, heads, d):
    """q, k and v as views of one packed projection, with the spread of scores that trained heads have."""
    hq, hk = heads
    t = _normal(g, rows, hq + 2 * hk, d)
    t[:, :hq] *= torch.exp2(_normal(g, 1, hq, 1).clamp(-1.5, 1.5))
    t = t.to(torch.bfloat16)
    return t[:, :hq], t[:, hq : hq + hk], t[:, hq + hk :]


def _pages(n, page):
    return (n + page - 1) // page


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    s = {"case": c}
    b16 = torch.bfloat16
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] in ("attn", "grad"):
        nq, nk = _lengths(c)
        s["nq"], s["nk"] = nq, nk
        s["cu_q"], s["cu_k"] = _ints(_sums(nq)), _ints(_sums(nk))
        tq, tk = sum(nq), sum(nk)
        s["q"], s["k"], s["v"] = _projection(g, tk, (c["hq"], c["hk"]), c["d"])
        s["q"] = s["q"][:tq]
        s["out"], s["lse"] = new(tq, c["hq"], c["d"], dtype=b16), new(tq, c["hq"])
        if c["op"] == "grad":
            done = _plain_attn(dict(s, case=dict(c, train=True)))
            s["out"], s["lse"] = done["out"], done["lse"]
            s["dout"] = (0.01 * _normal(g, tq, c["hq"], c["d"])).to(b16)
            grads = new(tk, c["hq"] + 2 * c["hk"], c["d"], dtype=b16)  # the gradient of the packed projection
            s["dq"], s["dk"], s["dv"] = grads[:tq, : c["hq"]], grads[:, c["hq"] : c["hq"] + c["hk"]], grads[:, c["hq"] + c["hk"] :]
    elif c["op"] == "paged":
        n, total = _requests(c)
        s["n"], s["total"] = n, total
        s["cu_q"], s["kv_lens"] = _ints(_sums(n)), _ints(total)
        width, count = _pages(max(total), c["page"]), [_pages(t, c["page"]) for t in total]
        order = torch.randperm(sum(count) + 3, generator=g, device="cuda").to(torch.int32)
        s["tables"] = torch.full((c["batch"], width), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(width, device="cuda")[None, :] < _ints(count)[:, None]
        s["tables"][at] = order[: sum(count)]
        pages = sum(count) + 3
        for name in ("k_cache", "v_cache"):
            s[name] = new(pages, c["page"], c["hk"], c["d"], dtype=b16).normal_(generator=g)
            # what lies behind a request's last token is of no request
            last = s["tables"].gather(1, (_ints(count, torch.int64) - 1)[:, None])[:, 0].long()
            stale = torch.arange(c["page"], device="cuda")[None, :] >= (_ints(total) - (_ints(count) - 1) * c["page"])[:, None]
            s[name][last] = s[name][last].masked_fill(stale[:, :, None, None], float("nan"))
        s["q"] = _projection(g, sum(n), (c["hq"], c["hk"]), c["d"])[0]
        s["out"] = new(sum(n), c["hq"], c["d"], dtype=b16)
    elif c["op"] == "tables":
        before, after = _growth(c)
        s["before"], s["after"] = _ints(before), _ints(after)
        held = [_pages(b, c["page"]) for b in before]
        wanted = sum(max(0, _pages(a, c["page"]) - h) for a, h in zip(after, held))
        n_pages = sum(held) + wanted + 17
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        s["tables"] = torch.full((c["batch"], c["width"]), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(c["width"], device="cuda")[None, :] < _ints(held)[:, None]
        s["tables"][at] = order[: sum(held)]
        s["free"] = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][: n_pages - sum(held)] = order[sum(held) :]
        s["n_free"], s["n_free_out"] = _ints([n_pages - sum(held)]), _ints([0])
        total = sum(max(0, a - b) for a, b in zip(after, before))
        s["total"] = total
        s["cu"], s["short"] = _ints([0] * (c["batch"] + 1)), _ints([0, 0])
        s["positions"], s["slots"] = _ints([0] * total, torch.int64), _ints([0] * total, torch.int64)
    else:
        _, s["k"], s["v"] = _projection(g, c["tokens"], (4 * c["hk"], c["hk"]), c["d"])
        for name in ("k_cache", "v_cache"):
            s[name] = new(c["pages"], c["page"], c["hk"], c["d"], dtype=b16).normal_(generator=g)
        # tokens fill pages one after the other, the pages lie anywhere
        order = torch.randperm(c["pages"], generator=g, device="cuda")
        t = torch.arange(c["tokens"], device="cuda") + c["page"] // 2
        s["slots"] = order[t // c["page"]] * c["page"] + t % c["page"]
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _grouped(q, k, v):
    """Heads first, as float32: q [Hk, G n, d] (all rows that read one key head), k and v [Hk, m, d]."""
    n, hq, d = q.shape
    hk = k.shape[1]
    rows = q.float().view(n, hk, hq // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
    return rows, k.float().transpose(0, 1), v.float().transpose(0, 1)


def _hidden(n, m, groups, causal, dev):
    """Whether query row (g, i) does not see key j, [1, G n, m] (None where all see all)."""
    if not causal:
        return None
    i = torch.arange(n, device=dev)[:, None] + (m - n)
    return (torch.arange(m, device=dev)[None, :] > i).repeat(groups, 1)[None]


def _back(rows, n, groups):
    """[Hk, G n, d] to [n, Hq, d]."""
    hk, _, d = rows.shape
    return rows.view(hk, groups, n, d).permute(2, 0, 1, 3).reshape(n, hk * groups, d)


def _attend(q, k, v, causal):
    """One sequence: out [n, Hq, d] float32 and the logarithm of each row's sum [n, Hq]."""
    n, hq, d = q.shape
    groups = hq // k.shape[1]
    rows, keys, values = _grouped(q, k, v)
    scores = (rows @ keys.transpose(1, 2)).mul_(d**-0.5)
    hidden = _hidden(n, k.shape[0], groups, causal, q.device)
    if hidden is not None:
        scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return _back((p @ values) / total, n, groups), _back(top + total.log(), n, groups)[:, :, 0]


def _plain_attn(s):
    c = s["case"]
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    a = b = 0
    for n, m in zip(s["nq"], s["nk"]):
        if n:
            out[a : a + n], lse[a : a + n] = _attend(s["q"][a : a + n], s["k"][b : b + m], s["v"][b : b + m], c["causal"])
        a, b = a + n, b + m
    return {"out": out, "lse": lse} if c["train"] else {"out": out}


def _gradients(dout, q, k, v, out, lse, causal):
    """One sequence: dq [n, Hq, d], dk and dv [m, Hk, d] in float32 from the forward's output and row sums."""
    n, hq, d = q.shape
    groups, scale = hq // k.shape[1], d**-0.5
    rows, keys, values = _grouped(q, k, v)
    grad, sums = _grouped(dout, k, v)[0], _grouped(lse[:, :, None], k, v)[0]
    p = (rows @ keys.transpose(1, 2)).mul_(scale).sub_(sums).exp_()
    hidden = _hidden(n, k.shape[0], groups, causal, q.device)
    if hidden is not None:
        p.masked_fill_(hidden, 0.0)
    dot = (grad * _grouped(out, k, v)[0]).sum(-1, keepdim=True)
    dv = p.transpose(1, 2) @ grad
    ds = (grad @ values.transpose(1, 2)).sub_(dot).mul_(p).mul_(scale)
    return _back(ds @ keys, n, groups), (ds.transpose(1, 2) @ rows).transpose(0, 1), dv.transpose(0, 1)


def _plain_grad(s):
    c = s["case"]
    dq, dk, dv = torch.empty_like(s["dq"]), torch.zeros_like(s["dk"]), torch.zeros_like(s["dv"])
    a = b = 0
    for n, m in zip(s["nq"], s["nk"]):
        if n:
            x, y = slice(a, a + n), slice(b, b + m)
            dq[x], dk[y], dv[y] = _gradients(s["dout"][x], s["q"][x], s["k"][y], s["v"][y], s["out"][x], s["lse"][x], c["causal"])
        a, b = a + n, b + m
    return {"dq": dq, "dk": dk, "dv": dv}


def _plain_paged(s):
    c = s["case"]
    out = torch.empty_like(s["out"])
    a = 0
    for b, (n, m) in enumerate(zip(s["n"], s["total"])):
        pages = s["tables"][b, : _pages(m, c["page"])].long()
        k, v = s["k_cache"][pages].flatten(0, 1)[:m], s["v_cache"][pages].flatten(0, 1)[:m]
        out[a : a + n] = _attend(s["q"][a : a + n], k, v, True)[0]
        a += n
    return {"out": out}


def _plain_tables(s):
    c = s["case"]
    page, before, after = c["page"], s["before"].long(), s["after"].long()
    held, need = (before + page - 1) // page, (after + page - 1) // page
    gained, lost = (need - held).clamp(min=0), (held - need).clamp(min=0)
    col = torch.arange(c["width"], device=held.device)[None, :]
    free, tables, n_free = s["free"].clone(), s["tables"].clone(), s["n_free"].long()
    # pages given back lie on top of the free ones, in the order of requests and of their pages
    back = (col >= need[:, None]) & (col < held[:, None])
    at = n_free + (lost.cumsum(0) - lost)[:, None] + col - need[:, None]
    ends = torch.cat((free, free.new_zeros(1)))  # one place for what is not given back
    ends.scatter_(0, torch.where(back, at, free.numel()).flatten(), tables.flatten())
    free = ends[:-1]
    top = n_free + lost.sum()
    # pages wanted come from the top, in the same order
    take = (col >= held[:, None]) & (col < need[:, None])
    at = top - 1 - ((gained.cumsum(0) - gained)[:, None] + col - held[:, None])
    tables = torch.where(take, free[torch.where(take, at, 0).clamp(min=0)], tables)
    tokens = (after - before).clamp(min=0)
    cu = torch.cat((tokens.new_zeros(1), tokens.cumsum(0)))
    t = torch.arange(s["total"], device=held.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    positions = before[b] + t - cu[b]
    slots = tables[b, positions // page].long() * page + positions % page
    return {"tables": tables, "free": free, "n_free": (top - gained.sum()).int(), "cu": cu.int(), "positions": positions,
            "slots": slots, "short": torch.zeros_like(s["short"])}


def _plain_write(s):
    for name, x in (("k_cache", s["k"]), ("v_cache", s["v"])):
        s[name].view(-1, *x.shape[1:])[s["slots"]] = x
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


PLAIN = {"attn": _plain_attn, "grad": _plain_grad, "paged": _plain_paged, "tables": _plain_tables, "write": _plain_write}


# ---------------------------------------------------------------------------------------- the framework's calls
def _own(s):
    from diffusion_transformer_flux_gb300 import _lib as L

    c = s["case"]
    if c["op"] == "attn":
        if "ws" not in s:
            s["ws"] = L.workspace(L.mmdit_varlen_attention_workspace_size(s["q"].shape[0], c["hq"], c["d"]))
        L.mmdit_varlen_attention_fwd(s["q"], s["k"], s["v"], s["out"], s["cu_q"], cu_k=s["cu_k"], causal=c["causal"],
                                     lse=s["lse"] if c["train"] else None, ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]} if c["train"] else {"out": s["out"]}
    if c["op"] == "grad":
        if "ws" not in s:
            s["ws"] = L.workspace(L.mmdit_varlen_attention_bwd_workspace_size(s["q"].shape[0], c["hq"], c["d"]))
        L.mmdit_varlen_attention_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["dq"], s["dk"], s["dv"],
                                     s["cu_q"], cu_k=s["cu_k"], causal=c["causal"], ws=s["ws"])
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    if c["op"] == "paged":
        longest, reach = max(s["n"]), max(s["total"])
        if "ws" not in s:
            s["ws"] = L.workspace(L.mmdit_paged_attention_workspace_size(s["q"].shape[0], c["batch"], c["hq"], c["hk"], c["d"],
                                                                         longest, reach))
        L.mmdit_paged_attention_fwd(s["q"], s["k_cache"], s["v_cache"], s["out"], s["tables"], s["kv_lens"], s["cu_q"],
                                    max_q=longest, max_kv=reach, ws=s["ws"])
        return {"out": s["out"]}
    if c["op"] == "tables":
        L.mmdit_block_tables(s["before"], s["after"], s["tables"], s["free"], s["n_free"], c["page"], s["n_free_out"], s["cu"],
                             s["positions"], s["slots"], s["short"])
        return {"tables": s["tables"], "free": s["free"], "n_free": s["n_free_out"], "cu": s["cu"], "positions": s["positions"],
                "slots": s["slots"], "short": s["short"]}
    L.mmdit_kv_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------- float64 definitions
def _softmax64(q, k, first):
    """Weights and row logarithms of query rows [n, d] that stand at first, first + 1, ... (None: see all keys)."""
    z = torch.einsum("id,jd->ij", q, k) / math.sqrt(q.shape[1])
    if first is not None:
        pos = first + torch.arange(q.shape[0], device=q.device)
        z = torch.where(torch.arange(k.shape[0], device=q.device) <= pos[:, None], z, torch.full_like(z, -math.inf))
    return torch.softmax(z, 1), torch.logsumexp(z, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "tables":
        return None  # whole numbers
    if c["op"] == "write":
        out = {}
        for name, x in (("k_cache", s["k"]), ("v_cache", s["v"])):
            page, slot = s["slots"] // c["page"], s["slots"] % c["page"]
            out[name] = s[name].double().index_put((page, slot), x.double())
        return out
    group = c["hq"] // c["hk"]
    if c["op"] == "grad":
        dq, dk, dv = (torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("dq", "dk", "dv"))
        a = b = 0
        for n, m in zip(s["nq"], s["nk"]):
            for h in range(c["hq"] if n else 0):
                q, k, v = (s[x][y, z].double() for x, y, z in (("q", slice(a, a + n), h), ("k", slice(b, b + m), h // group),
                                                               ("v", slice(b, b + m), h // group)))
                g, o = s["dout"][a : a + n, h].double(), s["out"][a : a + n, h].double()
                p, _ = _softmax64(q, k, m - n if c["causal"] else None)
                # dL/dz_ij = p_ij (g_i . v_j - g_i . o_i)
                dz = p * (torch.einsum("id,jd->ij", g, v) - torch.einsum("id,id->i", g, o)[:, None]) / math.sqrt(c["d"])
                dq[a : a + n, h] = dz @ k
                dk[b : b + m, h // group] += torch.einsum("ij,id->jd", dz, q)
                dv[b : b + m, h // group] += torch.einsum("ij,id->jd", p, g)
            a, b = a + n, b + m
        return {"dq": dq, "dk": dk, "dv": dv}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    a = b = 0
    for i, (n, m) in enumerate(zip(s["nq"], s["nk"]) if c["op"] == "attn" else zip(s["n"], s["total"])):
        if c["op"] == "paged":
            at = torch.arange(m, device="cuda")
            page, slot = s["tables"][i].long()[at // c["page"]], at % c["page"]
            keys, values = s["k_cache"][page, slot], s["v_cache"][page, slot]
        else:
            keys, values = s["k"][b : b + m], s["v"][b : b + m]
        for h in range(c["hq"] if n else 0):
            p, lse[a : a + n, h] = _softmax64(s["q"][a : a + n, h].double(), keys[:, h // group].double(),
                                              m - n if c["op"] == "paged" or c["causal"] else None)
            out[a : a + n, h] = p @ values[:, h // group].double()
        a, b = a + n, b + m
    return {"out": out, "lse": lse} if c["op"] == "attn" and c["train"] else {"out": out}


# ---------------------------------------------------------------------------------------- floors
def work(case):
    c = case
    if c["op"] in ("attn", "grad", "paged"):
        nq, nk = _requests(c) if c["op"] == "paged" else _lengths(c)
        tq, tk = sum(nq), sum(m for n, m in zip(nq, nk) if n)
        causal = c["op"] == "paged" or c["causal"]
        pairs = sum(n * (m - n) + n * (n + 1) // 2 if causal else n * m for n, m in zip(nq, nk))
        q, kv = 2 * tq * c["hq"] * c["d"], 2 * tk * c["hk"] * c["d"]
        if c["op"] == "grad":  # q, out, dout, lse and k, v in, dq, dk, dv out; five products
            return {"bytes": 4 * q + 4 * kv + 4 * tq * c["hq"], "flops": 10 * pairs * c["hq"] * c["d"]}
        sums = 4 * tq * c["hq"] if c.get("train") else 4 * sum(_pages(m, c["page"]) for m in nk) if c["op"] == "paged" else 0
        return {"bytes": 2 * q + 2 * kv + sums, "flops": 4 * pairs * c["hq"] * c["d"]}
    if c["op"] == "tables":
        before, after = _growth(c)
        moved = sum(abs(_pages(a, c["page"]) - _pages(b, c["page"])) for a, b in zip(after, before))
        tokens = sum(max(0, a - b) for a, b in zip(after, before))
        return {"bytes": 8 * moved + 16 * tokens + 12 * c["batch"], "flops": 0}
    return {"bytes": 8 * c["tokens"] * c["hk"] * c["d"] + 8 * c["tokens"], "flops": 0}
