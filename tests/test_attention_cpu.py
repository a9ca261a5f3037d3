"""Refusals of the text model's attention and cache: every argument check answers before CUDA is touched."""
import ctypes as C

import pytest
import torch

from diffusion_transformer_flux_gb300 import _lib as L
from diffusion_transformer_flux_gb300 import build_ext

A, B_, C_, D_, E_, F_, G_, H_, I_, J_, K_ = (0x100000 * i for i in range(1, 12))  # aligned addresses that nothing reads
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return L.load()


def heads(ptr, st=512, sh=128):
    return None if ptr is None else C.byref(L.HeadsView(ptr, st, sh))


def pages(ptr, sp=4096, st=256, sh=128):
    return None if ptr is None else C.byref(L.PagesView(ptr, sp, st, sh))


def _fwd(lib, batch=2, tq=64, tk=64, hq=4, hk=2, d=128, scale=0.1, q=heads(A), k=heads(B_, 256), v=heads(C_, 256), cu_q=D_,
         cu_k=D_, out=heads(E_), lse=F_, ws=G_, ws_bytes=1 << 30):
    return lib.mmdit_varlen_attention_fwd(batch, tq, tk, hq, hk, d, 1, scale, q, k, v, cu_q, cu_k, out, lse, ws, ws_bytes, None)


VIEWS = [
    (INVALID, None), (INVALID, heads(A + 8)), (INVALID, heads(A, 516)), (INVALID, heads(A, 512, 124)), (INVALID, heads(A, 64)),
    (INVALID, heads(A, 512, 0)), (INVALID, heads(A, -512)), (INVALID, heads(A, (1 << 36) + 8)),
]


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(batch=-1)), (INVALID, dict(tq=-1)), (INVALID, dict(tk=-1)), (INVALID, dict(hq=0)), (INVALID, dict(hk=0)),
    (INVALID, dict(d=0)), (INVALID, dict(hq=5)), (UNSUPPORTED, dict(d=132)), (UNSUPPORTED, dict(d=136)),
    (UNSUPPORTED, dict(d=100)), (UNSUPPORTED, dict(hq=258)), (UNSUPPORTED, dict(hq=65536, hk=65536)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (UNSUPPORTED, dict(tq=(1 << 30) + 1)), (UNSUPPORTED, dict(batch=(1 << 20) + 1)), (UNSUPPORTED, dict(tq=1 << 30, hq=1024, hk=1024)),
    (INVALID, dict(cu_q=None)), (INVALID, dict(cu_k=None)), (INVALID, dict(cu_q=D_ + 2)), (INVALID, dict(lse=F_ + 2)),
    (INVALID, dict(out=heads(A))), (INVALID, dict(out=heads(B_))), (INVALID, dict(out=heads(C_))),
    (INVALID, dict(out=heads(E_, 256))), (INVALID, dict(out=heads(E_, 128, 128))), (INVALID, dict(v=None)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=16)), (WORKSPACE, dict(ws=G_ + 16)),
] + [(s, dict(q=view)) for s, view in VIEWS])
def test_varlen_refusals(lib, status, kw):
    assert _fwd(lib, **kw) == status and (status == WORKSPACE or "varlen attention" in L.last_error())


def test_varlen_empty(lib):
    assert _fwd(lib, batch=0, q=None, k=None, v=None, out=None, cu_q=None, cu_k=None) == 0
    assert _fwd(lib, tq=0, q=None, k=None, v=None, out=None, cu_q=None, cu_k=None) == 0


def _bwd(lib, batch=2, tq=64, tk=64, hq=4, hk=2, d=128, scale=0.1, dout=heads(A), q=heads(B_), k=heads(C_, 256), v=heads(D_, 256),
         out=heads(E_), lse=F_, cu_q=G_, cu_k=G_, dq=heads(H_), dk=heads(I_, 256), dv=heads(J_, 256), ws=K_, ws_bytes=1 << 30):
    return lib.mmdit_varlen_attention_bwd(batch, tq, tk, hq, hk, d, 1, scale, dout, q, k, v, out, lse, cu_q, cu_k, dq, dk, dv, ws,
                                          ws_bytes, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(batch=-1)), (INVALID, dict(hq=3)), (UNSUPPORTED, dict(d=20)), (UNSUPPORTED, dict(hq=130)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(lse=None)), (INVALID, dict(lse=F_ + 1)), (INVALID, dict(cu_k=None)),
    (INVALID, dict(dout=None)), (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(out=None)),
    (INVALID, dict(dq=None)), (INVALID, dict(dk=None)), (INVALID, dict(dv=None)), (INVALID, dict(dk=heads(I_, 128))),
    (INVALID, dict(dq=heads(A))), (INVALID, dict(dq=heads(B_))), (INVALID, dict(dq=heads(C_))), (INVALID, dict(dq=heads(D_))),
    (INVALID, dict(dq=heads(E_))), (INVALID, dict(dk=heads(C_, 256))), (INVALID, dict(dk=heads(D_, 256))),
    (INVALID, dict(dv=heads(I_, 256))), (INVALID, dict(dk=heads(H_, 256))), (INVALID, dict(dv=heads(E_, 256))),
    (INVALID, dict(dv=heads(A, 256))), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=1024)),
])
def test_varlen_bwd_refusals(lib, status, kw):
    assert _bwd(lib, **kw) == status and (status == WORKSPACE or "varlen attention backward" in L.last_error())


def test_varlen_bwd_empty(lib):
    assert _bwd(lib, batch=0) == 0 and _bwd(lib, tq=0, tk=0) == 0


def _paged(lib, batch=2, tq=4, hq=4, hk=2, d=128, scale=0.1, q=heads(A), k=pages(B_), v=pages(C_), n_pages=8, page=16, tables=D_,
           width=4, lens=E_, cu_q=F_, max_q=1, max_kv=64, out=heads(G_), lse=H_, ws=I_, ws_bytes=1 << 30):
    return lib.mmdit_paged_attention_fwd(batch, tq, hq, hk, d, scale, q, k, v, n_pages, page, tables, width, lens, cu_q, max_q,
                                         max_kv, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(batch=-1)), (INVALID, dict(tq=-1)), (INVALID, dict(hq=3)), (UNSUPPORTED, dict(d=12)), (INVALID, dict(scale=0.0)),
    (INVALID, dict(page=0)), (INVALID, dict(n_pages=-1)), (INVALID, dict(n_pages=0)), (UNSUPPORTED, dict(page=4)),
    (UNSUPPORTED, dict(page=24)), (UNSUPPORTED, dict(page=1 << 21)), (UNSUPPORTED, dict(n_pages=(1 << 30) + 1)),
    (INVALID, dict(width=0)), (INVALID, dict(max_q=-1)), (INVALID, dict(max_kv=-1)), (UNSUPPORTED, dict(width=1 << 27)),
    (UNSUPPORTED, dict(batch=1 << 20, width=1 << 26, max_kv=0)), (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (INVALID, dict(out=None)), (INVALID, dict(k=pages(B_ + 8))), (INVALID, dict(k=pages(B_, 4100))), (INVALID, dict(v=pages(C_, 4096, 64))),
    (INVALID, dict(v=pages(C_, 4096, 256, 132))), (INVALID, dict(out=heads(A))), (INVALID, dict(out=heads(B_))),
    (INVALID, dict(out=heads(G_, 128))), (INVALID, dict(tables=None)), (INVALID, dict(lens=None)), (INVALID, dict(cu_q=None)),
    (INVALID, dict(tables=D_ + 2)), (INVALID, dict(lens=E_ + 1)), (INVALID, dict(lse=H_ + 2)), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(max_kv=0, width=1 << 20, ws_bytes=4096)),
])
def test_paged_refusals(lib, status, kw):
    assert _paged(lib, **kw) == status and (status == WORKSPACE or "paged attention" in L.last_error())


def test_paged_empty(lib):
    assert _paged(lib, batch=0) == 0 and _paged(lib, tq=0) == 0 and _paged(lib, max_q=0) == 0


def test_paged_workspace_covers_what_the_call_splits():
    """A call with fewer tokens or keys than the workspace was made for never asks for more."""
    size = L.mmdit_paged_attention_workspace_size
    for batch, hq, hk, d, max_q in ((1, 32, 8, 128, 1), (64, 32, 8, 128, 1), (8, 28, 4, 64, 4), (3, 4, 4, 96, 700)):
        sizes = [size(batch * max_q, batch, hq, hk, d, max_q, kv) for kv in (1, 512, 513, 4096, 100000)]
        assert all(s >= 256 for s in sizes) and max(sizes) < 1 << 32
    assert size(0, 4, 8, 8, 64, 1, 64) == size(4, 0, 8, 8, 64, 1, 64) == 256


def _tables(lib, batch=4, page=16, width=8, n_pages=32, before=A, after=B_, tables=C_, free=D_, n_free=E_, n_free_out=F_, cu=G_,
            cap=64, positions=H_, slots=I_, missing=J_):
    return lib.mmdit_block_tables(batch, page, width, n_pages, before, after, tables, free, n_free, n_free_out, cu, cap, positions,
                                  slots, missing, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(page=0)), (UNSUPPORTED, dict(page=12)), (INVALID, dict(n_pages=-1)), (INVALID, dict(batch=-1)),
    (INVALID, dict(width=0)), (INVALID, dict(cap=-1)), (UNSUPPORTED, dict(batch=1 << 20, width=1 << 11)),
    (UNSUPPORTED, dict(width=1 << 27)), (INVALID, dict(before=None)), (INVALID, dict(after=None)), (INVALID, dict(tables=None)),
    (INVALID, dict(free=None)), (INVALID, dict(n_free=None)), (INVALID, dict(n_free_out=None)), (INVALID, dict(cu=None)),
    (INVALID, dict(missing=None)), (INVALID, dict(before=A + 2)), (INVALID, dict(cu=G_ + 1)), (INVALID, dict(positions=H_ + 4)),
    (INVALID, dict(slots=I_ + 4)), (INVALID, dict(cu=A)), (INVALID, dict(tables=B_)), (INVALID, dict(missing=E_)),
    (INVALID, dict(slots=H_)), (INVALID, dict(cu=C_)), (INVALID, dict(n_free_out=D_)),
])
def test_block_tables_refusals(lib, status, kw):
    assert _tables(lib, **kw) == status and "block tables" in L.last_error()


def _write(lib, tokens=4, hk=2, d=128, k=heads(A, 256), v=heads(B_, 256), kc=pages(C_), vc=pages(D_), n_pages=8, page=16, slots=E_):
    return lib.mmdit_kv_cache_write(tokens, hk, d, k, v, kc, vc, n_pages, page, slots, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(tokens=-1)), (INVALID, dict(hk=0)), (INVALID, dict(d=0)), (UNSUPPORTED, dict(d=20)), (UNSUPPORTED, dict(d=520)),
    (UNSUPPORTED, dict(page=10)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(kc=None)), (INVALID, dict(vc=None)),
    (INVALID, dict(k=heads(A + 2, 256))), (INVALID, dict(kc=pages(C_, 4096, 128))), (INVALID, dict(vc=pages(D_, 256))),
    (INVALID, dict(kc=pages(D_))), (INVALID, dict(kc=pages(A))), (INVALID, dict(vc=pages(A))), (INVALID, dict(slots=None)),
    (INVALID, dict(slots=E_ + 4)),
])
def test_cache_write_refusals(lib, status, kw):
    assert _write(lib, **kw) == status and "cache write" in L.last_error()


def test_cache_write_empty(lib):
    assert _write(lib, tokens=0, k=None, v=None) == 0 and _write(lib, n_pages=0, kc=None, vc=None) == 0


def test_bindings_refuse_host_tensors(lib):
    x, c, i = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    lse = torch.zeros(2, 2)
    for call in (lambda: L.mmdit_varlen_attention_fwd(x, x, x, x, i), lambda: L.mmdit_varlen_attention_bwd(x, x, x, x, x, lse, x, x, x, i),
                 lambda: L.mmdit_paged_attention_fwd(x, c, c, x, i.view(1, 2), i[:1], i), lambda: L.mmdit_kv_cache_write(x, x, c, c, i.long()),
                 lambda: L.mmdit_block_tables(i, i, i.view(2, 1), i, i[:1], 16, i[:1], i, None, None, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_view_checks():
    """The shape, type and layout checks of the binding's views, on host tensors of a host `device`."""
    dev = torch.device("cpu")
    x = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    v = L._heads_view("x", x[:, :2], dev, 4, 2, 64)
    assert (v.ptr, v.stride_t, v.stride_h) == (x.data_ptr(), 384, 64)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    p = L._pages_view("c", c.transpose(1, 2).contiguous().transpose(1, 2), dev, c.shape)
    assert (p.stride_page, p.stride_t, p.stride_h) == (2048, 64, 1024)
    with pytest.raises(TypeError, match="dtype"):
        L._heads_view("x", x.float(), dev)
    with pytest.raises(TypeError, match="dtype"):
        L._pages_view("c", c.half(), dev)
    with pytest.raises(ValueError, match="adjacent"):
        L._heads_view("x", x.transpose(1, 2), dev)
    with pytest.raises(ValueError, match="adjacent"):
        L._pages_view("c", c.transpose(2, 3), dev)
    for bad in (dict(tokens=5), dict(heads=4), dict(d=128)):
        with pytest.raises(ValueError, match="shape"):
            L._heads_view("x", x, dev, **bad)
    with pytest.raises(ValueError, match="shape"):
        L._pages_view("c", c, dev, heads=3)
    with pytest.raises(ValueError, match="shape"):
        L._heads_view("x", c, dev)
    with pytest.raises(ValueError, match="meta"):
        L._heads_view("x", x, torch.device("meta"))


def test_varlen_bwd_workspace_serves_smaller_calls(lib):
    """It never shrinks as a call grows, also past 16384 queries."""
    size = L.mmdit_varlen_attention_bwd_workspace_size
    for heads, d in ((1, 64), (4, 8), (32, 128), (24, 64), (128, 128)):
        sizes = [size(t, heads, d) for t in (0, 1, 7, 128, 1000, 2048, 4096, 8191, 8192, 16383, 16384, 16385, 20000, 65536, 1 << 20)]
        assert sizes == sorted(sizes)
        assert sizes[1] >= 256 + 8 * heads
    assert [size(5000, h, 64) for h in (1, 2, 3, 16)] == sorted(size(5000, h, 64) for h in (1, 2, 3, 16))
    assert size(5000, 8, 64) <= size(5000, 8, 72) == size(5000, 8, 128)


# (tokens, batch, heads_q, heads_k, head_dim, max_q, max_kv) of calls that grow; each serves all before it
GROWING = [
    [(1, 1, 32, 8, 128, 1, 100), (1, 1, 32, 8, 128, 1, 32000), (300, 1, 32, 8, 128, 300, 32000), (1000, 1, 32, 8, 128, 1000, 32000),
     (4096, 1, 32, 8, 128, 4096, 32000), (8192, 1, 32, 8, 128, 8192, 32000), (8192, 1, 32, 8, 128, 8192, 200000)],
    [(8, 8, 28, 4, 64, 1, 500), (40, 40, 28, 4, 64, 1, 5000), (371, 40, 28, 4, 64, 333, 5000), (6000, 40, 28, 4, 64, 6000, 5000)],
    [(64, 64, 16, 1, 96, 1, 600), (64, 64, 16, 1, 96, 64, 16384), (2600, 64, 16, 1, 96, 700, 16384), (20000, 64, 16, 1, 96, 20000, 16384)],
]


@pytest.mark.parametrize("calls", GROWING)
def test_paged_workspace_serves_smaller_calls(lib, calls):
    """What a call asks for is enough for every call of fewer tokens, requests and keys, whatever these would ask for."""
    size = L.mmdit_paged_attention_workspace_size
    for i, large in enumerate(calls):
        for t, b, hq, hk, d, max_q, max_kv in calls[:i + 1]:
            kw = dict(batch=b, tq=t, hq=hq, hk=hk, d=d, max_q=max_q, max_kv=max_kv, width=1 << 14, ws_bytes=size(*large))
            # the check of q comes behind the workspace's
            assert _paged(lib, q=None, **kw) == INVALID and "q is NULL" in L.last_error(), (large, kw)
    for t, b, hq, hk, d, max_q, max_kv in calls:
        kw = dict(batch=b, tq=t, hq=hq, hk=hk, d=d, max_q=max_q, max_kv=max_kv, width=1 << 14)
        assert _paged(lib, q=None, ws_bytes=0, **kw) == WORKSPACE


@pytest.mark.parametrize("call", [_fwd, _bwd, _paged])
def test_scales_outside_float32_reach(lib, call):
    """1 / (scale log2(e)) times a log-sum, as the gradients form it, would overflow; 2^-100 and 2^100 pass to the next check."""
    for scale in (1e-40, 1e-38, 2.0 ** -101, 2.0 ** 101, 3e38):
        assert call(lib, scale=scale) == UNSUPPORTED and "2^-100" in L.last_error()
    for scale in (2.0 ** -100, 2.0 ** 100):
        assert call(lib, scale=scale, q=None) == INVALID and "q is NULL" in L.last_error()


def test_varlen_bwd_refuses_too_many_items_before_it_starts(lib):
    """Tiles of 128 rows of queries or of keys by key heads, counted in 31 bits with room for one more of each sequence."""
    for tq, tk in ((1 << 24, 128), (128, 1 << 24)):
        kw = dict(batch=1 << 20, tq=tq, tk=tk, hq=960, hk=960, d=8)
        views = dict(dout=heads(A, 8 * kw["hq"], 8), q=heads(B_, 8 * kw["hq"], 8), k=heads(C_, 8 * kw["hk"], 8), v=heads(D_, 8 * kw["hk"], 8),
                     out=heads(E_, 8 * kw["hq"], 8), dq=heads(H_, 8 * kw["hq"], 8), dk=heads(I_, 8 * kw["hk"], 8), dv=heads(J_, 8 * kw["hk"], 8))
        # lse NULL is refused behind the shapes: this call never starts
        few = dict(kw, batch=1 << 10)
        assert _bwd(lib, ws_bytes=1 << 40, lse=None, **few, **views) == INVALID
        assert _bwd(lib, ws_bytes=1 << 40, lse=None, **kw, **views) == UNSUPPORTED and "too many tiles" in L.last_error()
