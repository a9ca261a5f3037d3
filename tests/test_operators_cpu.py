"""Refusals of the language-model operators: every argument check answers before CUDA is touched."""
import ctypes as C

import pytest
import torch

from diffusion_transformer_flux_gb300 import _lib as L
from diffusion_transformer_flux_gb300 import build_ext

A, B_, C_, D_, E_, F_ = (0x10000 * i for i in range(1, 7))  # aligned addresses that nothing reads
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return L.load()


def _norm(lib, act=1, res_f32=0, rows=4, dim=256, eps=1e-6, x=A, ldx=None, res=B_, gain=C_, h=D_, y=E_, y_q=None,
          s_y=None, rstd=None):
    return lib.mmdit_add_rmsnorm_fwd(act, res_f32, rows, dim, eps, x, dim if ldx is None else ldx, res, gain, h, y, y_q,
                                     s_y, rstd, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(act=2)), (INVALID, dict(rows=-1)), (INVALID, dict(dim=0)), (UNSUPPORTED, dict(dim=252)),
    (UNSUPPORTED, dict(dim=16392)), (UNSUPPORTED, dict(dim=264, y_q=F_, s_y=A)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(ldx=128)), (INVALID, dict(ldx=260)), (INVALID, dict(x=None)),
    (INVALID, dict(x=A + 8)), (INVALID, dict(gain=None)), (INVALID, dict(res=B_ + 4)), (INVALID, dict(h=D_ + 2)),
    (INVALID, dict(res=None)), (INVALID, dict(y=None)), (INVALID, dict(y_q=F_)), (INVALID, dict(s_y=F_)),
    (INVALID, dict(y=A)), (INVALID, dict(y=B_)), (INVALID, dict(y_q=A, s_y=F_)), (INVALID, dict(y_q=E_, s_y=F_)), (INVALID, dict(h=A)), (INVALID, dict(h=E_)),
])
def test_norm_refusals(lib, status, kw):
    assert _norm(lib, **kw) == status and "RMSNorm" in L.last_error()


def test_norm_empty(lib):
    assert _norm(lib, rows=0, x=None, res=None, gain=None, h=None, y=None) == 0


def _norm_bwd(lib, act=1, res_f32=0, rows=4, dim=256, dy=A, h=B_, gain=C_, rstd=0x1004, dh_in=None, dh=D_, dx=None,
              dgain=None, ws=F_, ws_bytes=1 << 30):
    return lib.mmdit_add_rmsnorm_bwd(act, res_f32, rows, dim, dy, h, gain, rstd, dh_in, dh, dx, dgain, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(act=7)), (UNSUPPORTED, dict(dim=12)), (INVALID, dict(rstd=None)), (INVALID, dict(dy=None)),
    (INVALID, dict(dh=None)), (INVALID, dict(dh=A)), (INVALID, dict(dh=B_)), (INVALID, dict(dx=D_)),
    (INVALID, dict(dx=A)), (INVALID, dict(dx=E_, dh_in=E_)), (INVALID, dict(dgain=0x2008)), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(ws=F_ + 16)), (WORKSPACE, dict(ws_bytes=512)),
])
def test_norm_bwd_refusals(lib, status, kw):
    assert _norm_bwd(lib, **kw) == status


def _cast(lib, act=1, square=0, rows=100, cols=128, x=A, q=B_, s=C_, q_t=D_, s_t=E_):
    return lib.mmdit_fp8_block_cast(act, square, rows, cols, x, q, s, q_t, s_t, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(act=3)), (INVALID, dict(square=2)), (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)),
    (UNSUPPORTED, dict(cols=120)), (INVALID, dict(x=None)), (INVALID, dict(x=A + 8)), (INVALID, dict(q=None, q_t=None)),
    (INVALID, dict(q=B_ + 8)), (INVALID, dict(q_t=D_ + 8)), (INVALID, dict(s=None)), (INVALID, dict(s_t=None)),
    (INVALID, dict(q_t=None)), (INVALID, dict(square=1)), (INVALID, dict(square=1, s=None, s_t=None, q=None)),
    (UNSUPPORTED, dict(rows=(1 << 30) + 1)),
])
def test_cast_refusals(lib, status, kw):
    assert _cast(lib, **kw) == status and "block cast" in L.last_error()


def test_cast_empty(lib):
    assert _cast(lib, rows=0, x=None) == 0


def _linear(lib, M=4, N=128, K=256, x=A, s_x=0x1004, w=B_, s_w=0x2004, b=None, y=C_, y_f32=0, ws=F_, ws_bytes=256):
    return lib.mmdit_fp8_block_linear_fwd(M, N, K, x, s_x, w, s_w, b, y, y_f32, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=0)), (UNSUPPORTED, dict(N=12)),
    (UNSUPPORTED, dict(K=120)), (UNSUPPORTED, dict(M=(1 << 30) + 1)), (UNSUPPORTED, dict(N=(1 << 22) + 8)), (UNSUPPORTED, dict(K=(1 << 22) + 16)),
    (INVALID, dict(x=None)), (INVALID, dict(x=A + 8)), (INVALID, dict(w=None)), (INVALID, dict(y=C_ + 2)),
    (INVALID, dict(s_x=None)), (INVALID, dict(s_w=None)), (INVALID, dict(b=D_ + 2)), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(ws_bytes=255)), (WORKSPACE, dict(ws=F_ + 128)),
])
def test_linear_refusals(lib, status, kw):
    assert _linear(lib, **kw) == status


def test_linear_empty(lib):
    assert _linear(lib, M=0, x=None, w=None, y=None, s_x=None, s_w=None) == 0


def _linear_bwd(lib, M=4, N=128, K=256, dy=A, w_t=B_, s_w=0x1004, x_t=C_, s_xt=0x2004, dx=D_, dw=E_, db=0x7000,
                ws=F_, ws_bytes=1 << 30):
    return lib.mmdit_fp8_block_linear_bwd(M, N, K, dy, w_t, s_w, x_t, s_xt, dx, dw, db, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(N=-8)), (UNSUPPORTED, dict(N=4)), (UNSUPPORTED, dict(K=8)), (INVALID, dict(dy=None)),
    (INVALID, dict(w_t=None)), (INVALID, dict(s_w=None)), (INVALID, dict(x_t=C_ + 8)), (INVALID, dict(s_xt=None)),
    (INVALID, dict(dx=None, dw=None, db=None)), (INVALID, dict(dw=E_ + 4)), (INVALID, dict(db=0x7004)),
    (INVALID, dict(dx=D_ + 8)), (WORKSPACE, dict(ws_bytes=1024)), (WORKSPACE, dict(ws=None)),
])
def test_linear_bwd_refusals(lib, status, kw):
    assert _linear_bwd(lib, **kw) == status


def test_workspace_sizes(lib):
    assert L.mmdit_fp8_block_linear_workspace_size(4096, 4096, 4096) == 256
    # both casts of dy, their scales and the column sums
    M, N = 1000, 264
    floor = M * 272 + 3 * M * 4 + N * 1008 + 2 * (8 * N * 4)
    assert floor <= L.mmdit_fp8_block_linear_bwd_workspace_size(M, N, 512) <= floor + 256 * 6
    assert L.mmdit_fp8_block_linear_bwd_workspace_size(0, N, 512) == 256
    assert L.mmdit_add_rmsnorm_bwd_workspace_size(0, 64) == 256
    # at least one CTA's sums of dgain, at most one row's per row
    assert 256 + 64 * 4 <= L.mmdit_add_rmsnorm_bwd_workspace_size(3, 64) <= 256 + 3 * 64 * 4
    assert L.mmdit_add_rmsnorm_bwd_workspace_size(1 << 20, 4096) < 64 << 20


def _cfg(lib, rot=64, inter=1, theta=1e4, scaling=0, factor=1.0, orig=0.0, low=1.0, high=4.0, mscale=1.0):
    cfg = L.RopeCfg()
    return lib.mmdit_rope_config(C.byref(cfg), rot, inter, theta, scaling, factor, orig, low, high, mscale), cfg


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(rot=0)), (UNSUPPORTED, dict(rot=33)), (UNSUPPORTED, dict(rot=514)), (INVALID, dict(theta=0.5)),
    (INVALID, dict(theta=float("inf"))), (INVALID, dict(scaling=3)), (INVALID, dict(scaling=-1)),
    (INVALID, dict(scaling=1, factor=0.5)), (INVALID, dict(scaling=2, factor=2.0)),
    (INVALID, dict(scaling=2, factor=2.0, orig=100.0, low=4.0)), (INVALID, dict(mscale=float("nan"))),
])
def test_rope_config_refusals(lib, status, kw):
    assert _cfg(lib, **kw)[0] == status


def test_rope_config_turns(lib):
    """turns[j] is f_j / 2 pi in units of 2^-64, to a double's rounding."""
    import math

    from oracle import lm
    for kw, args in ((dict(), dict()), (dict(scaling=1, factor=8.0), dict(scaling="linear", factor=8.0)),
                     (dict(scaling=2, factor=8.0, orig=4096.0, high=32.0),
                      dict(scaling="by_parts", factor=8.0, orig_len=4096.0, high=32.0))):
        st, cfg = _cfg(lib, **kw)
        assert st == 0 and cfg.rot_dim == 64 and cfg.interleaved == 1
        f = lm.rope_frequencies(64, **args)
        for j in range(32):
            # a whole number: less than one unit below, beside the double's own rounding
            assert cfg.turns[j] == pytest.approx(f[j] / (2 * math.pi) * 2.0 ** 64, rel=1e-14, abs=1.0)
        assert not any(cfg.turns[32:])
    assert lib.mmdit_rope_config(None, 64, 1, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0) == INVALID


def _rope(lib, fn="mmdit_rope_fwd", act=1, cfg="ok", batch=1, seq=4, d=64, hq=2, q=(A, 512, 128, 64), qo=(B_, 512, 128, 64),
          hk=1, k=(C_, 256, 64, 64), ko=(D_, 256, 64, 64), pos=E_, pb=4, cos=None, sin=None):
    view = lambda v: None if v is None else L.RopeView(*v)  # noqa: E731
    c = _cfg(lib)[1] if cfg == "ok" else cfg
    return getattr(lib, fn)(act, c, batch, seq, d, hq, view(q), view(qo), hk, view(k), view(ko), pos, pb, cos, sin, None)


@pytest.mark.parametrize("fn", ["mmdit_rope_fwd", "mmdit_rope_bwd"])
@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(act=2)), (INVALID, dict(cfg=None)), (INVALID, dict(cfg=L.RopeCfg())), (INVALID, dict(seq=-1)),
    (INVALID, dict(hq=-1)), (UNSUPPORTED, dict(d=60)), (UNSUPPORTED, dict(d=520)), (INVALID, dict(d=56)),
    (INVALID, dict(q=None)), (INVALID, dict(qo=None)), (INVALID, dict(ko=None)), (INVALID, dict(k=None)),
    (INVALID, dict(q=(A + 8, 512, 128, 64))), (INVALID, dict(q=(A, 512, 128, 60))), (INVALID, dict(qo=(B_, 512, -128, 64))),
    (INVALID, dict(qo=(A, 512, 64, 256))), (INVALID, dict(pos=None)), (INVALID, dict(cos=E_, sin=F_)),
    (INVALID, dict(pos=None, cos=E_)), (INVALID, dict(pb=-4)), (UNSUPPORTED, dict(hq=65536, hk=1)), (UNSUPPORTED, dict(batch=65536)),
    (UNSUPPORTED, dict(seq=(1 << 30) + 1)), (INVALID, dict(qo=(B_, 512, 0, 64))), (INVALID, dict(batch=2, ko=(D_, 0, 64, 64))),
    (INVALID, dict(qo=(B_, 512, 128, 0))),
    (INVALID, dict(pos=E_ + 4)), (INVALID, dict(pos=None, cos=E_ + 2, sin=F_)),
])
def test_rope_refusals(lib, fn, status, kw):
    assert _rope(lib, fn, **kw) == status and "rope" in L.last_error()


@pytest.mark.parametrize("kw", [
    dict(qo=(B_, 512, 128, 56)), dict(qo=(B_, 512, 56, 64)), dict(batch=2, ko=(D_, 56, 64, 64)), dict(ko=(B_, 256, 64, 64)),
    dict(qo=(C_, 512, 128, 64)), dict(ko=(A, 256, 64, 64)),
])
def test_rope_refuses_overlapping_outputs(lib, kw):
    """Heads that start less than a head apart, q_out on k or k_out, k_out on q."""
    assert _rope(lib, **kw) == INVALID and ("overlap" in L.last_error() or "each other" in L.last_error())


def test_rope_empty(lib):
    assert _rope(lib, batch=0) == 0 and _rope(lib, seq=0) == 0


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.mmdit_add_rmsnorm_fwd(x, x[0], y=x)
    with pytest.raises(ValueError, match="CUDA"):
        L.mmdit_fp8_block_cast(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        L.mmdit_rope_fwd(L.make_rope_cfg(32), x.view(1, 2, 1, 64), x.view(1, 2, 1, 64))
    with pytest.raises(ValueError, match="scaling"):
        L.make_rope_cfg(32, scaling="cubic")
    with pytest.raises(L.MMDitError):
        L.make_rope_cfg(31)


def test_argument_checks():
    """The shape, type and layout checks of the binding, on host tensors of a host `device`."""
    dev = torch.device("cpu")
    t = torch.zeros(4, 6)
    assert L._arg("t", t, dev, torch.float32, 4, 6) == t.data_ptr() and L._arg("t", None, dev, torch.float32, 1) is None
    with pytest.raises(TypeError, match="dtype"):
        L._arg("t", t, dev, torch.uint8, 4, 6)
    with pytest.raises(ValueError, match="shape"):
        L._arg("t", t, dev, torch.float32, 6, 4)
    with pytest.raises(ValueError, match="contiguous"):
        L._arg("t", t.t(), dev, torch.float32, 6, 4)
    with pytest.raises(ValueError, match="cpu"):
        L._arg("t", t, torch.device("meta"), torch.float32, 4, 6)


def test_operands_updated_in_place_are_not_read_through_the_read_only_path():
    """__ldg is for memory that nothing writes during the kernel.  The header lets h be the residual, dh be dh_in and
    q and k be rotated in place: the kernels read these operands plainly."""
    import os
    import re

    csrc = os.path.join(os.path.dirname(build_ext.__file__), "csrc")
    read = lambda name: open(os.path.join(csrc, name)).read()  # noqa: E731
    raw8 = re.findall(r"struct Raw8<\w+> \{.*?\n\};", read("rowwise.cuh"), re.S)
    assert len(raw8) == 2
    for body in raw8:
        plain = re.search(r"void load_rw\(const \w+\* p\) \{(.*?)\}", body, re.S)
        assert plain and "__ldg" not in plain.group(1)
    norm = read("rmsnorm.cu")
    assert re.findall(r"\brr\[i\]\.(\w+)\(res", norm) == ["load_rw"]
    assert re.findall(r"\bin\[i\]\.(\w+)\(static_cast<const TR\*>\(a\.dh_in\)", norm) == ["load_rw"]
    rope = read("rope_apply.cu")
    assert re.search(r"struct Piece<__nv_bfloat16, 8> : Raw8<__nv_bfloat16> \{[^}]*void load\([^)]*\) \{ load_rw\(p\); \}", rope)
    # the heads themselves are read through Piece and load_v alone, neither of which takes the read-only path
    assert "__ldg" not in re.search(r"void load_v\(.*?\n\}", rope, re.S).group(0)
    assert all(m.startswith(("a.cos", "a.sin", "a.pos")) for m in re.findall(r"__ldg\(([^)]*)", rope))


def test_norm_gradient_workspace_of_the_most_rows(lib):
    """The header sets no limit on the rows: the launch shape must not leave 32 bits on the way."""
    most = L.mmdit_add_rmsnorm_bwd_workspace_size(1 << 20, 8)
    for rows in ((1 << 31) - 1, (1 << 31) - 7, (1 << 31) - 8):
        assert L.mmdit_add_rmsnorm_bwd_workspace_size(rows, 8) == most


def test_workspace_of_overlapping_elements_is_refused():
    """An expanded tensor has fewer bytes than elements; the library would write behind it."""
    dev = torch.device("cpu")
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(512, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            L._workspace_arg(ws, dev, lambda: 256, None)
    ws = torch.zeros(512, dtype=torch.uint8)
    assert L._workspace_arg(ws, dev, lambda: 256, None) is ws


@pytest.mark.parametrize("fn", ["mmdit_rope_fwd", "mmdit_rope_bwd"])
def test_rope_heads_without_their_other_half_are_refused(fn):
    """k_out without k was taken for a call on q alone and left as it was."""
    q = torch.zeros(1, 2, 1, 64)
    for kw in (dict(k_out=q), dict(k=q)):
        with pytest.raises(ValueError, match="go together"):
            getattr(L, fn)(L.RopeCfg(), q, q, **kw)
    with pytest.raises(ValueError, match="q_out"):
        getattr(L, fn)(L.RopeCfg(), q, None)


def test_launch_needs_no_private_name_of_torch(monkeypatch):
    """On a torch without the private calls the current stream and device come from the public ones."""
    import types

    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i=None: types.SimpleNamespace(cuda_stream=70 + (i or 0)))
    monkeypatch.setattr(L, "_lib", types.SimpleNamespace(f=lambda *a: seen.append(a) or 0))
    if hasattr(L, "_current_getters"):
        for name, get in zip(("_raw_stream", "_current_device"), L._current_getters()):
            monkeypatch.setattr(L, name, get)
    L._launch("f", torch.device("cuda", 0), None, 1, 2)
    L._launch("f", torch.device("cuda", 0), 5, 3)
    assert seen == [(1, 2, 70), (3, 5)]


def test_rope_config_refuses_an_mscale_that_float32_cannot_hold(lib):
    """The configuration keeps mscale as a float: a larger double became infinite."""
    for m in (1e39, -1e39, 1e308, float("inf")):
        assert _cfg(lib, mscale=m)[0] == INVALID
    st, cfg = _cfg(lib, mscale=3e38)
    assert st == 0 and cfg.mscale == pytest.approx(3e38)


def test_rope_config_holds_the_exact_frequencies_to_its_bound(lib):
    """turns[j] against f_j / 2 pi without a double's rounding, at the bound that the header states."""
    from decimal import Decimal

    from oracle import lm

    for rot, kw in ((128, dict()), (64, dict(theta=500000.0)), (96, dict(scaling="linear", factor=3.7)),
                    (128, dict(theta=500000.0, scaling="by_parts", factor=16.0, orig_len=8192.0, low=1.0, high=32.0)),
                    (128, dict(scaling="by_parts", factor=40.0, orig_len=4096.0, low=1.0, high=4.0))):
        cfg = L.make_rope_cfg(rot, **kw)
        steps = 5.0
        if kw.get("scaling") == "by_parts":
            steps = kw["factor"] * (5 * kw["high"] / (kw["high"] - kw["low"]) + 3) + 8
        for j, t in enumerate(lm.rope_turns_exact(rot, **kw)):
            assert abs(Decimal(cfg.turns[j]) - t * 2 ** 64) <= 1 + Decimal(steps) * t * 2 ** 11
