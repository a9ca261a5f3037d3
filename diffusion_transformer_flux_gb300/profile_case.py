"""Runs one library entry point on one seeded case, for profiling a kernel with ncu.

    python -m diffusion_transformer_flux_gb300.profile_case attention --batch 2 --seq 4608
    python -m diffusion_transformer_flux_gb300.profile_case double_block --seq-img 4096 --seq-txt 512
    python -m diffusion_transformer_flux_gb300.profile_case linear --m 4608 --n 12288 --k 3072
    python -m diffusion_transformer_flux_gb300.profile_case double_block_bwd --seq-img 4096 --seq-txt 512
    python -m diffusion_transformer_flux_gb300.profile_case fp8_attention --seq 4608
    python -m diffusion_transformer_flux_gb300.profile_case head_loss --seq-img 4096
    python -m diffusion_transformer_flux_gb300.profile_case modulation --jobs 4
    python -m diffusion_transformer_flux_gb300.profile_case blockwise_linear --m 4608 --n 12288 --k 3072
    python -m diffusion_transformer_flux_gb300.profile_case mxfp8_linear --m 4608 --n 12288 --k 3072
    python -m diffusion_transformer_flux_gb300.profile_case block_linear --m 4608 --n 12288 --k 4096
    python -m diffusion_transformer_flux_gb300.profile_case block_linear_bwd --m 4095 --n 4096 --k 4096
    python -m diffusion_transformer_flux_gb300.profile_case add_rmsnorm --m 4608 --k 4096
    python -m diffusion_transformer_flux_gb300.profile_case rope --batch 2 --seq 4608
    python -m diffusion_transformer_flux_gb300.profile_case varlen_attention --batch 2 --seq 4608 --head-dim 128
    python -m diffusion_transformer_flux_gb300.profile_case varlen_attention_bwd --batch 2 --seq 2304 --head-dim 128
    python -m diffusion_transformer_flux_gb300.profile_case paged_attention --batch 16 --seq 4096 --new 1
    python -m diffusion_transformer_flux_gb300.profile_case block_tables --batch 64 --new 2000
    python -m diffusion_transformer_flux_gb300.profile_case kv_cache_write --seq 9216

Inputs are drawn on the device (N(0,1) activations, N(0,0.02) weights); the case runs
--iters times and exits 0 only if every kernel finished its waits.
"""
from __future__ import annotations

import argparse

import torch

from . import _lib as L


def _w(*shape, std=0.02):
    return (torch.randn(*shape, device="cuda") * std).to(torch.bfloat16)


def _stream_w(D, F, d=128):
    return {"w_mod": _w(6 * D, D), "b_mod": _w(6 * D), "w_qkv": _w(3 * D, D), "b_qkv": _w(3 * D),
            "g_q": torch.ones(d, device="cuda", dtype=torch.bfloat16),
            "g_k": torch.ones(d, device="cuda", dtype=torch.bfloat16),
            "w_o": _w(D, D), "b_o": _w(D), "w_1": _w(F, D), "b_1": _w(F), "w_2": _w(D, F), "b_2": _w(D)}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["attention", "double_block", "single_block", "linear", "double_block_bwd",
                                     "fp8_attention", "head_loss", "modulation", "blockwise_linear",
                                     "mxfp8_linear", "block_linear", "block_linear_bwd", "block_cast", "add_rmsnorm",
                                     "add_rmsnorm_bwd", "rope", "varlen_attention", "varlen_attention_bwd", "paged_attention",
                                     "block_tables", "kv_cache_write"])
    ap.add_argument("--jobs", type=int, default=4)
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--seq", type=int, default=4608)
    ap.add_argument("--seq-img", type=int, default=4096)
    ap.add_argument("--seq-txt", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=3072)
    ap.add_argument("--mlp", type=int, default=12288)
    ap.add_argument("--m", type=int, default=4608)
    ap.add_argument("--n", type=int, default=12288)
    ap.add_argument("--k", type=int, default=3072)
    ap.add_argument("--iters", type=int, default=3)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--new", type=int, default=1)
    a = ap.parse_args()
    torch.manual_seed(0)
    L.load()
    wss = []
    if a.case == "fp8_attention":
        H = a.hidden // 128
        q, k, v = (torch.randn(a.batch, H, a.seq, 128, device="cuda").to(torch.bfloat16) for _ in range(3))
        scales = torch.full((3,), 32.0, device="cuda")
        out = torch.empty(a.batch, a.seq, a.hidden, device="cuda", dtype=torch.bfloat16)
        run = lambda: wss.append(L.mmdit_fp8_attention_fwd(q, k, v, scales[0:1], scales[1:2], scales[2:3], out))
    elif a.case == "head_loss":
        B, Si, D = a.batch, a.seq_img, a.hidden
        hw = int(round(Si ** 0.5))
        dims = L.make_dims(B, Si, 0, D, D // 128, a.mlp, L.MMDIT_BF16)
        x, vec = _w(B, Si, D, std=1.0), _w(B, D, std=1.0)
        z0, z1 = (torch.randn(B, 64, hw, hw, device="cuda") for _ in range(2))
        loss = torch.zeros(1, device="cuda")
        args = (dims, hw, hw, x, vec, _w(2 * D, D), _w(2 * D), _w(64, D), _w(64), z0, z1, loss)
        run = lambda: wss.append(L.mmdit_final_layer_loss_fwd(*args))
    elif a.case == "modulation":
        D = a.hidden
        vec = _w(a.batch, D, std=1.0)
        jobs = [(_w(6 * D, D), _w(6 * D), torch.empty(a.batch, 6 * D, device="cuda")) for _ in range(a.jobs)]
        run = lambda: L.mmdit_modulation_batched_fwd(vec, jobs)
    elif a.case == "attention":
        H = a.hidden // 128
        q, k, v = (torch.randn(a.batch, H, a.seq, 128, device="cuda").to(torch.bfloat16) for _ in range(3))
        out = torch.empty(a.batch, a.seq, a.hidden, device="cuda", dtype=torch.bfloat16)
        run = lambda: wss.append(L.mmdit_attention_fwd(q, k, v, out))
    elif a.case == "linear":
        x, w, b = _w(a.m, a.k, std=1.0), _w(a.n, a.k), _w(a.n)
        y = torch.empty(a.m, a.n, device="cuda", dtype=torch.bfloat16)
        run = lambda: wss.append(L.mmdit_linear_fwd(x, w, b, y))
    elif a.case == "blockwise_linear":
        x, w, b = _w(a.m, a.k, std=1.0), _w(a.n, a.k), _w(a.n)
        y = torch.empty(a.m, a.n, device="cuda", dtype=torch.bfloat16)
        run = lambda: wss.append(L.mmdit_fp8_blockwise_linear_fwd(x, w, b, y))
    elif a.case == "mxfp8_linear":
        x, w, b = _w(a.m, a.k, std=1.0), _w(a.n, a.k), _w(a.n)
        y = torch.empty(a.m, a.n, device="cuda", dtype=torch.bfloat16)
        run = lambda: wss.append(L.mmdit_fp8_mxfp8_linear_fwd(x, w, b, y))
    elif a.case in ("block_linear", "block_linear_bwd", "block_cast"):
        m, n, k = a.m, a.n, a.k
        t = lambda v: (v + 127) // 128
        e = lambda *s, dtype=torch.uint8: torch.empty(*s, dtype=dtype, device="cuda")
        x, w = _w(m, k, std=1.0), _w(n, k)
        xq, sx, xt, sxt = e(m, k), e(t(k), m, dtype=torch.float32), e(k, (m + 15) // 16 * 16), e(t(m), k, dtype=torch.float32)
        wq, sw, wt = e(n, k), e(t(n), t(k), dtype=torch.float32), e(k, (n + 15) // 16 * 16)
        cast = lambda: L.mmdit_fp8_block_cast(x, xq, sx, q_t=xt, s_t=sxt)
        cast()
        L.mmdit_fp8_block_cast(w, wq, sw, q_t=wt, square=True)
        if a.case == "block_cast":
            run = cast
        elif a.case == "block_linear":
            y, b = e(m, n, dtype=torch.bfloat16), _w(n)
            run = lambda: wss.append(L.mmdit_fp8_block_linear_fwd(xq, sx, wq, sw, b, y))
        else:
            dy, dx = _w(m, n, std=1e-3), e(m, k, dtype=torch.bfloat16)
            dw, db = e(n, k, dtype=torch.float32), e(n, dtype=torch.float32)
            ws = L.workspace(L.mmdit_fp8_block_linear_bwd_workspace_size(m, n, k))
            run = lambda: wss.append(L.mmdit_fp8_block_linear_bwd(dy, wt, sw, xt, sxt, dx=dx, dw=dw, db=db, ws=ws))
    elif a.case in ("add_rmsnorm", "add_rmsnorm_bwd"):
        x, res, gain = _w(a.m, a.k, std=1.0), _w(a.m, a.k, std=1.0).float(), _w(a.k, std=1.0)
        h, rstd = torch.empty_like(res), torch.empty(a.m, device="cuda")
        q, s = torch.empty(a.m, a.k, device="cuda", dtype=torch.uint8), torch.empty((a.k + 127) // 128, a.m, device="cuda")
        fwd = lambda: L.mmdit_add_rmsnorm_fwd(x, gain, residual=res, h=h, y_q=q, s_y=s, rstd=rstd)
        fwd()
        dh, dg = torch.empty_like(x), torch.empty(a.k, device="cuda")
        ws = L.workspace(L.mmdit_add_rmsnorm_bwd_workspace_size(a.m, a.k))
        xb = x.clone()
        run = fwd if a.case == "add_rmsnorm" else lambda: wss.append(
            L.mmdit_add_rmsnorm_bwd(x, xb, gain, rstd, dh, dh_in=x, dgain=dg, ws=ws))
    elif a.case == "rope":
        q = _w(a.batch, a.seq, 32, 128, std=1.0)
        k = _w(a.batch, a.seq, 8, 128, std=1.0)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        cfg, pos = L.make_rope_cfg(128, scaling="linear", factor=4.0), torch.arange(a.seq, device="cuda")
        run = lambda: L.mmdit_rope_fwd(cfg, q, qo, k=k, k_out=ko, positions=pos)
    elif a.case in ("varlen_attention", "varlen_attention_bwd"):  # 32 query and 8 key heads, causal
        T, d = a.batch * a.seq, a.head_dim
        q, k, v = _w(T, 32, d, std=1.0), _w(T, 8, d, std=1.0), _w(T, 8, d, std=1.0)
        cu = torch.arange(0, T + 1, a.seq, device="cuda", dtype=torch.int32)
        out, lse = torch.empty_like(q), torch.empty(T, 32, device="cuda")
        fwd = lambda: wss.append(L.mmdit_varlen_attention_fwd(q, k, v, out, cu, lse=lse))
        fwd()
        dout, grads = _w(T, 32, d, std=1.0), [torch.empty_like(t) for t in (q, k, v)]
        run = fwd if a.case == "varlen_attention" else lambda: wss.append(
            L.mmdit_varlen_attention_bwd(dout, q, k, v, out, lse, *grads, cu))
    elif a.case == "paged_attention":  # requests of a.seq tokens, the last a.new of them new
        d, page = a.head_dim, 16
        width = (a.seq + page - 1) // page
        kc, vc = (_w(a.batch * width, page, 8, d, std=1.0) for _ in range(2))
        tables = torch.randperm(a.batch * width, device="cuda").to(torch.int32).view(a.batch, width)
        lens = torch.full((a.batch,), a.seq, device="cuda", dtype=torch.int32)
        cu = torch.arange(0, a.batch * a.new + 1, a.new, device="cuda", dtype=torch.int32)
        q = _w(a.batch * a.new, 32, d, std=1.0)
        out = torch.empty_like(q)
        run = lambda: wss.append(L.mmdit_paged_attention_fwd(q, kc, vc, out, tables, lens, cu, max_q=a.new))
    elif a.case == "block_tables":  # requests of a.new tokens each
        page, width = 64, (a.new + 63) // 64
        i32 = lambda *s, fill=0: torch.full(s, fill, device="cuda", dtype=torch.int32)
        before, after, tables = i32(a.batch), i32(a.batch, fill=a.new), i32(a.batch, width, fill=-1)
        free, n = torch.arange(a.batch * width, device="cuda", dtype=torch.int32), i32(1, fill=a.batch * width)
        pos, slots = (torch.empty(a.batch * a.new, device="cuda", dtype=torch.int64) for _ in range(2))
        out = i32(1), i32(a.batch + 1)
        run = lambda: L.mmdit_block_tables(before, after, tables, free, n, page, *out, pos, slots, i32(2))
    elif a.case == "kv_cache_write":
        k, v = (_w(a.seq, 8, a.head_dim, std=1.0) for _ in range(2))
        kc, vc = (_w((a.seq + 63) // 64, 64, 8, a.head_dim) for _ in range(2))
        slots = torch.arange(a.seq, device="cuda")
        run = lambda: L.mmdit_kv_cache_write(k, v, kc, vc, slots)
    else:
        B, Si, St, D, F = a.batch, a.seq_img, a.seq_txt, a.hidden, a.mlp
        S = Si + St
        dims = L.make_dims(B, Si, St, D, D // 128, F, L.MMDIT_BF16)
        vec = _w(B, D, std=1.0)
        cos, sin = torch.rand(B, S, 64, device="cuda"), torch.rand(B, S, 64, device="cuda")
        if a.case == "double_block_bwd":
            wi, wt = _stream_w(D, F), _stream_w(D, F)
            xi, xt = _w(B, Si, D, std=1.0), _w(B, St, D, std=1.0)
            dyi, dyt = _w(B, Si, D, std=1e-3), _w(B, St, D, std=1e-3)
            dxi, dxt = torch.empty_like(xi), torch.empty_like(xt)
            dvec = torch.empty(B, D, device="cuda")
            g = [{n: torch.empty(tuple(w[n].shape), device="cuda") for n in L.STREAM_W_FIELDS} for w in (wi, wt)]
            ws = L.workspace(L.mmdit_double_block_bwd_workspace_size(dims))
            run = lambda: wss.append(L.mmdit_double_block_bwd(dims, wi, wt, vec, cos, sin, xi, xt, dyi, dyt, dxi, dxt,
                                                              dvec, g[0], g[1], ws=ws))
        elif a.case == "double_block":
            wi, wt = _stream_w(D, F), _stream_w(D, F)
            xi, xt = _w(B, Si, D, std=1.0), _w(B, St, D, std=1.0)
            yi, yt = torch.empty_like(xi), torch.empty_like(xt)
            ws = L.workspace(L.mmdit_double_block_workspace_size(dims))
            run = lambda: wss.append(L.mmdit_double_block_fwd(dims, wi, wt, vec, cos, sin, xi, xt, yi, yt, ws=ws))
        else:
            w = _stream_w(D, F)
            x = _w(B, S, D, std=1.0)
            y = torch.empty_like(x)
            ws = L.workspace(L.mmdit_single_block_workspace_size(dims))
            run = lambda: wss.append(L.mmdit_single_block_fwd(dims, w, vec, cos, sin, x, y, ws=ws))
    for _ in range(a.iters):
        run()
    torch.cuda.synchronize()
    for ws in wss:
        if L.mmdit_workspace_status(ws) != 0:
            raise SystemExit("a kernel gave up a bounded wait")
    print(f"{a.case}: {a.iters} iterations ok")


if __name__ == "__main__":
    main()
