"""Refusals of the feed-forward operators, before any CUDA call (no GPU
needed: the addresses are made up and never touched), and the binding's
checks of shapes, dtypes and layout."""
import ctypes

import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H

L = H.lib
OK, INVALID, MISALIGNED, OVERLAP, TOO_LARGE = 0, 1, 2, 3, 8
BASE = 0x7F0000000000
M24 = 0x1000000


def norm(x=BASE, xt=H.BF16, res=BASE + M24, w=BASE + 2 * M24, wt=H.F32, rows=64, cols=128, eps=1e-5, fmt=H.E4M3, block=0,
         q=BASE + 3 * M24, s=BASE + 4 * M24, ro=BASE + 5 * M24, y=BASE + 6 * M24, rstd=BASE + 7 * M24):
    return L.hq_rmsnorm_fp8(x, xt, res, w, wt, rows, cols, eps, fmt, block, q, s, ro, y, rstd, None)


def test_rmsnorm_rejections():
    assert norm(xt=3) == INVALID and norm(wt=-1) == INVALID and norm(fmt=2) == INVALID
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert norm(eps=eps) == INVALID
    assert norm(rows=-1) == INVALID and norm(cols=-1) == INVALID
    assert norm(rows=1 << 31) == TOO_LARGE and norm(cols=32769) == TOO_LARGE
    assert norm(block=-16) == INVALID and norm(block=8) == INVALID and norm(block=40) == INVALID
    assert norm(block=32, cols=120) == INVALID            # block-wise rows are whole 16-column units
    assert norm(res=None) == INVALID                      # residual_out without a residual
    assert "residual" in L.hq_last_error().decode()
    assert norm(x=None) == INVALID and norm(w=None) == INVALID and norm(q=None) == INVALID and norm(s=None) == INVALID
    assert norm(x=BASE + 1) == MISALIGNED and norm(xt=H.F32, y=BASE + 6 * M24 + 2) == MISALIGNED
    assert norm(w=BASE + 2 * M24 + 2) == MISALIGNED and norm(s=BASE + 4 * M24 + 2) == MISALIGNED
    assert norm(rstd=BASE + 7 * M24 + 1) == MISALIGNED
    assert norm(q=BASE + 64) == OVERLAP                   # codes over x
    assert norm(y=BASE + M24) == OVERLAP                  # y over the residual
    assert norm(ro=BASE + 256) == OVERLAP                 # the sum shifted against x
    assert norm(ro=BASE, res=BASE + 2) == OVERLAP         # in place over x, which the residual overlaps
    assert norm(s=BASE + 2 * M24) == OVERLAP              # scales over the weight
    assert norm(y=BASE + 5 * M24 + 16) == OVERLAP         # two outputs
    assert norm(ro=BASE, y=BASE) == OVERLAP               # in place is for the sum alone
    assert norm(rows=0, x=None, w=None, q=None, s=None) == OK and norm(cols=0, q=None) == OK
    assert norm(rows=0, cols=32769) == TOO_LARGE          # shapes are checked for an empty call too


def bwd(dy=BASE, h=BASE + M24, xt=H.BF16, dres=BASE + 2 * M24, w=BASE + 3 * M24, wt=H.BF16, rstd=BASE + 4 * M24, rows=64,
        cols=128, dx=BASE + 5 * M24, dw=BASE + 6 * M24, ws=BASE + 7 * M24, wsb=None):
    wsb = H.hq_rmsnorm_backward_workspace_bytes(64, 128) if wsb is None else wsb
    return L.hq_rmsnorm_backward(dy, h, xt, dres, w, wt, rstd, rows, cols, dx, dw, ws, wsb, None)


def test_rmsnorm_backward_rejections():
    assert H.hq_rmsnorm_backward_workspace_bytes(64, 128) > 0
    assert H.hq_rmsnorm_backward_workspace_bytes(-1, 128) == 0 and H.hq_rmsnorm_backward_workspace_bytes(8, 40000) == 0
    assert bwd(xt=9) == INVALID and bwd(wt=9) == INVALID and bwd(rows=-1) == INVALID
    assert bwd(rows=1 << 31) == TOO_LARGE and bwd(cols=32769) == TOO_LARGE
    for name in ("dy", "h", "w", "rstd", "dx"):
        assert bwd(**{name: None}) == INVALID
    assert bwd(ws=None) == INVALID and bwd(wsb=H.hq_rmsnorm_backward_workspace_bytes(64, 128) - 1) == INVALID
    assert "workspace" in L.hq_last_error().decode()
    assert bwd(dy=BASE + 1) == MISALIGNED and bwd(rstd=BASE + 4 * M24 + 2) == MISALIGNED
    assert bwd(wt=H.F32, dw=BASE + 6 * M24 + 2) == MISALIGNED and bwd(ws=BASE + 7 * M24 + 16) == MISALIGNED
    assert bwd(dx=BASE) == OVERLAP and bwd(dx=BASE + M24) == OVERLAP and bwd(dx=BASE + 2 * M24 + 2) == OVERLAP
    assert bwd(dw=BASE + 3 * M24) == OVERLAP and bwd(ws=BASE + 5 * M24) == OVERLAP
    assert bwd(cols=0) == OK and bwd(rows=0, dw=None, ws=None, wsb=0, dy=None) == OK


def act(xq=BASE, wq=BASE + M24, fmt=H.E4M3, xsl=64, wsl=128, bias=BASE + 4 * M24, a=H.ACT_GELU, res=BASE + 5 * M24, M=64,
        N=128, K=256, out=BASE + 6 * M24, zq=BASE + 7 * M24, zf=H.E4M3, zb=32, zs=BASE + 8 * M24):
    return L.hq_gemm_a8w8_act(xq, wq, fmt, BASE + 2 * M24, xsl, BASE + 3 * M24, wsl, bias, a, res, M, N, K, out, zq, zf,
                              zb, zs, None)


def test_gemm_act_rejections():
    assert act(a=-1) == INVALID and act(a=5) == INVALID and act(fmt=2) == INVALID and act(zf=2) == INVALID
    assert act(M=-1) == INVALID and act(K=250) == INVALID and act(N=100) == INVALID and act(xsl=3) == INVALID
    assert act(K=1 << 31) == TOO_LARGE
    assert act(zs=None) == INVALID and act(zq=None) == INVALID        # codes and scales together
    assert act(zb=64) == INVALID and act(zb=0) == INVALID
    assert act(N=136, wsl=136) == INVALID                             # whole 32-column blocks
    assert act(out=None) == INVALID and act(xq=None) == INVALID
    assert act(bias=BASE + 4 * M24 + 2) == MISALIGNED and act(res=BASE + 5 * M24 + 8) == MISALIGNED
    assert act(zq=BASE + 7 * M24 + 8) == MISALIGNED and act(zs=BASE + 8 * M24 + 2) == MISALIGNED
    assert act(out=BASE + 6 * M24 + 8) == MISALIGNED
    assert act(out=BASE) == OVERLAP and act(zq=BASE + M24) == OVERLAP and act(zs=BASE + 4 * M24) == OVERLAP
    assert act(res=BASE + 6 * M24 + 16) == OVERLAP                    # out shifted against the residual
    assert act(res=BASE + 7 * M24) == OVERLAP                         # codes over the residual
    assert act(zq=BASE + 6 * M24 + 1024) == OVERLAP                   # two outputs
    assert act(M=0, xsl=1, out=BASE + 6 * M24) in (OK, 4, 5, 6)       # nothing to compute: only the device checks are left


def abw(g=BASE, gt=H.BF16, zq=BASE + M24, zf=H.E4M3, zb=32, zs=BASE + 2 * M24, a=H.ACT_SILU, rows=64, cols=128,
        dz=BASE + 3 * M24, db=BASE + 4 * M24, ws=BASE + 5 * M24, wsb=None):
    wsb = H.hq_act_backward_workspace_bytes(64, 128) if wsb is None else wsb
    return L.hq_act_backward_fp8(g, gt, zq, zf, zb, zs, a, rows, cols, dz, db, ws, wsb, None)


def test_act_backward_rejections():
    assert H.hq_act_backward_workspace_bytes(64, 128) > 0 and H.hq_act_backward_workspace_bytes(-1, 16) == 0
    assert abw(gt=4) == INVALID and abw(zf=7) == INVALID and abw(a=0) == INVALID and abw(a=5) == INVALID
    assert abw(rows=-1) == INVALID and abw(cols=120) == INVALID and abw(zb=8) == INVALID and abw(zb=24) == INVALID
    assert abw(rows=1 << 31) == TOO_LARGE and abw(rows=1 << 21, cols=1 << 20) == TOO_LARGE
    for name in ("g", "zq", "zs", "dz"):
        assert abw(**{name: None}) == INVALID
    assert abw(ws=None) == INVALID and abw(wsb=16) == INVALID
    assert abw(g=BASE + 2) == MISALIGNED and abw(zq=BASE + M24 + 8) == MISALIGNED and abw(dz=BASE + 3 * M24 + 8) == MISALIGNED
    assert abw(zs=BASE + 2 * M24 + 1) == MISALIGNED and abw(db=BASE + 4 * M24 + 1) == MISALIGNED
    assert abw(ws=BASE + 5 * M24 + 8) == MISALIGNED
    assert abw(dz=BASE + 16) == OVERLAP                   # in place, but shifted
    assert abw(dz=BASE + M24) == OVERLAP and abw(db=BASE + 32) == OVERLAP and abw(ws=BASE + 2 * M24) == OVERLAP
    assert abw(cols=0) == OK and abw(rows=0, db=None, ws=None, wsb=0, g=None) == OK


def test_host_memory_is_refused():
    # CPU tensors reach the library's device check (or, without a driver, its first CUDA query): never a launch
    x, w = torch.zeros(2, 16), torch.ones(16)
    q, s = torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = L.hq_rmsnorm_fp8(p(x), H.F32, None, p(w), H.F32, 2, 16, 1e-5, H.E4M3, 0, p(q), p(s), None, None, None, None)
    assert st in (4, 6)
    assert bool((q == 0).all()) and bool((s == 0).all())


def test_binding_checks():
    x, w = torch.zeros(4, 32), torch.ones(32)
    bad = [
        lambda: H.hq_rmsnorm_fp8(x[0], w),
        lambda: H.hq_rmsnorm_fp8(x.long(), w),
        lambda: H.hq_rmsnorm_fp8(x, w[:16]),
        lambda: H.hq_rmsnorm_fp8(x, w, residual=x.half()),
        lambda: H.hq_rmsnorm_fp8(x, w, residual=x[:2]),
        lambda: H.hq_rmsnorm_fp8(x, w, residual_out=torch.zeros(4, 32)),
        lambda: H.hq_rmsnorm_fp8(x, w, residual=x, residual_out=torch.zeros(32, 4).t()),
        lambda: H.hq_rmsnorm_fp8(x, w, q=torch.zeros(4, 32)),
        lambda: H.hq_rmsnorm_fp8(x, w, block=16, scales=torch.zeros(4)),
        lambda: H.hq_rmsnorm_fp8(x, w, y_out=torch.zeros(4, 32).half()),
        lambda: H.hq_rmsnorm_fp8(x, w, rstd_out=torch.zeros(4).double()),
        lambda: H.hq_rmsnorm_backward(x, x, w, torch.ones(3)),
        lambda: H.hq_rmsnorm_backward(x, x.half(), w, torch.ones(4)),
        lambda: H.hq_rmsnorm_backward(x, x, w, torch.ones(4), dres=torch.zeros(4, 16)),
        lambda: H.hq_rmsnorm_backward(x, x, w, torch.ones(4), dweight=torch.zeros(32).half()),
        lambda: H.hq_rmsnorm_backward(x, x, w, torch.ones(4), dweight=w, need_dweight=False),
        lambda: H.hq_gemm_a8w8_act(x, x, w[:1], w[:1]),
        lambda: H.hq_gemm_a8w8_act(x.byte(), x[:, :16].byte(), w[:1], w[:1]),
        lambda: H.hq_gemm_a8w8_act(x.byte(), x.byte(), w[:1].half(), w[:1]),
        lambda: H.hq_gemm_a8w8_act(x.byte(), x.byte(), w[:1], w[:1], bias=torch.zeros(4)),
        lambda: H.hq_gemm_a8w8_act(x.byte(), x.byte(), w[:1], w[:1], residual=torch.zeros(4, 4)),
        lambda: H.hq_gemm_a8w8_act(x.byte(), x.byte(), w[:1], w[:1], ckpt=True),
        lambda: H.hq_act_backward_fp8(x, x.byte(), torch.ones(4, 2), H.ACT_SILU),
        lambda: H.hq_act_backward_fp8(x, x, torch.ones(4, 1), H.ACT_SILU),
        lambda: H.hq_act_backward_fp8(x, x.byte(), torch.ones(4, 1), H.ACT_SILU, dz=torch.zeros(32, 4).t()),
        lambda: H.hq_act_backward_fp8(x, x.byte(), torch.ones(4, 1), H.ACT_SILU, dbias=w, need_dbias=False),
        lambda: H.hq_act_backward_fp8(x, x.byte(), torch.ones(4, 1), H.ACT_SILU, block=0),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
