"""RMS norm with the residual's addition and FP8 output, and its backward
pass, on the GPU against the 64-bit plain forms of tests/_plain.py.

Error bounds (U = 2^-24): a row's f32 sum of squares passes each term through
at most sum_depth(cols) additions, all of one sign, so rstd is off by half
that many U and y = h w rstd by four roundings more.
"""
import ctypes

import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H
import _plain as P

pytestmark = pytest.mark.gpu
U = P.U


def rel_y(cols):
    return (P.sum_depth(cols) / 2 + 8) * U


def inputs(rows, cols, dtype, wdtype, residual, seed, offset=0):
    """Rows that start `offset` elements off the allocation."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def make(shape, dt, std, mean=0.0):
        flat = torch.empty(shape[0] * (shape[1] if len(shape) > 1 else 1) + offset, dtype=dt, device="cuda")
        v = flat[offset:].view(shape)
        v.copy_(torch.randn(shape, generator=g, device="cuda") * std + mean)
        return v

    x = make((rows, cols), dtype, 1.0)
    w = make((cols,), wdtype, 0.1, 1.0)
    r = make((rows, cols), dtype, 3.0) if residual else None
    return x, w, r


def check_forward(x, w, r, eps, fmt, block, q, scales, h_out, y_out, rstd):
    rows, cols = x.shape
    h = x.double() + (r.double() if r is not None else 0.0)
    want = (h.square().mean(1) + float(torch.tensor(eps, dtype=torch.float32))).rsqrt()
    rel = rel_y(cols)
    assert bool(((rstd.double() - want).abs() <= want * rel).all())
    y = h * w.double() * want[:, None]
    P.check_quantized(q, scales, y, block, fmt, rel)
    t = x.dtype
    if h_out is not None:
        assert bool(((h_out.double() - h).abs() <= h.abs() * (P.half(t) + 2 * U) + P.tiny(t)).all())
    if y_out is not None:
        assert bool(((y_out.double() - y).abs() <= y.abs() * (P.half(t) + 2 * rel) + P.tiny(t)).all())


def run_forward(x, w, r, eps, fmt, block, y=True):
    rows, cols = x.shape
    y_out = torch.empty_like(x) if y else None
    rstd = torch.empty(rows, device="cuda")
    q, s, h = H.hq_rmsnorm_fp8(x, w, eps, residual=r, fmt=fmt, block=block, y_out=y_out, rstd_out=rstd)
    torch.cuda.synchronize()
    return q, s, h, y_out, rstd


SHAPES = [(1, 1), (1, 8192), (2, 17), (3, 33), (7, 64), (16, 8192), (5, 1000), (130, 1408), (300, 1024), (33, 4100),
          (9, 8200), (1300, 256), (4, 16384), (3, 16400), (3, 28672), (2, 32768), (2, 32761), (1, 31)]


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                          (torch.float32, torch.float32), (torch.float32, torch.float16),
                                          (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_per_row(shape, dtype, wdtype):
    for residual, fmt in ((True, H.E4M3), (False, H.E5M2)):
        x, w, r = inputs(*shape, dtype, wdtype, residual, seed=shape[1] + fmt)
        q, s, h, y, rstd = run_forward(x, w, r, 1e-5, fmt, 0)
        check_forward(x, w, r, 1e-5, fmt, 0, q, s, h if residual else None, y, rstd)
        if not residual:
            assert h is x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape,block", [((3, 64), 16), ((5, 1408), 32), ((5, 1408), 128), ((17, 1040), 64),
                                         ((4, 8192), 128), ((3, 336), 48), ((2, 32768), 16), ((2, 4112), 400),
                                         ((6, 256), 4096), ((200, 2048), 256), ((9, 1024), 512), ((2, 28672), 32)],
                         ids=str)
def test_forward_block_wise(shape, block, dtype):
    for residual in (False, True):
        x, w, r = inputs(*shape, dtype, torch.float32, residual, seed=block)
        if shape[1] > 64:
            x[0, :block] = 0  # a block of zeros: scale 1
            if r is not None:
                r[0, :block] = 0
        for fmt in (H.E4M3, H.E5M2):
            q, s, h, y, rstd = run_forward(x, w, r, 1e-6, fmt, block)
            assert tuple(s.shape) == (shape[0], -(-shape[1] // block))
            check_forward(x, w, r, 1e-6, fmt, block, q, s, h if residual else None, y, rstd)


def test_codes_are_those_of_the_quantize_of_y():
    # with f32 rows y_out is y itself: its per-token and block-wise quantize give the same codes and scales
    x, w, r = inputs(37, 2064, torch.float32, torch.float32, True, seed=3)
    for block in (0, 48, 128):
        q, s, _, y, _ = run_forward(x, w, r, 1e-5, H.E4M3, block)
        q2, s2 = H.hq_quantize_fp8_blockwise(y, H.E4M3, block) if block else H.hq_quantize_fp8(y, H.E4M3, H.PER_TOKEN)
        assert torch.equal(q, q2) and torch.equal(s.reshape(-1), s2.reshape(-1))


def test_optional_outputs_do_not_change_the_others():
    x, w, r = inputs(65, 1024, torch.bfloat16, torch.bfloat16, True, seed=4)
    q, s, h, _, _ = run_forward(x, w, r, 1e-5, H.E4M3, 0)
    q2, s2, h2 = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(h, h2)
    # without residual_out (the C ABI's NULL): the same codes, nothing else written
    q3, s3 = torch.empty_like(q), torch.empty_like(s)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    H.check(H.lib.hq_rmsnorm_fp8(p(x), H.BF16, p(r), p(w), H.BF16, 65, 1024, 1e-5, H.E4M3, 0, p(q3), p(s3), None, None,
                                 None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    torch.cuda.synchronize()
    assert torch.equal(q, q3) and torch.equal(s, s3)


@pytest.mark.parametrize("shape", [(300, 1024), (3, 4099), (2, 32768), (17, 8192)], ids=str)
@pytest.mark.parametrize("which", ["x", "residual"])
def test_residual_stream_in_place(shape, which):
    x, w, r = inputs(*shape, torch.bfloat16, torch.bfloat16, True, seed=5)
    q, s, h, _, _ = run_forward(x, w, r, 1e-5, H.E4M3, 0)
    x2, r2 = x.clone(), r.clone()
    dst = x2 if which == "x" else r2
    q2, s2, h2 = H.hq_rmsnorm_fp8(x2, w, 1e-5, residual=r2, residual_out=dst)
    torch.cuda.synchronize()
    assert h2 is dst and torch.equal(h2, h) and torch.equal(q2, q) and torch.equal(s2, s)
    assert torch.equal(r2, r) if which == "x" else torch.equal(x2, x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("offset,cols", [(1, 1024), (3, 1408), (8, 1024), (4, 1032), (1, 4097)])
def test_rows_off_the_vector_grid(dtype, offset, cols):
    # views whose rows start off 16-byte boundaries, and buffers around the outputs left as they were
    rows = 11
    x, w, r = inputs(rows, cols, dtype, dtype, True, seed=6, offset=offset)
    buf = lambda dt: torch.full((rows * cols + 2 * offset + 64,), 77, dtype=dt, device="cuda")  # noqa: E731
    qb, hb, yb = buf(torch.uint8), buf(dtype), buf(dtype)
    view = lambda b: b[offset:offset + rows * cols].view(rows, cols)  # noqa: E731
    rstd = torch.empty(rows, device="cuda")
    q, s, h = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r, q=view(qb), residual_out=view(hb), y_out=view(yb), rstd_out=rstd)
    torch.cuda.synchronize()
    check_forward(x, w, r, 1e-5, H.E4M3, 0, q, s, h, view(yb), rstd)
    for b in (qb, hb, yb):
        assert bool((b[:offset] == 77).all()) and bool((b[offset + rows * cols:] == 77).all())


@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("cols", [1024, 1040, 8192])
def test_infinities_and_nan(block, cols):
    x, w, _ = inputs(6, cols, torch.bfloat16, torch.float32, False, seed=7)
    x[0, 5] = float("inf")     # rstd 0: y is NaN there and 0 elsewhere
    x[1, 9] = float("nan")     # the whole row
    x[2] = 0.0                 # y = 0, scale 1
    w[40] = float("inf")       # y infinite at a finite h
    w[41] = 0.0
    q, s, _, y, rstd = run_forward(x, w, None, 1e-5, H.E4M3, block)
    h = x.double()
    want = (h.square().mean(1) + float(torch.tensor(1e-5, dtype=torch.float32))).rsqrt()
    yy = h * w.double() * want[:, None]
    assert float(rstd[0]) == 0.0 and bool(torch.isnan(rstd[1]))
    assert bool((torch.isnan(y) == torch.isnan(yy)).all())
    P.check_quantized(q, s, yy, block, H.E4M3, rel_y(cols))
    assert bool((q[2, :40] == 0).all()) and bool((s[1] == 1).all())


def test_large_and_small_magnitudes():
    for scale in (1e-18, 1e-3, 1e4, 3e17):
        x, w, _ = inputs(3, 1000, torch.float32, torch.float32, False, seed=8)
        x = x * scale
        q, s, _, y, rstd = run_forward(x, w, None, 1e-30, H.E4M3, 0)
        check_forward(x, w, None, 1e-30, H.E4M3, 0, q, s, None, y, rstd)


def test_more_rows_than_the_grid_holds():
    x, w, r = inputs(20011, 136, torch.bfloat16, torch.bfloat16, True, seed=9)
    q, s, h, y, rstd = run_forward(x, w, r, 1e-5, H.E4M3, 0)
    check_forward(x, w, r, 1e-5, H.E4M3, 0, q, s, h, y, rstd)


def test_offsets_past_32_bits():
    # 140000 rows of 16384 columns: elements past 2^31
    rows, cols = 140000, 16384
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    q, s, _ = H.hq_rmsnorm_fp8(x, w, 1e-5)
    torch.cuda.synchronize()
    for lo in (0, 131070, rows - 3):
        sub = x[lo:lo + 3]
        q2, s2, _ = H.hq_rmsnorm_fp8(sub, w, 1e-5)
        assert torch.equal(q[lo:lo + 3], q2) and torch.equal(s[lo:lo + 3], s2)
    rstd = torch.full((rows,), 0.5, device="cuda")
    dx, _ = H.hq_rmsnorm_backward(x, x, w, rstd, need_dweight=False)
    dx2, _ = H.hq_rmsnorm_backward(x[-3:], x[-3:], w, rstd[-3:], need_dweight=False)
    assert torch.equal(dx[-3:], dx2)


# ---------------------------------------------------------------- backward
def check_backward(dy, h, w, rstd, dres, dx, dw):
    rows, cols = h.shape
    g, hd, wd, rs = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    xh, gw = hd * rs, g * wd
    mean = (gw * xh).mean(1, keepdim=True)
    want = rs * (gw - xh * mean) + (dres.double() if dres is not None else 0.0)
    # the mean's terms pass through sum_depth additions; the rest rounds a few times
    size = rs * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    tol = (P.sum_depth(cols) + 12) * U * size + P.half(dx.dtype) * want.abs() + P.tiny(dx.dtype)
    if dres is not None:
        tol = tol + 2 * U * dres.double().abs()
    assert bool(((dx.double() - want).abs() <= tol).all()), float(((dx.double() - want).abs() / tol).max())
    if dw is not None:
        wantw = (g * xh).sum(0)
        # a CTA's rows in order, at most 296 partial rows in eighths, then the eighths
        depth = rows / 128 + 64
        tolw = depth * U * (g * xh).abs().sum(0) + P.half(dw.dtype) * wantw.abs() + P.tiny(dw.dtype)
        assert bool(((dw.double() - wantw).abs() <= tolw).all()), float(((dw.double() - wantw).abs() / tolw).max())


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                          (torch.float32, torch.float32), (torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("shape", [(1, 1), (1, 8192), (2, 17), (7, 64), (300, 1024), (777, 4100), (5, 1000), (130, 1408),
                                   (9, 8200), (2500, 256), (4, 16384), (3, 16400), (3, 28672), (2, 32768), (2, 32761),
                                   (1000, 8192)], ids=str)
def test_backward(shape, dtype, wdtype):
    for with_dres in (False, True):
        h, w, dres = inputs(*shape, dtype, wdtype, with_dres, seed=shape[0])
        dy, _, _ = inputs(*shape, dtype, wdtype, False, seed=shape[0] + 1)
        rstd = (h.float().square().mean(1) + 1e-5).rsqrt()
        dx, dw = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=dres)
        torch.cuda.synchronize()
        check_backward(dy, h, w, rstd, dres, dx, dw)
        dx2, dw2 = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=dres)          # a fixed order: the same bits
        dx3, none = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=dres, need_dweight=False)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(dx, dx3) and none is None


@pytest.mark.parametrize("offset,cols", [(1, 1024), (8, 1024), (4, 1032), (3, 4097)])
def test_backward_off_the_vector_grid(offset, cols):
    h, w, dres = inputs(13, cols, torch.bfloat16, torch.bfloat16, True, seed=10, offset=offset)
    dy, _, _ = inputs(13, cols, torch.bfloat16, torch.bfloat16, False, seed=11, offset=offset)
    rstd = (h.float().square().mean(1) + 1e-5).rsqrt()
    dx, dw = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=dres)
    torch.cuda.synchronize()
    check_backward(dy, h, w, rstd, dres, dx, dw)


def test_backward_of_no_rows_writes_a_zero_gain_gradient():
    e = torch.empty((0, 72), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(72, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((72,), 5.0, dtype=torch.bfloat16, device="cuda")
    dx, dw = H.hq_rmsnorm_backward(e, e, w, torch.empty(0, device="cuda"), dweight=dw)
    torch.cuda.synchronize()
    assert dx.shape == (0, 72) and bool((dw == 0).all())
    q, s, h = H.hq_rmsnorm_fp8(e, w, 1e-5)
    assert q.shape == (0, 72) and s.shape == (0,)


def test_backward_is_the_gradient_by_differences():
    # the loss sum(c * y) in 64 bits, moved by +-t along random directions
    rows, cols, eps = 5, 96, 1e-5
    x, w, r = inputs(rows, cols, torch.float32, torch.float32, True, seed=12)
    h = x + r
    c = torch.randn(rows, cols, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    H.hq_rmsnorm_fp8(x, w, eps, residual=r, rstd_out=rstd)
    dx, dw = H.hq_rmsnorm_backward(c, h, w, rstd)

    def loss(hh, ww):
        return float((c.double() * hh * ww * (hh.square().mean(1, keepdim=True) + eps).rsqrt()).sum())

    for seed in range(4):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        dh, d = torch.randn(rows, cols, generator=g, device="cuda").double(), torch.randn(cols, generator=g, device="cuda").double()
        t = 1e-5
        num_h = (loss(h.double() + t * dh, w.double()) - loss(h.double() - t * dh, w.double())) / (2 * t)
        num_w = (loss(h.double(), w.double() + t * d) - loss(h.double(), w.double() - t * d)) / (2 * t)
        # differences are off by t^2 and 2^-53 / t of the loss's terms, the f32 gradient by ~1e-5 of its terms
        assert abs(num_h - float((dx.double() * dh).sum())) <= 1e-4 * float((dx.double() * dh).abs().sum())
        assert abs(num_w - float((dw.double() * d).sum())) <= 1e-4 * float((dw.double() * d).abs().sum())


# ----------------------------------------------------- streams and graphs
def test_another_stream_and_a_captured_graph():
    x, w, r = inputs(64, 1024, torch.bfloat16, torch.bfloat16, True, seed=13)
    dy, _, _ = inputs(64, 1024, torch.bfloat16, torch.bfloat16, False, seed=14)
    q, s, h, _, rstd = run_forward(x, w, r, 1e-5, H.E4M3, 0)
    dx, dw = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=r)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    q1, s1, h1 = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r, stream=st)
    dx1, dw1 = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=r, stream=st)
    st.synchronize()
    assert torch.equal(q, q1) and torch.equal(h, h1) and torch.equal(dx, dx1) and torch.equal(dw, dw1)
    graphs, outs = [], []
    for _ in range(2):  # two graphs, each with buffers of its own, replayed on two streams at once
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            qq, ss, hh = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r)
            outs.append((qq, ss, hh) + H.hq_rmsnorm_backward(dy, hh, w, rstd, dres=r))
        graphs.append(gr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, (q, s, h, dx, dw)):
            assert torch.equal(a, b)


# --------------------------- widths that are not a whole number of vectors
# (rows that share their first and last 16 bytes with their neighbours)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(2003, 1001), (1301, 257), (900, 4099), (150, 8191), (149, 12291), (5001, 25),
                                       (333, 100), (2401, 1004), (148, 8189), (301, 16369), (7, 24), (1, 1002)])
def test_rows_between_vectors(rows, cols, dtype):
    wdtype = torch.float32 if rows % 2 else dtype
    x, w, r = inputs(rows, cols, dtype, wdtype, True, seed=cols)
    for res in (r, None):
        guard = lambda dt: torch.full((rows * cols + 64,), 77, dtype=dt, device="cuda")  # noqa: E731
        view = lambda b: b[:rows * cols].view(rows, cols)  # noqa: E731
        qb, yb, hb = guard(torch.uint8), guard(dtype), guard(dtype)
        rstd = torch.empty(rows, device="cuda")
        q, s, h = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=res, q=view(qb), y_out=view(yb), rstd_out=rstd,
                                   residual_out=view(hb) if res is not None else None)
        torch.cuda.synchronize()
        check_forward(x, w, res, 1e-5, H.E4M3, 0, q, s, h if res is not None else None, view(yb), rstd)
        assert all(bool((b[rows * cols:] == 77).all()) for b in (qb, yb, hb))
    x2 = x.clone()
    q2, s2, h2 = H.hq_rmsnorm_fp8(x2, w, 1e-5, residual=r, residual_out=x2)
    q1, s1, h1 = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(s1, s2) and torch.equal(h1, h2)


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.float16),
                                          (torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,cols", [(2003, 1001), (1301, 257), (777, 4099), (150, 8191), (149, 12291), (5001, 25),
                                       (333, 100), (2401, 1004), (301, 16369), (7, 24), (1, 1002)])
def test_backward_of_rows_between_vectors(rows, cols, dtype, wdtype):
    for with_dres in (False, True):
        h, w, dres = inputs(rows, cols, dtype, wdtype, with_dres, seed=rows)
        dy, _, _ = inputs(rows, cols, dtype, wdtype, False, seed=rows + 1)
        rstd = (h.float().square().mean(1) + 1e-5).rsqrt()
        buf = torch.full((rows * cols + 64,), 77, dtype=dtype, device="cuda")
        dx, dw = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=dres, dx=buf[:rows * cols].view(rows, cols))
        torch.cuda.synchronize()
        check_backward(dy, h, w, rstd, dres, dx, dw)
        assert bool((buf[rows * cols:] == 77).all())
        dx2, dw2 = H.hq_rmsnorm_backward(dy, h, w, rstd, dres=dres)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1001, 4098, 60])
def test_neighbouring_rows_do_not_mix(cols, dtype):
    # rows of NaN leave the rows that share their vectors as they are
    rows = 997
    x, w, r = inputs(rows, cols, dtype, dtype, True, seed=12)
    q, s, h = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r)
    rstd = torch.rand(rows, device="cuda") + 0.5
    dx, _ = H.hq_rmsnorm_backward(x, r, w, rstd, dres=x)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[1::3] = True
    bad[-1] = False
    x2 = x.clone()
    x2[bad] = float("nan")
    q2, s2, h2 = H.hq_rmsnorm_fp8(x2, w, 1e-5, residual=r)
    dx2, _ = H.hq_rmsnorm_backward(x2, r, w, rstd, dres=x)
    torch.cuda.synchronize()
    for a, b in ((q, q2), (s, s2), (h, h2), (dx, dx2)):
        assert torch.equal(a[~bad], b[~bad])
    assert bool((q2[bad] == 0x7F).all()) and bool(torch.isnan(dx2[bad]).all())


# ------------------------------------------- rows split over a cluster's CTAs
WIDE = [(torch.bfloat16, 20480), (torch.bfloat16, 28672), (torch.float16, 16401), (torch.float32, 9600),
        (torch.float32, 18944), (torch.float32, 28672), (torch.float32, 32765)]


@pytest.mark.parametrize("dtype,cols", WIDE)
@pytest.mark.parametrize("rows", [1, 301])
def test_wide_rows(rows, dtype, cols):
    wdtype = torch.float32 if rows == 1 else dtype
    x, w, r = inputs(rows, cols, dtype, wdtype, True, seed=cols)
    dy, _, _ = inputs(rows, cols, dtype, wdtype, False, seed=cols + 1)
    for res, dres in ((r, dy), (None, None)):
        q, s, h, y, rstd = run_forward(x, w, res, 1e-5, H.E4M3, 0)
        check_forward(x, w, res, 1e-5, H.E4M3, 0, q, s, h if res is not None else None, y, rstd)
        dx, dw = H.hq_rmsnorm_backward(r, x, w, rstd, dres=dres)
        dx2, dw2 = H.hq_rmsnorm_backward(r, x, w, rstd, dres=dres)
        torch.cuda.synchronize()
        check_backward(r, x, w, rstd, dres, dx, dw)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    if cols % 16 == 0:
        for block in (32, 256):
            q, s, h, y, rstd = run_forward(x, w, r, 1e-5, H.E5M2, block)
            check_forward(x, w, r, 1e-5, H.E5M2, block, q, s, h, y, rstd)


@pytest.mark.parametrize("block", [0, 64])
def test_infinities_and_nan_in_wide_rows(block):
    for dtype, cols in ((torch.bfloat16, 28672), (torch.float32, 20480)):
        x, w, _ = inputs(200, cols, dtype, torch.float32, False, seed=13)
        clean = run_forward(x, w, None, 1e-5, H.E4M3, block)
        bad = torch.zeros(200, dtype=torch.bool, device="cuda")
        for k in range(0, 200, 7):
            x[k, (k * 997) % cols] = float("nan") if k % 2 else float("inf")
            bad[k] = True
        q, s, _, y, rstd = run_forward(x, w, None, 1e-5, H.E4M3, block)
        yy = x.double() * w.double() * rstd.double()[:, None]
        assert bool((torch.isnan(y) == torch.isnan(yy)).all())
        P.check_quantized(q[bad], s[bad], yy[bad], block, H.E4M3, rel_y(cols))
        for a, b in zip((q, s, y, rstd), (clean[0], clean[1], clean[3], clean[4])):
            assert torch.equal(a[~bad], b[~bad])


def test_wide_rows_on_two_streams_at_once():
    x, w, r = inputs(150, 28672, torch.bfloat16, torch.bfloat16, True, seed=14)
    q, s, h = H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r)
    rstd = torch.rand(150, device="cuda")
    dx, dw = H.hq_rmsnorm_backward(x, r, w, rstd)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    for _ in range(10):
        got.append(H.hq_rmsnorm_fp8(x, w, 1e-5, residual=r) + H.hq_rmsnorm_backward(x, r, w, rstd, stream=side))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, (q, s, h, dx, dw)))
    H.hq_check_device_error()
