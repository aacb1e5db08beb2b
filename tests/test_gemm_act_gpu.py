"""The a8w8 GEMM with bias, activation, residual and the 8-bit checkpoint, on
the GPU against 64-bit products of the same codes (tests/_plain.py).

Error bound of z: the tensor cores add 32 products a step into a f32
accumulator and may truncate, so each of the K / 32 steps is off by up to
2^-23 of the largest partial sum, which sum |x w| bounds; then two scale
products, the bias and their roundings.
"""
import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H
import _plain as P

pytestmark = pytest.mark.gpu
U = P.U

# M, N, K: every tile of the dispatch -- decode tiles of 64, 128, 208 and 256 columns at up to 16, 64 and 128 rows, the
# 1-CTA tiles, the CTA pair and its 512-column form -- with ragged edges
SHAPES = [(1, 8, 16), (1, 64, 48), (16, 72, 256), (13, 9504, 128), (3, 18984, 64), (16, 28672, 96), (40, 1024, 400),
          (64, 18960, 32), (50, 24000, 160), (64, 38016, 32), (128, 136, 144), (100, 12000, 64), (128, 24008, 48),
          (128, 38016, 32), (300, 272, 144), (260, 2304, 96), (1000, 1032, 4096), (700, 2048, 128), (4097, 2304, 64),
          (8200, 2048, 32), (129, 64, 8192)]


def operands(M, N, K, seed, fmt=0, per_tensor=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    top = P.FMAX[fmt] / 8
    xq = (r(M, K) * top / 2).clamp(-P.FMAX[fmt], P.FMAX[fmt]).to(P.F8[fmt]).view(torch.uint8)
    wq = (r(N, K) * top / 2).clamp(-P.FMAX[fmt], P.FMAX[fmt]).to(P.F8[fmt]).view(torch.uint8)
    xs = torch.rand(1 if per_tensor else M, generator=g, device="cuda") + 0.5
    ws = torch.rand(1 if per_tensor else N, generator=g, device="cuda") + 0.5
    ws = ws * (8.0 / top / top / max(K, 1) ** 0.5)
    bias = (r(N) * 0.5).bfloat16()
    res = r(M, N).bfloat16()
    return xq, wq, xs, ws, bias, res


def plain(xq, wq, xs, ws, bias, fmt=0):
    x, w = P.dec(xq, fmt), P.dec(wq, fmt)
    s = xs.double().reshape(-1, 1) * ws.double().reshape(1, -1)
    z = (x @ w.t()) * s
    size = (x.abs() @ w.abs().t()) * s
    err = (xq.shape[1] / 32 + 1) * 2 * U * size + 4 * U * z.abs()
    if bias is not None:
        z = z + bias.double()
        err = err + 2 * U * z.abs()
    return z, err


def check(out, z, err, act, res):
    want = P.act(z, act)
    tol = P.act_tol(z, act, err)
    if res is not None:
        want = want + res.double()
        tol = tol + 2 * U * want.abs()
    tol = tol + P.half(torch.bfloat16) * (want.abs() + tol) + P.tiny(torch.bfloat16)
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), "%d off, worst %g of its bound" % (int((off > tol).sum()), float((off / tol).max()))


# up to 16 rows, K split over clusters of 8, 4 and 2: fewer K blocks than CTAs, an uneven split, ragged tiles of columns
SHAPES += [(1, 8, 64), (2, 16, 16), (4, 1184, 1040), (7, 2056, 208), (8, 4104, 1024), (9, 40, 8192), (12, 3000, 2064),
           (15, 9480, 1168), (16, 8192, 28672), (11, 1024, 4096), (16, 9472, 2048), (5, 18952, 400)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bias_activation_residual(shape):
    M, N, K = shape
    xq, wq, xs, ws, bias, res = operands(M, N, K, seed=N)
    for act, b, r in ((H.ACT_NONE, True, True), (H.ACT_GELU, True, False), (H.ACT_SILU, False, True)):
        z, err = plain(xq, wq, xs, ws, bias if b else None)
        guard = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = guard[:M * N].view(M, N)
        got = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias if b else None, act=act, residual=res if r else None, out=out)
        torch.cuda.synchronize()
        assert got is out and bool((guard[M * N:] == 7.0).all())
        check(out, z, err, act, res if r else None)
    H.hq_check_device_error()


@pytest.mark.parametrize("act", [H.ACT_NONE, H.ACT_RELU, H.ACT_GELU, H.ACT_GELU_TANH, H.ACT_SILU])
@pytest.mark.parametrize("shape", [(5, 32, 16), (16, 9504, 64), (64, 64, 512), (300, 288, 144), (700, 2048, 128),
                                   (3, 18976, 32), (120, 25600, 32), (4100, 2304, 64), (8200, 2048, 32)], ids=str)
def test_checkpoint(shape, act):
    M, N, K = shape
    xq, wq, xs, ws, bias, res = operands(M, N, K, seed=act)
    xq[0] = 0
    z, err = plain(xq, wq, xs, ws, bias)
    for z_fmt in (H.E4M3, H.E5M2):
        out, zq, zs = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=act, residual=res, ckpt=True, z_fmt=z_fmt)
        torch.cuda.synchronize()
        check(out, z, err, act, res)
        P.check_quantized(zq, zs, z, 32, z_fmt, 0.0, err)
    # the checkpoint does not change the result
    same = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=act, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(same, out)
    H.hq_check_device_error()


def test_no_activation_is_the_plain_gemm():
    # without activation and residual: bit for bit the existing epilogue, bias or not, on the same tiles (up to 16 rows
    # another kernel sums in another order)
    for M, N, K in ((17, 8192, 512), (300, 272, 144), (700, 2048, 128), (8200, 2048, 32)):
        xq, wq, xs, ws, bias, _ = operands(M, N, K, seed=K)
        assert torch.equal(H.hq_gemm_a8w8_act(xq, wq, xs, ws), H.hq_gemm_a8w8(xq, wq, xs, ws))
        assert torch.equal(H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias), H.hq_gemm_a8w8_ex(xq, wq, xs, ws, bias=bias))


def test_e5m2_operands_and_per_tensor_scales():
    xq, wq, xs, ws, bias, res = operands(130, 264, 272, seed=1, fmt=1, per_tensor=True)
    z, err = plain(xq, wq, xs, ws, bias, fmt=1)
    out = H.hq_gemm_a8w8_act(xq, wq, xs, ws, H.E5M2, bias=bias, act=H.ACT_GELU_TANH, residual=res)
    torch.cuda.synchronize()
    check(out, z, err, H.ACT_GELU_TANH, res)


@pytest.mark.parametrize("shape", [(16, 8192, 64), (300, 272, 144), (8200, 2048, 32), (37, 104, 32)], ids=str)
def test_residual_updated_in_place(shape):
    xq, wq, xs, ws, bias, res = operands(*shape, seed=2)
    want = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_SILU, residual=res)
    stream = res.clone()
    got = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_SILU, residual=stream, out=stream)
    torch.cuda.synchronize()
    assert got is stream and torch.equal(got, want)


def test_empty_k_and_empty_outputs():
    xq = torch.empty((5, 0), dtype=torch.uint8, device="cuda")
    wq = torch.empty((64, 0), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    bias = torch.randn(64, device="cuda").bfloat16()
    res = torch.randn(5, 64, device="cuda").bfloat16()
    out, zq, zs = H.hq_gemm_a8w8_act(xq, wq, one, one, bias=bias, act=H.ACT_RELU, residual=res, ckpt=True)
    torch.cuda.synchronize()
    z = bias.double().expand(5, 64)
    check(out, z, torch.zeros_like(z), H.ACT_RELU, res)
    P.check_quantized(zq, zs, z.contiguous(), 32, 0, 0.0)
    none = H.hq_gemm_a8w8_act(xq[:0], wq, one, one, act=H.ACT_GELU)
    assert none.shape == (0, 64)


def test_special_values_reach_the_checkpoint():
    # NaN and infinite operands (E5M2 codes hold both), an infinite bias, and a row that overflows
    M, N, K = 40, 96, 32
    xq, wq, xs, ws, bias, _ = operands(M, N, K, seed=3)
    xq[3, 5] = 0x7F                     # NaN: the row
    bias = bias.clone()
    bias[33] = float("inf")
    bias[70] = float("nan")
    z, err = plain(xq, wq, xs, ws, bias)
    err = torch.nan_to_num(err, 0.0, 0.0)
    out, zq, zs = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_RELU, ckpt=True)
    torch.cuda.synchronize()
    P.check_quantized(zq, zs, z, 32, 0, 0.0, err)
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(out[:, 70]).all())
    assert bool(torch.isinf(out[4:, 33]).all()) and bool((zs[3] == 1).all())
    fin = torch.isfinite(z)
    check(torch.where(fin, out, torch.zeros_like(out)), torch.where(fin, z, torch.zeros_like(z)),
          torch.where(fin, err, torch.zeros_like(err)), H.ACT_RELU, None)


def test_captured_graphs_and_another_stream():
    xq, wq, xs, ws, bias, res = operands(2048, 1024, 256, seed=4)
    want = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_GELU, residual=res, ckpt=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_GELU, residual=res, ckpt=True, stream=st)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_GELU, residual=res, ckpt=True)
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, got):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("shape", [(1, 8192, 1024), (16, 1024, 4096), (5, 4096, 400)], ids=str)
def test_decode_calls_on_two_streams_at_once(shape):
    # cluster launches of two graphs interleaved on two streams, the residual stream updated in place by each
    xq, wq, xs, ws, bias, res = operands(*shape, seed=5)
    want = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_GELU, residual=res)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, streams = [], [res.clone(), res.clone()]
    for s in streams:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s.copy_(res)
            H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_GELU, residual=s, out=s)
        graphs.append(gr)
    for _ in range(20):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(streams[0], want) and torch.equal(streams[1], want)
    H.hq_check_device_error()


def test_scales_and_bias_off_the_vector_grid():
    # column scales and bias that start 4 bytes off a 16-byte boundary, rows of out 16 bytes off a 32-byte one
    for M, N, K in ((3, 1024, 256), (40, 520, 64), (200, 264, 256), (700, 2048, 128)):
        xq, wq, xs, ws, bias, res = operands(M, N, K, seed=N)
        z, err = plain(xq, wq, xs, ws, bias)
        ws1 = torch.empty(N + 1, device="cuda")[1:].copy_(ws)
        bias1 = torch.empty(N + 2, dtype=torch.bfloat16, device="cuda")[2:].copy_(bias)
        out = torch.empty(M * N + 8, dtype=torch.bfloat16, device="cuda")[8:].view(M, N)
        res1 = torch.empty(M * N + 8, dtype=torch.bfloat16, device="cuda")[8:].view(M, N).copy_(res)
        H.hq_gemm_a8w8_act(xq, wq, xs, ws1, bias=bias1, act=H.ACT_SILU, residual=res1, out=out)
        torch.cuda.synchronize()
        check(out, z, err, H.ACT_SILU, res)
