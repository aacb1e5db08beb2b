"""A feed-forward block on the FP8 path, forward and backward, through the
binding as a user chains it: norm (with the residual) -> up projection with
activation and checkpoint -> quantize -> down projection onto the residual
stream; then the activation's backward from the checkpoint, the weight and
input gradients through the quantize and the GEMM, and the norm's backward.

The references are 64-bit and take the quantized operands that the path
itself consumed, so each step is held to its own arithmetic; the whole
backward pass is compared with the derivative of the unquantized block
within the FP8 error.
"""
import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H
import _plain as P

pytestmark = pytest.mark.gpu

TOKENS, DIM, HIDDEN, EPS = 272, 256, 1024, 1e-5


def params(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    return {"x": n(TOKENS, DIM), "res": n(TOKENS, DIM, std=2.0), "gain": n(DIM, std=0.1) + 1, "up": n(HIDDEN, DIM, std=0.06),
            "bias": n(HIDDEN, std=0.1), "down": n(DIM, HIDDEN, std=0.03), "dout": n(TOKENS, DIM, std=0.01)}


def forward(p, act):
    s = {"rstd": torch.empty(TOKENS, device="cuda"), "y": torch.empty_like(p["x"])}
    s["yq"], s["ys"], s["h"] = H.hq_rmsnorm_fp8(p["x"], p["gain"], EPS, residual=p["res"], y_out=s["y"], rstd_out=s["rstd"])
    s["uq"], s["us"] = H.hq_quantize_fp8(p["up"], gran=H.PER_TOKEN)
    s["a"], s["zq"], s["zs"] = H.hq_gemm_a8w8_act(s["yq"], s["uq"], s["ys"], s["us"], bias=p["bias"], act=act, ckpt=True)
    s["aq"], s["as"] = H.hq_quantize_fp8(s["a"], gran=H.PER_TOKEN)
    s["dq"], s["ds"] = H.hq_quantize_fp8(p["down"], gran=H.PER_TOKEN)
    s["out"] = H.hq_gemm_a8w8_act(s["aq"], s["dq"], s["as"], s["ds"], residual=s["h"])
    return s


def linear_backward(g, w, x):
    """dX = g . w and dW = g^T . x of a layer x [M, K], w [N, K], g [M, N] on transposed FP8 codes."""
    gq, gt, gs = H.hq_quantize_fp8_transpose(g, H.E4M3, q=True)
    _, wt, ws = H.hq_quantize_fp8_transpose(w, H.E4M3)
    _, xt, xs = H.hq_quantize_fp8_transpose(x, H.E4M3)
    return H.hq_gemm_a8w8(gq, wt, gs, ws), H.hq_gemm_a8w8(gt, xt, gs, xs)


def backward(p, s, act):
    da, ddown = linear_backward(p["dout"], p["down"], s["a"])
    dz, dbias = H.hq_act_backward_fp8(da, s["zq"], s["zs"], act)
    dy, dup = linear_backward(dz, p["up"], s["y"])
    dx, dgain = H.hq_rmsnorm_backward(dy, s["h"], p["gain"], s["rstd"], dres=p["dout"])
    return {"x": dx, "gain": dgain, "up": dup, "bias": dbias, "down": ddown, "da": da, "dz": dz, "dy": dy}


@pytest.mark.parametrize("act", [H.ACT_RELU, H.ACT_GELU, H.ACT_GELU_TANH, H.ACT_SILU])
def test_block_forward_and_backward(act):
    p = params(act)
    s = forward(p, act)
    g = backward(p, s, act)
    torch.cuda.synchronize()
    H.hq_check_device_error()
    # each product from the codes it consumed; half a bf16 step and the f32 accumulation
    dec = lambda q, sc: P.dec(q, 0) * sc.double().reshape(-1, 1)  # noqa: E731
    z = dec(s["yq"], s["ys"]) @ dec(s["uq"], s["us"]).t() + p["bias"].double()
    size = dec(s["yq"], s["ys"]).abs() @ dec(s["uq"], s["us"]).abs().t()
    err = (DIM / 32 + 1) * 2 * P.U * size + 6 * P.U * z.abs()
    want = P.act(z, act)
    tol = P.act_tol(z, act, err) + P.half(torch.bfloat16) * want.abs() * 1.01 + 1e-30
    assert bool(((s["a"].double() - want).abs() <= tol).all())
    P.check_quantized(s["zq"], s["zs"], z, 32, 0, 0.0, err)
    o = dec(s["aq"], s["as"]) @ dec(s["dq"], s["ds"]).t() + s["h"].double()
    osize = dec(s["aq"], s["as"]).abs() @ dec(s["dq"], s["ds"]).abs().t()
    tol = (HIDDEN / 32 + 1) * 2 * P.U * osize + (P.half(torch.bfloat16) * 1.01 + 8 * P.U) * o.abs()
    assert bool(((s["out"].double() - o).abs() <= tol).all())
    # the whole against autograd of the unquantized block in 64 bits, with `h` as stored
    leaf = {k: p[k].double().requires_grad_() for k in ("gain", "up", "bias", "down")}
    h = s["h"].double().requires_grad_()
    y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * leaf["gain"]
    out = P.act(y @ leaf["up"].t() + leaf["bias"], act) @ leaf["down"].t() + h
    out.backward(p["dout"].double())
    leaf["x"] = h
    for k in ("x", "gain", "up", "bias", "down"):
        ref = leaf[k].grad
        # E4M3 products: every operand is off by up to 2^-4 of itself, independently: the result by some 3 % of its
        # norm per product, through at most four of them
        rel = float((g[k].double() - ref).norm() / ref.norm())
        assert rel <= 4 * 2.0 ** -4, (k, rel)


def test_block_captured_with_updates_in_place():
    # a whole step in one graph: the residual stream updated in place by the norm and by the down projection
    p = params(9)
    s = forward(p, H.ACT_GELU)
    want = backward(p, s, H.ACT_GELU)
    uq, us = H.hq_quantize_fp8(p["up"], gran=H.PER_TOKEN)
    dq, ds = H.hq_quantize_fp8(p["down"], gran=H.PER_TOKEN)
    stream = p["res"].clone()

    def step():
        yq, ys, h = H.hq_rmsnorm_fp8(p["x"], p["gain"], EPS, residual=stream, residual_out=stream)
        a = H.hq_gemm_a8w8_act(yq, uq, ys, us, bias=p["bias"], act=H.ACT_GELU)
        aq, as_ = H.hq_quantize_fp8(a, gran=H.PER_TOKEN)
        return H.hq_gemm_a8w8_act(aq, dq, as_, ds, residual=h, out=h)

    step()
    torch.cuda.synchronize()
    assert torch.equal(stream, s["out"])
    stream.copy_(p["res"])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
        got = backward(p, s, H.ACT_GELU)
    for _ in range(2):
        stream.copy_(p["res"])
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, s["out"])
        for k in want:
            assert torch.equal(got[k], want[k]), k


def test_decode_step_of_one_token():
    # one row through the forward chain is that row of the batch: every scale is per token
    p = params(10)
    s = forward(p, H.ACT_SILU)
    for r in (0, 100, TOKENS - 1):
        yq, ys, h = H.hq_rmsnorm_fp8(p["x"][r:r + 1], p["gain"], EPS, residual=p["res"][r:r + 1])
        torch.cuda.synchronize()
        assert torch.equal(h, s["h"][r:r + 1])
        # a row alone may be summed in another order: its codes are the batch's or the neighbours
        one, many = P.dec(yq, 0) * ys.double(), P.dec(s["yq"][r:r + 1], 0) * s["ys"][r].double()
        assert bool(((one - many).abs() <= 2.0 ** -3 * many.abs() + 2.0 ** -9 * float(ys)).all())
        yq, ys = s["yq"][r:r + 1], s["ys"][r:r + 1]
        a = H.hq_gemm_a8w8_act(yq, s["uq"], ys, s["us"], bias=p["bias"], act=H.ACT_SILU)
        # another tile adds the products in another grouping: the same value within the accumulation's error
        torch.cuda.synchronize()
        assert float((a.float() - s["a"][r:r + 1].float()).abs().max()) <= 2.0 ** -7 * float(s["a"][r].float().abs().max())


FIRST_CALLS = """
import torch
import fp8_dynamic_quantization_amax_b200 as H
n = lambda *s: torch.randn(s, device="cuda").bfloat16()
x, w, rstd = n(64, 1024), n(1024), torch.rand(64, device="cuda")
q = torch.randint(0, 100, (64, 1024), dtype=torch.uint8, device="cuda")
wq = torch.randint(0, 100, (2048, 1024), dtype=torch.uint8, device="cuda")
one, zs = torch.ones(1, device="cuda"), torch.rand(64, 32, device="cuda")

def calls():
    return [*H.hq_rmsnorm_fp8(x, w, 1e-5)[:2], *H.hq_rmsnorm_backward(x, x, w, rstd), *H.hq_act_backward_fp8(x, q, zs, 2),
            H.hq_gemm_a8w8_act(q, wq, one, one, act=2), H.hq_gemm_a8w8_act(q[:3], wq, one, one, act=2)]

torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    got = calls()
gr.replay()
torch.cuda.synchronize()
again = calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, again))
H.hq_check_device_error()
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    # kernels set up and loaded while a stream is being captured
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
