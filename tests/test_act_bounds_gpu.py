"""The activations and their slopes against 64 bits, each within the bound of
its own arithmetic (csrc/act.cuh), on the GPU.

Counted in U = 2^-24, f32's largest relative rounding error.  The erf GELU,
with a = |z| held at 5.6 and e = e^(-z^2 / 2):
  e      the hardware exp2's 2 ulp (4 U) and three roundings of its argument
         z^2 / 2: (4 + 1.5 z^2) U of itself
  slope  1/2 +- (1/2 - e Q): the polynomial's e |error| (1.13e-8 for f32, 2.72e-7
         for 16-bit gradients), its Horner steps (0.76 U), |e Q| (4 + 1.5 z^2) U
         <= 2 U, the difference (0.63 U) and the sum (1.13 U)
  value  max(z, 0) - a e P: the polynomial's a e |error| (9.0e-8), its Horner
         steps (0.89 U), a e P (5 + 1.5 z^2) U <= 1.1 U, one rounding
ReLU's slope is 0 or 1: dz is g or 0.  The sigmoid forms' slopes are counted in
tests/_plain.py (24 U).
"""
import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H
import _plain as P

pytestmark = pytest.mark.gpu
U = P.U
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def slope_bound(act, dtype):
    if act == H.ACT_RELU:
        return 0.0
    if act == H.ACT_GELU:
        return (1.13e-8 if dtype == torch.float32 else 2.72e-7) + (0.76 + 2 + 0.63 + 1.13) * U
    return 24 * U


def checkpoint(rows, cols, seed, std=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn((rows, cols), generator=g, device="cuda") * std
    zq, zs = H.hq_quantize_fp8_blockwise(z, H.E4M3, 32)
    # the value that the derivative is taken at: one f32 product
    zz = (P.dec(zq, 0).float() * zs[:, P.group_index(cols, 32)]).double()
    return zq, zs, zz, torch.randn((rows, cols), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", [H.ACT_RELU, H.ACT_GELU, H.ACT_GELU_TANH, H.ACT_SILU])
def test_slope_of_each_activation(act, dtype):
    zq, zs, z, g = checkpoint(515, 2064, seed=act)
    g = g.to(dtype)
    dz, _ = H.hq_act_backward_fp8(g, zq, zs, act, need_dbias=False)
    torch.cuda.synchronize()
    want = g.double() * P.act_slope(z, act)
    unit = slope_bound(act, dtype)
    # the f32 product, then the rounding to g's type (in f32 the same one; ReLU's product is exact)
    once = 0.0 if act == H.ACT_RELU else U if dtype == torch.float32 else U + P.half(dtype)
    tol = g.double().abs() * unit * (1 + once) + want.abs() * once + (0.0 if act == H.ACT_RELU else P.tiny(dtype))
    off = (dz.double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


def test_gelu_slope_in_f32_is_as_exact_as_plain_f32():
    zq, zs, z, _ = checkpoint(512, 4096, seed=7)
    one = torch.ones(z.shape, device="cuda")
    dz, _ = H.hq_act_backward_fp8(one, zq, zs, H.ACT_GELU, need_dbias=False)
    torch.cuda.synchronize()
    want = P.act_slope(z, H.ACT_GELU)
    norm = lambda t: float(t.double().norm() / want.norm())  # noqa: E731
    x = z.float()
    plain = 0.5 * (1.0 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (0.5 / torch.pi) ** 0.5
    off, theirs = norm(dz.double() - want), norm(plain.double() - want)
    # rounding the slope once costs up to U of its norm: twice that, and twice plain f32's error
    assert off <= 2 * U, off
    assert off <= 2 * theirs, (off, theirs)


def test_gelu_slope_at_zero_is_one_half():
    # codes 0x00 and 0x80 (plus and minus zero); the bias gradient of one row is dz
    codes = torch.tensor([0x00, 0x80] * 8, dtype=torch.uint8, device="cuda")[None]
    g = torch.linspace(-3, 5, 16, device="cuda")[None]
    dz, db = H.hq_act_backward_fp8(g, codes, torch.ones((1, 1), device="cuda"), H.ACT_GELU, block=16)
    torch.cuda.synchronize()
    assert torch.equal(dz, g / 2) and torch.equal(db, dz[0])


@pytest.mark.parametrize("rows", [5, 40, 300])
@pytest.mark.parametrize("act", [H.ACT_NONE, H.ACT_RELU, H.ACT_GELU, H.ACT_GELU_TANH, H.ACT_SILU])
def test_value_at_every_bf16(act, rows):
    # without columns of K the product is 0 and z the bias: every finite bf16, through the GEMM's kernels
    bits = torch.arange(65536, device="cuda").to(torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80].to(torch.int16)
    z16 = bits.view(torch.bfloat16).reshape(8, 8160)
    one = torch.ones(1, device="cuda")
    xq = torch.empty((rows, 0), dtype=torch.uint8, device="cuda")
    wq = torch.empty((8160, 0), dtype=torch.uint8, device="cuda")
    for bias in z16:
        out = H.hq_gemm_a8w8_act(xq, wq, one, one, bias=bias.contiguous(), act=act)
        torch.cuda.synchronize()
        assert torch.equal(out, out[:1].expand_as(out))
        z = bias.double()
        want = P.act(z, act)
        tol = torch.zeros_like(z)
        if act == H.ACT_GELU:
            tol = 9.0e-8 + (0.89 + 1.1) * U + U * want.abs()
        elif act in (H.ACT_GELU_TANH, H.ACT_SILU):
            x = z if act == H.ACT_SILU else 1.6 * (z + 0.044715 * z ** 3)
            # the argument: seven roundings of its products and constants, each U |x| of the sigmoid at most;
            # beyond x = -87.3 that leaves f32's normal numbers (1.2e-38) and is 0; |z| is below 88 there
            tol = (8 * x.abs().clamp(max=90) + 8) * U * want.abs() + 1.1e-36
        # none and ReLU: z or 0, as it is
        if act not in (H.ACT_NONE, H.ACT_RELU):
            tol = tol + P.half(torch.bfloat16) * (want.abs() + tol) + P.tiny(torch.bfloat16)
        off = (out[0].double() - want).abs()
        assert bool((off <= tol).all()), (float(bias[(off - tol).argmax()]), float((off - tol).max()))
