"""Plain 64-bit forms of the feed-forward operators and the error bounds their
tests use.  torch float64 on whatever device the inputs are on; written from
the definitions in include/hq.h, sharing no code with the CUDA path.

Bounds: U = 2^-24 is f32's largest relative rounding error, half(t) an output
type's.  A result may be off by half a step of its type beyond what the f32
arithmetic ahead of it can be off, which each test counts.
"""
import math

import torch

U = 2.0 ** -24
FMAX = (448.0, 57344.0)                 # E4M3, E5M2
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
MANT = (3, 2)
EMIN = (-6, -14)
ACTS = {1: "relu", 2: "gelu", 3: "gelu_tanh", 4: "silu"}


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the smallest step (subnormal) of a type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def dec(codes, fmt):
    return codes.view(F8[fmt]).double()


def sum_depth(cols):
    """Terms a f32 row sum passes through at most: 256 threads' strided sums, then the joins."""
    return cols / 256 + 48


def group_index(cols, block):
    return torch.arange(cols, device="cuda") // (block if block else cols)


def finite_amax(y, block):
    """Per row and block: the largest finite |y| (0 where there is none)."""
    rows, cols = y.shape
    idx = group_index(cols, block).to(y.device)
    a = torch.where(torch.isfinite(y), y.abs(), torch.zeros_like(y))
    out = torch.zeros((rows, int(idx[-1]) + 1), dtype=y.dtype, device=y.device)
    return out.scatter_reduce(1, idx.expand(rows, cols), a, "amax"), idx


def check_quantized(q, scales, y, block, fmt, rel, absolute=0.0):
    """Codes and scales against 64-bit y (finite or not), y itself being off
    by up to rel * |y| + absolute (a number, or a tensor like y) in f32."""
    rows, cols = y.shape
    if rows == 0:
        return
    absolute = torch.as_tensor(absolute, dtype=torch.float64, device=y.device).expand(rows, cols)
    amax, idx = finite_amax(y, block)
    nb = amax.shape[1]
    want = torch.where(amax > 0, amax / FMAX[fmt], torch.ones_like(amax))
    a_abs = torch.zeros_like(amax).scatter_reduce(1, idx.expand(rows, cols), absolute.contiguous(), "amax")
    got = scales.double().reshape(rows, nb)
    # the quotient and its reciprocal round once each
    tol = want * (rel + 3 * U) + a_abs / FMAX[fmt]
    assert bool(((got - want).abs() <= tol).all()), ((got - want).abs() / want).max()
    nan = torch.isnan(y)
    code = q.to(torch.int32)
    assert bool((code[nan] == 0x7F).all())
    inf = torch.isinf(y)
    big = (0x7E, 0x7B)[fmt]
    assert bool((code[inf] == torch.where(y[inf] > 0, big, big + 128)).all())
    fin = ~(nan | inf)
    s = got[:, idx]
    t = torch.where(fin, y / s, torch.zeros_like(y))          # the value the codes stand for, by the scale given out
    e = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -60))).clamp(min=EMIN[fmt])
    step = torch.exp2(e - MANT[fmt])
    err = torch.where(fin, (dec(q, fmt) - t).abs(), torch.zeros_like(t))
    # y m in f32 with m = 1/s to two roundings, then half a step of the format;
    # the largest element of a block may round above fmax and is held there
    bad = err > step / 2 + t.abs() * (rel + 4 * U) + absolute / s
    assert not bool(bad.any()), "codes off: %d, worst %g" % (int(bad.sum()), float((err - step / 2).max()))


def act(z, a):
    if a == 1:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if a == 2:
        return z * torch.special.ndtr(z)
    if a == 3:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if a == 4:
        return z * torch.sigmoid(z)
    return z


def act_slope(z, a):
    if a == 1:
        return (z > 0).to(z.dtype)
    if a == 2:
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    x, du = z, torch.ones_like(z)
    if a == 3:
        x = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    return torch.sigmoid(x) + z * du * torch.sigmoid(x) * torch.sigmoid(-x)


# Absolute error of the f32 slope: 7.5e-8 of the erf approximation; the slope
# is s + z x' e s s with e off by (4 |x| + 4) U and s by 2 U + (1 - s) of
# that, and |x z x' s (1 - s)| <= 1.3, |z x' s (1 - s)| <= 0.5: below 24 U.
SLOPE_TOL = 7.5e-8 + 24 * U


def act_tol(z, a, dz):
    """Error of act(z) in f32 for z off by dz: slopes are at most 1.13 in
    size; the erf form is off by 7.5e-8 |z|; sigmoid's argument is off by
    4 U |x|, so s (and the result) by (4 |x| + 8) U of itself."""
    out = act(z, a).abs()
    t = 1.13 * dz + 4 * U * out
    if a == 2:
        t = t + 7.5e-8 * z.abs() + (z * z + 12) * U * out
    if a in (3, 4):
        x = z if a == 4 else 1.6 * (z + 0.044715 * z ** 3)
        t = t + (4 * x.abs() + 8) * U * out
    return t
