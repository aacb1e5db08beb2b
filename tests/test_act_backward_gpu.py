"""The activation's backward pass from the 8-bit checkpoint, with the bias
gradient, on the GPU against the 64-bit plain forms of tests/_plain.py."""
import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H
import _plain as P

pytestmark = pytest.mark.gpu
U = P.U
ACTS = [H.ACT_RELU, H.ACT_GELU, H.ACT_GELU_TANH, H.ACT_SILU]
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def inputs(rows, cols, dtype, fmt, block, seed, std=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn((rows, cols), generator=g, device="cuda") * std
    zq, zs = H.hq_quantize_fp8_blockwise(z, fmt, block)
    return (torch.randn((rows, cols), generator=g, device="cuda")).to(dtype), zq, zs


def check(g, zq, zs, act, fmt, block, dz, db):
    rows, cols = g.shape
    idx = P.group_index(cols, block)
    z = P.dec(zq, fmt) * zs.double()[:, idx]
    want = g.double() * P.act_slope(z, act)
    # z is off by U |z| (slopes change by at most 0.8 per unit of z, 1.1 in the tanh form, and
    # |z| times that stays below 2 where it is not 0), the slope by SLOPE_TOL, the product rounds once
    unit = P.SLOPE_TOL + 4 * U
    off = (dz.double() - want).abs()
    tol = g.double().abs() * unit + P.half(g.dtype) * want.abs() + P.tiny(g.dtype)
    assert bool((off <= tol).all()), float((off / tol).max())
    if db is not None:
        total = want.sum(0)
        # a lane's rows in order (an eighth of a band), eight warps, the bands in eighths
        depth = rows / 64 + 64
        tol = (unit + depth * U) * g.double().abs().sum(0) * 1.2 + P.half(db.dtype) * total.abs() + P.tiny(db.dtype)
        assert bool(((db.double() - total).abs() <= tol).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,block", [((1, 16), 16), ((3, 16), 32), ((1, 4096), 32), ((65, 272), 32), ((2047, 528), 128),
                                         ((300, 1040), 48), ((33, 8192), 8192), ((1000, 64), 64), ((5, 28672), 32)],
                         ids=str)
def test_against_64_bits(shape, block, dtype, act):
    for fmt in (H.E4M3, H.E5M2):
        g, zq, zs = inputs(*shape, dtype, fmt, block, seed=shape[0] + act)
        dz, db = H.hq_act_backward_fp8(g, zq, zs, act, fmt, block)
        torch.cuda.synchronize()
        check(g, zq, zs, act, fmt, block, dz, db)
        dz2, db2 = H.hq_act_backward_fp8(g, zq, zs, act, fmt, block)        # a fixed order: the same bits
        dz3, none = H.hq_act_backward_fp8(g, zq, zs, act, fmt, block, need_dbias=False)
        own = g.clone()
        dz4, db4 = H.hq_act_backward_fp8(own, zq, zs, act, fmt, block, dz=own)   # in place
        torch.cuda.synchronize()
        assert torch.equal(dz, dz2) and torch.equal(db, db2) and torch.equal(dz, dz3) and none is None
        assert dz4 is own and torch.equal(dz, dz4) and torch.equal(db, db4)


@pytest.mark.parametrize("act", ACTS)
def test_every_code_and_extreme_scales(act):
    # all 256 codes in a row, at scales from where z is tiny to where e^-z overflows; NaN codes give NaN alone
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(7, 1)
    scale = torch.tensor([1e-30, 1e-3, 0.01, 0.1, 1.0, 1e5, 1e34], device="cuda")
    zs = scale[:, None].expand(7, 16).contiguous()
    g = torch.ones((7, 256), device="cuda")
    for fmt in (H.E4M3, H.E5M2):
        dz, _ = H.hq_act_backward_fp8(g, codes, zs, act, fmt, 16)
        torch.cuda.synchronize()
        z = (P.dec(codes, fmt) * scale[:, None].double()).float().double()   # f32: may overflow to infinity
        nan = torch.isnan(z)
        assert bool((torch.isnan(dz) == nan).all())
        lim = z.clamp(-80, 80)
        want = torch.where(z.abs() > 80, (z > 0).double(), P.act_slope(lim, act))
        off = (dz.double() - want).abs()[~nan]
        assert float(off.max()) <= P.SLOPE_TOL + 8 * U


def test_infinite_and_nan_gradients():
    g, zq, zs = inputs(40, 64, torch.bfloat16, 0, 32, seed=1)
    g[3, 7], g[4, 8] = float("inf"), float("nan")
    dz, db = H.hq_act_backward_fp8(g, zq, zs, H.ACT_GELU, 0, 32)
    torch.cuda.synchronize()
    assert bool(torch.isnan(dz[4, 8])) and bool(torch.isnan(db[8])) and not bool(torch.isfinite(dz[3, 7]))
    fin = torch.ones((40, 64), dtype=torch.bool, device="cuda")
    fin[3, 7] = fin[4, 8] = False
    assert bool(torch.isfinite(dz[fin]).all())
    keep = [c for c in range(64) if c not in (7, 8)]
    assert bool(torch.isfinite(db[keep]).all())


def test_no_rows_writes_a_zero_bias_gradient():
    g = torch.empty((0, 48), device="cuda")
    db = torch.full((48,), 3.0, device="cuda")
    dz, db = H.hq_act_backward_fp8(g, torch.empty((0, 48), dtype=torch.uint8, device="cuda"),
                                   torch.empty((0, 2), device="cuda"), H.ACT_SILU, dbias=db)
    torch.cuda.synchronize()
    assert dz.shape == (0, 48) and bool((db == 0).all())


def test_slope_is_the_difference_quotient_of_the_forward_pass():
    # act'(z) against (act(z + t) - act(z - t)) / 2t of the 64-bit activation; off by t^2 / 6 * |act'''| (< 4) and
    # 2^-52 |act| / t
    z = torch.linspace(-6, 6, 512, device="cuda").reshape(2, 256)
    zq, zs = H.hq_quantize_fp8_blockwise(z, H.E4M3, 32)
    zz = P.dec(zq, 0) * zs.double()[:, P.group_index(256, 32)]
    t = 1e-5
    for act in (H.ACT_GELU, H.ACT_GELU_TANH, H.ACT_SILU):
        num = (P.act(zz + t, act) - P.act(zz - t, act)) / (2 * t)
        dz, _ = H.hq_act_backward_fp8(torch.ones_like(z), zq, zs, act, need_dbias=False)
        torch.cuda.synchronize()
        assert float((dz.double() - num).abs().max()) <= P.SLOPE_TOL + 8 * U + 1e-9


def test_offsets_past_32_bits():
    rows, cols = 80000, 28672   # elements past 2^31
    g = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    zq = torch.randint(0, 120, (rows, cols), dtype=torch.uint8, device="cuda")
    zs = torch.full((rows, cols // 32), 0.01, device="cuda")
    dz, db = H.hq_act_backward_fp8(g, zq, zs, H.ACT_SILU)
    torch.cuda.synchronize()
    for lo in (0, 74890, rows - 2):
        sub, _ = H.hq_act_backward_fp8(g[lo:lo + 2], zq[lo:lo + 2], zs[lo:lo + 2], H.ACT_SILU, need_dbias=False)
        assert torch.equal(dz[lo:lo + 2], sub)
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(total)
    for lo in range(0, rows, 4000):
        z = P.dec(zq[lo:lo + 4000], 0).mul_(float(zs[0, 0]))
        total += P.act_slope(z, H.ACT_SILU).mul_(g[lo:lo + 4000]).sum(0)
        size += g[lo:lo + 4000].double().abs_().sum(0)
    tol = (P.SLOPE_TOL + 4 * U + (rows / 64 + 64) * U) * 1.2 * size + P.half(db.dtype) * total.abs()
    assert bool(((db.double() - total).abs() <= tol).all())


def test_captured_graphs_replayed_at_once():
    g, zq, zs = inputs(2000, 1024, torch.bfloat16, 0, 32, seed=2)
    want = H.hq_act_backward_fp8(g, zq, zs, H.ACT_GELU)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = H.hq_act_backward_fp8(g, zq, zs, H.ACT_GELU, stream=st)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(H.hq_act_backward_fp8(g, zq, zs, H.ACT_GELU))
        graphs.append(gr)
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(st):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs + [other]:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
