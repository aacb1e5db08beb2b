"""The activation GEMM on every tile that ragged and middling shapes are given
(csrc/act_tile.cuh; tests/test_act_tile_host.py checks that these shapes get
them): a last tile that is ragged in M and N, K of many blocks, more tiles
than run at once, with bias, residual, in place and with the checkpoint.
Bounds as in tests/test_gemm_act_gpu.py."""
import pytest
import torch

from fp8_dynamic_quantization_amax_b200 import _hq as H
import _plain as P
from test_gemm_act_gpu import check, operands, plain

pytestmark = pytest.mark.gpu

SHAPES = [("64", 133, 264, 1840), ("64", 129, 12320, 144), ("128", 2047, 1032, 2064), ("128", 900, 4640, 144),
          ("256", 257, 12328, 2064), ("256", 1100, 6432, 144), ("pair256", 1388, 1880, 4560),
          ("pair256", 133, 24416, 4112), ("pair512", 700, 6440, 16400), ("pair512", 2047, 8992, 28352)]


@pytest.mark.parametrize("tile,M,N,K", SHAPES, ids=str)
def test_ragged_tiles(tile, M, N, K):
    xq, wq, xs, ws, bias, res = operands(M, N, K, seed=N)
    z, err = plain(xq, wq, xs, ws, bias)
    guard = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[:M * N].view(M, N)
    H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_SILU, residual=res, out=out)
    torch.cuda.synchronize()
    assert bool((guard[M * N:] == 7.0).all())
    check(out, z, err, H.ACT_SILU, res)
    stream = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    stream[:M * N] = res.reshape(-1)
    same = stream[:M * N].view(M, N)
    H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_SILU, residual=same, out=same)
    torch.cuda.synchronize()
    assert torch.equal(same, out) and bool((stream[M * N:] == 7.0).all())
    if N % 32 == 0:
        zq = torch.full((M * N + 64,), 0x55, dtype=torch.uint8, device="cuda")
        zs = torch.full((M * N // 32 + 16,), 7.0, device="cuda")
        got = H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias, act=H.ACT_GELU, z_q=zq[:M * N].view(M, N),
                                 z_scales=zs[:M * N // 32].view(M, N // 32))
        torch.cuda.synchronize()
        check(got[0], z, err, H.ACT_GELU, None)
        P.check_quantized(got[1], got[2], z, 32, H.E4M3, 0.0, err)
        assert bool((zq[M * N:] == 0x55).all()) and bool((zs[M * N // 32:] == 7.0).all())
    H.hq_check_device_error()


@pytest.mark.parametrize("tile,M,N,K", [s for s in SHAPES if s[1] * s[2] * s[3] < 1 << 37], ids=str)
def test_the_same_bits_as_without_activation(tile, M, N, K):
    # no activation, no residual: bit for bit the plain epilogue's result, on whichever tile that takes; and again from
    # two graphs replayed at once
    xq, wq, xs, ws, bias, _ = operands(M, N, K, seed=K)
    want = H.hq_gemm_a8w8_ex(xq, wq, xs, ws, bias=bias)
    assert torch.equal(H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias), want)
    graphs, outs, side = [], [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(H.hq_gemm_a8w8_act(xq, wq, xs, ws, bias=bias))
        graphs.append(gr)
    for _ in range(5):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    H.hq_check_device_error()
