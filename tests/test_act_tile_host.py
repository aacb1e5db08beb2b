"""The activation GEMM's choice of tile (csrc/act_tile.cuh), as plain C++ on
the CPU: the GPU tests' shapes reach every tile, and any number of SMs gets
one that it can run."""
import os
import subprocess

import test_gemm_act_tiles_gpu as G

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_dynamic_quantization_amax_b200", "csrc")
TILES = {"64": (0, 128, 64, 1), "128": (1, 128, 128, 1), "256": (2, 128, 256, 1), "pair256": (3, 256, 256, 2),
         "pair512": (4, 256, 512, 2)}

PROGRAM = r"""
#include "act_tile.cuh"
#include <cstdio>
int main() {
  long long m, n, k, sms;
  while (std::scanf("%lld %lld %lld %lld", &m, &n, &k, &sms) == 4)
    std::printf("%d\n", static_cast<int>(hq::pick_act_tile(m, n, (k + 127) / 128, sms)));
}
"""


def picks(tmp_path, calls):
    src, exe = tmp_path / "tile.cpp", tmp_path / "tile"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    text = "".join("%d %d %d %d\n" % c for c in calls)
    r = subprocess.run([str(exe)], input=text, capture_output=True, text=True)
    assert r.returncode == 0, r.returncode
    return [int(v) for v in r.stdout.split()]


def test_the_gpu_shapes_reach_every_tile(tmp_path):
    got = picks(tmp_path, [(m, n, k, 148) for _, m, n, k in G.SHAPES])
    seen = {}
    for (name, m, n, k), p in zip(G.SHAPES, got):
        tile, rows, cols, sms = TILES[name]
        assert p == tile, (name, m, n, k, p)
        # not for the rules ahead of it: few rows, or whole CTA-pair tiles
        assert m > 128 and not (n % 256 == 0 and n >= 2048 and (m >= 4096 or (m >= 512 and m * n * k >= 2 ** 37)))
        assert m % rows != 0 and n % cols != 0          # a ragged last tile both ways
        tiles = -(-m // rows) * -(-n // cols)
        seen.setdefault(name, set()).update({"blocks" if n % 32 == 0 else "pieces" if n % 16 else "sectors",
                                             "rounds" if tiles > 148 // sms else "one", "deep" if k > 1024 else "short"})
    for name in TILES:  # a checkpoint's whole blocks, rows off 32-byte sectors, more tiles than run at once, many K blocks
        assert {"blocks", "pieces", "rounds", "deep"} <= seen[name], (name, seen[name])


def test_any_number_of_sms(tmp_path):
    sms = list(range(1, 160))
    got = picks(tmp_path, [(692, 9208, 28352, s) for s in sms])
    assert all(0 <= p <= 4 for p in got) and got[0] <= 2 and len(got) == len(sms)
