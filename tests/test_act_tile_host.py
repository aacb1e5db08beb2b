"""The activation GEMM's choice of tile (csrc/act_tile.cuh), as plain C++ on
the CPU: any number of SMs gets a tile that it can run."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_dynamic_quantization_amax_b200", "csrc")

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


def test_any_number_of_sms(tmp_path):
    sms = list(range(1, 160))
    got = picks(tmp_path, [(692, 9208, 28352, s) for s in sms])
    assert all(0 <= p <= 4 for p in got) and got[0] <= 2 and len(got) == len(sms)
