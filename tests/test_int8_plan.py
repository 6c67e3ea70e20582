"""Which kernels the int8 product takes for the shapes that its GPU tests are made of: a test whose shape goes to
another kernel than the one that it was written for fails here.  The choice is host code of its own
(csrc/int8_plan.h), compiled here by itself."""
import os
import subprocess

import pytest

from int8_shapes import TILES, WIDE, pitch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <stdio.h>
#include "csrc/int8_plan.h"
int main() {
  gemm_int8_desc d{};
  long long v[5];
  int type;
  while (scanf("%lld %lld %lld %lld %lld %d", v, v + 1, v + 2, v + 3, v + 4, &type) == 6) {
    d.M = v[0], d.N = v[1], d.K = v[2], d.lda = v[3], d.ldb = v[4], d.dtype_c = type;
    const auto p = dg::plan_of(d);
    if (p.wide) printf("%dx%d%s", dg::kWide, dg::kWide, p.tiles >= 0 ? " " : "");
    if (p.tiles == -1) printf("few");
    if (p.tiles >= 0) printf("%dx%d", dg::kTiles[p.tiles].bm, dg::kTiles[p.tiles].bn);
    printf("%s\n", p.tiles >= 0 && p.splits > 1 ? " cut" : "");
  }
}
"""
BF16, F32 = 0, 2


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "dense_gemm_design_amd"), "-o", str(at / "plan"),
                    str(at / "plan.cpp")], check=True)

    def ask(M, N, K, pitch, out):
        run = subprocess.run([str(at / "plan")], input=f"{M} {N} {K} {pitch} {pitch} {out}", capture_output=True,
                             text=True, check=True)
        return run.stdout.strip()
    return ask


@pytest.mark.parametrize("M,N,K,start,kernel", WIDE + TILES)
def test_shapes_reach_their_kernels(chosen, M, N, K, start, kernel):
    for out in (BF16, F32):
        assert chosen(M, N, K, pitch(K, start), out) == kernel


def test_every_kernel_has_its_shapes():
    sizes = {f"{m}x{n}" for m, n in ((64, 64), (64, 128), (128, 128), (128, 192), (192, 128), (192, 192),
                                     (128, 256), (256, 128), (256, 256))}
    for start in {s[3] for s in TILES}:
        assert sizes | {"few"} <= {k for s in WIDE + TILES for k in s[4].split() if s[3] == start}
    rounds = {-(-(-(-M // 256) * -(-N // 256)) // 256) for M, N, _, _, k in WIDE if k == "256x256"}
    assert rounds == {1, 2, 3}


def test_larger_products_take_larger_tiles(chosen):
    """What the kernels' measured times lead to, at 4096 columns."""
    want = {1: "few", 32: "few", 64: "64x64", 256: "64x64", 1024: "128x128", 8192: "256x256"}
    for M, kernel in want.items():
        assert chosen(M, 4096, 4096, 4096, BF16).split()[0] == kernel, M
