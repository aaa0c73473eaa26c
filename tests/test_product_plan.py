"""Which tiles the layer's products take, asked of the library's own rule on the host (no GPU): the sizes that stand for
a way of working in the GPU tests do run by it."""
import os
import shutil
import subprocess

import pytest

import product_tiles

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
DRIVER = r"""
#include <stdio.h>
#include <stdlib.h>
#include "gdn_mm.h"
// lines of: kind scales M N K segments outputs turned two-sided pairs
int main() {
    long long kind, sc, M, N, K, segs, outs, turned, dual, pairs;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &kind, &sc, &M, &N, &K, &segs, &outs, &turned, &dual, &pairs) == 10) {
        const gdn::MmPlan r = gdn::mm_plan((int)kind, (int)sc, M, N, K, (int)segs, (int)outs, turned, dual, pairs);
        printf("%d %d %d %d %zu\n", r.few, r.bm, r.splits, r.share, r.bytes);
    }
}
"""
BF16, F32, F8, F8X = 0, 1, 2, 3
PLAIN, BLOCK, GROUP, ROW = 0, 1, 2, 3


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not shutil.which(HIPCC):
        pytest.skip("hipcc not installed")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(DRIVER)
    subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-w", "-I",
                    os.path.join(ROOT, "gated_deltanet_chunked_04_amd", "csrc"), "-I", os.path.join(ROOT, "include"), str(at / "plan.cpp"),
                    "-o", str(at / "plan")], check=True, capture_output=True, text=True)

    def ask(kind, sc, M, N, K, segs=1, outs=1, turned=False, dual=False, pairs=False):
        line = " ".join(str(int(v)) for v in (kind, sc, M, N, K, segs, outs, turned, dual, pairs))
        out = subprocess.run([str(at / "plan")], input=line, capture_output=True, text=True, check=True).stdout.split()
        return dict(zip(("few", "rows", "splits", "share", "bytes"), map(int, out)))

    return ask


def tall(p):
    return not p["few"] and p["rows"] == 256 and not p["splits"]


def test_tall_tiles(plan):
    for M, N, K in product_tiles.MATMUL:
        assert K % 16 == 0 and K % 128 and K > 8 * 128 and M % 256 and N % 256
        for sc in (BLOCK, GROUP, ROW):
            assert tall(plan(F8, sc, M, N, K))
    for M, K, F in product_tiles.FFN8:
        assert K % 16 == 0 and K % 128 and K > 8 * 128 and M % 256 and F % 128
        assert tall(plan(F8, BLOCK, M, F, K, dual=True))
    for M, K, F in product_tiles.FORWARD:
        assert K % 8 == 0 and K % 64 and K > 8 * 64
        assert tall(plan(BF16, PLAIN, M, F, K, dual=True))
    for M, K, F in product_tiles.DX:
        assert K % 8 == 0 and 2 * F > 8 * 64 and F % 64 and min(M * F, M * K, F * K) >= 65536  # (not as pairs)
        assert tall(plan(BF16, PLAIN, M, K, F, segs=2, turned=True))
    for M, K, F in product_tiles.DW:
        assert K % 8 == 0 and M > 8 * 64 and M % 64 and min(M * F, M * K, F * K) >= 65536
        assert tall(plan(BF16, PLAIN, F, K, M, outs=2, turned=True))


def test_parts_hold_the_contraction(plan):
    """Parts begin at a multiple of four steps where scales come four steps at a time, none is empty, and they fit the workspace."""
    for kind, sc, M, N, K, unit, size in ((F8, GROUP, 130, 96, 3001, 4, 1), (F8X, BLOCK, 300, 200, 5120, 4, 1), (F8X, ROW, 64, 64, 20000, 1, 1),
                                          (BF16, PLAIN, 129, 500, 4096, 1, 2), (F32, PLAIN, 257, 300, 3000, 1, 4)):
        p = plan(kind, sc, M, N, K, turned=kind in (BF16, F32))
        steps = -(-K * size // 128)
        assert p["splits"] > 1 and p["share"] % unit == 0
        assert (p["splits"] - 1) * p["share"] < steps <= p["splits"] * p["share"]
        assert p["bytes"] == 4 * p["splits"] * M * N


def test_pairs_take_low_tiles(plan):
    """Tiles of 128 rows, which are pairs of 64."""
    for M, K, F in product_tiles.DX:
        p = plan(BF16, PLAIN, M, K, F, segs=2, turned=True, pairs=True)
        assert p["rows"] == 128 and not p["few"]
