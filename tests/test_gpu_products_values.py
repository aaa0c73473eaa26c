"""The layer's products on values at the ends of what their types hold: scales near the smallest normal one, infinities and
NaN beside ordinary values, contractions of nothing."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import products as ref
from test_gpu_products import BF, F32

pytestmark = pytest.mark.gpu

KINDS = [("row", False), ("group", False), ("block", False), ("group", True), ("block", True)]


@pytest.mark.parametrize("kind,turned", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("at", [-126, -125, -120, -110, -101, -100, -60, 0])
def test_quant_ties_by_small_scales(at, dt, kind, turned, gpu_lib):
    """Values half way between two 8-bit ones go to the even one, whatever the scale: 3, 5, 7 .. 13 x 2^at, by which all
    quotients here are exact."""
    ties = torch.tensor([n * 2.0 ** e for n in (17, 19, 21, 23, 25, 27, 29, 31) for e in range(-7, 4)], dtype=torch.float64)
    for m in (3, 5, 7) if dt == BF else (3, 5, 7, 9, 11, 13, 25, 27, 49):
        scale = m * 2.0 ** at
        v = torch.cat([torch.full((1,), 448.0, dtype=torch.float64), ties, -ties[:39]])[None]
        x = (v * scale).to(dt)
        assert x.shape == (1, 128) and torch.equal(x.double(), v * scale)
        q, s = gdn.gdn_quant_e4m3((x.t().contiguous() if turned else x).cuda(), quant=kind, transpose=turned)
        assert s.cpu().double().item() == scale
        want, gap = ref.e4m3_nearest(v)
        assert (gap == 0).sum() == 127  # ties indeed
        assert torch.equal(q.cpu().double(), want), (m, (q.cpu().double() != want).sum())


@pytest.mark.parametrize("M,N", [(5, 9), (70, 300)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_matmul_of_nothing_by_rows(M, N, dt, gpu_lib):
    """A contraction of length zero is zero whatever the scales of its rows are."""
    a, b = (torch.empty(n, 0).to(torch.float8_e4m3fn).cuda() for n in (M, N))
    for bad in (float("nan"), float("inf"), 1.0):
        y = gdn.gdn_matmul_e4m3(a, torch.full((M, 1), bad).cuda(), b, torch.full((N, 1), bad).cuda(), out_dtype=dt,
                                y=torch.full((M, N), 3.0, dtype=dt).cuda())
        assert (y == 0).all()
