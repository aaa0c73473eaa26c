"""The layer's products on values at the ends of what their types hold: scales near the smallest normal one, infinities and
NaN beside ordinary values, contractions of nothing."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import products as ref
from test_gpu_products import BF, F32, ffn_inputs
from test_gpu_products_edges import bound_of

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


# few rows over large weights, few columns under many rows, several tiles of each operand; rows that are whole chunks and not
@pytest.mark.parametrize("M,K,F", [(7, 8192, 1032), (1, 4104, 2056), (520, 120, 264), (65, 960, 136), (200, 72, 130), (9001, 264, 7), (130, 101, 99), (63, 1000, 1000)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_pairs_in_tiles(M, K, F, act, gpu_lib):
    """Gradients of gate and up kept as pairs of bf16: dx and the weights' gradients are off by their own rounding and 2^-15
    of the products' terms, in every tile."""
    x, wg, wu, d = ffn_inputs(M, K, F, BF, seed=M + K)
    dev = [t.cuda() for t in (x, wg, wu)]
    want = ref.ffn_bwd(x, wg, wu, d, act, F32)
    terms = bound_of(x, wg, wu, d, act)
    out = {k: torch.full((len(t) + 2, t.shape[1]), 9.0, dtype=BF).cuda() for k, t in (("dx", x), ("dw_gate", wg), ("dw_up", wu))}
    for kept in (True, False):
        pre = gdn.gdn_gated_ffn_pre(dev[0], dev[1]) if kept else None
        if kept:
            gdn.gdn_gated_ffn_fwd(*dev, pre=pre, activation=act)
        gdn.gdn_gated_ffn_bwd(*dev, d.cuda(), pre=pre, activation=act, out={k: t[1:-1] for k, t in out.items()})
        for k, (v, e) in want.items():
            got = out[k][1:-1].cpu().double()
            assert ((got - v).abs() <= 2.0 ** -8 * v.abs() + 1.01 * e + 2.0 ** -15 * terms[k]).all(), (k, kept)
            # in the 2-norm: its own rounding is 2^-9.2 of it, and a lost half of the pairs would make that 2^-8.7
            assert (got - v).norm() <= 1.12 * (v.to(BF).double() - v).norm() + 2.0 ** -15 * v.norm(), (k, kept)
            assert (out[k][0] == 9).all() and (out[k][-1] == 9).all(), "rows around the output were written"
