"""The layer's products on values at the ends of what their types hold: scales near the smallest normal one, infinities and
NaN beside ordinary values, contractions of nothing."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import products as ref
from test_gpu_products import BF, E4M3, F32, ffn_inputs, quantised
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
    a, b = (torch.empty(n, 0).to(E4M3).cuda() for n in (M, N))
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


# ---- infinities and NaN -------------------------------------------------------------------------


def sharing(x, kind):
    """For every value the largest absolute one that shares its scale (NaN above infinity above the rest)."""
    rows, cols = x.shape
    R, G = (128 if kind == "block" else 1), (cols if kind == "row" else 128)
    p = torch.nn.functional.pad(x.float().abs(), (0, -cols % G, 0, -rows % R))
    top = p.reshape(p.shape[0] // R, R, p.shape[1] // G, G).amax((1, 3))  # (amax keeps NaN)
    return top, top.repeat_interleave(R, 0).repeat_interleave(G, 1)[:rows, :cols]


def check_special(x, q, scale, kind):
    """x, as q holds it, with infinities and NaN: beside a NaN all is NaN, beside an infinity the finite values are 0, and
    what shares no scale with either is what it would be without them."""
    top, spread = sharing(x, kind)
    s = scale.cpu().reshape(top.shape)
    assert torch.equal(torch.isnan(s), torch.isnan(top)) and torch.equal(torch.isinf(s), torch.isinf(top))
    got = q.cpu().float().reshape(x.shape)
    assert torch.isnan(got[torch.isnan(spread)]).all()
    infinite = torch.isinf(spread)
    assert (got[infinite & torch.isfinite(x.float())] == 0).all() and torch.isnan(got[infinite & torch.isinf(x.float())]).all()
    whole = torch.isfinite(spread)
    calm = torch.where(whole, x.float(), torch.zeros(()))
    assert torch.equal(s[torch.isfinite(top)], ref.quant_scale(calm, kind)[torch.isfinite(top)])
    want, gap = ref.e4m3_nearest(calm.double() / ref.spread(ref.quant_scale(calm, kind), kind, *x.shape))
    off = (got.double() != want) & whole
    assert not (off & (gap > 2.0 ** -22)).any()  # (the quotient is rounded to fp32 first)


@pytest.mark.parametrize("kind,turned", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(300, 400), (131, 257), (4, 9000), (3, 40000), (9, 8)])
def test_quant_special_values(rows, cols, dt, kind, turned, gpu_lib):
    gen = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=gen)
    nan, inf = float("nan"), float("inf")
    x[-1, -1], x[0, 1], x[rows // 2, cols // 2], x[1, cols - 1] = nan, inf, -nan, -inf
    if rows > 256:
        x[256:, 256:384] = 1e-39  # below the smallest scale's 448th
        x[130:140, 130] = 3e38
    x = x.to(dt)
    q, s = gdn.gdn_quant_e4m3(x.cuda(), quant=kind, transpose=turned)
    check_special(x.t().contiguous() if turned else x, q, s, kind)


# few rows and split contractions (a quantisation behind the product), the product's own epilogue over whole and odd rows
@pytest.mark.parametrize("M,K,F", [(5, 256, 300), (70, 4100, 250), (257, 640, 129), (140, 150, 300), (300, 1040, 385)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn8_special_values(M, K, F, act, gpu_lib):
    """The e4m3 output of rows with NaN, infinities and values out of all proportion is the quantisation of the fp32 output."""
    x, xs = quantised(M, K, "group")
    wg, gs = quantised(F, K, "block", seed=1, scale=2 * K ** -0.5)
    wu, us = quantised(F, K, "block", seed=2, scale=K ** -0.5)
    x = x.float()
    x[0, K - 1] = float("nan")
    xs[1], xs[2, 0], xs[M - 1] = 1e25, float("inf"), 1e-30  # h: infinite where gates are positive, NaN, tiny
    args = [t.cuda() for t in (x.to(E4M3), xs, wg, gs, wu, us)]
    q, s = gdn.gdn_gated_ffn_e4m3(*args, activation=act, quant="group")
    h, _ = gdn.gdn_gated_ffn_e4m3(*args, activation=act, out_dtype=F32)
    h = h.cpu()
    assert torch.isnan(h[0]).all() and torch.isinf(h[1]).any() and torch.isfinite(h[3:]).all()
    check_special(h, q, s, "group")


# ---- what autograd refuses ----------------------------------------------------------------------


@pytest.mark.parametrize("op", ["linear_e4m3", "gated_ffn"])
def test_one_derivative(op, gpu_lib):
    """A second derivative, a forward-mode one and a vmap are refused, not answered wrongly."""
    def call(x, w):
        return gdn.linear_e4m3(x, w) if op == "linear_e4m3" else gdn.gated_ffn(x, w, w)

    gen = torch.Generator().manual_seed(0)
    x, w = (torch.randn(*s, generator=gen).cuda().requires_grad_() for s in ((6, 40), (24, 40)))
    dx, = torch.autograd.grad(call(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dx.sum(), w)
    with torch.autograd.forward_ad.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
        call(torch.autograd.forward_ad.make_dual(x.detach(), torch.ones_like(x)), w.detach())
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.vmap(call, in_dims=(0, None))(torch.stack([x.detach(), x.detach()]), w.detach())
