"""Products by tiles of 256 rows against the 64-bit forms: many steps of the contraction with every kind of scales, both
sides of the block, turned operands, remainders everywhere. Errors in the 2-norm beside the result's own rounding: what
else is in them are sums in 32 bits, the 8-bit instruction's cut (2^-13, as everywhere) and, in the block's gradients,
one more rounding of as many values (sqrt 2 in all; 1.35 to 1.44 at such sizes)."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
import product_tiles
from oracle import products as ref
from test_gpu_products import BF, close, ffn_inputs, quantised, scales_for

pytestmark = pytest.mark.gpu


def beside_rounding(got, value, factor, rel, what):
    value = value.reshape(got.shape)
    own = (value.to(BF).double() - value).norm()
    err = (got.cpu().double() - value).norm()
    assert err <= factor * own + rel * value.norm(), f"{what}: {(err / own).item():.3f} of its own rounding"


def framed(rows, cols):
    """An output with rows around it that nothing may write."""
    buf = torch.full((rows + 2, cols), 9.0, dtype=BF).cuda()
    return buf, buf[1:-1]


def untouched(*bufs):
    return all(bool((b[0] == 9).all() and (b[-1] == 9).all()) for b in bufs)


@pytest.mark.parametrize("kind", ["block", "group", "row"])
@pytest.mark.parametrize("M,N,K", product_tiles.MATMUL)
def test_matmul(M, N, K, kind, gpu_lib):
    a, sa = quantised(M, K, scales_for(kind), seed=1)
    b, sb = quantised(N, K, kind, seed=2, scale=K ** -0.5)
    value, s, bound = ref.matmul(a, sa, b, sb, kind)
    buf, y = framed(M, N)
    args = [t.cuda() for t in (a, sa, b, sb)]
    gdn.gdn_matmul_e4m3(*args, y=y)
    close(y, (value, bound + ref.CUT * s), kind)
    beside_rounding(y, value, 1.01, 2.0 ** -13, kind)
    assert untouched(buf) and torch.equal(y, gdn.gdn_matmul_e4m3(*args))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,F", product_tiles.FFN8)
def test_ffn8(M, K, F, act, gpu_lib):
    x, xs = quantised(M, K, "group")
    wg, gs = quantised(F, K, "block", seed=1, scale=2 * K ** -0.5)
    wu, us = quantised(F, K, "block", seed=2, scale=K ** -0.5)
    v = [ref.values(x, xs, "group"), ref.values(wg, gs, "block"), ref.values(wu, us, "block")]
    buf, h = framed(M, F)
    gdn.gdn_gated_ffn_e4m3(*[t.cuda() for t in (x, xs, wg, gs, wu, us)], activation=act, h=h)
    want = ref.ffn_fwd(*v, act, cut=ref.CUT)[0]
    close(h, want, "h")
    beside_rounding(h, want[0], 1.01, 2.0 ** -12, "h")
    assert untouched(buf)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,F", product_tiles.FORWARD + product_tiles.DX + product_tiles.DW)
def test_ffn(M, K, F, act, gpu_lib):
    x, wg, wu, d = ffn_inputs(M, K, F, BF, seed=3)
    dev = [t.cuda() for t in (x, wg, wu)]
    pre = gdn.gdn_gated_ffn_pre(dev[0], dev[1])
    want, a, u = ref.ffn_fwd(x, wg, wu, act)
    buf, h = framed(M, F)
    gdn.gdn_gated_ffn_fwd(*dev, activation=act, h=h, pre=pre)
    close(h, want, "h")
    close(pre[0], a, "gate")
    close(pre[1], u, "up")
    beside_rounding(h, want[0], 1.01, 2.0 ** -15, "h")
    bufs = {k: framed(*t.shape) for k, t in (("dx", x), ("dw_gate", wg), ("dw_up", wu))}
    for kept in (pre, None):
        gdn.gdn_gated_ffn_bwd(*dev, d.cuda(), activation=act, pre=kept, out={k: t for k, (_, t) in bufs.items()})
        grads = ref.ffn_bwd(x, wg, wu, d, act, BF, None if kept is None else pre.cpu())
        for k, (value, bound) in grads.items():
            close(bufs[k][1], (value, bound), k)
            beside_rounding(bufs[k][1], value, 1.5, 2.0 ** -15, k)
    assert untouched(buf, *(b for b, _ in bufs.values()))
