"""The layer's products where their ways of working meet: split contractions at odd and even addresses, tiles that end
inside each other, outputs that pass 32-bit offsets, operands and outputs inside larger buffers at odd addresses."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import products as ref
from test_gpu_products import BF, E4M3, F32, check_quant, close, ffn_inputs, near, quantised, rnd, scales_for

pytestmark = pytest.mark.gpu


# few tiles and long contractions: the contraction is split, with scales four steps at a time and without; memory rows that
# are whole chunks, and ones that are not
@pytest.mark.parametrize("M,N,K", [(130, 96, 3001), (70, 300, 4096), (257, 130, 2050), (65, 1, 1300), (100, 129, 1664), (300, 200, 5120)])
@pytest.mark.parametrize("kind", ["row", "group", "block"])
def test_matmul_split(M, N, K, kind, gpu_lib):
    a, sa = quantised(M, K, scales_for(kind), seed=3)
    b, sb = quantised(N, K, kind, seed=4, scale=K ** -0.5)
    y, s, bound = ref.matmul(a, sa, b, sb, kind)
    # the parts' sums are added one after the other: 32 of them at most
    bound = bound + 32 * 2 * ref.U * s
    args = [t.cuda() for t in (a, sa, b, sb)]
    got = gdn.gdn_matmul_e4m3(*args, out_dtype=F32)
    close(got, (y, bound), "fp32")
    assert torch.equal(got, gdn.gdn_matmul_e4m3(*args, out_dtype=F32))
    got = gdn.gdn_matmul_e4m3(*args)
    close(got, (y, bound + ref.CUT * s), "bf16")
    near(got, y, 2.0 ** -9 + 2.0 ** -13, "bf16")


# tiles of 128 rows and 256 columns met and passed by one, one step of the contraction and a bit, several tiles a side (tiles of
# 256 rows: test_gpu_products_tiles.py)
@pytest.mark.parametrize("M,N,K", [(255, 257, 128), (256, 256, 256), (257, 255, 144), (511, 513, 400), (1025, 129, 16), (129, 1025, 1008), (640, 2304, 512)])
def test_matmul_tiles(M, N, K, gpu_lib):
    for kind in ("block", "group", "row"):
        a, sa = quantised(M, K, scales_for(kind), seed=M)
        b, sb = quantised(N, K, kind, seed=N)
        y, s, bound = ref.matmul(a, sa, b, sb, kind)
        out = torch.full((M + 2, N), 9.0, dtype=BF).cuda()
        gdn.gdn_matmul_e4m3(*[t.cuda() for t in (a, sa, b, sb)], y=out[1:-1])
        close(out[1:-1], (y, bound + ref.CUT * s), kind)
        assert (out[0] == 9).all() and (out[-1] == 9).all(), "rows around the output were written"
        close(gdn.gdn_matmul_e4m3(*[t.cuda() for t in (a, sa, b, sb)], out_dtype=F32), (y, bound), kind + " fp32")


@pytest.mark.parametrize("M,K,F", [(70, 4096, 256), (70, 4100, 250), (257, 640, 129), (300, 1040, 385), (1030, 256, 1153)])
def test_ffn8_quantised_tiles(M, K, F, gpu_lib):
    """The e4m3 output is the quantisation of the fp32 one, whichever way it is made."""
    x, xs = quantised(M, K, "group")
    wg, gs = quantised(F, K, "block", seed=1, scale=2 * K ** -0.5)
    wu, us = quantised(F, K, "block", seed=2, scale=K ** -0.5)
    args = [t.cuda() for t in (x, xs, wg, gs, wu, us)]
    q, s = gdn.gdn_gated_ffn_e4m3(*args, quant="group")
    h, _ = gdn.gdn_gated_ffn_e4m3(*args, out_dtype=F32)
    check_quant(h.cpu(), q, s, "group", "of the fp32 output")
    v = [ref.values(x, xs, "group"), ref.values(wg, gs, "block"), ref.values(wu, us, "block")]
    close(h, ref.ffn_fwd(*v, "silu")[0], "fp32")


@pytest.mark.parametrize("M,K,F,dt", [(70, 2048, 136, BF), (3000, 40, 50, BF), (1500, 37, 61, BF), (1500, 37, 61, F32), (256, 264, 512, BF), (257, 520, 264, BF),
                                      (129, 128, 900, F32), (16, 256, 1024, BF), (1, 48, 2000, F32)])
def test_ffn_shapes(M, K, F, dt, gpu_lib):
    """Split and whole contractions in each of the gradients' products."""
    x, wg, wu, d = ffn_inputs(M, K, F, dt, seed=11)
    dev = [t.cuda() for t in (x, wg, wu)]
    pre = gdn.gdn_gated_ffn_pre(dev[0], dev[1])
    h, a, u = ref.ffn_fwd(x, wg, wu, "silu")
    close(gdn.gdn_gated_ffn_fwd(*dev, pre=pre), h, "h")
    close(pre[0], a, "gate")
    close(pre[1], u, "up")
    for kept in (pre, None):
        want = ref.ffn_bwd(x, wg, wu, d, "silu", dt, None if kept is None else pre.cpu())
        gr = gdn.gdn_gated_ffn_bwd(*dev, d.cuda(), pre=kept)
        for k in want:
            close(gr[k], want[k], k)
            near(gr[k], want[k][0], 4 * ref.HALF[dt] + 2.0 ** -18, k)


def inside(t, front, fill=7.0):
    """The same values in the middle of a larger buffer, `front` elements behind its start."""
    buf = torch.full((t.numel() + front + 11,), fill).to(t.dtype).cuda()
    view = buf[front:front + t.numel()].view(t.shape)
    view.copy_(t)
    return buf, view


@pytest.mark.parametrize("M,K,F", [(5, 64, 48), (70, 64, 128), (200, 33, 77), (300, 128, 264)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_ffn_at_odd_addresses(M, K, F, dt, gpu_lib):
    """Operands and outputs one element behind a vector's start: the same bits as at even addresses' other kernels within
    the bounds, and nothing around the outputs is written."""
    x, wg, wu, d = ffn_inputs(M, K, F, dt, seed=2)
    (_, xo), (_, go), (_, uo), (_, do) = (inside(t, 1) for t in (x, wg, wu, d))
    want, _, _ = ref.ffn_fwd(x, wg, wu, "gelu_tanh")
    hb, h = inside(torch.zeros(M, F, dtype=dt), 3)
    pb, pre = inside(torch.zeros(2, M, F), 1)
    gdn.gdn_gated_ffn_fwd(xo, go, uo, activation="gelu_tanh", h=h, pre=pre)
    close(h, want, "h")
    bufs = {k: inside(torch.zeros_like(t), 3) for k, t in (("dx", x), ("dw_gate", wg), ("dw_up", wu))}
    for kept in (pre, None):
        gdn.gdn_gated_ffn_bwd(xo, go, uo, do, activation="gelu_tanh", pre=kept, out={k: v for k, (_, v) in bufs.items()})
        grads = ref.ffn_bwd(x, wg, wu, d, "gelu_tanh", dt, None if kept is None else pre.cpu())
        for k, (_, v) in bufs.items():
            close(v, grads[k], k)
    for buf, t, front in [(hb, h, 3), (pb, pre, 1)] + [(b, v, 3) for b, v in bufs.values()]:
        assert (buf[:front] == 7).all() and (buf[front + t.numel():] == 7).all()


def test_ffn8_at_odd_addresses(gpu_lib):
    for M, K, F in ((5, 128, 130), (140, 256, 384)):
        x, xs = quantised(M, K, "group")
        wg, gs = quantised(F, K, "block", seed=1)
        wu, us = quantised(F, K, "block", seed=2)
        want = gdn.gdn_gated_ffn_e4m3(*[t.cuda() for t in (x, xs, wg, gs, wu, us)], quant="group")
        odd = [inside(t, 1)[1] for t in (x, xs, wg, gs, wu, us)]
        qb, q = inside(torch.zeros(M, F).to(E4M3), 5)
        sb, s = inside(torch.zeros(M, -(-F // 128)), 1)
        gdn.gdn_gated_ffn_e4m3(*odd, quant="group", h=q, scale=s)
        # the same products in another order: scales within its bound, values within a step
        assert torch.allclose(s, want[1], rtol=2.0 ** -10)
        assert (qb[:5].float() == 7).all() and (qb[5 + M * F:].float() == 7).all() and sb[0] == 7 and (sb[1 + s.numel():] == 7).all()
        near(q.float().cpu() * ref.spread(s, "group", M, F).float(), want[0].cpu().double() * ref.spread(want[1], "group", M, F), 2.0 ** -6, "h")


def test_workspaces_of_the_caller(gpu_lib):
    a, sa, b, sb = (t.cuda() for p in (quantised(200, 4096, "group"), quantised(160, 4096, "block", seed=1)) for t in p)
    want = gdn.gdn_matmul_e4m3(a, sa, b, sb)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    assert torch.equal(gdn.gdn_matmul_e4m3(a, sa, b, sb, workspace=ws), want)
    with pytest.raises(ValueError):
        gdn.gdn_matmul_e4m3(a, sa, b, sb, workspace=ws[:256])
    with pytest.raises(ValueError):
        gdn.gdn_matmul_e4m3(a, sa, b, sb, workspace=ws[8:])
    x, wg, wu, d = (t.cuda() for t in ffn_inputs(90, 64, 72, BF))
    full = gdn.gdn_gated_ffn_bwd(x, wg, wu, d)
    mine = gdn.gdn_gated_ffn_bwd(x, wg, wu, d, workspace=ws)
    assert all(torch.equal(full[k], mine[k]) for k in full)


def test_beyond_32_bits(gpu_lib):
    """Outputs of more than 2^31 elements: their last rows equal those of a call on these rows alone."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    M, N, K = 70016, 33024, 128
    a = torch.randn(M, K, device="cuda", generator=gen)
    qa, sa = gdn.gdn_quant_e4m3(a)
    qb, sb = gdn.gdn_quant_e4m3(torch.randn(N, K, device="cuda", generator=gen), quant="block")
    y = gdn.gdn_matmul_e4m3(qa, sa, qb, sb)
    for at in (0, 65000, M - 512):
        assert torch.equal(y[at:at + 512], gdn.gdn_matmul_e4m3(qa[at:at + 512].contiguous(), sa[at:at + 512].contiguous(), qb, sb))
    # quantisation of such a matrix, row by row and turned
    q, s = gdn.gdn_quant_e4m3(y)
    tail, ts = gdn.gdn_quant_e4m3(y[-256:].contiguous())
    assert torch.equal(q[-256:].view(torch.uint8), tail.view(torch.uint8)) and torch.equal(s[-256:], ts)
    del q, s
    q, s = gdn.gdn_quant_e4m3(y, transpose=True)
    tail, ts = gdn.gdn_quant_e4m3(y[-256:, -300:].contiguous(), transpose=True)
    assert torch.equal(q[-300:, -256:].contiguous().view(torch.uint8), tail.view(torch.uint8)) and torch.equal(s[-300:, -2:].contiguous(), ts)


def test_ffn_beyond_32_bits(gpu_lib):
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, K, F = 40064, 64, 28032  # gate and up: 2.2e9 fp32 values
    x = torch.randn(M, K, device="cuda", generator=gen).to(BF)
    wg, wu = (torch.randn(F, K, device="cuda", generator=gen).mul(K ** -0.5).to(BF) for _ in range(2))
    pre = gdn.gdn_gated_ffn_pre(x, wg)
    h = gdn.gdn_gated_ffn_fwd(x, wg, wu, pre=pre)
    few = slice(M - 512, M)
    p2 = gdn.gdn_gated_ffn_pre(x[few], wg)
    assert torch.equal(h[few], gdn.gdn_gated_ffn_fwd(x[few], wg, wu, pre=p2)) and torch.equal(pre[:, few], p2)
    dx = gdn.gdn_gated_ffn_bwd(x, wg, wu, h, pre=pre, need_dweight=False)["dx"]
    # (other rows may be split otherwise: within the order of the additions)
    other = gdn.gdn_gated_ffn_bwd(x[few], wg, wu, h[few], pre=p2, need_dweight=False)["dx"]
    assert ((dx[few].float() - other.float()).norm() <= 2.0 ** -7 * other.float().norm()).item()


def test_linear_does_what_is_asked(gpu_lib, monkeypatch):
    """Nothing is prepared or computed for gradients that nobody can ask for."""
    from gated_deltanet_chunked_04_amd import products

    x, w = rnd(3, 70, 200, dtype=BF).cuda().requires_grad_(), rnd(130, 200, seed=1).cuda().requires_grad_()
    kinds = []
    quant = products.gdn_quant_e4m3

    def counted(t, **kw):
        kinds.append((kw["quant"], kw.get("transpose", False)))
        return quant(t, **kw)

    monkeypatch.setattr(products, "gdn_quant_e4m3", counted)
    for mode in (torch.no_grad, torch.inference_mode):
        kinds.clear()
        with mode():
            y = gdn.linear_e4m3(x, w)
        assert kinds == [("group", False), ("block", False)] and not y.requires_grad
    kinds.clear()
    z = gdn.linear_e4m3(x, w)
    assert torch.equal(z, y) and kinds == [("group", False), ("block", False), ("group", True)]
    assert gdn.linear_e4m3(x.detach(), w.detach()).requires_grad is False and kinds[3:] == kinds[:2]
    kinds.clear()
    torch.autograd.grad(gdn.linear_e4m3(x, w.detach()).float().sum(), x)
    assert kinds == [("group", False), ("block", False), ("group", False), ("block", True)]
    kinds.clear()
    dw = torch.autograd.grad(gdn.linear_e4m3(x.detach(), w).float().sum(), w)[0]
    assert kinds == [("group", False), ("block", False), ("group", True), ("group", True)] and dw.dtype == F32


def test_ffn_some_gradients(gpu_lib):
    """gated_ffn's gradients one at a time are those asked for together."""
    x, wg, wu, d = (t.cuda() for t in ffn_inputs(70, 96, 136, BF, seed=5))
    leaves = [t.requires_grad_() for t in (x, wg, wu)]
    for recompute in (False, True):
        h = gdn.gated_ffn(*leaves, recompute=recompute)
        all_of = torch.autograd.grad(h, leaves, d, retain_graph=True)
        for i, leaf in enumerate(leaves):
            assert torch.equal(torch.autograd.grad(h, leaf, d, retain_graph=True)[0], all_of[i])
    with torch.no_grad():
        assert torch.equal(gdn.gated_ffn(*leaves), h)


# rows on both sides of what a workgroup's registers hold, its last vector whole and not
@pytest.mark.parametrize("cols", [2047, 2048, 2049, 4096, 4101, 8192, 8193, 20000, 32768, 32769, 70003])
@pytest.mark.parametrize("dt", [BF, F32])
def test_quant_long_rows(cols, dt, gpu_lib):
    x = rnd(5, cols, seed=cols, dtype=dt)
    x[1, -1], x[2, 0], x[3] = 50.0, -60.0, 0.0
    q, s = gdn.gdn_quant_e4m3(x.cuda(), quant="row")
    check_quant(x, q, s, "row", "row")


# bf16 gradients where they are few: all that rounds them to 8 bits is their own rounding, half a step a value at most (the
# gradients of gate and up are kept to 16 bits).
@pytest.mark.parametrize("M,K,F", [(1, 16, 16), (1, 1, 1), (16, 16, 2048), (16, 2048, 16), (3000, 16, 16), (1, 1024, 512), (129, 100, 70), (70, 1000, 333), (4096, 15, 64)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_few_gradients(M, K, F, act, gpu_lib):
    x, wg, wu, d = ffn_inputs(M, K, F, BF, seed=M + K)
    dev = [t.cuda() for t in (x, wg, wu)]
    pre = gdn.gdn_gated_ffn_pre(dev[0], dev[1])
    gdn.gdn_gated_ffn_fwd(*dev, pre=pre, activation=act)
    want = ref.ffn_bwd(x, wg, wu, d, act, F32)
    for kept in (pre, None):
        gr = gdn.gdn_gated_ffn_bwd(*dev, d.cuda(), pre=kept, activation=act)
        for k, (v, e) in want.items():
            err = (gr[k].cpu().double() - v).abs()
            # half a step of bf16 each; of the products' terms 2^-16 for the pairs beside fp32's own bound
            assert (err <= 2.0 ** -8 * v.abs() + 1.01 * e + 2.0 ** -15 * bound_of(x, wg, wu, d, act)[k]).all(), k


def bound_of(x, wg, wu, d, act):
    """Sums of the absolute terms of the gradients."""
    from oracle import products as ref

    x, wg, wu, d = (t.double() for t in (x, wg, wu, d))
    a, u = x @ wg.t(), x @ wu.t()
    f, df = ref._act(a, act)[:2]
    da, du = (d * u * df).abs(), (d * f).abs()
    return dict(dx=da @ wg.abs() + du @ wu.abs(), dw_gate=da.t() @ x.abs(), dw_up=du.t() @ x.abs())


def test_ffn_pairs_infinite(gpu_lib):
    """A gradient that bf16 has no value for is infinite, not NaN, and stays in its row of dx and its rows of the weights'."""
    x, wg, wu, d = (t.cuda() for t in ffn_inputs(20, 16, 24, BF, seed=7))
    d[3, 5] = 3.3e38
    u = (x.float() @ wu.float().t())[3, 5]
    x[3] *= (4 / u.abs()).to(BF)  # d_up up = 1.3e39
    gr = gdn.gdn_gated_ffn_bwd(x, wg, wu, d)
    rows = torch.arange(20, device="cuda") != 3
    assert torch.isfinite(gr["dx"][rows]).all() and not torch.isfinite(gr["dx"][3]).all()
    cols = torch.arange(24, device="cuda") != 5
    assert torch.isfinite(gr["dw_gate"][cols]).all() and torch.isfinite(gr["dw_up"][cols]).all()
    assert torch.isinf(gr["dw_gate"][5]).any() and not torch.isnan(gr["dw_gate"][5]).any()


# on both sides of what counts as few rows, over short rows and long ones
@pytest.mark.parametrize("M", [32, 33, 48, 49, 64, 65])
@pytest.mark.parametrize("K", [300, 3056, 3088, 3101])
def test_few_rows_or_tiles(M, K, gpu_lib):
    N = 200
    a, sa = quantised(M, K, scales_for("block"), seed=M)
    b, sb = quantised(N, K, "block", seed=K, scale=K ** -0.5)
    y, s, bound = ref.matmul(a, sa, b, sb, "block")
    bound = bound + 32 * 2 * ref.U * s
    close(gdn.gdn_matmul_e4m3(*[t.cuda() for t in (a, sa, b, sb)], out_dtype=F32), (y, bound), "fp32")
    x, wg, wu, _ = ffn_inputs(M, K // 2 // 8 * 8, 136, BF, seed=M)
    h = ref.ffn_fwd(x, wg, wu, "silu")[0]
    got = gdn.gdn_gated_ffn_fwd(x.cuda(), wg.cuda(), wu.cuda())
    close(got, h, "h")
