"""What a caller may ask for beyond the defaults: bf16 outputs of e4m3 operands with sums as in fp32 (products that cancel
beside small ones, and the fp32 outputs' values rounded once), and the gated block's bf16 gradients from gradients of gate and up
that are pairs of bf16 at any size."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import products as ref
from test_gpu_products import BF, E4M3, F32, close, ffn_inputs, quantised, rnd, scales_for
from test_gpu_products_edges import bound_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["row", "group", "block"])
@pytest.mark.parametrize("M,K", [(1, 24), (4, 128), (30, 8192), (130, 256), (300, 1040), (70, 9001), (600, 33)])
def test_matmul_cancelling(M, K, kind, gpu_lib):
    """448 x 448 - 448 x 448 + 1 + 1 ..: all that is left is what the 8-bit instruction drops."""
    a, b = torch.ones(M, K), torch.ones(40, K)
    a[:, 0], a[:, 1], b[:, 0], b[:, 1] = 448, -448, 448, 448
    kb = 1 if kind == "row" else -(-K // 128)
    sa, sb = torch.ones(M, kb), torch.ones(1 if kind == "block" else 40, kb)
    y = gdn.gdn_matmul_e4m3(a.to(E4M3).cuda(), sa.cuda(), b.to(E4M3).cuda(), sb.cuda(), exact=True)
    assert y.dtype == BF and (y.float() == torch.tensor(float(K - 2)).to(BF).float()).all()


# few rows, tiles of every way, split contractions, odd sizes
@pytest.mark.parametrize("kind", ["row", "group", "block"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 130, 300), (20, 300, 640), (40, 96, 3101), (64, 200, 1000), (130, 96, 3001), (70, 300, 4096), (257, 255, 144),
                                   (513, 260, 1152), (1500, 640, 1040), (700, 3000, 400)])
def test_matmul_is_the_fp32_output_rounded(M, N, K, kind, gpu_lib):
    a, sa = quantised(M, K, scales_for(kind), seed=M)
    b, sb = quantised(N, K, kind, seed=N)
    args = [t.cuda() for t in (a, sa, b, sb)]
    y = gdn.gdn_matmul_e4m3(*args, exact=True)
    assert torch.equal(y, gdn.gdn_matmul_e4m3(*args, out_dtype=F32).to(BF))
    value, s, bound = ref.matmul(a, sa, b, sb, kind)
    close(y, (value, bound + 32 * 2 * ref.U * s), "exact")  # (parts are added one after the other, 32 at most)
    f = gdn.gdn_matmul_e4m3(*args, out_dtype=F32, exact=True)
    assert torch.equal(f, gdn.gdn_matmul_e4m3(*args, out_dtype=F32))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,F", [(1, 16, 1), (3, 31, 130), (20, 2048, 256), (64, 1000, 128), (70, 4100, 250), (257, 640, 129), (1030, 256, 1153)])
def test_ffn8_is_the_fp32_output_rounded(M, K, F, act, gpu_lib):
    x, xs = quantised(M, K, "group")
    wg, gs = quantised(F, K, "block", seed=1, scale=2 * K ** -0.5)
    wu, us = quantised(F, K, "block", seed=2, scale=K ** -0.5)
    args = [t.cuda() for t in (x, xs, wg, gs, wu, us)]
    h, none = gdn.gdn_gated_ffn_e4m3(*args, activation=act, exact=True)
    f, _ = gdn.gdn_gated_ffn_e4m3(*args, activation=act, out_dtype=F32)
    assert none is None and h.dtype == BF and torch.equal(h, f.to(BF))
    # what is kept in 32 bits has such sums already
    q, s = gdn.gdn_gated_ffn_e4m3(*args, activation=act, quant="group", exact=True)
    q2, s2 = gdn.gdn_gated_ffn_e4m3(*args, activation=act, quant="group")
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("M,N,K", [(20, 40, 136), (130, 140, 260), (300, 264, 520)])
def test_linear_cancelling(M, N, K, gpu_lib):
    """The same along each of the three products' contractions, with values that quantise exactly."""
    def edge(n):
        e = torch.ones(n, dtype=torch.float64)
        e[::128], e[1::128] = 448, -448
        return e

    x = edge(M)[:, None] * edge(K)
    d = edge(M).abs()[:, None] * edge(N)
    w = torch.ones(N, K, dtype=torch.float64)
    for first in (0, 1):
        w[first::128], w[:, first::128] = 448, 448
    leaves = x.to(BF).cuda().requires_grad_(), w.to(BF).cuda().requires_grad_()
    y = gdn.linear_e4m3(*leaves, exact=True)
    dx, dw = torch.autograd.grad(y, leaves, d.to(BF).cuda())
    for got, want, what in ((y, x @ w.t(), "y"), (dx, d @ w, "dx"), (dw, d.t() @ x, "dw")):
        assert torch.equal(got.cpu(), want.to(BF)), what


def test_exact_in_a_graph(gpu_lib):
    """A captured step with exact sums, replayed with other inputs and eager work between."""
    M, K, F = 70, 256, 320
    x = rnd(M, K, dtype=BF).cuda()
    wg, wu = (gdn.gdn_quant_e4m3(rnd(F, K, seed=i, scale=K ** -0.5).cuda(), quant="block") for i in (1, 2))

    def step():
        q, s = gdn.gdn_quant_e4m3(x, quant="group")
        return gdn.gdn_matmul_e4m3(q, s, *wg, exact=True), gdn.gdn_gated_ffn_e4m3(q, s, *wg, *wu, exact=True)[0]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        outs = step()
    for k in range(3):
        x.copy_(rnd(M, K, seed=50 + k, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, step())), k
        torch.cuda.synchronize()


# all matrices of 65,536 values and more: rounded once, unless asked for
@pytest.mark.parametrize("M,K,F", [(300, 264, 520), (1000, 300, 257), (513, 1025, 130), (4101, 600, 331)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_pairs_asked_for(M, K, F, act, gpu_lib):
    assert min(M * K, M * F, K * F) >= 65536
    x, wg, wu, d = ffn_inputs(M, K, F, BF, seed=M)
    leaves = [t.cuda().requires_grad_() for t in (x, wg, wu)]
    want = ref.ffn_bwd(x, wg, wu, d, act, F32)
    terms = bound_of(x, wg, wu, d, act)
    for recompute in (False, True):
        grads = torch.autograd.grad(gdn.gated_ffn(*leaves, activation=act, recompute=recompute, pairs=True), leaves, d.cuda())
        for got, (k, (v, e)) in zip(grads, want.items()):
            got = got.cpu().double()
            own = (v.to(BF).double() - v).norm()
            assert ((got - v).abs() <= 2.0 ** -8 * v.abs() + 1.01 * e + 2.0 ** -15 * terms[k]).all(), k
            # its own rounding alone; rounded once it is 1.35 to 1.44 of that
            assert (got - v).norm() <= 1.12 * own + 2.0 ** -15 * v.norm(), k
    # (in fp32 there is nothing to ask for)
    dev = [t.detach().float() for t in leaves]
    a, b = (gdn.gdn_gated_ffn_bwd(*dev, d.cuda().float(), activation=act, pairs=p) for p in (False, True))
    assert all(torch.equal(a[k], b[k]) for k in a)
