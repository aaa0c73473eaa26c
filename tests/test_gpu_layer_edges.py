"""Edges of the layer operators on the GPU: 8-bit values that lie on a tie, gates that grow, packed batches with rows
of no sequence, and the shapes and chains behind them, against the plain 64-bit forms."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
import test_gpu_layer as base
from oracle import layer as ref
from test_gpu_layer import close, cu_dev, cuda, owned, packed, rnd, scan_inputs

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ---- RMS norm -----------------------------------------------------------------------------------


@pytest.mark.parametrize("rows,D", [(40, 5), (200, 64), (200, 300), (200, 512), (60, 2047), (30, 9000), (10, 20000), (6, 33001)])
def test_8_bit_values_are_the_nearest_quotients(rows, D, gpu_lib):
    """y / scale to nearest even, formed from the fp32 y: a call in the input's type gives that y, and the quotients of
    small whole numbers lie on 8-bit ties often."""
    gen = torch.Generator().manual_seed(D)
    x = torch.randint(-120, 121, (rows, D), generator=gen).float()
    x[::2] = torch.randn(len(x[::2]), D, generator=gen)
    w = torch.randint(1, 9, (D,), generator=gen).float() / 8
    y = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda())[0].cpu()
    for quant, G in (("row", D), ("group", 128)):
        q, _, scale = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda(), quant=quant)
        want = (y / scale.cpu().repeat_interleave(G, 1)[:, :D]).clamp(-448, 448).to(torch.float8_e4m3fn)
        bad = q.cpu().view(torch.uint8) != want.view(torch.uint8)
        # (a zero may carry either sign)
        bad &= (q.cpu().float() != 0) | (want.float() != 0)
        assert not bad.any(), (quant, int(bad.sum()), bad.numel())


def test_8_bit_values_beside_an_infinity(gpu_lib):
    """Where y overflows to infinity its scale is infinite, the values beside it 0 / inf = 0, itself NaN."""
    for D in (5, 64, 300, 40000):
        x, w = torch.ones(2, D).cuda(), torch.ones(D).cuda()
        w[3] = float("inf")
        for quant in ("row", "group"):
            q, _, scale = gdn.gdn_rmsnorm_fwd(x, w, quant=quant)
            q = q.float().cpu()
            assert torch.isinf(scale[:, 0]).all() and torch.isnan(q[:, 3]).all()
            assert (q[:, :3] == 0).all() and (q[:, 4] == 0).all()


# ---- gated scan: gates whose product over many tiles leaves fp32's range ------------------------


def check_scan(x, g, s0, cu=None, d_h=None, d_fin=None):
    """Forward and gradient (states kept and recomputed) against the 64-bit form."""
    B, T, D = x.shape
    cd, keep = cu_dev(cu), owned(B, T, cu)
    rows = lambda got, want, what: close(got[keep.cuda()], (want[0][keep], want[1][keep]), what)  # noqa: E731
    want_h, want_fin = ref.scan_fwd(x, g, s0, cu)
    states = gdn.gdn_gated_scan_states(x.cuda())
    h, fin = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), cuda(s0), cu_seqlens=cd, states=states)
    rows(h, want_h, "h")
    close(fin, want_fin, "final_state")
    d_h = torch.zeros_like(x) if d_h is None else d_h
    want = ref.scan_bwd(x, g, s0, d_h, d_fin, cu)
    for st in (states, None):
        gr = gdn.gdn_gated_scan_bwd(x.cuda(), g.cuda(), d_h.cuda(), cuda(s0), cuda(d_fin), cu_seqlens=cd, states=st)
        for k in ("dx", "dg"):
            rows(gr[k], want[k], k)
        close(gr["d_initial_state"], want["d_initial_state"], "d_initial_state")


def steps(T, D, *parts):
    """g [1, T, D], zero but for the parts (first token, one behind the last, gate)."""
    g = torch.zeros(1, T, D)
    for a, b, v in parts:
        g[:, a:b] = v
    return g


@pytest.mark.parametrize("D", [64, 130, 256, 2048])
def test_scan_growth_over_many_tiles(D, gpu_lib):
    """A tiny state grows by e^102 over 512 tokens, 128 of which grow by 1.3e11 at most."""
    T = 2048
    tiny = torch.full((1, D), 1e-36)
    check_scan(torch.zeros(1, T, D), steps(T, D, (512, 1024, 0.2)), tiny, d_fin=tiny)
    check_scan(torch.zeros(1, T, D), steps(T, D, (1024, 1536, 0.2)), tiny, d_fin=tiny)


@pytest.mark.parametrize("D", [64, 131, 256, 2048])
def test_scan_growth_then_decay_and_forgetting(D, gpu_lib):
    """Growth to 3e34 from a state and inputs, then decay, and a gate of -inf in half of the channels."""
    T = 4096
    g = steps(T, D, (1024, 2048, 0.1), (2048, 4096, -0.05))
    g[0, 3000, ::2] = float("-inf")
    x = rnd(1, T, D, scale=1e-12)
    x[:, 1500:] = 0
    x[:, 3000:] = rnd(1, T - 3000, D, seed=1)
    check_scan(x, g, torch.full((1, D), 1e-10), d_h=rnd(1, T, D, seed=2, scale=1e-12), d_fin=rnd(1, D, seed=3, scale=1e-10))


@pytest.mark.parametrize("D", [64, 131, 256, 2048])
def test_scan_decay_and_growth_that_undo_each_other(D, gpu_lib):
    """The product falls to e^-102 (or rises to e^102) over 1,024 tokens and comes back to 1."""
    T = 2048
    up, down = torch.full((1, D), 1e30), torch.full((1, D), 1e-30)
    check_scan(torch.zeros(1, T, D), steps(T, D, (0, 1024, -0.1), (1024, 2048, 0.1)), up, d_fin=down)
    check_scan(torch.zeros(1, T, D), steps(T, D, (0, 1024, 0.1), (1024, 2048, -0.1)), down, d_fin=up)


@pytest.mark.parametrize("D", [64, 256, 2048])
def test_scan_growth_behind_a_cancelled_state(D, gpu_lib):
    """An input cancels the state, and what it would have left from a zero state grows beyond the range (e^99 over 330
    tokens, which every part of the chain that holds them sees; 128 of them grow by e^38)."""
    T = 3000
    x, s0 = torch.zeros(1, T, D), torch.full((1, D), -1.0)
    for at in (0, 300, 1100):
        x.zero_()
        x[0, at] = 1.0
        check_scan(x, steps(T, D, (at + 1, at + 331, 0.3)), s0)
    d_h = torch.zeros(1, T, D)
    for at in (T - 1, 2500, 1700):
        d_h.zero_()
        d_h[0, at] = 1.0
        check_scan(torch.zeros(1, T, D), steps(T, D, (at - 330, at, 0.3)), None, d_h=d_h, d_fin=s0)


def test_scan_infinite_state_stays_infinite(gpu_lib):
    """Behind decay over many tiles (each product in range) an infinite state is infinite, not NaN."""
    T, D = 2048, 256
    s0 = torch.full((1, D), float("inf"))
    g = torch.full((1, T, D), -0.1)
    h, fin = gdn.gdn_gated_scan_fwd(torch.zeros(1, T, D).cuda(), g.cuda(), s0.cuda())
    assert torch.isposinf(h).all() and torch.isposinf(fin).all()
    gr = gdn.gdn_gated_scan_bwd(torch.zeros(1, T, D).cuda(), g.cuda(), torch.zeros(1, T, D).cuda(), torch.ones(1, D).cuda(), s0.cuda())
    assert torch.isposinf(gr["dx"]).all() and torch.isposinf(gr["d_initial_state"]).all()


# ---- packed batches with tokens of no sequence --------------------------------------------------


def litter():
    """Memory that the allocator hands out next holds NaN."""
    junk = [torch.full((1 << k,), float("nan"), device="cuda") for k in range(10, 21) for _ in range(4)]
    del junk


# the batch is padded behind (and in front): in one tile, several, as decoding takes it, and with nothing but padding
PADDED = [([5, 0, 30], 0, 29, 64), ([5, 0, 30], 3, 9, 131), ([300, 2, 400], 0, 322, 256), ([300, 2, 400], 70, 200, 130),
          ([1] * 40, 0, 24, 64), ([1] * 30 + [0] * 60, 2, 40, 130), ([0] * 700 + [50, 0], 9, 450, 256), ([0, 0], 0, 300, 64), ([0], 4, 0, 8)]


@pytest.mark.parametrize("lens,head,tail,D", PADDED)
@pytest.mark.parametrize("dt", [BF, F32])
def test_padding_gets_zeros(lens, head, tail, D, dt, gpu_lib):
    """Outputs and gradients that the package allocates hold zeros in rows of no sequence, whatever the inputs hold
    there; the other rows are what they are without the padding's values."""
    cu, T = packed(lens, head, tail)
    x, g, s0, N = scan_inputs(1, T, D, cu, dt, F32, True)
    keep, cd = owned(1, T, cu), cu_dev(cu)
    w, c0 = rnd(D, 4, seed=3).cuda(), rnd(N, 3, D, seed=4, dtype=dt).cuda()
    d = rnd(1, T, D, seed=5, dtype=dt)
    want = ref.scan_fwd(x, g, s0, cu)[0], ref.conv_fwd(x, w.cpu(), None, c0.cpu(), True, cu)[0]
    wantg = ref.scan_bwd(x, g, s0, d, None, cu), ref.conv_bwd(x, w.cpu(), None, c0.cpu(), d, None, True, cu)
    for t in (x, g, d):
        t[~keep] = float("nan")
    x, g, s0, d = x.cuda(), g.cuda(), s0.cuda(), d.cuda()

    def check(got, want, what):
        assert (got[~keep.cuda()] == 0).all(), what + ": padding"
        close(got[keep.cuda()], (want[0][keep], want[1][keep]), what)

    litter()
    check(gdn.gdn_gated_scan_fwd(x, g, s0, cu_seqlens=cd)[0], want[0], "h")
    litter()
    check(gdn.gdn_short_conv_fwd(x, w, None, c0, cu_seqlens=cd)[0], want[1], "y")
    states = gdn.gdn_gated_scan_states(x)
    gdn.gdn_gated_scan_fwd(x, g, s0, cu_seqlens=cd, states=states)
    for st in (states, None):
        litter()
        gr = gdn.gdn_gated_scan_bwd(x, g, d, s0, cu_seqlens=cd, states=st)
        for k in ("dx", "dg"):
            check(gr[k], wantg[0][k], k)
    litter()
    gr = gdn.gdn_short_conv_bwd(x, w, d, None, c0, cu_seqlens=cd)
    check(gr["dx"], wantg[1]["dx"], "dx")
    for k in ("dweight", "d_initial_state"):
        close(gr[k], wantg[1][k], k)


def test_padding_reaches_no_weight(gpu_lib):
    """A projection in front of and behind a convolution and a scan of a padded batch, whose loss takes the tokens
    alone: its weights' gradients are finite and those of the batch without padding."""
    cu, T = packed([70, 1, 130], 0, 55)
    real, cd = cu[-1], cu_dev(cu)
    u, gates = rnd(1, T, 32).cuda(), (-rnd(1, T, 64, seed=1).abs() * 0.1).cuda()
    up = rnd(1, real, 32, seed=2).cuda()
    grads = []
    for n in (T, real):
        litter()
        a, b = (rnd(64, 32, seed=3).cuda().requires_grad_(), rnd(32, 64, seed=4).cuda().requires_grad_())
        wc = rnd(64, 4, seed=5).cuda().requires_grad_()
        m, _ = gdn.short_conv(u[:, :n] @ a.t(), wc, cu_seqlens=cd)
        h, _ = gdn.gated_scan(m, gates[:, :n].contiguous(), cu_seqlens=cd)
        ((h @ b.t())[:, :real] * up).sum().backward()
        grads.append([a.grad, b.grad, wc.grad])
    for p, q in zip(*grads):
        assert torch.isfinite(p).all()
        # the same sums of at most 256 terms in another grouping: 256 half steps of the sum of absolute values, which is
        # about 16 times the sum where signs are random, taken of the largest weight
        assert (p - q).abs().max() <= 256 * ref.U * q.abs().max() * 16


# ---- chains over several groups of tiles --------------------------------------------------------

# A tile is 64 or 128 tokens; a group 8 to 64 tiles by the number of channels and the direction (512 to 8,192 tokens).
# Slow gates, so that what enters a group is much of its states.
LONG = [(2500, 2048), (5000, 512), (5000, 130), (5000, 259), (2600, 4096), (2600, 4099), (9001, 100)]
# sequences that start before a group's first token (from either end), at it and behind it, and that span groups
CUTS = [(4608, 2048, [512, 512, 1000, 24, 1, 511, 1536, 512]), (5300, 512, [1024, 1023, 2, 2047, 1204]), (5300, 131, [2047, 1, 2049, 1203]),
        (5300, 256, [4096, 0, 1204]), (3100, 4096, [1023, 2, 1023, 1052])]


@pytest.mark.parametrize("dt,gdt", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("T,D", LONG)
def test_scan_chain(T, D, dt, gdt, gpu_lib):
    x, g, s0, _ = scan_inputs(1, T, D, None, dt, gdt, True, decay=0.002)
    check_scan(x, g, s0, d_h=rnd(1, T, D, seed=7, dtype=dt), d_fin=rnd(1, D, seed=8, scale=30.0))


@pytest.mark.parametrize("T,D,lens", CUTS)
def test_scan_chain_of_packed_sequences(T, D, lens, gpu_lib):
    cu, _ = packed(lens)
    assert cu[-1] <= T
    x, g, s0, N = scan_inputs(1, T, D, cu, F32, F32, True, decay=0.002)
    check_scan(x, g, s0, cu, d_h=rnd(1, T, D, seed=7), d_fin=rnd(N, D, seed=8, scale=30.0))


# ---- norm: rows of a few columns and of more than registers hold --------------------------------


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,D", [(9, 2), (3, 5), (70, 7), (2, 16392), (2, 20001), (3, 32768), (2, 33001), (2, 65536)])
def test_rms_narrow_and_wide_rows(rows, D, dt, wdt, gpu_lib):
    """(The bounds' 64 terms a thread hold for 1,024 threads up to 65,536 columns.)"""
    base.test_rms(rows, D, dt, wdt, gpu_lib)


# ---- captured calls whose offsets change --------------------------------------------------------


@pytest.mark.parametrize("T,N,D", [(700, 5, 256), (60, 3, 131), (300, 400, 64)])
def test_graph_of_a_padded_batch(T, N, D, gpu_lib):
    """A captured forward and gradient, replayed with other inputs and other sequences (and other padding: rows that
    held results at the last replay), agrees with eager calls in every bit."""
    x, g, s0, _ = scan_inputs(1, T, D, [0] * (N + 1), BF, F32, True)
    bufs = [t.cuda() for t in (x, g, s0, rnd(D, 4, dtype=BF), rnd(N, 3, D, dtype=BF))] + [cu_dev([0] * N + [T])]

    def call(x, g, s0, w, c0, cu):
        m, cf = gdn.gdn_short_conv_fwd(x, w, None, c0, cu_seqlens=cu, output_final_state=True)
        states = gdn.gdn_gated_scan_states(m)
        h, f = gdn.gdn_gated_scan_fwd(m, g, s0, cu_seqlens=cu, states=states)
        gs = gdn.gdn_gated_scan_bwd(m, g, h, s0, f, cu_seqlens=cu, states=states)
        gc = gdn.gdn_short_conv_bwd(x, w, gs["dx"], None, c0, cf, cu_seqlens=cu)
        return [m, cf, h, f, *gs.values(), gc["dx"], gc["dweight"], gc["d_initial_state"]]

    call(*bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(*bufs)
    gen = torch.Generator().manual_seed(1)
    for it in range(5):
        cuts = sorted(torch.randint(0, T + 1, (N + 1,), generator=gen).tolist())
        fresh = scan_inputs(1, T, D, cuts, BF, F32, True, seed=10 * it + 1)[:3]
        for b, t in zip(bufs, (*fresh, rnd(D, 4, seed=it, dtype=BF), rnd(N, 3, D, seed=it, dtype=BF), torch.tensor(cuts, dtype=torch.int32))):
            b.copy_(t)
        graph.replay()
        want = call(*bufs)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (it, i)
        pad = ~owned(1, T, cuts).cuda()
        for i in (0, 2, 4, 5, 7):
            assert outs[i].shape == (1, T, D) and (outs[i][pad] == 0).all(), (it, i)
