"""The layer operators (gated scan, short convolution, RMS norm) on the GPU against the plain 64-bit forms, element
by element: an output may be off by half a step of its type plus what 32-bit arithmetic can lose on the way
(oracle/layer.py derives that bound)."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import layer as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -9, F32: 2.0 ** -24}  # half a step, relative to the power of two below the value
TINY = 1e-37  # results below fp32's normal range may be flushed


def close(got, want, what):
    value, bound = want
    got64 = got.detach().cpu().double()
    # half a step is at most HALF times the next power of two: 2 HALF times the value
    tol = 2 * HALF[got.dtype] * (value.abs() + bound) + bound + TINY
    bad = (got64 - value).abs() > tol
    assert not bad.any() and torch.isfinite(got64).all(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {((got64 - value).abs() / tol).max():.2f} of the bound")


def rnd(*shape, seed=0, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


def packed(lens, head=0, tail=0):
    cu = [head]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu, cu[-1] + tail


# (B, T, D) and packed batches: one token, tiles met and passed by one, ragged and empty sequences, tokens that
# belong to no sequence in front and behind, channels that fill vectors and ones that do not
ROWS = [(1, 128, 136), (5, 64, 130), (70, 17, 128), (130, 64, 3), (3, 128, 260), (2, 17, 64), (1, 1, 1), (3, 1, 64), (2, 5, 256), (1, 16, 513), (1, 63, 64), (1, 64, 128), (1, 65, 260), (2, 129, 96),
        (3, 200, 77), (1, 700, 520)]
PACKS = [([1], 0, 0, 8), ([0] * 200 + [20] + [0] * 300 + [90, 0] + [7] * 9, 3, 2, 132), ([2, 0, 3, 9, 1, 0, 0, 4] * 5, 0, 0, 131), ([0, 5, 0, 0, 70, 1, 1, 1, 64, 3, 0], 0, 0, 256), ([130, 200, 33], 7, 90, 72),
         ([0, 0], 0, 10, 16), ([1] * 70, 1, 1, 33), ([300, 2, 1, 90], 64, 64, 512)]
SHAPES = [("rows", s) for s in ROWS] + [("pack", s) for s in PACKS]


def shape_of(kind, s):
    if kind == "rows":
        return s[0], s[1], s[2], None
    cu, T = packed(s[0], s[1], s[2])
    return 1, T, s[3], cu


def cu_dev(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()


def owned(B, T, cu):
    m = torch.zeros(B * T, dtype=torch.bool)
    for p, q in ref.sequences(B, T, cu):
        m[p:q] = True
    return m.reshape(B, T)


def check_rows(got, want, keep, fill, what):
    """Rows of a sequence against the reference, the others still as they were."""
    value, bound = want
    close(got[keep.cuda()], (value[keep], bound[keep]), what)
    assert (got[~keep.cuda()] == fill).all(), what + ": rows outside every sequence were written"


# ---- gated scan ---------------------------------------------------------------------------------


def scan_inputs(B, T, D, cu, dt, gdt, state, seed=0, decay=0.2):
    N = B if cu is None else len(cu) - 1
    x = rnd(B, T, D, seed=seed, dtype=dt)
    g = (-torch.nn.functional.softplus(rnd(B, T, D, seed=seed + 1)) * decay).to(gdt)
    s0 = rnd(N, D, seed=seed + 2) if state else None
    return x, g, s0, N


@pytest.mark.parametrize("dt,gdt", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("kind,s", SHAPES)
def test_scan(kind, s, dt, gdt, gpu_lib):
    B, T, D, cu = shape_of(kind, s)
    for state in (False, True):
        x, g, s0, N = scan_inputs(B, T, D, cu, dt, gdt, state)
        keep, cd = owned(B, T, cu), cu_dev(cu)
        h = torch.full((B, T, D), 5.0, dtype=dt).cuda()
        states = gdn.gdn_gated_scan_states(x.cuda())
        want_h, want_fin = ref.scan_fwd(x, g, s0, cu)
        _, fin = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), cuda(s0), cu_seqlens=cd, h=h, states=states)
        check_rows(h, want_h, keep, 5.0, "h")
        close(fin, want_fin, "final_state")
        d_h, d_fin = rnd(B, T, D, seed=7, dtype=dt), rnd(N, D, seed=8) if state else None
        want = ref.scan_bwd(x, g, s0, d_h, d_fin, cu)
        got = []
        for st in (states, None):
            out = dict(dx=torch.full((B, T, D), 3.0, dtype=dt).cuda(), dg=torch.full((B, T, D), 3.0, dtype=gdt).cuda(),
                       d_initial_state=torch.empty(N, D).cuda())
            gdn.gdn_gated_scan_bwd(x.cuda(), g.cuda(), d_h.cuda(), cuda(s0), cuda(d_fin), cu_seqlens=cd, states=st, out=out)
            check_rows(out["dx"], want["dx"], keep, 3.0, "dx")
            check_rows(out["dg"], want["dg"], keep, 3.0, "dg")
            close(out["d_initial_state"], want["d_initial_state"], "d_initial_state")
            got.append(out)
        for k in got[0]:
            assert torch.equal(got[0][k], got[1][k]), k + ": kept and recomputed states differ"


def test_scan_long_and_repeatable(gpu_lib):
    """A sequence of many tiles, slow gates among them, against the sequential form; two runs agree in every bit."""
    x, g, s0, _ = scan_inputs(1, 9001, 68, None, F32, F32, True, decay=0.01)
    a = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), s0.cuda())
    b = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), s0.cuda())
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    want_h, want_fin = ref.scan_fwd(x, g, s0)
    close(a[0], want_h, "h")
    close(a[1], want_fin, "final_state")
    d_h = rnd(1, 9001, 68, seed=5)
    gr = [gdn.gdn_gated_scan_bwd(x.cuda(), g.cuda(), d_h.cuda(), s0.cuda()) for _ in range(2)]
    want = ref.scan_bwd(x, g, s0, d_h, None)
    for k in want:
        assert torch.equal(gr[0][k], gr[1][k])
        close(gr[0][k], want[k], k)


@pytest.mark.parametrize("T,D", [(70001, 8), (40000, 2048), (131072, 256)])
def test_scan_split_continues(T, D, gpu_lib):
    """Long sequences: a call of the whole equals two calls, the second from the first one's state."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, T, D, device="cuda", generator=gen)
    g = -torch.rand(1, T, D, device="cuda", generator=gen) * 0.1
    h, fin = gdn.gdn_gated_scan_fwd(x, g)
    cut = T // 2 + 13
    h1, s1 = gdn.gdn_gated_scan_fwd(x[:, :cut].contiguous(), g[:, :cut].contiguous())
    h2, s2 = gdn.gdn_gated_scan_fwd(x[:, cut:].contiguous(), g[:, cut:].contiguous(), s1)
    # both are within the 32-bit bound of the exact value; with gates of -0.05 on average a state remembers
    # about 20 tokens, whose errors of 4 half steps of |h| (up to ~20) each make the bound
    tol = 2 * 20 * 4.2 * ref.U * 40
    assert (torch.cat([h1, h2], 1) - h).abs().max() < tol and (s2 - fin).abs().max() < tol


def test_scan_packed_equals_single_calls(gpu_lib):
    lens = [500, 0, 1, 2000, 3, 64, 129]
    cu, T = packed(lens)
    x, g, s0, N = scan_inputs(1, T, 192, cu, BF, F32, True)
    x, g, s0 = x.cuda(), g.cuda(), s0.cuda()
    h, fin = gdn.gdn_gated_scan_fwd(x, g, s0, cu_seqlens=cu_dev(cu))
    for n, (p, q) in enumerate(zip(cu[:-1], cu[1:])):
        if p == q:
            assert torch.equal(fin[n], s0[n])
            continue
        h1, f1 = gdn.gdn_gated_scan_fwd(x[:, p:q].contiguous(), g[:, p:q].contiguous(), s0[n:n + 1])
        # the same values up to the order of the tiles: a bf16 step, 32-bit rounding in the state
        assert (h1.float() - h[:, p:q].float()).abs().max() <= 2 ** -7 * h1.float().abs().max()
        assert torch.allclose(f1[0], fin[n], rtol=1e-5, atol=1e-5)


def test_scan_steps_equal_prefill(gpu_lib):
    """Decoding in place, one token and then several per call, continues as the long call does."""
    x, g, s0, _ = scan_inputs(3, 40, 130, None, F32, F32, True)
    x, g = x.cuda(), g.cuda()
    want_h, want_fin = ref.scan_fwd(x, g, s0)
    state, outs, t = s0.cuda(), [], 0
    for n in [1] * 10 + [2, 3, 7, 18]:
        h, st = gdn.gdn_gated_scan_fwd(x[:, t:t + n].contiguous(), g[:, t:t + n].contiguous(), state, final_state=state)
        assert st is state
        outs.append(h)
        t += n
    close(torch.cat(outs, 1), want_h, "h")
    close(state, want_fin, "state")


def test_scan_in_place_state_of_long_rows(gpu_lib):
    x, g, s0, _ = scan_inputs(2, 5000, 64, None, BF, F32, True)
    _, fin = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), s0.cuda())
    state = s0.cuda()
    gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), state, final_state=state)
    assert torch.equal(state, fin)


def test_scan_in_place_state_of_packed_sequences(gpu_lib):
    """Sequences that start and end in one tile, in one wave and tiles apart."""
    for lens in ([300, 2, 3, 0, 1, 100, 700, 5], [1, 0, 2, 3, 1]):
        cu, T = packed(lens)
        x, g, s0, _ = scan_inputs(1, T, 260, cu, F32, F32, True)
        x, g, cd = x.cuda(), g.cuda(), cu_dev(cu)
        h, fin = gdn.gdn_gated_scan_fwd(x, g, s0.cuda(), cu_seqlens=cd)
        for _ in range(3):
            state = s0.cuda()
            h2, _ = gdn.gdn_gated_scan_fwd(x, g, state, cu_seqlens=cd, final_state=state)
            assert torch.equal(state, fin) and torch.equal(h, h2)


def test_scan_many_sequences(gpu_lib):
    """Thousands of short sequences, most of them empty in one case, equal a plain loop over the longest."""
    for lens in ([3] * 3000, ([0] * 9 + [41]) * 400, [5, 0, 8] * 700):
        cu, T = packed(lens)
        D, N = 128, len(lens)
        x, g, s0, _ = scan_inputs(1, T, D, cu, F32, F32, True)
        h, fin = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), s0.cuda(), cu_seqlens=cu_dev(cu))
        y, cf = gdn.gdn_short_conv_fwd(x.cuda(), rnd(D, 2, seed=5).cuda(), None, s0[:, None].contiguous().cuda(), activation=None,
                                       cu_seqlens=cu_dev(cu), output_final_state=True)
        start, n = torch.tensor(cu[:-1]), torch.tensor(lens)
        c, prev = s0.double(), s0.double()
        w = rnd(D, 2, seed=5).double()
        for t in range(max(lens)):
            on = n > t
            at = (start + t)[on]
            c[on] = g[0, at].double().exp() * c[on] + x[0, at].double()
            # 32 bits: 5 half steps a token of a state below 10, over at most 41 tokens
            assert (h[0].cpu().double()[at] - c[on]).abs().max() < 41 * 5 * ref.U * 10
            z = prev[on] * w[:, 0] + x[0, at].double() * w[:, 1]
            assert (y[0].cpu().double()[at] - z).abs().max() < 3 * ref.U * 40
            prev[on] = x[0, at].double()
        assert (fin.cpu().double() - c).abs().max() < 41 * 5 * ref.U * 10
        assert torch.equal(cf[:, 0].cpu().double(), prev)


@pytest.mark.parametrize("dt,gdt", [(BF, F32), (F32, F32)])
@pytest.mark.parametrize("s", [([1] * 90, 0, 0, 260), ([0] * 300 + [40, 1, 0, 16, 1, 17, 1, 1], 5, 3, 131),
                               ([1] * 300, 2, 0, 64), ([0] * 400 + [300], 0, 1, 130), ([1] * 128 + [400], 0, 0, 256),
                               ([1] * 600, 0, 0, 128)])
def test_scan_decoding_batches(s, dt, gdt, gpu_lib):
    """Packed batches of single tokens, among them long sequences between empty ones, and a long prefill."""
    test_scan("pack", s, dt, gdt, gpu_lib)


def test_states_of_many_empty_sequences(gpu_lib):
    """States (and their gradients) of 10,000 sequences without tokens pass through, those of the others do not."""
    lens = [0] * 5000 + [33, 0, 600] + [0] * 5000
    cu, T = packed(lens)
    for D in (64, 131):
        x, g, s0, N = scan_inputs(1, T, D, cu, F32, F32, True)
        some = torch.tensor(lens) == 0
        h, fin = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), s0.cuda(), cu_seqlens=cu_dev(cu))
        gr = gdn.gdn_gated_scan_bwd(x.cuda(), g.cuda(), h, s0.cuda(), s0.cuda() * 2, cu_seqlens=cu_dev(cu))
        assert torch.equal(fin.cpu()[some], s0[some]) and torch.equal(gr["d_initial_state"].cpu()[some], 2 * s0[some])
        assert (fin.cpu()[~some] != s0[~some]).all() and torch.isfinite(fin).all()
        w, c0 = rnd(D, 4, seed=9), rnd(N, 3, D, seed=10)
        y, cf = gdn.gdn_short_conv_fwd(x.cuda(), w.cuda(), None, c0.cuda(), cu_seqlens=cu_dev(cu), output_final_state=True)
        gc = gdn.gdn_short_conv_bwd(x.cuda(), w.cuda(), y, None, c0.cuda(), c0.cuda() * 2, cu_seqlens=cu_dev(cu))
        assert torch.equal(cf.cpu()[some], c0[some]) and torch.equal(gc["d_initial_state"].cpu()[some], 2 * c0[some])
        assert torch.equal(cf[5000].cpu(), x[0, 30:33]) and torch.equal(cf[5002].cpu(), x[0, -3:])


def test_nearly_all_sequences_empty(gpu_lib):
    """More sequences than 2^30: their numbers' sum passes 32 bits."""
    N, T, D = 1_200_000_000, 100, 8
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    cu[-1] = T
    x, w = rnd(1, T, D).cuda(), rnd(D, 4, seed=1).cuda()
    y, _ = gdn.gdn_short_conv_fwd(x, w, cu_seqlens=cu)
    assert torch.equal(y, gdn.gdn_short_conv_fwd(x, w)[0])
    g = -torch.ones(1, T, D).cuda()
    h, _ = gdn.gdn_gated_scan_fwd(torch.cat([x] * 6, 1), torch.cat([g] * 6, 1), cu_seqlens=cu * 6, output_final_state=False)
    want, _ = gdn.gdn_gated_scan_fwd(torch.cat([x] * 6, 1), torch.cat([g] * 6, 1))
    assert torch.equal(h, want)


def test_scan_gradient_of_many_sequences(gpu_lib):
    lens = [3, 0, 1, 9, 0, 0, 17, 2] * 20 + [0] * 50 + [70, 1]
    cu, T = packed(lens, 2, 5)
    x, g, s0, N = scan_inputs(1, T, 129, cu, BF, F32, True)
    d_h, d_fin = rnd(1, T, 129, seed=7, dtype=BF), rnd(N, 129, seed=8)
    want = ref.scan_bwd(x, g, s0, d_h, d_fin, cu)
    keep = owned(1, T, cu)
    got = gdn.gdn_gated_scan_bwd(x.cuda(), g.cuda(), d_h.cuda(), s0.cuda(), d_fin.cuda(), cu_seqlens=cu_dev(cu))
    for k in ("dx", "dg"):
        close(got[k][keep.cuda()], (want[k][0][keep], want[k][1][keep]), k)
    close(got["d_initial_state"], want["d_initial_state"], "d_initial_state")


def test_scan_gates_at_the_edges(gpu_lib):
    """-inf forgets, +growth from a zero state stays finite, and what one sequence holds (NaN, infinity) does not
    reach the next."""
    cu, T = packed([300, 400, 300])
    x, g, _, _ = scan_inputs(1, T, 64, cu, F32, F32, False)
    g[0, 100] = float("-inf")
    x[0, 650] = float("nan")
    x[0, 600, 3] = float("inf")
    h, fin = gdn.gdn_gated_scan_fwd(x.cuda(), g.cuda(), cu_seqlens=cu_dev(cu))
    assert torch.equal(h[0, 100].cpu(), x[0, 100])
    assert torch.isfinite(h[0, :600]).all() and torch.isnan(h[0, 650:700]).all() and torch.isfinite(h[0, 700:]).all()
    assert torch.isfinite(fin[0]).all() and torch.isnan(fin[1]).all() and torch.isfinite(fin[2]).all()
    d_h = rnd(1, T, 64, seed=3)
    d_h[0, 320] = float("nan")
    gr = gdn.gdn_gated_scan_bwd(x.cuda(), g.cuda(), d_h.cuda(), cu_seqlens=cu_dev(cu))
    assert torch.isfinite(gr["dx"][0, :300]).all() and torch.isfinite(gr["dx"][0, 321:]).all()
    assert (gr["dg"][0, 100] == 0).all()
    # gates above zero: a state that grows fourfold over a tile, against the sequential form
    x, g, s0, _ = scan_inputs(1, 200, 64, None, F32, F32, True)
    want_h, want_fin = ref.scan_fwd(x, -g * 0.1, s0)
    h, fin = gdn.gdn_gated_scan_fwd(x.cuda(), (-g * 0.1).cuda(), s0.cuda())
    close(h, want_h, "h")
    close(fin, want_fin, "final_state")
    # growth: the product of 64 gates overflows, but there is no state for it to act on until the input comes
    x = torch.zeros(1, 600, 64)
    x[0, 599] = 1.0
    h, fin = gdn.gdn_gated_scan_fwd(x.cuda(), torch.full((1, 600, 64), 2.0).cuda())
    assert (fin == 1).all() and (h[0, :599] == 0).all()


def test_scan_no_tokens(gpu_lib):
    s0 = rnd(2, 8).cuda()
    h, fin = gdn.gdn_gated_scan_fwd(torch.empty(2, 0, 8).cuda(), torch.empty(2, 0, 8).cuda(), s0)
    assert h.shape == (2, 0, 8) and torch.equal(fin, s0)
    gr = gdn.gdn_gated_scan_bwd(torch.empty(2, 0, 8).cuda(), torch.empty(2, 0, 8).cuda(), h, s0, s0 * 2)
    assert torch.equal(gr["d_initial_state"], s0 * 2)


def test_scan_beyond_32_bit_offsets(gpu_lib):
    """More than 2^31 elements: the last sequence of a packed batch equals a call of its own."""
    T, D, last = 530000, 4096, 150
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1, T, D, device="cuda", generator=gen, dtype=BF)
    g = (-torch.rand(1, T, D, device="cuda", generator=gen, dtype=BF) * 0.1)
    cu = torch.tensor([0, T - last, T], dtype=torch.int32).cuda()
    h, fin = gdn.gdn_gated_scan_fwd(x, g, cu_seqlens=cu)
    h1, f1 = gdn.gdn_gated_scan_fwd(x[:, T - last:].contiguous(), g[:, T - last:].contiguous())
    assert (h1.float() - h[:, T - last:].float()).abs().max() <= 2 ** -7 * h1.float().abs().max()
    assert torch.allclose(f1[0], fin[1], rtol=1e-5, atol=1e-5)


# ---- short convolution --------------------------------------------------------------------------


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("kind,s", SHAPES)
def test_conv(kind, s, dt, wdt, gpu_lib):
    B, T, D, cu = shape_of(kind, s)
    N = B if cu is None else len(cu) - 1
    for W, silu, bias, state in ((4, True, True, True), (3, False, False, True), (2, True, False, False)):
        x, w = rnd(B, T, D, dtype=dt), rnd(D, W, seed=1, dtype=wdt)
        b = rnd(D, seed=2, dtype=wdt) if bias else None
        s0 = rnd(N, W - 1, D, seed=3, dtype=dt) if state else None
        act = "silu" if silu else None
        keep, cd = owned(B, T, cu), cu_dev(cu)
        y = torch.full((B, T, D), 5.0, dtype=dt).cuda()
        _, fin = gdn.gdn_short_conv_fwd(x.cuda(), w.cuda(), cuda(b), cuda(s0), activation=act, cu_seqlens=cd, y=y,
                                        output_final_state=True)
        want_y, want_fin = ref.conv_fwd(x, w, b, s0, silu, cu)
        check_rows(y, want_y, keep, 5.0, "y")
        assert torch.equal(fin.cpu().double(), want_fin)
        d_y = rnd(B, T, D, seed=4, dtype=dt)
        d_fin = rnd(N, W - 1, D, seed=5, dtype=dt) if state else None
        out = dict(dx=torch.full((B, T, D), 3.0, dtype=dt).cuda(), dweight=torch.empty(D, W).cuda(),
                   dbias=torch.empty(D).cuda() if bias else None, d_initial_state=torch.empty(N, W - 1, D, dtype=dt).cuda())
        gdn.gdn_short_conv_bwd(x.cuda(), w.cuda(), d_y.cuda(), cuda(b), cuda(s0), cuda(d_fin), activation=act,
                               cu_seqlens=cd, out=out)
        want = ref.conv_bwd(x, w, b, s0, d_y, d_fin, silu, cu)
        check_rows(out["dx"], want["dx"], keep, 3.0, "dx")
        for k in ("dweight", "d_initial_state") + (("dbias",) if bias else ()):
            close(out[k], want[k], k)


def test_conv_long_sums_repeatable(gpu_lib):
    x, w, d_y = rnd(2, 6001, 40), rnd(40, 4, seed=1), rnd(2, 6001, 40, seed=2)
    gr = [gdn.gdn_short_conv_bwd(x.cuda(), w.cuda(), d_y.cuda()) for _ in range(2)]
    want = ref.conv_bwd(x, w, None, None, d_y, None, True)
    for k in ("dx", "dweight", "d_initial_state"):
        assert torch.equal(gr[0][k], gr[1][k])
        close(gr[0][k], want[k], k)


def test_conv_steps_equal_prefill(gpu_lib):
    x, w, s0 = rnd(3, 40, 130), rnd(130, 4, seed=1), rnd(3, 3, 130, seed=2)
    want, want_fin = ref.conv_fwd(x, w, None, s0, True)
    xd, state, outs, t = x.cuda(), s0.cuda(), [], 0
    for n in [1] * 10 + [2, 3, 9, 16]:
        y, st = gdn.gdn_short_conv_fwd(xd[:, t:t + n].contiguous(), w.cuda(), None, state, final_state=state)
        assert st is state
        outs.append(y)
        t += n
    close(torch.cat(outs, 1), want, "y")
    assert torch.equal(state.cpu().double(), want_fin)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_short_conv_fwd(xd[:, :17].contiguous(), w.cuda(), None, state, final_state=state)


def test_conv_nan_stays_in_its_sequence(gpu_lib):
    cu, T = packed([20, 30, 40])
    x, w = rnd(1, T, 64), rnd(64, 4, seed=1)
    x[0, 49] = float("nan")
    y, _ = gdn.gdn_short_conv_fwd(x.cuda(), w.cuda(), cu_seqlens=cu_dev(cu))
    assert torch.isnan(y[0, 49]).all() and torch.isfinite(y[0, :49]).all() and torch.isfinite(y[0, 50:]).all()
    d_y = rnd(1, T, 64, seed=2)
    d_y[0, 50] = float("nan")
    gr = gdn.gdn_short_conv_bwd(torch.nan_to_num(x).cuda(), w.cuda(), d_y.cuda(), cu_seqlens=cu_dev(cu))
    assert torch.isfinite(gr["dx"][0, :50]).all() and torch.isnan(gr["dx"][0, 50]).all() and torch.isfinite(gr["dx"][0, 51:]).all()
    big = torch.full((1, 8, 64), 1e30)
    y, _ = gdn.gdn_short_conv_fwd(big.cuda(), torch.ones(64, 4).cuda() * -1e3)
    assert (y == 0).all()  # silu of a value far below zero


# ---- RMS norm -----------------------------------------------------------------------------------

RMS_SHAPES = [(1, 1), (70, 8), (35, 255), (9, 256), (9, 257), (700, 136), (131, 31), (65, 32), (66, 33), (19, 127), (17, 128), (3, 1023), (5, 520), (3, 8), (2, 100), (5, 128), (7, 129), (4, 512), (3, 513), (2, 1000), (9, 1024), (3, 2047), (2, 2048),
              (300, 2056), (2, 4096), (2, 5120), (3, 8192), (2, 8200), (1, 16384), (70, 264)]


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,D", RMS_SHAPES)
def test_rms(rows, D, dt, wdt, gpu_lib):
    x, w = rnd(rows, D, dtype=dt), (rnd(D, seed=1, scale=0.3) + 1).to(wdt)
    for res in (None, rnd(rows, D, seed=2, dtype=dt, scale=3.0)):
        want, bound, r = ref.rms_fwd(x, res, w, 1e-6)
        y, kept, scale = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda(), cuda(res))
        assert scale is None and (kept is None) == (res is None)
        close(y, (want, bound), "y")
        if res is not None:
            assert torch.equal(kept.cpu(), r)
        for quant, G in (("row", D), ("group", 128)):
            check_quant(gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda(), cuda(res), quant=quant), want, bound, r if res is not None else None, G)
        d_y, d_res = rnd(rows, D, seed=3, dtype=dt), None if res is None else rnd(rows, D, seed=4, dtype=dt)
        gr = gdn.gdn_rmsnorm_bwd(r.cuda(), w.cuda(), d_y.cuda(), cuda(d_res))
        wantg = ref.rms_bwd(r, w, d_y, d_res, 1e-6)
        close(gr["dx"], wantg["dx"], "dx")
        close(gr["dweight"], wantg["dweight"], "dweight")


def check_quant(got, want, bound, r, G):
    q, kept, scale = got
    rows, D = want.shape
    groups = -(-D // G)
    assert q.dtype == torch.float8_e4m3fn and scale.shape == (rows, groups)
    if r is not None:
        assert torch.equal(kept.cpu(), r)
    v, s = q.cpu().float().double(), scale.cpu().double().repeat_interleave(G, 1)[:, :D]
    rel = ref.RSTD + 6 * ref.U  # the scale's and the value's relative error before the rounding to 8 bits
    amax = torch.stack([c.abs().amax(1) for c in want.split(G, 1)], 1)
    assert ((scale.cpu().double() - amax / 448).abs() <= rel * amax / 448 + TINY).all()
    exact = want / s
    # e4m3: half a step is 2^-4 of the power of two below the value, and 2^-10 below the smallest normal 2^-6
    step = torch.exp2(torch.floor(torch.log2(exact.abs().clamp(min=2.0 ** -6))))
    assert ((v - exact).abs() <= step * 2.0 ** -4 * (1 + 1e-6) + rel * exact.abs() + 2.0 ** -10 * 1e-3).all()
    top = torch.stack([c.abs().amax(1) for c in v.split(G, 1)], 1)
    assert (top == 448).all()


def test_rms_zero_rows_and_bad_values(gpu_lib):
    for D in (128, 300, 2048, 9000):
        x = rnd(6, D)
        x[1] = 0
        x[2, 5] = float("nan")
        x[3, 5] = float("inf")
        x[4] = 1e-30
        w = torch.ones(D)
        y, _, _ = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda())
        y = y.cpu()
        assert (y[1] == 0).all() and torch.isnan(y[2]).all()
        assert torch.isnan(y[3, 5]) and (y[3, 6:] == 0).all()
        assert torch.isfinite(y[[0, 4, 5]]).all()
        for quant in ("row", "group"):
            q, _, s = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda(), quant=quant)
            q, s = q.float().cpu(), s.cpu()
            assert (q[1] == 0).all() and (s[1] == 1).all()
            assert torch.isnan(s[2]).all() and torch.isnan(q[2]).all()
            assert torch.isnan(s[3, 0]) and torch.isnan(q[3, :100]).all()
            if quant == "group" and D > 128:
                assert (s[3, 1:] == 1).all() and (q[3, 128:] == 0).all()
            assert torch.isfinite(q[[0, 4, 5]]).all()
        gr = gdn.gdn_rmsnorm_bwd(x.cuda(), w.cuda(), rnd(6, D, seed=1).cuda())
        assert torch.isfinite(gr["dx"][[0, 1, 4, 5]]).all()


def test_rms_infinite_gradient(gpu_lib):
    """An infinity in d_y reaches its row as the formula says (mean(w d_y rh) infinite), also where the row's last
    columns are read along with their neighbours'."""
    for D in (12, 100, 300, 2044, 9001):
        r, w, d_y = rnd(2, D).abs() + 0.1, rnd(D, seed=1).abs() + 0.1, rnd(2, D, seed=2)
        r[:, ::3] *= -1
        at = D - 6  # before the columns that the last vector owns (8 ceil(D / 8) - 8 on), inside what it reads
        d_y[0, at] = float("inf")
        got = gdn.gdn_rmsnorm_bwd(r.cuda(), w.cuda(), d_y.cuda())
        rest = torch.arange(D) != at
        want = -torch.sign(r[0]) * torch.sign(r[0, at]) * float("inf")
        assert torch.equal(got["dx"][0].cpu()[rest], want[rest]), D
        close(got["dx"][1:], [v[1:] for v in ref.rms_bwd(r, w, torch.nan_to_num(d_y, posinf=0.0), None, 1e-6)["dx"]], "dx")


def test_rms_in_place_residual(gpu_lib):
    for D in (2048, 300, 20000):
        x, res, w = rnd(9, D, dtype=BF).cuda(), rnd(9, D, seed=1, dtype=BF).cuda(), torch.ones(D).cuda()
        y, kept, _ = gdn.gdn_rmsnorm_fwd(x, w, res)
        for which in ("x", "residual"):
            xc, rc = x.clone(), res.clone()
            y2, kept2, _ = gdn.gdn_rmsnorm_fwd(xc, w, rc, residual_out=xc if which == "x" else rc)
            assert torch.equal(y, y2) and torch.equal(kept, kept2)


def test_rms_many_rows_repeatable(gpu_lib):
    r, w, d_y = rnd(5000, 264, dtype=BF), rnd(264, seed=1, dtype=BF), rnd(5000, 264, seed=2, dtype=BF)
    gr = [gdn.gdn_rmsnorm_bwd(r.cuda(), w.cuda(), d_y.cuda()) for _ in range(2)]
    want = ref.rms_bwd(r, w, d_y, None, 1e-6)
    for k in want:
        assert torch.equal(gr[0][k], gr[1][k])
        close(gr[0][k], want[k], k)


def test_rms_wide_rows(gpu_lib):
    """Rows beyond what a workgroup holds in registers."""
    x, w = rnd(3, 40000, dtype=BF), rnd(40000, seed=1, dtype=BF)
    want, bound, _ = ref.rms_fwd(x, None, w, 1e-6)
    y, _, _ = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda())
    close(y, (want, bound * 3), "y")  # 40000 / 16384 as many terms in the sum
    d_y = rnd(3, 40000, seed=2, dtype=BF)
    gr = gdn.gdn_rmsnorm_bwd(x.cuda(), w.cuda(), d_y.cuda())
    want = ref.rms_bwd(x, w, d_y, None, 1e-6)
    close(gr["dx"], (want["dx"][0], want["dx"][1] * 3), "dx")
    close(gr["dweight"], (want["dweight"][0], want["dweight"][1] * 3), "dweight")


def test_rms_no_rows(gpu_lib):
    gr = gdn.gdn_rmsnorm_bwd(torch.empty(0, 64).cuda(), torch.ones(64).cuda(), torch.empty(0, 64).cuda())
    assert gr["dx"].shape == (0, 64) and (gr["dweight"] == 0).all()
    y, _, s = gdn.gdn_rmsnorm_fwd(torch.empty(0, 64).cuda(), torch.ones(64).cuda(), quant="row")
    assert y.shape == (0, 64) and s.shape == (0, 1)


# ---- what holds for all of them -----------------------------------------------------------------


def test_unaligned_buffers(gpu_lib):
    """Contiguous tensors that start off a 16-byte boundary give what aligned ones give."""
    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    for dt in (BF, F32):
        x, g, s0, _ = scan_inputs(2, 100, 256, None, dt, dt, True)
        want, want_fin = ref.scan_fwd(x, g, s0)
        h, fin = gdn.gdn_gated_scan_fwd(off(x), off(g), off(s0))
        close(h, want, "h")
        close(fin, want_fin, "final_state")
        d_h = rnd(2, 100, 256, seed=9, dtype=dt)
        gr, wantg = gdn.gdn_gated_scan_bwd(off(x), off(g), off(d_h), off(s0)), ref.scan_bwd(x, g, s0, d_h, None)
        for k in wantg:
            close(gr[k], wantg[k], k)
        w, c0 = rnd(256, 4, dtype=dt), rnd(2, 3, 256, seed=2, dtype=dt)
        y, _ = gdn.gdn_short_conv_fwd(off(x), off(w), None, off(c0))
        close(y, ref.conv_fwd(x, w, None, c0, True)[0], "y")
        gr = gdn.gdn_short_conv_bwd(off(x), off(w), off(d_h), None, off(c0))
        wantg = ref.conv_bwd(x, w, None, c0, d_h, None, True)
        for k in ("dx", "dweight", "d_initial_state"):
            close(gr[k], wantg[k], k)
        wn = rnd(256, seed=3, dtype=dt)
        y, _, _ = gdn.gdn_rmsnorm_fwd(off(x), off(wn))
        close(y, ref.rms_fwd(x, None, wn, 1e-6)[:2], "norm")
        gr, wantg = gdn.gdn_rmsnorm_bwd(off(x), off(wn), off(d_h)), ref.rms_bwd(x, wn, d_h, None, 1e-6)
        for k in wantg:
            close(gr[k], wantg[k], k)


def test_refusals(gpu_lib):
    x = torch.zeros(1, 8, 16, device="cuda")
    for bad in (x.double(), x.half(), x.transpose(1, 2), x[0]):
        with pytest.raises((TypeError, ValueError)):
            gdn.gdn_gated_scan_fwd(bad, bad)
        with pytest.raises((TypeError, ValueError)):
            gdn.gdn_short_conv_fwd(bad, torch.zeros(16, 4, device="cuda"))
    with pytest.raises((TypeError, ValueError)):
        gdn.gdn_rmsnorm_fwd(x.half(), torch.zeros(16, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(x, x[:, :4])
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(x, x.to(BF))
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(x, x, torch.zeros(2, 16, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(x, x, states=torch.zeros(2, 16, device="cuda"))
    long = torch.zeros(1, 300, 16, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(long, long, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        gdn.gdn_gated_scan_fwd(x, x, cu_seqlens=torch.tensor([0, 8]).cuda())
    with pytest.raises(TypeError):
        gdn.gdn_gated_scan_fwd(x, x, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(x.reshape(2, 4, 16), x.reshape(2, 4, 16), cu_seqlens=cu_dev([0, 8]))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_short_conv_fwd(x, torch.zeros(16, 5, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_short_conv_fwd(x, torch.zeros(16, 4, device="cuda"), activation="relu")
    with pytest.raises(ValueError):
        gdn.gdn_short_conv_fwd(x, torch.zeros(16, 4, device="cuda"), None, torch.zeros(1, 4, 16, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_rmsnorm_fwd(x, torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_rmsnorm_fwd(x, torch.zeros(16, device="cuda"), quant="column")
    with pytest.raises(gdn.GdnError):
        gdn.gdn_rmsnorm_fwd(x, torch.zeros(16, device="cuda"), eps=-1.0)


def test_offsets_out_of_order_stay_in_bounds(gpu_lib):
    """Offsets that decrease or lie outside give unspecified rows; everything around the buffers stays."""
    T, D = 200, 64
    pad = torch.full((3 * T, D), 7.0, device="cuda")
    out = pad[T:2 * T].view(1, T, D)
    x, g = rnd(1, T, D).cuda(), -torch.ones(1, T, D).cuda()
    for cu in ([0, 150, 20, 200], [-50, 100, 10 ** 6, 200], [200, 100, 0, 50]):
        gdn.gdn_gated_scan_fwd(x, g, cu_seqlens=cu_dev(cu), h=out)
        gdn.gdn_short_conv_fwd(x, rnd(D, 4).cuda(), cu_seqlens=cu_dev(cu), y=out, output_final_state=True)
        gdn.gdn_gated_scan_bwd(x, g, x.clone(), cu_seqlens=cu_dev(cu), out=dict(dx=out, dg=torch.empty_like(g), d_initial_state=torch.empty(3, D).cuda()))
        gdn.gdn_short_conv_bwd(x, rnd(D, 4).cuda(), x.clone(), cu_seqlens=cu_dev(cu),
                               out=dict(dx=out, dweight=torch.empty(D, 4).cuda(), d_initial_state=torch.empty(3, 3, D).cuda()))
        torch.cuda.synchronize()
        assert (pad[:T] == 7).all() and (pad[2 * T:] == 7).all()


def everything(x, g, s0, w, c0, wn, cu, ws):
    """Every operator once, forward and backward; ws: one workspace for all of them."""
    h, fin = gdn.gdn_gated_scan_fwd(x, g, s0, cu_seqlens=cu, workspace=ws)
    gs = gdn.gdn_gated_scan_bwd(x, g, h, s0, fin, cu_seqlens=cu, workspace=ws)
    y, cf = gdn.gdn_short_conv_fwd(x, w, None, c0, cu_seqlens=cu, output_final_state=True)
    gc = gdn.gdn_short_conv_bwd(x, w, y, None, c0, cf, cu_seqlens=cu, workspace=ws)
    q, kept, sc = gdn.gdn_rmsnorm_fwd(x, wn, y, quant="group")
    gn = gdn.gdn_rmsnorm_bwd(kept, wn, x, y, workspace=ws)
    return [h, fin, gs["dx"], gs["dg"], gs["d_initial_state"], y, cf, gc["dx"], gc["dweight"], gc["d_initial_state"],
            q.view(torch.uint8), kept, sc, gn["dx"], gn["dweight"]]


def all_inputs(seed, D=256, lens=(700, 0, 300, 1, 64)):
    cu, T = packed(list(lens))
    x, g, s0, N = scan_inputs(1, T, D, cu, BF, F32, True, seed=seed)
    w, c0, wn = rnd(D, 4, seed=seed + 3, dtype=BF), rnd(N, 3, D, seed=seed + 4, dtype=BF), rnd(D, seed=seed + 5, dtype=BF)
    return [t.cuda() for t in (x, g, s0, w, c0, wn)] + [cu_dev(cu)]


def test_graphs_share_a_workspace(gpu_lib):
    """Two captured graphs of all operators on one workspace, replayed in turn with other inputs and eager work in
    between, agree with eager calls in every bit each time."""
    ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    ins = [all_inputs(1), all_inputs(50, lens=(64, 1000, 5))]
    everything(*ins[0], ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(everything(*ins[k], ws))
        graphs.append(gr)
    for it in range(4):
        for k in (0, 1) if it % 2 else (1, 0):
            fresh = all_inputs(100 + 10 * it + k) if k == 0 else all_inputs(100 + 10 * it + k, lens=(64, 1000, 5))
            for a, b in zip(ins[k], fresh):
                a.copy_(b)
            ws.fill_(it * 50 + 3)
            graphs[k].replay()
            want = everything(*ins[k], None)
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(outs[k], want)):
                assert torch.equal(a, b), (it, k, i)


def test_two_streams_at_once(gpu_lib):
    ins = [all_inputs(1, D=512, lens=(5000, 3000)), all_inputs(2, D=512, lens=(100, 7900))]
    want = [everything(*i, None) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = everything(*ins[k], None)
        torch.cuda.synchronize()
        for k in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(got[k], want[k])), k


def test_kernel_timing_names(gpu_lib):
    gdn.gdn_profile_enable(True)
    try:
        everything(*all_inputs(1), None)
        seen = gdn.gdn_profile_read()
    finally:
        gdn.gdn_profile_enable(False)
    for name in ("gated_scan_fwd", "gated_scan_bwd", "short_conv_fwd", "short_conv_bwd", "rmsnorm_fwd", "rmsnorm_bwd"):
        assert seen[name][0] == 1 and seen[name][1] > 0, seen


# ---- a layer of them ----------------------------------------------------------------------------




def test_layer_together(gpu_lib):
    """One layer as it is used, packed sequences, in fp32: residual add and norm, short convolution, the gated delta
    rule on its q, k, v and a gated scan on its v; outputs, states and the gradients of every input against the
    same formulas in 64 bits under torch's automatic differentiation."""
    H, K, V = 1, 64, 64
    D = H * (2 * K + V)
    lens = [70, 0, 1, 130]
    cu, T = packed(lens)
    N = len(lens)
    leaves = dict(x=rnd(1, T, D), res=rnd(1, T, D, seed=1), wn=rnd(D, seed=2, scale=0.2) + 1, wc=rnd(D, 4, seed=3, scale=0.5),
                  c0=rnd(N, 3, D, seed=4), g=-rnd(1, T, H, seed=5).abs() * 0.1, beta=torch.sigmoid(rnd(1, T, H, seed=6)),
                  s0=rnd(N, H, V, K, seed=7, scale=0.1), gs=-rnd(1, T, H * V, seed=8).abs() * 0.1, h0=rnd(N, H * V, seed=9))
    ups = [rnd(1, T, H, V, seed=20), rnd(1, T, H * V, seed=21), rnd(1, T, D, seed=22), rnd(N, H, V, K, seed=23, scale=0.1),
           rnd(N, H * V, seed=24)]

    dev = {k: v.cuda().requires_grad_() for k, v in leaves.items()}
    cud = cu_dev(cu)
    n, kept = gdn.rms_norm(dev["x"], dev["wn"], dev["res"])
    m, _ = gdn.short_conv(n, dev["wc"], None, dev["c0"], cu_seqlens=cud)
    q, k, v = m.reshape(1, T, H, 2 * K + V).split([K, K, V], -1)
    o, sT = gdn.chunk_gated_delta_rule(q.contiguous(), k.contiguous(), v.contiguous(), dev["g"], dev["beta"],
                                       initial_state=dev["s0"], cu_seqlens=cud, qk_l2norm=True)
    h, hT = gdn.gated_scan(v.reshape(1, T, H * V).contiguous(), dev["gs"], dev["h0"], cu_seqlens=cud)
    outs = [o, h, kept, sT, hT]
    got = torch.autograd.grad(sum((a * u.cuda()).sum() for a, u in zip(outs, ups)), list(dev.values()))

    r64 = {k: v.double().requires_grad_() for k, v in leaves.items()}
    kept = r64["x"] + r64["res"]
    n = kept / torch.sqrt((kept * kept).mean(-1, keepdim=True) + 1e-6) * r64["wn"]
    os_, hs, sTs, hTs = [], [], [], []
    for i, (p, e) in enumerate(zip(cu[:-1], cu[1:])):
        ext = torch.cat([r64["c0"][i], n[0, p:e]])
        z = sum(ext[j:j + e - p] * r64["wc"][:, j] for j in range(4))
        m = z * torch.sigmoid(z)
        S, c = r64["s0"][i, 0], r64["h0"][i]
        for t in range(e - p):
            q, k, v = m[t].split([K, K, V])
            q, k = (u / torch.sqrt((u * u).sum() + 1e-6) for u in (q, k))
            a, b = r64["g"][0, p + t, 0].exp(), r64["beta"][0, p + t, 0]
            S = a * (S - b * torch.outer(S @ k, k)) + b * torch.outer(v, k)
            os_.append(S @ q)
            c = r64["gs"][0, p + t].exp() * c + v
            hs.append(c)
        sTs.append(S)
        hTs.append(c)
    refs = [torch.stack(os_).reshape(1, T, 1, V), torch.stack(hs).reshape(1, T, V), kept, torch.stack(sTs).unsqueeze(1), torch.stack(hTs)]
    want = torch.autograd.grad(sum((a * u.double()).sum() for a, u in zip(refs, ups)), list(r64.values()))
    # fp32 throughout: the delta rule's own bound for fp32 (1e-4 relative) holds the chain
    for a, b in zip(outs, refs):
        assert (a.detach().cpu().double() - b).norm() <= 1e-4 * b.norm()
    for name, a, b in zip(leaves, got, want):
        assert (a.cpu().double() - b).norm() <= 1e-4 * b.norm(), name


def test_layer_decodes_as_it_prefills(gpu_lib):
    """Norm, convolution and scan, token by token with states in place, against one call of the whole prompt."""
    B, T, D = 2, 24, 128
    x, res, g = rnd(B, T, D, dtype=BF).cuda(), rnd(B, T, D, seed=1, dtype=BF).cuda(), (-rnd(B, T, D, seed=2).abs() * 0.1).cuda()
    wn, wc = torch.ones(D, dtype=BF).cuda(), rnd(D, 4, seed=3, dtype=BF).cuda()
    n, _, _ = gdn.gdn_rmsnorm_fwd(x, wn, res)
    m, c_end = gdn.gdn_short_conv_fwd(n, wc, output_final_state=True)
    h, s_end = gdn.gdn_gated_scan_fwd(m, g)
    conv, state, hs = torch.zeros(B, 3, D, dtype=BF).cuda(), torch.zeros(B, D).cuda(), []
    for t in range(T):
        xt, rt, gt = (a[:, t:t + 1].contiguous() for a in (x, res, g))
        n, _, _ = gdn.gdn_rmsnorm_fwd(xt, wn, rt)
        m, _ = gdn.gdn_short_conv_fwd(n, wc, None, conv, final_state=conv)
        ht, _ = gdn.gdn_gated_scan_fwd(m, gt, state, final_state=state)
        hs.append(ht)
    assert torch.equal(conv, c_end)
    # the same 32-bit steps in another grouping: a bf16 step of h at most
    assert (torch.cat(hs, 1).float() - h.float()).abs().max() <= 2 ** -7 * h.float().abs().max()
    assert torch.allclose(state, s_end, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("name", ["scan", "conv", "rms"])
def test_autograd_and_differences(name, gpu_lib):
    """The wrappers' gradients against central differences of their own forward in fp32, along one direction."""
    T, D, N, cu = 90, 48, 3, cu_dev([0, 30, 31, 90])
    if name == "scan":
        ins = [rnd(1, T, D), -rnd(1, T, D, seed=1).abs() * 0.2, rnd(N, D, seed=2)]
        fn = lambda x, g, s: gdn.gated_scan(x, g, s, cu_seqlens=cu)  # noqa: E731
    elif name == "conv":
        ins = [rnd(1, T, D), rnd(D, 3, seed=1), rnd(D, seed=2), rnd(N, 2, D, seed=3)]
        fn = lambda x, w, b, s: gdn.short_conv(x, w, b, s, cu_seqlens=cu, output_final_state=True)  # noqa: E731
    else:
        ins = [rnd(T, D), rnd(D, seed=1), rnd(T, D, seed=2)]
        fn = lambda x, w, r: gdn.rms_norm(x, w, r)  # noqa: E731
    leaves = [t.cuda().requires_grad_() for t in ins]
    outs = fn(*leaves)
    ups = [rnd(*o.shape, seed=30 + i).cuda() for i, o in enumerate(outs)]
    got = torch.autograd.grad(sum((o * u).sum() for o, u in zip(outs, ups)), leaves)
    eps = 1e-2
    for i, t in enumerate(ins):
        v = rnd(*t.shape, seed=60 + i)
        vals = []
        for sign in (1, -1):
            moved = [u.cuda() for u in ins]
            moved[i] = (t + sign * eps * v).cuda()
            vals.append([(o.double() * u.double()).sum().item() for o, u in zip(fn(*moved), ups)])
        diff = sum(a - b for a, b in zip(*vals)) / (2 * eps)
        want = (got[i].double() * v.cuda().double()).sum().item()
        # the difference is off by eps^2 / 6 of the third derivative along v, and by the outputs' rounding
        # (half steps of sums of ~1e4 terms) over eps: a thousandth of the gradient's length covers both
        size = (got[i].double().norm() * v.double().norm()).item()
        assert abs(diff - want) < 1e-3 * size, (name, i, diff, want, size)


def test_partial_gradients(gpu_lib):
    """Only one output used, only some inputs asking, gradients handed in expanded."""
    x, g = rnd(2, 70, 32).cuda().requires_grad_(), (-rnd(2, 70, 32, seed=1).abs()).cuda()
    _, fin = gdn.gated_scan(x, g)
    fin.sum().backward()
    want = ref.scan_bwd(x, g, None, torch.zeros(2, 70, 32), torch.ones(2, 32))["dx"]
    close(x.grad, want, "dx")
    w = rnd(32).cuda().requires_grad_()
    y = gdn.rms_norm(x.detach(), w)
    y.sum().backward()
    close(w.grad, ref.rms_bwd(x, w, torch.ones(2, 70, 32), None, 1e-6)["dweight"], "dweight")
    wc = rnd(32, 4, dtype=BF).cuda().requires_grad_()
    y, _ = gdn.short_conv(x.detach().to(BF), wc)
    y.sum().backward()
    assert wc.grad.dtype == BF and wc.grad.shape == (32, 4)
    res = x.detach().clone().requires_grad_()
    xx = x.detach().clone().requires_grad_()
    y, kept = gdn.rms_norm(xx, w.detach(), res)
    (kept.sum() + y.sum()).backward()
    assert torch.equal(xx.grad, res.grad)
    xx.grad.zero_()
    assert not torch.equal(xx.grad, res.grad)  # two gradients, not one buffer
