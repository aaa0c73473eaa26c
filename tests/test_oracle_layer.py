"""The plain 64-bit forms of the layer operators (oracle/layer.py) pinned on the CPU: hand-worked values, torch's
automatic differentiation and central differences of a literal forward, splitting a sequence in two."""
import math

import pytest
import torch

from oracle import layer as ref

torch.manual_seed(0)
CU = [0, 0, 4, 5, 5, 12]


def rnd(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


def test_scan_by_hand():
    x = torch.tensor([[[1.0], [2.0], [4.0]]])
    g = torch.tensor([[[math.log(0.5)], [math.log(0.25)], [float("-inf")]]]).double()
    (h, _), (fin, _) = ref.scan_fwd(x, g, torch.tensor([[8.0]]))
    assert torch.allclose(h.flatten(), torch.tensor([5.0, 3.25, 4.0]).double(), atol=1e-12)
    assert fin.item() == 4.0


def test_conv_by_hand():
    x = torch.tensor([[[1.0], [2.0], [3.0]]])
    (y, _), fin = ref.conv_fwd(x, torch.tensor([[10.0, 1.0]]), torch.tensor([0.5]), torch.tensor([[[7.0]]]), False)
    assert y.flatten().tolist() == [71.5, 12.5, 23.5]
    assert fin.item() == 3.0
    (y, _), _ = ref.conv_fwd(x, torch.tensor([[0.0, 1.0]]), None, None, True)
    assert torch.allclose(y.flatten(), torch.tensor([1.0, 2.0, 3.0]).double() / (1 + torch.exp(-torch.tensor([1.0, 2.0, 3.0]).double())))


def test_rms_by_hand():
    y, _, r = ref.rms_fwd(torch.tensor([[2.0, 3.0]]), torch.tensor([[1.0, 1.0]]), torch.tensor([1.0, 2.0]), 0.0)
    s = math.sqrt(12.5)
    assert r.tolist() == [[3.0, 4.0]]
    assert torch.allclose(y, torch.tensor([[3 / s, 8 / s]]).double())


def _loss(out, ups):
    return sum((o * u).sum() for o, u in zip(out, ups) if u is not None)


def _literal_scan(x, g, s0, cu):
    D = x.shape[2]
    h, fin = [], []
    for n, (p, q) in enumerate(ref.sequences(1, x.shape[1], cu)):
        c = s0[n]
        for t in range(p, q):
            c = g[0, t].exp() * c + x[0, t]
            h.append(c)
        fin.append(c)
    return torch.stack(h).reshape(1, -1, D), torch.stack(fin)


def _literal_conv(x, w, b, s0, cu):
    W = w.shape[1]
    y, fin = [], []
    for n, (p, q) in enumerate(ref.sequences(1, x.shape[1], cu)):
        e = [s0[n, i] for i in range(W - 1)] + [x[0, t] for t in range(p, q)]
        for t in range(q - p):
            z = b + sum(w[:, j] * e[t + j] for j in range(W))
            y.append(z / (1 + torch.exp(-z)))
        fin.append(torch.stack(e[len(e) - W + 1:]))
    return torch.stack(y).unsqueeze(0), torch.stack(fin)


def _literal_rms(r, w):
    return (r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-3) * w, r)


def _cases():
    T, D, N = CU[-1], 3, len(CU) - 1
    scan_in = [rnd(1, T, D), -rnd(1, T, D, seed=1).abs() * 0.5, rnd(N, D, seed=2)]
    scan_up = [rnd(1, T, D, seed=3), rnd(N, D, seed=4)]
    bw = ref.scan_bwd(*scan_in, *scan_up, CU)
    yield "scan", lambda *i: _literal_scan(*i, CU), scan_in, scan_up, [bw["dx"], bw["dg"], bw["d_initial_state"]]
    for W in (2, 3, 4):
        conv_in = [rnd(1, T, D), rnd(D, W, seed=1), rnd(D, seed=2), rnd(N, W - 1, D, seed=3)]
        conv_up = [rnd(1, T, D, seed=4), rnd(N, W - 1, D, seed=5)]
        bw = ref.conv_bwd(*conv_in, *conv_up, True, CU)
        yield (f"conv{W}", lambda *i: _literal_conv(*i, CU), conv_in, conv_up,
               [bw["dx"], bw["dweight"], bw["dbias"], bw["d_initial_state"]])
    rms_in = [rnd(5, 7), rnd(7, seed=1)]
    rms_up = [rnd(5, 7, seed=2), rnd(5, 7, seed=3)]
    bw = ref.rms_bwd(*rms_in, *rms_up, 1e-3)
    yield "rms", _literal_rms, rms_in, rms_up, [bw["dx"], bw["dweight"]]


@pytest.mark.parametrize("name,fn,ins,ups,want", list(_cases()), ids=[c[0] for c in _cases()])
def test_gradients(name, fn, ins, ups, want):
    leaves = [t.clone().requires_grad_() for t in ins]
    grads = torch.autograd.grad(_loss(fn(*leaves), ups), leaves)
    for got, (value, _) in zip(grads, want):
        assert torch.allclose(got, value, rtol=1e-11, atol=1e-12), name
    eps = 1e-6
    for i, t in enumerate(ins):
        v = rnd(*t.shape, seed=40 + i)
        up, down = [list(ins), list(ins)]
        up[i], down[i] = t + eps * v, t - eps * v
        diff = (_loss(fn(*up), ups) - _loss(fn(*down), ups)) / (2 * eps)
        # differences of a smooth function: off by eps^2 of the third derivative and 2^-53 / eps of the value
        assert abs(diff - (want[i][0] * v).sum()) < 1e-7 * (1 + abs(diff)), (name, i)


def test_forward_matches_literal():
    T, D, N = CU[-1], 3, len(CU) - 1
    x, g, s0 = rnd(1, T, D), -rnd(1, T, D, seed=1).abs(), rnd(N, D, seed=2)
    (h, _), (fin, _) = ref.scan_fwd(x, g, s0, CU)
    h2, fin2 = _literal_scan(x, g, s0, CU)
    assert torch.allclose(h, h2) and torch.allclose(fin, fin2)
    w, b, c0 = rnd(D, 4), rnd(D, seed=3), rnd(N, 3, D, seed=4)
    (y, _), fin = ref.conv_fwd(x, w, b, c0, True, CU)
    y2, fin2 = _literal_conv(x, w, b, c0, CU)
    assert torch.allclose(y, y2) and torch.equal(fin, fin2)


def test_bounds_hold_in_32_bits():
    """The bounds are bounds: the literal forms in 32 bits stay inside them."""
    x, g, s0 = rnd(1, 300, 5).float(), (-rnd(1, 300, 5, seed=1).abs() * 0.05).float(), rnd(1, 5, seed=2).float()
    (h, e), _ = ref.scan_fwd(x, g, s0)
    h32, _ = _literal_scan(x, g, s0, [0, 300])
    assert ((h32.double() - h).abs() <= e).all()
    w, b, c0 = rnd(5, 4).float(), rnd(5, seed=3).float(), rnd(1, 3, 5, seed=4).float()
    (y, e), _ = ref.conv_fwd(x, w, b, c0, True)
    y32, _ = _literal_conv(x, w, b, c0, [0, 300])
    assert ((y32.double() - y).abs() <= e).all()
