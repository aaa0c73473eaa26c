"""The plain 64-bit forms of the layer's products (oracle/products.py) pinned on the CPU: hand-worked values, torch's
8-bit type, its automatic differentiation and central differences."""
import math

import pytest
import torch

from oracle import products as ref


def rnd(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


def test_scales_by_hand():
    x = torch.zeros(130, 129)
    x[0, 0], x[3, 127], x[2, 128], x[129, 5] = 448.0, -896.0, 1.0, 3.5
    assert ref.quant_scale(x, "row").flatten()[[0, 1, 2, 3, 129]].tolist() == [1.0, 1.0, torch.tensor(1.0).div(448).item(), 2.0, 3.5 / 448]
    g = ref.quant_scale(x, "group")
    assert g.shape == (130, 2) and g[0].tolist() == [1.0, 1.0] and g[2].tolist() == [1.0, torch.tensor(1.0).div(448).item()]
    b = ref.quant_scale(x, "block")
    assert b.shape == (2, 2) and b.flatten().tolist() == [2.0, torch.tensor(1.0).div(448).item(), 3.5 / 448, 1.0]
    assert ref.quant_scale(torch.full((1, 1), 1e-40), "row").item() == 2.0 ** -126


def test_nearest_is_the_types():
    """Against torch's conversion from fp32, for values that are no ties in fp32."""
    v = torch.cat([rnd(20000).mul(60), rnd(2000).mul(0.02), torch.arange(-448, 449).double()])
    near, gap = ref.e4m3_nearest(v)
    want = v.float().to(torch.float8_e4m3fn).double()
    far = gap > 2.0 ** -22
    assert torch.equal(near[far], want[far])
    tie = torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10], dtype=torch.float64)  # to even: 16, 20, 0, 2^-8
    near, gap = ref.e4m3_nearest(tie)
    assert near.tolist() == [16.0, 20.0, 0.0, 2.0 ** -8] and gap.tolist() == [0.0] * 4


@pytest.mark.parametrize("kind", ["row", "group", "block"])
def test_matmul_by_hand(kind):
    a, b = torch.ones(2, 130), torch.ones(3, 130)
    sa = torch.tensor([[2.0], [3.0]]) if kind == "row" else torch.tensor([[2.0, 5.0], [3.0, 7.0]])
    sb = {"row": torch.tensor([[1.0], [10.0], [100.0]]), "group": torch.tensor([[1.0, 2], [10, 20], [100, 200]]),
          "block": torch.tensor([[1.0, 10.0]])}[kind]
    y, s, _ = ref.matmul(a, sa, b, sb, kind)
    want = {"row": [[260.0, 2600, 26000], [390, 3900, 39000]],
            "group": [[256 + 20.0, 2760, 27600], [384 + 28.0, 4120, 41200]],
            "block": [[256 + 100.0] * 3, [384 + 140.0] * 3]}[kind]
    assert y.tolist() == want and torch.equal(s, y)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn(act):
    M, K, F = 5, 7, 6
    x, wg, wu, d = rnd(M, K), rnd(F, K, seed=1), rnd(F, K, seed=2), rnd(M, F, seed=3)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    a, u = leaves[0] @ leaves[1].t(), leaves[0] @ leaves[2].t()
    f = torch.nn.functional.silu(a) if act == "silu" else torch.nn.functional.gelu(a, approximate="tanh")
    (h, bound), _, _ = ref.ffn_fwd(x, wg, wu, act)
    assert torch.allclose(h, f * u, rtol=1e-13, atol=1e-14) and (bound > 0).all()
    want = torch.autograd.grad((f * u * d).sum(), leaves)
    got = ref.ffn_bwd(x, wg, wu, d, act, torch.float32)
    for k, w, at in zip(("dx", "dw_gate", "dw_up"), want, (0, 1, 2)):
        assert torch.allclose(got[k][0], w, rtol=1e-12, atol=1e-13), k
        # and against central differences along a direction: the error is of the step's square
        v = rnd(*w.shape, seed=9)
        step = 1e-5
        ends = []
        for sgn in (1, -1):
            ins = [x, wg, wu]
            ins[at] = ins[at] + sgn * step * v
            ends.append((ref.ffn_fwd(*ins, act)[0][0] * d).sum())
        assert math.isclose((ends[0] - ends[1]).item() / (2 * step), (got[k][0] * v).sum().item(), rel_tol=1e-6, abs_tol=1e-6), k
    pre = torch.stack([x @ wg.t(), x @ wu.t()])
    kept = ref.ffn_bwd(x, wg, wu, d, act, torch.float32, pre)
    assert all(torch.equal(kept[k][0], got[k][0]) and (kept[k][1] <= got[k][1]).all() for k in got)
