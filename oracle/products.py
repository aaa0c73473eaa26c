"""Plain 64-bit forms of the layer's products (quantisation to e4m3, the product of e4m3 matrices, the gated
feed-forward block and its gradients), on the CPU, and how far a computation in 32 bits may be from them.

Test infrastructure only. Every function takes the tensors the kernels take and upcasts them exactly. The second
value of a pair is an absolute bound, element by element, on the error before the result is rounded to the output's
type; U is half a step of fp32. A matrix instruction may cut where an addition would round, so an addition counts 2 U."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value
C = 2 * math.sqrt(2 / math.pi)


def f64(t):
    return None if t is None else t.detach().cpu().double()


def spread(scale, kind, rows, cols):
    """A quantised matrix's scales, one for every value."""
    s = f64(scale)
    if kind == "row":
        return s.reshape(rows, 1).expand(rows, cols)
    s = s.reshape(-1, s.shape[-1])
    if kind == "block":
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def values(q, scale, kind):
    """What a quantised matrix stands for (leading dimensions flattened)."""
    q = f64(q)
    q = q.reshape(-1, q.shape[-1])
    return q * spread(scale, kind, *q.shape)


def quant_scale(x, kind):
    """The fp32 scales of a matrix: the largest absolute value / 448 rounded once, 2^-126 at least, 1 for zeros."""
    x = x.detach().cpu().float()
    x = x.reshape(-1, x.shape[-1])
    rows, cols = x.shape
    R, G = (128 if kind == "block" else 1), (cols if kind == "row" else 128)
    p = torch.nn.functional.pad(x.abs(), (0, -cols % G, 0, -rows % R))
    amax = p.reshape(p.shape[0] // R, R, p.shape[1] // G, G).amax((1, 3))
    s = (amax / torch.full_like(amax, 448.0)).clamp(min=2.0 ** -126)
    return torch.where(amax == 0, torch.ones_like(s), s)


def e4m3_nearest(v):
    """64-bit values to the nearest e4m3 value (half way: the even one), and how far each lies from half way between
    two of them, relative to the value."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    n = a / step
    near = torch.round(n)  # half to even
    gap = ((n - torch.floor(n)) - 0.5).abs() * step / a.clamp(min=2.0 ** -40)
    return torch.sign(v) * (near * step).clamp(max=448.0), gap


def matmul(a, a_scale, b, b_scale, kind):
    """(y, sum of the absolute products, bound of fp32 arithmetic): a block's 128 products are added in some order, its
    sum is scaled (a product of scales, a fused product) and the blocks are added."""
    akind = "row" if kind == "row" else "group"
    x, w = values(a, a_scale, akind), values(b, b_scale, kind)
    y, s = x @ w.t(), x.abs() @ w.abs().t()
    K = x.shape[1]
    return y, s, (2 * min(K, 128) + 2 * -(-K // 128) + 4) * U * s if kind != "row" else (2 * K + 4) * U * s


# the 8-bit matrix instruction cuts the products of a group of eight 2^-13 below the largest: 8 x 2^-13 of it at most
CUT = 2.0 ** -10


def _act(a, act):
    """(f, f', p, p', s) of f = a s, s = sigmoid(p)."""
    p = a if act == "silu" else C * (a + 0.044715 * a ** 3)
    dp = torch.ones_like(a) if act == "silu" else C * (1 + 3 * 0.044715 * a ** 2)
    s = torch.sigmoid(p)
    return a * s, s + a * s * (1 - s) * dp, p, dp, s


def ffn_fwd(x, wg, wu, act, cut=0.0):
    """((h, bound), (gate, bound), (up, bound)); cut: of the sums of absolute products, beside fp32's."""
    x, wg, wu = f64(x), f64(wg), f64(wu)
    K = x.shape[-1]
    a, u = x @ wg.t(), x @ wu.t()
    ea, eu = ((2 * K * U + cut) * (x.abs() @ w.abs().t()) for w in (wg, wu))
    f, _, p, _, s = _act(a, act)
    # exp is off by (2 + |p|) half steps and its argument by 4 |p|, the sigmoid by (1 - s) of that and 4 more; |f'| < 1.2
    ef = 1.2 * ea + (6 + (1 - s) * (4 + 6 * p.abs())) * U * f.abs()
    return (f * u, ef * u.abs() + (f.abs() + ef) * eu + U * (f * u).abs()), (a, ea), (u, eu)


def ffn_bwd(x, wg, wu, d_h, act, dtype, pre=None):
    """dict of (value, bound) for dx, dw_gate, dw_up. pre: gate and up as the backward was given them, or None. The
    gradients of gate and up are rounded to dtype."""
    x, wg, wu, d = f64(x), f64(wg), f64(wu), f64(d_h)
    _, (a, ea), (u, eu) = ffn_fwd(x, wg, wu, act)
    if pre is not None:
        (a, u), ea, eu = f64(pre), torch.zeros_like(ea), torch.zeros_like(eu)
    f, df, p, dp, s = _act(a, act)
    one = (8 + (1 - s) * (4 + 6 * p.abs())) * U
    ef = 1.2 * ea + one * f.abs()
    slope = a.abs() * s * dp.abs()
    # |f''| < 1; 1 - s is off by U itself
    edf = ea + (one + 4 * U) * (s + slope * (1 - s)) + 2 * U * slope
    da, du = d * u * df, d * f
    eda = d.abs() * (u.abs() * edf + eu * (df.abs() + edf)) + 2 * U * da.abs()
    edu = d.abs() * ef + U * du.abs()
    eda = eda + HALF[dtype] * (da.abs() + eda)
    edu = edu + HALF[dtype] * (du.abs() + edu)

    def product(terms, n):
        v = sum(p @ q for p, _, q in terms)
        e = sum((ep + 2 * n * U * (p.abs() + ep)) @ q.abs() for p, ep, q in terms)
        return v, e

    F, M = wg.shape[0], x.shape[0]
    return dict(dx=product([(da, eda, wg), (du, edu, wu)], 2 * F), dw_gate=product([(da.t(), eda.t(), x)], M),
                dw_up=product([(du.t(), edu.t(), x)], M))
