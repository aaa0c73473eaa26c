"""The readme's fenced Python lines on the products of a layer, run as they stand."""
import os
import re

import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_products_lines_run(gpu_lib):
    with open(os.path.join(ROOT, "README.md")) as f:
        serve, train = re.findall(r"```python\n(.*?)```", f.read().split("### The products of a layer")[1], re.S)
    gen = torch.Generator(device="cuda").manual_seed(0)

    def r(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)

    B, T, D, N, F = 2, 5, 256, 384, 320
    ws = dict(w=r(N, D, scale=D ** -0.5), w_gate=r(F, D, scale=D ** -0.5), w_up=r(F, D, scale=D ** -0.5), w_down=r(D, F, scale=F ** -0.5))
    ns = dict(gdn=gdn, torch=torch, x=r(B, T, D), w_norm=torch.ones(D, device="cuda").to(torch.bfloat16), stream=r(B, T, D), **ws)
    exec(serve, ns)
    assert ns["qkv"].shape == (B, T, N) and ns["x"].shape == (B, T, D) and ns["h8"].dtype == torch.float8_e4m3fn
    # the same in fp32: each 8-bit rounding is off by at most 2^-4 of its value; two of them meet in qkv, six in x
    s = ns["stream"].float()
    n = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6)
    f = {k: t.float() for k, t in ws.items()}
    qkv = n @ f["w"].t()
    x = (torch.nn.functional.silu(n @ f["w_gate"].t()) * (n @ f["w_up"].t())) @ f["w_down"].t()
    assert (ns["qkv"].float() - qkv).norm() < 2 * 2.0 ** -4 * qkv.norm()
    assert (ns["x"].float() - x).norm() < 6 * 2.0 ** -4 * x.norm()

    ns = dict(gdn=gdn, x=r(B, T, D).requires_grad_(), w=r(D, D, scale=D ** -0.5).requires_grad_(),
              w_gate=ws["w_gate"].requires_grad_(), w_up=ws["w_up"].requires_grad_())
    exec(train, ns)
    assert ns["h"].shape == (B, T, F)
    assert all(torch.isfinite(ns[k].grad).all() and ns[k].grad.abs().sum() > 0 for k in ("x", "w", "w_gate", "w_up"))
