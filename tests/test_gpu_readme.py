"""The Python lines of the readme's section on use, run as they stand."""
import os

import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def blocks():
    """The indented blocks behind "From Python:"."""
    with open(os.path.join(ROOT, "README.md")) as f:
        lines = f.read().split("From Python:")[1].split("\n")
    out, cur = [], []
    for line in lines + [""]:
        if line.startswith("    "):
            cur.append(line[4:])
        elif cur:
            out.append("\n".join(cur))
            cur = []
    return out


def test_python_lines_run(gpu_lib):
    gen = torch.Generator(device="cuda").manual_seed(0)

    def r(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=gen).to(dtype)

    N, T, H, K, V, D = 2, 40, 2, 64, 64, 192
    f32 = torch.float32
    unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype)  # noqa: E731
    rule, step, layer, decode = blocks()
    ns = dict(gdn=gdn, K=K, q=unit(r(1, T, H, K)), k=unit(r(1, T, H, K)), v=r(1, T, H, V), g=-r(1, T, H, dtype=f32).abs(),
              beta=torch.sigmoid(r(1, T, H, dtype=f32)), s0=r(N, H, V, K, dtype=f32),
              cu=torch.tensor([0, 15, T], dtype=torch.int32).cuda())
    exec(rule, ns)
    assert ns["o"].shape == (1, T, H, V) and ns["final_state"].shape == (N, H, V, K)
    ns.update(q_t=unit(r(N, 1, H, K)), k_t=unit(r(N, 1, H, K)), v_t=r(N, 1, H, V), g_t=-r(N, 1, H, dtype=f32).abs(),
              beta_t=torch.sigmoid(r(N, 1, H, dtype=f32)))
    exec(step, ns)
    assert ns["o_t"].shape == (N, 1, H, V) and ns["state"] is ns["final_state"]

    ns = dict(gdn=gdn, x=r(N, T, D), w=r(D), stream=r(N, T, D), w_conv=r(D, 4), conv_state=None, g=-r(N, T, D, dtype=f32).abs(), state=None)
    exec(layer, ns)
    for name in ("y", "stream", "qkv", "h"):
        assert ns[name].shape == (N, T, D), name
    assert ns["y8"].dtype == torch.float8_e4m3fn and ns["scale"].shape == (N, T, 2)

    ns.update(x_t=r(N, 1, D), stream_t=r(N, 1, D), g_t=-r(N, 1, D, dtype=f32).abs())
    held = {k: ns[k] for k in ("stream_t", "conv_state", "state")}
    before = {k: t.clone() for k, t in held.items()}
    exec(decode, ns)
    for k, t in held.items():  # in place
        assert ns[k] is t and not torch.equal(t, before[k]), k
    want = before["state"] * ns["g_t"][:, 0].exp() + ns["x_t"][:, 0].float()
    assert torch.allclose(held["state"], want, rtol=1e-5, atol=1e-5)
    assert torch.equal(held["conv_state"][:, :-1], before["conv_state"][:, 1:]) and torch.equal(held["conv_state"][:, -1:], ns["y_t"])
    for name in ("y_t", "qkv_t", "h_t"):
        assert ns[name].shape == (N, 1, D) and torch.isfinite(ns[name]).all(), name
