"""Cases for the matrix products around the gated delta rule: quantisation to e4m3, the product of e4m3 matrices
with scales for blocks of 128, the linear layer that trains through both, and the gated feed-forward block in bf16,
fp32 and e4m3.

run() computes them in plain torch operations, or with `own` through this repository's package. Quantised tensors
are e4m3 with fp32 scales, scale = max|x| / 448 over a row ("row"), over 128 columns of a row ("group") or over
128 x 128 values ("block"); a value stands for e4m3 x scale."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
E4M3_MAX = 448.0
GELU_C = math.sqrt(2 / math.pi)


def listed():
    return [
        # the heads' outputs of a 32K prompt (16 heads x 128), ahead of an output projection in 8 bits
        dict(name="quant_act", op="quant", M=32768, N=2048, dtype="bf16", quant="group", transpose=False),
        # a ragged batch's gradient, turned for the weight gradient's product: groups along the tokens
        dict(name="quant_turn_odd", op="quant", M=5003, N=1001, dtype="fp32", quant="group", transpose=True),
        # decoding a batch of 16 through the q, k, v projection: the weights are read once, latency counts
        dict(name="mm_step", op="mm", M=16, N=6144, K=2048, scales="block", out="bf16"),
        # the q, k, v projection of a 32K prompt
        dict(name="mm_prefill", op="mm", M=32768, N=6144, K=2048, scales="block", out="bf16"),
        # a weight gradient: 32K tokens contracted, groups along them in both operands
        dict(name="mm_wgrad", op="mm", M=6144, N=2048, K=32768, scales="group", out="fp32"),
        # odd sizes, one scale a row: a head of unusual width in an 8-bit model
        dict(name="mm_odd", op="mm", M=1003, N=777, K=1001, scales="row", out="fp32"),
        # training a projection in 8 bits: output, input gradient, weight gradient
        dict(name="linear_train", op="linear", M=8192, N=6144, K=2048, dtype="bf16"),
        # decoding one token through the gated block
        dict(name="ffn_step", op="ffn", mode="fwd", M=1, K=2048, F=5632, dtype="bf16", act="silu"),
        # training the gated block on 8K tokens: the largest
        dict(name="ffn_train", op="ffn", mode="train", M=8192, K=2048, F=8192, dtype="bf16", act="silu"),
        # a ragged fp32 training batch, odd widths
        dict(name="ffn_train_odd", op="ffn", mode="train", M=1037, K=515, F=999, dtype="fp32", act="gelu_tanh"),
        # decoding a batch of 16 through the gated block in 8 bits, output quantised for the product behind it
        dict(name="ffn8_step", op="ffn8", M=16, K=2048, F=8192, act="silu", quant="group"),
        # prefill of 16K tokens through the gated block in 8 bits
        dict(name="ffn8_prefill", op="ffn8", M=16384, K=2048, F=8192, act="silu", quant="group"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.4 or n < 64 else n // 64 * 64


def draw(rng):
    op = rng.choice(["quant", "mm", "mm", "linear", "ffn", "ffn", "ffn8"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "quant":
        N = _width(rng, 16, 16384)
        quant = rng.choice(["row", "group", "group", "block"])
        return dict(op=op, M=_log_int(rng, 1, max(1, min(65536, (1 << 26) // N))), N=N, dtype=dtype, quant=quant,
                    transpose=quant != "row" and rng.random() < 0.4)
    K = _width(rng, 16, 8192)
    N = _width(rng, 16, 8192)
    most = {"mm": 1 << 38, "linear": 1 << 36, "ffn": 1 << 36 if dtype == "bf16" else 1 << 34, "ffn8": 1 << 37}[op]
    M = _log_int(rng, 1, max(1, min(32768, most // (N * K))))
    if op == "mm":
        return dict(op=op, M=M, N=N, K=K, scales=rng.choice(["block", "block", "group", "row"]), out=rng.choice(["bf16", "fp32"]))
    if op == "linear":
        return dict(op=op, M=M, N=N, K=K, dtype=dtype)
    act = rng.choice(["silu", "silu", "gelu_tanh"])
    if op == "ffn":
        return dict(op=op, mode=rng.choice(["fwd", "train"]), M=M, K=K, F=N, dtype=dtype, act=act)
    return dict(op=op, M=M, K=K, F=N, act=act, quant=rng.choice(["group", "group", "none"]))


# --- inputs ------------------------------------------------------------------------------------------------------


def _tiles(t, rows, cols):
    """[R, rows, C, cols] of a matrix padded with zeros to whole tiles."""
    M, N = t.shape
    t = torch.nn.functional.pad(t, (0, -N % cols, 0, -M % rows))
    return t.reshape(t.shape[0] // rows, rows, t.shape[1] // cols, cols)


def _quantise(t, quant):
    """(e4m3 values, scales) of an fp32 matrix."""
    M, N = t.shape
    v = _tiles(t, 128 if quant == "block" else 1, N if quant == "row" else 128)
    amax = v.abs().amax((1, 3))
    # (a division by a number would be a product with its reciprocal, which moves values off ties of the 8-bit rounding)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, E4M3_MAX))
    q = (v / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.reshape(v.shape[0] * v.shape[1], -1)[:M, :N]
    return q.to(torch.float8_e4m3fn), scale


def _values(q, scale, quant):
    """What a quantised matrix stands for, in 32 bits."""
    v = _tiles(q.float(), 128 if quant == "block" else 1, q.shape[1] if quant == "row" else 128)
    v = v * scale[:, None, :, None]
    return v.reshape(v.shape[0] * v.shape[1], -1)[:q.shape[0], :q.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7 + 3)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * scale

    def stream(rows, cols):
        # a layer's inputs: a few channels are much larger than the others
        return normal(rows, cols) * (1 + 8 * (torch.rand(cols, device="cuda", generator=gen) < 0.01))

    s, op = dict(case=dict(case)), case["op"]
    M = case["M"]
    if op == "quant":
        s["x"] = stream(M, case["N"]).to(DT[case["dtype"]])
        return s
    K, N = case["K"], case.get("N", case.get("F"))
    if op == "mm":
        s["a"], s["a_scale"] = _quantise(stream(M, K), "row" if case["scales"] == "row" else "group")
        s["b"], s["b_scale"] = _quantise(normal(N, K, scale=K ** -0.5), case["scales"])
    elif op == "linear":
        dt = DT[case["dtype"]]
        s["x"], s["w"], s["dy"] = stream(M, K).to(dt), normal(N, K, scale=K ** -0.5).to(dt), normal(M, N).to(dt)
    elif op == "ffn":
        dt = DT[case["dtype"]]
        s["x"] = normal(M, K).to(dt)
        s["w_gate"], s["w_up"] = normal(N, K, scale=K ** -0.5).to(dt), normal(N, K, scale=K ** -0.5).to(dt)
        if case["mode"] == "train":
            s["d_h"] = normal(M, N).to(dt)
    else:
        s["x"], s["x_scale"] = _quantise(stream(M, K), "group")
        for k in ("gate", "up"):
            s["w_" + k], s[k + "_scale"] = _quantise(normal(N, K, scale=K ** -0.5), "block")
    return s


# --- plain forms -------------------------------------------------------------------------------------------------


def _turn(t):
    return t.t().contiguous()


def _plain_quant(s):
    case = s["case"]
    x = s["x"].float()
    q, scale = _quantise(_turn(x) if case["transpose"] else x, case["quant"])
    return {"q": q, "scale": scale}


def _plain_mm(s):
    kind = s["case"]["scales"]
    a = _values(s["a"], s["a_scale"], "row" if kind == "row" else "group")
    return {"y": (a @ _values(s["b"], s["b_scale"], kind).t()).to(DT[s["case"]["out"]])}


def _plain_linear(s):
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()

    def rounded(t, quant):
        return _values(*_quantise(t, quant), quant)

    y = rounded(x, "group") @ rounded(w, "block").t()
    dx = rounded(dy, "group") @ rounded(w, "block")
    dw = rounded(_turn(dy), "group") @ rounded(_turn(x), "group").t()
    return {"y": y.to(s["x"].dtype), "dx": dx.to(s["x"].dtype), "dw": dw.to(s["w"].dtype)}


def _slope(a, act):
    """(sigmoid's argument p, dp/da): both activations are a sigmoid(p)."""
    if act == "silu":
        return a, 1.0
    return 2 * GELU_C * (a + 0.044715 * a * a * a), 2 * GELU_C * (1 + 3 * 0.044715 * a * a)


def _plain_ffn(s):
    case = s["case"]
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    a, u = x @ wg.t(), x @ wu.t()
    p, dp = _slope(a, case["act"])
    sig = 1 / (1 + torch.exp(-p))
    out = {"h": (a * sig * u).to(s["x"].dtype)}
    if case["mode"] == "train":
        dh = s["d_h"].float()
        da, du = dh * u * (sig + a * sig * (1 - sig) * dp), dh * (a * sig)
        out["dx"] = (da @ wg + du @ wu).to(s["x"].dtype)
        out["dw_gate"] = (da.t() @ x).to(s["w_gate"].dtype)
        out["dw_up"] = (du.t() @ x).to(s["w_up"].dtype)
    return out


def _plain_ffn8(s):
    case = s["case"]
    x = _values(s["x"], s["x_scale"], "group")
    a = x @ _values(s["w_gate"], s["gate_scale"], "block").t()
    u = x @ _values(s["w_up"], s["up_scale"], "block").t()
    h = a / (1 + torch.exp(-_slope(a, case["act"])[0])) * u
    if case["quant"] == "none":
        return {"h": h.to(torch.bfloat16)}
    q, scale = _quantise(h, "group")
    return {"h": q, "scale": scale}


# --- the framework's calls ---------------------------------------------------------------------------------------


def _own(s):
    import gated_deltanet_chunked_04_amd as gdn

    case = s["case"]
    op = case["op"]
    if op == "quant":
        q, scale = gdn.gdn_quant_e4m3(s["x"], quant=case["quant"], transpose=case["transpose"])
        return {"q": q, "scale": scale}
    if op == "mm":
        return {"y": gdn.gdn_matmul_e4m3(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DT[case["out"]])}
    if op == "linear":
        x, w = s["x"].detach().requires_grad_(), s["w"].detach().requires_grad_()
        y = gdn.linear_e4m3(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    if op == "ffn":
        x, wg, wu, act = s["x"], s["w_gate"], s["w_up"], case["act"]
        if case["mode"] == "fwd":
            return {"h": gdn.gdn_gated_ffn_fwd(x, wg, wu, activation=act)}
        pre = gdn.gdn_gated_ffn_pre(x, wg)
        h = gdn.gdn_gated_ffn_fwd(x, wg, wu, activation=act, pre=pre)
        return {"h": h, **gdn.gdn_gated_ffn_bwd(x, wg, wu, s["d_h"], activation=act, pre=pre)}
    h, scale = gdn.gdn_gated_ffn_e4m3(s["x"], s["x_scale"], s["w_gate"], s["gate_scale"], s["w_up"], s["up_scale"],
                                      activation=case["act"], quant=None if case["quant"] == "none" else "group")
    return {"h": h} if scale is None else {"h": h, "scale": scale}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "mm": _plain_mm, "linear": _plain_linear, "ffn": _plain_ffn, "ffn8": _plain_ffn8}[state["case"]["op"]](state)


def _scales(rows, cols, quant):
    """Bytes of a quantised matrix's scales."""
    return 4 * (-(-rows // 128) if quant == "block" else rows) * (1 if quant == "row" else -(-cols // 128))


def work(case):
    op, M = case["op"], case["M"]
    if op == "quant":
        N = case["N"]
        r, c = (N, M) if case["transpose"] else (M, N)
        return {"bytes": M * N * (SIZE[case["dtype"]] + 1) + _scales(r, c, case["quant"]), "flops": 3 * M * N}
    K, N = case["K"], case.get("N", case.get("F"))
    if op == "mm":
        kind = case["scales"]
        return {"bytes": M * K + N * K + _scales(M, K, "row" if kind == "row" else "group") + _scales(N, K, kind) + M * N * SIZE[case["out"]],
                "flops": 2 * M * N * K}
    if op == "linear":
        # x, w and dy read, y, dx and dw written
        return {"bytes": SIZE[case["dtype"]] * 2 * (M * K + N * K + M * N), "flops": 6 * M * N * K}
    if op == "ffn":
        e = SIZE[case["dtype"]]
        fwd = e * (M * K + 2 * N * K + M * N)
        if case["mode"] == "fwd":
            return {"bytes": fwd, "flops": 4 * M * N * K}
        # what the two directions read in common is counted for each: the gradient comes long after the forward
        return {"bytes": fwd + e * (2 * M * K + 4 * N * K + M * N), "flops": 12 * M * N * K}
    out = 2 * M * N if case["quant"] == "none" else M * N + _scales(M, N, "group")
    return {"bytes": M * K + 2 * N * K + _scales(M, K, "group") + 2 * _scales(N, K, "block") + out, "flops": 4 * M * N * K}


# --- 64 bits, from the definitions -------------------------------------------------------------------------------


def _spread(scale, quant, shape):
    """A scale for every value of a matrix, in 64 bits."""
    s = scale.double()
    if quant == "row":
        return s.expand(shape)
    if quant == "block":
        s = s.repeat_interleave(128, 0)
    return s.repeat_interleave(128, 1)[:shape[0], :shape[1]]


def _exact_quant(x, quant):
    """(x / scale before its rounding to 8 bits, scale), the scale rounded to the 32 bits that hold it."""
    rows = x.split(128, 0) if quant == "block" else [x]
    strips = []
    for r in rows:
        parts = [r] if quant == "row" else r.split(128, 1)
        strips.append(torch.stack([p.abs().max().reshape(1) if quant == "block" else p.abs().amax(1) for p in parts], 1))
    scale = (torch.cat(strips) / E4M3_MAX).float().double()
    scale = scale.masked_fill(scale == 0, 1.0)
    return x / _spread(scale, quant, x.shape), scale


def _held(x, quant):
    """The values that x stands for after quantisation."""
    q, scale = _exact_quant(x, quant)
    return q.float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double() * _spread(scale, quant, x.shape)


def _exact_act(a, act):
    """(activation, its derivative)."""
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    t = torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * a ** 2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        x = s["x"].double()
        q, scale = _exact_quant(x.t() if case["transpose"] else x, case["quant"])
        return {"q": q, "scale": scale}
    if op == "mm":
        a = s["a"].double() * _spread(s["a_scale"], "row" if case["scales"] == "row" else "group", s["a"].shape)
        b = s["b"].double() * _spread(s["b_scale"], case["scales"], s["b"].shape)
        return {"y": torch.mm(a, b.t())}
    if op == "linear":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        wq = _held(w, "block")
        return {"y": torch.mm(_held(x, "group"), wq.t()), "dx": torch.mm(_held(dy, "group"), wq),
                "dw": torch.mm(_held(dy.t(), "group"), _held(x.t(), "group").t())}
    if op == "ffn":
        x, wg, wu = (s[k].double() for k in ("x", "w_gate", "w_up"))
        a, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        f, df = _exact_act(a, case["act"])
        out = {"h": f * u}
        if case["mode"] == "train":
            dh = s["d_h"].double()
            du = dh * f
            da = dh * u * df
            out.update(dx=torch.mm(da, wg).addmm_(du, wu), dw_gate=torch.mm(da.t(), x), dw_up=torch.mm(du.t(), x))
        return out
    x = s["x"].double() * _spread(s["x_scale"], "group", s["x"].shape)
    a = torch.mm(x, (s["w_gate"].double() * _spread(s["gate_scale"], "block", s["w_gate"].shape)).t())
    u = torch.mm(x, (s["w_up"].double() * _spread(s["up_scale"], "block", s["w_up"].shape)).t())
    h = _exact_act(a, case["act"])[0] * u
    if case["quant"] == "none":
        return {"h": h}
    q, scale = _exact_quant(h, "group")
    return {"h": q, "scale": scale}
