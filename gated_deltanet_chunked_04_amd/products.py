"""The products of a layer: quantisation to e4m3, the product of e4m3 matrices, and the gated feed-forward block.

Like the rest of the package these functions carry the C ABI's names (include/gdn.h) and only marshal
tensors into it; every step of the computation runs in the HIP library. Tensors are contiguous, on one
device; work runs on that device's current stream. Quantised tensors are torch.float8_e4m3fn beside fp32
scales: a value stands for e4m3 x scale.

  gdn_quant_e4m3                to e4m3, a scale per row, per 128 columns or per 128 x 128; also transposed
  gdn_matmul_e4m3               a b^T of two quantised matrices
  gdn_gated_ffn_fwd / _bwd      h = act(x w_gate^T) (x w_up^T), and its gradients
  gdn_gated_ffn_pre(x, w_gate)  the buffer that carries gate and up from the forward to the backward
  gdn_gated_ffn_e4m3            the block on quantised x and weights, h quantised or not
  linear_e4m3, gated_ffn        with autograd
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from ._abi import (GDN_ACT_GELU_TANH, GDN_ACT_SILU, GDN_DTYPE_BF16, GDN_FLAG_EXACT_SUMS, GDN_FLAG_GRAD_PAIRS, GDN_OUT_E4M3, GDN_OUT_SAME, GDN_SCALE_BLOCK,
                   GDN_SCALE_GROUP, GDN_SCALE_ROW, GdnFfnDesc, GdnMatmulDesc, GdnQuantDesc, load_library)
from .layer import _DTYPES, _bytes, _dense, _dtype, _like, _out, _run, _scratch

_SCALES = {"row": GDN_SCALE_ROW, "group": GDN_SCALE_GROUP, "block": GDN_SCALE_BLOCK}
_GATES = {"silu": GDN_ACT_SILU, "gelu_tanh": GDN_ACT_GELU_TANH}
E4M3 = torch.float8_e4m3fn


def _matrix(name, t):
    """(rows, columns) of a contiguous device tensor [..., columns]."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous device tensor [..., columns]")
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else t.shape[:-1].numel()
    return rows, cols


def _weight(name, t, cols, dtype, device):
    """Rows of a weight matrix [rows, cols]."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a tensor of 2 dimensions")
    _like(name, t, (t.shape[0], cols), dtype, device)
    return t.shape[0]


def _blocks(n) -> int:
    return -(-n // 128)


def _scales_of(name, t, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous fp32 scales on {device}")


# ---- quantisation -------------------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _quant_desc(rows, cols, dtype, scales, transpose):
    return ctypes.byref(GdnQuantDesc(rows, cols, dtype, scales, transpose))


def gdn_quant_e4m3(x, *, quant="group", transpose=False, q=None, scale=None):
    """x [..., D], bf16 or fp32, to e4m3. Returns (q, scale): scale = max|x| / 448 over the values that share it.

    quant 'row': scale [..., 1]; 'group': a scale per 128 columns, [..., ceil(D/128)]; 'block': x is taken as
    [rows, D], a scale per 128 x 128 values, [ceil(rows/128), ceil(D/128)]. transpose (not with 'row') gives
    q [D, rows], with the scales of that matrix: 'group' [D, ceil(rows/128)], 'block' [ceil(D/128), ceil(rows/128)]."""
    kind = _SCALES.get(quant)
    if kind is None:
        raise ValueError("quant: expected 'row', 'group' or 'block'")
    rows, cols = _matrix("x", x)
    dtype = _dtype(x)
    if transpose:
        if quant == "row":
            raise ValueError("transpose: not with quant='row'")
        qshape = (cols, rows)
        sshape = (cols if quant == "group" else _blocks(cols), _blocks(rows))
    else:
        qshape = tuple(x.shape)
        sshape = (_blocks(rows), _blocks(cols)) if quant == "block" else (*x.shape[:-1], 1 if quant == "row" else _blocks(cols))
    q, pq = _out("q", q, x, qshape, E4M3, x.device)
    scale, ps = _out("scale", scale, x, sshape, torch.float32, x.device)
    _run(load_library().gdn_quant_e4m3, x.device, _quant_desc(rows, cols, dtype, kind, 1 if transpose else 0), x.data_ptr(), pq, ps)
    return q, scale


# ---- product of e4m3 matrices -------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _matmul_plan(M, N, K, out_dtype, scales, exact):
    """(descriptor, its workspace size)."""
    desc = GdnMatmulDesc(M, N, K, out_dtype, scales, GDN_FLAG_EXACT_SUMS if exact else 0)
    return ctypes.byref(desc), _bytes("gdn_matmul_e4m3_workspace_size", desc)


def gdn_matmul_e4m3(a, a_scale, b, b_scale, *, out_dtype=torch.bfloat16, exact=False, y=None, workspace=None):
    """y = a b^T of quantised a [..., K] and b [N, K]: [..., N] in out_dtype, bf16 or fp32.

    b_scale is [ceil(N/128), ceil(K/128)] or [N, ceil(K/128)] with a_scale [..., ceil(K/128)], or [N, 1] with
    a_scale [..., 1] (what gdn_quant_e4m3 and gdn_rmsnorm_fwd give). With fp32 the products and sums are fp32's;
    bf16 takes the 8-bit matrix instruction, whose sums of eight products drop what lies about 2^-13 below the
    largest of them (include/gdn.h): twice as fast, and for activations and weights far below bf16's rounding. Where
    large products cancel, exact=True gives fp32's products and sums, rounded to bf16 at the end."""
    M, K = _matrix("a", a)
    if a.dtype != E4M3:
        raise TypeError("a: expected torch.float8_e4m3fn")
    out = _DTYPES.get(out_dtype)
    if out is None:
        raise TypeError("out_dtype: expected torch.bfloat16 or torch.float32")
    dev = a.device
    N = _weight("b", b, K, E4M3, dev)
    _scales_of("a_scale", a_scale, dev)
    _scales_of("b_scale", b_scale, dev)
    lead, kb = a.shape[:-1], _blocks(K)
    ashape, bshape = tuple(a_scale.shape), tuple(b_scale.shape)
    if ashape == (*lead, kb) and bshape == (_blocks(N), kb):
        kind = GDN_SCALE_BLOCK
    elif ashape == (*lead, kb) and bshape == (N, kb):
        kind = GDN_SCALE_GROUP
    elif ashape == (*lead, 1) and bshape == (N, 1):
        kind = GDN_SCALE_ROW
    else:
        raise ValueError(f"scales {ashape} and {bshape} fit no kind: a [..., {kb}] with b [{_blocks(N)}, {kb}] or [{N}, {kb}], "
                         f"or a [..., 1] with b [{N}, 1]")
    ref, need = _matmul_plan(M, N, K, out, kind, bool(exact))
    y, py = _out("y", y, a, (*lead, N), out_dtype, dev)
    pw, wb, ws = _scratch(need, a, workspace)
    _run(load_library().gdn_matmul_e4m3, dev, ref, a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), py, pw, wb)
    return y


# ---- gated feed-forward block -------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _ffn_plan(rows, K, F, dtype, activation, backward, pairs):
    """(descriptor, its workspace size) of one of the two directions."""
    desc = GdnFfnDesc(rows, K, F, dtype, activation, GDN_OUT_SAME, GDN_FLAG_GRAD_PAIRS if pairs else 0)
    return ctypes.byref(desc), _bytes("gdn_gated_ffn_bwd_workspace_size" if backward else "gdn_gated_ffn_fwd_workspace_size", desc)


@functools.lru_cache(maxsize=1024)
def _ffn8_plan(rows, K, F, dtype, activation, out_type, exact):
    desc = GdnFfnDesc(rows, K, F, dtype, activation, out_type, GDN_FLAG_EXACT_SUMS if exact else 0)
    return ctypes.byref(desc), _bytes("gdn_gated_ffn_e4m3_workspace_size", desc)


def _gate(activation) -> int:
    code = _GATES.get(activation)
    if code is None:
        raise ValueError("activation: expected 'silu' or 'gelu_tanh'")
    return code


def _ffn_call(x, w_gate, w_up, activation, backward=False, pairs=False):
    """(descriptor, workspace bytes, rows, K, F)."""
    rows, K = _matrix("x", x)
    dtype = _dtype(x)
    F = _weight("w_gate", w_gate, K, x.dtype, x.device)
    _like("w_up", w_up, (F, K), x.dtype, x.device)
    if w_up is None:
        raise ValueError("w_up is required")
    return (*_ffn_plan(rows, K, F, dtype, _gate(activation), backward, pairs), rows, K, F)


def gdn_gated_ffn_pre(x, w_gate):
    """The buffer (fp32 device tensor [2, rows, F]) in which gdn_gated_ffn_fwd(pre=...) leaves gate and up for
    gdn_gated_ffn_bwd(pre=...) on the same inputs."""
    rows, K = _matrix("x", x)
    F = _weight("w_gate", w_gate, K, x.dtype, x.device)
    return torch.empty((2, rows, F), dtype=torch.float32, device=x.device)


def gdn_gated_ffn_fwd(x, w_gate, w_up, *, activation="silu", h=None, pre=None, workspace=None):
    """h = act(x w_gate^T) (x w_up^T): [..., F] in x's type.

    x [..., K] bf16 or fp32; w_gate, w_up [F, K] in x's type; activation 'silu' or 'gelu_tanh'. pre (see
    gdn_gated_ffn_pre) receives what gdn_gated_ffn_bwd needs of the forward."""
    ref, need, rows, K, F = _ffn_call(x, w_gate, w_up, activation)
    dev = x.device
    h, ph = _out("h", h, x, (*x.shape[:-1], F), x.dtype, dev)
    pp = _like("pre", pre, (2, rows, F), torch.float32, dev)
    pw, wb, ws = _scratch(need, x, workspace)
    _run(load_library().gdn_gated_ffn_fwd, dev, ref, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), ph, pp, pw, wb)
    return h


def gdn_gated_ffn_bwd(x, w_gate, w_up, d_h, *, activation="silu", pre=None, need_dx=True, need_dweight=True,
                      pairs=False, workspace=None, out=None):
    """Gradients of <d_h, h>: dict(dx, dw_gate, dw_up) in x's type, None where not needed; `out` may hold them
    preallocated. pre: what gdn_gated_ffn_fwd(pre=...) wrote for these inputs, or None (gate and up are computed
    again). The gradients of gate and up are rounded to x's type, the operands' type of the products behind, which in
    bf16 makes the error sqrt 2 times the results' own rounding; to a pair of bf16, which adds nothing to it, where rows
    F, rows K or F K is below 65,536, and with pairs=True at any size (8,192 x 2,048 x 8,192: 1,040 us to 2,690)."""
    ref, need, rows, K, F = _ffn_call(x, w_gate, w_up, activation, True, bool(pairs))
    dev, shape = x.device, x.shape
    if d_h is None:
        raise ValueError("d_h is required")
    pd = _like("d_h", d_h, (*shape[:-1], F), x.dtype, dev)
    pp = _like("pre", pre, (2, rows, F), torch.float32, dev)
    if out is None:
        out = {"dx": torch.empty_like(x) if need_dx else None,
               "dw_gate": torch.empty_like(w_gate) if need_dweight else None,
               "dw_up": torch.empty_like(w_up) if need_dweight else None}
    elif (out.get("dw_gate") is None) != (out.get("dw_up") is None):
        raise ValueError("out: dw_gate and dw_up come together")
    px = _like("out['dx']", out.get("dx"), shape, x.dtype, dev)
    pg = _like("out['dw_gate']", out.get("dw_gate"), (F, K), x.dtype, dev)
    pu = _like("out['dw_up']", out.get("dw_up"), (F, K), x.dtype, dev)
    pw, wb, ws = _scratch(need, x, workspace)
    _run(load_library().gdn_gated_ffn_bwd, dev, ref, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), pp, pd, px, pg, pu, pw, wb)
    return out


def gdn_gated_ffn_e4m3(x, x_scale, w_gate, gate_scale, w_up, up_scale, *, activation="silu", quant=None,
                       out_dtype=torch.bfloat16, exact=False, h=None, scale=None, workspace=None):
    """The block on quantised x [..., K] (scales per 128 columns) and weights [F, K] (scales per 128 x 128). Returns
    (h, scale or None): h [..., F] in out_dtype (bf16 by the 8-bit matrix instruction, or with exact=True and in fp32
    with fp32's products and sums; see gdn_matmul_e4m3), or with quant='group' in e4m3 with scales per 128 columns,
    quantised from its fp32 values."""
    rows, K = _matrix("x", x)
    if x.dtype != E4M3:
        raise TypeError("x: expected torch.float8_e4m3fn")
    if quant not in (None, "group"):
        raise ValueError("quant: expected None or 'group'")
    dtype = _DTYPES.get(out_dtype)
    if dtype is None:
        raise TypeError("out_dtype: expected torch.bfloat16 or torch.float32")
    dev, lead, kb = x.device, x.shape[:-1], _blocks(K)
    F = _weight("w_gate", w_gate, K, E4M3, dev)
    if w_up is None or x_scale is None or gate_scale is None or up_scale is None:
        raise ValueError("w_up and all scales are required")
    sshape = (-(-F // 128), kb)
    pu = _like("w_up", w_up, w_gate.shape, E4M3, dev)
    pxs = _like("x_scale", x_scale, (*lead, kb), torch.float32, dev)
    pgs = _like("gate_scale", gate_scale, sshape, torch.float32, dev)
    pus = _like("up_scale", up_scale, sshape, torch.float32, dev)
    ref, need = _ffn8_plan(rows, K, F, GDN_DTYPE_BF16 if quant else dtype, _gate(activation), GDN_OUT_E4M3 if quant else GDN_OUT_SAME,
                           bool(exact))
    h, ph = _out("h", h, x, (*lead, F), E4M3 if quant else out_dtype, dev)
    if quant:
        scale, psc = _out("scale", scale, x, (*lead, _blocks(F)), torch.float32, dev)
    elif scale is not None:
        raise ValueError("scale without quant")
    else:
        psc = None
    pw, wb, ws = _scratch(need, x, workspace)
    _run(load_library().gdn_gated_ffn_e4m3, dev, ref, x.data_ptr(), pxs, w_gate.data_ptr(), pgs, pu, pus, ph, psc, pw, wb)
    return h, scale


# ---- autograd -----------------------------------------------------------------------------------


class _LinearE4m3(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, need_dx, need_dw, exact):
        q, s = gdn_quant_e4m3(x, quant="group")
        y = gdn_matmul_e4m3(q, s, *gdn_quant_e4m3(weight, quant="block"), out_dtype=x.dtype, exact=exact)
        # of x the backward needs what the weight gradient contracts: its columns, in e4m3
        turned = gdn_quant_e4m3(x, quant="group", transpose=True) if need_dw else (None, None)
        ctx.save_for_backward(weight if need_dx else None, *turned)
        ctx.w_dtype, ctx.exact = weight.dtype, exact
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        weight, xq, xs = ctx.saved_tensors
        d_y = _dense(d_y)
        dx = dw = None
        if weight is not None:
            q, s = gdn_quant_e4m3(d_y, quant="group")
            dx = gdn_matmul_e4m3(q, s, *gdn_quant_e4m3(weight, quant="block", transpose=True), out_dtype=d_y.dtype, exact=ctx.exact)
        if xq is not None:
            q, s = gdn_quant_e4m3(d_y, quant="group", transpose=True)
            dw = gdn_matmul_e4m3(q, s, xq, xs, out_dtype=ctx.w_dtype, exact=ctx.exact)
        return dx, dw, None, None, None


def linear_e4m3(x, weight, *, exact=False):
    """y = x weight^T through e4m3, with autograd (x, weight): y [..., N] in x's type.

    x [..., K] and weight [N, K], each bf16 or fp32, are quantised on the way (x per 128 columns, weight per 128 x
    128), and so is the gradient that comes back (per 128 columns for dx, per 128 tokens for the weight's). Held for
    the backward: x in e4m3, quantised along its tokens. exact: sums as in fp32 in the three products' bf16 outputs
    too (gdn_matmul_e4m3)."""
    rows, K = _matrix("x", x)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[1] != K:
        raise ValueError(f"weight: expected [N, {K}]")
    if weight.device != x.device:
        raise ValueError(f"weight: expected a tensor on {x.device}")
    grad = torch.is_grad_enabled()
    return _LinearE4m3.apply(x, weight, grad and x.requires_grad, grad and weight.requires_grad, bool(exact))


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, keep, pairs):
        pre = gdn_gated_ffn_pre(x, w_gate) if keep else None
        h = gdn_gated_ffn_fwd(x, w_gate, w_up, activation=activation, pre=pre)
        ctx.save_for_backward(x, w_gate, w_up, pre)
        ctx.activation, ctx.pairs = activation, pairs
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, d_h):
        x, w_gate, w_up, pre = ctx.saved_tensors
        need = ctx.needs_input_grad
        gr = gdn_gated_ffn_bwd(x, w_gate, w_up, _dense(d_h), activation=ctx.activation, pre=pre, need_dx=need[0],
                               need_dweight=need[1] or need[2], pairs=ctx.pairs)
        return gr["dx"], gr["dw_gate"] if need[1] else None, gr["dw_up"] if need[2] else None, None, None, None


def gated_ffn(x, w_gate, w_up, *, activation="silu", recompute=False, pairs=False):
    """gdn_gated_ffn_fwd with autograd (x, w_gate, w_up): h [..., F] in x's type. gate and up are held in fp32 for
    the backward (8 bytes per value of h), or with recompute computed again there. pairs: see gdn_gated_ffn_bwd."""
    keep = not recompute and torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up))
    return _GatedFfn.apply(x, w_gate, w_up, activation, keep, bool(pairs))
