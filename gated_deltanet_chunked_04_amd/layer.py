"""The operators around the gated delta rule in a layer: gated scan, short convolution and RMS norm.

Like the rest of the package these functions carry the C ABI's names (include/gdn.h) and only marshal
tensors into it; every step of the computation runs in the HIP library. Tensors are contiguous, on one
device; work runs on that device's current stream. Tokens in front of a packed batch's first sequence and
behind its last one get zeros in outputs and gradients that these functions allocate, and leave a caller's
own as they were.

  gdn_gated_scan_fwd / _bwd     h_t = exp(g_t) h_{t-1} + x_t per channel, and its gradients
  gdn_gated_scan_states(x)      the buffer that carries the forward's states to the backward
  gdn_short_conv_fwd / _bwd     causal convolution of 2 to 4 taps per channel, silu or none behind it
  gdn_rmsnorm_fwd / _bwd        RMS norm, residual addition in front, 8-bit output with scales behind
  gated_scan, short_conv, rms_norm   the same with autograd
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from ._abi import (GDN_ACT_NONE, GDN_ACT_SILU, GDN_DTYPE_BF16, GDN_DTYPE_FP32, GDN_FLAG_ZERO_OUTSIDE, GDN_OUT_E4M3,
                   GDN_OUT_SAME, GdnConvDesc, GdnRmsnormDesc, GdnScanDesc, check, load_library)

_DTYPES = {torch.bfloat16: GDN_DTYPE_BF16, torch.float32: GDN_DTYPE_FP32}
_ACTIVATIONS = {None: GDN_ACT_NONE, "silu": GDN_ACT_SILU}
_QUANT = {"row": 0, "group": 128}
SCAN_TILE = 64  # tokens between two kept states of the gated scan


def _dtype(t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported input dtype {t.dtype} (bf16 or fp32)")
    return code


def _lead(name, x, dims):
    if not isinstance(x, torch.Tensor) or x.dim() != dims or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous device tensor of {dims} dimensions")


def _like(name, t, shape, dtype, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {tuple(shape)} {dtype} tensor on {device}")
    return t.data_ptr()


def _out(name, t, x, shape, dtype, device):
    """(tensor, pointer) of a caller's output, or of a new one (empty_like is the quicker call where it serves)."""
    if t is None:
        t = torch.empty_like(x) if dtype == x.dtype and shape == x.shape else x.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    return t, _like(name, t, shape, dtype, device)


def _outs(out, x, device, **want):
    """(dict, its pointers in order) of a backward's outputs, name=(shape, dtype, whether a new dict has it): new
    ones, or the caller's, which must hold all but the ones that may be left out (a state's or a bias's)."""
    if out is None:
        out = {k: _out(k, None, x, shape, dtype, device)[0] if need else None for k, (shape, dtype, need) in want.items()}
        return (out, *(None if t is None else t.data_ptr() for t in out.values()))
    for k in ("dx", "dg", "dweight"):
        if k in want and want[k][2] and out.get(k) is None:
            raise ValueError(f"out[{k!r}] is required")
    return (out, *(_like(f"out[{k!r}]", out.get(k), shape, dtype, device) for k, (shape, dtype, _) in want.items()))


def _second_type(name, t, x) -> int:
    if not isinstance(t, torch.Tensor) or (t.dtype != x.dtype and t.dtype != torch.float32):
        raise ValueError(f"{name}: expected {x.dtype} or fp32")
    return _DTYPES[t.dtype]


def _packing(x, cu_seqlens, new):
    """(N, flags) of a packed batch; new: the outputs are, and get zeros in rows of no sequence."""
    if (not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device
            or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 2):
        raise TypeError(f"cu_seqlens must be a contiguous int32 tensor [N+1], N >= 1, on {x.device}")
    if x.shape[0] != 1:
        raise ValueError("cu_seqlens needs B = 1")
    return cu_seqlens.numel() - 1, GDN_FLAG_ZERO_OUTSIDE if new else 0


# The current stream's handle. The first form gives it without building a Stream object (0.1 against 1.9 us of a
# decoding call's 10); it is not in torch's public interface, so the public one stands in where it is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device) -> int:
    return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _run(fn, device, *args):
    """One call of the library on `device`'s current stream, with `device` current."""
    if torch.cuda.current_device() == device.index:
        status = fn(*args, _stream_of(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream_of(device))
    if status:
        check(status, fn.__name__)


def _scratch(nbytes, x, workspace):
    """(pointer, bytes, the tensor to keep alive) of a caller's workspace or of a new one."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = x.new_empty(nbytes, dtype=torch.uint8)
        return workspace.data_ptr(), nbytes, workspace
    if (not isinstance(workspace, torch.Tensor) or workspace.device != x.device or not workspace.is_contiguous()
            or workspace.data_ptr() % 256):
        raise ValueError(f"workspace must be a contiguous tensor on {x.device} at a 256-byte aligned address")
    size = workspace.numel() * workspace.element_size()
    if size < nbytes:
        raise ValueError(f"workspace too small: {size} bytes, {nbytes} needed")
    return workspace.data_ptr(), size, workspace


def _bytes(name, desc) -> int:
    n = ctypes.c_size_t()
    check(getattr(load_library(), name)(ctypes.byref(desc), ctypes.byref(n)), name)
    return n.value


# ---- gated scan ---------------------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _scan_plan(B, T, D, dtype, g_dtype):
    """(descriptor of an unpacked call, its forward's and its backward's workspace sizes): by sizes and types alone,
    never changed afterwards."""
    desc = GdnScanDesc(B, T, D, dtype, g_dtype)
    return (ctypes.byref(desc), _bytes("gdn_gated_scan_fwd_workspace_size", desc),
            _bytes("gdn_gated_scan_bwd_workspace_size", desc))


def _scan_call(x, g, cu_seqlens, new):
    """(descriptor, forward and backward workspace bytes, N)."""
    _lead("x", x, 3)
    dtype, g_dtype = _dtype(x), _second_type("g", g, x)
    B, T, D = x.shape
    ref, fwd, bwd = _scan_plan(B, T, D, dtype, g_dtype)
    if cu_seqlens is None:
        return ref, fwd, bwd, B
    N, flags = _packing(x, cu_seqlens, new)
    return ctypes.byref(GdnScanDesc(B, T, D, dtype, g_dtype, N, flags, cu_seqlens.data_ptr())), fwd, bwd, N


def gdn_gated_scan_states(x):
    """The buffer (fp32 device tensor) in which gdn_gated_scan_fwd(states=...) leaves the state that
    enters every 64th token, for gdn_gated_scan_bwd(states=...) on the same inputs."""
    _lead("x", x, 3)
    B, T, D = x.shape
    return torch.empty((-(-B * T // SCAN_TILE), D), dtype=torch.float32, device=x.device)


def _check_states(states, x):
    if states is None:
        return None
    B, T, D = x.shape
    p = _like("states", states, (-(-B * T // SCAN_TILE), D), torch.float32, x.device)
    if p % 256:
        raise ValueError("states must start at a 256-byte aligned address")
    return p or None


def gdn_gated_scan_fwd(x, g, initial_state=None, *, cu_seqlens=None, output_final_state=True, h=None,
                       final_state=None, states=None, workspace=None):
    """h_t = exp(g_t) h_{t-1} + x_t per sequence and channel. Returns (h, final_state or None).

    x [B,T,D] bf16 or fp32; g [B,T,D] natural-log decay, in x's type or fp32; initial_state [N,D] fp32
    or None (zeros); cu_seqlens int32 device tensor [N+1] (B = 1), no host copy needed. final_state may be
    initial_state itself (updated in place). states (see gdn_gated_scan_states) receives what
    gdn_gated_scan_bwd needs of the forward."""
    ref, need, _, N = _scan_call(x, g, cu_seqlens, h is None)
    shape, dev = x.shape, x.device
    pg = _like("g", g, shape, g.dtype, dev)
    p0 = _like("initial_state", initial_state, (N, shape[2]), torch.float32, dev)
    h, ph = _out("h", h, x, shape, x.dtype, dev)
    if output_final_state and final_state is not None and final_state is initial_state:
        pT = p0
    elif output_final_state:
        final_state, pT = _out("final_state", final_state, x, (N, shape[2]), torch.float32, dev)
    else:
        final_state = pT = None
    ps = _check_states(states, x)
    pw, wb, ws = _scratch(need, x, workspace)
    _run(load_library().gdn_gated_scan_fwd, dev, ref, x.data_ptr(), pg, p0, ph, pT, ps, pw, wb)
    return h, final_state


def gdn_gated_scan_bwd(x, g, d_h, initial_state=None, d_final_state=None, *, cu_seqlens=None, states=None,
                       need_d_initial_state=True, workspace=None, out=None):
    """Gradients of <d_h, h> + <d_final_state, final_state>: dict(dx, dg, d_initial_state); `out` may hold
    them preallocated. states: what gdn_gated_scan_fwd(states=...) wrote for these inputs, or None (the
    states are recomputed)."""
    ref, _, need, N = _scan_call(x, g, cu_seqlens, out is None)
    shape, dev = x.shape, x.device
    if d_h is None:
        raise ValueError("d_h is required")
    pg = _like("g", g, shape, g.dtype, dev)
    p0 = _like("initial_state", initial_state, (N, shape[2]), torch.float32, dev)
    pd = _like("d_h", d_h, shape, x.dtype, dev)
    pT = _like("d_final_state", d_final_state, (N, shape[2]), torch.float32, dev)
    out, px, pdg, pd0 = _outs(out, x, dev, dx=(shape, x.dtype, True), dg=(shape, g.dtype, True),
                              d_initial_state=((N, shape[2]), torch.float32, need_d_initial_state))
    ps = _check_states(states, x)
    pw, wb, ws = _scratch(need, x, workspace)
    _run(load_library().gdn_gated_scan_bwd, dev, ref, x.data_ptr(), pg, p0, pd, pT, ps, px, pdg, pd0, pw, wb)
    return out


# ---- short convolution --------------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _conv_plan(B, T, D, W, dtype, w_dtype, activation):
    """(descriptor of an unpacked call, its backward's workspace size)."""
    desc = GdnConvDesc(B, T, D, W, dtype, w_dtype, activation)
    return ctypes.byref(desc), _bytes("gdn_short_conv_bwd_workspace_size", desc)


def _conv_call(x, weight, bias, activation, cu_seqlens, new):
    """(descriptor, backward workspace bytes, N, W, pointers of weight and bias)."""
    _lead("x", x, 3)
    dtype, w_dtype = _dtype(x), _second_type("weight", weight, x)
    if activation not in _ACTIVATIONS:
        raise ValueError("activation: expected 'silu' or None")
    if weight.dim() != 2:
        raise ValueError("weight: expected [D, W]")
    B, T, D = x.shape
    W = weight.shape[1]
    pw = _like("weight", weight, (D, W), weight.dtype, x.device)
    pb = _like("bias", bias, (D,), weight.dtype, x.device)
    act = _ACTIVATIONS[activation]
    ref, bwd = _conv_plan(B, T, D, W, dtype, w_dtype, act)
    if cu_seqlens is None:
        return ref, bwd, B, W, pw, pb
    N, flags = _packing(x, cu_seqlens, new)
    return ctypes.byref(GdnConvDesc(B, T, D, W, dtype, w_dtype, act, N, flags, cu_seqlens.data_ptr())), bwd, N, W, pw, pb


def gdn_short_conv_fwd(x, weight, bias=None, initial_state=None, *, activation="silu", cu_seqlens=None,
                       output_final_state=False, y=None, final_state=None):
    """y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}). Returns (y, final_state or None).

    x [B,T,D] bf16 or fp32; weight [D,W], W in {2, 3, 4}, and bias [D] in x's type or fp32; activation
    'silu' or None; initial_state [N,W-1,D] in x's type: the inputs before each sequence's first token,
    oldest first (zeros if None). The final state is a sequence's last W-1 inputs; a final_state tensor
    asks for it, and may be initial_state itself for up to 16 tokens per row (decoding)."""
    ref, _, N, W, pw, pb = _conv_call(x, weight, bias, activation, cu_seqlens, y is None)
    shape, dev = x.shape, x.device
    sshape = (N, W - 1, shape[2])
    p0 = _like("initial_state", initial_state, sshape, x.dtype, dev)
    y, py = _out("y", y, x, shape, x.dtype, dev)
    pT = None
    if final_state is not None and final_state is initial_state:
        pT = p0
    elif final_state is not None or output_final_state:
        final_state, pT = _out("final_state", final_state, x, sshape, x.dtype, dev)
    _run(load_library().gdn_short_conv_fwd, dev, ref, x.data_ptr(), pw, pb, p0, py, pT)
    return y, final_state


def gdn_short_conv_bwd(x, weight, d_y, bias=None, initial_state=None, d_final_state=None, *, activation="silu",
                       cu_seqlens=None, need_d_initial_state=True, workspace=None, out=None):
    """Gradients of <d_y, y> + <d_final_state, final_state>: dict(dx, dweight, dbias, d_initial_state), dweight
    and dbias in fp32, dbias None without a bias; `out` may hold them preallocated."""
    ref, need, N, W, pw, pb = _conv_call(x, weight, bias, activation, cu_seqlens, out is None)
    shape, dev = x.shape, x.device
    D = shape[2]
    sshape = (N, W - 1, D)
    if d_y is None:
        raise ValueError("d_y is required")
    p0 = _like("initial_state", initial_state, sshape, x.dtype, dev)
    pd = _like("d_y", d_y, shape, x.dtype, dev)
    pT = _like("d_final_state", d_final_state, sshape, x.dtype, dev)
    out, px, pdw, pdb, pd0 = _outs(out, x, dev, dx=(shape, x.dtype, True), dweight=((D, W), torch.float32, True),
                                   dbias=((D,), torch.float32, bias is not None),
                                   d_initial_state=(sshape, x.dtype, need_d_initial_state))
    ws_p, wb, ws = _scratch(need, x, workspace)
    _run(load_library().gdn_short_conv_bwd, dev, ref, x.data_ptr(), pw, pb, p0, pd, pT, px, pdw, pdb, pd0, ws_p, wb)
    return out


# ---- RMS norm -----------------------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def _rms_plan(rows, D, dtype, w_dtype, out_type, scale_group, eps):
    """(descriptor, the backward's workspace size)."""
    desc = GdnRmsnormDesc(rows, D, dtype, w_dtype, out_type, scale_group, eps)
    return ctypes.byref(desc), _bytes("gdn_rmsnorm_bwd_workspace_size", desc)


def _rms_call(name, x, weight, eps, out_type=GDN_OUT_SAME, scale_group=0):
    """(descriptor, backward workspace bytes, pointer of weight)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous device tensor [..., D]")
    D = x.shape[-1]
    ref, bwd = _rms_plan(x.numel() // D if D else 0, D, _dtype(x), _second_type("weight", weight, x), out_type,
                         scale_group, eps)
    return ref, bwd, _like("weight", weight, (D,), weight.dtype, x.device)


def gdn_rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, quant=None, y=None, residual_out=None, scale=None):
    """r = x + residual, y = r weight / sqrt(mean(r^2) + eps) over the last dimension. Returns
    (y, residual_out or None, scale or None).

    x [..., D] bf16 or fp32; weight [D] in x's type or fp32; residual like x or None. residual_out receives r
    in x's type (it may be residual or x itself). quant None gives y in x's type; 'row' and 'group' give
    it as torch.float8_e4m3fn with fp32 scales of every row ([..., 1]) or of every 128 columns
    ([..., ceil(D/128)]): y stands for y.float() * scale."""
    if quant is not None and quant not in _QUANT:
        raise ValueError("quant: expected None, 'row' or 'group'")
    ref, _, pw = _rms_call("x", x, weight, eps, *((GDN_OUT_SAME, 0) if quant is None else (GDN_OUT_E4M3, _QUANT[quant])))
    shape, dev, D = x.shape, x.device, x.shape[-1]
    pr = _like("residual", residual, shape, x.dtype, dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
        po = None
    else:
        residual_out, po = _out("residual_out", residual_out, x, shape, x.dtype, dev)
    if quant is None:
        if scale is not None:
            raise ValueError("scale without quant")
        ydt, psc = x.dtype, None
    else:
        ydt = torch.float8_e4m3fn
        sshape = (*shape[:-1], 1 if quant == "row" else -(-D // 128))
        scale, psc = _out("scale", scale, x, sshape, torch.float32, dev)
    y, py = _out("y", y, x, shape, ydt, dev)
    _run(load_library().gdn_rmsnorm_fwd, dev, ref, x.data_ptr(), pr, pw, py, psc, po)
    return y, residual_out, scale


def gdn_rmsnorm_bwd(r, weight, d_y, d_residual=None, *, eps=1e-6, need_dweight=True, workspace=None, out=None):
    """Gradients of <d_y, y> + <d_residual, residual_out> from r (the forward's residual_out, or x where there
    was no residual): dict(dx, dweight), dx being the gradient of x and of residual alike, dweight fp32;
    `out` may hold them preallocated."""
    ref, need, pw = _rms_call("r", r, weight, eps)
    shape, dev, D = r.shape, r.device, r.shape[-1]
    if d_y is None:
        raise ValueError("d_y is required")
    pd = _like("d_y", d_y, shape, r.dtype, dev)
    pr = _like("d_residual", d_residual, shape, r.dtype, dev)
    if out is not None:
        need_dweight = out.get("dweight") is not None
    out, px, pdw = _outs(out, r, dev, dx=(shape, r.dtype, True), dweight=((D,), torch.float32, need_dweight))
    ws_p, wb, ws = _scratch(need, r, workspace)
    _run(load_library().gdn_rmsnorm_bwd, dev, ref, r.data_ptr(), pw, pd, pr, px, pdw, ws_p, wb)
    return out


# ---- autograd -----------------------------------------------------------------------------------


def _dense(t: Optional[torch.Tensor]):
    return None if t is None else t.contiguous()


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, initial_state, cu_seqlens, grad):
        states = gdn_gated_scan_states(x) if grad else None
        h, final = gdn_gated_scan_fwd(x, g, initial_state, cu_seqlens=cu_seqlens, states=states)
        ctx.save_for_backward(x, g, initial_state, cu_seqlens, states)
        ctx.set_materialize_grads(False)
        return h, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_h, d_final):
        x, g, s0, cu, states = ctx.saved_tensors
        gr = gdn_gated_scan_bwd(x, g, torch.zeros_like(x) if d_h is None else _dense(d_h), s0, _dense(d_final),
                                cu_seqlens=cu, states=states, need_d_initial_state=s0 is not None)
        return gr["dx"], gr["dg"], gr["d_initial_state"], None, None


def gated_scan(x, g, initial_state=None, *, cu_seqlens=None, output_final_state=True):
    """gdn_gated_scan_fwd with autograd (x, g, initial_state): (h, final_state or None). The state entering
    every 64th token is held for the backward, which recomputes h from there."""
    grad = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, g, initial_state))
    h, final = _GatedScan.apply(x, g, initial_state, cu_seqlens, grad)
    return h, (final if output_final_state else None)


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, activation, cu_seqlens, output_final_state):
        y, final = gdn_short_conv_fwd(x, weight, bias, initial_state, activation=activation, cu_seqlens=cu_seqlens,
                                      output_final_state=output_final_state)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y, d_final):
        x, w, b, s0, cu = ctx.saved_tensors
        gr = gdn_short_conv_bwd(x, w, torch.zeros_like(x) if d_y is None else _dense(d_y), b, s0, _dense(d_final),
                                activation=ctx.activation, cu_seqlens=cu, need_d_initial_state=s0 is not None)
        return (gr["dx"], gr["dweight"].to(w.dtype), None if b is None else gr["dbias"].to(b.dtype),
                gr["d_initial_state"], None, None, None)


def short_conv(x, weight, bias=None, initial_state=None, *, activation="silu", cu_seqlens=None,
               output_final_state=False):
    """gdn_short_conv_fwd with autograd (x, weight, bias, initial_state): (y, final_state or None)."""
    return _ShortConv.apply(x, weight, bias, initial_state, activation, cu_seqlens, output_final_state)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, kept, _ = gdn_rmsnorm_fwd(x, weight, residual, eps=eps)
        ctx.save_for_backward(x if residual is None else kept, weight)
        ctx.eps = eps
        ctx.added = residual is not None
        ctx.set_materialize_grads(False)
        return y, kept

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y, d_kept):
        r, w = ctx.saved_tensors
        gr = gdn_rmsnorm_bwd(r, w, torch.zeros_like(r) if d_y is None else _dense(d_y), _dense(d_kept), eps=ctx.eps,
                             need_dweight=ctx.needs_input_grad[1])
        dw = None if gr["dweight"] is None else gr["dweight"].to(w.dtype)
        return gr["dx"], dw, gr["dx"] if ctx.added else None, None


def rms_norm(x, weight, residual=None, *, eps=1e-6):
    """gdn_rmsnorm_fwd (in x's type) with autograd (x, weight, residual): y, or (y, residual_out) with a
    residual."""
    y, kept = _RmsNorm.apply(x, weight, residual, eps)
    return y if residual is None else (y, kept)
