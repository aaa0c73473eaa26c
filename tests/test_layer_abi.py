"""The layer operators' entry points on the host (no GPU): sizes, and refusals before anything is launched."""
import ctypes

import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from gated_deltanet_chunked_04_amd import _abi

P = ctypes.c_void_p(0x10000)
Q = ctypes.c_void_p(0x20000)
R = ctypes.c_void_p(0x30000)
S = ctypes.c_void_p(0x40000)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


def scan_desc(B=2, T=300, D=96, dtype=0, g_dtype=1, **kw):
    d = _abi.GdnScanDesc(B=B, T=T, D=D, dtype=dtype, g_dtype=g_dtype)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def conv_desc(B=2, T=300, D=96, width=4, dtype=0, w_dtype=0, activation=1, **kw):
    d = _abi.GdnConvDesc(B=B, T=T, D=D, width=width, dtype=dtype, w_dtype=w_dtype, activation=activation)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def rms_desc(rows=7, D=96, dtype=0, w_dtype=0, out_type=0, scale_group=0, eps=1e-6, **kw):
    d = _abi.GdnRmsnormDesc(rows=rows, D=D, dtype=dtype, w_dtype=w_dtype, out_type=out_type, scale_group=scale_group, eps=eps)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def size(fn, d):
    n = ctypes.c_size_t()
    assert fn(ctypes.byref(d), ctypes.byref(n)) == 0
    return n.value


def test_sizes(lib):
    # one fp32 state per channel for every 64 tokens begun
    assert size(lib.gdn_gated_scan_states_size, scan_desc(B=2, T=300, D=96)) == 10 * 96 * 4
    assert size(lib.gdn_gated_scan_states_size, scan_desc(B=1, T=0, D=96)) == 0
    for fn in (lib.gdn_gated_scan_fwd_workspace_size, lib.gdn_gated_scan_bwd_workspace_size):
        a = size(fn, scan_desc(B=2, T=300))
        assert a == size(fn, scan_desc(B=1, T=600)) == size(fn, scan_desc(B=1, T=600, dtype=1))
        assert size(fn, scan_desc(B=1, T=0)) == 0
        assert fn(ctypes.byref(scan_desc()), None) == 1 and fn(None, ctypes.byref(ctypes.c_size_t())) == 1
    assert size(lib.gdn_short_conv_bwd_workspace_size, conv_desc()) > 0
    assert size(lib.gdn_rmsnorm_bwd_workspace_size, rms_desc()) > 0


@pytest.mark.parametrize("change,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(dtype=2), 1), (dict(g_dtype=2), 1),
    (dict(dtype=1, g_dtype=0), 1), (dict(flags=1), 1), (dict(cu_seqlens=0x1000), 1),
    (dict(B=1, cu_seqlens=0x1000, num_seqs=0), 1), (dict(B=1 << 20, T=1 << 20), 2), (dict(B=1, T=1 << 31), 2),
    (dict(D=1 << 25), 2)])
def test_scan_refusals(lib, change, code):
    d = scan_desc(**change)
    n = ctypes.c_size_t(BIG)
    assert lib.gdn_gated_scan_fwd(ctypes.byref(d), P, Q, None, R, None, None, S, n, None) == code
    assert lib.gdn_gated_scan_bwd(ctypes.byref(d), P, Q, None, R, None, None, S, ctypes.c_void_p(0x50000), None, S, n, None) == code
    assert lib.gdn_gated_scan_states_size(ctypes.byref(d), ctypes.byref(n)) == code


def test_grids_beyond_32_bits(lib):
    """More threads than a launch can count: refused before anything is launched."""
    n = ctypes.c_size_t(1 << 50)
    out = ctypes.c_void_p(0x50000)
    assert lib.gdn_rmsnorm_fwd(ctypes.byref(rms_desc(rows=5_000_000, D=4)), P, None, Q, R, None, None, None) == 2
    assert lib.gdn_rmsnorm_fwd(ctypes.byref(rms_desc(rows=2_000_000_000, D=512)), P, None, Q, R, None, None, None) == 2
    assert lib.gdn_rmsnorm_bwd(ctypes.byref(rms_desc(rows=5_000_000, D=4)), P, Q, R, None, S, None, S, n, None) == 2
    assert lib.gdn_gated_scan_fwd(ctypes.byref(scan_desc(B=1, T=2_000_000_000, D=1024)), P, Q, None, R, None, None, S, n, None) == 2
    assert lib.gdn_gated_scan_fwd(ctypes.byref(scan_desc(B=200_000_000, T=1, D=64)), P, Q, None, R, None, None, S, n, None) == 2
    assert lib.gdn_gated_scan_bwd(ctypes.byref(scan_desc(B=1, T=2_000_000_000, D=1024)), P, Q, None, R, None, P, S, out, None, S, n, None) == 2
    assert lib.gdn_short_conv_fwd(ctypes.byref(conv_desc(B=200_000_000, T=1, D=64)), P, Q, None, None, R, None, None) == 2
    assert lib.gdn_short_conv_bwd(ctypes.byref(conv_desc(B=1, T=2_000_000_000, D=4096)), P, Q, None, None, R, None, S, out, None, None, S, n, None) == 2


def test_scan_workspace_of_decoding(lib):
    """Short rows need none; packed sequences never more than the unpacked call of their size."""
    fn = lib.gdn_gated_scan_fwd_workspace_size
    for B, T in ((1000, 1), (1000, 16), (10, 64)):
        assert size(fn, scan_desc(B=B, T=T)) == size(lib.gdn_gated_scan_bwd_workspace_size, scan_desc(B=B, T=T)) == 0
    assert size(fn, scan_desc(B=10, T=65)) > 0
    for N in (1, 50, 300):
        assert size(fn, scan_desc(B=1, T=1000, cu_seqlens=0x1000, num_seqs=N)) <= size(fn, scan_desc(B=1, T=1000))


def test_scan_refused_buffers(lib):
    d = scan_desc()
    r = ctypes.byref(d)
    n = ctypes.c_size_t(size(lib.gdn_gated_scan_fwd_workspace_size, d))
    fwd = lib.gdn_gated_scan_fwd
    assert fwd(r, None, Q, None, R, None, None, S, n, None) == 1
    assert fwd(r, P, None, None, R, None, None, S, n, None) == 1
    assert fwd(r, P, Q, None, None, None, None, S, n, None) == 1
    assert fwd(r, P, Q, None, P, None, None, S, n, None) == 1      # h is x
    assert fwd(r, P, Q, None, Q, None, None, S, n, None) == 1      # h is g
    assert fwd(r, P, Q, None, R, None, None, None, n, None) == 3
    assert fwd(r, P, Q, None, R, None, None, S, ctypes.c_size_t(n.value - 1), None) == 3
    assert fwd(r, P, Q, None, R, None, None, ctypes.c_void_p(0x40010), n, None) == 3
    assert fwd(r, P, Q, None, R, None, ctypes.c_void_p(0x50010), S, n, None) == 3
    n = ctypes.c_size_t(size(lib.gdn_gated_scan_bwd_workspace_size, d))
    T_, U_ = ctypes.c_void_p(0x50000), ctypes.c_void_p(0x60000)
    bwd = lib.gdn_gated_scan_bwd
    assert bwd(r, P, Q, None, None, None, None, T_, U_, None, S, n, None) == 1
    assert bwd(r, P, Q, None, R, None, None, T_, T_, None, S, n, None) == 1   # dx is dg
    assert bwd(r, P, Q, None, R, None, None, R, U_, None, S, n, None) == 1    # dx is d_h
    assert bwd(r, P, Q, None, R, None, None, T_, U_, None, S, ctypes.c_size_t(n.value - 1), None) == 3
    f = ctypes.cast(T_, ctypes.c_void_p)
    assert bwd(r, P, Q, None, R, f, None, U_, ctypes.c_void_p(0x70000), f, S, n, None) == 1


@pytest.mark.parametrize("change,code", [
    (dict(width=1), 2), (dict(width=5), 2), (dict(activation=2), 1), (dict(w_dtype=3), 1), (dict(dtype=1, w_dtype=0), 1),
    (dict(D=0), 1), (dict(T=-1), 1), (dict(B=0), 1), (dict(flags=4), 1), (dict(cu_seqlens=0x1000, num_seqs=2), 1),
    (dict(B=1 << 20, T=1 << 20), 2)])
def test_conv_refusals(lib, change, code):
    d = conv_desc(**change)
    n = ctypes.c_size_t(BIG)
    assert lib.gdn_short_conv_fwd(ctypes.byref(d), P, Q, None, None, R, None, None) == code
    assert lib.gdn_short_conv_bwd(ctypes.byref(d), P, Q, None, None, R, None, S, ctypes.c_void_p(0x50000), None, None, S, n, None) == code


def test_conv_refused_buffers(lib):
    fwd = lib.gdn_short_conv_fwd
    d = conv_desc(T=17)
    r = ctypes.byref(d)
    assert fwd(r, None, Q, None, None, R, None, None) == 1
    assert fwd(r, P, None, None, None, R, None, None) == 1
    assert fwd(r, P, Q, None, None, P, None, None) == 1
    # a state updated in place: only for a few tokens of unpacked rows
    assert fwd(r, P, Q, None, S, R, S, None) == 1
    packed = conv_desc(B=1, T=4, cu_seqlens=0x1000, num_seqs=2)
    assert fwd(ctypes.byref(packed), P, Q, None, S, R, S, None) == 1
    n = ctypes.c_size_t(size(lib.gdn_short_conv_bwd_workspace_size, d))
    bwd, dw = lib.gdn_short_conv_bwd, ctypes.c_void_p(0x50000)
    assert bwd(r, P, Q, None, None, R, None, S, None, None, None, S, n, None) == 1        # no dweight
    assert bwd(r, P, Q, None, None, R, None, R, dw, None, None, S, n, None) == 1          # dx is d_y
    assert bwd(r, P, Q, None, None, R, None, S, dw, None, None, None, n, None) == 3
    assert bwd(r, P, Q, None, None, R, None, S, dw, None, None, S, ctypes.c_size_t(n.value - 1), None) == 3


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), 1), (dict(D=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(out_type=2), 1), (dict(scale_group=64, out_type=1), 1), (dict(scale_group=128), 1), (dict(dtype=5), 1),
    (dict(dtype=1, w_dtype=0), 1), (dict(flags=1), 1), (dict(rows=1 << 31), 2), (dict(D=1 << 25), 2)])
def test_rms_refusals(lib, change, code):
    d = rms_desc(**change)
    scale = P if d.out_type == 1 else None
    assert lib.gdn_rmsnorm_fwd(ctypes.byref(d), P, None, Q, R, scale, None, None) == code
    assert lib.gdn_rmsnorm_bwd(ctypes.byref(d), P, Q, R, None, S, None, S, ctypes.c_size_t(BIG), None) == code


def test_rms_refused_buffers(lib):
    fwd, bwd = lib.gdn_rmsnorm_fwd, lib.gdn_rmsnorm_bwd
    r = ctypes.byref(rms_desc())
    assert fwd(r, P, None, None, R, None, None, None) == 1
    assert fwd(r, P, S, Q, R, None, None, None) == 1       # a residual needs residual_out
    assert fwd(r, P, None, Q, R, None, S, None) == 1       # and residual_out a residual
    assert fwd(r, P, None, Q, P, None, None, None) == 1    # y is x
    assert fwd(r, P, S, Q, S, None, S, None) == 1          # y is the residual
    assert fwd(r, P, None, Q, R, S, None, None) == 1       # scales without 8 bits
    q = ctypes.byref(rms_desc(out_type=1))
    assert fwd(q, P, None, Q, R, None, None, None) == 1    # 8 bits without scales
    n = ctypes.c_size_t(size(lib.gdn_rmsnorm_bwd_workspace_size, rms_desc()))
    assert bwd(r, P, Q, None, None, S, None, S, n, None) == 1
    assert bwd(r, P, Q, R, S, S, None, S, n, None) == 1    # dx is d_residual
    assert bwd(r, P, Q, R, None, S, None, None, n, None) == 3
    assert bwd(r, P, Q, R, None, S, None, S, ctypes.c_size_t(n.value - 1), None) == 3


def test_python_refuses_host_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        gdn.gdn_gated_scan_fwd(x, x)
    with pytest.raises(ValueError):
        gdn.gdn_short_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        gdn.gdn_rmsnorm_fwd(x, torch.zeros(8))
    with pytest.raises(ValueError):
        gdn.rms_norm(x, torch.zeros(8))


def test_zero_outside_flag(lib):
    """Taken by the operators that know sequences, alone; other bits beside it are refused."""
    n = ctypes.c_size_t(BIG)
    assert _abi.GDN_FLAG_ZERO_OUTSIDE == 128
    for flags, code in ((128, 0), (129, 1), (256, 1), (-1, 1)):
        assert lib.gdn_gated_scan_fwd_workspace_size(ctypes.byref(scan_desc(flags=flags)), ctypes.byref(n)) == code
        assert lib.gdn_short_conv_bwd_workspace_size(ctypes.byref(conv_desc(flags=flags)), ctypes.byref(n)) == code
        assert lib.gdn_rmsnorm_bwd_workspace_size(ctypes.byref(rms_desc(flags=flags)), ctypes.byref(n)) == 1
