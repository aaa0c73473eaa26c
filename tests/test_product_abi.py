"""The entry points of the layer's products on the host (no GPU): sizes, and refusals before anything is launched."""
import ctypes

import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from gated_deltanet_chunked_04_amd import _abi

P, Q, R, S, V, W, X = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(7))
BIG = ctypes.c_size_t(1 << 45)


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


def quant_desc(rows=7, cols=300, dtype=0, scales=1, transpose=0, **kw):
    d = _abi.GdnQuantDesc(rows=rows, cols=cols, dtype=dtype, scales=scales, transpose=transpose)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def mm_desc(M=7, N=300, K=200, out_dtype=0, scales=2, **kw):
    d = _abi.GdnMatmulDesc(M=M, N=N, K=K, out_dtype=out_dtype, scales=scales)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def ffn_desc(rows=7, K=96, F=200, dtype=0, activation=1, out_type=0, **kw):
    d = _abi.GdnFfnDesc(rows=rows, K=K, F=F, dtype=dtype, activation=activation, out_type=out_type)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def size(fn, d):
    n = ctypes.c_size_t()
    assert fn(ctypes.byref(d), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=2), 1), (dict(scales=3), 1), (dict(scales=-1), 1),
    (dict(transpose=2), 1), (dict(scales=0, transpose=1), 1), (dict(flags=1), 1), (dict(rows=1 << 31), 2),
    (dict(cols=1 << 31), 2), (dict(rows=2_000_000_000, scales=0), 2)])
def test_quant_refusals(lib, change, code):
    assert lib.gdn_quant_e4m3(ctypes.byref(quant_desc(**change)), P, Q, R, None) == code


def test_quant_refused_buffers(lib):
    r = ctypes.byref(quant_desc())
    for args in ((None, Q, R), (P, None, R), (P, Q, None), (P, P, R), (P, Q, P), (P, Q, Q)):
        assert lib.gdn_quant_e4m3(r, *args, None) == 1
    assert lib.gdn_quant_e4m3(None, P, Q, R, None) == 1
    d = quant_desc()
    d.reserved[3] = 1
    assert lib.gdn_quant_e4m3(ctypes.byref(d), P, Q, R, None) == 1
    assert lib.gdn_quant_e4m3(ctypes.byref(quant_desc(rows=0)), None, None, None, None) == 0  # nothing to do


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=-1), 1), (dict(out_dtype=2), 1), (dict(scales=3), 1), (dict(flags=1), 1),
    (dict(M=1 << 31), 2), (dict(N=1 << 31), 2), (dict(K=1 << 31), 2)])
def test_matmul_refusals(lib, change, code):
    r = ctypes.byref(mm_desc(**change))
    assert lib.gdn_matmul_e4m3(r, P, Q, R, S, V, W, BIG, None) == code
    assert lib.gdn_matmul_e4m3_workspace_size(r, ctypes.byref(ctypes.c_size_t())) == code


def test_matmul_refused_buffers(lib):
    r = ctypes.byref(mm_desc())
    fn = lib.gdn_matmul_e4m3
    for i in range(5):
        args = [P, Q, R, S, V]
        args[i] = None
        assert fn(r, *args, W, BIG, None) == 1
    for i in range(4):
        args = [P, Q, R, S, V]
        args[4] = args[i]  # y is an input
        assert fn(r, *args, W, BIG, None) == 1
    assert fn(ctypes.byref(mm_desc(M=0)), None, None, None, None, None, None, 0, None) == 0
    assert lib.gdn_matmul_e4m3_workspace_size(r, None) == 1


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), 1), (dict(K=0), 1), (dict(F=0), 1), (dict(dtype=2), 1), (dict(activation=0), 1),
    (dict(activation=3), 1), (dict(out_type=2), 1), (dict(flags=1), 1), (dict(rows=1 << 31), 2), (dict(K=1 << 25), 2),
    (dict(F=1 << 25), 2)])
def test_ffn_refusals(lib, change, code):
    r, n = ctypes.byref(ffn_desc(**change)), ctypes.byref(ctypes.c_size_t())
    assert lib.gdn_gated_ffn_fwd(r, P, Q, R, S, None, X, BIG, None) == code
    assert lib.gdn_gated_ffn_bwd(r, P, Q, R, None, S, V, None, None, X, BIG, None) == code
    assert lib.gdn_gated_ffn_e4m3(r, P, Q, R, S, V, W, X, None, ctypes.c_void_p(0x100000), BIG, None) == code
    for fn in (lib.gdn_gated_ffn_fwd_workspace_size, lib.gdn_gated_ffn_bwd_workspace_size, lib.gdn_gated_ffn_e4m3_workspace_size):
        assert fn(r, n) == code


def test_ffn_refused_buffers(lib):
    r = ctypes.byref(ffn_desc())
    for i in range(4):
        args = [P, Q, R, S]
        args[i] = None
        assert lib.gdn_gated_ffn_fwd(r, *args, None, X, BIG, None) == 1
    for h in (P, Q, R):
        assert lib.gdn_gated_ffn_fwd(r, P, Q, R, h, None, X, BIG, None) == 1
    assert lib.gdn_gated_ffn_fwd(r, P, Q, R, S, S, X, BIG, None) == 1
    assert lib.gdn_gated_ffn_fwd(ctypes.byref(ffn_desc(out_type=1)), P, Q, R, S, None, X, BIG, None) == 1

    bwd, big = lib.gdn_gated_ffn_bwd, size(lib.gdn_gated_ffn_bwd_workspace_size, ffn_desc())
    assert big > 0
    assert bwd(r, P, Q, R, None, None, V, None, None, X, BIG, None) == 1             # no d_h
    assert bwd(r, P, Q, R, None, S, V, W, None, X, BIG, None) == 1                   # one weight's gradient alone
    assert bwd(r, P, Q, R, None, S, V, W, W, X, BIG, None) == 1                      # both in one place
    for out in (P, Q, R, S):
        assert bwd(r, P, Q, R, None, S, out, None, None, X, BIG, None) == 1
    assert bwd(r, P, Q, R, None, S, V, None, None, None, BIG, None) == 3
    assert bwd(r, P, Q, R, None, S, V, None, None, X, ctypes.c_size_t(big - 1), None) == 3
    assert bwd(r, P, Q, R, None, S, V, None, None, ctypes.c_void_p(0x70010), BIG, None) == 3

    f8, Y, Z = lib.gdn_gated_ffn_e4m3, ctypes.c_void_p(0x80000), ctypes.c_void_p(0x90000)
    q = ctypes.byref(ffn_desc(out_type=1))
    for i in range(7):
        args = [P, Q, R, S, V, W, X]
        args[i] = None
        assert f8(r, *args, None, Z, BIG, None) == 1
    assert f8(r, P, Q, R, S, V, W, X, Y, Z, BIG, None) == 1       # scales without 8 bits
    assert f8(q, P, Q, R, S, V, W, X, None, Z, BIG, None) == 1    # 8 bits without scales
    assert f8(q, P, Q, R, S, V, W, X, Q, Z, BIG, None) == 1       # h's scales in place of x's
    need = size(lib.gdn_gated_ffn_e4m3_workspace_size, ffn_desc(rows=1000, out_type=1))
    if need:
        assert f8(ctypes.byref(ffn_desc(rows=1000, out_type=1)), P, Q, R, S, V, W, X, Y, Z, ctypes.c_size_t(need - 1), None) == 3


def test_python_refuses_host_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    q = x.to(torch.float8_e4m3fn)
    one = torch.ones(4, 1)
    with pytest.raises(ValueError):
        gdn.gdn_quant_e4m3(x)
    with pytest.raises(ValueError):
        gdn.gdn_quant_e4m3(x, quant="column")
    with pytest.raises(ValueError):
        gdn.gdn_matmul_e4m3(q, one, q, one)
    with pytest.raises(ValueError):
        gdn.gdn_gated_ffn_fwd(x, w, w)
    with pytest.raises(ValueError):
        gdn.gdn_gated_ffn_e4m3(q, one, q, one, q, one)
    with pytest.raises(ValueError):
        gdn.linear_e4m3(x, w)
    with pytest.raises(ValueError):
        gdn.gated_ffn(x, w, w)
