"""Outputs of the layer's products in the place of one of their inputs are refused before anything is launched (no GPU)."""
import ctypes

import pytest

from test_product_abi import BIG, ffn_desc, lib, mm_desc  # noqa: F401

ARGS = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(10)]


@pytest.mark.parametrize("dtype", [0, 1])
def test_ffn_pre_is_no_input(lib, dtype):  # noqa: F811
    x, wg, wu, h, pre, ws = ARGS[:6]
    need = ctypes.c_size_t()
    d = ffn_desc(rows=0, dtype=dtype)
    assert lib.gdn_gated_ffn_fwd_workspace_size(ctypes.byref(d), ctypes.byref(need)) == 0
    assert lib.gdn_gated_ffn_fwd(ctypes.byref(d), x, wg, wu, h, pre, ws, BIG, None) == 0  # nothing to do
    d = ffn_desc(dtype=dtype)
    for taken in (x, wg, wu, h):
        assert lib.gdn_gated_ffn_fwd(ctypes.byref(d), x, wg, wu, h, taken, ws, BIG, None) == 1


def test_ffn8_outputs_are_no_inputs(lib):  # noqa: F811
    x, xs, wg, gs, wu, us, h, hs, ws = ARGS[:9]
    fn = lib.gdn_gated_ffn_e4m3
    assert fn(ctypes.byref(ffn_desc(rows=0, out_type=1)), x, xs, wg, gs, wu, us, h, hs, ws, BIG, None) == 0
    quant, plain = (ctypes.byref(ffn_desc(out_type=t)) for t in (1, 0))
    for taken in (x, xs, wg, gs, wu, us):
        assert fn(quant, x, xs, wg, gs, wu, us, taken, hs, ws, BIG, None) == 1
        assert fn(plain, x, xs, wg, gs, wu, us, taken, None, ws, BIG, None) == 1
        assert fn(quant, x, xs, wg, gs, wu, us, h, taken, ws, BIG, None) == 1
    assert fn(quant, x, xs, wg, gs, wu, us, h, h, ws, BIG, None) == 1


def test_flags(lib):  # noqa: F811
    """Exact sums may be asked for where the operands are e4m3, and nothing else."""
    n = ctypes.byref(ctypes.c_size_t())
    for flags, code in ((0, 0), (256, 0), (128, 1), (257, 1), (-1, 1)):
        assert lib.gdn_matmul_e4m3_workspace_size(ctypes.byref(mm_desc(flags=flags)), n) == code
        assert lib.gdn_gated_ffn_e4m3_workspace_size(ctypes.byref(ffn_desc(flags=flags)), n) == code
        assert lib.gdn_gated_ffn_fwd_workspace_size(ctypes.byref(ffn_desc(flags=flags)), n) == (1 if flags else 0)
        assert lib.gdn_gated_ffn_bwd_workspace_size(ctypes.byref(ffn_desc(flags=flags)), n) == (1 if flags else 0)


def test_flag_of_pairs(lib):  # noqa: F811
    """Pairs of bf16 at any size may be asked of the block's backward, and of nothing else; they want a larger workspace."""
    n = ctypes.c_size_t()
    sizes = {}
    for dtype in (0, 1):
        for flags in (0, 512):
            d = ffn_desc(rows=700, K=800, F=900, dtype=dtype, flags=flags)
            assert lib.gdn_gated_ffn_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
            sizes[dtype, flags] = n.value
            assert lib.gdn_gated_ffn_fwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == (1 if flags else 0)
            assert lib.gdn_gated_ffn_e4m3_workspace_size(ctypes.byref(d), ctypes.byref(n)) == (1 if flags else 0)
    assert sizes[0, 512] >= sizes[0, 0] + 2 * 700 * 900 * 2 and sizes[1, 512] == sizes[1, 0]
    assert lib.gdn_gated_ffn_bwd_workspace_size(ctypes.byref(ffn_desc(flags=513)), ctypes.byref(n)) == 1
    x, wg, wu, d_h, dx, ws = ARGS[:6]
    d = ffn_desc(rows=700, K=800, F=900, flags=512)
    assert lib.gdn_gated_ffn_bwd(ctypes.byref(d), x, wg, wu, None, d_h, dx, None, None, ws, ctypes.c_size_t(sizes[0, 512] - 1), None) == 3
