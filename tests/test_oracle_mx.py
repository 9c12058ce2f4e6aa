"""The microscaled oracle against values worked out by hand, and the library's
refusals for these formats (no kernel is launched here)."""
import ctypes

import numpy as np
import pytest

from oracle import mx

qb = pytest.importorskip("bit_nf4_quantized_encode_b200")
lib = qb._lib
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUP, ERR_CUDA, ERR_WS = 0, -1, -2, -3, -4, -5, -6


def test_nearest_code_ties_go_to_the_even_code():
    v = np.array([0.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.9])
    assert mx.nearest_code(v).tolist() == [0, 0, 1, 2, 1, 2, 4, 4, 6, 6, 7, 7]


def test_e4m3_levels():
    lv = mx.e4m3_levels()
    assert lv[1] == 2.0 ** -9 and lv[8] == 2.0 ** -6 and lv[126] == 448.0 and np.all(np.diff(lv) > 0)
    assert mx.nearest_e4m3(np.array([0.0, 2.0 ** -10, 2.0 ** -10 * 1.01, 448.0, 17.0, 19.0])).tolist() == \
        [0, 0, 1, 126, 88, 90]                       # 16, 18, 20 are bytes 88, 89, 90


def test_mxfp4_block_by_hand():
    x = np.zeros((1, 40))
    x[0, :4] = [7.0, -5.0, 0.5, 0.26]                # amax 7: E = 0
    x[0, 32:] = [0.03125] * 8                        # amax 2^-5: E = -7, 2^-5 / 2^-7 = 4
    codes, sb, g = mx.quantize(x, "mxfp4")
    assert g is None and sb.tolist() == [[127, 120]]
    assert codes[0, :4].tolist() == [7, 14, 1, 1] and codes[0, 32:].tolist() == [6] * 8


def test_nvfp4_global_scale_by_hand():
    assert mx.global_scale(2688.0) == 1.0 and mx.global_scale(2689.0) == 2.0 and mx.global_scale(0.0) == 1.0
    assert mx.global_scale(2.0 ** -133) == 2.0 ** -126
    x = np.full((1, 16), 6.0)                        # g = 2^-8: 6 <= 2688 g; S = e4m3(256) = 256, code of 6
    codes, sb, g = mx.quantize(x, "nvfp4")
    assert g.tolist() == [2.0 ** -8] and mx.e4m3_levels()[sb[0, 0]] == 256 and codes.tolist() == [[7] * 16]


@pytest.mark.parametrize("fmt,per_row", [("mxfp4", False), ("nvfp4", False), ("nvfp4", True)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (100, 1000), (129, 64), (4096, 11008)])
def test_sizes(fmt, per_row, rows, cols):
    sz = qb.qlora_mx_sizes(rows, cols, fmt, per_row)
    assert sz["codes"] == rows * -(-cols // 32) * 16
    assert sz["scales"] == mx.tile_scales(np.zeros((rows, -(-cols // mx.BLOCK[fmt])), np.uint8)).size
    assert sz["global_scale"] == (0 if fmt == "mxfp4" else 4 * (rows if per_row else 1))
    assert (sz["codes"], sz["scales"]) == qb._mx_bytes(rows, cols, fmt)


def _t(rows=64, cols=64, fmt=0, per_row=0, base=0x10000):
    return qb._MxTensorC(base, base + 0x10000, base + 0x20000, rows, cols, fmt, per_row)


def test_size_refusals():
    f = lib.qlora_mx_sizes
    assert f(-1, 4, 0, 0, None, None, None, None) == ERR_SHAPE
    assert f(4, 1 << 31, 0, 0, None, None, None, None) == ERR_SHAPE
    assert f(4, 4, 2, 0, None, None, None, None) == ERR_UNSUP
    assert f(4, 4, 0, 1, None, None, None, None) == ERR_UNSUP        # a scale per row is NVFP4's
    assert f(4, 4, 1, 2, None, None, None, None) == ERR_UNSUP


def test_quantize_refusals():
    f, w, ws = lib.qlora_mx_quantize, 0x100000, 0x200000
    assert f(w, 0, None, ws, 1 << 20, None) == ERR_NULL
    assert f(None, 0, _t(), ws, 1 << 20, None) == ERR_NULL
    assert f(w + 2, 0, _t(), ws, 1 << 20, None) == ERR_ALIGN
    assert f(w, 2, _t(), ws, 1 << 20, None) == ERR_UNSUP
    assert f(w, 1, _t(fmt=1, per_row=1), ws, 1 << 20, None) == ERR_UNSUP
    assert f(w, 0, _t(fmt=2), ws, 1 << 20, None) == ERR_UNSUP
    assert f(w, 0, _t(per_row=1), ws, 1 << 20, None) == ERR_UNSUP
    assert f(w, 0, _t(rows=-1), ws, 1 << 20, None) == ERR_SHAPE
    big = _t(rows=1024, cols=1024, fmt=1)
    assert f(w, 0, big, None, 0, None) == ERR_NULL                   # one global scale needs the work buffer
    assert f(w, 0, big, ws, 64, None) == ERR_WS
    assert f(w, 0, big, ws + 4, 1 << 20, None) == ERR_ALIGN
    assert qb.qlora_mx_sizes(1024, 1024, "nvfp4")["workspace"] and not qb.qlora_mx_sizes(100, 1000, "nvfp4")["workspace"]
    for field in ("codes", "scales", "global_scale"):
        nul, mis = _t(fmt=1), _t(fmt=1)
        setattr(nul, field, None)
        setattr(mis, field, getattr(mis, field) + 8)
        assert f(w, 0, nul, ws, 1 << 20, None) == ERR_NULL
        assert f(w, 0, mis, ws, 1 << 20, None) == ERR_ALIGN
    assert f(None, 0, _t(rows=0), None, 0, None) == OK


def test_dequantize_refusals():
    f = lib.qlora_mx_dequantize
    assert f(None, 0x1000, None) == ERR_NULL
    assert f(_t(), None, None) == ERR_NULL
    assert f(_t(), 0x1002, None) == ERR_ALIGN
    assert f(_t(cols=0), None, None) == OK


def test_binding_refuses_buffers_that_do_not_hold_the_matrix():
    import torch
    cpu = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        qb.MXTensor(cpu, cpu, None, 4, 32).c_struct()
    with pytest.raises(ValueError, match="fmt"):
        qb.MXTensor(cpu, cpu, None, 4, 32, "fp4").c_struct()
    with pytest.raises(ValueError, match="nvfp4"):
        qb.empty_mx(4, 4, "cpu", "mxfp4", per_row=True)
    with pytest.raises(ValueError, match="bf16"):
        qb.qlora_mx_quantize(torch.zeros(4, 32))


def test_linear_refusals():
    p, s = 0x100000, ctypes.c_float(0.5)
    f, b, size = lib.qlora_mx_linear_fwd, lib.qlora_mx_linear_bwd, lib.qlora_mx_linear_workspace_size
    W = _t(64, 128)
    args = lambda w=W, x=p, m=4, a=p, bb=p, r=8, y=p, xa=None, ws=p, n=1 << 40: (w, x, m, a, bb, r, s, y, xa, ws, n, None)  # noqa: E731
    assert f(*args(w=None)) == ERR_NULL and f(*args(x=None)) == ERR_NULL and f(*args(a=None)) == ERR_NULL
    assert f(*args(x=p + 2)) == ERR_ALIGN and f(*args(xa=p + 4)) == ERR_ALIGN and f(*args(y=p + 8)) == ERR_ALIGN
    assert f(*args(m=0)) == ERR_SHAPE and f(*args(r=12)) == ERR_SHAPE and f(*args(r=264)) == ERR_SHAPE
    assert f(*args(r=-8)) == ERR_SHAPE
    assert f(*args(w=_t(64, 72))) == ERR_SHAPE and f(*args(w=_t(60, 128))) == ERR_SHAPE
    assert f(*args(w=_t(0, 128))) == ERR_SHAPE and f(*args(w=_t(64, 128, 7))) == ERR_UNSUP
    assert f(*args(w=_t(64, 128, 1, 1))) == ERR_UNSUP                     # a scale per weight row with an adapter
    far = _t((1 << 31) - 256, (1 << 31) - 256)                           # more scale tiles than 32 bits count
    assert f(far, p, 4, None, None, 0, s, p, None, p, 1 << 62, None) == ERR_SHAPE
    assert b(far, None, p, 4, None, None, 0, s, None, p, None, None, p, 1 << 62, None) == ERR_SHAPE
    assert f(*args(n=64)) == ERR_WS and f(W, p, 4, None, None, 0, s, p, None, p, 64, None) == ERR_WS
    assert f(W, p, 4, p, p, 8, ctypes.c_float(float("inf")), p, None, p, 1 << 40, None) == ERR_SHAPE
    bargs = lambda dx=p, da=p, x=p, r=8, xa=None, n=1 << 40: (W, x, p, 4, p, p, r, s, xa, dx, da, p, p, n, None)  # noqa: E731
    assert b(*bargs(dx=None, r=0)) == ERR_NULL and b(*bargs(da=None)) == ERR_NULL and b(*bargs(x=None)) == ERR_NULL
    assert b(*bargs(xa=p + 2)) == ERR_ALIGN and b(*bargs(n=64)) == ERR_WS
    assert size(64, 128, 3, 4, 8, None, None) == ERR_UNSUP and size(64, 100, 0, 4, 8, None, None) == ERR_SHAPE
    assert size(64, 100, 0, 4, 0, None, None) == OK and size(0, 100, 0, 4, 0, None, None) == ERR_SHAPE


def test_moe_refusals():
    p = 0x100000
    f, size = lib.qlora_mx_moe_fwd, lib.qlora_mx_moe_workspace_size
    W13, W2 = _t(4 * 2 * 128, 256), _t(4 * 256, 128)
    args = lambda a=W13, b=W2, r=p, e=4, x=p, m=3, k=2, y=p, ids=p, pr=p, ws=p, n=1 << 40: \
        (a, b, r, e, x, m, k, y, ids, pr, ws, n, None)  # noqa: E731
    for key in ("a", "b", "r", "x", "y", "ids", "pr", "ws"):
        assert f(*args(**{key: None})) == ERR_NULL
    for key in ("r", "x", "y", "ids", "pr", "ws"):
        assert f(*args(**{key: p + 4})) == ERR_ALIGN
    for kw in (dict(m=0), dict(m=17), dict(k=0), dict(k=5), dict(e=0), dict(e=5), dict(a=_t(1024, 200)), dict(b=_t(1024, 120)),
               dict(b=_t(1000, 128))):
        assert f(*args(**kw)) == ERR_SHAPE, kw
    assert f(*args(a=_t(1024, 256, 1))) == ERR_UNSUP
    assert f(*args(n=64)) == ERR_WS
    assert size(257, 256, 128, 1, 1, None) == ERR_SHAPE and size(32, 256, 128, 1, 17, None) == ERR_SHAPE
    assert size(4, 256, 128, 16, 4, None) == OK
