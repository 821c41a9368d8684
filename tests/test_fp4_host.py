"""Argument checks of the 4-bit entry points: they answer before anything is launched, so this
file needs no GPU (the pointers are never dereferenced)."""

import ctypes

import pytest

import tenant_serving_b200 as bd

P = ctypes.c_void_p(0x1000)      # aligned
M = ctypes.c_void_p(0x1008)      # 8-byte aligned
U = ctypes.c_void_p(0x1002)      # 2-byte aligned
BIG = 1 << 40
NV, MX = bd.BD_FP4_NV, bd.BD_FP4_MX


@pytest.fixture(scope="module")
def lib():
    from tenant_serving_b200 import build
    build.build()
    return bd.lib()


def test_scale_bytes(lib):
    f = bd.bd_fp4_scales_bytes
    assert f(1, 32, NV) == 512 and f(128, 64, NV) == 512 and f(129, 64, NV) == 1024 and f(128, 96, NV) == 1024
    assert f(1, 32, MX) == 512 and f(128, 128, MX) == 512 and f(128, 160, MX) == 1024
    assert f(14336, 4096, NV) == 14336 * 4096 // 16
    for rows, cols, fmt in ((0, 64, NV), (4, 48, NV), (4, 0, MX), (4, 64, 2), (4, 64, -1), ((1 << 24) + 1, 64, NV),
                            (4, (1 << 24) + 32, NV)):
        assert f(rows, cols, fmt) == 0
    assert bd.fp4_scales_shape(300, 416, NV) == (3, 7, 512)


def _quant(lib, x=P, dtype=bd.BD_BF16, rows=8, cols=64, ld=64, fmt=NV, codes=P, scales=P, row=P, hat=P,
           hat_dtype=bd.BD_F32):
    return lib.bd_quantize_fp4(x, dtype, rows, cols, ld, fmt, codes, scales, row, hat, hat_dtype, None)


@pytest.mark.parametrize("kw,code", [
    ({"dtype": 3}, bd.BD_ERR_DTYPE), ({"hat_dtype": bd.BD_F16}, bd.BD_ERR_DTYPE), ({"fmt": 2}, bd.BD_ERR_CONFIG),
    ({"rows": 0}, bd.BD_ERR_SHAPE), ({"cols": 40, "ld": 40}, bd.BD_ERR_SHAPE), ({"cols": 0}, bd.BD_ERR_SHAPE),
    ({"ld": 56}, bd.BD_ERR_SHAPE), ({"ld": (1 << 31) + 8}, bd.BD_ERR_SHAPE), ({"x": None}, bd.BD_ERR_NULL),
    ({"codes": None}, bd.BD_ERR_NULL), ({"scales": None}, bd.BD_ERR_NULL), ({"row": None}, bd.BD_ERR_NULL),
    ({"x": M}, bd.BD_ERR_ALIGN), ({"ld": 68}, bd.BD_ERR_ALIGN), ({"codes": M}, bd.BD_ERR_ALIGN),
    ({"scales": M}, bd.BD_ERR_ALIGN), ({"row": U}, bd.BD_ERR_ALIGN), ({"hat": M}, bd.BD_ERR_ALIGN)])
def test_quantize_refusals(lib, kw, code):
    assert _quant(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    ({"dt": bd.BD_F16}, bd.BD_ERR_DTYPE), ({"fmt": 7}, bd.BD_ERR_CONFIG), ({"rows": 0}, bd.BD_ERR_SHAPE),
    ({"cols": 33}, bd.BD_ERR_SHAPE), ({"c": None}, bd.BD_ERR_NULL), ({"s": None}, bd.BD_ERR_NULL),
    ({"out": None}, bd.BD_ERR_NULL), ({"c": M}, bd.BD_ERR_ALIGN), ({"s": M}, bd.BD_ERR_ALIGN),
    ({"r": U}, bd.BD_ERR_ALIGN), ({"out": M}, bd.BD_ERR_ALIGN)])
def test_dequantize_refusals(lib, kw, code):
    a = {"c": P, "s": P, "r": P, "fmt": NV, "rows": 4, "cols": 64, "out": P, "dt": bd.BD_F32} | kw
    assert lib.bd_dequantize_fp4(a["c"], a["s"], a["r"], a["fmt"], a["rows"], a["cols"], a["out"], a["dt"], None) == code


@pytest.mark.parametrize("kw,code", [
    ({"fmt": 2}, bd.BD_ERR_CONFIG), ({"rows": 0}, bd.BD_ERR_SHAPE), ({"cols": 31}, bd.BD_ERR_SHAPE),
    ({"s": None}, bd.BD_ERR_NULL), ({"out": None}, bd.BD_ERR_NULL), ({"out": M}, bd.BD_ERR_ALIGN)])
def test_prepare_scales_refusals(lib, kw, code):
    a = {"s": P, "fmt": NV, "rows": 4, "cols": 64, "out": P} | kw
    assert lib.bd_prepare_fp4_scales(a["s"], a["fmt"], a["rows"], a["cols"], a["out"], None) == code


PRODUCT = [
    ({"dt": bd.BD_F16}, bd.BD_ERR_DTYPE), ({"fmt": 2}, bd.BD_ERR_CONFIG), ({"fmt": -1}, bd.BD_ERR_CONFIG),
    ({"d_out": 0}, bd.BD_ERR_SHAPE), ({"d_in": 80}, bd.BD_ERR_SHAPE), ({"d_in": 0}, bd.BD_ERR_SHAPE),
    ({"t": -1}, bd.BD_ERR_SHAPE), ({"t": 65537}, bd.BD_ERR_SHAPE), ({"d_out": (1 << 24) + 1}, bd.BD_ERR_SHAPE),
    ({"wc": None}, bd.BD_ERR_NULL), ({"ws": None}, bd.BD_ERR_NULL), ({"x": None}, bd.BD_ERR_NULL),
    ({"y": None}, bd.BD_ERR_NULL), ({"wc": M}, bd.BD_ERR_ALIGN), ({"ws": M}, bd.BD_ERR_ALIGN),
    ({"wr": U}, bd.BD_ERR_ALIGN), ({"x": M}, bd.BD_ERR_ALIGN), ({"y": M}, bd.BD_ERR_ALIGN),
    ({"work": None}, bd.BD_ERR_WORKSPACE), ({"wb": 16}, bd.BD_ERR_WORKSPACE), ({"work": M}, bd.BD_ERR_ALIGN),
    ({"t": 0, "x": None, "work": None}, bd.BD_OK)]
DEFAULTS = {"wc": P, "ws": P, "wr": P, "x": P, "xs": P, "xr": P, "fmt": NV, "d_out": 8, "d_in": 64, "t": 4, "y": P,
            "dt": bd.BD_BF16, "work": P, "wb": BIG}


@pytest.mark.parametrize("kw,code", PRODUCT + [({"xs": None}, bd.BD_ERR_NULL), ({"xs": M}, bd.BD_ERR_ALIGN),
                                               ({"xr": U}, bd.BD_ERR_ALIGN)])
def test_matmul_refusals(lib, kw, code):
    a = DEFAULTS | kw
    assert lib.bd_matmul_fp4(a["wc"], a["ws"], a["wr"], a["x"], a["xs"], a["xr"], a["fmt"], a["d_out"], a["d_in"],
                             a["t"], a["y"], a["dt"], a["work"], a["wb"], None) == code


@pytest.mark.parametrize("kw,code", PRODUCT)
def test_linear_refusals(lib, kw, code):
    a = DEFAULTS | kw
    assert lib.bd_linear_fp4(a["wc"], a["ws"], a["wr"], a["fmt"], a["d_out"], a["d_in"], a["x"], a["t"], a["y"],
                             a["dt"], a["work"], a["wb"], None) == code


@pytest.mark.parametrize("kw,code", PRODUCT + [
    ({"ids": None}, bd.BD_ERR_NULL), ({"n": 16385}, bd.BD_ERR_SHAPE), ({"n": -1}, bd.BD_ERR_SHAPE),
    ({"sdt": bd.BD_BF16}, bd.BD_ERR_DTYPE), ({"ids": M}, bd.BD_ERR_ALIGN), ({"tab": None}, bd.BD_ERR_NULL)])
def test_apply_refusals(lib, kw, code):
    a = DEFAULTS | {"ids": P, "n": 2, "sdt": bd.BD_F16, "tab": P} | kw
    assert lib.bd_apply_multi_fp4(a["wc"], a["ws"], a["wr"], a["fmt"], a["d_out"], a["d_in"], a["tab"], a["n"],
                                  a["sdt"], a["ids"], a["x"], a["t"], a["y"], a["dt"], a["work"], a["wb"],
                                  None) == code


def test_workspace_sizes(lib):
    assert bd.bd_matmul_fp4_workspace_size(8, 64, 4) >= 16
    # the limbs of 512 tokens, four or six rows of codes each
    assert bd.bd_linear_fp4_workspace_size(4096, 4096, 512) >= 512 * 6 * 2048
    assert bd.bd_linear_fp4_workspace_size(4096, 4096, 65536) > bd.bd_linear_fp4_workspace_size(4096, 4096, 512)
    for bad in ((0, 64, 4), (8, 48, 4), (8, 64, -1), (8, 64, 65537)):
        assert bd.bd_linear_fp4_workspace_size(*bad) == 0
    assert bd.bd_apply_fp4_workspace_size(4096, 4096, 512, 10) >= 512 * 4096 * 4
    # sizes that the call accepts are the ones it was told
    n = bd.bd_linear_fp4_workspace_size(8, 64, 4)
    lib = bd.lib()
    assert lib.bd_linear_fp4(P, P, P, NV, 8, 64, P, 4, P, bd.BD_F32, P, n // 4, None) == bd.BD_ERR_WORKSPACE


def test_wrappers_refuse_cpu_tensors():
    import torch
    c, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((1, 1, 512), dtype=torch.uint8)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: bd.bd_quantize_fp4(x, NV), lambda: bd.bd_dequantize_fp4(c, s, None, NV),
                 lambda: bd.bd_linear_fp4(c, s, None, x, NV), lambda: bd.bd_matmul_fp4(c, s, None, c, s, None, NV),
                 lambda: bd.bd_prepare_fp4_scales(c, NV, 4, 64)):
        with pytest.raises(ValueError):
            call()
