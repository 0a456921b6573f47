"""Refusals of the calls over rows in 8 bits that need no GPU: every bad argument is refused
before the device is touched, in C and in the binding."""
import ctypes

import pytest
import torch

c = ctypes
F16, F32, F64, BF16 = 0, 1, 2, 3
A, B, C, D, E, G, H, W = (0x100000 * i for i in range(1, 9))    # never dereferenced: the call fails first


@pytest.fixture(scope="module")
def lib():
    import fac_second_order_amd._lib as L
    return L


def i64(*v):
    return (c.c_int64 * max(1, len(v)))(*v)


def i32(*v):
    return (c.c_int32 * max(1, len(v)))(*v)


def ptrs(*v):
    return (c.c_void_p * max(1, len(v)))(*v)


def quantize(so, rows=4, cols=8, dt=F16, x=A, ldx=8, mask=None, pow2=1, q=B, ldq=8, s=C):
    return so.kfac_quantize_rows(rows, cols, dt, x, ldx, mask, pow2, q, ldq, s, None)


def test_quantize_refusals(lib):
    so = lib._lib
    past = quantize(so)
    assert past not in (0, -1)                    # good arguments stop at the device
    assert quantize(so, rows=-1) == -1 and quantize(so, cols=-1) == -1
    assert quantize(so, dt=F64) == -2 and quantize(so, dt=9) == -2
    assert quantize(so, x=None) == -1 and quantize(so, q=None) == -1 and quantize(so, s=None) == -1
    assert quantize(so, x=A + 1) == -1 and quantize(so, dt=F32, x=A + 2) == -1 and quantize(so, s=C + 2) == -1
    assert quantize(so, x=A + 2) == past and quantize(so, q=B + 1) == past
    assert quantize(so, ldx=7) == -1 and quantize(so, ldq=7) == -1 and b"overlap" in so.kfac_last_error()
    assert quantize(so, rows=1, ldx=0, ldq=0) == past
    assert quantize(so, pow2=2) == -1 and quantize(so, pow2=0) == past
    assert quantize(so, q=A + 10) == -1 and quantize(so, s=A + 16) == -1 and quantize(so, s=B + 28) == -1
    assert quantize(so, s=B + 32) == past
    assert quantize(so, mask=B + 3) == -1 and quantize(so, mask=C + 15) == -1 and quantize(so, mask=A) == past
    assert quantize(so, ldx=64, ldq=128, q=A + 16) == past    # rows between each other's
    assert quantize(so, ldx=64, ldq=128, q=A + 15) == -1
    assert quantize(so, rows=0, x=None, q=None, s=None) == past


def dequantize(so, rows=4, cols=8, q=A, ldq=8, s=B, dt=BF16, x=C, ldx=8):
    return so.kfac_dequantize_rows(rows, cols, q, ldq, s, dt, x, ldx, None)


def test_dequantize_refusals(lib):
    so = lib._lib
    past = dequantize(so)
    assert past not in (0, -1)
    assert dequantize(so, rows=-1) == -1 and dequantize(so, dt=F64) == -2
    for k in ("q", "s", "x"):
        assert dequantize(so, **{k: None}) == -1
    assert dequantize(so, s=B + 1) == -1 and dequantize(so, x=C + 1) == -1
    assert dequantize(so, ldq=7) == -1 and dequantize(so, ldx=7) == -1
    assert dequantize(so, x=A) == -1 and dequantize(so, x=B + 8) == -1
    assert dequantize(so, cols=0, q=None, s=None, x=None) == past


def linear(so, rows=4, c_in=8, c_out=6, dt=BF16, x=A, ldx=8, mask=None, q=B, ldq=8, s=C, w=D, ldw=8, v=E, b=G, y=H, ldy=6,
           ws=W, wsb=1 << 19):
    return so.kfac_linear_q8(rows, c_in, c_out, dt, x, ldx, mask, q, ldq, s, w, ldw, v, b, y, ldy, ws, wsb, None)


def test_linear_refusals(lib):
    so, sz = lib._lib, c.c_size_t()
    past = linear(so)
    assert past not in (0, -1)
    for k in ("rows", "c_in", "c_out"):
        assert linear(so, **{k: -1}) == -1
    assert linear(so, c_in=1 << 17, ldx=1 << 17, ldq=1 << 17, ldw=1 << 17) == -2
    assert so.kfac_linear_q8_workspace(1, 1 << 17, 1, c.byref(sz)) == -2
    assert so.kfac_linear_q8_workspace(1, -1, 1, c.byref(sz)) == -1
    assert so.kfac_linear_q8_workspace(1, 1, 1, None) == -1
    assert so.kfac_linear_q8_workspace(1, (1 << 17) - 1, 1, c.byref(sz)) == 0
    assert linear(so, dt=F64) == -2
    for k in ("q", "s", "w", "v", "y"):
        assert linear(so, **{k: None}) == -1
    assert linear(so, x=None) == past and linear(so, b=None) == past
    assert linear(so, x=None, mask=A) == -1
    for k in ("ldx", "ldq", "ldw"):
        assert linear(so, **{k: 7}) == -1
    assert linear(so, ldy=5) == -1 and linear(so, y=H + 1) == -1 and linear(so, b=G + 1) == -1 and linear(so, v=E + 2) == -1
    for at in (A, B, C, D, E, G):
        assert linear(so, y=at) == -1
    assert linear(so, q=A) == -1 and linear(so, q=D) == -1 and linear(so, s=E) == -1 and linear(so, s=B + 4) == -1
    assert linear(so, mask=B) == -1 and linear(so, mask=C) == -1 and linear(so, mask=H) == -1 and linear(so, mask=A) == past
    assert linear(so, x=None, q=D) == past         # given codes are inputs
    assert linear(so, ws=W + 4) in (past, -3)


def grad(so, rows=4, c_in=8, c_out=6, dt=F16, g=A, ldg=6, q=B, ldq=8, s=C, dw=D, ldw=9, db=D + 32, inc=9, acc=0, ws=W,
         wsb=1 << 19):
    return so.kfac_weight_grad_q8(rows, c_in, c_out, dt, g, ldg, q, ldq, s, dw, ldw, db, inc, acc, ws, wsb, None)


def test_weight_grad_refusals(lib):
    so, sz = lib._lib, c.c_size_t()
    past = grad(so)
    assert past not in (0, -1)
    for k in ("rows", "c_in", "c_out"):
        assert grad(so, **{k: -1}) == -1
    assert grad(so, dt=F64) == -2 and so.kfac_weight_grad_q8_workspace(1, 1, 1, F64, c.byref(sz)) == -2
    assert so.kfac_weight_grad_q8_workspace(1, 1, 1, F16, None) == -1
    assert so.kfac_weight_grad_q8_workspace(-1, 1, 1, F16, c.byref(sz)) == -1
    assert so.kfac_weight_grad_q8_workspace(1, 1 << 30, 1 << 30, F16, c.byref(sz)) == -2
    for k in ("g", "q", "s", "dw"):
        assert grad(so, **{k: None}) == -1
    assert grad(so, db=None) == past
    assert grad(so, g=A + 1) == -1 and grad(so, s=C + 1) == -1 and grad(so, dw=D + 2) == -1 and grad(so, db=E + 2) == -1
    assert grad(so, ldg=5) == -1 and grad(so, ldq=7) == -1 and grad(so, ldw=7) == -1 and grad(so, db=E, inc=0) == -1
    assert grad(so, acc=2) == -1 and grad(so, acc=1) == past
    assert grad(so, db=D + 28) == -1                 # inside the rows of dweight
    assert grad(so, ldw=8) == -1                     # then the column behind them is the next row's first
    for at in (A, B, C):
        assert grad(so, dw=at, db=None) == -1 and grad(so, db=at) == -1
    assert grad(so, rows=0, g=None, q=None, s=None) == past


def factors(so, rows=(4,), cols=(8,), bias=(1,), q=(A,), ld=(8,), s=(B,), A_packed=(C,), full=None, decay=0.0, ws=W,
            wsb=1 << 19, count=None):
    return so.kfac_factors_q8(len(rows) if count is None else count, i32(*rows), i32(*cols), i32(*bias), ptrs(*q), i64(*ld),
                              ptrs(*s), ptrs(*A_packed), None if full is None else ptrs(*full), c.c_float(decay), ws, wsb, None)


def test_factors_refusals(lib):
    so, sz = lib._lib, c.c_size_t()
    past = factors(so)
    assert past not in (0, -1)
    for decay in (-0.1, 1.1, float("nan")):
        assert factors(so, decay=decay) == -1
    assert factors(so, count=-1) == -1 and factors(so, rows=(-1,)) == -1 and factors(so, cols=(0,)) == -1
    assert factors(so, bias=(2,)) == -1
    assert factors(so, q=(None,)) == -1 and factors(so, s=(None,)) == -1 and factors(so, A_packed=(None,)) == -1
    assert factors(so, ld=(7,)) == -1 and factors(so, s=(B + 2,)) == -1 and factors(so, A_packed=(C + 2,)) == -1
    assert factors(so, full=(D + 2,)) == -1 and factors(so, full=(None,)) == past and factors(so, full=(D,)) == past
    assert factors(so, full=(C,)) == -1 and factors(so, A_packed=(A,)) == -1 and factors(so, full=(B,)) == -1
    two = dict(rows=(4, 4), cols=(8, 8), bias=(0, 1), q=(A, A), ld=(8, 8), s=(B, B))
    assert factors(so, A_packed=(C, C + 36 * 4), **two) == past      # one checkpoint read twice
    assert factors(so, A_packed=(C, C + 35 * 4), **two) == -1
    assert so.kfac_factors_q8_workspace(1, i32(4), i32(8), i32(1), None) == -1
    assert so.kfac_factors_q8_workspace(1, None, i32(8), i32(1), c.byref(sz)) == -1
    assert so.kfac_factors_q8_workspace(1, i32(4), i32(1 << 30), i32(1), c.byref(sz)) == -2
    assert so.kfac_factors_q8_workspace(0, None, None, None, c.byref(sz)) == 0


def test_workspace_is_apart(lib):
    """A workspace that a result lies in is refused, by the bytes that the call uses of it."""
    so, sz = lib._lib, c.c_size_t()
    assert so.kfac_factors_q8_workspace(1, i32(5000), i32(64), i32(1), c.byref(sz)) == 0 and sz.value > 0
    big = dict(rows=(5000,), cols=(64,), ld=(64,), q=(0x40000000,), s=(0x50000000,), ws=0x60000000, wsb=1 << 28)
    past = factors(so, A_packed=(0x60000000 + sz.value,), **big)
    assert past not in (0, -1)
    assert factors(so, A_packed=(0x60000000 + sz.value - 4,), **big) == -1
    assert so.kfac_weight_grad_q8_workspace(5000, 64, 64, F16, c.byref(sz)) == 0 and sz.value > 0
    big = dict(rows=5000, c_in=64, c_out=64, g=0x30000000, ldg=64, q=0x40000000, ldq=64, s=0x50000000, ldw=64, db=None,
               ws=0x60000000, wsb=1 << 28)
    assert grad(so, dw=0x60000000 + sz.value, **big) == past
    assert grad(so, dw=0x60000000 + sz.value - 4, **big) == -1
    assert grad(so, dw=D, **{**big, "g": 0x60000000}) == -1


# the binding -------------------------------------------------------------------

def rows(r, k, dt):
    return torch.zeros(r, k, dtype=dt)


I8, H16, F = torch.int8, torch.float16, torch.float32


@pytest.mark.parametrize("call", [
    lambda L: L.kfac_quantize_rows(rows(4, 8, torch.float64), rows(4, 8, I8), torch.zeros(4)),
    lambda L: L.kfac_quantize_rows(torch.zeros(4, 8, 2), rows(4, 8, I8), torch.zeros(4)),
    lambda L: L.kfac_quantize_rows(rows(8, 4, F).T, rows(4, 8, I8), torch.zeros(4)),
    lambda L: L.kfac_quantize_rows(rows(4, 8, F), rows(4, 8, torch.uint8), torch.zeros(4)),
    lambda L: L.kfac_quantize_rows(rows(4, 8, F), rows(4, 8, I8), torch.zeros(4, dtype=torch.float64)),
    lambda L: L.kfac_quantize_rows(rows(4, 8, F), rows(4, 8, I8), torch.zeros(5)),
    lambda L: L.kfac_quantize_rows(rows(4, 8, F), rows(4, 8, I8), torch.zeros(4), mask=torch.ones(4)),
    lambda L: L.kfac_quantize_rows(torch.zeros(4, 1, dtype=F).expand(4, 8), rows(4, 8, I8), torch.zeros(4)),
    lambda L: L.kfac_dequantize_rows(rows(4, 8, I8), torch.zeros(4), rows(4, 8, I8)),
    lambda L: L.kfac_linear_q8(rows(4, 8, F), rows(4, 8, I8), torch.zeros(4), rows(6, 8, I8), torch.zeros(6), rows(4, 6, H16)),
    lambda L: L.kfac_linear_q8(rows(4, 7, F), rows(4, 8, I8), torch.zeros(4), rows(6, 8, I8), torch.zeros(6), rows(4, 6, F)),
    lambda L: L.kfac_linear_q8(None, rows(4, 8, I8), torch.zeros(4), rows(6, 8, I8), torch.zeros(6), rows(4, 6, F),
                               bias=torch.zeros(6, dtype=H16)),
    lambda L: L.kfac_weight_grad_q8(rows(4, 6, F), rows(4, 8, I8), torch.zeros(4), rows(6, 8, H16)),
    lambda L: L.kfac_weight_grad_q8(rows(4, 6, F), rows(4, 8, I8), torch.zeros(4), rows(6, 8, F), dbias=torch.zeros(5)),
    lambda L: L.kfac_factors_q8([rows(4, 8, I8)], [torch.zeros(4)], [torch.zeros(35)]),
    lambda L: L.kfac_factors_q8([rows(4, 8, F)], [torch.zeros(4)], [torch.zeros(36)]),
])
def test_binding_refuses_types(lib, call):
    with pytest.raises(TypeError):
        call(lib)


@pytest.mark.parametrize("call", [
    lambda L: L.kfac_quantize_rows(rows(4, 8, F), rows(4, 7, I8), torch.zeros(4)),
    lambda L: L.kfac_linear_q8(None, rows(4, 8, I8), torch.zeros(4), rows(6, 9, I8), torch.zeros(6), rows(4, 6, F)),
    lambda L: L.kfac_linear_q8(None, rows(5, 8, I8), torch.zeros(5), rows(6, 8, I8), torch.zeros(6), rows(4, 6, F)),
    lambda L: L.kfac_weight_grad_q8(rows(4, 6, F), rows(5, 8, I8), torch.zeros(5), rows(6, 8, F)),
    lambda L: L.kfac_weight_grad_q8(rows(4, 6, F), rows(4, 8, I8), torch.zeros(4), rows(6, 9, F)),
    lambda L: L.kfac_factors_q8([rows(4, 8, I8)], [torch.zeros(4)] * 2, [torch.zeros(36)]),
    lambda L: L.kfac_factors_q8([rows(4, 8, I8)], [torch.zeros(4)], [torch.zeros(36)], bias=[True, False]),
    lambda L: L.kfac_factors_q8_workspace([4], [8, 8], False),
    # tensors of the host: a device is asked for last
    lambda L: L.kfac_quantize_rows(rows(4, 8, F), rows(4, 8, I8), torch.zeros(4)),
    lambda L: L.kfac_factors_q8([rows(4, 8, I8)], [torch.zeros(4)], [torch.zeros(36)]),
])
def test_binding_refuses_sizes_and_devices(lib, call):
    with pytest.raises(ValueError):
        call(lib)


def test_products_of_more_tiles_than_a_launch_takes(lib):
    so, sz = lib._lib, c.c_size_t()
    assert so.kfac_linear_q8_workspace(1 << 20, 8, 1 << 20, c.byref(sz)) == -2 and b"tiles" in so.kfac_last_error()
    assert so.kfac_linear_q8_workspace((1 << 20) - 256, 8, 1 << 20, c.byref(sz)) == 0
    assert so.kfac_linear_q8_workspace((1 << 31) - 1, 8, (1 << 31) - 1, c.byref(sz)) == -2
    assert so.kfac_linear_q8_workspace((1 << 31) - 1, 8, 1, c.byref(sz)) == 0


def test_workspace_of_factors(lib):
    """It does not grow with the layers, and one row needs none."""
    L = lib
    assert L.kfac_factors_q8_workspace([1], [8192], True) == 0
    one = L.kfac_factors_q8_workspace([7], [7920], True)
    assert 0 < one < 160 << 20
    assert one <= L.kfac_factors_q8_workspace([7] * 5, [7920, 7904, 7888, 7872, 7856], True) < 160 << 20
    small = L.kfac_factors_q8_workspace([300], [64], True)
    assert 0 < small < 1 << 20
    assert L.kfac_factors_q8_workspace([300] * 7, [64] * 7, True) <= 7 * (1 << 20)
    for rows, cols, n in [(100, 8192, 3), (2048, 8192, 5), (32768, 64, 100), (8192, 4096, 40), (32768, 1000, 9), (5, 12, 64)]:
        assert L.kfac_factors_q8_workspace([rows] * n, [cols] * n, True) <= 256 << 20


def test_factors_that_are_left_out(lib):
    """All of a layer's arrays are NULL, or none; what is left out is not looked at."""
    so = lib._lib
    past = factors(so)
    two = dict(rows=(4, 4), cols=(8, 8), bias=(0, 1), ld=(8, 0))
    assert factors(so, q=(A, None), s=(B, None), A_packed=(C, None), **two) == past
    assert factors(so, q=(None,), s=(None,), A_packed=(None,)) == past
    for k, v in (("q", A), ("s", B), ("A_packed", C)):
        assert factors(so, **{**dict(q=(None,), s=(None,), A_packed=(None,)), k: (v,)}) == -1
    with pytest.raises(ValueError):    # in the binding too: then a device is asked for
        lib.kfac_factors_q8([rows(4, 8, I8)], [torch.zeros(4)], [None])
