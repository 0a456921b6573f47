"""Rows in 8 bits, the integer product, and the gradient and factor formed from them, on the
GPU against fp64.

Bounds. Codes and scales are equal to the oracle's. A value read back is one fp32 product and one
rounding to its type. The integer product's sum is exact; its conversion, two products and the
sum with the bias are four roundings of 2^-24 of |part| + |bias|, and one to the type. Gradients and
factors are sums of exact products in fp32, whose partial sums never exceed the sum of the
magnitudes: n terms lose at most n 2^-23 of that (2^-23 where the matrix unit cuts instead of
rounding), and a few more roundings follow. Inputs whose sums stay whole numbers below 2^24 are
exact in any order: there the results are equal."""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from loss_cases import FLOOR, HALF_STEP, U, host64
from oracle import q8_oracle as qo

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F16, BF16, F32]


def host(t):
    return t.detach().cpu().numpy()


def pitched(rows, cols, dtype, pad=0, fill=7):
    """A [rows, cols] tensor whose rows lie cols + pad apart, and the buffer that it is a part of."""
    wide = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    return wide[:, :cols], wide


def rows_of(seed, rows, cols, dtype, pad=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    out, _ = pitched(rows, cols, dtype, pad)
    out.copy_(x.to(dtype))
    return out


def quantize(kfac, x, mask=None, pow2=True, pad=0):
    q, wide = pitched(*x.shape, torch.int8, pad)
    scale = torch.full((x.shape[0],), 7.0, device="cuda")
    kfac.kfac_quantize_rows(x, q, scale, mask=mask, pow2=pow2)
    torch.cuda.synchronize()
    assert (wide[:, x.shape[1]:] == 7).all()
    return q, scale


def same(a, b):
    return np.array_equal(np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64), equal_nan=True)


COLS = [1, 2, 3, 7, 8, 15, 16, 17, 63, 64, 65, 255, 257, 1001, 1024, 2049, 4096, 4099, 8200, 16400, 40001]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_quantize_rows(kfac_gpu, dtype, cols):
    for pow2 in (True, False):
        for pad in (0, 5):
            rows = 5 if cols > 2000 else 37
            x = rows_of(cols + pad, rows, cols, dtype, pad, spread=3.0 if dtype != F16 else 0.5)
            mask = torch.tensor([t % 3 != 1 for t in range(rows)], device="cuda")
            for m in (None, mask, mask.to(torch.uint8) * 2):
                q, s = quantize(kfac_gpu, x, m, pow2, pad)
                want, scale = qo.quantize_rows(host64(x), None if m is None else host(m), pow2)
                assert same(host(s), scale) and same(host(q), want), (cols, pow2, pad)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_half(kfac_gpu, dtype):
    """Quotients at, just below and just above every half step."""
    top = 127.0
    for s in (1.0, 2.0 ** -9):
        halves = torch.arange(-126, 127, dtype=torch.float64) + 0.5
        near = torch.cat([halves, halves * (1 + 2.0 ** -20), halves * (1 - 2.0 ** -20), torch.tensor([top, -top])]) * s
        x = near.to(dtype).cuda().repeat(3, 1).contiguous()
        for pow2 in (True, False):
            q, scale = quantize(kfac_gpu, x, None, pow2)
            want, ws = qo.quantize_rows(host64(x), None, pow2)
            assert same(host(scale), ws) and same(host(q), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [1, 9, 300, 5000])
def test_quantize_special_rows(kfac_gpu, dtype, cols):
    inf, nan, big = float("inf"), float("nan"), torch.finfo(dtype).max
    rows = [inf, -inf, nan, 0.0, -0.0, big, -big, torch.finfo(dtype).smallest_normal, torch.finfo(dtype).tiny / 4, 1.0]
    x = torch.zeros(len(rows), cols)
    x[:, cols // 2] = torch.tensor(rows)
    x[-1, 0] = 1.0
    x = x.to(dtype).cuda()
    for mask in (None, torch.tensor([0, 1] * 5, device="cuda", dtype=torch.uint8)):
        for pow2 in (True, False):
            q, s = quantize(kfac_gpu, x, mask, pow2)
            want, scale = qo.quantize_rows(host64(x), None if mask is None else host(mask), pow2)
            assert same(host(s), scale) and same(host(q), want)
            out = torch.full_like(x, 7.0)
            kfac_gpu.kfac_dequantize_rows(q, s, out)
            v = qo.row_values(want, scale)
            assert (host64(out)[np.isnan(scale)] != host64(out)[np.isnan(scale)]).all()
            fine = ~np.isnan(scale)
            assert np.isfinite(host64(out)[fine]).all()
            if pow2:
                assert same(host64(out)[fine], np.clip(v[fine], -big, big))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 7, 2), (65, 129, 0), (33, 1001, 7), (17, 4096, 0), (2, 20003, 1)])
def test_dequantize_rows(kfac_gpu, dtype, rows, cols, pad):
    g = torch.Generator().manual_seed(rows)
    for pow2 in (True, False):
        q, _ = pitched(rows, cols, torch.int8, pad)
        q.copy_(torch.randint(-128, 128, (rows, cols), generator=g))
        s = torch.exp2(torch.randint(-9, 9, (rows,), generator=g).float()) if pow2 else torch.rand(rows, generator=g) + 0.1
        out, wide = pitched(rows, cols, dtype, pad)
        kfac_gpu.kfac_dequantize_rows(q, s.cuda(), out)
        v = qo.row_values(host(q), s.numpy())
        err = np.abs(host64(out) - v)
        if pow2:
            assert not err.any()
        else:
            assert (err <= np.abs(v) * (U + (HALF_STEP[dtype] if dtype != F32 else 0)) * 1.01).all()
        assert (wide[:, cols:] == 7).all()


def codes(seed, rows, cols, pad=0, most=127):
    g = torch.Generator().manual_seed(seed)
    q, _ = pitched(rows, cols, torch.int8, pad)
    q.copy_(torch.randint(-most, most + 1, (rows, cols), generator=g))
    return q


LINEAR = [(1, 1, 1), (1, 64, 5), (1, 1000, 1001), (2, 4096, 64), (3, 17, 33), (5, 4099, 130), (8, 256, 256), (16, 512, 100),
          (17, 96, 257), (31, 2048, 1000), (64, 128, 64), (65, 65, 65), (128, 4096, 128), (200, 333, 777), (257, 1024, 512),
          (513, 160, 300), (1024, 64, 1024), (1000, 2500, 260)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,c_in,c_out", LINEAR)
def test_linear(kfac_gpu, dtype, rows, c_in, c_out):
    for pad, biased, given in ((0, True, False), (3, False, True)):
        x = rows_of(rows + pad, rows, c_in, dtype, pad)
        w, v = codes(c_in, c_out, c_in, pad), torch.rand(c_out, device="cuda") * 0.01 + 0.001
        b = torch.randn(c_out, device="cuda").to(dtype) if biased else None
        mask = torch.tensor([t % 5 != 3 for t in range(rows)], device="cuda") if pad else None
        q, q_wide = pitched(rows, c_in, torch.int8, pad)
        s = torch.full((rows,), 7.0, device="cuda")
        y, wide = pitched(rows, c_out, dtype, pad)
        if given:
            kfac_gpu.kfac_quantize_rows(x, q, s, mask=mask)
            kfac_gpu.kfac_linear_q8(None, q, s, w, v, y, bias=b)
        else:
            kfac_gpu.kfac_linear_q8(x, q, s, w, v, y, bias=b, mask=mask)
        want_q, want_s = qo.quantize_rows(host64(x), None if mask is None else host(mask))
        assert same(host(q), want_q) and same(host(s), want_s)
        want, size = qo.linear(want_q, want_s, host(w), host64(v), None if b is None else host64(b))
        bound = 4 * U * size * 1.01 + (HALF_STEP[dtype] * np.abs(want) * 1.01 if dtype != F32 else 0) + FLOOR[dtype]
        assert (np.abs(host64(y) - want) <= bound).all()
        assert (wide[:, c_out:] == 7).all() and (q_wide[:, c_in:] == 7).all()


def test_linear_sums_are_exact(kfac_gpu):
    """Every code at its largest, sums up to 2^31: no int32 overflows, none is rounded before its end."""
    c_in = 131071
    q = torch.full((3, c_in), -128, dtype=torch.int8, device="cuda")
    q[1] = 127
    w = torch.full((2, c_in), -128, dtype=torch.int8, device="cuda")
    w[1, ::2] = 127
    one = torch.ones(3, device="cuda")
    y = torch.zeros(3, 2, device="cuda")
    kfac_gpu.kfac_linear_q8(None, q, one, w, one[:2].contiguous(), y)
    want = host(q).astype(np.int64) @ host(w).astype(np.int64).T
    assert same(host(y), want.astype(np.float32))


def grads_of(seed, rows, cols, dtype, pad=0, whole=False):
    g = torch.Generator().manual_seed(seed)
    out, _ = pitched(rows, cols, dtype, pad)
    out.copy_(torch.randint(-3, 4, (rows, cols), generator=g) if whole else torch.randn(rows, cols, generator=g) * 0.01)
    return out


def scales_of(seed, rows, zeros=True):
    g = torch.Generator().manual_seed(seed)
    s = torch.exp2(torch.randint(-2, 2, (rows,), generator=g).float())
    if zeros and rows > 1:
        s[torch.rand(rows, generator=g) < 0.2] = 0.0
    return s.cuda()


def grad(kfac, g, q, s, biased, matrix, accumulate=False, start=0.0):
    c_out, c_in = g.shape[1], q.shape[1]
    out = torch.full((c_out, c_in + (1 if biased else 0)), start, device="cuda")
    if matrix or not biased:
        dw, db = out[:, :c_in], out[:, c_in] if biased else None
    else:
        dw, db = out[:, :c_in].contiguous(), out[:, c_in].contiguous()
    kfac.kfac_weight_grad_q8(g, q, s, dw, dbias=db, accumulate=accumulate)
    torch.cuda.synchronize()
    return host64(dw), None if db is None else host64(db)


GRAD = [(1, 1, 1), (1, 200, 3), (2, 8, 8), (7, 33, 65), (31, 130, 127), (32, 128, 128), (33, 129, 257), (64, 256, 256),
        (65, 300, 40), (300, 1001, 77), (513, 64, 1000), (2048, 100, 60), (2049, 260, 250), (5000, 31, 17), (4100, 513, 300)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,c_in,c_out", GRAD)
def test_weight_grad_of_whole_numbers(kfac_gpu, dtype, rows, c_in, c_out):
    for pad, biased, matrix in ((0, True, True), (3, True, False), (1, False, False)):
        q, s = codes(rows + pad, rows, c_in, pad, most=20), scales_of(rows, rows)
        g = grads_of(c_in, rows, c_out, dtype, pad, whole=True)
        dw, db, size, _ = qo.weight_grad(host64(g), host(q), host(s))
        assert size.max() * 4 < 2 ** 24
        got, gb = grad(kfac_gpu, g, q, s, biased, matrix)
        assert same(got, dw) and (not biased or same(gb, db))
        got, gb = grad(kfac_gpu, g, q, s, biased, matrix, accumulate=True, start=5.0)
        assert same(got, dw + 5) and (not biased or same(gb, db + 5))


# sizes that fill the card with large tiles: the last ones ragged, one list of rows and several, few and many steps
LARGE = [(300, 2048, 2048), (1111, 1032, 4104), (256, 2056, 2000), (8300, 1024, 4096), (700, 4104, 1040), (333, 8192, 520),
         (1001, 2051, 2049), (640, 777, 1001), (33000, 40, 24), (9001, 130, 9)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,c_in,c_out", LARGE)
def test_large_weight_grad_of_whole_numbers(kfac_gpu, dtype, rows, c_in, c_out):
    q, s = codes(rows, rows, c_in, 8 if rows % 2 else 0, most=20), scales_of(rows, rows, zeros=rows != 300)
    g = grads_of(c_in, rows, c_out, dtype, 8 if rows % 2 else 0, whole=True)
    g[s == 0] = float("nan")
    live = s != 0
    # sums of whole numbers below 2^53: exact in any order, also on the GPU
    a = (q.double() * s.double()[:, None])[live].cuda()
    want = host64(g[live].double().T.contiguous() @ a)
    bias = host64(g[live].double().sum(0))
    got, gb = grad(kfac_gpu, g, q, s, True, rows % 2 == 0)
    assert same(got, want) and same(gb, bias)
    got, gb = grad(kfac_gpu, g, q, s, True, rows % 2 == 1, accumulate=True, start=5.0)
    assert same(got, want + 5) and same(gb, bias + 5)
    s[:] = 0
    got, gb = grad(kfac_gpu, g, q, s, True, True)
    assert not got.any() and not gb.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,c_in,c_out", [(33, 129, 57), (300, 256, 260), (1500, 70, 300)])
def test_weight_grad(kfac_gpu, dtype, rows, c_in, c_out):
    x = rows_of(1, rows, c_in, dtype, spread=0.5)
    q, s = quantize(kfac_gpu, x)
    g = grads_of(2, rows, c_out, dtype)
    dw, db, size, bsize = qo.weight_grad(host64(g), host(q), host(s))
    got, gb = grad(kfac_gpu, g, q, s, True, True)
    n = rows * (3 if dtype == F32 else 1) + 8
    assert (np.abs(got - dw) <= n * 2 * U * size).all()
    assert (np.abs(gb - db) <= n * 2 * U * bsize).all()
    say(dtype, rows, "relF", np.linalg.norm(got - dw) / np.linalg.norm(dw))


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_rows_that_take_no_part(kfac_gpu, dtype):
    """Gradients of rows with scale 0 may hold anything; a row with scale NaN shows everywhere."""
    rows, c_in, c_out = 150, 40, 30
    q, s = codes(1, rows, c_in, most=20), scales_of(2, rows)
    g = grads_of(3, rows, c_out, dtype, whole=True)
    dw, db, _, _ = qo.weight_grad(host64(g), host(q), host(s))
    g[s == 0] = float("nan")
    q[s == 0] = 111
    got, gb = grad(kfac_gpu, g, q, s, True, True)
    assert same(got, dw) and same(gb, db)
    s[:] = 0
    got, gb = grad(kfac_gpu, g, q, s, True, True)
    assert not got.any() and not gb.any()
    s[77] = float("nan")
    g[77] = 1.0
    q[77] = 0
    got, gb = grad(kfac_gpu, g, q, s, True, True)
    assert np.isnan(got).all() and (gb == 1).all()
    # an infinite gradient reaches its own outputs alone
    s[:] = 1
    g[:] = 1
    g[3, 4] = float("inf")
    q[:] = 1
    got, gb = grad(kfac_gpu, g, q, s, True, True)
    assert (got[4] == np.inf).all() and gb[4] == np.inf and np.isfinite(np.delete(got, 4, 0)).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_of_far_scales(kfac_gpu, dtype):
    """Rows of very different size: exact where the documentation says so."""
    rows = 24
    e = torch.arange(rows) - 20.0
    s = torch.exp2(e).cuda()
    q = codes(5, rows, 50)
    g = torch.zeros(rows, rows, dtype=dtype, device="cuda")
    g.fill_diagonal_(1.0)  # output o is row o alone
    got, _ = grad(kfac_gpu, g, q, s, False, False)
    assert same(got, qo.row_values(host(q), host64(s)))
    for far in (2.0 ** 100, 2.0 ** -100):
        got, _ = grad(kfac_gpu, g, q, s * far, False, False)
        assert same(got, qo.row_values(host(q), host64(s) * far))


def factors(kfac, layers, bias, full=False, decay=0.0, start=None, **kw):
    """Packed factors (and the full ones) of [(q, s)]."""
    orders = [q.shape[1] + (1 if bias else 0) for q, _ in layers]
    packed = [torch.full((d * (d + 1) // 2,), 3.0, device="cuda") if start is None else start[i].clone()
              for i, d in enumerate(orders)]
    fulls = [torch.full((d, d), 9.0, device="cuda") for d in orders] if full else None
    kfac.kfac_factors_q8([q for q, _ in layers], [s for _, s in layers], packed, A_full=fulls, bias=bias, ema_decay=decay,
                         **kw)
    torch.cuda.synchronize()
    if full:
        for f, p, d in zip(fulls, packed, orders):
            i, j = np.triu_indices(d)
            assert same(host(f)[i, j], host(p))
            assert (host(f)[np.tril_indices(d, -1)] == 9).all()
    return packed


FACTOR = [(1, 1), (1, 5), (2, 64), (31, 128), (33, 129), (64, 255), (65, 257), (300, 100), (513, 384), (2048, 60),
          (2049, 130), (5000, 33), (4100, 300)]


@pytest.mark.parametrize("rows,cols", FACTOR)
def test_factor_of_whole_numbers(kfac_gpu, rows, cols):
    for pad, bias in ((0, True), (3, False)):
        q, s = codes(rows + pad, rows, cols, pad, most=9), scales_of(cols, rows)
        raw, size = qo.factor_packed(host(q), host(s), bias)
        live = int((host(s) != 0).sum())
        assert size.max() * live * 16 < 2 ** 24
        got = host(factors(kfac_gpu, [(q, s)], bias, full=True)[0])
        inv = np.float32(1) / np.float32(live) if live else np.float32(0)
        want = (raw * live).astype(np.float32) * inv
        # the corner is 1; others one product with the rounded 1 / C, in either order of a power of two
        if bias and live:
            want[-1] = 1
        assert same(got, want), (rows, cols, np.abs(got - want).max())


@pytest.mark.parametrize("rows,cols", [(700, 2051), (300, 1500), (6200, 1032), (13000, 520), (128, 4096), (20000, 64)])
def test_large_factor_of_whole_numbers(kfac_gpu, rows, cols):
    for bias in (True, False):
        q, s = codes(rows, rows, cols, 3, most=4), scales_of(cols, rows, zeros=rows != 300)
        live = s != 0
        n = int(live.sum())
        a = (q.double() * s.double()[:, None])[live]
        if bias:
            a = torch.cat([a, torch.ones_like(a[:, :1])], 1)
        sums = a.T.contiguous() @ a  # whole numbers of sixteenths: exact in any order
        i, j = torch.triu_indices(a.shape[1], a.shape[1], device="cuda")
        want = host(sums[i, j]).astype(np.float32) * (np.float32(1) / np.float32(n))
        if bias:
            want[-1] = 1
        assert float((a.abs().T @ a.abs()).max()) * 16 < 2 ** 24
        assert same(host(factors(kfac_gpu, [(q, s)], bias, full=cols < 2000)[0]), want)
        both = factors(kfac_gpu, [(q, s)] * 2 + [(q[:50], s[:50])], bias)
        assert same(host(both[0]), want) and same(host(both[1]), want)


def test_factors_of_many_layers(kfac_gpu):
    """More layers than one launch takes, of every kind of tile."""
    layers = [(codes(i, 40 + 211 * i, w, most=9), scales_of(i, 40 + 211 * i))
              for i, w in enumerate([3, 8, 17, 64, 120, 129, 200, 256, 300, 31, 5, 40, 72, 88, 96, 104, 112, 136, 144, 152])]
    for (q, s), p in zip(layers, factors(kfac_gpu, layers, True, full=True)):
        want, size = qo.factor_packed(host(q), host(s), True)
        assert (np.abs(host64(p) - want) <= 3 * U * size).all()  # exact sums, 1 / C and one product


def test_factors_of_several_layers(kfac_gpu):
    layers, xs = [], []
    for i, (rows, cols) in enumerate([(700, 130), (33, 260), (1, 7), (2500, 64), (90, 40)]):
        x = rows_of(i, rows, cols, F16, pad=i, spread=0.5)
        xs.append(x)
        layers.append(quantize(kfac_gpu, x, pad=i))
    alone = [factors(kfac_gpu, [l], True)[0] for l in layers]
    together = factors(kfac_gpu, layers, True, full=True)
    for (q, s), a, t in zip(layers, alone, together):
        assert same(host(a), host(t))
        want, size = qo.factor_packed(host(q), host(s), True)
        assert (np.abs(host64(a) - want) <= (q.shape[0] + 8) * 2 * U * size).all()
        say(q.shape, "relF", np.linalg.norm(host64(a) - want) / np.linalg.norm(want))
    old = [torch.rand_like(p) for p in together]
    blended = factors(kfac_gpu, layers, True, full=True, decay=0.75, start=old)
    for (q, s), o, b in zip(layers, old, blended):
        want, size = qo.factor_packed(host(q), host(s), True, host64(o), 0.75)
        assert (np.abs(host64(b) - want) <= (q.shape[0] + 12) * 2 * U * size).all()


def test_factor_of_scales(kfac_gpu):
    """Rows of every scale there is: each adds up by itself; a scale that is none makes the factor NaN."""
    rows, cols = 700, 40
    q = codes(9, rows, cols, most=9)
    s = torch.exp2((torch.arange(rows) % 200 - 100).float() / 2).floor().clamp(min=2.0 ** -50).cuda()
    s = torch.exp2(torch.log2(s).floor())
    want, size = qo.factor_packed(host(q), host(s), True)
    got = host64(factors(kfac_gpu, [(q, s)], True)[0])
    assert (np.abs(got - want) <= (150 + 8) * 2 * U * size).all()       # a sum of 2^12 at most 150 scales' sums
    # the same rows, all far away: powers of two throughout, infinite where a float is
    for far in (2.0 ** 30, 2.0 ** -30):
        again = host(factors(kfac_gpu, [(q, s * far)], False)[0])
        with np.errstate(over="ignore"):
            assert same(again, (host64(factors(kfac_gpu, [(q, s)], False)[0]) * far * far).astype(np.float32))
    for bad in (1.5, float("nan"), float("inf"), -1.0, 2.0 ** -130):
        t = s.clone()
        t[5] = bad
        assert np.isnan(host(factors(kfac_gpu, [(q, t)], False)[0])).all()


@pytest.mark.parametrize("rows, cols", [(6000, 200), (20000, 70), (900, 1040), (8192, 17)])
def test_factor_of_full_sums(kfac_gpu, rows, cols):
    """Codes of one size and columns of one sign: sums as large as they get, of scales that do not fit into 32 bits."""
    sign = torch.where(torch.arange(cols) % 3 == 0, -127, 127).to(torch.int8).cuda()
    q = sign.expand(rows, cols).contiguous()
    s = torch.exp2(-(torch.arange(rows) % 9).float()).cuda()
    want, size = qo.factor_packed(host(q), host(s), True)
    got = host64(factors(kfac_gpu, [(q, s)], True)[0])
    # at most 9 scales' exact sums a block, 5 blocks, the mean and the blending: each rounds once or twice
    assert (np.abs(got - want) <= (9 + 5 + 8) * 2 * U * size).all()


def test_rows_far_apart(kfac_gpu):
    """Rows 2^32 bytes apart, beside a layer of ordinary ones in one call: whole numbers, so that nothing is rounded."""
    close = codes(3, 3, 40, most=9)
    wide = torch.empty(2 ** 33 + 64, dtype=torch.int8, device="cuda")
    far = wide.as_strided((3, 40), (2 ** 32, 1))
    far.copy_(close)
    s = torch.tensor([1.0, 0.0, 2.0], device="cuda")
    q, t = codes(4, 5000, 64, most=9), torch.ones(5000, device="cuda")
    alone = [host(factors(kfac_gpu, [layer], True)[0]) for layer in ((close, s), (q, t), (close, s))]
    together = factors(kfac_gpu, [(far, s), (q, t), (close, s)], True)
    for a, b in zip(alone, together):
        assert same(a, host(b))
    assert same(alone[0], qo.factor_packed(host(close), host(s), True)[0])
    g = codes(5, 3, 30, most=9).half()
    for a, b in zip(grad(kfac_gpu, g, close, s, True, False), grad(kfac_gpu, g, far, s, True, False)):
        assert same(a, b)


@pytest.mark.parametrize("bias", [True, False])
def test_factor_without_rows(kfac_gpu, bias):
    q, s = codes(1, 70, 50), torch.zeros(70, device="cuda")
    none = (torch.zeros(0, 50, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda"))
    for layer in ((q, s), none):
        assert not host(factors(kfac_gpu, [layer], bias, full=True)[0]).any()
        old = [torch.rand(51 * 52 // 2 if bias else 50 * 51 // 2, device="cuda")]
        assert same(host(factors(kfac_gpu, [layer], bias, full=True, decay=0.9, start=old)[0]), host(old[0]))


def test_nothing_to_do(kfac_gpu):
    e8, e32 = torch.zeros(0, 5, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    x = torch.zeros(0, 5, device="cuda")
    kfac_gpu.kfac_quantize_rows(x, e8, e32)
    kfac_gpu.kfac_dequantize_rows(e8, e32, x)
    w, v = codes(1, 4, 5), torch.ones(4, device="cuda")
    kfac_gpu.kfac_linear_q8(x, e8, e32, w, v, torch.zeros(0, 4, device="cuda"))
    # no input channels: the bias alone, and the bias gradient alone
    q, s = torch.zeros(3, 0, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda")
    y = torch.full((3, 4), 9.0, device="cuda")
    b = torch.arange(4.0, device="cuda")
    kfac_gpu.kfac_linear_q8(None, q, s, torch.zeros(4, 0, dtype=torch.int8, device="cuda"), v, y, bias=b)
    assert same(host(y), np.tile(np.arange(4.0), (3, 1)))
    g, db = torch.ones(3, 4, device="cuda"), torch.full((4,), 9.0, device="cuda")
    kfac_gpu.kfac_weight_grad_q8(g, q, s, torch.zeros(4, 0, device="cuda"), dbias=db)
    assert same(host(db), [3] * 4)
    # no rows: zeros, or what was there
    dw = torch.full((4, 5), 9.0, device="cuda")
    kfac_gpu.kfac_weight_grad_q8(torch.zeros(0, 4, device="cuda"), e8, e32, dw, accumulate=True)
    assert (dw == 9).all()
    kfac_gpu.kfac_weight_grad_q8(torch.zeros(0, 4, device="cuda"), e8, e32, dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("dtype, apart", [(F32, 2 ** 30), (F32, 2 ** 30 + 8), (F16, 2 ** 31), (BF16, 2 ** 31 - 8)])
def test_gradient_rows_far_apart(kfac_gpu, dtype, apart):
    """Rows of gradients up to 2^32 bytes and more apart, beside the same rows close to each other: whole numbers."""
    close = codes(6, 3, 30, most=9).to(dtype)
    wide = torch.empty(2 * apart + 64, dtype=dtype, device="cuda")
    far = wide.as_strided((3, 30), (apart, 1))
    far.copy_(close)
    q, s = codes(7, 3, 40, most=9), torch.tensor([1.0, 0.0, 2.0], device="cuda")
    want = grad(kfac_gpu, close, q, s, True, False)
    dw, db, _, _ = qo.weight_grad(host64(close), host(q), host(s))
    assert same(want[0], dw) and same(want[1], db)
    for a, b in zip(want, grad(kfac_gpu, far, q, s, True, False)):
        assert same(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [40, 5])     # in tiles, and too few columns for one
def test_weight_grad_of_the_largest_rows(kfac_gpu, dtype, cols):
    """Rows up to the largest finite number: s q is finite, and so is what a small gradient makes of it."""
    top = float(torch.finfo(F32).max)
    x = torch.zeros(40, cols, device="cuda")
    x[:] = torch.linspace(-1, 1, cols, device="cuda") * top
    x[1::2] *= 0.6
    x[5], x[6, 0] = 0.0, top
    q, s = quantize(kfac_gpu, x)
    assert {2.0 ** 121, 2.0 ** 122} < set(s.tolist())
    g = torch.zeros(40, 40, dtype=dtype, device="cuda")
    g.fill_diagonal_(2.0 ** -9)
    s[5] = 2.0 ** 118       # its codes are 0
    got, gb = grad(kfac_gpu, g, q, s, True, False)
    assert same(got, qo.row_values(host(q), host64(s)) * 2.0 ** -9) and (gb == 2.0 ** -9).all()


@pytest.mark.parametrize("rows", [2, 40, 1500])
@pytest.mark.parametrize("cols", [40, 5])
def test_bias_gradient_of_far_scales(kfac_gpu, rows, cols):
    """A row that fp16 cannot hold beside the largest scale has its share of the bias gradient all the same."""
    q = codes(8, rows, cols, most=9)
    s = torch.full((rows,), 2.0 ** -100, device="cuda")
    s[0] = 2.0 ** 100
    for dtype in TYPES:
        g = grads_of(9, rows, 40, dtype, whole=True)
        _, gb = grad(kfac_gpu, g, q, s, True, False)
        assert same(gb, host64(g).sum(0))


def test_quantize_halves_of_the_smallest_scales(kfac_gpu):
    """Scales next to 2^-126, whose halves are no floats: quotients half a last place beside every half step."""
    S = 2 ** 23 + 1 + 2 * np.arange(400, dtype=np.int64)           # scales in units of 2^-149
    x = np.zeros((len(S), 1 + 2 * 127), dtype=np.float64)
    x[:, 0] = 127 * S
    for k in range(127):
        x[:, 1 + 2 * k] = ((2 * k + 1) * S) // 2                   # (k + 1/2) S is half a whole number
        x[:, 2 + 2 * k] = -((2 * k + 1) * S + 1) // 2
    x = (x * 2.0 ** -149).astype(np.float32)
    q, s = quantize(kfac_gpu, torch.from_numpy(x).cuda(), None, False)
    want, scale = qo.quantize_rows(x, None, False)
    assert same(host(s), scale) and len(set(scale)) > 200
    assert same(host(q), want)


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 2044])
def test_the_longest_rows(kfac_gpu, cols):
    at = torch.tensor([0, 5, 2 ** 30 + 1, cols - 2050, cols - 9, cols - 1], device="cuda")
    x = torch.zeros(1, cols, dtype=F16, device="cuda")
    x[0, at] = torch.tensor([1.0, -2.0, 3.0, 127.0, -5.0, 6.0], dtype=F16, device="cuda")
    q, s = quantize(kfac_gpu, x)
    assert float(s) == 1.0 and q[0, at].tolist() == [1, -2, 3, 127, -5, 6]
    assert int(torch.count_nonzero(q)) == 6
    x.fill_(9.0)
    kfac_gpu.kfac_dequantize_rows(q, s, x)
    assert x[0, at].tolist() == [1, -2, 3, 127, -5, 6] and int(torch.count_nonzero(x)) == 6
    q.fill_(9)
    kfac_gpu.kfac_quantize_rows(x, q, s, mask=torch.zeros(1, dtype=torch.bool, device="cuda"))
    assert float(s) == 0.0 and not q.any()


def test_more_rows_than_a_launch_takes(kfac_gpu):
    """2^26 rows are a launch's at four a block, 2^32 groups of 8 elements one's that are read back."""
    rows = 2 ** 26 + 3
    x = torch.ones(rows, 2, dtype=F16, device="cuda")
    x[-4:] = 3.0
    mask = torch.ones(rows, dtype=torch.bool, device="cuda")
    mask[-2] = mask[-40] = False
    q, s = quantize(kfac_gpu, x, mask)
    assert bool((q[:-4] == 64).sum() == 2 * (rows - 5)) and not q[-40].any()
    assert q[-4:].tolist() == [[96, 96], [96, 96], [0, 0], [96, 96]]
    assert s[-4:].tolist() == [2.0 ** -5, 2.0 ** -5, 0.0, 2.0 ** -5] and float(s[-40]) == 0.0 and float(s[0]) == 2.0 ** -6
    del x, q, s, mask
    rows = 2 ** 31 - 1
    q = torch.ones(rows, 9, dtype=torch.int8, device="cuda")
    s = torch.ones(rows, device="cuda")
    q[-1], s[-2] = 5, 0.5
    out = torch.zeros(rows, 9, dtype=F16, device="cuda")
    kfac_gpu.kfac_dequantize_rows(q, s, out)
    for part in out[:-2].split(2 ** 28):
        assert bool((part == 1).all())
    assert (out[-2] == 0.5).all() and (out[-1] == 5).all()


def test_more_channels_than_a_launch_of_few_rows_takes(kfac_gpu):
    for c_out in (2 ** 25, 2 ** 26 + 40):
        w = torch.ones(c_out, 16, dtype=torch.int8, device="cuda")
        w[-1] = 3
        v = torch.ones(c_out, device="cuda")
        v[-2] = 0.5
        q, s = torch.ones(2, 16, dtype=torch.int8, device="cuda"), torch.tensor([1.0, 2.0], device="cuda")
        y = torch.zeros(2, c_out, device="cuda")
        kfac_gpu.kfac_linear_q8(None, q, s, w, v, y)
        assert bool((y[:, :-2] == torch.tensor([[16.0], [32.0]], device="cuda")).all())
        assert y[:, -2:].tolist() == [[8.0, 48.0], [16.0, 96.0]]


@pytest.mark.parametrize("rows", [3, 40])
def test_linear_of_rows_without_columns(kfac_gpu, rows):
    """Their checkpoint is written: a scale of 1, or 0 where the mask says so."""
    x, q = torch.zeros(rows, 0, device="cuda"), torch.zeros(rows, 0, dtype=torch.int8, device="cuda")
    w, v, b = torch.zeros(4, 0, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"), torch.arange(4.0, device="cuda")
    mask = torch.arange(rows, device="cuda") != 1
    for m, want in ((None, [1.0] * rows), (mask, mask.float().tolist())):
        s, y = torch.full((rows,), float("nan"), device="cuda"), torch.full((rows, 4), 9.0, device="cuda")
        kfac_gpu.kfac_linear_q8(x, q, s, w, v, y, bias=b, mask=m)
        assert s.tolist() == want and same(host(y), np.tile(np.arange(4.0), (rows, 1)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [5, 20, 300])
def test_linear_of_weights_that_are_no_numbers(kfac_gpu, dtype, rows):
    """A channel whose weights held a NaN is NaN in every row but those that take no part: their y is the bias."""
    c_out = 130
    x = rows_of(3, rows, 64, dtype)
    mask = torch.arange(rows, device="cuda") % 3 != 1
    w, v = codes(4, c_out, 64), torch.ones(c_out, device="cuda")
    w[7], v[7], v[9] = 0, float("nan"), float("inf")
    b = torch.randn(c_out, device="cuda").to(dtype)
    q, s = torch.zeros(rows, 64, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
    for bias in (b, None):
        y = torch.full((rows, c_out), 9.0, dtype=dtype, device="cuda")
        kfac_gpu.kfac_linear_q8(x, q, s, w, v, y, bias=bias, mask=mask)
        alone = torch.zeros_like(b) if bias is None else b
        assert torch.equal(y[~mask], alone.expand(rows, c_out)[~mask])
        assert torch.isnan(y[mask][:, 7]).all() and torch.isfinite(y[:, :7]).all()


@pytest.mark.parametrize("rows, cols, octaves", [(8192, 300, 22), (8192, 70, 22), (8192, 1500, 20), (100352, 200, 15),
                                                 (100352, 64, 20)])
def test_factor_is_deterministic(kfac_gpu, rows, cols, octaves):
    """The same bits from run to run, over scales that do not fit into 32 bits together."""
    q = codes(rows, rows, cols) | 64                            # sums far from 0
    g = torch.Generator().manual_seed(cols)
    s = torch.exp2(-torch.randint(0, octaves, (rows,), generator=g).float()).cuda()
    first = factors(kfac_gpu, [(q, s)], True)[0]
    want, size = qo.factor_packed(host(q[:, :64]), host(s), True) if cols == 64 else (None, None)
    for _ in range(6):
        assert torch.equal(factors(kfac_gpu, [(q, s)], True)[0], first)
    if want is not None:
        assert (np.abs(host64(first) - want) <= (octaves + 60) * 2 * U * size).all()


@pytest.mark.parametrize("rows", [63, 200, 440])
@pytest.mark.parametrize("cols", [33, 130, 900, 2600])
def test_factor_does_not_know_the_rows_order(kfac_gpu, rows, cols):
    """Rows of one scale add up exactly: in any order of the rows of a block the same bits."""
    q = codes(rows, rows, cols) | 64
    s = torch.exp2(-(torch.arange(rows) % 23).float()).cuda()
    first = factors(kfac_gpu, [(q, s)], True)[0]
    for seed in range(4):
        p = torch.randperm(rows, generator=torch.Generator().manual_seed(seed)).cuda()
        assert torch.equal(factors(kfac_gpu, [(q[p].contiguous(), s[p].contiguous())], True)[0], first)


@pytest.mark.parametrize("rows, cols", [(70, 40), (9000, 40), (300, 900)])
def test_factor_of_a_scale_that_is_none(kfac_gpu, rows, cols):
    """All of it is NaN, the bias column's own entry too, whatever the other rows are."""
    q = codes(1, rows, cols, most=9)
    for bad in (1.5, float("nan"), float("inf"), -1.0, 2.0 ** -130):
        s = torch.ones(rows, device="cuda")
        s[rows - 3] = bad
        old = [torch.rand((cols + 1) * (cols + 2) // 2, device="cuda")]
        for decay in (0.0, 0.5):
            assert np.isnan(host(factors(kfac_gpu, [(q, s)], True, full=False, decay=decay, start=old)[0])).all()
        s[:] = 0
        s[rows - 3] = bad
        assert np.isnan(host(factors(kfac_gpu, [(q, s)], True)[0])).all()


def far_copy(q, apart):
    """The same rows, `apart` bytes from each other."""
    wide = torch.empty((len(q) - 1) * apart + 4096, dtype=torch.int8, device="cuda")
    far = wide.as_strided(q.shape, (apart, 1))
    far.copy_(q)
    return far


@pytest.mark.parametrize("rows, cols", [(1, 1), (5, 7), (64, 15), (700, 3), (3000, 8), (9000, 15), (100352, 2), (40000, 12)])
@pytest.mark.parametrize("bias", [True, False])
def test_factor_of_few_columns(kfac_gpu, rows, cols, bias):
    """No row is lost for its size: the last column has entries in rows alone that are 2^-40 of the others."""
    q = codes(rows, rows, cols, pad=1)
    s = torch.exp2(-(torch.arange(rows) % 5).float()).cuda()
    if rows > 2:
        small = torch.arange(rows, device="cuda") % 3 == 1
        s[small] *= 2.0 ** -40
        q[~small, -1] = 0
        s[2] = 0.0
    want, size = qo.factor_packed(host(q), host(s), bias)
    first = factors(kfac_gpu, [(q, s)], bias, full=True)[0]
    # 10 scales' exact sums a block, 128 blocks at most, the mean: each rounds once or twice
    assert (np.abs(host64(first) - want) <= (10 + 128 + 8) * 2 * U * size).all()
    assert torch.equal(factors(kfac_gpu, [(q, s)], bias)[0], first)
    several = factors(kfac_gpu, [(q, s)] * 3 + [(codes(1, 30, 40), torch.ones(30, device="cuda"))], bias)
    assert all(torch.equal(several[k], first) for k in range(3))
    old = [torch.rand_like(first)]
    got = factors(kfac_gpu, [(q, s)], bias, full=True, decay=0.75, start=old)[0]
    want, size = qo.factor_packed(host(q), host(s), bias, host64(old[0]), 0.75)
    assert (np.abs(host64(got) - want) <= (10 + 128 + 12) * 2 * U * size).all()
    for bad in (1.5, float("nan"), float("inf"), -1.0, 2.0 ** -130):
        t = s.clone()
        t[rows // 2] = bad
        assert np.isnan(host(factors(kfac_gpu, [(q, t)], bias)[0])).all()


@pytest.mark.parametrize("cols", [5, 40, 203])
def test_factor_of_rows_far_apart(kfac_gpu, cols):
    """The same bits as those of the rows close to each other, also over scales that are far from each other."""
    close = codes(2, 5, cols)
    far = far_copy(close, 2 ** 32 + 1)
    for s in ([1.0, 2.0, 4.0, 0.0, 1.0], [1.0, 2.0 ** -60, 2.0 ** 30, 2.0 ** -60, 0.5], [1.0, 2.0 ** -130, 1.0, 1.0, 1.0],
              [float("inf")] + [1.0] * 4):
        s = torch.tensor(s, device="cuda")
        for bias in (True, False):
            a, b = (host(factors(kfac_gpu, [(q, s)], bias, full=True)[0]) for q in (close, far))
            assert same(a, b)
            if (s == 2.0 ** -60).any():
                want, size = qo.factor_packed(host(close), host(s), bias)
                assert (np.abs(a - want) <= 12 * 2 * U * size).all()
            else:
                assert np.isnan(a).all() == (not torch.isfinite(s).all() or bool((s == 2.0 ** -130).any()))


def test_factors_of_wide_layers(kfac_gpu):
    """Layers whose sums take more room than a call has run one after another; scales that do not fit together."""
    rows, cols = 9, 7920
    q = codes(rows, rows, cols)
    s = torch.exp2(torch.tensor([0.0, -30, -60, -1, 0, -2, -90, -30, 5])).cuda()
    narrow = (codes(2, 300, 70, most=9), scales_of(3, 300))
    need = kfac_gpu.kfac_factors_q8_workspace([rows] * 4 + [300], [cols] * 4 + [70], True)
    ws = torch.full((need + 256 + 4096,), 9, dtype=torch.uint8, device="cuda")
    at = -ws.data_ptr() % 256
    got = factors(kfac_gpu, [(q, s)] * 4 + [narrow], True, workspace=ws[at:at + need])
    assert (ws[at + need:] == 9).all()
    assert all(torch.equal(got[0], p) for p in got[1:4])
    a = torch.cat([q.double() * s.double()[:, None], torch.ones(rows, 1, device="cuda", dtype=torch.float64)], 1)
    i, j = torch.triu_indices(cols + 1, cols + 1, device="cuda")
    want, size = (t.T.contiguous() @ t / rows for t in (a, a.abs()))
    assert bool(((got[0].double() - want[i, j]).abs() <= (rows + 8) * 2 * U * size[i, j]).all())
    want, size = qo.factor_packed(host(narrow[0]), host(narrow[1]), True)
    assert (np.abs(host64(got[4]) - want) <= 3 * U * size).all()


@pytest.mark.parametrize("rows,c_in,c_out", [(16, 600, 4097), (17, 1024, 4096), (17, 1025, 4096), (32, 1100, 4097), (33, 1025, 100),
                                             (20, 2000, 64), (32, 1030, 4090), (18, 40, 8200)])
@pytest.mark.parametrize("dtype", TYPES)
def test_linear_next_to_few_rows(kfac_gpu, dtype, rows, c_in, c_out):
    test_linear(kfac_gpu, dtype, rows, c_in, c_out)
