"""Refusals of the losses, the clipping and the bounded update that need no GPU: every bad
argument is refused before the device is touched, in C and in the binding."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

c = ctypes
F16, F32, F64, BF16 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import fac_second_order_amd._lib as L
    return L


def f(v):
    return c.c_float(v)


def ptrs(*v):
    return (c.c_void_p * max(1, len(v)))(*v)


def i64(*v):
    return (c.c_int64 * max(1, len(v)))(*v)


def i32(*v):
    return (c.c_int32 * max(1, len(v)))(*v)


A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000    # never dereferenced: the call fails first


def norm(so, n=i64(4), dt=i32(F32), g=None, out=A, count=1):
    return so.kfac_grad_norm(count, n, dt, ptrs(B) if g is None else g, out, None, 0, None)


def test_grad_norm_refusals(lib):
    so, sz = lib._lib, c.c_size_t()
    assert so.kfac_grad_norm_workspace(1, i64(-1), c.byref(sz)) == -1
    assert b"numel[0]" in so.kfac_last_error()
    assert so.kfac_grad_norm_workspace(1, i64((1 << 40) + 1), c.byref(sz)) == -1
    assert so.kfac_grad_norm_workspace(-1, i64(1), c.byref(sz)) == -1
    assert so.kfac_grad_norm_workspace(1, None, c.byref(sz)) == -1
    assert so.kfac_grad_norm_workspace(1, i64(1), None) == -1
    many = i64(*[1 << 40] * 40)
    assert so.kfac_grad_norm_workspace(40, many, c.byref(sz)) == -2
    assert so.kfac_grad_norm_workspace(0, None, c.byref(sz)) == 0 and sz.value > 0
    assert norm(so, out=None) == -1 and norm(so, out=A + 2) == -1
    assert norm(so, dt=i32(F64)) == -2 and norm(so, dt=i32(17)) == -2 and norm(so, dt=None) == -1
    assert norm(so, g=ptrs(None)) == -1 and norm(so, g=ptrs(B + 2)) == -1
    assert norm(so, dt=i32(BF16), g=ptrs(B + 1)) == -1
    assert norm(so, n=i64(0), g=ptrs(None)) not in (-1, 0)      # nothing to read: past the arguments


def test_units_of_a_call_stay_countable(lib):
    """4096 elements a unit, and unit numbers that stay below 2^31 with a grid of 1024 added."""
    so, sz = lib._lib, c.c_size_t()
    most = ((1 << 31) - 1 - 1024) * 4096 - 7 * (1 << 40)
    assert so.kfac_grad_norm_workspace(8, i64(*[1 << 40] * 7, most), c.byref(sz)) == 0
    assert so.kfac_grad_norm_workspace(8, i64(*[1 << 40] * 7, most + 1), c.byref(sz)) == -2


def clip(so, n=(4, 4), dt=(F32, F32), g=(A, B), odt=(F32, F32), out=(C, D), top=1.0, norm_at=0x500000):
    return so.kfac_grad_clip(len(n), i64(*n), i32(*dt), ptrs(*g), i32(*odt), ptrs(*out), f(top), norm_at, None, 0, None)


def test_grad_clip_refusals(lib):
    so = lib._lib
    past = clip(so)
    assert past not in (0, -1)                     # good arguments stop at the device or the workspace
    for top in (0.0, -1.0, float("inf"), float("nan")):
        assert clip(so, top=top) == -1
    assert clip(so, odt=(BF16, F32)) == -2         # neither the gradient's type nor fp32
    assert clip(so, dt=(BF16, F16), odt=(BF16, F32)) == past
    assert clip(so, out=(None, D)) == -1 and clip(so, out=(C + 2, D)) == -1
    assert clip(so, out=(A, B)) == past            # in place
    assert clip(so, dt=(F16, F32), out=(A, D)) == -1 and b"overlaps" in so.kfac_last_error()
    assert clip(so, out=(A + 4, D)) == -1
    assert clip(so, out=(C, C)) == -1 and b"overlap" in so.kfac_last_error()
    assert clip(so, out=(C, C + 12)) == -1
    assert clip(so, out=(C, C + 16)) == past
    assert clip(so, out=(B, A)) == -1              # one tensor's output is another's input
    assert clip(so, g=(A, A), out=(A, D)) == -1    # the same gradient twice, once in place
    assert clip(so, g=(A, A), out=(A, A)) == -1
    assert clip(so, g=(A, A)) == past
    assert clip(so, norm_at=C + 4) == -1 and clip(so, norm_at=A + 8) == -1


def trust(so, n=(4, 4), P=(A, B), dt=(F32, F16), g=(C, D), fisher=None, w=(0x500000, 0x600000), lr=0.1, delta=1e-3,
          shift=0.0, step=0x700000):
    return so.kfac_trust_update(len(n), i64(*n), ptrs(*P), i32(*dt), ptrs(*g), None if fisher is None else ptrs(*fisher),
                                f(shift), ptrs(*w), f(lr), f(delta), step, None, 0, None)


def test_trust_update_refusals(lib):
    so = lib._lib
    past = trust(so)
    assert past not in (0, -1)
    for bad in (-0.1, float("nan"), float("inf")):
        assert trust(so, lr=bad) == -1
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert trust(so, delta=bad) == -1
    assert trust(so, shift=float("nan")) == -1 and trust(so, step=None) == -1
    assert trust(so, dt=(F64, F16)) == -2
    assert trust(so, g=(None, D)) == -1 and b"fisher" in so.kfac_last_error()
    assert trust(so, g=(None, D), fisher=(0x800000, None)) == past
    assert trust(so, g=(None, D), fisher=(None, None)) == -1
    assert trust(so, P=(None, B)) == -1 and trust(so, w=(None, 0x600000)) == -1 and trust(so, w=(0x500002, 0x600000)) == -1
    assert trust(so, w=(A, 0x600000)) == -1 and trust(so, w=(C, 0x600000)) == -1      # P, g
    assert trust(so, w=(B, 0x600000)) == -1 and trust(so, w=(0x500000, 0x500008)) == -1
    assert trust(so, g=(None, D), fisher=(0x500008, None)) == -1
    assert trust(so, step=0x500004) == -1
    assert trust(so, g=(A, D)) == past             # the gradient may be the preconditioned one


def policy(so, rows=2, vocab=8, dt=F32, z=A, ld=8, token=B, mask=None, seqs=0, begin=None, old=C, ref=None, adv=C,
           low=0.2, high=0.2, kl=0.0, by=0, scale=1.0, logp=D, stats=D, d=None, ldd=0):
    return so.kfac_policy_loss(rows, vocab, dt, z, ld, token, mask, seqs, begin, old, ref, adv, f(low), f(high), f(kl),
                               by, f(scale), logp, stats, d, ldd, None, 0, None)


def test_policy_loss_refusals(lib):
    so, sz = lib._lib, c.c_size_t()
    for rows, vocab, seqs in ((-1, 4, 0), (4, 0, 0), (4, -3, 0), (4, (1 << 30) + 1, 0), (4, 4, -1)):
        assert so.kfac_policy_loss_workspace(rows, vocab, seqs, c.byref(sz)) == -1
    assert so.kfac_policy_loss_workspace(4, 4, 0, None) == -1
    assert so.kfac_policy_loss_workspace(1 << 22, 4, 0, c.byref(sz)) == -2          # rows of a call
    assert so.kfac_policy_loss_workspace((1 << 22) - 1, 4, 0, c.byref(sz)) == 0
    past = policy(so)
    assert past not in (0, -1)
    assert policy(so, dt=F64) == -2 and policy(so, dt=9) == -2
    assert policy(so, z=None) == -1 and policy(so, z=A + 2) == -1 and policy(so, dt=BF16, z=A + 1) == -1
    assert policy(so, ld=7) == -1 and policy(so, token=None) == -1 and policy(so, token=B + 4) == -1
    assert policy(so, old=None) == -1 and policy(so, adv=C + 1) == -1 and policy(so, logp=None) == -1
    assert policy(so, stats=None) == -1 and policy(so, rows=0, stats=None) == -1
    assert policy(so, low=-0.1) == -1 and policy(so, low=1.5) == -1 and policy(so, low=float("nan")) == -1
    assert policy(so, high=-0.1) == -1 and policy(so, high=float("inf")) == -1
    assert policy(so, kl=0.1) == -1 and b"ref_logp" in so.kfac_last_error()
    assert policy(so, kl=0.1, ref=C) == past and policy(so, kl=float("nan"), ref=C) == -1
    assert policy(so, scale=float("inf")) == -1 and policy(so, by=2) == -1
    assert policy(so, seqs=2) == -1 and policy(so, begin=B) == -1 and policy(so, seqs=1, begin=B + 1) == -1
    assert policy(so, seqs=1, begin=B) == past
    assert policy(so, d=A, ldd=8) == past          # in place
    assert policy(so, d=A, ldd=9) == -1 and policy(so, d=A + 4, ldd=8) == -1 and policy(so, d=A + 32, ldd=8) == -1
    assert policy(so, d=A + 64, ldd=8) == past
    assert policy(so, d=0x900000, ldd=7) == -1


def prefer(so, rows=2, vocab=8, dt=F32, z=A, ld=8, token=B, mask=None, pairs=1, begin=B, ref=None, beta=0.1, smooth=0.0,
           scale=1.0, seq=C, margin=C, loss=D, d=None, ldd=0):
    return so.kfac_preference_loss(rows, vocab, dt, z, ld, token, mask, pairs, begin, ref, f(beta), f(smooth), f(scale),
                                   seq, margin, loss, d, ldd, None, 0, None)


def test_preference_loss_refusals(lib):
    so, sz = lib._lib, c.c_size_t()
    for rows, vocab, pairs in ((-1, 4, 1), (4, 0, 1), (4, 4, -1), (4, 4, 1 << 30)):
        assert so.kfac_preference_loss_workspace(rows, vocab, pairs, c.byref(sz)) == -1
    past = prefer(so)
    assert past not in (0, -1)
    assert prefer(so, pairs=-1) == -1 and prefer(so, pairs=1 << 30) == -1
    assert prefer(so, begin=None) == -1 and prefer(so, begin=B + 2) == -1
    assert prefer(so, beta=float("nan")) == -1 and prefer(so, smooth=-0.1) == -1 and prefer(so, smooth=1.1) == -1
    assert prefer(so, scale=float("nan")) == -1 and prefer(so, ref=C + 2) == -1
    assert prefer(so, seq=None) == -1 and prefer(so, margin=None) == -1 and prefer(so, loss=None) == -1
    assert prefer(so, z=None) == -1 and prefer(so, ld=3) == -1 and prefer(so, dt=F64) == -2
    assert prefer(so, d=A + 16, ldd=8) == -1 and prefer(so, d=A, ldd=8) == past


def test_results_lie_apart_from_inputs(lib):
    """A result that shares bytes with an input is refused: its writer and the input's readers run at
    the same time. Rows 2, vocab 8, float32: 64 bytes of logits, 8 of a float for each row."""
    so = lib._lib
    mine = dict(stats=0x500000, logp=0x600000, old=0x700000, ref=0x800000, adv=0x900000, mask=0xa00000, seqs=2, begin=0xb00000,
                d=0xc00000, ldd=8)
    past = policy(so, **mine)
    assert past not in (0, -1)
    for name in ("logp", "stats"):
        for what in ("old", "ref", "adv", "mask", "begin"):
            assert policy(so, **{**mine, name: mine[what]}) == -1 and b"overlaps an input" in so.kfac_last_error()
        assert policy(so, **{**mine, name: A + 60}) == -1 and policy(so, **{**mine, name: B + 12}) == -1
    assert policy(so, **{**mine, "logp": 0x700004}) == -1 and policy(so, **{**mine, "logp": 0x6ffffc}) == -1
    assert policy(so, **{**mine, "logp": 0x700008}) == past and policy(so, **{**mine, "logp": 0x6ffff8}) == past
    assert policy(so, **{**mine, "stats": 0x6ffff4}) == -1 and policy(so, **{**mine, "logp": 0xb00008}) == -1
    for what in ("old", "ref", "adv", "mask", "begin"):
        assert policy(so, **{**mine, "d": mine[what]}) == -1
    assert policy(so, **{**mine, "d": 0x6fffc4}) == -1 and policy(so, **{**mine, "d": 0x6fffc0}) == past
    pair = dict(seq=0x500000, margin=0x600000, loss=0x700000, ref=0x800000, mask=0xa00000, begin=0xb00000, d=0xc00000, ldd=8)
    past = prefer(so, **pair)
    assert past not in (0, -1)
    for name in ("seq", "margin", "loss", "d"):
        for what in ("ref", "mask", "begin"):
            assert prefer(so, **{**pair, name: pair[what]}) == -1 and b"overlaps an input" in so.kfac_last_error()
        assert prefer(so, **{**pair, name: B + 8}) == -1                     # the last token
    assert prefer(so, **{**pair, "seq": 0x7ffffc}) == -1 and prefer(so, **{**pair, "seq": 0x7ffff8}) == past
    assert prefer(so, **{**pair, "margin": 0x7ffffc}) == past


def test_binding_refuses_other_devices(lib):
    """Tensors that are not on the current device, here on the CPU, are refused before their
    addresses reach the library."""
    x, y = torch.zeros(4), torch.zeros(4)
    one = torch.zeros(1)
    with pytest.raises(ValueError, match="device"):
        lib.kfac_grad_norm([x], one)
    with pytest.raises(ValueError, match="device"):
        lib.kfac_grad_clip([x], [y], 1.0, one)
    with pytest.raises(ValueError, match="device"):
        lib.kfac_trust_update([x], [x], [y], 0.1, 1.0, torch.zeros(2))
    z, t = torch.zeros(4, 3), torch.zeros(4, dtype=torch.long)
    with pytest.raises(ValueError, match="device"):
        lib.kfac_policy_loss(z, t, x, x, y, torch.zeros(4))
    with pytest.raises(ValueError, match="device"):
        lib.kfac_preference_loss(z, t, torch.zeros(3, dtype=torch.int32), one, one, one)
    with pytest.raises(TypeError, match="rows, vocab"):
        lib.kfac_policy_loss(z[0], t, x, x, y, torch.zeros(4))


@pytest.fixture
def anywhere(lib, monkeypatch):
    """The binding's checks behind the one of the device, on CPU tensors; a call that passes
    them all stops in the library at the missing device."""
    monkeypatch.setattr(lib, "_on_device", lambda tensors, what: None)
    monkeypatch.setattr(lib, "_stream", lambda stream: None)
    return lib


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would reach a device")
def test_binding_checks(anywhere):
    L = anywhere
    x, one, two = torch.zeros(4), torch.zeros(1), torch.zeros(2)
    with pytest.raises(TypeError, match="contiguous"):
        L.kfac_grad_norm([torch.zeros(4, 4).t()], one)
    with pytest.raises(TypeError, match="dtype"):
        L.kfac_grad_norm([x.double()], one)
    with pytest.raises(TypeError, match="norm"):
        L.kfac_grad_norm([x], one.double())
    with pytest.raises(ValueError, match="out"):
        L.kfac_grad_clip([x], [torch.zeros(5)], 1.0, one)
    with pytest.raises(ValueError, match="out"):
        L.kfac_grad_clip([x], [], 1.0, one)
    with pytest.raises(TypeError, match="float32"):
        L.kfac_trust_update([x.half()], [x], [x], 0.1, 1.0, two)
    with pytest.raises(ValueError, match="size"):
        L.kfac_trust_update([x], [torch.zeros(3)], [x.clone()], 0.1, 1.0, two)
    with pytest.raises(ValueError, match="size"):
        L.kfac_trust_update([x], [], [x.clone()], 0.1, 1.0, two)
    with pytest.raises(ValueError, match="fisher"):
        L.kfac_trust_update([x], [None], [x.clone()], 0.1, 1.0, two)
    with pytest.raises(ValueError, match="size"):
        L.kfac_trust_update([x], [None], [x.clone()], 0.1, 1.0, two, fisher=[torch.zeros(3)])
    with pytest.raises(TypeError, match="fisher"):
        L.kfac_trust_update([x], [None], [x.clone()], 0.1, 1.0, two, fisher=[x.half()])
    z, t = torch.zeros(4, 3), torch.zeros(4, dtype=torch.long)
    good = dict(logits=z, token=t, old_logp=x, advantage=x, logp=x.clone(), stats=torch.zeros(4))

    def policy(**kw):
        return L.kfac_policy_loss(**{**good, **kw})

    with pytest.raises(L.KfacError):
        policy()
    for bad in (dict(token=t.int()), dict(token=t[:3]), dict(old_logp=x.double()), dict(advantage=torch.zeros(8)[::2]),
                dict(logits=z.double()), dict(logits=torch.zeros(3, 4).t()), dict(mask=x), dict(dlogits=z[:3]),
                dict(dlogits=z.half()), dict(logits=torch.zeros(1, 3).expand(4, 3)), dict(stats=torch.zeros(3)),
                dict(seq_begin=torch.zeros(3)), dict(ref_logp=x[:2]), dict(mask=torch.ones(3, dtype=torch.bool))):
        with pytest.raises(TypeError):
            policy(**bad)
    with pytest.raises(ValueError):
        policy(seq_begin=torch.zeros(0, dtype=torch.int32))
    begin = torch.zeros(3, dtype=torch.int32)
    fine = dict(logits=z, token=t, seq_begin=begin, seq_logp=two, margin=one, loss=one.clone())
    with pytest.raises(L.KfacError):
        L.kfac_preference_loss(**fine)
    with pytest.raises(ValueError, match="pair"):
        L.kfac_preference_loss(**{**fine, "seq_begin": begin[:2]})
    for bad in (dict(seq_logp=one), dict(margin=two), dict(loss=torch.zeros(0)), dict(ref_logp=one)):
        with pytest.raises(TypeError):
            L.kfac_preference_loss(**{**fine, **bad})


def test_tensors_of_a_generator_are_looked_at(anywhere):
    """Tensors may come from anything that is iterable: none gets lost to the first look."""
    L = anywhere
    bad = [torch.zeros(4, dtype=torch.float64)]
    one = torch.zeros(1)
    with pytest.raises(TypeError, match="dtype"):
        L.kfac_grad_norm((t for t in bad), one)
    with pytest.raises(TypeError, match="dtype"):
        L.kfac_grad_clip((t for t in bad), (t for t in bad), 1.0, one)
    assert L._listed((t for t in [torch.zeros(3), torch.zeros(5)]), "grad")[0] == [3, 5]


def test_a_workspace_smaller_than_its_alignment_has_no_bytes(lib):
    """The bytes behind the aligned address of a tiny workspace are none, not a wrapped count."""
    big = torch.zeros(600, dtype=torch.uint8)
    at = (-big.data_ptr()) % 256 + 1                     # one byte past an aligned address
    assert lib._ws(big[at:at + 8], 100, "cpu")[1] == 0
    assert lib._ws(big[at:at + 300], 100, "cpu")[1] == 45


def test_a_stream_of_another_device_is_refused(lib):
    there = SimpleNamespace(device=torch.device("cuda", 1))
    for workspace in (None, torch.zeros(8)):
        with pytest.raises(ValueError, match="stream"):
            lib._call_ws(workspace, None, (), torch.device("cuda", 0), there)


def test_a_workspace_of_repeated_bytes_is_refused(lib):
    """An expanded tensor has more elements than bytes."""
    with pytest.raises(TypeError, match="contiguous"):
        lib._call_ws(torch.zeros(1).expand(1 << 20), None, (), torch.device("cpu"), None)
