"""The losses over logits on the GPU against their fp64 definitions, element by element
within derived bounds (tests/loss_cases.py), at the sizes, masks and layouts where they can
go wrong."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import say
from loss_cases import FLOOR, HALF_STEP, U, grad_bound, host64, logits, row_errors
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _vec(g, n, scale=1.0):
    return (torch.randn(n, generator=g) * scale).cuda()


def _policy(kfac, z, token, old, adv, ref=None, mask=None, begin=None, grad=True, dlogits=None, **kw):
    rows = z.shape[0]
    logp = torch.full((rows,), 7.0, device="cuda")
    stats = torch.full((4,), 7.0, device="cuda")
    if grad and dlogits is None:
        dlogits = torch.full(z.shape, 7.0, dtype=z.dtype, device="cuda")
    kfac.kfac_policy_loss(z, token, old, adv, logp, stats, dlogits=dlogits, ref_logp=ref, mask=mask, seq_begin=begin,
                          **kw)
    torch.cuda.synchronize()
    return stats, logp, dlogits


def _check_policy(got, z0, token, old, adv, ref=None, mask=None, begin=None, by_sequence=False, clip_low=0.2,
                  clip_high=0.2, kl_coef=0.0, grad_scale=1.0):
    """z0: the logits before the call."""
    stats, logp, d = got
    dtype = z0.dtype
    z, tok, old, adv = host64(z0), token.cpu().numpy(), host64(old), host64(adv)
    ref = None if ref is None else host64(ref)
    mask = None if mask is None else mask.cpu().numpy()
    begin = None if begin is None else begin.cpu().tolist()
    # the library holds its options as floats
    low, high, beta, scale = (float(np.float32(v)) for v in (clip_low, clip_high, kl_coef, grad_scale))
    want, want_l, want_d = lo.policy_loss(z, tok, old, adv, ref, mask, begin, by_sequence, low, high, beta, scale)
    err = row_errors(z)
    inside = ~np.isnan(want_l)
    counted = inside & (want_l != 0)
    lp = host64(logp)
    assert (lp[~inside] == 7.0).all()
    assert (np.abs(lp - want_l)[inside] <= (err + U * np.abs(want_l) * 1.01)[inside]).all()
    # weights and slopes again, row by row, for the bounds
    spans = [(0, len(tok))] if begin is None else list(zip(begin[:-1], begin[1:]))
    n = [int(counted[a:b].sum()) for a, b in spans]
    weight = np.zeros(len(tok))
    for (a, b), k in zip(spans, n):
        if k:
            weight[a:b] = counted[a:b] / (k * sum(v > 0 for v in n) if by_sequence else sum(n))
    l = np.where(counted, want_l, 0.0)
    r = np.where(counted, np.exp(l - np.where(counted, old, 0)), 1.0)
    a = np.where(counted, adv, 0.0)
    edge = np.minimum(np.abs(r - (1 - low)), np.abs(r - (1 + high)))
    assert (edge[counted] > 2 * (err * r)[counted]).all(), "an input on the bound decides nothing"
    e = np.exp(np.where(counted, ref - l, 0)) if ref is not None else np.ones(len(tok))
    held = np.clip(r, 1 - low, 1 + high) * a
    active = r * a <= held
    st = host64(stats)
    u_out = 1.01 * U
    tol_part = (weight * np.abs(r * a) * err).sum()
    tol_kl = (weight * np.abs(e - 1) * err + weight * err ** 2).sum()
    assert abs(st[1] - want[1]) <= tol_part + u_out * abs(want[1]) + 1e-14
    assert abs(st[2] - want[2]) <= tol_kl + u_out * abs(want[2]) + 1e-14
    assert abs(st[0] - want[0]) <= tol_part + beta * tol_kl + u_out * abs(want[0]) + 1e-14
    assert abs(st[3] - want[3]) <= u_out * want[3] + 1e-14
    if d is None:
        return
    slope = np.where(active, -r * a, 0.0) - (beta * (e - 1) if ref is not None else 0.0)
    coef = scale * weight * slope
    coef_err = scale * weight * (np.abs(r * a) * active + beta * e) * 1.01 * err + np.abs(coef) * u_out
    have = host64(d)
    assert (have[~inside] == 7.0).all()
    bound = grad_bound(np.nan_to_num(want_d), z, tok, coef, coef_err, err, dtype)
    off = np.abs(have - want_d)[inside] / bound[inside]
    say("policy", tuple(z.shape), dtype, "gradient at", float(np.max(off, initial=0.0)), "of its bound")
    assert (off <= 1).all()
    assert not have[inside & ~counted].any()


def _policy_inputs(seed, rows, vocab, dtype, pad=0, offset=0):
    z, token, g = logits(seed, rows, vocab, dtype, pad, offset)
    lp = np.array([lo.row_logp(row, y)[0] for row, y in zip(host64(z), token.cpu().numpy())])
    lp = torch.from_numpy(lp).float()
    old = (lp + 0.25 * torch.randn(rows, generator=g)).cuda()
    ref = (lp + 0.3 * torch.randn(rows, generator=g)).cuda()
    return z, token, old, _vec(g, rows), ref


VOCABS = [1, 2, 7, 8, 9, 63, 64, 65, 255, 256, 257, 513, 1000, 1023, 2048, 2049, 4097, 5003]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy_vocabularies(kfac_gpu, dtype, vocab):
    rows = 5
    z, token, old, adv, ref = _policy_inputs(100 + vocab, rows, vocab, dtype)
    kw = dict(ref=ref, kl_coef=0.1, grad_scale=float(rows))
    _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", [16383, 16384, 32001, 65537, 131072, 131075, 163841])
def test_policy_long_rows(kfac_gpu, dtype, vocab):
    """Rows up to and past what a block keeps in registers, for every type."""
    z, token, old, adv, ref = _policy_inputs(vocab, 3, vocab, dtype)
    kw = dict(ref=ref, kl_coef=0.1, grad_scale=3.0)
    _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)


@pytest.mark.parametrize("rows", [1, 2, 31, 257, 1025, 2050])
def test_policy_row_counts(kfac_gpu, rows):
    z, token, old, adv, ref = _policy_inputs(rows, rows, 37, F32)
    _check_policy(_policy(kfac_gpu, z, token, old, adv), z, token, old, adv)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (24, 0)])
def test_policy_pitches_and_alignments(kfac_gpu, dtype, pad, offset):
    for vocab in (40, 1003):
        z, token, old, adv, ref = _policy_inputs(7, 6, vocab, dtype, pad, offset)
        buf = torch.full((6 * (vocab + 2) + 3,), 7.0, dtype=dtype, device="cuda")
        d = buf[3:].view(6, vocab + 2)[:, :vocab]
        kw = dict(ref=ref, kl_coef=0.1, grad_scale=6.0)
        _check_policy(_policy(kfac_gpu, z, token, old, adv, dlogits=d, **kw), z, token, old, adv, **kw)
        assert (buf[:3] == 7).all() and (buf[3:].view(6, vocab + 2)[:, vocab:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [33, 1000, 20011])
def test_policy_in_place(kfac_gpu, dtype, vocab):
    z, token, old, adv, ref = _policy_inputs(8, 4, vocab, dtype)
    z0 = z.clone()
    kw = dict(ref=ref, kl_coef=0.1, grad_scale=4.0)
    apart = _policy(kfac_gpu, z0, token, old, adv, **kw)
    got = _policy(kfac_gpu, z, token, old, adv, dlogits=z, **kw)
    assert all(torch.equal(a, b) for a, b in zip(apart, got))
    _check_policy(got, z0, token, old, adv, **kw)


LAYOUTS = [[0, 12], [0, 5, 12], [2, 2, 9, 9, 11], [0, 0, 0], [12, 12], [0, 1, 2, 3], [3, 12]]


@pytest.mark.parametrize("begin", LAYOUTS)
@pytest.mark.parametrize("by_sequence", [False, True])
@pytest.mark.parametrize("masked", ["none", "some", "a sequence", "all"])
def test_policy_sequences_and_masks(kfac_gpu, begin, by_sequence, masked):
    """Empty sequences, sequences that the mask empties, rows before the first and behind
    the last sequence; what does not count holds NaN."""
    rows, vocab = 12, 70
    z, token, old, adv, ref = _policy_inputs(9, rows, vocab, BF16)
    mask = {"none": None, "some": torch.arange(rows) % 3 != 1, "a sequence": torch.arange(rows) >= 5,
            "all": torch.zeros(rows, dtype=torch.bool)}[masked]
    token[3], token[10] = -100, vocab
    off = torch.zeros(rows, dtype=torch.bool)
    off[[3, 10]] = True
    if mask is not None:
        off |= ~mask
    off |= torch.tensor([not begin[0] <= t < begin[-1] for t in range(rows)])
    z0 = z.clone()
    z[off.cuda()] = float("nan")
    for t in (old, adv, ref):
        t[off.cuda()] = float("nan")
    mask = None if mask is None else mask.cuda()
    b = torch.tensor(begin, dtype=torch.int32, device="cuda")
    kw = dict(ref=ref, mask=mask, begin=b, by_sequence=by_sequence, kl_coef=0.2, grad_scale=10.0)
    got = _policy(kfac_gpu, z, token, old, adv, **kw)
    if not z.isfinite().any():
        assert not host64(got[0]).any()
    _check_policy(got, z0, token, old, adv, **kw)


def test_policy_many_sequences(kfac_gpu):
    """More sequences than a block has threads, empty ones among them."""
    rows = 1500
    z, token, old, adv, ref = _policy_inputs(10, rows, 11, F32)
    begin = torch.tensor([min(rows, t - t % 3) for t in range(rows + 1)], dtype=torch.int32, device="cuda")
    for by in (False, True):
        kw = dict(begin=begin, by_sequence=by, grad_scale=float(rows))
        _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)


def test_policy_loss_alone_and_kl_reported(kfac_gpu):
    z, token, old, adv, ref = _policy_inputs(11, 9, 300, F16)
    kw = dict(ref=ref, kl_coef=0.0, clip_low=0.1, clip_high=0.3)
    got = _policy(kfac_gpu, z, token, old, adv, grad=False, **kw)
    assert got[2] is None
    _check_policy(got, z, token, old, adv, **kw)
    with_grad = _policy(kfac_gpu, z, token, old, adv, **kw)
    assert torch.equal(got[0], with_grad[0]) and torch.equal(got[1], with_grad[1])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_policy_lowest_values_and_infinities(kfac_gpu, dtype):
    """Masked vocabularies (-inf or the type's lowest value), rows of nothing but the lowest
    value (a uniform distribution), large logits."""
    low = torch.finfo(dtype).min
    for vocab in (24, 3000):
        z, token, old, adv, ref = _policy_inputs(12, 6, vocab, dtype)
        z[0, : vocab // 2] = float("-inf")
        z[1, vocab // 2:] = low
        z[2] = low
        z[3, : vocab - 1] = float("-inf")
        z[4] *= 1000
        z[5, ::2] = torch.finfo(dtype).max
        token[:] = torch.tensor([vocab - 1, 0, 3, vocab - 1, int(z[4].argmax()), 2], device="cuda")
        old = torch.tensor([lo.row_logp(a, b)[0] for a, b in zip(host64(z), token.tolist())]).float().cuda() + 0.05
        _check_policy(_policy(kfac_gpu, z, token, old, adv), z, token, old, adv)


@pytest.mark.parametrize("vocab", [24, 3000])
def test_policy_bad_rows_stay_their_own(kfac_gpu, vocab):
    """NaN, +inf or nothing but -inf make a row NaN, and no other."""
    z, token, old, adv, ref = _policy_inputs(13, 5, vocab, F32)
    z[0, 3], z[1, 4] = float("nan"), float("inf")
    z[2] = float("-inf")
    stats, logp, d = _policy(kfac_gpu, z, token, old, adv)
    assert logp[:3].isnan().all() and logp[3:].isfinite().all()
    assert d[:3].isnan().all() and d[3:].isfinite().all()
    assert stats[0].isnan()


def test_policy_edges_of_the_call(kfac_gpu):
    e = torch.empty(0, device="cuda")
    z = torch.empty(0, 5, device="cuda")
    stats = torch.full((4,), 7.0, device="cuda")
    kfac_gpu.kfac_policy_loss(z, e.long(), e, e, e, stats, dlogits=z)
    assert not stats.any()


@pytest.mark.parametrize("dtype", [F16, F32])
def test_rows_past_32_bit_offsets(kfac_gpu, dtype):
    """Rows that begin past 2^31 elements and 2^32 bytes into the tensor."""
    vocab, ld = 9, (1 << 30) + 3
    z0, token, old, adv, ref = _policy_inputs(14, 3, vocab, dtype)
    flat = torch.empty(2 * ld + vocab, dtype=dtype, device="cuda")
    z = flat.as_strided((3, vocab), (ld, 1))
    z.copy_(z0)
    got = _policy(kfac_gpu, z, token, old, adv, grad_scale=3.0)
    _check_policy(got, z0, token, old, adv, grad_scale=3.0)
    z.copy_(z0)
    got = _policy(kfac_gpu, z0, token, old, adv, dlogits=z, grad_scale=3.0)
    _check_policy(got, z0, token, old, adv, grad_scale=3.0)


def test_policy_gradient_against_differences(kfac_gpu):
    """The written gradient against central differences of the fp64 loss on the same
    logits. h = 1e-5: the differences are off by h^2/6 of a third derivative that the ratio,
    the advantage and the KL keep below 50 (1e-9), and by eps/h (1e-10)."""
    rows, vocab = 4, 6
    z, token, old, adv, ref = _policy_inputs(15, rows, vocab, F32)
    kw = dict(kl_coef=0.5, clip_low=0.3, clip_high=0.2)
    _, _, d = _policy(kfac_gpu, z, token, old, adv, ref=ref, **kw)
    x, have = host64(z), host64(d)
    tok = token.cpu().numpy()

    def f():
        return lo.policy_loss(x, tok, host64(old), host64(adv), host64(ref), low=0.3, high=0.2, kl_coef=0.5)[0][0]

    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + 1e-5
        up = f()
        x[i] = keep - 1e-5
        down = f()
        x[i] = keep
        assert abs(have[i] - (up - down) / 2e-5) <= 2e-8 + row_errors(x).max() * 4


# ---------------------------------------------------------------------------
# preference
# ---------------------------------------------------------------------------

def _prefer(kfac, z, token, begin, ref=None, mask=None, grad=True, dlogits=None, **kw):
    pairs = begin.numel() // 2
    seq, margin, loss = (torch.full((n,), 7.0, device="cuda") for n in (2 * pairs, pairs, 1))
    if grad and dlogits is None:
        dlogits = torch.full(z.shape, 7.0, dtype=z.dtype, device="cuda")
    kfac.kfac_preference_loss(z, token, begin, seq, margin, loss, dlogits=dlogits, ref_logp=ref, mask=mask, **kw)
    torch.cuda.synchronize()
    return loss, margin, seq, dlogits


def _check_prefer(got, z0, token, begin, ref=None, mask=None, beta=0.1, label_smoothing=0.0, grad_scale=1.0):
    loss, margin, seq, d = (None if t is None else host64(t) for t in got)
    z, tok, begin = host64(z0), token.cpu().numpy(), begin.cpu().tolist()
    ref = None if ref is None else host64(ref)
    mask = None if mask is None else mask.cpu().numpy()
    beta, smooth, scale = (float(np.float32(v)) for v in (beta, label_smoothing, grad_scale))
    want, x, sums, want_d = lo.preference_loss(z, tok, begin, ref, mask, beta, smooth, scale)
    pairs = len(x)
    err = row_errors(z)
    counted = np.array([(mask is None or bool(mask[t])) and 0 <= tok[t] < z.shape[1] for t in range(len(tok))])
    spans = list(zip(begin[:-1], begin[1:]))
    seq_err = np.array([err[a:b][counted[a:b]].sum() for a, b in spans])
    u_out = 1.01 * U
    assert (np.abs(seq - sums) <= seq_err + u_out * np.abs(sums)).all()
    x_err = abs(beta) * (seq_err[:pairs] + seq_err[pairs:])
    assert (np.abs(margin - x) <= x_err + u_out * np.abs(x) + 1e-14).all()
    # the loss changes by at most |dx| with x
    assert abs(loss[0] - want) <= (x_err.mean() if pairs else 0.0) + u_out * abs(want) + 1e-14
    if d is None:
        return
    inside = np.zeros(len(tok), dtype=bool)
    coef, coef_err = np.zeros(len(tok)), np.zeros(len(tok))
    for i in range(pairs):
        slope = scale * (smooth - 1 / (1 + math.exp(x[i]))) * beta / pairs
        for k, sign in ((i, 1), (pairs + i, -1)):
            a, b = spans[k]
            inside[a:b] = True
            coef[a:b] = sign * slope
            # sig' <= 1/4
            coef_err[a:b] = abs(scale * beta) / pairs * x_err[i] / 4 + abs(slope) * u_out
    assert (d[~inside] == 7.0).all()
    assert not d[inside & ~counted].any()
    bound = grad_bound(np.nan_to_num(want_d), z, tok, coef, coef_err, err, z0.dtype)
    off = np.abs(d - want_d)[inside] / bound[inside]
    say("preference", tuple(z.shape), z0.dtype, "gradient at", float(np.max(off, initial=0.0)), "of its bound")
    assert (off <= 1).all()


def _offsets(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", VOCABS)
def test_prefer_vocabularies(kfac_gpu, dtype, vocab):
    z, token, g = logits(200 + vocab, 9, vocab, dtype)
    begin, ref = _offsets(0, 2, 4, 5, 9), _vec(g, 4, 2.0)
    kw = dict(ref=ref, beta=0.3, label_smoothing=0.1, grad_scale=9.0)
    _check_prefer(_prefer(kfac_gpu, z, token, begin, **kw), z, token, begin, **kw)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", [16384, 65537, 131075, 163841])
def test_prefer_long_rows(kfac_gpu, dtype, vocab):
    z, token, g = logits(vocab, 4, vocab, dtype)
    begin = _offsets(0, 1, 4)
    kw = dict(beta=0.3, grad_scale=4.0)
    _check_prefer(_prefer(kfac_gpu, z, token, begin, **kw), z, token, begin, **kw)


@pytest.mark.parametrize("begin", [[0, 6, 12], [0, 0, 0], [2, 5, 5, 7, 11], [0, 12, 12], [12, 12, 12], [5],
                                   [0, 1, 2, 3, 4, 5, 6, 7, 8]])
@pytest.mark.parametrize("masked", ["none", "some", "a sequence", "all"])
def test_prefer_sequences_and_masks(kfac_gpu, begin, masked):
    rows, vocab = 12, 70
    z, token, g = logits(20, rows, vocab, F16)
    mask = {"none": None, "some": torch.arange(rows) % 3 != 1, "a sequence": torch.arange(rows) >= 5,
            "all": torch.zeros(rows, dtype=torch.bool)}[masked]
    token[3], token[10] = -100, vocab
    off = torch.zeros(rows, dtype=torch.bool)
    off[[3, 10]] = True
    if mask is not None:
        off |= ~mask
    off |= torch.tensor([not begin[0] <= t < begin[-1] for t in range(rows)])
    z0 = z.clone()
    z[off.cuda()] = float("nan")
    mask = None if mask is None else mask.cuda()
    ref = _vec(g, len(begin) - 1)
    b = _offsets(*begin)
    for kw in (dict(ref=ref, beta=0.5, label_smoothing=0.2), dict(beta=0.5)):
        kw.update(mask=mask, grad_scale=12.0)
        _check_prefer(_prefer(kfac_gpu, z, token, b, **kw), z0, token, b, **kw)


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 5), (24, 0)])
def test_prefer_pitches_in_place_and_alone(kfac_gpu, pad, offset):
    z, token, g = logits(21, 10, 515, BF16, pad, offset)
    z0 = z.clone()
    begin = _offsets(0, 4, 10)
    kw = dict(beta=0.2, grad_scale=10.0)
    alone = _prefer(kfac_gpu, z, token, begin, grad=False, **kw)
    _check_prefer(alone, z0, token, begin, **kw)
    got = _prefer(kfac_gpu, z, token, begin, dlogits=z, **kw)
    assert all(torch.equal(a, b) for a, b in zip(alone[:3], got[:3]))
    _check_prefer(got, z0, token, begin, **kw)


def test_prefer_many_pairs(kfac_gpu):
    rows = 1200
    z, token, g = logits(22, rows, 13, F32)
    begin = torch.tensor([t - t % 2 for t in range(rows + 1)], dtype=torch.int32, device="cuda")
    kw = dict(beta=0.4, label_smoothing=0.05, grad_scale=float(rows))
    _check_prefer(_prefer(kfac_gpu, z, token, begin, **kw), z, token, begin, **kw)


def test_prefer_long_sequences(kfac_gpu):
    rows = 2100
    z, token, g = logits(23, rows, 13, F32, std=1.0)
    begin = _offsets(0, 1000, 2100)
    kw = dict(beta=0.01, grad_scale=float(rows))
    _check_prefer(_prefer(kfac_gpu, z, token, begin, **kw), z, token, begin, **kw)


def test_prefer_extreme_margins(kfac_gpu):
    """Margins so large that the sigmoid is 0 or 1 in fp64."""
    z, token, g = logits(24, 4, 8, F32)
    begin = _offsets(0, 1, 2, 3, 4)
    ref = torch.tensor([3000.0, -3000.0, -3000.0, 3000.0], device="cuda")
    for smooth in (0.0, 0.1):
        kw = dict(ref=ref, beta=1.0, label_smoothing=smooth, grad_scale=4.0)
        loss, margin, seq, d = got = _prefer(kfac_gpu, z, token, begin, **kw)
        assert all(t.isfinite().all() for t in got)
        want, x, _, want_d = lo.preference_loss(host64(z), token.cpu().numpy(), begin.tolist(), host64(ref), None, 1.0,
                                                float(np.float32(smooth)), 4.0)
        assert abs(float(loss) - want) <= 1e-6 * want
        assert np.abs(host64(d) - want_d).max() <= 2e-5


# ---------------------------------------------------------------------------
# calls: streams, graphs, repeats
# ---------------------------------------------------------------------------

def test_losses_repeat_bit_for_bit(kfac_gpu):
    z, token, old, adv, ref = _policy_inputs(30, 300, 777, BF16)
    begin = _offsets(0, 100, 150, 220, 299)
    kw = dict(ref=ref, begin=begin, by_sequence=True, kl_coef=0.1)
    a, b = (_policy(kfac_gpu, z, token, old, adv, **kw) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (_prefer(kfac_gpu, z, token, begin) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_losses_on_another_stream(kfac_gpu):
    """The stream argument, with the call's own workspace, while the current stream goes on
    allocating."""
    z, token, old, adv, ref = _policy_inputs(31, 200, 3001, F16)
    begin = _offsets(0, 60, 200)
    want_p = _policy(kfac_gpu, z, token, old, adv)
    want_q = _prefer(kfac_gpu, z, token, begin)
    side = torch.cuda.Stream()
    logp, stats, d = torch.empty(200, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(z)
    seq, margin, loss, d2 = (torch.empty(2, device="cuda"), torch.empty(1, device="cuda"),
                             torch.empty(1, device="cuda"), torch.empty_like(z))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        kfac_gpu.kfac_policy_loss(z, token, old, adv, logp, stats, dlogits=d, stream=side)
        torch.full((1 << 16,), float("nan"), device="cuda")
        kfac_gpu.kfac_preference_loss(z, token, begin, seq, margin, loss, dlogits=d2, stream=side)
        torch.full((1 << 16,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(stats, want_p[0]) and torch.equal(logp, want_p[1]) and torch.equal(d, want_p[2])
    assert torch.equal(loss, want_q[0]) and torch.equal(seq, want_q[2]) and torch.equal(d2, want_q[3])


def test_losses_in_a_graph(kfac_gpu):
    """Both losses captured with one workspace and replayed on new inputs, eager calls and
    synchronisations between the replays."""
    rows, vocab = 40, 1500
    z, token, old, adv, ref = _policy_inputs(32, rows, vocab, BF16)
    begin = _offsets(0, 10, 22, 30, 40)
    need = max(kfac_gpu.kfac_policy_loss_workspace(rows, vocab, 4),
               kfac_gpu.kfac_preference_loss_workspace(rows, vocab, 2))
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    out = {n: torch.empty(k, device="cuda") for n, k in
           (("logp", rows), ("stats", 4), ("seq", 4), ("margin", 2), ("loss", 1))}
    d1, d2 = torch.empty_like(z), torch.empty_like(z)

    def calls():
        kfac_gpu.kfac_policy_loss(z, token, old, adv, out["logp"], out["stats"], dlogits=d1, ref_logp=ref,
                                  seq_begin=begin, by_sequence=True, kl_coef=0.1, workspace=ws)
        kfac_gpu.kfac_preference_loss(z, token, begin, out["seq"], out["margin"], out["loss"], dlogits=d2,
                                      workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(4):
        z.copy_(_policy_inputs(40 + k, rows, vocab, BF16)[0])
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in (*out.values(), d1, d2)]
        for t in (*out.values(), d1, d2):
            t.fill_(3.0)
        calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(have, (*out.values(), d1, d2))), k


def test_two_calls_at_once(kfac_gpu):
    """Two streams, a workspace each."""
    ins = [_policy_inputs(50 + k, 130, 4000, BF16) for k in range(2)]
    want = [_policy(kfac_gpu, *i[:4], ref=i[4], kl_coef=0.1) for i in ins]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty(130, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(i[0])) for i in ins]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (z, token, old, adv, ref), (logp, stats, d) in zip(streams, ins, outs):
            with torch.cuda.stream(s):
                kfac_gpu.kfac_policy_loss(z, token, old, adv, logp, stats, dlogits=d, ref_logp=ref, kl_coef=0.1)
    torch.cuda.synchronize()
    for (logp, stats, d), w in zip(outs, want):
        assert torch.equal(stats, w[0]) and torch.equal(logp, w[1]) and torch.equal(d, w[2])


def _refused(kfac, call, **kw):
    with pytest.raises(kfac.KfacError, match="overlap"):
        call(**kw)


def test_results_lie_apart_from_each_other(kfac_gpu):
    """A result inside another one or the workspace is refused, before any launch; one between the
    rows of the gradient is not."""
    rows, vocab = 6, 10
    z, token, old, adv, ref = _policy_inputs(60, rows, vocab, F32)
    buf = torch.zeros(rows * 24 + 64, device="cuda")
    wide = buf[:rows * 24].view(rows, 24)
    d = wide[:, :vocab]

    def policy(**kw):
        own = dict(logp=torch.zeros(rows, device="cuda"), stats=torch.zeros(4, device="cuda"), dlogits=d)
        kfac_gpu.kfac_policy_loss(z, token, old, adv, **{**own, **kw})

    one = torch.zeros(rows + 4, device="cuda")
    _refused(kfac_gpu, policy, logp=one[:rows], stats=one[rows - 1:rows + 3])
    _refused(kfac_gpu, policy, stats=wide[0, 9:13])              # the last element of the first row
    _refused(kfac_gpu, policy, stats=wide[1, :4])
    _refused(kfac_gpu, policy, stats=buf[22:26])                 # past the first row's end, into the second
    _refused(kfac_gpu, policy, logp=wide[rows - 1, 9:9 + rows])  # the last element of all
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    _refused(kfac_gpu, policy, stats=ws[1024:1040].view(F32), workspace=ws)
    _refused(kfac_gpu, policy, workspace=ws, dlogits=ws[512:512 + rows * vocab * 4].view(F32).view(rows, vocab))
    assert not buf.any() and not one.any() and not ws.any()
    want = _policy(kfac_gpu, z, token, old, adv)
    for at in (10, 20):                                          # right behind a row, right before the next
        policy(stats=wide[2, at:at + 4])
        assert torch.equal(wide[2, at:at + 4], want[0]) and torch.equal(d, want[2])
    policy(logp=wide[rows - 1, 10:10 + rows])
    assert torch.equal(wide[rows - 1, 10:10 + rows], want[1]) and torch.equal(d, want[2])
    begin = _offsets(0, 2, 6)
    buf.zero_()

    def prefer(**kw):
        own = dict(seq_logp=torch.zeros(2, device="cuda"), margin=torch.zeros(1, device="cuda"),
                   loss=torch.zeros(1, device="cuda"), dlogits=d)
        kfac_gpu.kfac_preference_loss(z, token, begin, **{**own, **kw})

    _refused(kfac_gpu, prefer, seq_logp=one[:2], margin=one[1:2])
    _refused(kfac_gpu, prefer, margin=one[:1], loss=one[:1])
    _refused(kfac_gpu, prefer, loss=wide[3, 2:3])
    _refused(kfac_gpu, prefer, seq_logp=wide[3, 9:11])
    _refused(kfac_gpu, prefer, loss=ws[:4].view(F32), workspace=ws)
    assert not buf.any() and not one.any()
    prefer(seq_logp=one[:2], margin=one[2:3], loss=wide[0, 10:11])
    torch.cuda.synchronize()
    got = _prefer(kfac_gpu, z, token, begin)
    assert torch.equal(wide[0, 10:11], got[0]) and torch.equal(one[2:3], got[1]) and torch.equal(d, got[3])


def test_bounds_are_the_types_own():
    for t in (F32, F16, BF16):
        assert HALF_STEP[t] == torch.finfo(t).eps / 2
        assert FLOOR[t] <= torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
