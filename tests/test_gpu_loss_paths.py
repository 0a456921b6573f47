"""The losses and the clipping at the sizes where their launches change: rows held by a wave, by
blocks of every size and by none; counts that the blocks take for themselves, in slices, by
sequence, over many sequences; sums in one step and in two; gradients that pass the caches by;
tables sent to the device; and what the calls allow beside that."""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from loss_cases import U, grad_bound, host64, logits, row_errors
from oracle import loss_oracle as lo
from test_gpu_grads import _check_clip, _check_trust, _clip, _norm, _tensors, _trust
from test_gpu_loss import BF16, F16, F32, _check_policy, _check_prefer, _offsets, _policy, _policy_inputs, _prefer, _vec

pytestmark = pytest.mark.gpu


# 16-byte groups of a row at which its threads change: a wave of 4 groups, 256 threads of 4 and 8,
# 512 of 8 and 16, 1024 of 16 and 19, a row in memory
EDGES = [256, 1024, 2048, 4096, 8192, 16384, 19456]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("groups", EDGES)
@pytest.mark.parametrize("offset", [0, 1])
def test_rows_on_both_sides_of_an_edge(kfac_gpu, dtype, groups, offset):
    """Rows of exactly that many groups, one element fewer and a whole group more; offset 1: no row
    begins at a multiple of 16 bytes. By sequence: the rows are then held whole; otherwise so few
    are cut into parts."""
    ev = 4 if dtype == F32 else 8
    for vocab in (groups * ev - 1, groups * ev, groups * ev + ev):
        z, token, old, adv, ref = _policy_inputs(vocab + offset, 2, vocab, dtype, 0, offset)
        token[1] = vocab - 1
        old[1] = lo.row_logp(host64(z[1]), vocab - 1)[0] + 0.1
        for by in (dict(), dict(begin=_offsets(0, 1, 2), by_sequence=True)):
            kw = dict(ref=ref, kl_coef=0.1, grad_scale=2.0, **by)
            _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)
        kw = dict(beta=0.3, grad_scale=2.0)
        _check_prefer(_prefer(kfac_gpu, z, token, _offsets(0, 1, 2), **kw), z, token, _offsets(0, 1, 2), **kw)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("groups", [4096, 8192, 19456])
@pytest.mark.parametrize("offset", [0, 1])
def test_rows_without_a_gradient(kfac_gpu, dtype, groups, offset):
    """Rows of which nothing but l is wanted, at the lengths where they stay in memory; -inf in whole
    groups, and the maximum in the first, a middle and the last element."""
    ev = 4 if dtype == F32 else 8
    for vocab in (groups * ev - 1, groups * ev, groups * ev + ev):
        z, token, old, adv, ref = _policy_inputs(vocab + offset + 1, 3, vocab, dtype, 0, offset)
        for t, j in enumerate((0, vocab // 2, vocab - 1)):
            z[t, vocab // 4: vocab // 4 + 5000] = float("-inf")
            z[t, j] = 14.0
            token[t] = j
            old[t] = lo.row_logp(host64(z[t]), j)[0] + 0.1
        kw = dict(ref=ref, kl_coef=0.1, begin=_offsets(0, 1, 3), by_sequence=True)
        _check_policy(_policy(kfac_gpu, z, token, old, adv, grad=False, **kw), z, token, old, adv, **kw)
        kw = dict(ref=_vec(torch.Generator().manual_seed(1), 2), beta=0.3)
        _check_prefer(_prefer(kfac_gpu, z, token, _offsets(0, 1, 3), grad=False, **kw), z, token, _offsets(0, 1, 3), **kw)


@pytest.mark.parametrize("rows", [1, 3, 63, 64, 65])
@pytest.mark.parametrize("dtype,vocab", [(F32, 4097), (F32, 4100), (F32, 8191), (F32, 8193), (BF16, 8199), (BF16, 8200),
                                         (F16, 16385), (BF16, 50001), (F32, 262143), (F32, 262144)])
def test_few_long_rows(kfac_gpu, rows, dtype, vocab):
    """Rows in parts of 1024 groups, up to 64 parts and one more; up to 64 rows and one more."""
    if rows > 3 and vocab > 60000:
        rows = {63: 4, 64: 5, 65: 6}[rows]
    z, token, old, adv, ref = _policy_inputs(rows + vocab, rows, vocab, dtype, 0, 1)
    mask = torch.arange(rows) % 5 != 3
    begin = None if rows < 60 else _offsets(2, 30, rows - 1)
    kw = dict(ref=ref, kl_coef=0.1, grad_scale=float(rows), mask=mask.cuda(), begin=begin)
    z0 = z.clone()
    got = _policy(kfac_gpu, z, token, old, adv, **kw)
    _check_policy(got, z0, token, old, adv, **kw)
    alone = _policy(kfac_gpu, z, token, old, adv, grad=False, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], alone[:2]))
    again = _policy(kfac_gpu, z, token, old, adv, dlogits=z, **kw)
    inside = torch.arange(rows, device="cuda") >= 0 if begin is None else \
        (torch.arange(rows, device="cuda") >= 2) & (torch.arange(rows, device="cuda") < rows - 1)
    assert torch.equal(got[0], again[0]) and torch.equal(got[2][inside], again[2][inside])
    assert torch.equal(again[2][~inside], z0[~inside])


@pytest.mark.parametrize("by_sequence", [False, True])
def test_long_rows_of_masked_and_bad_values(kfac_gpu, by_sequence):
    """Whole parts of -inf or of the lowest value, rows of nothing else, NaN and +inf in one part."""
    low = torch.finfo(F32).min
    begin = _offsets(0, 3, 8) if by_sequence else None
    z, token, old, adv, ref = _policy_inputs(3, 8, 20000, F32)
    z[0, :9000] = float("-inf")
    z[1, 4096:] = low
    z[2] = low
    z[3, :19999] = float("-inf")
    token[:4] = torch.tensor([19999, 5, 12345, 19999], device="cuda")
    old = torch.tensor([lo.row_logp(a, b)[0] for a, b in zip(host64(z), token.tolist())]).float().cuda() + 0.05
    kw = dict(begin=begin, by_sequence=by_sequence, grad_scale=8.0)
    _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)
    z[4, 17000], z[5, 3], z[6] = float("nan"), float("inf"), float("-inf")
    stats, logp, d = _policy(kfac_gpu, z, token, old, adv, **kw)
    assert logp[4:7].isnan().all() and logp[[0, 1, 2, 3, 7]].isfinite().all()
    assert d[4:7].isnan().all() and d[[0, 1, 2, 3, 7]].isfinite().all() and stats[0].isnan()


@pytest.mark.parametrize("place", [0, 1, 6, 7, 8, 9, 1022, 1023, 1024, 1029])
@pytest.mark.parametrize("offset", [0, 3])
def test_the_token_anywhere_in_its_row(kfac_gpu, place, offset):
    """In front of the first aligned group, in the first and last group, behind the last."""
    for dtype in (F32, BF16):
        z, token, old, adv, ref = _policy_inputs(place, 3, 1030, dtype, 1, offset)
        token[:] = place
        old = torch.tensor([lo.row_logp(a, place)[0] for a in host64(z)]).float().cuda() - 0.1
        kw = dict(grad_scale=3.0)
        _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)


@pytest.mark.parametrize("rows", [255, 256, 257, 1023, 1024, 1025, 4096, 4097, 9001, 40000])
@pytest.mark.parametrize("layout", ["none", "one", "few", "few by sequence", "many by sequence"])
def test_counts(kfac_gpu, rows, layout):
    z, token, old, adv, ref = _policy_inputs(rows, rows, 7, F32)
    # of tens of thousands of ratios some lie within fp32's reach of a bound: those rows move off it
    ratio = torch.exp(torch.log_softmax(z.double(), 1).gather(1, token[:, None])[:, 0] - old.double())
    old[torch.minimum((ratio - 0.8).abs(), (ratio - 1.2).abs()) < 1e-3] += 0.01
    begin = {"none": None, "one": [3, rows - 2], "few": [0, rows // 5, rows // 2, rows - 1],
             "few by sequence": [0, rows // 5, rows // 5, rows // 2, rows - 1],
             "many by sequence": list(range(0, rows + 1, 7))}[layout]
    if begin is not None:
        begin = _offsets(*begin)
    mask = torch.rand(rows, generator=torch.Generator().manual_seed(rows)) < 0.8
    mask[: rows // 8] = False
    kw = dict(begin=begin, by_sequence=layout.endswith("by sequence"), mask=mask.cuda(), grad_scale=float(rows))
    _check_policy(_policy(kfac_gpu, z, token, old, adv, **kw), z, token, old, adv, **kw)


@pytest.mark.parametrize("rows,layout", [(16384, "none"), (16385, "none"), (7168, "many by sequence"),
                                         (7175, "many by sequence")])
def test_counts_on_both_sides_of_an_edge(kfac_gpu, rows, layout):
    """The last rows that are summed in one step; 1024 sequences and one more."""
    test_counts(kfac_gpu, rows, layout)


@pytest.mark.parametrize("rows,pairs", [(300, 1), (5000, 1), (9000, 1), (9000, 2), (9000, 4), (9000, 8), (9000, 9),
                                        (20000, 16), (3000, 40), (2000, 500)])
def test_pairs(kfac_gpu, rows, pairs):
    """Sequences of one row to thousands over one wave to eight, losses of one block and of several."""
    z, token, g = logits(rows + pairs, rows, 9, F32, std=1.0)
    cuts = torch.sort(torch.randint(0, rows + 1, (2 * pairs - 1,), generator=g)).values.tolist()
    begin = _offsets(1, *[max(1, c) for c in cuts], rows)
    kw = dict(ref=_vec(g, 2 * pairs, 3.0), beta=0.02, label_smoothing=0.1, grad_scale=float(rows))
    for grad in (True, False):
        _check_prefer(_prefer(kfac_gpu, z, token, begin, grad=grad, **kw), z, token, begin, **kw)


@pytest.mark.parametrize("rows,vocab,dtype", [(300, 131072, BF16), (1100, 20000, F32), (17000, 1000, F32)])
def test_gradients_past_the_caches(kfac_gpu, rows, vocab, dtype):
    """Gradients of more than 64 MB, stored past the caches; also in place."""
    z, token, old, adv, ref = _policy_inputs(rows, rows, vocab, dtype)
    assert z.numel() * z.element_size() > 64 << 20
    z0 = z.clone()
    ratio = torch.exp(torch.log_softmax(z.double(), 1).gather(1, token[:, None])[:, 0] - old.double())
    old[torch.minimum((ratio - 0.8).abs(), (ratio - 1.2).abs()) < 1e-3] += 0.01    # off the bounds, as above
    kw = dict(ref=ref, kl_coef=0.1, grad_scale=float(rows))
    got = _policy(kfac_gpu, z, token, old, adv, **kw)
    _check_policy(got, z0, token, old, adv, **kw)
    again = _policy(kfac_gpu, z, token, old, adv, dlogits=z, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    z = z0.clone()
    begin = _offsets(0, rows // 4, rows // 2, rows - 10, rows - 3)
    kw = dict(beta=0.001, grad_scale=float(rows))
    got = _prefer(kfac_gpu, z, token, begin, **kw)
    _check_prefer(got, z0, token, begin, **kw)
    z[rows - 3:] = 7.0
    again = _prefer(kfac_gpu, z, token, begin, dlogits=z, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_many_rows_of_a_gradient_launch(kfac_gpu):
    """More rows than one launch of the preference gradient takes, in blocks of a wave a row and of
    a row each."""
    for rows, vocab, dtype in ((262200, 3, F16), (65600, 2060, F16)):
        z, token, g = logits(rows, rows, vocab, dtype, std=1.0, device="cuda")
        begin = _offsets(0, rows // 3, rows - 5)
        seq, margin, loss = (torch.empty(n, device="cuda") for n in (2, 1, 1))
        d = torch.full_like(z, 7.0)
        kfac_gpu.kfac_preference_loss(z, token, begin, seq, margin, loss, dlogits=d, beta=1e-4, grad_scale=float(rows))
        torch.cuda.synchronize()
        assert (d[rows - 5:] == 7).all()
        x = float(margin)
        slope = -float(rows) * 1e-4 / (1 + np.exp(x))
        for t in (0, 1, rows // 3 - 1, rows // 3, rows - 262200 // 4 * 3, rows - 65540 if rows > 65540 else 5, rows - 6):
            if t < 0:
                continue
            p = torch.softmax(z[t].double(), 0)
            p[token[t]] -= 1
            want = -p * slope * (1 if t < rows // 3 else -1)
            # fp16 result of a coefficient known to 1e-4 (a margin of sums over 10^5 rows, off by
            # beta * rows * err_l / 4 = 2e-5) and of fp32 operations
            assert ((d[t].double() - want).abs() <= want.abs() * (2.0 ** -11 + 2e-4) + 2.0 ** -25).all(), t
        say("preference gradient over", rows, "rows")


@pytest.mark.parametrize("rows,vocab,pairs", [(262200, 3, 12), (1500, 40, 9), (1500, 40, 40)])
def test_the_loss_of_several_shares(kfac_gpu, rows, vocab, pairs):
    """More pairs than one block takes: their shares are added by the gradient's launch, the first of two
    where the rows are many, or by one of their own without a gradient, to the same bits."""
    z, token, g = logits(rows + pairs, rows, vocab, F32, std=1.0)
    cuts = torch.linspace(2, rows - 3, 2 * pairs + 1).int().tolist()
    begin = _offsets(*cuts)
    d = torch.full((rows, vocab), 7.0, device="cuda")
    kw = dict(beta=1e-3, grad_scale=float(rows))
    loss, margin, seq, _ = _prefer(kfac_gpu, z, token, begin, dlogits=d, **kw)
    alone = _prefer(kfac_gpu, z, token, begin, grad=False, **kw)
    assert torch.equal(loss, alone[0]) and torch.equal(margin, alone[1]) and torch.equal(seq, alone[2])
    x = host64(margin)
    # the loss moves by at most as much as a margin, which is off by half a step as it stands
    assert abs(float(loss) - np.logaddexp(0, -x).mean()) <= U * (np.abs(x).mean() + 1.01 * float(loss)) + 1e-14
    assert (d[:cuts[0]] == 7).all() and (d[cuts[-1]:] == 7).all()
    one = torch.nn.functional.one_hot(token, vocab).double()
    side = np.repeat([1.0, -1.0], pairs)
    slope = np.tile(-rows * 1e-3 / (1 + np.exp(x)) / pairs, 2) * side
    coef = torch.from_numpy(np.repeat(slope, np.diff(cuts))).cuda()[:, None]
    want = coef * (one - z.double().softmax(1))[cuts[0]:cuts[-1]]
    # l of a row is off by less than 1e-5, a softmax of 40 elements by 2e-5 of itself; the coefficient by
    # a quarter of its margin's half step and its own
    err = 2e-5 + U * (float(np.abs(x).max()) / 4 + 2)
    assert ((d[cuts[0]:cuts[-1]] - want).abs() <= err * coef.abs()).all()


def test_losses_without_rows(kfac_gpu):
    e = torch.empty(0, device="cuda")
    z = torch.empty(0, 5, device="cuda")
    out = torch.full((4,), 7.0, device="cuda")
    begin = torch.zeros(5, dtype=torch.int32, device="cuda")
    kfac_gpu.kfac_policy_loss(z, e.long(), e, e, e, out, dlogits=z, seq_begin=begin, by_sequence=True)
    assert not out.any()
    seq, margin, loss = (torch.full((n,), 7.0, device="cuda") for n in (4, 2, 1))
    ref = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    kfac_gpu.kfac_preference_loss(z, e.long(), begin, seq, margin, loss, dlogits=z, ref_logp=ref, beta=0.5)
    assert not seq.any() and margin.tolist() == [1.0, 1.0]           # 0.5 ((0 - 1) - (0 - 3))
    assert abs(float(loss) - np.log1p(np.exp(-1.0))) < 1e-7
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = torch.ones(3, 5, device="cuda")
    kfac_gpu.kfac_preference_loss(z, torch.zeros(3, dtype=torch.long, device="cuda"), none, e, e, loss, dlogits=z)
    assert float(loss) == 0.0 and (z == 1).all()


def test_offsets_that_decrease_stay_inside(kfac_gpu):
    """Offsets out of order or out of range: no result is promised, and no write outside the
    rows. The buffers around the gradient are checked."""
    rows, vocab = 50, 40
    z, token, old, adv, ref = _policy_inputs(5, rows, vocab, F32)
    for begin in ([0, 40, 10, 50], [-5, 20, 1000, 2000000000], [30, 0, 0, 0], [2000000000, -2000000000, 7, 3]):
        buf = torch.full((rows + 2, vocab), 7.0, device="cuda")
        b = _offsets(*begin, rows)
        kfac_gpu.kfac_policy_loss(z, token, old, adv, torch.empty(rows, device="cuda"), torch.empty(4, device="cuda"),
                                  dlogits=buf[1:-1], seq_begin=b, by_sequence=True)
        kfac_gpu.kfac_preference_loss(z, token, b, torch.empty(4, device="cuda"), torch.empty(2, device="cuda"),
                                      torch.empty(1, device="cuda"), dlogits=buf[1:-1])
        torch.cuda.synchronize()
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()


@pytest.mark.parametrize("count,size", [(108, 5000), (109, 5000), (150, 1 << 20), (64, 4097), (65, 4096), (4100, 50),
                                        (300, 1)])
def test_tables_of_tensors(kfac_gpu, count, size):
    """Tables in the arguments (of an update, to 108 tensors) and sent ahead; 150 MB and 600 MB of gradients, found
    in the caches again and not; one to three steps of the search for a unit's tensor."""
    sizes = [size + i % 3 for i in range(count)]
    grads = _tensors(count, sizes, [F32, BF16] if size < 1 << 20 else [F32])
    outs, norm = _clip(kfac_gpu, grads, 0.5)
    assert _norm(kfac_gpu, grads) == norm
    if size < 1 << 20:
        _check_clip(outs, norm, grads, 0.5)
        P, w = _tensors(count + 1, sizes, [F32]), _tensors(count + 2, sizes, [F32])
        w0 = [t.clone() for t in w]
        g = [(p * 0.1).to(t.dtype) for p, t in zip(P, grads)]
        _check_trust(_trust(kfac_gpu, P, g, w, 0.1, 1e-4), w, w0, P, g, 0.1, 1e-4)
        return
    want = float(sum(t.double().square().sum() for t in grads).sqrt())
    assert abs(norm - want) <= 1.01 * U * want
    c = 0.5 / want
    for o, t in zip(outs, grads):
        assert ((o.double() - t.double() * c).abs() <= 2.02 * U * (t.double() * c).abs()).all()


@pytest.mark.parametrize("count", [138, 139, 194, 195])
def test_tables_on_both_sides_of_an_edge(kfac_gpu, count):
    """The most tensors whose tables the clipping and the norm take in their arguments, and one more."""
    test_tables_of_tensors(kfac_gpu, count, 5000)


def test_a_call_of_one_block_and_of_more(kfac_gpu):
    """Sixteen units go to one block, seventeen do not; the sums agree to fp64."""
    for n in (16 * 4096, 16 * 4096 + 1):
        t = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
        outs, norm = _clip(kfac_gpu, [t], 0.5)
        _check_clip(outs, norm, [t], 0.5)
        outs, norm = _clip(kfac_gpu, [t[:4096 * 8], t[4096 * 8:]], 0.5)
        _check_clip(outs, norm, [t[:4096 * 8], t[4096 * 8:]], 0.5)


def test_workspace_that_is_too_small_is_refused(kfac_gpu):
    z, token, old, adv, ref = _policy_inputs(6, 8, 40, F32)
    small = torch.empty(100, dtype=torch.uint8, device="cuda")
    with pytest.raises(kfac_gpu.KfacError, match="WORKSPACE"):
        kfac_gpu.kfac_policy_loss(z, token, old, adv, torch.empty_like(old), torch.empty(4, device="cuda"), workspace=small)
    with pytest.raises(kfac_gpu.KfacError, match="WORKSPACE"):
        kfac_gpu.kfac_grad_norm([z.contiguous()], torch.empty(1, device="cuda"), workspace=small)
    with pytest.raises(ValueError, match="device"):
        kfac_gpu.kfac_grad_norm([z.contiguous()], torch.empty(1, device="cuda"), workspace=small.cpu())
    with pytest.raises(ValueError, match="device"):
        kfac_gpu.kfac_policy_loss(z, token.cpu(), old, adv, torch.empty_like(old), torch.empty(4, device="cuda"))


def test_workspaces_hold_anything_before_a_call(kfac_gpu):
    """Nothing of an earlier call, or of other use, is taken for this one's."""
    z, token, old, adv, ref = _policy_inputs(7, 700, 300, F16)
    begin = _offsets(*range(0, 701, 2))
    grads = _tensors(9, [50000] * 120, [BF16])
    want = None
    for fill in (0, 255, 127):
        ws = torch.full((1 << 20,), fill, dtype=torch.uint8, device="cuda")
        logp, stats, d = torch.empty(700, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(z)
        kfac_gpu.kfac_policy_loss(z, token, old, adv, logp, stats, dlogits=d, ref_logp=ref, kl_coef=0.1, seq_begin=begin,
                                  by_sequence=True, workspace=ws)
        ws.fill_(fill)
        seq, margin, loss, d2 = (torch.empty(350, device="cuda"), torch.empty(175, device="cuda"),
                                 torch.empty(1, device="cuda"), torch.empty_like(z))
        kfac_gpu.kfac_preference_loss(z, token, begin, seq, margin, loss, dlogits=d2, workspace=ws)
        ws.fill_(fill)
        norm, outs = torch.empty(1, device="cuda"), [torch.empty_like(t) for t in grads]
        kfac_gpu.kfac_grad_clip(grads, outs, 0.1, norm, workspace=ws)
        torch.cuda.synchronize()
        got = [logp, stats, d, seq, margin, loss, d2, norm, *outs]
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        want = got


def _unlikely(dtype, vocab):
    """Two rows, the first with a logit of -inf at its token."""
    z, token, old, adv, ref = _policy_inputs(77, 2, vocab, dtype)
    z[0, int(token[0])] = float("-inf")
    return z, token, old, adv, ref


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", [24, 3000])
@pytest.mark.parametrize("smooth", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("first", [True, False])
def test_prefer_a_token_without_probability(kfac_gpu, dtype, vocab, smooth, first):
    """l of -inf: a margin of -inf or +inf, a loss that is infinite or has none of it, and a gradient
    whose sigmoid is 0 or 1: with no error but the row's own, the rounding of the coefficient (1 u)
    and those of grad_bound."""
    z, token, *_ = _unlikely(dtype, vocab)
    if not first:
        z, token = z.flip(0), token.flip(0)
    loss, margin, seq, d = _prefer(kfac_gpu, z, token, _offsets(0, 1, 2), beta=0.5, label_smoothing=smooth)
    zz, tok = host64(z), token.cpu().numpy()
    want, x, sums, want_d = lo.preference_loss(zz, tok, [0, 1, 2], beta=0.5, smooth=smooth)
    assert float(loss) == want and float(margin) == x[0] and host64(seq)[0 if first else 1] == -np.inf
    coef = np.array([1.0, -1.0]) * (smooth - (1.0 if first else 0.0)) * 0.5
    bound = grad_bound(want_d, zz, tok, coef, np.abs(coef) * U, row_errors(zz), dtype)
    assert (np.abs(host64(d) - want_d) <= bound).all()


@pytest.mark.parametrize("vocab", [24, 3000, 4100])
def test_policy_a_token_without_probability(kfac_gpu, vocab):
    """l of -inf: the ratio is 0, the KL infinite, and without a KL term the row has no gradient."""
    z, token, old, adv, ref = _unlikely(F32, vocab)
    adv = adv.abs()
    stats, logp, d = (host64(t) for t in _policy(kfac_gpu, z, token, old, adv, ref=ref))
    want, want_l, want_d = lo.policy_loss(host64(z), token.cpu().numpy(), host64(old), host64(adv), host64(ref))
    assert logp[0] == -np.inf and stats[2] == np.inf == want[2] and not d[0].any() and not want_d[0].any()
    # |error| of l, and of the ratio of row 1 relative to it, weighted by 1/2
    err = row_errors(host64(z))[1]
    ratio = np.exp(want_l[1] - host64(old)[1])
    assert abs(logp[1] - want_l[1]) <= err + 1.01 * U * abs(want_l[1])
    assert np.abs(stats[:2] - want[:2]).max() <= 0.5 * ratio * host64(adv)[1] * err + 1.01 * U * abs(want[1])
    assert stats[3] == np.float32(want[3])


def _launches(kfac, call):
    """Kernel launches of a call by name."""
    kfac.kfac_timing_reset()
    kfac.kfac_timing_enable(True)
    try:
        call()
    finally:
        kfac.kfac_timing_enable(False)
    counts = {kfac.kfac_kernel_name(i): kfac.kfac_timing_read(i)[1] for i in range(kfac.kfac_timing_kernels())}
    kfac.kfac_timing_reset()
    return {k: n for k, n in counts.items() if n}


@pytest.mark.parametrize("rows,vocab,pairs,own", [(3000, 64, 1, True), (3001, 64, 1, False), (20000, 100, 1, False),
                                                  (3001, 2, 16, False), (65536, 16, 4, False), (1000, 1000, 4, True)])
def test_rows_that_form_their_own_coefficient(kfac_gpu, rows, vocab, pairs, own):
    """A row's wave adds up its whole pair, which is quadratic in the rows: above 3000 of them, however few
    bytes they have, each sequence is added up once, by a kernel of its own."""
    z, token, g = logits(rows + pairs, rows, vocab, F32 if rows * vocab < 1 << 21 else BF16, std=1.0)
    begin = _offsets(*[rows * i // (2 * pairs) for i in range(2 * pairs)], rows)
    got = []
    launched = _launches(kfac_gpu, lambda: got.extend(_prefer(kfac_gpu, z, token, begin, beta=1e-3, grad_scale=float(rows))))
    assert ("pref_pairs_kernel" in launched) != own and launched["pref_grad_kernel"] == 1
    _check_prefer(got, z, token, begin, beta=1e-3, grad_scale=float(rows))


@pytest.mark.parametrize("rows,seqs,own", [(12500, 2, True), (12501, 2, False), (12500, 1000, True), (12501, 1000, False),
                                           (40000, 300, True), (40001, 300, False), (100000, 16, False)])
def test_rows_that_count_the_sequences(kfac_gpu, rows, seqs, own):
    """Every row's wave looks through the counts of all sequences, up to 200000 steps of 64 of them over all
    rows; beyond that they are counted once. Slices of a sequence count each: 16 at 12500 rows in two."""
    vocab = 5
    z, token, g = logits(rows + seqs, rows, vocab, F32)
    cuts = [rows * i // seqs for i in range(seqs)] + [rows]
    cuts[1] = cuts[0]                                         # an empty one
    begin = _offsets(*cuts)
    l = torch.log_softmax(z.double(), 1).gather(1, token[:, None])[:, 0]
    got = []
    launched = _launches(kfac_gpu, lambda: got.extend(_policy(kfac_gpu, z, token, l.float(), torch.ones_like(l).float(),
                                                               begin=begin, by_sequence=True, grad_scale=float(rows))))
    assert ("loss_nonempty_kernel" in launched) != own
    # ratios of 1 and advantages of 1: the rows' weights, which add up to 1, are the slopes
    lengths = np.diff(cuts)
    weight = np.repeat(1.0 / ((lengths > 0).sum() * np.maximum(lengths, 1)), lengths)
    stats, logp, d = got
    err = row_errors(host64(z)).max() + U * float(l.abs().max())
    assert abs(float(stats[1]) + 1.0) <= 2 * err + U
    want = (z.double().softmax(1) - torch.nn.functional.one_hot(token, vocab)) * torch.from_numpy(weight * rows).cuda()[:, None]
    bound = torch.from_numpy(weight * rows).cuda()[:, None] * (4 * err + 6 * U)
    assert ((d.double() - want).abs() <= bound).all()
