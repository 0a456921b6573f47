"""Host-side checks of the network capture (no GPU): the weight layout matches the
patch columns of the K-FAC activation factor, and the hooks record every layer with
the geometry the library expects."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle
from oracle import loss_oracle as lo

cap_mod = pytest.importorskip("fac_second_order_amd.capture")


@pytest.mark.parametrize("k,s,p,bias", [(3, 2, 1, False), (1, 1, 0, True), (7, 2, 3, False)])
def test_weight_matrix_matches_patch_columns(k, s, p, bias):
    """conv2d(x, W) equals X W_mat^T with X the oracle's im2col patches: the matrix
    layout the capture gives the library is the one its factor A is built on."""
    torch.manual_seed(0)
    conv = torch.nn.Conv2d(5, 4, k, s, p, bias=bias).double()
    x = torch.randn(2, 5, 9, 9, dtype=torch.float64)
    y = conv(x).permute(0, 2, 3, 1).reshape(-1, 4).detach().numpy()
    X = oracle.im2col_nhwc(x.permute(0, 2, 3, 1).numpy(), k, k, s, s, p, p, bias)
    W = cap_mod.KfacCapture._to_matrix(conv).double().numpy()
    assert np.allclose(X @ W.T, y, rtol=1e-12, atol=1e-12)


def test_matrix_round_trip():
    torch.manual_seed(1)
    for m in (torch.nn.Conv2d(3, 6, 3, 1, 1, bias=False), torch.nn.Linear(7, 5)):
        before = [t.detach().clone() for t in m.parameters()]
        mat = cap_mod.KfacCapture._to_matrix(m)
        for t in m.parameters():
            t.data.zero_()
        cap_mod.KfacCapture._from_matrix(m, mat)
        for b, t in zip(before, m.parameters()):
            assert torch.equal(b, t.data)


def test_hooks_record_every_layer():
    torch.manual_seed(2)
    model = cap_mod.ResNet50(classes=10)
    cap = cap_mod.KfacCapture(model)
    x = torch.randn(2, 3, 32, 32)
    loss = F.cross_entropy(model(x), torch.tensor([1, 7]))
    loss.backward()
    layers, bns = cap._geometry()
    assert len(layers) == 54 and len(bns) == 53
    for L, a, g in zip(layers, cap.act, cap.gout):
        assert (L.h + 2 * L.ph - L.kh) // L.sh + 1 == L.h_out
        assert a.dtype == torch.float16 and a.is_contiguous() and a.shape == (L.n, L.h, L.w, L.c_in) or \
            a.shape == (L.n, L.c_in)
        assert g.dtype == torch.float16 and g.is_contiguous()
    assert layers[0].c_in == 3 and layers[0].kh == 7 and layers[-1].c_out == 10 and layers[-1].bias == 1
    assert sum(L.kh == 3 for L in layers) == 16 and sum(L.sh == 2 for L in layers) == 7
    for B, xh, gb in zip(bns, cap.xhat, cap.bgout):
        assert xh.shape == (B.n, B.hw, B.c) == gb.shape and xh.is_contiguous() and gb.is_contiguous()
    # the classifier's captured output gradient is n times the batch-mean gradient
    logits = model(x)
    p = torch.softmax(logits.detach(), 1)
    p[[0, 1], [1, 7]] -= 1
    assert torch.allclose(cap.gout[-1].float(), p.half().float(), atol=2e-3)
    cap.remove()


class Recorder:
    """Stands in for KfacStep: what a step was given."""

    def __init__(self, layers, bns, dev, **kw):
        self.made, self.options, self.calls = (layers, bns), kw, []

    def step(self, *args, **kw):
        # layers of None: those it was made for
        kw["layers"], kw["bn_layers"] = kw["layers"] or self.made[0], kw["bn_layers"] or self.made[1]
        if kw["bn_fisher"] is not None:
            kw["bn_fisher"] = (kw["bn_fisher"][0] or self.made[1], *kw["bn_fisher"][1:])
        self.calls.append(([list(a) for a in args], kw))   # the lists are filled again by the next pass


def test_a_batch_of_another_size_has_its_own_geometry(monkeypatch):
    """The step of a smaller or larger batch names that many samples: the library reads what the
    tensors hold. A backward pass that is missing is refused."""
    monkeypatch.setattr(cap_mod, "KfacStep", Recorder)
    torch.manual_seed(4)
    model = cap_mod.ResNet50(classes=10).to(memory_format=torch.channels_last)
    cap = cap_mod.KfacCapture(model)
    for n in (3, 2, 4):
        F.cross_entropy(model(torch.randn(n, 3, 32, 32)), torch.arange(n)).backward()
        cap.step(0.1)
        (act, gout, grads, xhat, bgout), kw = cap.kstep.calls[-1]
        for L, a, g in zip(kw["layers"], act, gout):
            assert L.n == n == a.shape[0] == g.shape[0]
        for B, x, g in zip(kw["bn_layers"], xhat, bgout):
            assert B.n == n == x.shape[0] == g.shape[0]
    model(torch.randn(3, 3, 32, 32))
    with pytest.raises(RuntimeError, match="batches"):
        cap.step(0.1)
    cap.remove()


@pytest.mark.parametrize("fmt", [torch.contiguous_format, torch.channels_last])
def test_matrix_of_a_weight_that_has_its_order(fmt):
    """A 1x1 convolution's fp32 weight lies in memory as its matrix does, in either format: what the
    step writes there is the weight."""
    torch.manual_seed(5)
    for m in (torch.nn.Conv2d(6, 4, 1, bias=False), torch.nn.Conv2d(6, 4, 3, bias=False), torch.nn.Linear(6, 4, bias=False)):
        m = m.to(memory_format=fmt)
        mat = cap_mod.KfacCapture._to_matrix(m)
        mat.mul_(2.0).add_(1.0)
        want = mat.clone()
        cap_mod.KfacCapture._from_matrix(m, mat)
        assert torch.equal(cap_mod.KfacCapture._to_matrix(m), want)


# ---------------------------------------------------------------------------
# the backward passes of the losses, the library's calls replaced by the oracle
# ---------------------------------------------------------------------------

def _np(t):
    return None if t is None else t.detach().double().numpy() if t.is_floating_point() else t.numpy()


def _oracle_policy(z, token, old_logp, advantage, logp, stats, dlogits=None, ref_logp=None, mask=None, seq_begin=None,
                   by_sequence=False, clip_low=0.2, clip_high=0.2, kl_coef=0.0, grad_scale=1.0):
    token = token.reshape(-1)
    begin = None if seq_begin is None else seq_begin.tolist()
    st, l, d = lo.policy_loss(_np(z), _np(token), _np(old_logp), _np(advantage), _np(ref_logp), _np(mask), begin,
                              by_sequence, clip_low, clip_high, kl_coef, grad_scale)
    stats.copy_(torch.from_numpy(st))
    logp.copy_(torch.from_numpy(np.nan_to_num(l)))
    if dlogits is not None:
        dlogits.copy_(torch.from_numpy(np.nan_to_num(d)))


def _oracle_preference(z, token, begin, seq_logp, margin, loss, dlogits=None, ref_logp=None, mask=None, beta=0.1,
                       label_smoothing=0.0, grad_scale=1.0):
    value, x, sums, d = lo.preference_loss(_np(z), _np(token), begin.tolist(), _np(ref_logp), _np(mask), beta,
                                           label_smoothing, grad_scale)
    loss.fill_(value)
    margin.copy_(torch.from_numpy(x))
    seq_logp.copy_(torch.tensor(sums))
    dlogits.copy_(torch.from_numpy(np.nan_to_num(d)))


@pytest.fixture
def passes(monkeypatch):
    monkeypatch.setattr(cap_mod, "KfacStep", Recorder)
    monkeypatch.setattr(cap_mod.K, "kfac_policy_loss", _oracle_policy)
    monkeypatch.setattr(cap_mod.K, "kfac_preference_loss", _oracle_preference)


class Net(torch.nn.Module):
    def __init__(self, per=1):
        super().__init__()
        self.a, self.b, self.per = torch.nn.Linear(5, 6), torch.nn.Linear(6, 4 * per), per

    def forward(self, x):
        return self.b(torch.tanh(self.a(x))).view(x.shape[0] * self.per, 4)

    def kfac_modules(self):
        return [(self.a, None), (self.b, None)]


class ConvNet(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.c, self.n, self.b = torch.nn.Conv2d(3, 4, 3, 1, 1, bias=False), torch.nn.BatchNorm2d(4), torch.nn.Linear(4, 4)

    def forward(self, x):
        return self.b(torch.relu(self.n(self.c(x))).mean((2, 3)))

    def kfac_modules(self):
        return [(self.c, self.n), (self.b, None)]


TOL = dict(rtol=2.0 ** -10, atol=2.0 ** -10)      # fp16 tensors of numbers up to 1, and of some up to 3


def _score_grads(net, x, y, weights, outs):
    """Gradients at `outs` (captured by forward hooks) of sum_t weights[t] log p(y_t)."""
    seen = {}
    hooks = [m.register_forward_hook(lambda mod, i, o, k=k: seen.__setitem__(k, o)) for k, m in enumerate(outs)]
    l = torch.log_softmax(net(x), 1).gather(1, y[:, None])[:, 0]
    got = torch.autograd.grad((l * weights).sum(), [seen[k] for k in range(len(outs))])
    for h in hooks:
        h.remove()
    return got


ROWS = 7
TOKEN = torch.tensor([1, 0, 3, 2, -100, 1, 0])
DRAWN = torch.tensor([3, 1, 0, 2, 2, 0, 1])
MASK = torch.tensor([1, 1, 0, 1, 1, 0, 1], dtype=torch.bool)
BEGIN = torch.tensor([0, 3, 6], dtype=torch.int32)
COUNTED = torch.tensor([1, 1, 0, 1, 0, 0, 0], dtype=torch.bool)     # 4 has no token, 6 no sequence


def _policy_kw():
    g = torch.Generator().manual_seed(6)
    return dict(old_logp=-1.4 + 0.1 * torch.randn(ROWS, generator=g), advantage=torch.randn(ROWS, generator=g),
                ref_logp=torch.full((ROWS,), -1.3), mask=MASK, seq_begin=BEGIN, by_sequence=True, kl_coef=0.2)


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_factors_take_scores_of_the_rows_that_count(passes, monkeypatch, loss):
    """gout of the step: d log p(y) at each layer, coefficient 1, of the rows that count alone, whatever the
    loss weighs them by; the weights' gradients are the loss's and nothing else."""
    torch.manual_seed(7)
    net = Net()
    cap = cap_mod.KfacCapture(net)
    monkeypatch.setattr(cap, "_draw", lambda z: DRAWN)
    x = torch.randn(ROWS, 5)
    net.a.weight.grad = before = torch.ones(6, 5)                     # an earlier pass's
    logits = net(x)
    if loss == "policy":
        cap.policy_backward(logits, TOKEN, **_policy_kw())
        kw = {k: _np(v) if torch.is_tensor(v) else v for k, v in _policy_kw().items()}
        want = lo.policy_loss(_np(logits), _np(TOKEN), kw["old_logp"], kw["advantage"], kw["ref_logp"], kw["mask"],
                              BEGIN.tolist(), True, kl_coef=0.2)[2]
    else:
        cap.preference_backward(logits, TOKEN, BEGIN, mask=MASK, beta=0.5)
        want = lo.preference_loss(_np(logits), _np(TOKEN), BEGIN.tolist(), None, _np(MASK), 0.5)[3]
    logits = net(x)                                                    # (also: a later forward alone changes no .grad)
    ref = torch.autograd.grad(logits, list(net.parameters()), torch.from_numpy(np.nan_to_num(want)).float())
    assert net.a.weight.grad is before
    for p, w in zip(net.parameters(), ref):
        assert torch.allclose(p.grad, w + (1.0 if p is net.a.weight else 0.0), rtol=1e-5, atol=1e-6)
    score = _score_grads(net, x, DRAWN, COUNTED.float(), [net.a, net.b])
    net.zero_grad()                                                    # the gradients above took the scores away
    if loss == "policy":
        cap.policy_backward(net(x), TOKEN, **_policy_kw())
    else:
        cap.preference_backward(net(x), TOKEN, BEGIN, mask=MASK, beta=0.5)
    cap.step(0.1)
    (act, gout, grads, _, _), kw = cap.kstep.calls[-1]
    assert torch.equal(act[0], x[COUNTED].half()) and kw["refresh"]
    assert all(L.n == 3 == a.shape[0] == g.shape[0] for L, a, g in zip(kw["layers"], act, gout))
    assert all(L.n == ROWS for L in cap.kstep.made[0])
    for g, s in zip(gout, score):
        assert torch.allclose(g.float(), s[COUNTED], **TOL) and s[COUNTED].abs().max() > 0.1
    one_hot = gout[1].float() + torch.softmax(logits.detach()[COUNTED], 1)
    assert torch.allclose(one_hot, F.one_hot(DRAWN[COUNTED], 4).float(), **TOL)
    cap.remove()


def test_padding_changes_nothing(passes, monkeypatch):
    """Rows that do not count, in front, between and behind, change neither the factors' tensors nor the
    weights' gradients; NaN among their logits does not either."""
    torch.manual_seed(8)
    net = Net()
    x, token, drawn = torch.randn(4, 5), torch.tensor([0, 3, 1, 2]), torch.tensor([1, 1, 0, 2])
    old, adv = torch.full((4,), -1.4), torch.tensor([0.5, -0.3, 1.0, 0.2])
    at = torch.tensor([1, 2, 4, 5])
    got = []
    for padded in (False, True):
        cap = cap_mod.KfacCapture(net)
        net.zero_grad()
        ins = [x, token, old, adv, drawn]
        mask = None
        if padded:
            wide = [torch.full((7, *t.shape[1:]), 9, dtype=t.dtype) for t in ins]
            for w, t in zip(wide, ins):
                w[at] = t
            ins, mask = wide, torch.zeros(7, dtype=torch.bool)
            mask[at] = True
        monkeypatch.setattr(cap, "_draw", lambda z, y=ins[4]: y.clamp(max=3))
        cap.policy_backward(net(ins[0]), ins[1], ins[2], ins[3], mask=mask)
        cap.step(0.0)
        (act, gout, grads, _, _), kw = cap.kstep.calls[-1]
        got.append((*act, *gout, *[torch.tensor(L.n) for L in kw["layers"]]))
        grads_of = [g.clone() for g in grads]
        got.append(grads_of)
        cap.remove()
    assert all(torch.equal(a, b) for a, b in zip(got[0], got[2]))
    assert all(torch.allclose(a, b, rtol=1e-5, atol=1e-7) for a, b in zip(got[1], got[3]))


def test_several_rows_of_a_sample(passes, monkeypatch):
    """Three rows a sample: its score is the sum of its rows', times sqrt(samples / rows) of those that count,
    so that the mean of its square over the samples estimates the mean over the rows."""
    torch.manual_seed(9)
    net = Net(per=3)
    cap = cap_mod.KfacCapture(net)
    drawn = torch.randint(0, 4, (12,))
    monkeypatch.setattr(cap, "_draw", lambda z: drawn)
    x = torch.randn(4, 5)
    mask = torch.ones(12, dtype=torch.bool)
    mask[[0, 3, 4, 5, 10]] = False                                     # the second sample has none left
    cap.policy_backward(net(x), torch.zeros(4, 3, dtype=torch.long), torch.full((12,), -1.4), torch.ones(12), mask=mask)
    cap.step(0.1)
    (act, gout, *_), kw = cap.kstep.calls[-1]
    kept = torch.tensor([0, 2, 3])
    assert torch.equal(act[0], x[kept].half()) and all(L.n == 3 for L in kw["layers"])
    score = _score_grads(net, x, drawn, mask.float(), [net.a, net.b])
    for g, s in zip(gout, score):
        assert torch.allclose(g.float(), s[kept] * (3 / 7) ** 0.5, **TOL)
    cap.remove()


@pytest.mark.parametrize("masked", [False, True])
def test_convolutions_and_batchnorm_take_scores(passes, monkeypatch, masked):
    """A convolution's score times sqrt(positions), BatchNorm's Fisher from the scores, its gradient from the
    loss, over all samples."""
    torch.manual_seed(10)
    net = ConvNet()
    cap = cap_mod.KfacCapture(net)
    drawn = torch.tensor([1, 0, 3, 2, 2])
    monkeypatch.setattr(cap, "_draw", lambda z: drawn)
    x = torch.randn(5, 3, 6, 6)
    mask = torch.tensor([True, True, not masked, True, True])
    old, adv = torch.full((5,), -1.4), torch.tensor([0.5, -0.3, 1.0, 0.2, 0.1])
    score = _score_grads(net, x, drawn, mask.float(), [net.c, net.n, net.b])
    cap.policy_backward(net(x), torch.zeros(5, dtype=torch.long), old, adv, mask=mask)
    bgout = cap.bgout[0].clone()
    cap.step(0.1)
    (act, gout, grads, xhat, bn_gout), kw = cap.kstep.calls[-1]
    n = 5 - masked
    assert [L.n for L in kw["layers"]] == [n, n] and [B.n for B in kw["bn_layers"]] == [5]
    assert torch.allclose(gout[0].float(), 6 * score[0].permute(0, 2, 3, 1)[mask], **TOL)
    assert torch.allclose(gout[1].float(), score[2][mask], **TOL)
    assert torch.equal(bn_gout[0], bgout) and xhat[0].shape == (5, 36, 4)
    bns, fx, fg = kw["bn_fisher"]
    assert [B.n for B in bns] == [n] and torch.equal(fx[0], cap.xhat[0][mask])
    assert torch.allclose(fg[0].float(), score[1].permute(0, 2, 3, 1).reshape(5, 36, 4)[mask], **TOL)
    # the gradient of gamma and beta: the mean over the samples of the captured products
    s = torch.stack([(bgout.float() * cap.xhat[0].float()).sum(1).mean(0), bgout.float().sum(1).mean(0)])
    assert torch.allclose(s, torch.stack([net.n.weight.grad, net.n.bias.grad]), rtol=1e-2, atol=1e-3)
    cap.remove()


def test_passes_of_a_stale_step_and_of_another_loss(passes, monkeypatch):
    """No second pass where the next step keeps its curvature; an ordinary loss behind takes its own
    gradients; a batch without a row that counts keeps the curvature there is."""
    torch.manual_seed(11)
    net = Net()
    cap = cap_mod.KfacCapture(net, refresh_every=2)
    drawn = []
    monkeypatch.setattr(cap, "_draw", lambda z: drawn.append(1) or torch.zeros(z.shape[0], dtype=torch.long))
    x, one = torch.randn(3, 5), torch.ones(3)
    call = lambda **kw: cap.policy_backward(net(x), torch.zeros(3, dtype=torch.long), -one, one, **kw)  # noqa: E731
    for refresh in (True, False, True):
        call()
        cap.step(0.1)
        assert cap.kstep.calls[-1][1]["refresh"] == refresh
    assert len(drawn) == 2
    cap.calls = 4
    F.cross_entropy(net(x), torch.zeros(3, dtype=torch.long)).backward()
    cap.step(0.1)
    assert all(a is b for a, b in zip(cap.kstep.calls[-1][0][1], cap.gout)) and len(drawn) == 2
    assert cap.kstep.calls[-1][1]["bn_fisher"] is None
    cap.calls = 6
    call(mask=torch.zeros(3, dtype=torch.bool))
    cap.step(0.1)
    assert not cap.kstep.calls[-1][1]["refresh"]
    cap.calls = 0
    call(mask=torch.zeros(3, dtype=torch.bool))
    cap.step(0.1)
    (act, gout, *_), kw = cap.kstep.calls[-1]
    assert kw["refresh"] and len(act[0]) == 3 and not any(g.any() for g in gout)
    cap.remove()


def test_drawn_tokens_follow_the_model():
    """40000 draws of three choices: each share within five standard deviations, 5 sqrt(p (1 - p) / n) <= 0.0125;
    a choice of no probability is never drawn."""
    torch.manual_seed(12)
    p = torch.tensor([0.5, 0.2, 0.0, 0.3])
    y = cap_mod.KfacCapture._draw(p.log().expand(40000, 4))
    share = torch.bincount(y, minlength=4) / 40000
    assert (share - p).abs().max() <= 0.0125 and share[2] == 0
    assert cap_mod.KfacCapture._draw(torch.zeros(0, 4)).shape == (0,)
    bad = cap_mod.KfacCapture._draw(torch.full((2, 4), float("nan")))
    assert ((bad >= 0) & (bad < 4)).all()


class HalfHead(torch.nn.Module):
    def __init__(self, d, choices):
        super().__init__()
        self.fc = torch.nn.Linear(d, choices)

    def forward(self, x):
        return self.fc(x).half()

    def kfac_modules(self):
        return [(self.fc, None)]


@pytest.mark.parametrize("loss", ["policy", "preference"])
@pytest.mark.parametrize("given", [None, 256.0])
def test_fp16_logits_keep_the_softmax_of_a_mean(passes, loss, given):
    """Of 1024 rows of 4096 fp16 logits every softmax entry of the loss's mean is below half the smallest
    fp16: the weights' gradients hold it all the same, added to what the leaves held; so does what the
    hooks were handed. An element of the logits' gradient is off by half a step of fp16, 2^-11 of it, or
    by 2^-25 / scale where it is a subnormal; a sum of 1024 in fp32 by 1024 * 2^-24 of its terms at most."""
    torch.manual_seed(13)
    rows, choices, d = 1024, 4096, 3
    net = HalfHead(d, choices)
    cap = cap_mod.KfacCapture(net)
    x, token = torch.randn(rows, d), torch.randint(0, choices, (rows,))
    logits = net(x)
    if loss == "policy":
        old, adv = torch.full((rows,), -8.3), torch.randn(rows)
        cap.policy_backward(logits, token, old, adv, grad_scale=given)
        want, scale = lo.policy_loss(_np(logits), _np(token), _np(old), _np(adv))[2], given or 1024.0
    else:
        begin = torch.arange(0, rows + 1, 8, dtype=torch.int32)       # 64 pairs
        net.fc.bias.grad = held = torch.full((choices,), 0.5)
        cap.preference_backward(logits, token, begin, beta=0.1, grad_scale=given)
        want, scale = lo.preference_loss(_np(logits), _np(token), begin.tolist(), None, None, 0.1)[3], given or 512.0
        assert net.fc.bias.grad is held
        held -= 0.5
    off = np.abs(want) * (2.0 ** -11 + rows * 2.0 ** -24) + 2.0 ** -25 / scale
    base = 2.0 ** -24 * (0.5 if loss == "preference" else 0.0)         # beside what was there
    got = net.fc.bias.grad.double().numpy()
    assert (np.abs(got - want.sum(0)) <= off.sum(0) * 1.01 + base).all()
    got = net.fc.weight.grad.double().numpy()
    xs = np.abs(_np(x))
    assert (np.abs(got - want.T @ _np(x)) <= (off.T @ xs) * 1.01 + rows * 2.0 ** -24 * (np.abs(want).T @ xs)).all()
    # n times the gradient, rounded to fp16 once more from fp16
    seen = cap.gout[0].double().numpy()
    assert (np.abs(seen - rows * want) <= rows * off * 1.01 + np.abs(rows * want) * 2.0 ** -11 * 1.01 + 2.0 ** -25).all()
    assert np.abs(want[np.arange(rows), token.numpy()]).max() > 1e-4 > np.abs(np.sort(want, 1)[:, 1:-1]).max()
    cap.remove()


def test_scales_of_other_types_and_refusals(passes):
    torch.manual_seed(14)
    net = Net()
    cap = cap_mod.KfacCapture(net)
    scale = cap_mod.KfacCapture._scale
    for z in (torch.zeros(1), torch.zeros(1, dtype=torch.bfloat16)):
        assert scale(None, z, 4096) == 1.0 and scale(8, z, 4096) == 8.0
    z = torch.zeros(1, dtype=torch.float16)
    assert [scale(None, z, x) for x in (0, 0.3, 1, 7, 4096, 1 << 20)] == [1, 1, 1, 4, 4096, 1 << 14]
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="grad_scale"):
            cap.policy_backward(net(torch.randn(3, 5)), torch.zeros(3, dtype=torch.long), torch.zeros(3), torch.ones(3),
                                grad_scale=bad)
    got = []
    for s in (None, 64.0):                                             # a power of two: the same bits in fp32
        net.zero_grad()
        torch.manual_seed(15)
        cap.policy_backward(net(torch.randn(3, 5)), torch.zeros(3, dtype=torch.long), -torch.ones(3), torch.ones(3),
                            grad_scale=s)
        got.append([p.grad.clone() for p in net.parameters()] + [g.clone() for g in cap.gout])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    cap.remove()


def test_a_layer_that_the_logits_do_not_reach(passes, monkeypatch):
    """A second head with a loss of its own, in a graph of its own: its factors take that loss's gradients
    over all samples, beside those of the logits' scores."""
    class Two(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.policy, self.value = torch.nn.Linear(5, 4), torch.nn.Linear(5, 1)

        def kfac_modules(self):
            return [(self.policy, None), (self.value, None)]

    torch.manual_seed(16)
    net = Two()
    cap = cap_mod.KfacCapture(net)
    drawn = torch.tensor([0, 1, 2, 3])
    monkeypatch.setattr(cap, "_draw", lambda z: drawn)
    x, mask = torch.randn(4, 5), torch.tensor([True, False, True, True])
    logits, value = net.policy(x), net.value(x)
    cap.policy_backward(logits, torch.zeros(4, dtype=torch.long), -torch.ones(4), torch.ones(4), mask=mask)
    value.square().mean().backward()
    cap.step(0.1)
    (act, gout, *_), kw = cap.kstep.calls[-1]
    assert [L.n for L in kw["layers"]] == [3, 4] and kw["refresh"]
    assert torch.equal(act[0], x[mask].half()) and torch.equal(act[1], x.half())
    assert torch.allclose(gout[0].float(), (F.one_hot(drawn, 4) - torch.softmax(logits.detach(), 1))[mask], **TOL)
    assert torch.allclose(gout[1].float(), 2 * value.detach(), **TOL)
    cap.remove()


def test_a_forward_before_the_step_leaves_the_scores(passes, monkeypatch):
    """A forward pass with gradients on between the loss's backward pass and the step, as of an evaluation,
    does not put the loss's gradients in the scores' place; another loss's backward pass does."""
    torch.manual_seed(17)
    net = Net()
    cap = cap_mod.KfacCapture(net)
    x, one = torch.randn(3, 5), torch.ones(3)
    cap.policy_backward(net(x), torch.zeros(3, dtype=torch.long), -one, 0.001 * one)
    score = [s.clone() for s in cap.score]
    net(x)
    cap.step(0.1)
    assert all(torch.equal(a, b) for a, b in zip(cap.kstep.calls[-1][0][1], score))
    F.cross_entropy(net(x), torch.zeros(3, dtype=torch.long)).backward()
    assert cap.score == [None, None]
    cap.remove()
