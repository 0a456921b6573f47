"""The losses, the clipping and the bounded update as a K-FAC step uses them: KfacStep with
max_grad_norm and trust_radius, and a policy trained through KfacCapture from the loss over
its logits to the bounded update of its weights."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import synth
from gpu_helpers import host, relF, say
from loss_cases import U, host64
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

LAYERS = [synth.Layer("c3x3", 2, 6, 6, 8, 6, 6, 16, 3, 3, 1, 1, 1, 1, 1),
          synth.Layer("c1x1s2", 2, 6, 6, 16, 3, 3, 24, 1, 1, 2, 2, 0, 0, 1),
          synth.Layer("c1x1", 2, 4, 4, 1040, 4, 4, 12, 1, 1, 1, 1, 0, 0, 1),
          synth.Layer("fc", 4, 1, 1, 40, 1, 1, 10, 1, 1, 1, 1, 0, 0, 1)]
BNS = [synth.BNLayer("bn1", 2, 36, 16), synth.BNLayer("bn2", 2, 9, 24)]


def _inputs(grad_dtype=torch.float32):
    rng = synth.layer_rng(77, 0)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dict(act=[to(synth.relu_normal_f16(rng, l.act_shape)) for l in LAYERS],
                gout=[to(synth.normal_f16(rng, l.gout_shape, 0.1)) for l in LAYERS],
                grads=[to(synth.normal_f32(rng, (l.d_g, l.d_a), 0.1)).to(grad_dtype) for l in LAYERS],
                xhat=[to(synth.normal_f16(rng, b.shape)) for b in BNS],
                bn_gout=[to(synth.normal_f16(rng, b.shape)) for b in BNS])


def _params():
    rng = synth.layer_rng(78, 0)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return ([to(synth.normal_f32(rng, (l.d_g, l.d_a), 0.05)) for l in LAYERS],
            [to(synth.normal_f32(rng, (2, b.c))) for b in BNS])


def _relative(a, b):
    return float(torch.linalg.vector_norm(a.double() - b.double()) / torch.linalg.vector_norm(b.double()))


@pytest.mark.parametrize("side_stream", [True, False])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
def test_step_clips_what_it_preconditions(kfac_gpu, side_stream, grad_dtype):
    ins = _inputs(grad_dtype)
    keep = [g.clone() for g in ins["grads"]]
    st = kfac_gpu.KfacStep(LAYERS, BNS, "cuda", max_grad_norm=0.75, side_stream=side_stream)
    assert bool(st.side) == side_stream
    st.step(**ins)
    norm = lo.global_norm([host64(g) for g in keep])
    assert norm > 0.75 and abs(float(st.grad_norm) - norm) <= 1.01 * U * norm
    assert all(torch.equal(a, b) for a, b in zip(keep, ins["grads"]))       # the caller's are not touched
    for c, g in zip(st.clipped, keep):
        ref = host64(g) * (0.75 / norm)
        assert (np.abs(host64(c) - ref) <= 2.02 * U * np.abs(ref)).all()
    plain = kfac_gpu.KfacStep(LAYERS, BNS, "cuda", side_stream=side_stream)
    plain.step(**{**ins, "grads": st.clipped})
    assert all(torch.equal(a, b) for a, b in zip(st.out, plain.out))


@pytest.mark.parametrize("side_stream", [True, False])
@pytest.mark.parametrize("radius", [1e9, 1e-3])
@pytest.mark.parametrize("refresh", [True, False])
def test_step_is_bounded(kfac_gpu, side_stream, radius, refresh):
    """The update is s P for all parameters, s the rate or what the radius allows."""
    ins = _inputs()
    lr = 0.2
    st = kfac_gpu.KfacStep(LAYERS, BNS, "cuda", trust_radius=radius, side_stream=side_stream)
    if not refresh:
        st.step(**ins)
        ins["grads"] = [g * 2 for g in ins["grads"]]
    w, p = _params()
    w0, p0 = _params()
    st.step(**ins, weights=w, bn_params=p, lr=lr, refresh=refresh)
    torch.cuda.synchronize()
    P = [host64(t) for t in st.out + st.bn_pre]
    g = [host64(t) for t in ins["grads"]] + [None] * len(BNS)
    fisher = [None] * len(LAYERS) + [host64(t) for t in st.fisher]
    s, q = lo.trust_step(P, g, float(np.float32(lr)), float(np.float32(radius)), fisher, float(np.float32(st.bn_shift)))
    assert q > 0 and (s == float(np.float32(lr))) == (radius == 1e9)
    assert abs(float(st.trust[0]) - s) <= s * 1.1 * U and abs(float(st.trust[1]) - q) <= q * 1.1 * U
    for new, old, d in zip(w + p, w0 + p0, P):
        ref = host64(old) - s * d
        assert (np.abs(host64(new) - ref) <= 1.1 * U * (np.abs(ref) + s * np.abs(d))).all()
    say("bounded step: s", s, "predicted KL", 0.5 * s * s * q, "radius", radius)
    # the options leave the preconditioned gradients as they are
    plain = kfac_gpu.KfacStep(LAYERS, BNS, "cuda", side_stream=side_stream)
    if not refresh:
        plain.step(**{**ins, "grads": [t / 2 for t in ins["grads"]]})
    plain.step(**ins, refresh=refresh)
    assert all(torch.equal(a, b) for a, b in zip(st.out + st.bn_pre, plain.out + plain.bn_pre))


def test_step_on_another_stream(kfac_gpu):
    ins = _inputs()
    got = []
    for stream in (None, torch.cuda.Stream()):
        st = kfac_gpu.KfacStep(LAYERS, BNS, "cuda", max_grad_norm=0.5, trust_radius=1e-3)
        w, p = _params()
        torch.cuda.synchronize()
        st.step(**ins, weights=w, bn_params=p, lr=0.2, stream=stream)
        torch.cuda.synchronize()
        got.append(w + p + [st.trust, st.grad_norm])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("side_stream", [True, False])
@pytest.mark.parametrize("samples", [1, 2, 5])
def test_step_of_fewer_and_of_more_samples(kfac_gpu, side_stream, samples):
    """A step made for one batch size takes another: the bits of a step made for that one."""
    layers = [dataclasses.replace(l, n=samples) for l in LAYERS]
    bns = [dataclasses.replace(b, n=samples) for b in BNS]
    rng = synth.layer_rng(79, 0)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    ins = dict(act=[to(synth.relu_normal_f16(rng, l.act_shape)) for l in layers],
               gout=[to(synth.normal_f16(rng, l.gout_shape, 0.1)) for l in layers],
               grads=[to(synth.normal_f32(rng, (l.d_g, l.d_a), 0.1)) for l in layers],
               xhat=[to(synth.normal_f16(rng, b.shape)) for b in bns],
               bn_gout=[to(synth.normal_f16(rng, b.shape)) for b in bns])
    got = []
    for made, kw in ((layers, {}), (LAYERS, dict(layers=layers, bn_layers=bns))):
        st = kfac_gpu.KfacStep(made, bns if not kw else BNS, "cuda", side_stream=side_stream, trust_radius=1e-3)
        w, p = _params()
        st.step(**ins, weights=w, bn_params=p, lr=0.2, **kw)
        torch.cuda.synchronize()
        got.append(st.A_packed + st.G_packed + st.fisher + st.out + st.bn_pre + w + p + [st.trust])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_step_whose_workspace_is_too_small(kfac_gpu):
    """Many more samples than the step was made for: a larger workspace, on the call's stream."""
    one = [synth.Layer("c3x3", 1, 8, 8, 64, 8, 8, 64, 3, 3, 1, 1, 1, 1, 1)]
    many = [dataclasses.replace(one[0], n=200)]
    rng = synth.layer_rng(80, 0)
    act = torch.from_numpy(synth.relu_normal_f16(rng, many[0].act_shape)).cuda()
    gout = torch.from_numpy(synth.normal_f16(rng, many[0].gout_shape, 0.1)).cuda()
    grad = torch.randn(64, many[0].d_a, device="cuda")
    want = kfac_gpu.KfacStep(many, (), "cuda")
    st = kfac_gpu.KfacStep(one, (), "cuda")
    assert kfac_gpu.kfac_factors_workspace(many) + 256 > st.workspace.numel()
    want.step([act], [gout], [grad])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side):
        st.step([act], [gout], [grad], layers=many, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(st.out[0], want.out[0]) and torch.equal(st.A_packed[0], want.A_packed[0])


def _plain_policy(z, token, old, adv, ref, beta):
    l = torch.log_softmax(z, 1).gather(1, token[:, None])[:, 0]
    r, d = (l - old).exp(), ref - l
    return (-torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv) + beta * (d.exp() - d - 1)).mean()


def test_policy_training_step(kfac_gpu):
    """A ResNet-50 as a policy over its classes: log-probabilities of the choices, the loss's
    backward pass through the network, clipping, preconditioning, the bounded update."""
    from fac_second_order_amd.capture import KfacCapture, ResNet50
    torch.manual_seed(31)
    classes, n = 10, 8
    model = ResNet50(classes).cuda().to(memory_format=torch.channels_last)
    cap = KfacCapture(model, damping=1e-1, max_grad_norm=0.5, trust_radius=1e-3)
    x = torch.randn(n, 3, 32, 32, device="cuda").to(memory_format=torch.channels_last)
    token = torch.randint(0, classes, (n,), device="cuda")
    adv = torch.randn(n, device="cuda")
    with torch.no_grad():
        start = torch.log_softmax(model(x), 1).gather(1, token[:, None])[:, 0]
    old, ref = start - 0.1 * torch.rand(n, device="cuda"), start + 0.1
    for t in range(2):
        model.zero_grad(set_to_none=True)
        logits = model(x)
        stats, logp = cap.policy_backward(logits, token, old, adv, ref_logp=ref, kl_coef=0.3)
        z = logits.detach().double().requires_grad_()
        loss = _plain_policy(z, token, old.double(), adv.double(), ref.double(), float(np.float32(0.3)))
        loss.backward()
        # fp32 logits of a 10-way choice: err_l below 64 u, ratios and KL slopes below 4
        assert abs(float(stats[0]) - float(loss.detach())) <= 4 * 64 * U + U * abs(float(loss.detach()))
        got = cap.gout[-1].double() / n                 # what the hook of the classifier was handed, in f16
        assert (got - z.grad).abs().max() <= z.grad.abs().max() * 2.0 ** -11 * 1.01 + 4 * 64 * U + 2.0 ** -25 / n
        assert _relative(model.fc.bias.grad, z.grad.sum(0)) <= 1e-5
        grads = [cap._to_matrix(m, grad=True) for m, _ in cap.pairs]
        w0 = cap._to_matrix(model.fc)
        cap.step(lr=0.05)
        torch.cuda.synchronize()
        st = cap.kstep
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        s, q = (float(v) for v in st.trust.double())
        say("policy step", t, "loss", float(stats[0]), "norm", norm, "s", s, "predicted KL", 0.5 * s * s * q)
        assert abs(float(st.grad_norm) - norm) <= 2 * U * norm
        assert _relative(st.clipped[-1], grads[-1] * min(1.0, 0.5 / norm)) <= 4 * U
        assert s > 0 and 0.5 * s * s * abs(q) <= 1e-3 * (1 + 4 * U)
        assert relF(host(cap._to_matrix(model.fc)), host64(w0) - s * host64(st.out[-1])) <= 2 * U
        assert int(st.info.abs().sum()) == 0
    cap.remove()


def test_preference_training_step(kfac_gpu):
    from fac_second_order_amd.capture import KfacCapture, ResNet50
    torch.manual_seed(32)
    classes, pairs, per = 10, 2, 2
    n = 2 * pairs * per
    model = ResNet50(classes).cuda().to(memory_format=torch.channels_last)
    cap = KfacCapture(model, damping=1e-1, trust_radius=1e-3)
    x = torch.randn(n, 3, 32, 32, device="cuda").to(memory_format=torch.channels_last)
    token = torch.randint(0, classes, (n,), device="cuda")
    begin = torch.arange(0, n + 1, per, dtype=torch.int32, device="cuda")
    ref = torch.randn(2 * pairs, device="cuda")
    logits = model(x)
    loss, margin, seq = cap.preference_backward(logits, token, begin, ref_logp=ref, beta=0.5)
    z = logits.detach().double().requires_grad_()
    l = torch.log_softmax(z, 1).gather(1, token[:, None])[:, 0].view(2 * pairs, per).sum(1)
    gain = l - ref.double()
    m = 0.5 * (gain[:pairs] - gain[pairs:])
    want = torch.nn.functional.softplus(-m).mean()
    want.backward()
    # four rows a pair: the margin is off by at most 0.5 * 4 * 64 u from the rows
    assert (margin.double() - m).abs().max() <= 128 * U + 2 * U * float(m.detach().abs().max())
    assert abs(float(loss) - float(want.detach())) <= 128 * U + U * float(want.detach())
    got = cap.gout[-1].double() / n
    assert (got - z.grad).abs().max() <= z.grad.abs().max() * 2.0 ** -11 * 1.01 + 128 * U + 2.0 ** -25 / n
    cap.step(lr=0.05)
    torch.cuda.synchronize()
    s, q = (float(v) for v in cap.kstep.trust.double())
    assert s > 0 and 0.5 * s * s * abs(q) <= 1e-3 * (1 + 4 * U)
    cap.remove()


class Head(torch.nn.Module):
    """One softmax layer, its logits in a type."""

    def __init__(self, d, choices, dtype=torch.float32, std=0.02):
        super().__init__()
        self.fc, self.dtype = torch.nn.Linear(d, choices), dtype
        with torch.no_grad():
            self.fc.weight.normal_(0, std)
            self.fc.bias.normal_(0, std)

    def forward(self, x):
        return self.fc(x).to(self.dtype)

    def kfac_modules(self):
        return [(self.fc, None)]


@pytest.mark.parametrize("loss", ["policy", "preference"])
@pytest.mark.parametrize("size", [0.1, 1.0, 10.0])
@pytest.mark.parametrize("masked", [False, True])
def test_radius_is_the_kl_of_the_model(kfac_gpu, loss, size, masked):
    """The KL divergence of the model across a step, measured in fp64 over the rows that count, is the radius
    it was given, whatever the loss weighs the rows by; rows that do not count, of other inputs, take no part.

    One softmax layer near the uniform distribution: its Fisher is A x (diag p - p p^T) but for p's own
    spread (logits of 0.08: some percent). G is estimated from 4096 (2048) drawn tokens: for a fixed direction u
    the square of u . score, whitened, has a mean of 1 and at most 7 as its largest value with 8 choices, so the
    estimate's deviation is at most sqrt(6 / 2048) = 0.054, and 0.2 is 3.7 of them. To second order: the step
    moves logits by sqrt(2e-3) = 0.045, and the third order is at most that part of the second. 0.2 + 0.05."""
    from fac_second_order_amd.capture import KfacCapture
    torch.manual_seed(41)
    rows, d, choices, radius = 4096, 16, 8, 1e-3
    net = Head(d, choices).cuda()
    cap = KfacCapture(net, damping=1e-6, trust_radius=radius)
    x = torch.randn(rows, d, device="cuda")
    token = torch.randint(0, choices, (rows,), device="cuda")
    mask = None
    if masked:
        mask = torch.arange(rows, device="cuda") % 2 == 0
        x[~mask] *= 20.0
    with torch.no_grad():
        before = torch.log_softmax(net(x).double(), 1)
    old = before.gather(1, token[:, None])[:, 0].float()
    if loss == "policy":
        cap.policy_backward(net(x), token, old, size * torch.randn(rows, device="cuda"), mask=mask)
    else:
        begin = torch.arange(0, rows + 1, 64, dtype=torch.int32, device="cuda")
        cap.preference_backward(net(x), token, begin, mask=mask, beta=0.01 * size)
    cap.step(lr=1e20)
    with torch.no_grad():
        after = torch.log_softmax(net(x).double(), 1)
    kl = (before.exp() * (before - after)).sum(1)
    kl = float(kl.mean() if mask is None else kl[mask].mean())
    s, q = (float(v) for v in cap.kstep.trust.double())
    say(loss, "size", size, "masked", masked, "KL", kl, "predicted", 0.5 * s * s * q)
    assert abs(0.5 * s * s * q - radius) <= radius * 8 * U
    assert abs(kl - radius) <= 0.25 * radius
    cap.remove()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_scores_of_the_factors(kfac_gpu, dtype):
    """What the factors of a step are formed from, by the library: a one-hot row less the softmax, in the
    logits' type (half a step of it, one of fp16, and 8 u of fp32) for rows that count, zeros elsewhere; G is
    their second moment over the rows that count, A that of their inputs."""
    from fac_second_order_amd.capture import KfacCapture
    torch.manual_seed(42)
    rows, d, choices = 300, 24, 11
    net = Head(d, choices, dtype, std=0.5).cuda()
    cap = KfacCapture(net, damping=1e-2)
    x = torch.randn(rows, d, device="cuda")
    mask = torch.arange(rows, device="cuda") % 3 != 1
    token = torch.randint(0, choices, (rows,), device="cuda")
    token[5], mask[6] = -100, True
    counted = mask & (token >= 0)
    logits = net(x)
    cap.policy_backward(logits, token, torch.full((rows,), -2.4, device="cuda"), torch.randn(rows, device="cuda"),
                        mask=mask)
    score = host64(cap.score[0])
    p = np.exp(host64(torch.log_softmax(logits.detach().double(), 1)))
    on = host64(counted.float()) != 0
    assert not score[~on].any()
    m = int(on.sum())
    # the library's row is rows / counted times the score, rounded to the type, times counted / rows, to fp16
    drawn = np.abs(score + p - 1.0).argmin(1)
    one = np.zeros_like(p)
    one[np.arange(rows), drawn] = 1.0
    half = torch.finfo(dtype).eps / 2 + 2.0 ** -11 + 8 * U
    floor = 2.0 ** -25 * (1 + m / rows)                                 # subnormals of fp16
    assert (np.abs(score - (one - p))[on] <= (np.abs(one - p) * half * 1.01 + 64 * U * p + 4 * U + floor)[on]).all()
    cap.step(0.0)
    torch.cuda.synchronize()
    G = (score[on].T @ score[on]) / m
    a = np.concatenate([host64(cap.act[0]), np.ones((rows, 1))], 1)[on]
    A = a.T @ a / m
    iu = np.triu_indices(choices)
    assert np.linalg.norm(host64(cap.kstep.G_packed[0]) - G[iu]) <= 1e-5 * np.linalg.norm(G)
    iu = np.triu_indices(d + 1)
    assert np.linalg.norm(host64(cap.kstep.A_packed[0]) - A[iu]) <= 1e-5 * np.linalg.norm(A)
    cap.remove()


@pytest.mark.parametrize("loss", ["policy", "preference"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_weight_gradients_of_a_mean_over_many_rows(kfac_gpu, loss, dtype):
    """2048 rows of 20000 choices: a softmax entry of the loss's mean is below the smallest fp16, 2^-24 = 6.0e-8
    (policy: |advantage| / 2048 / 20000, at most 3.7e-8 on average; preference: beta / (2 pairs) / 20000 = 4.9e-8).
    The weights' gradients against fp64, off by the rounding of the logits' gradient: half a step of
    its type and 8 u, or half the smallest subnormal of fp16 over the scale (2048, 512); the row's error of l
    twice (its softmax and its coefficient, which is below 2 and whose slope is); 2048 u for the sums."""
    from fac_second_order_amd.capture import KfacCapture
    torch.manual_seed(43)
    rows, choices, d = 2048, 20000, 4
    net = Head(d, choices, dtype, std=0.3).cuda()
    cap = KfacCapture(net)
    x = torch.randn(rows, d, device="cuda")
    token = torch.randint(0, choices, (rows,), device="cuda")
    logits = net(x)
    z = logits.detach().double()
    lp = torch.log_softmax(z, 1)
    l, one = lp.gather(1, token[:, None])[:, 0], torch.nn.functional.one_hot(token, choices)
    if loss == "policy":
        adv = torch.randn(rows, device="cuda").clamp(-1.5, 1.5)
        cap.policy_backward(logits, token, l.float(), adv)
        coef, scale = -adv.double() / rows, 2048.0
    else:
        begin = torch.arange(0, rows + 1, 16, dtype=torch.int32, device="cuda")   # 64 pairs
        ref = l.view(-1, 16).sum(1).float()                                       # margins of about 0
        cap.preference_backward(logits, token, begin, ref_logp=ref, beta=0.125)
        x_i = 0.125 * ((l.view(-1, 16).sum(1) - ref.double()).view(2, 64))
        c = -0.125 / 64 / (1 + (x_i[0] - x_i[1]).exp())
        coef, scale = torch.cat([c, -c]).repeat_interleave(16), 512.0
    want = coef[:, None] * (one - lp.exp())
    err = U * (choices / 64 + 40 + 6 * float((z.amax(1) - z.amin(1)).max()))
    tiny = {torch.float16: 2.0 ** -25 / scale, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}[dtype]
    # a margin adds up 32 rows' errors, a quarter of which its slope sees
    bound = want.abs() * (torch.finfo(dtype).eps / 2 + 4 * err + rows * U) + coef.abs()[:, None] * lp.exp() * 4 * err + tiny
    bound = bound + want.abs() * (8 * err if loss == "preference" else 0.0)
    assert ((net.fc.bias.grad.double() - want.sum(0)).abs() <= bound.sum(0) * 1.01).all()
    off = (net.fc.weight.grad.double() - want.T @ x.double()).abs()
    assert (off <= (bound.T @ x.double().abs()) * 1.01 + rows * U * (want.abs().T @ x.double().abs())).all()
    entries = want.abs().clone()
    entries.scatter_(1, token[:, None], 0.0)
    assert float(entries.median()) < 2.0 ** -24
    cap.remove()


def test_logits_of_any_layout_reach_the_loss(kfac_gpu):
    """Logits [batch, time, vocab], also as a transposed view: the same loss and gradients."""
    from fac_second_order_amd.capture import KfacCapture

    class Net(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.fc = torch.nn.Linear(6, 5)

        def kfac_modules(self):
            return [(self.fc, None)]

    torch.manual_seed(33)
    net = Net().cuda()
    cap = KfacCapture(net)
    x = torch.randn(12, 6, device="cuda")
    token = torch.randint(0, 5, (12,), device="cuda")
    old, adv = torch.full((12,), -1.6, device="cuda"), torch.randn(12, device="cuda")
    got = []
    for shape in (lambda z: z, lambda z: z.view(3, 4, 5), lambda z: z.t().contiguous().t()):
        net.zero_grad()
        stats, logp = cap.policy_backward(shape(net.fc(x)), token, old, adv, clip_high=5.0, clip_low=0.9)
        got.append((stats.clone(), logp, net.fc.weight.grad.clone()))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    cap.remove()
