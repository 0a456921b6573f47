"""Layers that keep their input in 8 bits, on the GPU: a model's forward and backward passes and
its step against the formulas in fp64, and the calls together on streams and in graphs.

Bounds. Weight gradients are fp32 sums of exact products (n 2^-23 of the sum of the magnitudes, as in the
tests of the calls), rounded once to the weights' type: by half a step of it, relative where numbers are
normal and half the distance of the subnormals (2^-25 for fp16, below 2^-14) where they are not. Factors likewise. Inverses and steps
amplify a factor's difference by its condition number."""
import numpy as np
import pytest
import torch

from gpu_helpers import relF, say
from loss_cases import FLOOR, HALF_STEP, U, host64
from oracle import q8_oracle as qo

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


class Mlp(torch.nn.Module):
    def __init__(self, sizes, dtype=F32, bias=True):
        super().__init__()
        self.layers = torch.nn.ModuleList(torch.nn.Linear(a, b, bias=bias, dtype=dtype) for a, b in zip(sizes, sizes[1:]))

    def forward(self, x):
        for i, m in enumerate(self.layers):
            x = m(torch.relu(x) if i else x)
        return x

    def kfac_modules(self):
        return [(m, None) for m in self.layers]


def watched(net):
    """Inputs, outputs and gradients at the outputs of the layers, as passes go through them."""
    seen = {}

    def forward(i):
        def hook(mod, inp, out):
            seen["x", i], seen["y", i] = inp[0].detach().clone(), out.detach().clone()
            if out.requires_grad:
                out.register_hook(lambda g: seen.__setitem__(("g", i), g.detach().clone()))
        return hook

    for i, m in enumerate(net.layers):
        m.register_forward_hook(forward(i))
    return seen


def grad_close(got, want, size, terms, dtype):
    bound = terms * 2 * U * size + (HALF_STEP[dtype] * np.abs(want) * 1.01 + FLOOR[dtype] if dtype != F32 else 0)
    off = np.abs(host64(got) - want)
    if (off > bound).any():
        at = np.unravel_index(np.argmax(off - bound), off.shape)
        say("worst", at, host64(got)[at], want[at], "off", off[at], "bound", bound[at])
    return (off <= bound).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("matmul", [None, "int8"])
@pytest.mark.parametrize("rows", [1, 7, 130])
def test_passes_of_a_model(kfac_gpu, dtype, matmul, rows):
    from fac_second_order_amd.capture import KfacCapture
    torch.manual_seed(1)
    net = Mlp([33, 64, 40, 9], dtype, bias=rows != 7).cuda()
    cap = KfacCapture(net, checkpoint="int8", matmul=matmul)
    seen = watched(net)
    x = torch.randn(rows, 33, device="cuda").to(dtype).requires_grad_()
    out = net(x)
    c = torch.randn_like(out)
    out.backward(c)
    for i, m in enumerate(net.layers):
        cp = cap.act[i]
        q, s = qo.quantize_rows(host64(seen["x", i]))
        assert np.array_equal(host64(cp.q), q) and np.array_equal(host64(cp.scale), s)
        g = host64(seen["g", i])
        dw, db, size, bsize = qo.weight_grad(g, q, s)
        terms = rows * (3 if dtype == F32 else 1) + 8
        assert grad_close(m.weight.grad, dw, size, terms, dtype)
        assert m.bias is None or grad_close(m.bias.grad, db, bsize, terms, dtype)
        if matmul:
            wq, ws = qo.quantize_rows(host64(m.weight), pow2=False)
            y, ysize = qo.linear(q, s, wq, ws, None if m.bias is None else host64(m.bias))
            assert (np.abs(host64(seen["y", i]) - y) <= 4 * U * ysize * 1.01 + HALF_STEP[dtype] * np.abs(y) * 1.01 + 1e-7).all()
        else:
            assert torch.equal(seen["y", i], torch.nn.functional.linear(seen["x", i], m.weight, m.bias))
    assert torch.equal(x.grad, seen["g", 0] @ net.layers[0].weight)
    # gradients add up, as autograd's do
    before = [m.weight.grad.clone() for m in net.layers]
    net(x).backward(c)
    for m, b in zip(net.layers, before):
        assert torch.equal(m.weight.grad, b + b)
    # a pass without gradients keeps nothing
    acts = list(cap.act)
    with torch.no_grad():
        again = net(x)
    assert torch.equal(again, out) and all(a is b for a, b in zip(acts, cap.act)) and not cap.made
    cap.remove()


def test_gradients_against_differences(kfac_gpu):
    """d(sum c y)/dW by central differences of the product that the backward pass belongs to: the values of
    the checkpoint times W, linear in W, so that only fp32's rounding is left."""
    torch.manual_seed(2)
    x, W, b = (torch.randn(*s, device="cuda") for s in ((20, 11), (6, 11), (6,)))
    c = torch.randn(20, 6, device="cuda")
    W.requires_grad_(), b.requires_grad_()
    from fac_second_order_amd import checkpoint as ck
    y, cp = ck.linear(x, W, b)
    (c * y).sum().backward()
    v = cp.values(F32).double()
    assert torch.equal(v, cp.q.double() * cp.scale.double()[:, None])

    def f(W, b):
        return float((c.double() * (v @ W.T + b)).sum())

    h, Wd, bd = 0.25, W.detach().double(), b.detach().double()
    for o, k in ((0, 0), (3, 10), (5, 4)):
        E = torch.zeros_like(Wd)
        E[o, k] = h
        diff = (f(Wd + E, bd) - f(Wd - E, bd)) / (2 * h)
        assert abs(diff - float(W.grad[o, k])) <= 68 * 2 * U * float((c[:, o].abs().double() * v[:, k].abs()).sum()) + 1e-9
        e = torch.zeros_like(bd)
        e[o] = h
        diff = (f(Wd, bd + e) - f(Wd, bd - e)) / (2 * h)
        assert abs(diff - float(b.grad[o])) <= 68 * 2 * U * float(c[:, o].abs().sum()) + 1e-9


@pytest.mark.parametrize("sizes", [[40, 64, 24], [33, 1100, 50]])   # the second one inverts on two streams
def test_step_of_checkpoints(kfac_gpu, sizes):
    from fac_second_order_amd.capture import KfacCapture
    from fac_second_order_amd.step import KfacStep
    torch.manual_seed(3)
    rows = 300
    net = Mlp(sizes).cuda()
    cap = KfacCapture(net, damping=0.1, checkpoint="int8")
    w0 = [cap._to_matrix(m).clone() for m in net.layers]
    for call in range(2):
        net.zero_grad()
        x = torch.randn(rows, sizes[0], device="cuda")
        logits = net(x)
        torch.nn.functional.cross_entropy(logits, torch.randint(0, sizes[-1], (rows,), device="cuda")).backward()
        old = None if call == 0 else [host64(p) for p in cap.kstep.A_packed]
        grads = [cap._to_matrix(m, grad=True).clone() for m in net.layers]
        acts, gouts = list(cap.act), list(cap.gout)
        cap.step(0.05)
        for l, a in enumerate(acts):
            want, size = qo.factor_packed(host64(a.q), host64(a.scale), True, None if old is None else old[l],
                                          0.95 if call else 0.0)
            assert (np.abs(host64(cap.kstep.A_packed[l]) - want) <= (rows + 12) * 2 * U * size).all()
        if call == 0:
            # the same step from the values in fp16, which holds them exactly: the path of other layers
            st = KfacStep(*cap._geometry(), "cuda", damping=0.1)
            w = [m.clone() for m in w0]
            st.step([a.values(F16) for a in acts], gouts, grads, weights=w, lr=0.05)
            assert torch.equal(acts[0].values(F16).float(), acts[0].values(F32))
            for l, (a, b) in enumerate(zip(st.out, cap.kstep.out)):
                cond = sum(float(np.linalg.norm(host64(f), 2)) / 0.316 + 1 for f in (st.A_inv[l].inverse(), st.G_inv[l].inverse()))
                say("layer", l, "P against the fp16 path", relF(host64(b), host64(a)), "condition", cond)
                assert relF(host64(b), host64(a)) <= cond * 2.0 ** -17
    assert not any(torch.equal(cap._to_matrix(m), w) for m, w in zip(net.layers, w0))
    assert all(torch.isfinite(p).all() for p in net.parameters())
    cap.remove()


@pytest.mark.parametrize("matmul", [None, "int8"])
def test_policy_step_of_rows_that_count(kfac_gpu, matmul):
    """The factors of a policy's step are those of the rows that count, from their checkpoints."""
    from fac_second_order_amd.capture import KfacCapture
    torch.manual_seed(4)
    rows, d, choices = 200, 30, 12
    net = Mlp([d, 48, choices]).cuda()
    cap = KfacCapture(net, damping=1e-3, trust_radius=1e-3, checkpoint="int8", matmul=matmul)
    x = torch.randn(rows, d, device="cuda")
    mask = torch.arange(rows, device="cuda") % 3 != 0
    x[~mask] *= 50
    token = torch.randint(0, choices, (rows,), device="cuda")
    logits = net(x)
    old = torch.log_softmax(logits.detach(), 1).gather(1, token[:, None])[:, 0]
    cap.policy_backward(logits, token, old, torch.randn(rows, device="cuda"), mask=mask)
    acts = [a.index_select(0, mask.nonzero()[:, 0]) for a in cap.act]
    cap.step(lr=1.0)
    for l, a in enumerate(acts):
        want, size = qo.factor_packed(host64(a.q), host64(a.scale), True)
        assert (np.abs(host64(cap.kstep.A_packed[l]) - want) <= (rows + 8) * 2 * U * size).all()
    s, q = (float(v) for v in cap.kstep.trust)
    assert abs(0.5 * s * s * q - 1e-3) <= 1e-3 * 8 * U
    cap.remove()


def test_autocast(kfac_gpu):
    from fac_second_order_amd.capture import KfacCapture
    torch.manual_seed(5)
    net = Mlp([32, 24, 8]).cuda()
    cap = KfacCapture(net, checkpoint="int8")
    x = torch.randn(50, 32, device="cuda")
    with torch.autocast("cuda", dtype=BF16):
        out = net(x)
    assert out.dtype == BF16
    out.float().square().sum().backward()
    assert all(m.weight.grad.dtype == F32 for m in net.layers)
    q, s = qo.quantize_rows(host64(x.to(BF16)))
    assert np.array_equal(host64(cap.act[0].q), q)
    cap.remove()


# the calls together ---------------------------------------------------------------

class Chain:
    """A layer's pass: product and checkpoint, weight gradient, factor, reading back."""

    def __init__(self, kfac, rows, c_in, c_out, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kfac, self.g = kfac, g
        self.x = torch.randn(rows, c_in, generator=g, device="cuda").to(dtype)
        self.gout = (torch.randn(rows, c_out, generator=g, device="cuda") * 0.1).to(dtype)
        self.w = torch.randint(-127, 128, (c_out, c_in), generator=g, device="cuda").to(torch.int8)
        self.ws = torch.rand(c_out, generator=g, device="cuda") * 0.01
        self.mask = torch.rand(rows, generator=g, device="cuda") < 0.8
        d = c_in + 1
        e = lambda *s, t=F32: torch.full(s, 7, dtype=t, device="cuda")  # noqa: E731
        self.q, self.s, self.y, self.back = e(rows, c_in, t=torch.int8), e(rows), e(rows, c_out, t=dtype), e(rows, c_in, t=dtype)
        self.dw, self.A, self.full = e(c_out, d), e(d * (d + 1) // 2), torch.zeros(d, d, device="cuda")
        need = max(kfac.kfac_linear_q8_workspace(rows, c_in, c_out), kfac.kfac_factors_q8_workspace([rows], [c_in], True),
                   kfac.kfac_weight_grad_q8_workspace(rows, c_in, c_out, dtype))
        self.ws_bytes = torch.empty(need + 256, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        k, c_in = self.kfac, self.x.shape[1]
        kw = dict(workspace=self.ws_bytes, stream=stream)
        k.kfac_linear_q8(self.x, self.q, self.s, self.w, self.ws, self.y, mask=self.mask, **kw)
        k.kfac_weight_grad_q8(self.gout, self.q, self.s, self.dw[:, :c_in], dbias=self.dw[:, c_in], **kw)
        k.kfac_factors_q8([self.q], [self.s], [self.A], [self.full], bias=True, **kw)
        k.kfac_dequantize_rows(self.q, self.s, self.back, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.q, self.s, self.y, self.dw, self.A, self.full, self.back)]


CHAINS = [(1, 64, 48), (3, 40, 33), (200, 130, 65), (700, 512, 1031), (3000, 1032, 264)]


@pytest.mark.parametrize("rows,c_in,c_out", CHAINS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_calls_together_are_deterministic(kfac_gpu, rows, c_in, c_out, dtype):
    """Run to run, on another stream, two at once with their own workspaces, and captured and replayed
    between eager work: the same bits."""
    a, b = (Chain(kfac_gpu, rows, c_in, c_out, dtype, seed) for seed in (1, 2))
    a.run(), b.run()
    torch.cuda.synchronize()
    want_a, want_b = a.outputs(), b.outputs()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for c in (a, b):
        for t in (c.q, c.s, c.y, c.dw, c.A, c.back):
            t.fill_(1)
    torch.cuda.synchronize()
    a.run(stream=s1), b.run(stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.outputs() + b.outputs(), want_a + want_b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for turn in range(3):
        for t in (a.q, a.s, a.y, a.dw, a.A, a.back):
            t.fill_(turn + 2)
        b.run()                                   # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.outputs(), want_a)), turn
        assert all(torch.equal(x, y) for x, y in zip(b.outputs(), want_b)), turn
    # the graph takes new inputs
    a.x.copy_(b.x), a.gout.copy_(b.gout), a.w.copy_(b.w), a.ws.copy_(b.ws), a.mask.copy_(b.mask)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.outputs(), want_b))


def test_workspace_guard(kfac_gpu):
    """A workspace that is too small is refused, and nothing behind one is written."""
    c = Chain(kfac_gpu, 3000, 520, 264, BF16, 3)
    need = kfac_gpu.kfac_weight_grad_q8_workspace(3000, 520, 264, BF16)
    assert need > 0
    big = torch.full((need + 8192,), 9, dtype=torch.uint8, device="cuda")
    at = -big.data_ptr() % 256
    kfac_gpu.kfac_quantize_rows(c.x, c.q, c.s)
    with pytest.raises(kfac_gpu.KfacError):
        kfac_gpu.kfac_weight_grad_q8(c.gout, c.q, c.s, c.dw[:, :520], dbias=c.dw[:, 520], workspace=big[at:at + need - 256])
    kfac_gpu.kfac_weight_grad_q8(c.gout, c.q, c.s, c.dw[:, :520], dbias=c.dw[:, 520], workspace=big[at:at + need])
    torch.cuda.synchronize()
    assert (big[at + need:] == 9).all() and (big[:at] == 9).all()


@pytest.mark.parametrize("sizes, rows", [([600, 1100, 700, 40], 3000), ([40, 1500, 9, 520, 64], 700)])
def test_two_streams_give_the_bits_of_one(kfac_gpu, sizes, rows):
    """Factors of checkpoints that are formed in several calls, over scales that do not fit into 32 bits."""
    from fac_second_order_amd.capture import KfacCapture
    from fac_second_order_amd.step import KfacStep
    torch.manual_seed(6)
    net = Mlp(sizes).cuda()
    cap = KfacCapture(net, damping=0.1, checkpoint="int8")
    x = torch.randn(rows, sizes[0], device="cuda") * torch.exp2(-(torch.arange(rows, device="cuda") % 23).float())[:, None]
    torch.nn.functional.cross_entropy(net(x), torch.randint(0, sizes[-1], (rows,), device="cuda")).backward()
    layers, _ = cap._geometry()
    grads = [cap._to_matrix(m, grad=True) for m in net.layers]
    steps = [KfacStep(layers, (), "cuda", damping=0.1, side_stream=side) for side in (True, False)]
    assert steps[0].side and not steps[1].side
    for turn in range(2):
        for st in steps:
            st.step(cap.act, cap.gout, grads, ema_decay=0.5 * turn)
        torch.cuda.synchronize()
        for a, b in zip(*([*st.A_packed, *st.G_packed, *st.out] for st in steps)):
            assert torch.equal(a, b)
    cap.remove()
