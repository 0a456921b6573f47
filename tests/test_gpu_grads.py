"""The gradient norm, the clipping and the bounded update on the GPU against fp64.

Bounds: squares and products are summed in fp64 (errors below 1e-12 of the sum of their
magnitudes), so a norm, step or q is off by its rounding to fp32, 2^-24. A clipped element is
c g with c rounded to fp32 and the product rounded to fp32 (2 * 2^-24) and then to its type.
w - s P is one fused operation: 2^-24 of the result and 2^-24 of s |P| from s."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import say
from loss_cases import FLOOR, HALF_STEP, U, host64
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
SIZES = [1, 3, 4, 7, 8, 255, 257, 0, 4096, 16383, 16384, 16385, 40001]


def _tensors(seed, sizes, dtypes, offset=0, scale=0.1):
    """Tensors of `sizes` with the types in turn, `offset` elements into a buffer of their own."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = (torch.randn(n + offset, generator=g) * scale).to(dtypes[i % len(dtypes)]).cuda()
        out.append(t[offset:])
    return out


def _norm(kfac, grads, **kw):
    norm = torch.full((1,), 7.0, device="cuda")
    kfac.kfac_grad_norm(grads, norm, **kw)
    torch.cuda.synchronize()
    return float(norm)


def _clip(kfac, grads, max_norm, widen=False, **kw):
    outs = [torch.full_like(t, 7.0, dtype=F32 if widen else t.dtype) for t in grads]
    norm = torch.full((1,), 7.0, device="cuda")
    kfac.kfac_grad_clip(grads, outs, max_norm, norm, **kw)
    torch.cuda.synchronize()
    return outs, float(norm)


def _check_clip(outs, norm, grads, max_norm):
    want = lo.global_norm([host64(t) for t in grads])
    c = lo.clip_scale(want, float(np.float32(max_norm)))
    assert abs(norm - want) <= want * (U * 1.01 + 1e-12)
    for o, t in zip(outs, grads):
        ref = host64(t) * c
        bound = np.abs(ref) * ((2 * U + (HALF_STEP[o.dtype] if o.dtype != F32 else 0)) * 1.01 if c != 1 else 0)
        assert (np.abs(host64(o) - ref) <= bound + (FLOOR[o.dtype] if c != 1 else 0)).all()


@pytest.mark.parametrize("dtypes", [[F32], [F16], [BF16], [F32, BF16, F16]])
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("widen", [False, True])
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clip_types_sizes_alignments(kfac_gpu, dtypes, offset, widen, max_norm):
    grads = _tensors(1, SIZES, dtypes, offset)
    outs, norm = _clip(kfac_gpu, grads, max_norm, widen)
    _check_clip(outs, norm, grads, max_norm)
    assert _norm(kfac_gpu, grads) == norm


@pytest.mark.parametrize("n", SIZES + [1 << 20, 3000001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_clip_one_tensor(kfac_gpu, n, dtype):
    grads = _tensors(2, [n], [dtype])
    outs, norm = _clip(kfac_gpu, grads, 0.01)
    _check_clip(outs, norm, grads, 0.01)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 129, 700])
def test_clip_many_tensors(kfac_gpu, count):
    grads = _tensors(3, [1 + (37 * i) % 900 for i in range(count)], [F32, BF16, F16])
    outs, norm = _clip(kfac_gpu, grads, 1.0, widen=True)
    _check_clip(outs, norm, grads, 1.0)


@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clip_in_place(kfac_gpu, max_norm):
    grads = _tensors(4, SIZES, [F32, BF16, F16])
    before = [t.clone() for t in grads]
    norm = torch.empty(1, device="cuda")
    kfac_gpu.kfac_grad_clip(grads, grads, max_norm, norm)
    torch.cuda.synchronize()
    _check_clip(grads, float(norm), before, max_norm)


def test_norm_edges(kfac_gpu):
    assert _norm(kfac_gpu, []) == 0.0
    assert _norm(kfac_gpu, [torch.zeros(0, device="cuda")] * 3) == 0.0
    assert _norm(kfac_gpu, [torch.zeros(5, device="cuda")]) == 0.0
    big = torch.full((1000,), 3e37, device="cuda")        # the squares do not fit in fp32
    assert _norm(kfac_gpu, [big]) == math.inf             # 3e37 sqrt(1000) = 9.5e38: past the largest float
    want = lo.global_norm([host64(big[:100])])            # 3e38
    assert abs(_norm(kfac_gpu, [big[:100]]) - want) <= want * U * 1.01
    tiny = torch.full((1000,), 1e-40, device="cuda")      # nor do these
    want = lo.global_norm([host64(tiny)])
    assert abs(_norm(kfac_gpu, [tiny]) - want) <= FLOOR[F32]
    same = torch.full((4,), 1.0, device="cuda")
    assert _norm(kfac_gpu, [same, same, same, same]) == 4.0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_clip_leaves_what_is_not_finite(kfac_gpu, bad):
    grads = _tensors(5, [100, 20000], [F32, BF16])
    grads[1][777] = bad
    outs, norm = _clip(kfac_gpu, grads, 0.5)
    assert (math.isnan(norm) if math.isnan(bad) else norm == math.inf)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, grads))
    huge = [torch.full((16,), 3e38, device="cuda")]       # a norm past the largest float
    outs, norm = _clip(kfac_gpu, huge, 0.5)
    assert norm == math.inf and torch.equal(outs[0], huge[0])


@pytest.mark.parametrize("dtypes", [[F32], [BF16], [F32, BF16]])
@pytest.mark.parametrize("n,scale", [(1000, 5e36), (70001, 5e35)])
@pytest.mark.parametrize("max_norm", [1e-3, 1e-9, 1e-30])
@pytest.mark.parametrize("widen", [False, True])
def test_clip_by_a_factor_below_the_smallest_float(kfac_gpu, dtypes, n, scale, max_norm, widen):
    """A norm of 1e38 and a small bound: their quotient is no normal float (6e-42, with 12 bits) or none at
    all, the clipped gradients are ordinary numbers."""
    grads = _tensors(6, [n] * len(dtypes), dtypes, scale=scale)
    outs, norm = _clip(kfac_gpu, grads, max_norm, widen)
    assert math.isfinite(norm) and max_norm / norm < 2.0 ** -126
    _check_clip(outs, norm, grads, max_norm)
    assert all(o.any() for o in outs)


@pytest.mark.parametrize("n", [4, 100000])
def test_clip_in_place_by_a_factor_that_rounds_to_a_power(kfac_gpu, n):
    """max / norm = 2^-126 (1 - 2^-31): its first part rounds to 1, and the gradients are scaled all the same."""
    t = torch.zeros(n, device="cuda")
    t[0], t[1] = 2.0 ** 100, 2.0 ** 85
    norm = torch.empty(1, device="cuda")
    kfac_gpu.kfac_grad_clip([t], [t], 2.0 ** -26, norm)
    torch.cuda.synchronize()
    assert float(norm) == 2.0 ** 100 and t[:2].tolist() == [2.0 ** -26, 2.0 ** -41]


def test_norm_past_32_bit_offsets(kfac_gpu):
    """One tensor of more than 2^31 elements and 2^32 bytes, values at its ends and about 2^31."""
    n = (1 << 31) + 70001
    t = torch.zeros(n, dtype=F16, device="cuda")
    for at, v in ((0, 1.0), ((1 << 31) - 1, 2.0), (1 << 31, 4.0), (n - 1, 8.0)):
        t[at] = v
    assert _norm(kfac_gpu, [t]) == float(np.float32(math.sqrt(85.0)))
    norm = torch.empty(1, device="cuda")
    kfac_gpu.kfac_grad_clip([t], [t], math.sqrt(85.0) / 2, norm)
    torch.cuda.synchronize()
    assert [float(t[i]) for i in (0, (1 << 31) - 1, 1 << 31, n - 1)] == [0.5, 1.0, 2.0, 4.0]
    assert int(torch.count_nonzero(t[: 1 << 30])) + int(torch.count_nonzero(t[1 << 30:])) == 4


def _trust(kfac, P, g, w, lr, delta, **kw):
    step = torch.full((2,), 7.0, device="cuda")
    kfac.kfac_trust_update(P, g, w, lr, delta, step, **kw)
    torch.cuda.synchronize()
    return step


def _check_trust(step, w, w0, P, g, lr, delta, fisher=None, shift=0.0):
    lr, delta, shift = (float(np.float32(v)) for v in (lr, delta, shift))
    ps = [host64(p) for p in P]
    gs = [None if t is None else host64(t) for t in g]
    fs = None if fisher is None else [None if t is None else host64(t) for t in fisher]
    s, q = lo.trust_step(ps, gs, lr, delta, fs, shift)
    size = sum(float((np.abs(p) * np.abs(p * (fs[i] + shift) if gs[i] is None else gs[i])).sum())
               for i, p in enumerate(ps))
    q_err = 1e-12 * size
    assert abs(float(step[1]) - q) <= abs(q) * U * 1.01 + q_err
    rel = (q_err / abs(q) if q else 0.0) + 1.01 * U
    assert abs(float(step[0]) - s) <= s * rel
    say("trust: step", float(step[0]), "q", q)
    for new, old, p in zip(w, w0, ps):
        ref = host64(old) - s * p
        assert (np.abs(host64(new) - ref) <= 1.01 * U * np.abs(ref) + s * np.abs(p) * rel * 1.01).all()


@pytest.mark.parametrize("dtypes", [[F32], [F16], [BF16], [F32, BF16, F16]])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("lr,delta", [(0.1, 1e9), (0.5, 1e-4)])
def test_trust_types_sizes(kfac_gpu, dtypes, offset, lr, delta):
    P = _tensors(10, SIZES, [F32], offset)
    w = _tensors(11, SIZES, [F32], offset)
    g = [(p * 0.3).to(dtypes[i % len(dtypes)]) for i, p in enumerate(P)]
    w0 = [t.clone() for t in w]
    step = _trust(kfac_gpu, P, g, w, lr, delta)
    _check_trust(step, w, w0, P, g, lr, delta)
    assert (float(step[0]) == float(np.float32(lr))) == (delta == 1e9)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_trust_diagonal_entries(kfac_gpu, sign):
    sizes = [512, 30, 0, 2 * 2048, 7]
    P = _tensors(12, sizes, [F32])
    w = _tensors(13, sizes, [F32])
    fisher = [None if i == 0 else t.abs() for i, t in enumerate(_tensors(14, sizes, [F32]))]
    g = [P[0] * 0.01 * sign] + [None] * 4
    w0 = [t.clone() for t in w]
    step = _trust(kfac_gpu, P, g, w, 5.0, 1e-3, fisher=fisher, shift=1e-3)
    _check_trust(step, w, w0, P, g, 5.0, 1e-3, fisher, 1e-3)


def test_trust_edges(kfac_gpu):
    step = _trust(kfac_gpu, [], [], [], 0.25, 1.0)
    assert step.tolist() == [0.25, 0.0]
    P, w = _tensors(15, [300], [F32]), _tensors(16, [300], [F32])
    w0 = w[0].clone()
    assert _trust(kfac_gpu, P, [torch.zeros_like(P[0])], w, 0.25, 1.0)[0] == 0.25     # q = 0: the rate
    assert torch.equal(w[0], torch.addcmul(w0, P[0], torch.tensor(-0.25, device="cuda")))
    for bad in (float("nan"), float("inf")):
        w0 = w[0].clone()
        g = P[0].clone()
        g[7] = bad
        step = _trust(kfac_gpu, P, [g], w, 0.25, 1.0)
        assert step[0] == 0 and not step[1].isfinite() and torch.equal(w[0], w0)
    w0 = w[0].clone()
    assert _trust(kfac_gpu, P, [P[0]], w, 0.0, 1.0)[0] == 0 and torch.equal(w[0], w0)
    _trust(kfac_gpu, P, [P[0]], w, 1.0, 1.0)       # the gradient may be the preconditioned one


def test_calls_repeat_bit_for_bit(kfac_gpu):
    grads = _tensors(20, SIZES + [1000003], [F32, BF16, F16])
    (a, na), (b, nb) = (_clip(kfac_gpu, grads, 0.3) for _ in range(2))
    assert na == nb and all(torch.equal(x, y) for x, y in zip(a, b))
    P = _tensors(21, SIZES + [1000003], [F32])
    w = [_tensors(22, SIZES + [1000003], [F32]) for _ in range(2)]
    s = [_trust(kfac_gpu, P, grads, v, 0.3, 1e-3) for v in w]
    assert torch.equal(*s) and all(torch.equal(x, y) for x, y in zip(*w))


def test_calls_on_another_stream(kfac_gpu):
    grads = _tensors(23, SIZES * 3, [F32, BF16])
    want, norm = _clip(kfac_gpu, grads, 0.3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in grads]
    got = torch.empty(1, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        kfac_gpu.kfac_grad_clip(grads, outs, 0.3, got, stream=side)
        torch.full((1 << 13,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    assert float(got) == norm and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_in_a_graph(kfac_gpu):
    """Clipping and the bounded update captured with one workspace, replayed on new
    gradients, eager calls between the replays."""
    sizes = SIZES + [200003]
    grads, P, w = _tensors(24, sizes, [BF16]), _tensors(25, sizes, [F32]), _tensors(26, sizes, [F32])
    outs = [torch.empty_like(t, dtype=F32) for t in grads]
    norm, step = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    ws = torch.empty(kfac_gpu.kfac_grad_norm_workspace(sizes) + 256, dtype=torch.uint8, device="cuda")

    def calls():
        kfac_gpu.kfac_grad_clip(grads, outs, 0.3, norm, workspace=ws)
        kfac_gpu.kfac_trust_update(P, outs, w, 0.5, 1e-4, step, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(4):
        for t, new in zip(grads, _tensors(30 + k, sizes, [BF16])):
            t.copy_(new)
        w0 = [t.clone() for t in w]
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in (*outs, *w, norm, step)]
        for t, v in zip(w, w0):
            t.copy_(v)
        for t in (*outs, norm, step):
            t.fill_(3.0)
        calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(have, (*outs, *w, norm, step))), k


@pytest.mark.parametrize("n", [300, 70001])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_trust_leaves_alone_what_a_float_does_not_hold(kfac_gpu, n, sign):
    """P and g finite, and q finite in fp64 (n 1e40) but no float: the step is 0, w stays and q
    shows it; one launch and several."""
    P, g = [torch.full((n,), 1e20, device="cuda")], [torch.full((n,), sign * 1e20, device="cuda")]
    w = _tensors(17, [n], [F32])
    w0 = w[0].clone()
    assert _trust(kfac_gpu, P, g, w, 0.25, 1.0).tolist() == [0.0, sign * math.inf]
    assert torch.equal(w[0], w0)
    # n 1e32 is one
    P, g = [torch.full((n,), 1e16, device="cuda")], [torch.full((n,), sign * 1e16, device="cuda")]
    step = _trust(kfac_gpu, P, g, w, 0.25, 1e30)
    assert step[0] > 0 and step[1].isfinite() and not torch.equal(w[0], w0)
