"""Host-side checks of layers that keep their input in 8 bits (no GPU): options and their
refusals, what a step does with checkpoints among its activations, and that the capture leaves a
model as it found it."""
from types import SimpleNamespace

import pytest
import torch

from test_capture import Net, Recorder

cap_mod = pytest.importorskip("fac_second_order_amd.capture")
step_mod = pytest.importorskip("fac_second_order_amd.step")
ck = pytest.importorskip("fac_second_order_amd.checkpoint")


def held(rows, cols, first=1):
    return ck.Checkpoint(torch.full((rows, cols), first, dtype=torch.int8), torch.ones(rows))


def test_options():
    for kw in ({"checkpoint": "int4"}, {"checkpoint": 8}, {"matmul": "int8"}, {"checkpoint": "int8", "matmul": "fp8"}):
        with pytest.raises(ValueError):
            cap_mod.KfacCapture(Net(), **kw)


def test_what_a_checkpoint_is():
    for q, s in ((torch.zeros(3, 4), torch.ones(3)), (torch.zeros(3, dtype=torch.int8), torch.ones(3)),
                 (torch.zeros(3, 4, dtype=torch.int8), torch.ones(4)),
                 (torch.zeros(3, 4, dtype=torch.int8), torch.ones(3, dtype=torch.float64))):
        with pytest.raises(TypeError):
            ck.Checkpoint(q, s)
    with pytest.raises(ValueError):
        ck.Checkpoint.empty(torch.zeros(2, 3, 4))
    c = ck.Checkpoint(torch.arange(12, dtype=torch.int8).view(4, 3), torch.arange(4.0))
    some = c.index_select(0, torch.tensor([2, 0]))
    assert some.q.tolist() == [[6, 7, 8], [0, 1, 2]] and some.scale.tolist() == [2, 0]
    assert len(c) == 4 and tuple(c.shape) == (4, 3) and c.device == torch.device("cpu")
    with pytest.raises(ValueError):
        c.index_select(1, torch.tensor([0]))
    with pytest.raises(ValueError):     # no CPU path
        ck.Checkpoint.of(torch.zeros(2, 3))
    with pytest.raises(ValueError):
        ck.linear(torch.zeros(2, 3), torch.zeros(4, 3), None)


def test_capture_leaves_the_model(monkeypatch):
    monkeypatch.setattr(cap_mod, "KfacStep", Recorder)
    net = Net()
    own = lambda x: x  # noqa: E731
    net.a.forward = own
    cap = cap_mod.KfacCapture(net, checkpoint="int8")
    assert net.a.forward is not own and "forward" in net.b.__dict__
    with torch.no_grad():
        assert torch.equal(net.b(torch.ones(2, 6)), torch.nn.functional.linear(torch.ones(2, 6), net.b.weight, net.b.bias))
    with pytest.raises(ValueError):     # with gradients the input is kept: on a GPU
        net.b(torch.ones(2, 6))
    cap.remove()
    assert net.a.forward is own and "forward" not in net.b.__dict__
    plain = cap_mod.KfacCapture(net)
    assert "forward" not in net.b.__dict__
    plain.remove()


def layer(n, c_in, c_out, bias=1, **kw):
    f = dict(n=n, h=1, w=1, c_in=c_in, h_out=1, w_out=1, c_out=c_out, kh=1, kw=1, sh=1, sw=1, ph=0, pw=0, bias=bias)
    return SimpleNamespace(**{**f, **kw})


class Calls:
    """Stands in for the library of a step: what it was called with."""

    def __init__(self, monkeypatch):
        self.q8, self.plain = [], []
        K = step_mod.K
        for name in ("kfac_factors_workspace", "kfac_pack_sym_workspace", "kfac_invert_workspace",
                     "kfac_precondition_workspace"):
            monkeypatch.setattr(K, name, lambda *a, **k: 64)
        monkeypatch.setattr(K, "kfac_factors_q8_workspace", lambda rows, cols, bias: 100000)
        monkeypatch.setattr(K, "kfac_factors_q8", lambda *a: self.q8.append(a))
        monkeypatch.setattr(K, "kfac_factors_full", lambda *a: self.plain.append(a))
        monkeypatch.setattr(K, "kfac_factors", lambda *a: self.plain.append(a))
        for name in ("kfac_invert", "kfac_precondition"):
            monkeypatch.setattr(K, name, lambda *a, **k: None)


def test_step_forms_factors_of_checkpoints(monkeypatch):
    calls = Calls(monkeypatch)
    layers = [layer(5, 3, 4), layer(5, 4, 2, bias=0), layer(5, 2, 2)]
    st = step_mod.KfacStep(layers, device="cpu")
    small = st.workspace.numel()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    act = [held(5, 3), torch.zeros(5, 4), held(5, 2, 7)]
    gout = [torch.zeros(5, 4), torch.zeros(5, 2), torch.zeros(5, 2)]
    st.step(act, gout, [torch.zeros(4, 4), torch.zeros(2, 4), torch.zeros(2, 3)], ema_decay=0.5)
    (q, s, packed, full, bias, decay, ws, stream), = calls.q8
    assert [t.data_ptr() for t in q] == [act[0].q.data_ptr(), act[2].q.data_ptr()]
    assert [t.data_ptr() for t in packed] == [st.A_packed[0].data_ptr(), st.A_packed[2].data_ptr()]
    assert [t.data_ptr() for t in full] == [st.full[0].data_ptr(), st.full[2].data_ptr()]
    assert bias == [1, 1] and decay == 0.5 and ws.numel() >= 100000 > small
    (_, a, g, *_), = calls.plain
    assert a[0] is None and a[2] is None and a[1] is act[1] and g == gout
    # nothing but checkpoints: no other factor call
    calls.q8.clear(), calls.plain.clear()
    st.factors([held(5, 3), held(5, 4), held(5, 2)], [None] * 3)
    assert len(calls.q8) == 1 and not calls.plain and calls.q8[0][3] is None and calls.q8[0][4] == [1, 0, 1]
    # a stale step looks at none
    calls.q8.clear()
    st.step([None] * 3, [None] * 3, [None] * 3, refresh=False)
    assert not calls.q8


@pytest.mark.parametrize("act,lay", [(held(5, 4), layer(5, 3, 4)), (held(4, 3), layer(5, 3, 4)),
                                     (held(5, 3), layer(5, 3, 4, kh=3)), (held(5, 3), layer(5, 3, 4, h=2, w=2, h_out=2, w_out=2))])
def test_step_refuses_other_checkpoints(monkeypatch, act, lay):
    calls = Calls(monkeypatch)
    st = step_mod.KfacStep([lay], device="cpu")
    with pytest.raises(ValueError):
        st.step([act], [torch.zeros(5, 4)], [torch.zeros(4, 4)])
    assert not calls.q8 and not calls.plain


class Tenfold(torch.nn.Linear):
    def forward(self, input):
        return 10 * super().forward(input)


def test_layers_with_a_forward_of_their_own():
    """A class's forward, and one set on a layer, are what runs; their inputs are kept as without the option."""
    net = Net()
    net.a = Tenfold(5, 6)
    plain = net.b.forward
    net.b.forward = lambda x: plain(x) - 3
    x = torch.randn(2, 5)
    want = net(x).detach()
    cap = cap_mod.KfacCapture(net, checkpoint="int8", matmul="int8")
    with torch.no_grad():
        assert torch.equal(net(x), want)
    seen = []
    handle = net.b.register_forward_pre_hook(lambda m, inp: seen.append(inp[0].detach()))
    out = net(x)
    assert torch.equal(out, want) and not cap.made
    assert torch.equal(cap.act[0], x.half()) and torch.equal(cap.act[1], seen[0].half())
    out.sum().backward()
    assert torch.equal(net.a.weight.grad, torch.autograd.grad(net(x).sum(), net.a.weight)[0])
    handle.remove()
    cap.remove()
    assert "forward" not in net.a.__dict__ and torch.equal(net(x), want)


@pytest.mark.parametrize("kw", [{}, {"checkpoint": "int8"}, {"checkpoint": "int8", "matmul": "int8"}])
def test_copies_of_a_model(kw):
    """A copy computes with its own weights, in 16 bits or more, and nothing of its passes is captured."""
    import copy
    net = Net()
    fourfold = lambda x: torch.nn.functional.linear(x, net.b.weight) * 4  # noqa: E731
    net.b.forward = fourfold
    cap = cap_mod.KfacCapture(net, **kw)
    for twin in (copy.deepcopy(net), copy.deepcopy(copy.deepcopy(net))):
        assert twin.b.forward is fourfold
        with torch.no_grad():
            for p in twin.a.parameters():
                p.zero_()
            assert not twin.a(torch.ones(2, 5)).any()
        x = torch.ones(3, 5)
        twin.a(x).sum().backward()
        assert torch.equal(twin.a.weight.grad, torch.full((6, 5), 3.0)) and net.a.weight.grad is None
        assert cap.n == 0 and not cap.made and cap.act == cap.gout == [None, None]
    alone = copy.deepcopy(net.a)
    with torch.no_grad():
        alone.bias.fill_(2)
        alone.weight.zero_()
        assert (alone(torch.ones(1, 5)) == 2).all()
    cap.remove()
    assert "forward" not in net.a.__dict__ and net.b.forward is fourfold


def test_copies_of_normalised_models(monkeypatch):
    import copy
    from test_capture import ConvNet
    net = ConvNet()
    cap = cap_mod.KfacCapture(net)
    copy.deepcopy(net)(torch.randn(2, 3, 4, 4)).sum().backward()
    assert cap.xhat == cap.bgout == [None] and cap.act == cap.gout == [None, None]


def test_input_by_name():
    net = Net()
    cap = cap_mod.KfacCapture(net, checkpoint="int8")
    x = torch.randn(2, 5)
    with torch.no_grad():
        assert torch.equal(net.a(input=x), torch.nn.functional.linear(x, net.a.weight, net.a.bias))
    cap.remove()


def test_parts_of_a_step_plan_for_all_of_it(monkeypatch):
    calls = Calls(monkeypatch)
    st = step_mod.KfacStep([layer(5, 3, 4), layer(5, 4, 2, bias=0), layer(5, 2, 2)], device="cpu")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    act, none = [held(5, 3), torch.zeros(5, 4), held(5, 2, 7)], [None] * 3
    st._factors_full(st.layers, [act[0], None, None], act, none, 0.5, None)
    (q, s, packed, full, *_), = calls.q8
    assert [t.data_ptr() for t in q] == [act[0].q.data_ptr(), act[2].q.data_ptr()]
    assert packed[0] is st.A_packed[0] and packed[1] is None and full[0] is st.full[0] and full[1] is None
    calls.q8.clear()
    st._factors_full(st.layers, [None, act[1], None], act, none, 0.5, None)
    assert not calls.q8 and len(calls.plain) == 1


def test_a_copy_is_captured_like_its_original():
    import copy
    net = Net()
    cap = cap_mod.KfacCapture(net, checkpoint="int8")
    twin = copy.deepcopy(net)
    cap.remove()
    cap = cap_mod.KfacCapture(twin, checkpoint="int8")
    with pytest.raises(ValueError):     # its layers keep their inputs in 8 bits: on a GPU
        twin.a(torch.ones(2, 5))
    cap.remove()
    assert torch.equal(twin(torch.ones(2, 5)), net(torch.ones(2, 5)))


def test_shallow_copies_of_layers():
    """Replicas and other copies that share a layer's attributes compute with their own weights."""
    import copy
    net = Net()
    cap = cap_mod.KfacCapture(net, checkpoint="int8")
    x = torch.randn(2, 5)
    for twin in (net.a._replicate_for_data_parallel(), copy.copy(net.a)):
        twin.__dict__["_parameters"] = {}
        twin.weight, twin.bias = torch.nn.Parameter(torch.zeros(6, 5)), torch.nn.Parameter(torch.full((6,), 2.0))
        for _ in range(2):
            out = twin(x)
            assert torch.equal(out, torch.full((2, 6), 2.0))
            out.sum().backward()
            assert twin.bias.grad is not None and net.a.bias.grad is None
            with torch.no_grad():
                want = torch.nn.functional.linear(x, net.a.weight, net.a.bias)
                assert torch.equal(net.a(x), want) and torch.equal(net.a.forward(x), want)
        assert cap.act == [None, None] and cap.n == 0 and not cap.made
    with pytest.raises(ValueError):     # the layer itself keeps its input: on a GPU
        net.a(x)
    cap.remove()
    assert not net.a._forward_pre_hooks and "forward" not in net.a.__dict__
