"""One K-FAC step over a fixed set of layers: device buffers plus the sequence of
library calls (factors, written packed and as the upper triangle the inversion
reads -> damped inverses -> preconditioning, and the BatchNorm diagonal). Python only allocates and sequences; every number is computed
by libkfac's HIP kernels.

Step order follows Osawa et al. (CVPR 2019): stage 1-2 of their Figure 1 (factors
from the forward activations and backward gradients), eq. (6) (inverses of the
damped factors), eq. (7) (preconditioned gradients) and, when parameters are
given, eq. (8) (the update with learning rate lr); BatchNorm uses the diagonal
Fisher (Section 1, contributions)."""
import math

import torch

from . import _lib as K
from .checkpoint import Checkpoint


def side_split(n_all, min_order=1024):
    """Indices of the matrices whose inverses go to the second stream: those of order
    more than half the largest, when the largest order is at least min_order (a sweep
    of 8 block steps or more; below that the events cost more than the overlap gains)
    and the split leaves matrices on both streams; else none."""
    n_max = max(n_all) if n_all else 0
    long_ = [i for i, n in enumerate(n_all) if 2 * n > n_max + 2]
    if n_max < min_order or len(long_) in (0, len(n_all)):
        return []
    return long_


def _bound(v, what):
    """v, None or a number whose float32 is positive and finite."""
    if v is not None and not 0.0 < float(torch.tensor(float(v), dtype=torch.float32)) < math.inf:
        raise ValueError(f"{what} must be positive and finite")
    return v


def _same_but_samples(given, made, fields, what):
    """`given`, layers that differ from `made` in n alone; `made` where it is None."""
    if given is None:
        return made
    names = [f for f, _ in fields if f != "n"]
    if len(given) != len(made) or any(getattr(a, f) != getattr(b, f) for a, b in zip(given, made) for f in names):
        raise ValueError(f"{what} may differ in n alone from those the step was made for")
    return given


class KfacStep:
    """Buffers for `layers` (objects with the kfac_layer fields) and `bn_layers`
    (objects with n, hw, c). Tikhonov damping gamma puts sqrt(gamma) on each
    Kronecker factor (float32-rounded) and gamma on the BN diagonal. precond_accum
    "f64" sums the preconditioning products in fp64 (kfac_precondition_ex).
    refine_inverse applies one fp64-residual refinement step to every inverse
    (kfac_invert_refine), which keeps a full symmetric copy of each factor.

    side_stream: when the largest order is 1024 or more, the inverses of the factors
    whose order is more than half the largest order (their block sweep is the long
    tail of the batch, a chain of latency-bound launches that leaves most compute
    units idle) run on a second stream, together with the preconditioning of their
    layers, while the caller's stream inverts the rest, preconditions their layers
    and does the BatchNorm step. The step joins the two streams before it returns;
    results are the same bits as with one stream.

    max_grad_norm: step() first clips the layers' weight gradients by their global norm
    (kfac_grad_clip) into fp32 copies of its own, which it then preconditions; the
    gradients may be float16, bfloat16 or float32. self.grad_norm holds the norm.

    trust_radius: step() updates the parameters last and together, by the step s P
    whose quadratic form s^2/2 <P, F P> = s^2/2 <P, gradient> is at most this
    (kfac_trust_update): s is lr where that is smaller. self.trust holds s and <P, gradient>.
    F is the damped curvature of the call's own factors. The form predicts the KL
    divergence of the model's distribution where that is its Fisher: gout (and bn_fisher)
    the gradients of log-probabilities of outcomes drawn from the model, one sample each, as
    KfacCapture.policy_backward takes them. Of a loss's own gradients it predicts none: F
    then scales with the loss.

    act: tensors as kfac_factors takes them, or for fully connected layers a Checkpoint of
    their rows, whose factor kfac_factors_q8 forms."""

    def __init__(self, layers, bn_layers=(), device="cuda", damping=1e-3, bn_shift=None,
                 in_dtype=torch.float16, precond_accum="f32", refine_inverse=False, side_stream=True,
                 max_grad_norm=None, trust_radius=None):
        self.layers = list(layers)
        self.bn_layers = list(bn_layers)
        self.device = torch.device(device)
        if precond_accum not in ("f32", "f64"):
            raise ValueError("precond_accum must be 'f32' or 'f64'")
        self.accum = K.KFAC_F64 if precond_accum == "f64" else K.KFAC_F32
        self.shift = float(torch.tensor(math.sqrt(damping), dtype=torch.float32))
        self.bn_shift = float(damping if bn_shift is None else bn_shift)
        self.d_a = [l.c_in * l.kh * l.kw + (1 if l.bias else 0) for l in self.layers]
        self.d_g = [l.c_out for l in self.layers]
        dev = self.device
        f32 = torch.float32
        self.A_packed = [torch.empty(d * (d + 1) // 2, dtype=f32, device=dev) for d in self.d_a]
        self.G_packed = [torch.empty(d * (d + 1) // 2, dtype=f32, device=dev) for d in self.d_g]
        # factor k of the inverse batch: A of every layer, then G of every layer
        self.n_all = self.d_a + self.d_g
        self.full = [torch.empty(d, d, dtype=f32, device=dev) for d in self.n_all]
        self.packed_all = self.A_packed + self.G_packed
        # matrices (indices into n_all) inverted on the second stream, and the layers
        # preconditioned there
        long_ = side_split(self.n_all) if side_stream and not refine_inverse else []
        L = len(self.layers)
        self.side = long_
        self.main = [i for i in range(len(self.n_all)) if i not in long_]
        self.side_layers = sorted({i % L for i in long_})
        self.main_layers = [l for l in range(L) if l not in self.side_layers]
        self._info_main = torch.zeros(len(self.main), dtype=torch.int32, device=dev)
        self._info_side = torch.zeros(len(self.side), dtype=torch.int32, device=dev)
        self.out = [torch.empty(g, a, dtype=f32, device=dev) for g, a in zip(self.d_g, self.d_a)]
        self.refine = bool(refine_inverse)
        self.factor_full = [torch.empty(d, d, dtype=f32, device=dev) for d in self.n_all] if self.refine else []
        self.max_grad_norm = _bound(max_grad_norm, "max_grad_norm")
        self.trust_radius = _bound(trust_radius, "trust_radius")
        self.grad_norm = self.trust = None
        self.clipped = []
        if max_grad_norm is not None:
            self.clipped = [torch.empty_like(o) for o in self.out]
            self.grad_norm = torch.zeros(1, dtype=f32, device=dev)
        if trust_radius is not None:
            self.trust = torch.zeros(2, dtype=f32, device=dev)
        self.fisher = [torch.zeros(2, b.c, dtype=f32, device=dev) for b in self.bn_layers]
        self.bn_pre = [torch.empty(2, b.c, dtype=f32, device=dev) for b in self.bn_layers]
        self.in_code = K.KFAC_F16 if in_dtype == torch.float16 else K.KFAC_F32
        sizes = [K.kfac_factors_workspace(self.layers, self.in_code),
                 K.kfac_pack_sym_workspace(self.n_all),
                 K.kfac_invert_workspace(self.n_all),
                 K.kfac_precondition_workspace(self.d_g, self.d_a)]
        if self.refine:
            sizes.append(K.kfac_invert_refine_workspace(self.n_all))
        if self.bn_layers:
            sizes.append(K.kfac_bn_diag_workspace(self.bn_layers))
        if max_grad_norm is not None or trust_radius is not None:
            sizes.append(K.kfac_grad_norm_workspace([o.numel() for o in self.out] +
                                                    [f.numel() for f in self.fisher]))
        # one workspace serves every call on the caller's stream: they run one after
        # another; the second stream has its own
        self.workspace = torch.empty(max(sizes) + 256, dtype=torch.uint8, device=dev)
        self.stream2 = None
        if self.side:
            sub = lambda v, idx: [v[i] for i in idx]  # noqa: E731
            side_ws = max(K.kfac_invert_workspace(sub(self.n_all, self.side)),
                          K.kfac_precondition_workspace(sub(self.d_g, self.side_layers),
                                                        sub(self.d_a, self.side_layers)))
            self.workspace2 = torch.empty(side_ws + 256, dtype=torch.uint8, device=dev)
            self.stream2 = torch.cuda.Stream(device=dev)

    @property
    def info(self):
        """Breakdown index of every inverse (order of n_all: A factors, then G)."""
        out = torch.zeros(len(self.n_all), dtype=torch.int32, device=self.device)
        if self.main:
            out[self.main] = self._info_main
        if self.side:
            out[self.side] = self._info_side
        return out

    @property
    def A_inv(self):
        return self.full[:len(self.layers)]

    @property
    def G_inv(self):
        return self.full[len(self.layers):]

    def factors(self, act, gout, ema_decay=0.0, stream=None):
        act = self._factors_of_checkpoints(self.layers, act, act, None, ema_decay, stream)
        if any(t is not None for t in (*act, *gout)):
            K.kfac_factors(self.layers, act, gout, self.A_packed, self.G_packed, ema_decay,
                           self.workspace, stream)

    def _factors_of_checkpoints(self, layers, act, every, full, ema_decay, stream):
        """Forms the factors of the layers whose act is a Checkpoint; act without those. `every`: the step's, of which
        act may be a part."""
        if not any(isinstance(a, Checkpoint) for a in act):
            return act
        at = [l for l, a in enumerate(every) if isinstance(a, Checkpoint)]
        held = [every[l] for l in at]
        rows, cols, bias = [len(a) for a in held], [a.shape[1] for a in held], [layers[l].bias for l in at]
        self._room(K.kfac_factors_q8_workspace(rows, cols, bias), stream)
        K.kfac_factors_q8([a.q for a in held], [a.scale for a in held],
                          [self.A_packed[l] if act[l] is not None else None for l in at],
                          None if full is None else [full[l] if act[l] is not None else None for l in at], bias, ema_decay,
                          self.workspace, stream)
        return [None if isinstance(a, Checkpoint) else a for a in act]

    @staticmethod
    def _check_checkpoints(layers, act):
        for l, a in zip(layers, act):
            if isinstance(a, Checkpoint):
                if (l.h, l.w, l.kh, l.kw, l.h_out, l.w_out) != (1,) * 6 or tuple(a.shape) != (l.n, l.c_in):
                    raise ValueError("a Checkpoint is of a fully connected layer's [n, c_in] rows")

    def _make_room(self, layers, bn_layers, stream):
        """A workspace that also serves these layers, where they are not those of the step."""
        need = 0 if layers is self.layers else K.kfac_factors_workspace(layers, self.in_code)
        if bn_layers is not self.bn_layers and bn_layers:
            need = max(need, K.kfac_bn_diag_workspace(bn_layers))
        self._room(need, stream)

    def _room(self, need, stream):
        if self.workspace.numel() < need + 256:
            on = torch.cuda.current_stream(self.device) if stream is None else stream
            self.workspace.record_stream(on)  # calls in flight there use the old one
            with torch.cuda.stream(on):
                self.workspace = torch.empty(need + 256, dtype=torch.uint8, device=self.device)

    def _factors_full(self, layers, act, every, gout, ema_decay, stream):
        # the packed factors (the stored state) and the upper triangles that kfac_invert
        # reads, from the same kernels: no separate unpack pass
        L = len(self.layers)
        act = self._factors_of_checkpoints(layers, act, every, self.full[:L], ema_decay, stream)
        if all(t is None for t in (*act, *gout)):
            return
        K.kfac_factors_full(layers, act, gout, self.A_packed, self.G_packed, self.full[:L], self.full[L:],
                            ema_decay, self.workspace, stream)

    # With the second stream, the caller's stream forms its factors in 2 calls,
    # preconditions in 4 and runs the BatchNorm step in 2 (groups of layers of about
    # equal work). A pivot block of the long sweeps needs a whole compute unit, and while
    # a launch of many small blocks runs, the units it frees go to its own next blocks:
    # the pivot waits for the launch to drain (up to 0.3 ms behind one preconditioning
    # or BatchNorm launch). Shorter launches bound that wait; more calls cost more than
    # they save (measured: 6 preconditioning calls or 3 factor calls were slower).
    MAIN_CALLS = {"factors": 2, "precondition": 4, "bn": 2}

    @staticmethod
    def _groups(idx, cost, parts):
        """idx (in order) cut into at most `parts` runs of about equal summed cost."""
        total = sum(cost(i) for i in idx)
        out, cur, acc = [], [], 0.0
        for i in idx:
            cur.append(i)
            acc += cost(i)
            if len(out) < parts - 1 and acc >= total * (len(out) + 1) / parts:
                out.append(cur)
                cur = []
        if cur:
            out.append(cur)
        return out

    def _sub(self, v, idx):
        return [v[i] for i in idx]

    def _factor_cost(self, l):
        # products of a layer's two factors: rows x order^2, the 3x3 A factors at about a
        # third (formed from shift products)
        L = self.layers[l]
        rows = L.n * L.h_out * L.w_out
        return rows * (self.d_a[l] ** 2 / (3.0 if L.kh == 3 and L.sh == 1 else 1.0) + self.d_g[l] ** 2)

    def _factor_inputs(self, act, gout):
        """(act, gout) lists of the side matrices' factors and of all the others, with
        None where a factor is left to the other call."""
        L = len(self.layers)
        side = set(self.side)
        first = ([a if l in side else None for l, a in enumerate(act)],
                 [g if l + L in side else None for l, g in enumerate(gout)])
        rest = ([None if l in side else a for l, a in enumerate(act)],
                [None if l + L in side else g for l, g in enumerate(gout)])
        return first, rest

    def invert(self, stream=None):
        """Unpacks and inverts every damped factor on `stream` (the side split is
        applied by step())."""
        self._unpack(stream)
        self._invert(self.main, self._info_main, self.workspace, stream)
        if self.side:
            self._invert(self.side, self._info_side, self.workspace, stream)
        self._refine(stream)

    def _unpack(self, stream):
        # kfac_invert reads only the upper triangle: unpack that half
        K.kfac_pack_sym(self.n_all, self.full, self.packed_all, 2, self.workspace, stream)

    def _invert(self, idx, info, ws, stream):
        if idx:
            K.kfac_invert(self._sub(self.n_all, idx), self._sub(self.full, idx), self._sub(self.full, idx),
                          [self.shift] * len(idx), info, None, ws, stream)

    def _refine(self, stream):
        if self.refine:
            K.kfac_pack_sym(self.n_all, self.factor_full, self.packed_all, 1, self.workspace, stream)
            K.kfac_invert_refine(self.n_all, self.factor_full, [self.shift] * len(self.n_all), self.full,
                                 self.workspace, stream)

    def precondition(self, grads, weights=None, lr=0.0, stream=None):
        """self.out <- preconditioned gradients; with weights (fp32 [d_g, d_a] per layer)
        also weights -= lr * self.out, in the same kernel."""
        self._precondition(list(range(len(self.layers))), grads, weights, lr, self.workspace, stream)

    def _precondition(self, ls, grads, weights, lr, ws, stream):
        if not ls:
            return
        sub = self._sub
        d_g, d_a, G, A, g, o = (sub(self.d_g, ls), sub(self.d_a, ls), sub(self.G_inv, ls), sub(self.A_inv, ls),
                                sub(grads, ls), sub(self.out, ls))
        w = sub(weights, ls) if weights is not None else None
        if self.accum == K.KFAC_F64:
            K.kfac_precondition_ex(d_g, d_a, G, A, g, o, w, lr, self.accum, ws, stream)
        elif w is None:
            K.kfac_precondition(d_g, d_a, G, A, g, o, ws, stream)
        else:
            K.kfac_precondition_update(d_g, d_a, G, A, g, o, w, lr, ws, stream)

    def bn(self, xhat, bn_gout, ema_decay=0.0, bn_params=None, lr=0.0, stream=None):
        """BN Fisher and preconditioned gradients; with bn_params (fp32 [2, c]: gamma,
        beta) also bn_params -= lr * self.bn_pre."""
        self._bn(list(range(len(self.bn_layers))), self.bn_layers, xhat, bn_gout, ema_decay, bn_params, lr, stream)

    def _bn(self, idx, bn_layers, xhat, bn_gout, ema_decay, bn_params, lr, stream):
        if not idx:
            return
        sub = self._sub
        if bn_params is None:
            K.kfac_bn_diag(sub(bn_layers, idx), sub(xhat, idx), sub(bn_gout, idx), sub(self.fisher, idx),
                           sub(self.bn_pre, idx), ema_decay, self.bn_shift, self.workspace, stream)
        else:
            K.kfac_bn_update(sub(bn_layers, idx), sub(xhat, idx), sub(bn_gout, idx), sub(self.fisher, idx),
                             sub(self.bn_pre, idx), sub(bn_params, idx), lr, ema_decay, self.bn_shift,
                             self.workspace, stream)

    def clip(self, grads, stream=None):
        """The gradients to precondition: clipped by their global norm into self.clipped,
        or as they are without max_grad_norm."""
        if self.max_grad_norm is None:
            return grads
        K.kfac_grad_clip(grads, self.clipped, self.max_grad_norm, self.grad_norm, self.workspace, stream)
        return self.clipped

    def _bounded_update(self, grads, weights, bn_params, lr, stream):
        # every parameter that the step updates takes part in the bound
        P, g, w, fisher = [], [], [], []
        if weights is not None:
            P, g, w, fisher = list(self.out), list(grads), list(weights), [None] * len(self.out)
        if bn_params is not None:
            P, w = P + self.bn_pre, w + list(bn_params)
            g, fisher = g + [None] * len(self.bn_pre), fisher + self.fisher
        K.kfac_trust_update(P, g, w, lr, self.trust_radius, self.trust, fisher, self.bn_shift, self.workspace, stream)

    def step(self, act, gout, grads, xhat=(), bn_gout=(), ema_decay=0.0, refresh=True,
             weights=None, bn_params=None, lr=0.0, stream=None, layers=None, bn_layers=None,
             bn_fisher=None):
        """One step. refresh=False is a stale-curvature step: factors and inverses are
        kept, the gradients are preconditioned with them, and BN divides its fresh
        gradient by the stored Fisher (decay 1 keeps it). Given weights and/or
        bn_params, those are updated in place with learning rate lr. layers, bn_layers:
        those of this call where its tensors have another number of samples, n. bn_fisher:
        (bn_layers, xhat, gout) that the BatchNorm Fisher is formed from where that is not the
        loss's own gradient; xhat and bn_gout then give the gradient alone."""
        # refused here, before the factors and the Fisher have taken the batch in
        if self.trust_radius is not None and not 0.0 <= lr < math.inf:
            raise ValueError("lr must be finite and >= 0")
        layers = _same_but_samples(layers, self.layers, K.kfac_layer._fields_, "layers")
        bn_layers = _same_but_samples(bn_layers, self.bn_layers, K.kfac_bn._fields_, "bn_layers")
        if refresh:
            self._check_checkpoints(layers, act)
        self._make_room(layers, bn_layers, stream)
        if bn_fisher is not None:
            fisher_layers = _same_but_samples(bn_fisher[0], self.bn_layers, K.kfac_bn._fields_, "bn_layers")
            self._make_room(layers, fisher_layers, stream)
            bn_fisher = (fisher_layers, *bn_fisher[1:])
        grads = self.clip(grads, stream)
        args = (layers, bn_layers, act, gout, grads, xhat, bn_gout, bn_fisher, ema_decay, refresh)
        if self.trust_radius is not None:
            self._step(*args, None, None, lr, stream)
            self._bounded_update(grads, weights, bn_params, lr, stream)
        else:
            self._step(*args, weights, bn_params, lr, stream)

    def _bn_groups(self, groups, bn_layers, xhat, bn_gout, bn_fisher, ema_decay, bn_params, lr, stream):
        if bn_fisher is not None:  # the gradient that this divides is not the loss's: only its Fisher stays
            for part in groups:
                self._bn(part, *bn_fisher, ema_decay, None, lr, stream)
            ema_decay = 1.0
        for part in groups:
            self._bn(part, bn_layers, xhat, bn_gout, ema_decay, bn_params, lr, stream)

    def _step(self, layers, bn_layers, act, gout, grads, xhat, bn_gout, bn_fisher, ema_decay, refresh, weights,
              bn_params, lr, stream):
        all_bn = list(range(len(bn_layers)))
        if not refresh:
            self.precondition(grads, weights, lr, stream)
            self._bn(all_bn, bn_layers, xhat, bn_gout, 1.0, bn_params, lr, stream)
            return
        if not self.side:
            self._factors_full(layers, act, act, gout, ema_decay, stream)
            self._invert(self.main, self._info_main, self.workspace, stream)
            self._refine(stream)
            self.precondition(grads, weights, lr, stream)
            self._bn_groups([all_bn], bn_layers, xhat, bn_gout, bn_fisher, ema_decay, bn_params, lr, stream)
            return
        main = torch.cuda.current_stream(self.device) if stream is None else stream
        side = self.stream2
        # the long sweeps' factors first, so that their inverses start while the other
        # factors are formed (a factor call plans its row splits over every layer,
        # whichever inputs it is given: the same bits as one call)
        first, rest = self._factor_inputs(act, gout)
        self._factors_full(layers, first[0], act, first[1], ema_decay, main)
        formed = torch.cuda.Event()
        formed.record(main)
        side.wait_event(formed)
        try:
            self._invert(self.side, self._info_side, self.workspace2, side)
            lay = [l for l in range(len(self.layers)) if rest[0][l] is not None or rest[1][l] is not None]
            for part in self._groups(lay, self._factor_cost, self.MAIN_CALLS["factors"]):
                ps = set(part)
                self._factors_full(layers, [a if l in ps else None for l, a in enumerate(rest[0])], act,
                                   [g if l in ps else None for l, g in enumerate(rest[1])], ema_decay,
                                   main)
            self._invert(self.main, self._info_main, self.workspace, main)
            main_inverses = torch.cuda.Event()
            main_inverses.record(main)
            pcost = lambda l: self.d_g[l] * self.d_a[l] * (self.d_g[l] + self.d_a[l])  # noqa: E731
            for part in self._groups(self.main_layers, pcost, self.MAIN_CALLS["precondition"]):
                self._precondition(part, grads, weights, lr, self.workspace, main)
            bcost = lambda b: self.bn_layers[b].n * self.bn_layers[b].hw * self.bn_layers[b].c  # noqa: E731
            self._bn_groups(self._groups(all_bn, bcost, self.MAIN_CALLS["bn"]), bn_layers, xhat, bn_gout, bn_fisher,
                            ema_decay, bn_params, lr, main)
            side.wait_event(main_inverses)  # the side layers' other factor
            self._precondition(self.side_layers, grads, weights, lr, self.workspace2, side)
        finally:
            # whatever was issued on the second stream is ordered before the caller's
            # later work, also when a call above raised
            joined = torch.cuda.Event()
            joined.record(side)
            main.wait_event(joined)
