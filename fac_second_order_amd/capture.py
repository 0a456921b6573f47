"""Stage 1-2 capture from a network's own forward and backward passes.

Osawa et al. (CVPR 2019), Figure 1 and Section 3: K-FAC takes each layer's input
activations in the forward pass and the gradients at its outputs in the backward
pass, forms the Kronecker factors from them (eq. 5), and updates the parameters with
the preconditioned gradients (eq. 7-8); BatchNorm uses the diagonal Fisher. This
module wires a PyTorch model to the library: hooks hand each convolution's and the
classifier's input and output gradient, and each BatchNorm's normalised input and
output gradient, to KfacStep in the layouts of include/kfac.h. PyTorch runs the
network (forward, backward, loss); every K-FAC number is computed by libkfac. For a
policy, whose rows of logits score the choice that was made, the loss and its gradient
at the logits are the library's too (policy_backward, preference_backward), and the
factors are formed from a backward pass of their own.

Layout conventions (the library's):
  * activations and output gradients NHWC fp16; a convolution weight [c_out, c_in,
    kh, kw] is the K-FAC matrix [c_out, (i*kw + j)*c_in + ci] (plus a last bias
    column for the classifier);
  * the loss is a batch mean, so the gradient a hook sees is 1/n of the per-sample
    gradient; it is multiplied by n on capture (the factor G is a per-sample second
    moment, eq. 5, and the BatchNorm Fisher is over per-sample gradients);
  * after policy_backward or preference_backward that does not hold: a row's gradient
    carries its advantage, its clip and its weight. Their factors take the gradients of
    log p(y), y drawn from the model at every row that counts (eq. 3, the Fisher), with
    coefficient 1; rows that do not count are in neither factor.
"""
import copy
import math
import threading
import types
from dataclasses import dataclass

import torch
import torch.nn as nn

from . import _lib as K
from . import checkpoint as ck
from .step import KfacStep


# ---------------------------------------------------------------------------
# ResNet-50 (He et al., 2016), v1 layout: the stride of a downsampling bottleneck
# sits on its first 1x1 convolution and on the projection.
# ---------------------------------------------------------------------------

class Bottleneck(nn.Module):
    def __init__(self, c_in, width, c_out, stride):
        super().__init__()
        self.c1 = nn.Conv2d(c_in, width, 1, stride, 0, bias=False)
        self.b1 = nn.BatchNorm2d(width)
        self.c2 = nn.Conv2d(width, width, 3, 1, 1, bias=False)
        self.b2 = nn.BatchNorm2d(width)
        self.c3 = nn.Conv2d(width, c_out, 1, 1, 0, bias=False)
        self.b3 = nn.BatchNorm2d(c_out)
        self.proj = None
        if stride != 1 or c_in != c_out:
            self.proj = nn.Conv2d(c_in, c_out, 1, stride, 0, bias=False)
            self.bp = nn.BatchNorm2d(c_out)
        self.act = nn.ReLU()

    def forward(self, x):
        y = self.act(self.b1(self.c1(x)))
        y = self.act(self.b2(self.c2(y)))
        y = self.b3(self.c3(y))
        s = self.bp(self.proj(x)) if self.proj is not None else x
        return self.act(y + s)

    def kfac_modules(self):
        """(conv, its BatchNorm) in the order the layers are numbered."""
        out = [(self.c1, self.b1), (self.c2, self.b2), (self.c3, self.b3)]
        if self.proj is not None:
            out.append((self.proj, self.bp))
        return out


class ResNet50(nn.Module):
    def __init__(self, classes=1000):
        super().__init__()
        self.conv1 = nn.Conv2d(3, 64, 7, 2, 3, bias=False)
        self.bn1 = nn.BatchNorm2d(64)
        self.act = nn.ReLU()
        self.pool = nn.MaxPool2d(3, 2, 1)
        blocks = []
        c = 64
        for n_blocks, width, c_out, stride in [(3, 64, 256, 1), (4, 128, 512, 2), (6, 256, 1024, 2),
                                               (3, 512, 2048, 2)]:
            for b in range(n_blocks):
                blocks.append(Bottleneck(c, width, c_out, stride if b == 0 else 1))
                c = c_out
        self.blocks = nn.Sequential(*blocks)
        self.fc = nn.Linear(2048, classes)

    def forward(self, x):
        x = self.pool(self.act(self.bn1(self.conv1(x))))
        x = self.blocks(x)
        return self.fc(torch.flatten(x.mean((2, 3)), 1))

    def kfac_modules(self):
        """Convolutions (with their BatchNorm) and the classifier (BatchNorm None), in
        forward order: conv1, then per bottleneck c1, c2, c3 and the projection."""
        out = [(self.conv1, self.bn1)]
        for blk in self.blocks:
            out.extend(blk.kfac_modules())
        out.append((self.fc, None))
        return out


# ---------------------------------------------------------------------------
# capture
# ---------------------------------------------------------------------------

@dataclass(frozen=True)
class LayerGeom:
    """The kfac_layer fields of one captured layer."""
    n: int
    h: int
    w: int
    c_in: int
    h_out: int
    w_out: int
    c_out: int
    kh: int
    kw: int
    sh: int
    sw: int
    ph: int
    pw: int
    bias: int


@dataclass(frozen=True)
class BnGeom:
    n: int
    hw: int
    c: int


def _nhwc_half(x):
    """[n, c, h, w] (any memory format) or [n, c] -> contiguous NHWC fp16."""
    if x.dim() == 2:
        return x.detach().to(torch.float16).contiguous()
    return x.detach().permute(0, 2, 3, 1).to(torch.float16).contiguous()


class _Taken:
    """The forward of a fully connected layer while a capture has it: `run`, which keeps the layer's
    input, or is `before`, what the layer itself was given for a forward (None: nothing). A copy of the layer has what
    the layer had before: the capture is not the copy's."""

    def __init__(self, layer, before, run):
        self.layer, self.before, self.run = layer, before, run
        self.calling = threading.local()

    def note(self):
        """A pre-hook of the layer: whose forward is about to be called. A shallow copy (a replica) has this very one."""
        def hook(mod, args):
            if mod.__dict__.get("forward") is self:
                self.calling.layer = mod
        return hook

    def __call__(self, *args, **kwargs):
        layer, self.calling.layer = getattr(self.calling, "layer", None), None
        if layer is None or layer is self.layer or self.before is not None:
            return self.run(*args, **kwargs)
        return type(layer).forward(layer, *args, **kwargs)

    def __deepcopy__(self, memo):
        if self.before is not None:
            return copy.deepcopy(self.before, memo)
        layer = copy.deepcopy(self.layer, memo)  # that of the copy, where it is the layer that is being copied
        return types.MethodType(type(layer).forward, layer)


class KfacCapture:
    """K-FAC for a model whose `kfac_modules()` lists (Conv2d or Linear, BatchNorm2d
    or None) pairs. Call `step(lr)` after `loss.backward()`: it forms the factors
    from the captured tensors, inverts them (every `refresh`-th call), preconditions
    the weight gradients and updates the weights and the BatchNorm parameters in
    place (eq. 8) through libkfac. precond_accum and refine_inverse are passed to
    KfacStep: "f64" sums the preconditioning products in fp64, refine_inverse takes
    one fp64-residual refinement step of every inverse. A real gradient lies in the
    range of its layer's factors, so where a factor is rank-deficient (batch smaller
    than its order) and the damping small, the preconditioning products cancel and
    amplify the inverses' fp32 error; the two options remove most of it. max_grad_norm
    and trust_radius are passed to KfacStep too: they bound the layers' weight gradients
    before those are preconditioned (BatchNorm's are not clipped), and the step that is
    taken. After policy_backward or preference_backward,
    whose factors are the model's Fisher, trust_radius bounds its predicted KL divergence
    (the mean over the rows that count, to second order and as far as the Kronecker factors
    hold); after another loss's backward pass it bounds the quadratic form of that loss's
    second moment.

    checkpoint="int8": the fully connected layers keep their input rows in 8 bits (Checkpoint),
    for autograd and the step together, instead of the input itself for autograd and, where that is no
    fp16, a copy in fp16 for the step. What else keeps the input decides what is saved: four layers of
    4096 with 8192 rows hold 384 MiB after the forward pass instead of 768 in bf16 behind GELUs, and instead
    of 576 behind ReLUs, which keep their outputs; in fp16 instead of 512 behind GELUs, but of 320 behind
    ReLUs, where the option costs memory. Their weight
    gradients and factors are those of the values that are kept (a row's error is at most
    1/127 of its largest entry), their outputs and the gradients at their inputs are what they were.
    matmul="int8", with it: their products are formed in 8-bit integers too (kfac_linear_q8), with
    a scale for each row and each output, also in passes without gradients; the gradients at their inputs
    take the weights as they are. Both are of layers whose product is nn.Linear's: one with a forward of its
    own, its class's or set on it, runs that, and its input is kept as without them."""

    def __init__(self, model, damping=1e-3, ema_decay=0.95, refresh_every=1, precond_accum="f32",
                 refine_inverse=False, max_grad_norm=None, trust_radius=None, checkpoint=None, matmul=None):
        if checkpoint not in (None, "int8") or matmul not in (None, "int8"):
            raise ValueError("checkpoint and matmul must be None or 'int8'")
        if matmul and not checkpoint:
            raise ValueError("matmul='int8' needs checkpoint='int8': the quantised input is the checkpoint")
        self.model = model
        self.precond_accum = precond_accum
        self.refine_inverse = bool(refine_inverse)
        self.max_grad_norm, self.trust_radius = max_grad_norm, trust_radius
        self.pairs = list(model.kfac_modules())
        self.damping = damping
        self.ema_decay = ema_decay
        self.refresh_every = refresh_every
        self.n = 0
        self.act = [None] * len(self.pairs)
        self.gout = [None] * len(self.pairs)
        self.bns = [bn for _, bn in self.pairs if bn is not None]
        self.xhat = [None] * len(self.bns)
        self.bgout = [None] * len(self.bns)
        # the gradients of the drawn tokens' log-probabilities, while a pass takes them what it
        # multiplies them by, and which samples hold one that counts
        self.score = [None] * len(self.pairs)
        self.bscore = [None] * len(self.bns)
        self.score_scale = self.counted = None
        # of a running backward pass: what its gradients are multiplied by, and if it is one behind a score pass
        self.loss_scale, self.own_loss = 1.0, False
        self.kstep = None
        self.calls = 0
        self.hooks = []
        # checkpoints that a layer's running forward pass has made, until its hook takes them
        self.made, self.int8 = {}, matmul == "int8"
        self.wrapped = []
        for i, (m, _) in enumerate(self.pairs):
            if checkpoint and isinstance(m, nn.Linear) and type(m).forward is nn.Linear.forward:
                before = m.__dict__.get("forward")
                plain = getattr(m.forward, "__func__", None) is nn.Linear.forward and m.forward.__self__ is m
                self.wrapped.append((m, before))
                m.forward = _Taken(m, None if plain else before, self._checkpointed(i, m) if plain else before)
                self.hooks.append(m.register_forward_pre_hook(m.forward.note()))
            self.hooks.append(m.register_forward_hook(self._fwd(i)))
            self.hooks.append(m.register_full_backward_hook(self._bwd(i)))
        for i, bn in enumerate(self.bns):
            self.hooks.append(bn.register_forward_hook(self._bn_fwd(i)))
            self.hooks.append(bn.register_full_backward_hook(self._bn_bwd(i)))

    def remove(self):
        for h in self.hooks:
            h.remove()
        self.hooks = []
        for m, before in self.wrapped:
            if before is None:
                del m.forward
            else:
                m.forward = before
        self.wrapped = []

    # layers that keep their input in 8 bits ------------------------------------
    def _checkpointed(self, i, m):
        def forward(input):
            if torch.is_grad_enabled():
                y, self.made[i] = ck.linear(input, m.weight, m.bias, self.int8)
                return y
            return ck.linear(input, m.weight, m.bias, True)[0] if self.int8 else nn.functional.linear(input, m.weight, m.bias)
        return forward

    # hooks: a copy of the model has them too, and its passes are not the capture's -------
    def _fwd(self, i):
        def hook(mod, inp, out):
            if mod is self.pairs[i][0] and torch.is_grad_enabled():
                self.n = inp[0].shape[0]
                made = self.made.pop(i, None)
                self.act[i] = _nhwc_half(inp[0]) if made is None else made
        return hook

    def _bwd(self, i):
        def hook(mod, grad_in, grad_out):
            if mod is not self.pairs[i][0]:
                return
            g = grad_out[0]
            if self.score_scale is None:
                self.gout[i] = _nhwc_half(g * (self.n / self.loss_scale))
                if not self.own_loss:
                    self.score[i] = None
                return
            # a convolution's Fisher is the sum over its positions, which its factors average
            places = math.sqrt(g.shape[2] * g.shape[3]) if g.dim() == 4 else 1.0
            self.score[i] = _nhwc_half(g.float() * (self.score_scale * places))
        return hook

    def _bn_fwd(self, i):
        def hook(mod, inp, out):
            if mod is self.bns[i] and torch.is_grad_enabled():
                x = inp[0].detach().float()
                var, mean = torch.var_mean(x, dim=(0, 2, 3), unbiased=False, keepdim=True)
                xh = (x - mean) * torch.rsqrt(var + mod.eps)
                self.xhat[i] = xh.permute(0, 2, 3, 1).reshape(x.shape[0], -1, x.shape[1]).to(
                    torch.float16).contiguous()
        return hook

    def _bn_bwd(self, i):
        def hook(mod, grad_in, grad_out):
            if mod is not self.bns[i]:
                return
            if self.score_scale is None:
                to, g = self.bgout, grad_out[0] * (self.n / self.loss_scale)
                if not self.own_loss:
                    self.bscore[i] = None
            else:
                to, g = self.bscore, grad_out[0].float() * self.score_scale
            to[i] = g.permute(0, 2, 3, 1).reshape(g.shape[0], -1, g.shape[1]).to(torch.float16).contiguous()
        return hook

    # geometry and parameter layouts -------------------------------------------
    def _layers_of(self, *tensors):
        """Layers of (act, gout, xhat, bgout) for a call; (None, None) where they are those the step was made for."""
        return (None, None) if [t.shape for ts in tensors for t in ts] == self.shapes else self._geometry(*tensors)

    def _geometry(self, act=None, gout=None, xhat=None, bgout=None):
        """Layers of captured tensors, of the last passes' if none are given."""
        if act is None:
            act, gout, xhat, bgout = self.act, self.gout, self.xhat, self.bgout
        layers = []
        for a, g in (*zip(act, gout), *zip(xhat, bgout)):
            if a.shape[0] != g.shape[0]:
                raise RuntimeError("the last forward and the last backward pass are of different batches")
        for (m, _), a, g in zip(self.pairs, act, gout):
            if isinstance(m, nn.Conv2d):
                n, h, w, c_in = a.shape
                _, h_out, w_out, c_out = g.shape
                layers.append(LayerGeom(n, h, w, c_in, h_out, w_out, c_out, m.kernel_size[0], m.kernel_size[1],
                                        m.stride[0], m.stride[1], m.padding[0], m.padding[1],
                                        1 if m.bias is not None else 0))
            else:
                n, c_in = a.shape
                layers.append(LayerGeom(n, 1, 1, c_in, 1, 1, g.shape[1], 1, 1, 1, 1, 0, 0,
                                        1 if m.bias is not None else 0))
        bns = [BnGeom(x.shape[0], x.shape[1], x.shape[2]) for x in xhat]
        return layers, bns

    @staticmethod
    def _to_matrix(m, grad=False):
        w = m.weight.grad if grad else m.weight.data
        if isinstance(m, nn.Conv2d):
            mat = w.permute(0, 2, 3, 1).reshape(w.shape[0], -1)
        else:
            mat = w
        if m.bias is not None:
            b = m.bias.grad if grad else m.bias.data
            mat = torch.cat([mat, b[:, None]], 1)
        return mat.float().contiguous()

    @staticmethod
    def _from_matrix(m, mat):
        if m.bias is not None:
            m.bias.data.copy_(mat[:, -1])
            mat = mat[:, :-1]
        elif mat.data_ptr() == m.weight.data_ptr():
            return  # a weight whose memory has the matrix's order: _to_matrix gave it itself
        if isinstance(m, nn.Conv2d):
            c_out, c_in, kh, kw = m.weight.shape
            m.weight.data.copy_(mat.reshape(c_out, kh, kw, c_in).permute(0, 3, 1, 2))
        else:
            m.weight.data.copy_(mat)

    # losses over the model's logits ----------------------------------------------
    @staticmethod
    def _logit_rows(logits):
        """[..., vocab] logits as rows for the library, and a gradient of their size."""
        z = logits.detach().reshape(-1, logits.shape[-1])
        if z.stride(1) != 1 or (z.shape[0] > 1 and z.stride(0) < z.shape[1]):
            z = z.contiguous()
        return z, torch.zeros(z.shape, dtype=z.dtype, device=z.device)

    @staticmethod
    def _row_counts(z, token, mask, seq_begin):
        """Which rows count, as the losses decide it."""
        token = token.reshape(-1)
        counts = (token >= 0) & (token < z.shape[1])
        if mask is not None:
            counts &= mask.reshape(-1) != 0
        if seq_begin is not None:
            at = torch.arange(z.shape[0], device=z.device)
            counts &= (at >= seq_begin[0]) & (at < seq_begin[-1])
        return counts

    @staticmethod
    def _draw(z):
        """A token for every row from the model's distribution: the largest of z - log e, with
        exponential numbers e."""
        e = torch.empty(z.shape, dtype=torch.float32, device=z.device).exponential_().log_()
        return torch.sub(z, e, out=e).argmax(1)

    @staticmethod
    def _leaves(out):
        """The leaves that a backward pass from `out` reaches."""
        seen, todo, found = set(), [out.grad_fn], []
        while todo:
            fn = todo.pop()
            if fn is None or fn in seen:
                continue
            seen.add(fn)
            if type(fn).__name__ == "AccumulateGrad":
                found.append(fn.variable)
            todo.extend(f for f, _ in fn.next_functions)
        return found

    def _score_pass(self, logits, z, counts):
        """A backward pass of log p(y) of the rows that count, with coefficient 1 and y drawn from
        the model: self.score and self.bscore. No leaf's gradient changes."""
        leaves = self._leaves(logits)
        if not leaves:
            return
        rows = z.shape[0]
        y, d = self._draw(z), torch.empty(z.shape, dtype=z.dtype, device=z.device)
        one, logp, unused = (torch.ones(rows, dtype=torch.float32, device=z.device) for _ in range(3))
        stats = torch.empty(4, dtype=torch.float32, device=z.device)
        # -1 for the advantage, and l itself for the old log-probability: the loss is -(-r) with r = 1 and
        # nothing to clip it below, its gradient that of l; rows / counted at a row
        K.kfac_policy_loss(z, y, one, one, logp, stats, mask=counts)
        K.kfac_policy_loss(z, y, logp, -one, unused, stats, dlogits=d, mask=counts, clip_low=1.0, clip_high=0.0,
                           grad_scale=float(rows))
        # the samples that hold the rows: the model's inputs in their order, or else all of them
        whole = self.n > 0 and rows % self.n == 0
        samples = counts.view(self.n, rows // self.n).any(1) if whole else torch.ones(self.n, dtype=torch.bool, device=z.device)
        # times counted / rows a row's score has coefficient 1; a factor divides by the samples that hold
        # one that counts, where the mean over the rows divides by the rows
        scale = (counts.sum() * samples.sum()).float().sqrt() / max(rows, 1)
        self.counted = (samples.to("cpu", non_blocking=True), torch.cuda.Event() if z.is_cuda else None)
        if z.is_cuda:
            self.counted[1].record()
        self.score_scale = scale
        try:
            torch.autograd.grad(logits, leaves, d.view(logits.shape), retain_graph=True)
        finally:
            self.score_scale = None

    @staticmethod
    def _scale(given, z, x):
        """grad_scale: the one given, or 1, or for fp16 logits the largest power of two up to x, from 1 to 2^14
        (a coefficient of 4 times that is still an fp16)."""
        if given is not None:
            if not 0.0 < given < math.inf:
                raise ValueError("grad_scale must be positive and finite")
            return float(given)
        return 2.0 ** min(14, math.floor(math.log2(x))) if z.dtype == torch.float16 and x >= 1 else 1.0

    def _backward(self, logits, z, d, counts, scale):
        """The backward pass of a loss whose gradient at the logits is d / scale, behind the one that the factors
        of the next step are formed from, if it forms any."""
        self.score, self.bscore = [None] * len(self.score), [None] * len(self.bscore)
        if self.calls % self.refresh_every == 0:
            self._score_pass(logits, z, counts)
        held = [] if scale == 1.0 else [(p, p.grad) for p in self._leaves(logits)]
        for p, _ in held:
            p.grad = None
        self.loss_scale, self.own_loss = scale, True
        try:
            logits.backward(d.view(logits.shape))
        finally:
            self.loss_scale, self.own_loss = 1.0, False
            for p, before in held:
                if p.grad is not None:
                    p.grad.div_(scale)
                p.grad = before if p.grad is None else p.grad if before is None else before.add_(p.grad)

    def policy_backward(self, logits, token, old_logp, advantage, ref_logp=None, mask=None, seq_begin=None,
                        by_sequence=False, clip_low=0.2, clip_high=0.2, kl_coef=0.0, grad_scale=None):
        """Backward pass of the clipped policy loss with a KL term (kfac_policy_loss) over
        the model's logits [..., vocab], one token, old log-probability and advantage for
        each row, the rows those of the model's inputs in their order. The factors of the next
        step come from a second backward pass through the same graph (torch's generator
        draws its tokens), which the leaves' gradients do not see, but hooks on tensors and retained
        gradients do. The gradients run through the network multiplied by grad_scale, which is
        divided out of what arrives at the leaves and the hooks: by default 1, and for fp16 logits the rows'
        number, as a power of two up to 2^14, since a mean over rows leaves most of a softmax below what an
        fp16 holds. Returns (stats, logp): the loss, its surrogate part, the mean KL and the clipped share; the
        rows' log-probabilities."""
        z, d = self._logit_rows(logits)
        scale = self._scale(grad_scale, z, z.shape[0])
        logp = torch.zeros(z.shape[0], dtype=torch.float32, device=z.device)
        stats = torch.zeros(4, dtype=torch.float32, device=z.device)
        K.kfac_policy_loss(z, token, old_logp, advantage, logp, stats, dlogits=d, ref_logp=ref_logp, mask=mask,
                           seq_begin=seq_begin, by_sequence=by_sequence, clip_low=clip_low, clip_high=clip_high,
                           kl_coef=kl_coef, grad_scale=scale)
        self._backward(logits, z, d, self._row_counts(z, token, mask, seq_begin), scale)
        return stats, logp

    def preference_backward(self, logits, token, seq_begin, ref_logp=None, mask=None, beta=0.1, label_smoothing=0.0,
                            grad_scale=None):
        """Backward pass of the preference loss (kfac_preference_loss) over the model's
        logits [..., vocab], whose rows are the preferred sequences and then the others, and a
        second one for the factors; grad_scale as in policy_backward, for fp16 logits about
        pairs / beta by default, which makes a row's coefficient 1. Returns (loss, margin, seq_logp)."""
        z, d = self._logit_rows(logits)
        pairs = seq_begin.numel() // 2
        scale = self._scale(grad_scale, z, pairs / abs(beta) if beta else 1.0)
        seq_logp, margin, loss = (torch.zeros(n, dtype=torch.float32, device=z.device) for n in (2 * pairs, pairs, 1))
        K.kfac_preference_loss(z, token, seq_begin, seq_logp, margin, loss, dlogits=d, ref_logp=ref_logp, mask=mask,
                               beta=beta, label_smoothing=label_smoothing, grad_scale=scale)
        self._backward(logits, z, d, self._row_counts(z, token, mask, seq_begin), scale)
        return loss, margin, seq_logp

    # the K-FAC step -------------------------------------------------------------
    def _curvature(self):
        """What a step forms its factors from, (act, gout, xhat, BatchNorm gout): of the layers that a score pass
        reached its tensors of the samples that count, of the others the loss's; None where no sample counts."""
        taken = tuple(list(ts) for ts in (self.act, self.gout, self.xhat, self.bgout))
        if all(g is None for g in (*self.score, *self.bscore)):
            return taken
        host, copied = self.counted
        if copied is not None:
            copied.synchronize()
        kept = host.nonzero()[:, 0]
        if not len(kept):
            return None
        some = kept.to(self.act[0].device) if len(kept) < len(host) else None
        for ins, outs, scores in ((taken[0], taken[1], self.score), (taken[2], taken[3], self.bscore)):
            for i, g in enumerate(scores):
                if g is None:
                    continue
                outs[i] = g
                if some is not None and len(g) == len(ins[i]) == len(host):
                    ins[i], outs[i] = ins[i].index_select(0, some), g.index_select(0, some)
        return taken

    def step(self, lr):
        if any(a is None for a in self.act) or any(g is None for g in self.gout):
            raise RuntimeError("step() needs one forward and backward pass with the hooks in place")
        dev = self.act[0].device
        passes = self.act, self.gout, self.xhat, self.bgout
        if self.kstep is None:
            layers, bns = self._geometry()
            self.shapes = [t.shape for ts in passes for t in ts]
            self.kstep = KfacStep(layers, bns, dev, damping=self.damping, precond_accum=self.precond_accum,
                                  refine_inverse=self.refine_inverse, max_grad_norm=self.max_grad_norm,
                                  trust_radius=self.trust_radius)
            self.master = [self._to_matrix(m) for m, _ in self.pairs]
            self.bn_master = [torch.stack([bn.weight.data.float(), bn.bias.data.float()]).contiguous()
                              for bn in self.bns]
        grads = [self._to_matrix(m, grad=True) for m, _ in self.pairs]
        refresh = self.calls % self.refresh_every == 0
        decay = 0.0 if self.calls == 0 else self.ema_decay
        act, gout, bn_fisher = self.act, self.gout, None
        layers, bns = self._layers_of(*passes)
        if refresh:
            taken = self._curvature()
            if taken is None and self.calls:  # no row counts: there is no curvature in the batch
                refresh = False
            elif taken is not None:
                act, gout, xhat, bgout = taken
                layers, fisher_bns = self._layers_of(*taken)
                if any(g is not None for g in self.bscore):
                    bn_fisher = (fisher_bns, xhat, bgout)
        self.kstep.step(act, gout, grads, self.xhat, self.bgout, ema_decay=decay, refresh=refresh,
                        weights=self.master, bn_params=self.bn_master, lr=lr, layers=layers, bn_layers=bns,
                        bn_fisher=bn_fisher)
        self.calls += 1
        for (m, _), mat in zip(self.pairs, self.master):
            self._from_matrix(m, mat)
        for bn, p in zip(self.bns, self.bn_master):
            bn.weight.data.copy_(p[0])
            bn.bias.data.copy_(p[1])
