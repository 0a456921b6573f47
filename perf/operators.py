"""What is measured of the operators around a K-FAC step: the policy and preference
losses over a model's logits with their gradients, the global gradient norm with
clipping, and the update whose length is bounded by its predicted KL divergence.

`run` computes them from elementary torch operations, or, with `own` set, through the
package's entry points. Formulas, with z the logits of a row, y its token, l = z[y] -
log sum exp z, p = softmax z:

  clip    norm = sqrt(sum of g^2 over all tensors); out = g * min(1, max_norm / norm)
  trust   q = sum of P * g over all tensors (g = P * (F + shift) where the Fisher is
          diagonal); w <- w - min(lr, sqrt(2 delta / |q|)) * P
  policy  r = exp(l - old), d = ref - l: sum of weight * (-min(r A, clip(r) A) +
          kl (exp(d) - d - 1)), and its gradient in the logits
  prefer  x = beta ((L_c - R_c) - (L_r - R_r)), L the sum of l over a sequence: mean of
          (1 - e) softplus(-x) + e softplus(x), and its gradient in the logits
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the weight gradients of ResNet-50 in their K-FAC matrix form, before preconditioning
        {"name": "clip resnet50 f32", "op": "clip", "set": "resnet50", "width": 0, "ffn": 0, "depth": 0, "vocab": 0,
         "type": "f32", "out": "f32", "packed": False, "clip": True},
        # one perceptron's gradients: the call's own cost
        {"name": "norm mlp f32", "op": "clip", "set": "mlp", "width": 64, "ffn": 0, "depth": 3, "vocab": 0,
         "type": "f32", "out": "f32", "packed": False, "clip": False},
        # a decoder's bf16 gradients with f32 gains, widened to the f32 that preconditioning reads
        {"name": "clip decoder bf16", "op": "clip", "set": "decoder", "width": 2048, "ffn": 8192, "depth": 12,
         "vocab": 32768, "type": "bf16", "out": "f32", "packed": False, "clip": True},
        # the step of ResNet-50 with its BatchNorm parameters
        {"name": "trust resnet50 f32", "op": "trust", "set": "resnet50", "width": 0, "ffn": 0, "depth": 0, "vocab": 0,
         "type": "f32", "packed": False},
        # a small policy's step, f16 gradients
        {"name": "trust mlp f16", "op": "trust", "set": "mlp", "width": 64, "ffn": 0, "depth": 3, "vocab": 0,
         "type": "f16", "packed": False},
        # a batch of decisions among the 1000 outputs of ResNet-50's classifier
        {"name": "policy 256x1000 f32", "op": "policy", "rows": 256, "vocab": 1000, "pad": 0, "type": "f32",
         "seqs": 0, "by_seq": False, "kl": 0.0, "grad": True},
        # a batch of answers to prompts, averaged by answer, held near a reference
        {"name": "policy 2048x32000 bf16", "op": "policy", "rows": 2048, "vocab": 32000, "pad": 0, "type": "bf16",
         "seqs": 8, "by_seq": True, "kl": 0.04, "grad": True},
        # long answers over a large vocabulary
        {"name": "policy 4096x131072 bf16", "op": "policy", "rows": 4096, "vocab": 131072, "pad": 0, "type": "bf16",
         "seqs": 4, "by_seq": False, "kl": 0.04, "grad": True},
        # a few single tokens, an odd vocabulary
        {"name": "policy 4x50001 f16", "op": "policy", "rows": 4, "vocab": 50001, "pad": 0, "type": "f16",
         "seqs": 0, "by_seq": False, "kl": 0.04, "grad": True},
        # two pairs of short answers
        {"name": "prefer 48x1000 f32", "op": "prefer", "rows": 48, "vocab": 1000, "pad": 0, "type": "f32",
         "seqs": 4, "smooth": 0.0, "grad": True},
        # eight pairs of answers to prompts
        {"name": "prefer 2048x32000 bf16", "op": "prefer", "rows": 2048, "vocab": 32000, "pad": 0, "type": "bf16",
         "seqs": 16, "smooth": 0.1, "grad": True},
        # four pairs of long answers, an odd vocabulary in rows of a padded head
        {"name": "prefer 4096x50001 f16", "op": "prefer", "rows": 4096, "vocab": 50001, "pad": 47, "type": "f16",
         "seqs": 8, "smooth": 0.0, "grad": True},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["clip", "trust", "policy", "policy", "prefer", "prefer"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("clip", "trust"):
        if op == "trust":
            kind = rng.choice(["f32", "f16"])
        if rng.random() < 0.5:
            case = {"op": op, "set": "mlp", "width": _between(rng, 8, 4096), "ffn": 0, "depth": rng.randint(1, 8),
                    "vocab": 0}
        else:
            width = _between(rng, 96, 1536)
            case = {"op": op, "set": "decoder", "width": width, "ffn": rng.randint(2 * width, 4 * width),
                    "depth": rng.randint(1, 12), "vocab": _between(rng, 500, 40000)}
        case.update({"type": kind, "packed": rng.random() < 0.3})
        if op == "clip":
            case.update({"out": rng.choice([kind, "f32"]), "clip": rng.random() < 0.8})
        return case
    vocab = _between(rng, 2, 131072)
    rows = _between(rng, 4 if op == "prefer" else 1, 4096)
    case = {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, 0, 1, 24]), "type": kind,
            "grad": rng.random() < 0.8}
    if BYTES[kind] * rows * (vocab + case["pad"]) * (2 if op == "prefer" else 1) > 2 * 4096 * 131072:
        case["rows"] = rows = max(4, rows // 4)
    if op == "policy":
        seqs = rng.choice([0, min(rows, _between(rng, 1, 64))])
        case.update({"seqs": seqs, "by_seq": seqs > 0 and rng.random() < 0.5, "kl": rng.choice([0.0, 0.04, 0.2])})
    else:
        case.update({"seqs": 2 * min(rows // 2, _between(rng, 1, 32)), "smooth": rng.choice([0.0, 0.1])})
    return case


# ---------------------------------------------------------------------------
# layouts
# ---------------------------------------------------------------------------

def _resnet50():
    """(order of G, order of A with its bias column) of the 53 convolutions and the classifier."""
    stages = [(3, 64, 64, 256), (4, 256, 128, 512), (6, 512, 256, 1024), (3, 1024, 512, 2048)]
    shapes = [(64, 3 * 49 + 1)]
    for blocks, c_in, width, c_out in stages:
        for b in range(blocks):
            shapes += [(width, (c_in if b == 0 else c_out) + 1), (width, 9 * width + 1), (c_out, width + 1)]
            shapes += [(c_out, c_in + 1)] if b == 0 else []
    return shapes + [(1000, 2049)]


def _shapes(case):
    """Shapes of the tensors, and for each whether it is a gain kept in f32."""
    w, f = case["width"], case["ffn"]
    if case["set"] == "resnet50":
        return [(s, False) for s in _resnet50()]
    if case["set"] == "mlp":
        return [((w, w + 1), False)] * case["depth"] + [((16, w + 1), False)]
    layer = [((w,), True), ((w, w), False), ((w // 4, w), False), ((w // 4, w), False), ((w, w), False), ((w,), True),
             ((f, w), False), ((f, w), False), ((w, f), False)]
    return [((case["vocab"], w), False)] + layer * case["depth"] + [((w,), True), ((case["vocab"], w), False)]


def _views(shapes, kinds, packed, device):
    """One zeroed buffer for each type and its views: every tensor begins at a multiple of 64
    elements, or right behind the one before it."""
    used, where = {}, []
    for shape, kind in zip(shapes, kinds):
        n = math.prod(shape)
        at = used.get(kind, 0)
        where.append((kind, at, n))
        used[kind] = at + (n if packed else -(-n // 64) * 64)
    flat = {k: torch.zeros(n, dtype=TYPES[k], device=device) for k, n in used.items()}
    return flat, [flat[k][at:at + n].view(s) for (k, at, n), s in zip(where, shapes)]


def _lengths(rows, seqs):
    """Ragged lengths of `seqs` sequences over about 31/32 of `rows`; with 8 or more of them, one is empty."""
    share = [0 if seqs >= 8 and i == 3 else 1 + (5 * i + 2) % 7 for i in range(seqs)]
    used = rows - rows // 32
    ends = [used * sum(share[:i + 1]) // sum(share) for i in range(seqs)]
    return [e - b for b, e in zip([0] + ends, ends)]


def _prompt(length, i):
    """How many leading rows of sequence i are a prompt, which the mask takes out; all of every fifth."""
    return length if i % 5 == 4 else length // 4


def _counted(case):
    """(rows in sequences, rows that count)."""
    if not case["seqs"]:
        return case["rows"], case["rows"]
    ls = _lengths(case["rows"], case["seqs"])
    return sum(ls), sum(n - _prompt(n, i) for i, n in enumerate(ls))


def work(case):
    if case["op"] in ("clip", "trust"):
        sizes = [(math.prod(s), "f32" if gain else case["type"]) for s, gain in _shapes(case)]
        n = sum(k for k, _ in sizes)
        read = sum(k * BYTES[t] for k, t in sizes)
        if case["op"] == "trust":
            bn = 2 * sum(g for g, _ in _resnet50()[:-1]) if case["set"] == "resnet50" else 0
            return {"bytes": read + 12 * n + 16 * bn, "flops": 4 * n + 6 * bn}
        wide = sum(k * (4 if case["out"] == "f32" else BYTES[t]) for k, t in sizes) if case["clip"] else 0
        return {"bytes": read + wide, "flops": 2 * n + (n if case["clip"] else 0)}
    inside, counted = _counted(case)
    size = BYTES[case["type"]] * case["vocab"]
    grad = 1 if case["grad"] else 0
    return {"bytes": size * (counted + grad * inside) + 32 * case["rows"],
            "flops": case["vocab"] * counted * (4 + 4 * grad)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] in ("clip", "trust"):
        shapes, gains = zip(*_shapes(case))
        kinds = ["f32" if k else case["type"] for k in gains]
        s["flat"], s["grad"] = _views(shapes, kinds, case["packed"], dev)
        if case["op"] == "clip":
            for i, t in enumerate(s["grad"]):
                t.copy_(normal(*t.shape) * (0.002 * (1 + i % 5)))
            outs = ["f32" if case["out"] == "f32" else k for k in kinds]
            s["out_flat"], s["out"] = _views(shapes, outs, case["packed"], dev)
            s["max_norm"] = 1.0 if sum(t.numel() for t in s["grad"]) > 250000 else 0.05
            s["norm"] = torch.zeros(1, device=dev)
            s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device=dev)
            return s
        f32 = ["f32"] * len(shapes)
        bn = [(2, c) for c, _ in _resnet50()[:-1]] if case["set"] == "resnet50" else []
        s["p_flat"], s["p"] = _views(list(shapes) + bn, f32 + ["f32"] * len(bn), case["packed"], dev)
        s["w_flat"], s["w"] = _views(list(shapes) + bn, f32 + ["f32"] * len(bn), case["packed"], dev)
        s["f_flat"], s["fisher"] = _views(bn, ["f32"] * len(bn), False, dev) if bn else ({}, [])
        for p, w in zip(s["p"], s["w"]):
            p.copy_(normal(*p.shape) * 0.02)
            w.copy_(normal(*w.shape) * 0.05)
        for p, t in zip(s["p"], s["grad"]):  # the Fisher's block is positive: P and g point the same way
            t.copy_(p * (normal(*t.shape) * 0.3 + 1) * 0.01)
        for t in s["fisher"]:
            t.copy_(normal(*t.shape).square() * 0.01)
        s["grad"] = s["grad"] + [None] * len(bn)
        s["fisher"] = [None] * len(shapes) + s["fisher"]
        s["shift"], s["lr"], s["delta"] = 1e-3, 0.1, 1e-3
        if sum(t.numel() for t in s["p"]) < 250000:
            s["delta"] = 1e-7
        s["step"] = torch.zeros(2, device=dev)
        s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device=dev)
        return s

    rows, vocab = case["rows"], case["vocab"]
    kind = TYPES[case["type"]]
    z = torch.empty(rows, vocab + case["pad"], dtype=kind, device=dev)
    s["token"] = torch.randint(0, vocab, (rows,), generator=g, device=dev)
    logp = torch.empty(rows, device=dev)
    for a in range(0, rows, 256):  # a model's scores: the token that was taken stands out
        part = normal(z[a:a + 256].shape[0], z.shape[1]) * 2.5
        part.scatter_add_(1, s["token"][a:a + 256, None], normal(part.shape[0], 1) * 2 + 6)
        z[a:a + 256] = part.to(kind)
        part = z[a:a + 256, :vocab].float()
        logp[a:a + 256] = part.gather(1, s["token"][a:a + 256, None])[:, 0] - torch.logsumexp(part, 1)
    s["logits"] = z[:, :vocab]
    s["dlogits"] = torch.zeros(rows, vocab, dtype=kind, device=dev) if case["grad"] else None
    s["begin"], s["mask"] = None, None
    lengths = _lengths(rows, case["seqs"]) if case["seqs"] else []
    if lengths:
        s["begin"] = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=dev)
        keep = [j >= _prompt(n, i) for i, n in enumerate(lengths) for j in range(n)]
        s["mask"] = torch.tensor(keep + [True] * (rows - len(keep)), device=dev)
    if case["op"] == "policy":
        s["old"] = logp + 0.2 * normal(rows)
        s["ref"] = logp + 0.3 * normal(rows) if case["kl"] else None
        s["advantage"] = normal(rows)
        s["logp"] = torch.zeros(rows, device=dev)
        s["stats"] = torch.zeros(4, device=dev)
    else:
        lp = (logp * s["mask"]).double()
        s["ref"] = torch.stack([lp[a:a + n].sum() for a, n in zip(s["begin"].tolist(), lengths)]).float()
        s["ref"] += 3 * normal(len(lengths))
        s["seq_logp"] = torch.zeros(len(lengths), device=dev)
        s["margin"] = torch.zeros(len(lengths) // 2, device=dev)
        s["loss"] = torch.zeros(1, device=dev)
    s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device=dev)
    return s


LOW, HIGH, BETA = 0.2, 0.28, 0.1


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _scores(s):
    """Probabilities of every row in f32 and the log-probability of its token in f64."""
    z = s["logits"].float()
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    picked = z.gather(1, s["token"][:, None])
    return e / total, ((picked - top).double() - total.double().log())[:, 0]


def _place(s):
    """For every row its sequence, whether it lies in one, and whether it counts."""
    rows = s["logits"].shape[0]
    at = torch.arange(rows, device=s["logits"].device)
    if s["begin"] is None:
        inside = at >= 0
        return at * 0, inside, inside if s["mask"] is None else s["mask"]
    begin = s["begin"].long()
    seq = (at[:, None] >= begin[None, 1:]).sum(1)
    inside = (at >= begin[0]) & (seq < begin.numel() - 1)
    return seq.clamp(max=begin.numel() - 2), inside, inside & s["mask"]


def _gradient(s, p, coef):
    """coef * (one-hot of the token - p), a row each, into the rows' own type."""
    d = -p
    d.scatter_add_(1, s["token"][:, None], torch.ones_like(coef)[:, None].float())
    return (d * coef.float()[:, None]).to(s["logits"].dtype)


def _plain_policy(s):
    case = s["case"]
    p, logp = _scores(s)
    seq, inside, counted = _place(s)
    n = counted.double()
    if case["by_seq"]:
        per = torch.zeros(s["begin"].numel() - 1, dtype=torch.float64, device=n.device).index_add_(0, seq, n)
        weight = n / (per[seq].clamp(min=1) * (per > 0).sum().clamp(min=1))
    else:
        weight = n / n.sum().clamp(min=1)
    zero = torch.zeros_like(logp)
    ratio = torch.where(counted, logp - s["old"], zero).exp()
    a = torch.where(counted, s["advantage"].double(), zero)
    plain, held = ratio * a, ratio.clamp(1 - LOW, 1 + HIGH) * a
    over = plain > held
    part = (weight * -torch.minimum(plain, held)).sum()
    slope = torch.where(over, zero, -plain)
    kl = torch.zeros_like(part)
    if case["kl"]:
        d = torch.where(counted, s["ref"] - logp, zero)
        kl = (weight * (d.expm1() - d)).sum()
        slope = slope - case["kl"] * d.expm1()
    stats = torch.stack([part + case["kl"] * kl, part, kl, (weight * over).sum()]).float()
    out = {"stats": stats, "logp": torch.where(counted, logp, zero).float()}
    if case["grad"]:
        out["dlogits"] = _gradient(s, p, case["rows"] * weight * slope)
    return out


def _plain_prefer(s):
    case = s["case"]
    p, logp = _scores(s)
    seq, inside, counted = _place(s)
    pairs = s["margin"].numel()
    sums = torch.zeros(2 * pairs, dtype=torch.float64, device=logp.device)
    sums.index_add_(0, seq, torch.where(counted, logp, torch.zeros_like(logp)))
    gain = sums - s["ref"].double()
    x = BETA * (gain[:pairs] - gain[pairs:])
    e = case["smooth"]
    # softplus(-x) = max(-x, 0) + log(1 + exp(-|x|)), softplus(x) = softplus(-x) + x
    soft = (-x).clamp(min=0) + (-x.abs()).exp().log1p()
    loss = ((1 - e) * soft + e * (soft + x)).mean()
    slope = (e - 1 / (1 + x.exp())) * BETA / pairs  # e sig(x) - (1 - e) sig(-x) = e - sig(-x)
    out = {"loss": loss.float().view(1), "margin": x.float(), "seq_logp": sums.float()}
    if case["grad"]:
        out["dlogits"] = _gradient(s, p, case["rows"] * torch.cat([slope, -slope])[seq] * counted)
    return out


def _plain_clip(s):
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grad"]]).sum().sqrt()
    out = {"norm": norm.float().view(1)}
    if s["case"]["clip"]:
        coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
        [o.copy_(t.float() * coef) for o, t in zip(s["out"], s["grad"])]
        out.update(s["out_flat"])
    return out


def _plain_trust(s):
    def dot(p, t, f):
        return (p * (p * (f + s["shift"]) if t is None else t.float())).sum(dtype=torch.float64)

    q = torch.stack([dot(p, t, f) for p, t, f in zip(s["p"], s["grad"], s["fisher"])]).sum()
    step = (2 * s["delta"] / q.abs()).sqrt().clamp(max=s["lr"])
    [w.sub_(p * step.float()) for w, p in zip(s["w"], s["p"])]
    return {"step": torch.stack([step, q]).float(), "w": s["w_flat"]["f32"]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import fac_second_order_amd as kfac
    case, ws = s["case"], s["workspace"]
    if case["op"] == "clip":
        if not case["clip"]:
            kfac.kfac_grad_norm(s["grad"], s["norm"], workspace=ws)
            return {"norm": s["norm"]}
        kfac.kfac_grad_clip(s["grad"], s["out"], s["max_norm"], s["norm"], workspace=ws)
        return {"norm": s["norm"], **s["out_flat"]}
    if case["op"] == "trust":
        kfac.kfac_trust_update(s["p"], s["grad"], s["w"], s["lr"], s["delta"], s["step"], fisher=s["fisher"],
                               shift=s["shift"], workspace=ws)
        return {"step": s["step"], "w": s["w_flat"]["f32"]}
    if case["op"] == "policy":
        kfac.kfac_policy_loss(s["logits"], s["token"], s["old"], s["advantage"], s["logp"], s["stats"],
                              dlogits=s["dlogits"], ref_logp=s["ref"], mask=s["mask"], seq_begin=s["begin"],
                              by_sequence=case["by_seq"], clip_low=LOW, clip_high=HIGH, kl_coef=case["kl"],
                              grad_scale=float(case["rows"]), workspace=ws)
        out = {"stats": s["stats"], "logp": s["logp"]}
    else:
        kfac.kfac_preference_loss(s["logits"], s["token"], s["begin"], s["seq_logp"], s["margin"], s["loss"],
                                  dlogits=s["dlogits"], ref_logp=s["ref"], mask=s["mask"], beta=BETA,
                                  label_smoothing=case["smooth"], grad_scale=float(case["rows"]), workspace=ws)
        out = {"loss": s["loss"], "margin": s["margin"], "seq_logp": s["seq_logp"]}
    if case["grad"]:
        out["dlogits"] = s["dlogits"]
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"clip": _plain_clip, "trust": _plain_trust, "policy": _plain_policy, "prefer": _plain_prefer}[op](state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grad"]))
        out = {"norm": torch.tensor([norm], dtype=torch.float64)}
        if case["clip"]:
            scale = min(1.0, s["max_norm"] / norm)
            kinds = ["f32" if o.dtype == torch.float32 else case["type"] for o in s["out"]]
            for kind in s["out_flat"]:
                flat = torch.zeros(s["out_flat"][kind].numel(), dtype=torch.float64, device="cuda")
                for t, o, k in zip(s["grad"], s["out"], kinds):
                    if k == kind:
                        a = o.storage_offset()
                        flat[a:a + o.numel()] = t.double().view(-1) * scale
                out[kind] = flat
        return out
    if case["op"] == "trust":
        q = 0.0
        for p, t, f in zip(s["p"], s["grad"], s["fisher"]):
            p = p.double().view(-1)
            q += float(p @ (p * (f.double().view(-1) + s["shift"]) if t is None else t.double().view(-1)))
        step = min(s["lr"], math.sqrt(2 * s["delta"] / abs(q)))
        w = s["w_flat"]["f32"].double() - step * s["p_flat"]["f32"].double()
        return {"step": torch.tensor([step, q], dtype=torch.float64), "w": w}

    rows, vocab = s["logits"].shape
    spans = [(0, rows)]
    if s["begin"] is not None:
        ends = s["begin"].tolist()
        spans = list(zip(ends[:-1], ends[1:]))
    keep = [True] * rows if s["mask"] is None else s["mask"].tolist()
    owner = [None] * rows
    for i, (a, b) in enumerate(spans):
        for t in range(a, b):
            owner[t] = i if keep[t] else None
    logp = torch.empty(rows, dtype=torch.float64)
    chunk = max(1, (1 << 27) // vocab)
    for a in range(0, rows, chunk):
        part = torch.log_softmax(s["logits"][a:a + chunk].double(), 1)
        logp[a:a + chunk] = part.gather(1, s["token"][a:a + chunk, None])[:, 0].cpu()
    lp, slope = logp.tolist(), [0.0] * rows
    sizes = [sum(owner[t] == i for t in range(a, b)) for i, (a, b) in enumerate(spans)]
    if case["op"] == "policy":
        old, adv = s["old"].double().tolist(), s["advantage"].double().tolist()
        ref = s["ref"].double().tolist() if case["kl"] else lp
        full = sum(n > 0 for n in sizes)
        part, kl, over, shown = 0.0, 0.0, 0.0, [0.0] * rows
        for t in range(rows):
            if owner[t] is None:
                continue
            weight = 1 / (full * sizes[owner[t]]) if case["by_seq"] else 1 / sum(sizes)
            r, d = math.exp(lp[t] - old[t]), ref[t] - lp[t]
            held = min(max(r, 1 - LOW), 1 + HIGH)
            part -= weight * min(r * adv[t], held * adv[t])
            kl += weight * (math.expm1(d) - d)
            slope[t] = -case["kl"] * math.expm1(d)
            if r * adv[t] > held * adv[t]:
                over += weight
            else:
                slope[t] -= r * adv[t]
            slope[t] *= weight * rows
            shown[t] = lp[t]
        kl = kl if case["kl"] else 0.0
        out = {"stats": torch.tensor([part + case["kl"] * kl, part, kl, over], dtype=torch.float64),
               "logp": torch.tensor(shown, dtype=torch.float64)}
    else:
        pairs = len(spans) // 2
        sums = [math.fsum(lp[t] for t in range(a, b) if owner[t] == i) for i, (a, b) in enumerate(spans)]
        gain = [v - r for v, r in zip(sums, s["ref"].double().tolist())]
        x = [BETA * (gain[i] - gain[pairs + i]) for i in range(pairs)]
        e, loss = case["smooth"], 0.0
        for i in range(pairs):
            below, above = (math.log1p(math.exp(-abs(x[i]))) + max(v, 0.0) for v in (-x[i], x[i]))
            loss += ((1 - e) * below + e * above) / pairs
            rise = math.exp(-above)  # sig(-x)
            for k, sign in ((i, 1), (pairs + i, -1)):
                for t in range(*spans[k]):
                    if owner[t] is not None:
                        slope[t] = sign * BETA / pairs * rows * (e * math.exp(-below) - (1 - e) * rise)
        out = {"loss": torch.tensor([loss], dtype=torch.float64), "margin": torch.tensor(x, dtype=torch.float64),
               "seq_logp": torch.tensor(sums, dtype=torch.float64)}
    if case["grad"]:
        full = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
        coef = torch.tensor(slope, dtype=torch.float64, device="cuda")[:, None]
        for a in range(0, rows, chunk):
            part = torch.softmax(s["logits"][a:a + chunk].double(), 1).mul_(-1)
            part.scatter_add_(1, s["token"][a:a + chunk, None], torch.ones_like(part[:, :1]))
            full[a:a + chunk] = part * coef[a:a + chunk]
        out["dlogits"] = full
    return out
