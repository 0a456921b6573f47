"""Plain fp64 definitions of the losses over logits, the gradient norm with clipping
and the update bounded by its predicted KL divergence.

TEST INFRASTRUCTURE ONLY, as ``kfac_oracle``: NumPy, row by row, from the formulas of
include/kfac.h, sharing no code with the HIP library. Inputs are the exact values of
the arrays that the library was given. Pinned in ``tests/test_loss_oracle.py`` by
central differences, closed forms and invariants.
"""
import math

import numpy as np

__all__ = ["row_logp", "policy_loss", "preference_loss", "global_norm", "clip_scale", "trust_step"]


def row_logp(z, y):
    """(log-probability of y, softmax) of one row of logits."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max()
    e = np.exp(z - m)
    s = e.sum()
    return (z[y] - m) - math.log(s), e / s


def _spans(rows, begin):
    return [(0, rows)] if begin is None else list(zip(begin[:-1], begin[1:]))


def _counts(token, mask, t, vocab):
    return (mask is None or bool(mask[t])) and 0 <= token[t] < vocab


def policy_loss(z, token, old, adv, ref=None, mask=None, begin=None, by_sequence=False, low=0.2, high=0.2,
                kl_coef=0.0, scale=1.0):
    """stats (loss, surrogate part, KL, clipped share), logp and dlogits; rows outside
    every sequence are NaN in both."""
    rows, vocab = z.shape
    logp = np.full(rows, np.nan)
    grad = np.full((rows, vocab), np.nan)
    spans = _spans(rows, begin)
    kept = [[t for t in range(a, b) if _counts(token, mask, t, vocab)] for a, b in spans]
    full = sum(1 for k in kept if k)
    total = sum(len(k) for k in kept)
    part = kl = over = 0.0
    for (a, b), k in zip(spans, kept):
        logp[a:b], grad[a:b] = 0.0, 0.0
        for t in k:
            weight = 1.0 / (full * len(k)) if by_sequence else 1.0 / total
            l, p = row_logp(z[t], token[t])
            r, A = math.exp(l - old[t]), float(adv[t])
            held = min(max(r, 1.0 - low), 1.0 + high) * A
            part -= weight * min(r * A, held)
            slope = 0.0 if r * A > held else -r * A
            over += weight if r * A > held else 0.0
            if ref is not None:
                d = float(ref[t]) - l
                kl += weight * (math.expm1(d) - d if d < math.inf else d)
                slope -= kl_coef * math.expm1(d) if kl_coef else 0.0
            logp[t] = l
            one = np.zeros(vocab)
            one[token[t]] = 1.0
            grad[t] = scale * weight * slope * (one - p)
    return np.array([part + (kl_coef * kl if kl_coef else 0.0), part, kl, over]), logp, grad


def _softplus(x):
    return max(x, 0.0) + math.log1p(math.exp(-abs(x)))


def preference_loss(z, token, begin, ref=None, mask=None, beta=0.1, smooth=0.0, scale=1.0):
    """loss, margins, sequence sums and dlogits (NaN outside every sequence)."""
    rows, vocab = z.shape
    spans = _spans(rows, begin)
    pairs = len(spans) // 2
    grad = np.full((rows, vocab), np.nan)
    probs, sums = {}, []
    for a, b in spans:
        grad[a:b] = 0.0
        ls = []
        for t in range(a, b):
            if _counts(token, mask, t, vocab):
                l, probs[t] = row_logp(z[t], token[t])
                ls.append(l)
        sums.append(math.fsum(ls))
    ref = [0.0] * (2 * pairs) if ref is None else [float(v) for v in ref]
    x = [beta * ((sums[i] - ref[i]) - (sums[pairs + i] - ref[pairs + i])) for i in range(pairs)]
    loss = sum(share * _softplus(v) for x_i in x for share, v in ((1 - smooth, -x_i), (smooth, x_i)) if share)
    loss = loss / pairs if pairs else 0.0
    for i in range(pairs):
        slope = (smooth - math.exp(-_softplus(x[i]))) * beta / pairs
        for s, sign in ((i, 1.0), (pairs + i, -1.0)):
            for t in range(*spans[s]):
                if t in probs:
                    one = np.zeros(vocab)
                    one[token[t]] = 1.0
                    grad[t] = scale * sign * slope * (one - probs[t])
    return loss, np.array(x), np.array(sums), grad


def global_norm(tensors):
    return math.sqrt(math.fsum(float((np.asarray(t, dtype=np.float64).ravel() ** 2).sum()) for t in tensors))


def clip_scale(norm, max_norm):
    return max_norm / norm if math.isfinite(norm) and norm > max_norm else 1.0


def trust_step(P, g, lr, delta, fisher=None, shift=0.0):
    """(step, q): g[i] None takes P (fisher + shift) for the gradient."""
    q = 0.0
    for i, p in enumerate(P):
        p = np.asarray(p, dtype=np.float64).ravel()
        gi = p * (np.asarray(fisher[i], dtype=np.float64).ravel() + shift) if g[i] is None else \
            np.asarray(g[i], dtype=np.float64).ravel()
        q += float(p @ gi)
    return (lr if q == 0 else min(lr, math.sqrt(2 * delta / abs(q)))), q
