"""Inputs and derived error bounds of the GPU tests of the losses over logits.

u = 2^-24 is half a step of fp32. The library forms, for a row of logits z with maximum m,
e_j = exp2((z_j - m) log2 e): the difference and the product are rounded once each and the
constant once, so the exponent is off by at most 2.5 u |z_j - m|, and the exponential by one
step (2 u) more. The sum of the e_j, formed by at least 64 lanes and then joined over at most
40 partial sums with a rescaling each, is off by u (vocab / 64 + 40) from its additions,
and by 2.5 u |z_j - m| for its terms and as much again for the rescalings. Terms further
than 40 below the maximum weigh e^-40 and are not felt. So with spread = min(max - min, 40)

    |error of log sum| <= err_l = u (vocab / 64 + 40 + 6 spread),

and l itself, formed in fp64 from there, has no other error until it is rounded to fp32.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half the distance of the smallest subnormals
FLOOR = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def host64(t):
    return t.detach().double().cpu().numpy()


def row_errors(z):
    """err_l of every row."""
    out = []
    for row in z:
        fin = row[np.isfinite(row)]
        spread = min(float(fin.max() - fin.min()), 40.0) if fin.size else 0.0
        out.append(U * (z.shape[1] / 64 + 40 + 6 * spread))
    return np.array(out)


def softmax_rows(z):
    with np.errstate(invalid="ignore"):
        e = np.exp(z - z.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def grad_bound(ref, z, token, coef, coef_err, err_l, dtype):
    """Bound of |dlogits - ref|: p is off by 2 err_l of itself, the coefficient by coef_err, the
    fp32 operations by 3 u, and the result is rounded once to its type."""
    p = softmax_rows(z)
    one = np.zeros_like(p)
    ok = (token >= 0) & (token < z.shape[1])
    one[np.nonzero(ok)[0], token[ok]] = 1
    return (np.abs(coef)[:, None] * p * 2 * err_l[:, None] + coef_err[:, None] * np.abs(one - p)
            + np.abs(ref) * (3 * U + HALF_STEP[dtype]) * 1.01 + FLOOR[dtype])


def logits(seed, rows, vocab, dtype, pad=0, offset=0, std=2.0, device="cuda"):
    """[rows, vocab] view at a pitch of vocab + pad, `offset` elements into its buffer, and tokens."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    ld = vocab + pad
    flat = torch.randn(offset + rows * ld, generator=g) * std
    z = flat.to(dtype).to(device)[offset:].view(rows, ld)[:, :vocab]
    return z, torch.randint(0, vocab, (rows,), generator=g).to(device), g
