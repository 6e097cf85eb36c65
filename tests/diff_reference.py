"""Differential attention in 64 bits, one query pair at a time, and what the
kernels' outputs may be off from it.

With A_j = sum_t p_jt |v_t| (the map's average of |v|) and S = sum_i |q_i k_i| of a
key, the errors are, relative to A_j:
  logits    MMA steps of 16 products in fp32, d / 16 of them, each off by at most 17
            truncations of 2^-23 of what it has summed: e_s = scale * max S * (d / 16) *
            17 * 2^-23, once in p's numerator and once in the denominator
  2^x       2^-22, and the product with scale * log2 e 2^-23 of the logit, both twice
  P.V       n / 16 steps for each of `terms` bf16 terms, 17 * 2^-23 each
  p         two terms: a remainder of 2^-8 rounded to 2^-8 of itself, 2^-16.  One term:
            2^-8 of each p, independent from key to key, so sum_t p_t e_t v_t is beyond
            7 * 2^-8 sqrt(sum_t p_t^2 v_t^2) once in 10^10 (Hoeffding: 2 exp(-7^2 / 2))
x = O1 - lambda O2 is then off by E = E1 + |lambda| E2; the norm's factor r by r rms(E)
relative, the rest of the fp32 steps by 2^-20, and out is rounded to bf16: 2^-8.
"""
import math

import torch

MMA = 17 * 2.0 ** -23


def pairs(q, keys, values, lens, scale, lam, weight, eps, out_scale, by_head, terms):
    """q [m][hq][d], keys and values [hkv][n][d], row i sees the first lens[i] of the n:
    (out [m][hq / 2][2 d], tolerance of the same shape), fp64."""
    m, hq, d = q.shape
    hkv, n = keys.shape[:2]
    per = hq // hkv
    q, keys, values = q.double(), keys.double(), values.double()
    lam = lam.double()
    weight = weight.double() if weight is not None else None
    out = torch.zeros((m, hq // 2, 2 * d), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    if n == 0:
        return out, tol
    seen = torch.arange(n, device=q.device)[None, :] < lens[:, None]
    for h in range(hq // 2):
        group = h // per
        v = torch.cat([values[2 * group], values[2 * group + 1]], dim=1)
        x, E = torch.zeros_like(out[:, 0]), torch.zeros_like(out[:, 0])
        for j in range(2):
            i = 2 * h + j
            k = keys[i // per] if by_head else keys[2 * group + j]
            logit = (q[:, i] @ k.T * scale).masked_fill(~seen, -math.inf)
            top = logit.amax(dim=1, keepdim=True)
            p = torch.exp(logit - torch.where(torch.isinf(top), 0.0, top))
            total = p.sum(dim=1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)
            size = (q[:, i].abs() @ k.abs().T * scale).masked_fill(~seen, 0.0).amax(dim=1)
            rel = 2 * (size * (d / 16 * MMA + 2.0 ** -23) + 2.0 ** -22) + terms * (n / 16 + 1) * MMA + 2.0 ** -16
            e = rel[:, None] * (p @ v.abs())
            if terms == 1:
                e = e + 7 * 2.0 ** -8 * torch.sqrt(p.square() @ v.square())
            sign = 1.0 if j == 0 else -float(lam[h])
            x += sign * (p @ v)
            E += abs(sign) * e
        y, bound = x * out_scale, E * abs(out_scale)
        if weight is not None:
            r = torch.rsqrt(x.square().mean(dim=1, keepdim=True) + eps)
            rms = torch.sqrt(E.square().mean(dim=1, keepdim=True))
            y = x * r * weight * out_scale
            bound = (r * weight.abs() * (E + x.abs() * r * rms)) * abs(out_scale)
        out[:, h] = y
        tol[:, h] = bound * (1 + 2.0 ** -8) + (2.0 ** -8 + 2.0 ** -20) * y.abs() + 1e-30
    return out, tol


def check(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst by {float((err - tol).max()):.3g}, "
                           f"first at {bad.nonzero()[0].tolist()}")
