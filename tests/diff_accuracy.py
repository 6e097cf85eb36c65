"""What differential attention's outputs are off by on average, beside the bounds on
each component of tests/diff_reference.py.

A rounding to bf16 is off by at most half a step, 2^-8 of the value, and by a 1 / sqrt 3
of that on average; roundings of different values are independent.  So with y the output,
x = O1 - lambda O2 and f what the norm and the scale multiply x by, the mean square of
the error is at most
    (2^-8)^2 / 3 y^2                                        the output's own rounding
    + f^2 sum_j lambda_j^2 (2^-8)^2 / 3 sum_t p_jt^2 v_t^2  one bf16 term a probability
                                                            (two: 2^-16 in place of 2^-8)
(the norm takes out of an error what lies along x, which only lowers it), and to its root
come the fp32 steps of f (|O1| + |lambda O2|), each as far off as its bound at the worst."""
import math

import torch

from tests import diff_reference as dr

MARGIN = 1.25     # of the mean over some thousand components from what is expected of it


def expected(q, keys, values, seen, scale, lam, weight, eps, out_scale, by_head, terms):
    """Arguments as diff_reference.pairs: (out, bound of each component for this many
    terms, bound of the error's root mean square over all components)."""
    out, tol = dr.pairs(q, keys, values, seen, scale, lam, weight, eps, out_scale, by_head, terms)
    m, hq, d = q.shape
    hkv, n = keys.shape[:2]
    per = hq // hkv
    square, steps = torch.zeros_like(out), torch.zeros_like(out)
    late = torch.arange(n, device=q.device)[None, :] >= seen[:, None]
    for h in range(hq // 2):
        g = h // per
        v = torch.cat([values[2 * g], values[2 * g + 1]], dim=1).double()
        o, p2 = [], []
        worst = 0.0
        for j in range(2):
            k = (keys[(2 * h + j) // per] if by_head else keys[2 * g + j]).double()
            at = q[:, 2 * h + j].double()
            p = torch.softmax((at @ k.T * scale).masked_fill(late, -math.inf), dim=1)
            o.append(p @ v)
            p2.append(p.square() @ v.square())
            size = (at.abs() @ k.abs().T * abs(scale)).masked_fill(late, 0.0).amax()
            worst = max(worst, float(2 * (size * (d / 16 * dr.MMA + 2.0 ** -23) + 2.0 ** -22)
                                     + terms * (n / 16 + 1) * dr.MMA + 2.0 ** -20))
        a = abs(float(lam[h]))
        x = o[0] - float(lam[h]) * o[1]
        f = torch.full_like(x, abs(out_scale))
        if weight is not None:
            f = f * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + eps) * weight.double().abs()
        unit = (2.0 ** -8 if terms == 1 else 2.0 ** -16) ** 2 / 3
        square[:, h] = f.square() * unit * (p2[0] + a * a * p2[1])
        steps[:, h] = f * worst * (o[0].abs() + a * o[1].abs())
    square += (2.0 ** -8) ** 2 / 3 * out.square()
    return out, tol, float(MARGIN * square.mean().sqrt() + steps.square().mean().sqrt())


def check(got, q, keys, values, seen, scale, lam, weight, eps, out_scale, by_head, terms, what):
    want, tol, rms = expected(q, keys, values, seen, scale, lam, weight, eps, out_scale, by_head, terms)
    dr.check(got, want, tol, what)
    err = float((got.double() - want).square().mean().sqrt())
    assert err <= rms, f"{what}: off by {err:.3g} on average, expected at most {rms:.3g}"
