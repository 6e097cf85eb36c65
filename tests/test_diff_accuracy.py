"""The bounds that differential attention is held to find what they are there for: the
definition rounded to bf16 passes, and every mistake planted in the definition (on the
CPU) fails."""
import math

import pytest
import torch

from tests import diff_accuracy as da
from tests import diff_reference as dr


def inputs(n, m, d, hq, hkv, rho, lam, norm, seed=0):
    """m rows over up to n keys; the two maps' queries correlated by rho, on equal keys."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    k, v, q = rand(hkv, n, d), rand(hkv, n, d).bfloat16(), 2 * rand(m, hq, d)
    if rho:
        k[1::2] = k[0::2]
        q[:, 1::2] = rho * q[:, 0::2] + math.sqrt(1 - rho * rho) * q[:, 1::2]
    weight = 1 + 0.2 * rand(2 * d) if norm else None
    return dict(q=q.bfloat16(), keys=k.bfloat16(), values=v, seen=n - m + 1 + torch.arange(m), scale=d ** -0.5,
                lam=torch.full((hq // 2,), lam), weight=weight, eps=1e-5, out_scale=0.2 if norm else 1.0, by_head=False)


def definition(x, **other):
    a = dict(x, **other)
    return dr.pairs(a["q"], a["keys"], a["values"], a["seen"], a["scale"], a["lam"], a["weight"], a["eps"],
                    a["out_scale"], a["by_head"], 2)[0]


def rounded_maps(x):
    """The definition with each probability rounded to bf16 once (its sum is not)."""
    q, k, v, lam = x["q"].double(), x["keys"].double(), x["values"].double(), x["lam"].double()
    per = q.shape[1] // k.shape[0]
    late = torch.arange(k.shape[1])[None, :] >= x["seen"][:, None]
    out = []
    for h in range(q.shape[1] // 2):
        g, o = h // per, []
        for j in range(2):
            s = (q[:, 2 * h + j] @ k[2 * g + j].T * x["scale"]).masked_fill(late, -math.inf)
            p = torch.exp(s - s.amax(dim=1, keepdim=True))
            o.append(p.bfloat16().double() @ torch.cat([v[2 * g], v[2 * g + 1]], dim=1) / p.sum(dim=1, keepdim=True))
        y = o[0] - lam[h] * o[1]
        if x["weight"] is not None:
            y = y * torch.rsqrt(y.square().mean(dim=1, keepdim=True) + x["eps"]) * x["weight"].double()
        out.append(y * x["out_scale"])
    return torch.stack(out, dim=1)


SHAPES = [(1, 1), (6, 6), (40, 40), (340, 40)]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("terms", [1, 2])
@pytest.mark.parametrize("rho,lam", [(0.0, 0.5), (0.99, 0.8), (0.999, 1.0)])
@pytest.mark.parametrize("n,m", SHAPES)
def test_the_definition_passes(n, m, rho, lam, terms, norm):
    x = inputs(n, m, 64, 4, 2, rho, lam, norm)
    da.check(definition(x).bfloat16(), **x, terms=terms, what=f"{n} keys")
    if terms == 1:
        da.check(rounded_maps(x).bfloat16(), **x, terms=1, what=f"{n} keys, rounded maps")


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("terms", [1, 2])
@pytest.mark.parametrize("n,m", SHAPES[1:])
def test_wrong_weights_and_scales_fail(n, m, terms, norm):
    x = inputs(n, m, 64, 4, 2, 0.0, 0.8, norm)
    # a scale that is 1% off shows with two terms and more than a few keys; 1% of it moves the
    # output of few keys, and of one term's bound, less than the roundings do
    scale = 1.01 if terms == 2 and n >= 40 else 1.1
    for wrong in (dict(lam=x["lam"] * 1.02), dict(scale=x["scale"] * scale), dict(seen=(x["seen"] - 1).clamp_min(1)),
                  dict(keys=x["keys"].flip(0)), dict(values=x["values"].flip(0)),
                  dict(out_scale=x["out_scale"] * 1.01)):
        with pytest.raises(AssertionError):
            da.check(definition(x, **wrong).bfloat16(), **x, terms=terms, what="planted")


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rho,lam", [(0.99, 0.8), (0.99, 1.0), (0.999, 0.8), (0.999, 1.0)])
@pytest.mark.parametrize("n,m", SHAPES[2:])
def test_rounded_maps_fail_where_they_are_alike(n, m, rho, lam, norm):
    """What the difference takes out of two maps that are alike leaves the roundings of
    both: with one bf16 term a probability the output is off by several roundings."""
    x = inputs(n, m, 64, 4, 2, rho, lam, norm)
    with pytest.raises(AssertionError):
        da.check(rounded_maps(x).bfloat16(), **x, terms=2, what="planted")
