"""Differential prefill with two bf16 terms a probability, held to the bounds of two terms
and to the average error (tests/diff_accuracy.py); maps that are alike, few keys, the form
with one term, and prefill beside decode."""
import math

import numpy as np
import pytest
import torch

import pa_workloads as wl
from tests import diff_accuracy as da
from tests.test_gpu_diff import Batch, chunked, pa  # noqa: F401

pytestmark = pytest.mark.gpu

bits = wl.bf16_bits


def check(x, out, terms, what=""):
    for s in range(len(x.lens)):
        seen = x.lens[s] - x.chunk + 1 + torch.arange(x.chunk, device="cuda")
        da.check(out[s], x.q[s], x.k[s], x.v[s], seen, x.scale, x.lam, x.weight, x.eps, x.out_scale,
                 x.keys == "head", terms, f"{what} sequence {s}, {x.chunk} of {x.lens[s]} tokens")


def alike(x, rho, lam):
    """The second map's queries correlated with the first's, on equal keys."""
    x.pool[:, 0, 1::2] = x.pool[:, 0, 0::2]
    for k in x.k:
        k[1::2] = k[0::2]
    noise = x.q[..., 1::2, :].float()
    x.q[..., 1::2, :] = (rho * x.q[..., 0::2, :].float() + math.sqrt(1 - rho * rho) * noise).bfloat16()
    x.lam.fill_(lam)
    return x


@pytest.mark.parametrize("b", [8, 16, 32, 64])
@pytest.mark.parametrize("per", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_diff_within_two_terms(pa, d, per, b):  # noqa: F811
    x = chunked([0, 1, 127, 300], 40, 2 * per, 2, d, b, seed=b + per, norm=per != 2, keys="head" if b == 32 else "map")
    check(x, x.prefill(pa), 2, f"d={d} R={per} b={b}")
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("chunk", [1, 2, 3, 17, 64, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_diff_of_few_keys(pa, d, chunk):  # noqa: F811
    """The first rows of a prompt, and chunks whose rows see a few cached keys."""
    x = chunked([0, 0, 1, 5], chunk, 8, 4, d, 16, seed=chunk)
    check(x, x.prefill(pa), 2)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rho,lam", [(0.99, 0.8), (0.99, 1.0), (0.999, 0.8), (0.999, 1.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_diff_of_maps_that_are_alike(pa, d, rho, lam, norm):  # noqa: F811
    """What the operator is for: most of both maps cancels, and what is left is as exact
    as when nothing does.  Decode's rows are held to the same."""
    x = alike(chunked([0, 260, 1500], 70, 8, 4, d, 16, seed=31, norm=norm), rho, lam)
    out = x.prefill(pa).clone()
    check(x, out, 2, "prefill")
    last = torch.empty((3, 4, 2 * d), dtype=torch.bfloat16, device="cuda")
    pa.decode_diff(last, x.q[:, -1].contiguous(), x.pool, x.tables, x.lens_dev, x.max_len, x.scale,
                   workspace=x.workspace(pa), **x.weights())
    for s in range(3):
        seen = torch.tensor([x.lens[s]], device="cuda")
        a = (x.q[s, -1:], x.k[s], x.v[s], seen, x.scale, x.lam, x.weight, x.eps, x.out_scale, False, 2)
        want, tol, _ = da.expected(*a)
        da.check(last[s:s + 1], *a, "decode")
        # one token's output from a chunk and from a decode step: two roundings of values that
        # both lie within the bound of the fp32 steps (tol less the rounding's 2^-8)
        apart = (last[s].double() - out[s, -1].double()).abs()
        steps = (tol[0] - 2.0 ** -8 * want[0].abs()).clamp_min(0)
        assert (apart <= 2.0 ** -7 * want[0].abs() * (1 + 2.0 ** -7) + 2 * steps).all()
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("d,per,keys", [(64, 1, "map"), (128, 2, "head"), (128, 8, "map"), (64, 4, "head")])
def test_prefill_diff_of_one_term(pa, d, per, keys):  # noqa: F811
    """The flag reaches the kernel, and its rounding is the one that is said."""
    x = chunked([0, 3, 200, 700], 90, 4 * per, 4, d, 16, seed=32, keys=keys)
    two = x.prefill(pa).clone()
    one = x.prefill(pa, one_term=True)
    assert not torch.equal(one, two)
    check(x, one, 1)
    check(x, two, 2)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("one_term", [False, True])
def test_prefill_diff_equal_maps_cancel_with_either(pa, one_term):  # noqa: F811
    x = Batch([300, 77, 150], 8, 4, 128, 16, seed=6, keys="head", chunk=70)
    x.q[:, :, 1::2] = x.q[:, :, 0::2]
    x.lam.fill_(1.0)
    x.prefill(pa, one_term=one_term)
    assert torch.equal(x.out, torch.zeros_like(x.out)) and pa.get_device_error() == 0


@pytest.mark.parametrize("ctas", [2, 6, 152])
def test_prefill_diff_hand_overs_of_either(pa, ctas):  # noqa: F811
    """The same bits however the units are dealt to the clusters, with either form, and in
    a graph."""
    x = chunked([0, 500, 3, 100], 70, 16, 2, 128, 16, seed=33)
    for one_term in (False, True):
        pa.set_prefill_ctas(0)
        want = x.prefill(pa, one_term=one_term).clone()
        pa.set_prefill_ctas(ctas)
        graph, ctx = torch.cuda.CUDAGraph(), x.ctx_dev
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            pa.prefill_diff(x.out, x.q, x.pool, x.tables, ctx, 500, x.scale, one_term=one_term, **x.weights())
        for _ in range(2):
            x.out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(bits(x.out), bits(want))
    pa.set_prefill_ctas(0)
    assert pa.get_device_error() == 0
