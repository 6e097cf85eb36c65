"""Rotation, compaction and beam selection where a call could go wrong beside
others, at far offsets or in the last bits, and with checks that an unwritten
component fails."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

from oracle import operators as ref
from tests import test_gpu_operators as ops
from tests.written import check_written

pytestmark = pytest.mark.gpu

pa = ops.pa
cuda, normal, f64 = ops.cuda, ops.normal, ops.f64


# ---------------------------------------------------------------------------
# every component is written
# ---------------------------------------------------------------------------

@pytest.fixture()
def written(monkeypatch):
    """The checks of test_gpu_operators.py, with one that NaN fails."""
    monkeypatch.setattr(ops, "check_rotated", lambda got, want, size, what: check_written(f64(got), want, size, what))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,heads", [(128, 128, 8), (64, 32, 3), (80, 24, 2), (96, 20, 7), (72, 10, 1),
                                         (1024, 1024, 1), (1024, 6, 2), (256, 64, 33)])
def test_rotate_writes_every_component(pa, written, d, rot, heads, interleaved):
    ops.test_rotate(pa, d, rot, heads, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_and_far_rotations_write_every_component(pa, written, interleaved):
    ops.test_rotate_inverse_is_the_gradient(pa, interleaved)
    ops.test_rotate_positions_beyond_32_bits(pa)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,b,rot", [(1, 4, 2, 64, 16, 64), (64, 64, 8, 128, 16, 128), (37, 28, 4, 64, 32, 32),
                                              (130, 8, 1, 128, 8, 48), (9, 3, 3, 80, 5, 20), (5, 0, 2, 128, 64, 128),
                                              (3, 71, 1, 64, 4, 6), (700, 6, 2, 64, 16, 64)])
def test_rotate_and_cache_writes_every_component(pa, written, n, hq, hkv, d, b, rot, interleaved):
    ops._cached(pa, n, hq, hkv, d, b, rot, interleaved, seed=n + d, mscale=1.0 if n % 2 else 0.875)


@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("d,b,rot,interleaved", [(128, 16, None, False), (128, 16, 128, False), (64, 32, 32, True),
                                                 (80, 4, 24, True), (128, 64, 20, False), (256, 16, 10, False),
                                                 (72, 5, 6, True)])
def test_compaction_writes_every_component(pa, written, d, b, rot, interleaved, fork):
    ops.test_compact_subsets(pa, d, b, rot, interleaved, fork)


@pytest.mark.parametrize("rot", [None, 64])
def test_compaction_in_clusters_writes_every_component(pa, written, rot):
    ops.test_compact_long_in_place(pa, 8, rot)


# ---------------------------------------------------------------------------
# host threads at once
# ---------------------------------------------------------------------------

def test_compaction_from_several_host_threads(pa):
    """Eight threads compact pools of different head sizes and keep widths, each on a
    stream of its own: the same kernels with different needs of shared memory.  All
    calls succeed, and each pool ends as it does when its thread is alone.  (Calls of
    the C ABI with arguments made beforehand: little but the library's own work then
    keeps the threads apart.)"""
    from paged_kv_cache_167_gb300 import binding
    calls, void = 3000, ctypes.c_void_p
    plans = []
    for seed, (d, L, fork) in enumerate([(128, 6000, False), (64, 6000, False), (128, 300, True), (32, 2500, False)] * 2):
        rng = np.random.default_rng(seed)
        keep = np.concatenate([np.arange(64), 64 + ops._scattered(rng, L - 64, L // 2)])
        nb, src, dst, keep, counts = ops._compaction([L], [keep], 16, seed, fork)
        src = cuda(src)
        plans.append((normal((nb, 2, 8, 16, d), seed), src, cuda(dst) if fork else src, cuda(np.asarray([L], np.int32)),
                      cuda(keep), cuda(counts)))

    def run(plan, stream):
        pool, src, dst, lens, keep, counts = plan
        desc = binding.pool_desc(pool)
        args = (ctypes.byref(desc), void(src.data_ptr()), void(dst.data_ptr()), src.shape[1], void(lens.data_ptr()),
                void(keep.data_ptr()), keep.shape[1], void(counts.data_ptr()), void(0), 1, None,
                void(stream.cuda_stream))
        call = pa.lib().pa_compact_tokens
        return sum(call(*args) != 0 for _ in range(calls))

    alone = []
    for pool, *rest in plans:
        alone.append(pool.clone())
        assert run((alone[-1], *rest), torch.cuda.current_stream()) == 0
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    refused, start = [None] * len(plans), threading.Barrier(len(plans))

    def work(i):
        start.wait()
        refused[i] = run(plans[i], streams[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(plans))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(plans)
    for (pool, *_rest), want in zip(plans, alone):
        assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    assert pa.get_device_error() == 0


# ---------------------------------------------------------------------------
# far offsets inside a block
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("hkv,rot,fork", [(1, None, False), (1, 128, False), (2, 128, True), (1, 32, True)])
def test_compaction_in_blocks_of_more_than_2_31_elements(pa, hkv, rot, fork):
    """Rows either side of 2^31 elements from the beginning of a head's slab in one
    block: a warp's few, one CTA's and a cluster's."""
    d, far = 128, 2 ** 24
    B = far + 1000
    pool = torch.zeros((2 if fork else 1, 2, hkv, B, d), dtype=torch.bfloat16, device="cuda")
    before = normal((2, hkv, 2000, d), 3)
    w, freqs = (ref.angular_frequencies(rot), cuda(pa.rotary_frequencies(rot))) if rot else (None, None)
    src = cuda(np.zeros((1, 1), np.int32))
    dst = cuda(np.ones((1, 1), np.int32)) if fork else src
    rng = np.random.default_rng(4)
    for count, start in ((6, far - 2), (15, far - 8), (900, far - 500)):
        pool[0, :, :, far - 1000:] = before
        keep = start + 1 + ops._scattered(rng, B - start - 1, count)
        pa.compact_tokens(pool, src, dst, cuda(np.asarray([B], np.int32)), cuda(keep.astype(np.int32)[None]),
                          cuda(np.asarray([count], np.int32)), starts=cuda(np.asarray([start], np.int32)), freqs=freqs)
        assert pa.get_device_error() == 0
        moved = before[:, :, torch.as_tensor(keep - (far - 1000), device="cuda")]
        got = pool[-1, :, :, start:start + count]
        assert torch.equal(got[1], moved[1])
        if rot is None:
            assert torch.equal(got[0], moved[0])
        else:
            rows = f64(moved[0]).transpose(1, 0, 2)
            want, size = zip(*(ref.rotate(rows[i], start + i - int(keep[i]), w, False) for i in range(count)))
            check_written(f64(got[0].transpose(0, 1)), np.stack(want), np.stack(size), f"{count} rows")
        # nothing else was touched
        if fork:
            assert torch.equal(pool[0, :, :, far - 1000:], before)
        else:
            at = far - 1000
            assert torch.equal(pool[0, :, :, at:start], before[:, :, :start - at])
            assert torch.equal(pool[0, :, :, start + count:], before[:, :, start + count - at:])
        pool[:, :, :, far - 1000:] = 0
        for block in pool:
            for slab in block:
                assert int(torch.count_nonzero(slab.view(torch.int64).view(-1))) == 0


# ---------------------------------------------------------------------------
# the error of a row's log sum
# ---------------------------------------------------------------------------

def _log_sum_bound(mean_distance):
    """The header's bound of a row's log sum, for rows whose elements lie
    mean_distance below the maximum, weighted by their probability.  Relative errors
    of the sum of exponentials: the hardware's 2^x, 2^-22; the argument x log2(e) - c,
    rounded once, of size at most distance * log2(e) + 1/2: 2^-24 (distance + 0.4) in
    nats; log2(e) as fp32, 2^-26 distance; a thread's sum, at most four levels of
    additions of a chunk and a compensated running sum (2 * 2^-24), 6 * 2^-24; the
    integer units (at most 640 slices, half a unit of 2^-32 each) and the logarithm,
    2^-23."""
    return 2.0 ** -24 * (4 + (mean_distance + 0.4) + mean_distance / 4 + 6 + 2)


def _log_sum_error(pa, x, lse):
    """Selects one candidate of each row under a beam score that cancels the log sum
    nearly, so that fp32 holds the rest: the error of the log sum itself."""
    best = x.float().amax(-1).double().cpu().numpy()[:, 0]
    s = torch.as_tensor((lse - best).astype(np.float32), device="cuda")[:, None]
    scores = ops._select(pa, x, s, 1)[0].double().cpu().numpy()[:, 0]
    exact = s.double().cpu().numpy()[:, 0] + best - lse
    # (the score is an fp64 difference of numbers up to |best|, and one fp32 rounding of the rest)
    return np.abs(scores - exact) - 2.0 ** -24 * np.abs(exact) - 2.0 ** -50 * np.abs(best)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 130])
@pytest.mark.parametrize("V", [4097, 50257, 128256, 131072, 1000003])
def test_log_sum_of_equal_logits(pa, V, rows, dtype):
    """All roundings of a row of one value go the same way."""
    values = [0.0, 30.625, 6.9375, -11.3125, 0.7109375, 5.5, -0.109375, 100.5]
    for value in values:
        x = torch.full((rows, 1, V), value, dtype=dtype, device="cuda")
        err = _log_sum_error(pa, x, np.full(rows, value + math.log(V)))
        assert err.max() <= _log_sum_bound(0.0), (value, float(err.max()))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [50257, 128256])
def test_log_sum_of_a_peak_and_equal_tails(pa, V, dtype):
    """One maximum over a tail of one value: an argument rounded alike V times."""
    for top, below in ((3.0, 11.5), (-20.0, 11.5), (40.25, 9.75), (0.0, 23.0), (7.0, 0.015625)):
        x = torch.full((2, 1, V), top - below, dtype=torch.float32, device="cuda")
        x[:, 0, V // 3] = top
        x = x.to(dtype)
        tail = float(x[0, 0, 0])
        weight = (V - 1) * math.exp(tail - top)
        lse = top + math.log1p(weight)
        err = _log_sum_error(pa, x, np.full(2, lse))
        assert err.max() <= _log_sum_bound((top - tail) * weight / (1 + weight)), (top, below, float(err.max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [6, 140])
def test_log_sum_of_random_logits(pa, rows, dtype):
    V = 32003
    x = (torch.randn((rows, 1, V), generator=torch.Generator().manual_seed(rows)) * 3).to(dtype).cuda()
    lse, distance = np.zeros(rows), np.zeros(rows)
    for i in range(rows):
        y = f64(x[i, 0])
        p = np.exp(y - y.max())
        lse[i] = y.max() + math.log(math.fsum(p))
        distance[i] = ((y.max() - y) * p).sum() / p.sum()
    assert (_log_sum_error(pa, x, lse) <= _log_sum_bound(distance)).all()


# ---------------------------------------------------------------------------
# logits that fp64 scores cannot tell apart
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("G", [1, 80])
def test_selection_orders_a_row_by_its_logits(pa, G):
    """Logits of 0 and of 2^-80 give one fp64 score.  Within a row the larger logit
    comes first, in a short selection and in a longer one, in one slice and across
    slices; between rows of equal scores the lower row does."""
    V = 20001
    x = torch.full((G, 2, V), -1.0, device="cuda")
    x[:, :, 5], x[:, :, 6], x[:, :, 19000] = 0.0, 2.0 ** -80, 2.0 ** -70
    s = torch.full((G, 2), -2.0, device="cuda")
    for n in range(1, 8):
        scores, parents, tokens = ops._select(pa, x, s, n)
        flat = (parents * V + tokens).cpu().numpy()
        want = [19000, 6, 5, V + 19000, V + 6, V + 5, 0][:n]
        assert (flat == np.asarray(want)).all(), (n, flat[0])
        assert bool((scores[:, :6] == scores[:, :1]).all())
    assert pa.get_device_error() == 0
