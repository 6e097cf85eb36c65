"""Rotation, compaction and beam selection where a call could go wrong beside
others, at far offsets or in the last bits."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from tests import test_gpu_operators as ops

pytestmark = pytest.mark.gpu

pa = ops.pa
cuda, normal, f64 = ops.cuda, ops.normal, ops.f64


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
