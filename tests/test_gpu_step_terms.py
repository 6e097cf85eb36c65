"""The serving loop of tests/test_gpu_step_together.py (tables on the GPU, positions of
three axes, differential attention of chunks, then of single tokens) with every output,
of a chunk or of a decode step, held to the bounds of two bf16 terms a probability and to
the average error of their roundings; the maps alike, as trained ones are in part."""
import math

import pytest
import torch

from tests import diff_accuracy as da
from tests.test_gpu_step_together import Loop, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rho", [0.0, 0.98])
@pytest.mark.parametrize("d,hq,hkv,b,norm,keys", [(128, 16, 4, 16, True, "map"), (64, 8, 2, 32, True, "head"),
                                                  (64, 4, 4, 8, False, "map")])
def test_serving_loop_within_two_terms(pa, d, hq, hkv, b, norm, keys, rho):  # noqa: F811
    B, chunk, steps = 4, 45, 3
    x = Loop(pa, B, hq, hkv, d, b, 0, norm, keys, seed=d + b)
    g = torch.Generator(device="cuda").manual_seed(2)
    empty = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    i64 = torch.int64

    def draw(n):
        rows = torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda")
        if rho:      # the second map's queries and keys close to the first's
            for lo, hi in ((0, hq), (hq, hq + hkv)):
                first = rows[:, lo:hi:2]
                rows[:, lo + 1:hi:2] = rho * first + math.sqrt(1 - rho * rho) * rows[:, lo + 1:hi:2]
        return rows.bfloat16()

    turned, outs, kinds = [], [], []
    ws = empty(pa.decode_diff_workspace_size(x.pool, B, hq, 24 * b), dtype=torch.uint8)
    for n in (chunk, chunk) + (1,) * steps:
        rows, rot = draw(B * n), empty(B * n, hq, d)
        out = empty(B, n, hq // 2, 2 * d) if n > 1 else empty(B, hq // 2, 2 * d)
        x.step(torch.full((B,), n, dtype=torch.int32, device="cuda"), rows, empty(B * n, dtype=i64),
               empty(B * n, dtype=i64), empty(3, B * n, dtype=i64), rot, out, workspace=None if n > 1 else ws)
        turned.append(rot.view(B, n, hq, d))
        outs.append(out.view(B, n, hq // 2, 2 * d))
        kinds.append("chunk" if n > 1 else "decode")
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    total = 2 * chunk + steps
    assert x.lens.tolist() == [total] * B
    t = torch.arange(total, device="cuda")
    for s in range(B):
        blk = x.tables[s].long()[t // b]
        k, v = x.pool[blk, 0, :, t % b].transpose(0, 1), x.pool[blk, 1, :, t % b].transpose(0, 1)
        at = 0
        for q, out, kind in zip(turned, outs, kinds):
            n = q.shape[1]
            da.check(out[s], q[s], k, v, t[at:at + n] + 1, x.scale, x.lam, x.weight, 1e-5, 1.0, keys == "head", 2,
                     f"sequence {s}, {kind} at {at}")
            at += n
