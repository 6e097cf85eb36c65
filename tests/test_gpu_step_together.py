"""The operators of a step together, as a serving loop uses them: tables and slots
built on the GPU, positions of three axes turned and stored at those slots,
differential attention of the prompts' chunks, then of single tokens, several
decode steps captured in one graph.  The cache is compared with the inputs turned
in 64 bits, the outputs with the definition over the tokens so far."""
import numpy as np
import pytest
import torch

from oracle import operators as ref
from tests import diff_reference as dr

pytestmark = pytest.mark.gpu

ANGLE, HALF_STEP = 2.0 ** -19, 2.0 ** -8


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_167_gb300 as pa
    assert torch.cuda.is_available(), "a CUDA device is required"
    pa.get_device_error(clear=True)
    return pa


class Loop:
    """Device state of a serving loop; every array of fixed size, none read by the host."""

    def __init__(self, pa, B, hq, hkv, d, b, room, norm, keys, seed):
        self.pa, self.hq, self.hkv, self.d, self.b, self.keys = pa, hq, hkv, d, b, keys
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        i32 = torch.int32
        blocks = 200
        self.blocks = blocks
        self.pool = torch.full((blocks, 2, hkv, b, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.tables = torch.full((B, 24), -1, dtype=i32, device="cuda")
        self.free = torch.as_tensor(rng.permutation(blocks).astype(np.int32), device="cuda")
        self.cursor = torch.zeros(1, dtype=i32, device="cuda")
        self.cursor_out = torch.zeros(1, dtype=i32, device="cuda")
        self.ctx = torch.zeros(B, dtype=i32, device="cuda")
        self.lens = torch.zeros(B, dtype=i32, device="cuda")
        self.starts = torch.zeros(B + 1, dtype=i32, device="cuda")
        self.offsets = torch.as_tensor(rng.integers(-50, 50, size=B).astype(np.int32), device="cuda")
        axes = [d // 2 - 2 * (d // 6), d // 6, d // 6]
        self.axis = pa.rotary_axes(axes, "cycled")
        self.w = ref.angular_frequencies(d)
        self.freqs = torch.as_tensor(pa.rotary_frequencies(d), device="cuda")
        self.lam = torch.rand(hq // 2, generator=g, device="cuda")
        self.weight = 1 + 0.1 * torch.randn(2 * d, generator=g, device="cuda") if norm else None
        self.scale = d ** -0.5

    def step(self, new, qkv, slots, positions, by_axis, rot, out, workspace=None):
        """One step: `new` tokens of each sequence, qkv [tokens][hq + 2 hkv][d]."""
        pa, hq, hkv, B = self.pa, self.hq, self.hkv, len(self.ctx)
        pa.extend_tables(self.tables, self.lens, self.starts, positions, slots, self.ctx, new, self.free, self.cursor,
                         self.cursor_out, self.b, self.blocks, position_offsets=self.offsets)
        # time goes on with the text; height and width trail it (as behind an image)
        by_axis[0].copy_(positions)
        torch.sub(positions, 3, out=by_axis[1])
        torch.sub(positions, 11, out=by_axis[2])
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pa.rotate_and_cache(self.pool, rot, q, k, v, by_axis, slots, self.freqs, axes=self.axis)
        weights = dict(lam=self.lam, norm_weight=self.weight, keys=self.keys)
        if workspace is None:
            chunk = qkv.shape[0] // B
            pa.prefill_diff(out, rot.view(B, chunk, hq, self.d), self.pool, self.tables, self.ctx, 24 * self.b - chunk,
                            self.scale, **weights)
        else:
            pa.decode_diff(out, rot, self.pool, self.tables, self.lens, 24 * self.b, self.scale, workspace=workspace,
                           **weights)
        self.ctx.copy_(self.lens)
        self.cursor.copy_(self.cursor_out)


@pytest.mark.parametrize("d,hq,hkv,b,norm,keys", [(128, 16, 4, 16, True, "map"), (64, 4, 4, 8, False, "map"),
                                                  (64, 8, 2, 32, True, "head"), (128, 8, 2, 64, True, "map")])
def test_serving_loop(pa, d, hq, hkv, b, norm, keys):
    B, chunk, steps = 5, 37, 4
    x = Loop(pa, B, hq, hkv, d, b, 0, norm, keys, seed=d + b)
    i64, bf = torch.int64, torch.bfloat16
    empty = lambda *s, dtype=bf: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda n: torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda").to(bf)  # noqa: E731

    history = []        # (qkv rows, turned queries, output) of each step, [B][tokens]
    # two chunks of prompt tokens
    for _ in range(2):
        n = B * chunk
        qkv, out, rot = draw(n), empty(B, chunk, hq // 2, 2 * d), empty(n, hq, d)
        x.step(torch.full((B,), chunk, dtype=torch.int32, device="cuda"), qkv, empty(n, dtype=i64),
               empty(n, dtype=i64), empty(3, n, dtype=i64), rot, out)
        history.append((qkv.view(B, chunk, -1, d), rot.view(B, chunk, hq, d), out))
    # decode steps: one graph of one step, replayed; new inputs in the same buffer
    new = torch.ones(B, dtype=torch.int32, device="cuda")
    qkv, out, rot = draw(B), empty(B, hq // 2, 2 * d), empty(B, hq, d)
    slots, positions, by_axis = empty(B, dtype=i64), empty(B, dtype=i64), empty(3, B, dtype=i64)
    ws = empty(pa.decode_diff_workspace_size(x.pool, B, hq, 24 * b), dtype=torch.uint8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.step(new, qkv, slots, positions, by_axis, rot, out, workspace=ws)
    for _ in range(steps):
        qkv.copy_(draw(B))
        graph.replay()
        history.append((qkv.clone().view(B, 1, -1, d), rot.clone().view(B, 1, hq, d),
                        out.clone().view(B, 1, hq // 2, 2 * d)))
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0

    total = 2 * chunk + steps
    assert x.lens.tolist() == [total] * B
    taken = x.cursor_out.item()
    assert taken == B * -(-total // b)
    used = x.tables[:, :-(-total // b)].flatten().tolist()
    assert sorted(used) == sorted(x.free[:taken].tolist())
    rows, turned, outs = (torch.cat([h[i] for h in history], dim=1) for i in range(3))   # [B][total][..][d]
    t = torch.arange(total, device="cuda")
    for s in range(B):
        blk = x.tables[s].long()[t // b]
        cached, values = x.pool[blk, 0, :, t % b], x.pool[blk, 1, :, t % b]       # [total][hkv][d]
        assert torch.equal(values, rows[s, :, hq + hkv:])
        # queries and cached keys against the inputs turned in 64 bits, some of them
        off = int(x.offsets[s])
        for i in sorted({*range(0, total, 9), *range(total - steps, total)}):
            pos = [i + off, i + off - 3, i + off - 11]
            want, size = ref.rotate_axes(rows[s, i, :hq + hkv].double().cpu().numpy(), pos, list(x.axis), x.w, False)
            got = torch.cat([turned[s, i], cached[i]]).double().cpu().numpy()
            assert (np.abs(got - want) <= HALF_STEP * np.abs(want) + ANGLE * (1 + HALF_STEP) * size).all()
        # the outputs, from the queries and the cache as they are; one term a probability in the chunks
        want, tol = dr.pairs(turned[s], cached.transpose(0, 1), values.transpose(0, 1), t + 1, x.scale, x.lam,
                             x.weight, 1e-5, 1.0, keys == "head", terms=1)
        dr.check(outs[s], want, tol, f"sequence {s}")
