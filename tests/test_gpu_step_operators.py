"""A step's tables, positions and slots, and rotary positions of several axes,
against plain restatements (oracle/operators.py), through the C ABI.

Tables, positions, slots, lengths and the cursor are whole numbers: equal.
Rotated components: the kernel and its bounds are those of one axis (2^-19 (|a| +
|b|) mscale before the one rounding to bf16, half a step of which is 2^-8
relative); each pair sees one axis's position."""
import numpy as np
import pytest
import torch

import pa_workloads as wl
from oracle import operators as ref

pytestmark = pytest.mark.gpu

bits = wl.bf16_bits
ANGLE = 2.0 ** -19
HALF_STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_167_gb300 as pa
    assert torch.cuda.is_available(), "a CUDA device is required"
    pa.get_device_error(clear=True)
    return pa


def cuda(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype)), device="cuda")


def normal(shape, seed):
    return wl.randn_bf16(shape, torch.Generator().manual_seed(seed)).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------------------
# a step's tables
# ---------------------------------------------------------------------------

class Step:
    """Device arrays of one call, the outputs full of a value it never writes."""

    def __init__(self, tables, ctx, new, free, cursor, b, num_blocks, max_tokens, offsets=None):
        self.host = (tables, ctx, new, free, cursor, b, num_blocks, max_tokens, offsets)
        i32 = np.int32
        self.tables, self.ctx, self.new = cuda(tables, i32), cuda(ctx, i32), cuda(new, i32)
        self.free, self.cursor = cuda(free, i32), cuda([cursor], i32)
        self.offsets = cuda(offsets, i32) if offsets is not None else None
        n = len(ctx)
        full = lambda size, dtype: torch.full((size,), -77, dtype=dtype, device="cuda")  # noqa: E731
        self.lens, self.starts, self.cursor_out = full(n, torch.int32), full(n + 1, torch.int32), full(1, torch.int32)
        self.positions, self.slots = full(max_tokens, torch.int64), full(max_tokens, torch.int64)

    def call(self, pa, stream=None):
        b, blocks = self.host[5:7]
        pa.extend_tables(self.tables, self.lens, self.starts, self.positions, self.slots, self.ctx, self.new,
                         self.free, self.cursor, self.cursor_out, b, blocks, position_offsets=self.offsets,
                         stream=stream)

    def check(self, pa, clear=True):
        tables, ctx, new, free, cursor, b, blocks, most, offsets = self.host
        want = ref.extend_tables(tables, ctx, new, free, cursor, b, blocks, most, offsets)
        assert self.tables.tolist() == want["tables"]
        assert self.lens.tolist() == want["lens"]
        assert self.starts.tolist() == want["starts"]
        assert self.cursor_out.tolist() == [want["cursor"]]
        assert self.positions.tolist() == want["positions"]
        assert self.slots.tolist() == want["slots"]
        if clear:
            assert pa.get_device_error(clear=True) == want["errors"]
        return want


def make(n, b, ctx_top, new_of, seed, room=0, short=None, offsets=True, width=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_top + 1, size=n)
    new = np.array([new_of(rng) for _ in range(n)], np.int64)
    have, end = -(-ctx // b), -(-(ctx + new) // b)
    width = width or max(int(end.max()) if n else 1, 1)
    blocks = int(end.sum()) + 9
    ids = rng.permutation(blocks)
    tables = np.full((n, width), -1, np.int64)
    at = 0
    for s in range(n):
        tables[s, :have[s]] = ids[at:at + have[s]]
        at += have[s]
    free = ids[at:]
    cursor = 4
    if short is not None:
        free = free[:cursor + int(short * (end - have).sum())]
    off = rng.integers(-3000, 3000, size=n) if offsets else None
    return Step(tables, ctx, new, free, cursor, b, blocks, int(new.sum()) + room, off)


ONE = lambda rng: 1                                              # noqa: E731
MIXED = lambda rng: int(rng.choice([0, 1, 1, 1, 2, 40]))         # noqa: E731


@pytest.mark.parametrize("n,b,ctx_top,new_of,room", [
    (1, 16, 0, ONE, 0), (1, 16, 37, lambda r: 5001, 3), (64, 16, 850, ONE, 0), (64, 4, 9, MIXED, 17),
    (511, 8, 100, ONE, 0), (512, 16, 100, MIXED, 1), (513, 16, 100, MIXED, 1), (1025, 32, 64, ONE, 600),
    (5000, 16, 20, MIXED, 100), (3, 1, 5, lambda r: 700, 0), (2, 17, 50, lambda r: 333, 5),
    (40, 64, 3, lambda r: 0, 12), (2000, 16, 30, lambda r: int(r.integers(0, 400) == 0) * 3000, 0)])
def test_extend_tables(pa, n, b, ctx_top, new_of, room):
    s = make(n, b, ctx_top, new_of, seed=n + b, room=room)
    s.call(pa)
    s.check(pa)
    s.call(pa)                  # again: the same step gives the same step
    s.check(pa)


@pytest.mark.parametrize("n", [5, 600, 3000])
@pytest.mark.parametrize("short", [0.0, 0.3, 0.97])
def test_extend_runs_out_of_blocks(pa, n, short):
    """Sequences behind the last free block are not served, those that want none are."""
    s = make(n, 4, 30, MIXED, seed=n, short=short)
    s.call(pa)
    s.check(pa)


@pytest.mark.parametrize("n", [6, 700])
@pytest.mark.parametrize("share", [0.0, 0.5, 0.999])
def test_extend_runs_out_of_places(pa, n, share):
    s = make(n, 8, 30, MIXED, seed=n + 1)
    tables, ctx, new, free, cursor, b, blocks, most, off = s.host
    Step(tables, ctx, new, free, cursor, b, blocks, int(most * share), off)
    s = Step(tables, ctx, new, free, cursor, b, blocks, int(most * share), off)
    s.call(pa)
    s.check(pa)


def test_extend_bad_inputs(pa):
    """Lengths below zero or beyond the table, ids out of range (in the list and in the
    table), a cursor behind the list: reported, and the other sequences are served."""
    big = 2 ** 31 - 1
    tables = [[0, 1, -1, -1], [2, -1, -1, -1], [99, -1, -1, -1], [-1, 3, -1, -1], [4, 5, 6, 7], [8, -1, -1, -1]]
    ctx, new = [-1, 3, 2, 6, 16, 1], [4, 2, 1, 1, 1, -2]
    s = Step(tables, ctx, new, [20, 55, 21, 22], 1, 4, 30, 12)
    s.call(pa)
    s.check(pa)
    s = Step(tables, [big, 0, 1, 6, 12, 1], [big, big, 5, 1, 4, 3], [20, 21], 0, 4, 30, 40)
    s.call(pa)
    s.check(pa)
    for cursor in (-1, 3, 2 ** 30):
        s = Step(tables, [1, 3, 2, 6, 16, 1], [1, 2, 1, 1, 0, 1], [20, 21], cursor, 4, 100, 12)
        s.call(pa)
        s.check(pa)


def test_extend_nothing(pa):
    """No sequences, no new tokens, no places, no free blocks."""
    s = make(0, 16, 0, ONE, seed=1, room=700, width=3)
    s.call(pa)
    s.check(pa)
    s = make(700, 16, 50, lambda r: 0, seed=2)
    s.call(pa)
    s.check(pa)
    s = make(3, 16, 14, lambda r: 1, seed=3, short=0.0, width=2)
    s.call(pa)
    s.check(pa)


@pytest.mark.parametrize("n,room,b", [(600, 0, 16), (4096, 100000, 7), (20011, 50, 16), (70001, 0, 32),
                                      (300000, 9, 16)])
def test_extend_many_sequences(pa, n, room, b):
    """Sequences by the thousands, with and without a range of places for each CTA of a
    cluster, pieces of more than 128; against sums of the lengths."""
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, 3 * b, size=n)
    new = rng.choice([0, 1, 1, 1, 2, 9], size=n)
    have, end = -(-ctx // b), -(-(ctx + new) // b)
    need = end - have
    ids = rng.permutation(int(end.sum()) + 10)
    tables = np.full((n, 5), -1, np.int64)
    tables[np.arange(5)[None, :] < have[:, None]] = ids[:have.sum()]
    s = Step(tables, ctx, new, ids[have.sum():], 3, b, len(ids), int(new.sum()) + room)
    s.call(pa)
    first = np.cumsum(new) - new
    assert np.array_equal(s.starts.cpu().numpy(), np.append(first, new.sum()))
    assert np.array_equal(s.lens.cpu().numpy(), ctx + new) and s.cursor_out.item() == 3 + need.sum()
    fresh = (np.arange(5)[None, :] >= have[:, None]) & (np.arange(5)[None, :] < end[:, None])
    tables[fresh] = ids[have.sum() + 3:][:need.sum()]      # row by row, in the sequences' order
    assert np.array_equal(s.tables.cpu().numpy(), tables)
    seq = np.repeat(np.arange(n), new)
    pos = ctx[seq] + np.arange(len(seq)) - first[seq]
    want = np.full(s.slots.numel(), -1)
    want[:len(seq)] = tables[seq, pos // b] * b + pos % b
    assert np.array_equal(s.slots.cpu().numpy(), want)
    want[:] = 0
    want[:len(seq)] = pos
    assert np.array_equal(s.positions.cpu().numpy(), want) and pa.get_device_error() == 0


def test_extend_many_sequences_far_tables(pa):
    """More sequences than a scan holds by far, and a table row beyond 2^31 bytes."""
    s = make(20000, 16, 3, ONE, seed=5, width=2)
    wide = torch.full((20000, 30000), -1, dtype=torch.int32, device="cuda")
    wide[:, :2] = s.tables
    s.tables = wide
    s.call(pa)
    want_starts = np.arange(20001)
    assert np.array_equal(s.starts.cpu().numpy(), want_starts)
    ctx, free = s.host[1], np.asarray(s.host[3])
    fresh = ctx == 0
    slots = s.slots.cpu().numpy()
    assert np.array_equal(slots[fresh], free[4:4 + fresh.sum()] * 16)
    rows = s.tables[:, 0].cpu().numpy()
    assert np.array_equal(slots[~fresh], rows[~fresh].astype(np.int64) * 16 + ctx[~fresh])
    assert s.cursor_out.item() == 4 + int(fresh.sum()) and pa.get_device_error() == 0


def test_extend_captured_steps(pa):
    """Three decode steps and a chunk, captured once and replayed: the lengths and the
    cursor go round on the device; and two calls at once on two streams."""
    n, b = 37, 4
    s = make(n, b, 11, lambda r: int(r.integers(0, 3)), seed=9, room=20, width=40)
    tables, ctx, new, free, cursor, _, _, most, off = s.host
    blocks = 4000
    free = np.concatenate([np.asarray(free), np.arange(int(np.max(free)) + 1000, int(np.max(free)) + 2500)])
    s = Step(tables, ctx, new, free, cursor, b, blocks, most, off)
    state = (np.asarray(tables), np.asarray(ctx), cursor)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.call(pa)
    torch.cuda.synchronize()
    s = Step(tables, ctx, new, free, cursor, b, blocks, most, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call(pa)
        lens, cur = s.lens.clone(), s.cursor_out.clone()
        s.ctx.copy_(s.lens)
        s.cursor.copy_(s.cursor_out)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = ref.extend_tables(state[0], state[1], new, free, state[2], b, blocks, most, off)
        assert s.tables.tolist() == want["tables"] and lens.tolist() == want["lens"]
        assert s.slots.tolist() == want["slots"] and s.positions.tolist() == want["positions"]
        assert cur.item() == want["cursor"]
        state = (want["tables"], want["lens"], want["cursor"])
    assert pa.get_device_error() == 0
    two = [make(900, 16, 90, MIXED, seed=20 + i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for one, stream in zip(two, streams):
            one.call(pa, stream=stream)
    torch.cuda.synchronize()
    for one in two:
        one.check(pa)


def test_extend_refusals(pa):
    s = make(3, 16, 20, ONE, seed=4)
    call = lambda **kw: pa.extend_tables(*[kw.get(k, v) for k, v in dict(  # noqa: E731
        tables=s.tables, lens=s.lens, starts=s.starts, positions=s.positions, slots=s.slots, ctx=s.ctx, new=s.new,
        free=s.free, cursor=s.cursor, cursor_out=s.cursor_out, b=16, blocks=99).items()])
    with pytest.raises(ValueError):
        call(starts=s.lens)
    with pytest.raises(ValueError):
        call(positions=s.positions[:-1])
    with pytest.raises(TypeError):
        call(positions=s.positions.int())
    with pytest.raises(TypeError):
        call(ctx=s.ctx.cpu())
    for kw in (dict(lens=s.ctx), dict(cursor_out=s.cursor)):       # what is read must not be written
        with pytest.raises(pa.PagedAttentionError) as e:
            call(**kw)
        assert e.value.status == 1
    assert pa.get_device_error() == 0


# ---------------------------------------------------------------------------
# positions of several axes
# ---------------------------------------------------------------------------

FAR = [[0, 7, 131071, 2 ** 40 + 5, -3], [1, 0, 12, 2 ** 33, 5], [100000, 3, 3, -2 ** 35, 6], [2, 2, 9, 9, 2 ** 20]]


def turned(x, positions, axis, w, interleaved, mscale):
    both = [ref.rotate_axes(x[n], [p[n] for p in positions], axis, w, interleaved, mscale) for n in range(len(x))]
    return np.stack([y for y, _ in both]), np.stack([s for _, s in both])


def check_turned(got, want, size, what):
    err = np.abs(f64(got) - want)
    bound = np.where(size > 0, HALF_STEP * np.abs(want) + ANGLE * (1 + HALF_STEP) * size, 0.0)
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} components off, worst {float((err - bound).max()):.3g}"


def exact_fractions(pairs, seed):
    """Frequencies that are multiples of 2^-48 of a turn, and the angles in fp64 they
    stand for: positions of 2^40 then have phases that fp64 reduces exactly."""
    rng = np.random.default_rng(seed)
    turns = rng.integers(1, 2 ** 40, size=pairs).astype(np.int64) << 16
    return turns


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("order", ["blocks", "cycled"])
@pytest.mark.parametrize("d,sections,heads", [(128, [16, 24, 24], 9), (80, [12, 12], 16), (64, [8, 3, 1, 4], 2),
                                              (72, [5, 0, 2], 3), (8, [1, 1], 1), (256, [128], 5),
                                              (1024, [100, 200, 212], 1), (40, [2, 2, 2], 7)])
def test_rotate_axes(pa, d, sections, heads, order, interleaved):
    n_axes, rot = len(sections), 2 * sum(sections)
    axis = pa.rotary_axes(sections, order)
    turns = exact_fractions(sum(sections), seed=d)
    positions = np.asarray(FAR[:n_axes], np.int64)
    x = normal((5, heads, d), seed=d + heads)
    # each pair's phase reduced in whole numbers, then turned by one position of 1
    want, size = np.zeros((5, heads, d)), np.zeros((5, heads, d))
    for n in range(5):
        phase = [(int(positions[a, n]) * int(t)) % 2 ** 64 / 2.0 ** 64 for a, t in zip(axis, turns)]
        want[n], size[n] = ref.rotate(f64(x)[n], 1, [2 * np.pi * f for f in phase], interleaved, 1.25)
    out = torch.full_like(x, float("nan"))
    freqs = cuda(turns)
    pa.rotate(out, x, cuda(positions), freqs, interleaved=interleaved, mscale=1.25, axes=axis)
    check_turned(out, want, size, f"d={d} {order}")
    # rows of positions that lie apart, a strided x, in place: the same bits
    apart = torch.zeros((n_axes, 11), dtype=torch.int64, device="cuda")
    apart[:, 3:8] = cuda(positions)
    wide = normal((5, heads + 2, d), seed=1)
    wide[:, 1:1 + heads] = x
    again = torch.empty_like(x)
    pa.rotate(again, wide[:, 1:1 + heads], apart[:, 3:8], freqs, interleaved=interleaved, mscale=1.25, axes=axis)
    pa.rotate(x, x, cuda(positions), freqs, interleaved=interleaved, mscale=1.25, axes=axis)
    assert np.array_equal(bits(again), bits(out)) and np.array_equal(bits(x), bits(out))
    assert pa.get_device_error() == 0


def test_rotate_axes_of_equal_positions_is_one_axis(pa):
    """Text: equal positions on every axis give the bits of the call with one."""
    x = normal((700, 6, 128), seed=2)
    pos = torch.arange(700, device="cuda") * 37 - 100
    freqs = cuda(pa.rotary_frequencies(128))
    one, three = torch.empty_like(x), torch.empty_like(x)
    pa.rotate(one, x, pos, freqs)
    pa.rotate(three, x, pos.expand(3, 700).contiguous(), freqs, axes=pa.rotary_axes([16, 24, 24]))
    assert np.array_equal(bits(one), bits(three))


@pytest.mark.parametrize("heads,d,rot", [(1, 128, 128), (2, 128, 64), (3, 80, 48), (5, 64, 64), (16, 80, 48),
                                         (9, 1024, 1024), (80, 128, 128), (31, 64, 32)])
def test_rotate_axes_many_tokens(pa, heads, d, rot):
    """Calls that fill the GPU, few heads and many: each axis on its own gives, for its pairs,
    the bits of the call with that axis's position for all."""
    n = 6007 if heads < 80 else 700
    x = normal((n, heads, d), seed=heads)
    axis = pa.rotary_axes([rot // 2 - rot // 4 - 1, rot // 4, 1], "cycled")
    pos = torch.stack([torch.arange(n, device="cuda") * 3, torch.arange(n, device="cuda") // 7 + 10 ** 6,
                       5 - torch.arange(n, device="cuda")])
    freqs = cuda(pa.rotary_frequencies(rot))
    got, one = torch.empty_like(x), torch.empty_like(x)
    pa.rotate(got, x, pos, freqs, axes=axis)
    for a in range(3):
        pa.rotate(one, x, pos[a].contiguous(), freqs)
        pairs = cuda(np.nonzero(axis == a)[0])
        for part in (pairs, pairs + rot // 2):
            assert torch.equal(got[:, :, part].view(torch.int16), one[:, :, part].view(torch.int16))
    assert torch.equal(got[:, :, rot:], x[:, :, rot:]) and pa.get_device_error() == 0


@pytest.mark.parametrize("heads", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("d,rot", [(16, 16), (24, 16), (32, 32)])
def test_rotate_axes_small_heads_many_tokens(pa, heads, d, rot):
    """Tokens of one or two chunks, of which a CTA could hold more than a block has places."""
    n = 100003
    x = normal((n, heads, d), seed=heads)
    pos = torch.arange(n, device="cuda") * 5 - 1000
    freqs = cuda(pa.rotary_frequencies(rot))
    one, two = torch.empty_like(x), torch.empty_like(x)
    pa.rotate(one, x, pos, freqs)
    pa.rotate(two, x, pos.expand(2, n).contiguous(), freqs, axes=pa.rotary_axes([rot // 2 - 3, 3], "cycled"))
    assert np.array_equal(bits(one), bits(two)) and pa.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (0, 2), (4, 2), (64, 8)])
def test_rotate_and_cache_axes_many_tokens(pa, hq, hkv):
    """The same with the slot writer, against the call with one axis: equal positions."""
    n, d, b = 5003, 128, 16
    q, k, v = normal((n, max(hq, 1), d), seed=1), normal((n, hkv, d), seed=2), normal((n, hkv, d), seed=3)
    slots = torch.randperm(5008, generator=torch.Generator().manual_seed(4))[:n].cuda()
    slots[::5] = -1
    pos = torch.arange(n, device="cuda") + 77
    freqs = cuda(pa.rotary_frequencies(d))
    pools, outs = [], []
    for axes in (None, pa.rotary_axes([16, 24, 24])):
        pool, out = torch.zeros((313, 2, hkv, b, d), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(q)
        pa.rotate_and_cache(pool, out if hq else None, q if hq else None, k, v,
                            pos if axes is None else pos.expand(3, n).contiguous(), slots, freqs, axes=axes)
        pools.append(pool)
        outs.append(out)
    assert torch.equal(pools[0], pools[1]) and torch.equal(outs[0], outs[1]) and pa.get_device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_axes_inverse_is_the_gradient(pa, interleaved):
    """R^T g by the inverse call, against the formula and against the columns of R (the
    forward call on unit vectors, each entry rounded once, two a column)."""
    d, sections = 32, [3, 4, 5]
    axis = pa.rotary_axes(sections, "cycled")
    w = ref.angular_frequencies(24)
    freqs, positions = cuda(pa.rotary_frequencies(24)), [[17], [1234], [-8]]
    g = normal((1, 1, d), seed=8)
    back = torch.empty_like(g)
    pa.rotate(back, g, cuda(positions, np.int64), freqs, interleaved=interleaved, mscale=1.5, inverse=True, axes=axis)
    want, size = turned(f64(g), [[-p[0]] for p in positions], axis, w, interleaved, 1.5)
    check_turned(back, want, size, "inverse")
    units = torch.eye(d, dtype=torch.bfloat16, device="cuda").reshape(d, 1, d)
    columns = torch.empty_like(units)
    pa.rotate(columns, units, cuda(np.repeat(np.asarray(positions, np.int64), d, axis=1)), freqs,
              interleaved=interleaved, mscale=1.5, axes=axis)
    slope = f64(columns)[:, 0] @ f64(g)[0, 0]
    bound = (HALF_STEP * np.abs(f64(columns)[:, 0]) + 2 * ANGLE * 1.5) @ np.abs(f64(g)[0, 0])
    off = np.abs(f64(back)[0, 0] - slope)
    assert (off <= bound + HALF_STEP * np.abs(want[0, 0]) + 2 * ANGLE * size[0, 0]).all()


@pytest.mark.parametrize("n,hq,hkv,d,b,sections,order,interleaved", [
    (1, 8, 2, 128, 16, [16, 24, 24], "blocks", False), (64, 64, 8, 128, 16, [24, 20, 20], "cycled", False),
    (333, 7, 1, 64, 32, [4, 6, 6], "cycled", True), (1500, 12, 4, 128, 8, [16, 16], "blocks", True),
    (40, 0, 3, 72, 4, [4, 5, 0, 6], "blocks", False)])
def test_rotate_and_cache_axes(pa, n, hq, hkv, d, b, sections, order, interleaved):
    rng = np.random.default_rng(n)
    axis = pa.rotary_axes(sections, order)
    w = ref.angular_frequencies(2 * sum(sections))
    freqs = cuda(pa.rotary_frequencies(2 * sum(sections)))
    positions = rng.integers(0, 5000, size=(len(sections), n)).astype(np.int64)
    blocks = n // b + 4
    slots = rng.permutation(blocks * b)[:n].astype(np.int64)
    slots[rng.random(n) < 0.2] = -1
    qkv = normal((n, hq + 2 * hkv, d), seed=n + d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    layered = normal((blocks, 2, 2, hkv, b, d), seed=3)
    before = layered.clone()
    out = torch.full((n, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pa.rotate_and_cache(layered, out if hq else None, q if hq else None, k, v, cuda(positions), cuda(slots), freqs,
                        interleaved=interleaved, layer=1, axes=axis)
    some = np.unique(rng.integers(0, n, size=40))       # the restatement takes a token at a time
    if hq:
        want, size = turned(f64(q)[some], positions[:, some], axis, w, interleaved, 1.0)
        check_turned(out[cuda(some)], want, size, "q")
        assert not torch.isnan(out).any()
    want, size = turned(f64(k)[some], positions[:, some], axis, w, interleaved, 1.0)
    real = slots[some] >= 0
    at = slots[some][real]
    check_turned(layered[cuda(at // b), 0, 1, :, cuda(at % b)], want[real], size[real], "k")
    real = slots >= 0
    at = slots[real]
    assert torch.equal(layered[cuda(at // b), 1, 1, :, cuda(at % b)], v[cuda(np.nonzero(real)[0])])
    # the rest of the pool, the other layer among it, as it was
    before[cuda(at // b), :, 1, :, cuda(at % b)] = layered[cuda(at // b), :, 1, :, cuda(at % b)]
    assert torch.equal(layered, before)
    assert pa.get_device_error() == 0


def test_axes_refusals_of_the_binding(pa):
    x, freqs, axis = normal((4, 2, 16), seed=1), cuda(pa.rotary_frequencies(16)), pa.rotary_axes([3, 5])
    pos = torch.zeros((2, 4), dtype=torch.int64, device="cuda")
    out = torch.empty_like(x)
    bad = [dict(axes=axis[:-1]), dict(axes=axis, positions=pos[:, :3]), dict(axes=axis, positions=pos[0]),
           dict(axes=axis, positions=pos.T.contiguous().T)]
    for kw in bad:
        with pytest.raises(ValueError):
            pa.rotate(out, x, kw.pop("positions", pos), freqs, **kw)
    for kw in (dict(axes=axis.tolist()), dict(axes=axis.astype(np.int32)), dict(axes=axis, positions=pos.int()),
               dict(axes=axis, positions=pos.cpu())):
        with pytest.raises((TypeError, ValueError)):
            pa.rotate(out, x, kw.pop("positions", pos), freqs, **kw)
    with pytest.raises(pa.PagedAttentionError):
        pa.rotate(out, x, pos[:1], freqs, axes=axis)       # a pair by an axis that has no positions
    assert pa.get_device_error() == 0
