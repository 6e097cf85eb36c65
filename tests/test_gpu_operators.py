"""Rotary positions with the slot writer, compaction of cached tokens and beam
selection against their fp64 restatements (oracle/operators.py), through the
C ABI.

Tolerances.  A rotated component is a cos - b sin with the angle's phase reduced
exactly: the phase's fp32 value and the product with 2 pi are off by 2^-24 each,
relative to at most pi (2^-21.3 together), and the hardware's sine and cosine by
2^-20.5, so cos and sin are off by less than 2^-19.8; the three fp32 operations
and the scale add 4 * 2^-24.  Together less than 2^-19 (|a| + |b|) mscale.  The
rounding to bf16 is off by half a step, 2^-8 relative.  Values are moved bit for
bit.

Scores: one fp32 rounding of the fp64 score (2^-24 relative) plus the error of
the log-sum-exp, which is the relative error of its sum of exponentials: 2^-22
(the hardware's 2^x), 2^-23 T for arguments down to -T below the maximum (their
difference and their product with log2 e, each rounded), and one 2^-24 per
addition of the at most k elements a thread sums.  Terms below e^-24 of the
maximum are less than 2^-34 of the sum each and less than 2^-18 of it together
at these vocabularies, so T = 24 with 2^-23 * T of their own share is ample.
"""
import math

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


def cuda(a):
    return torch.as_tensor(a, device="cuda")


def normal(shape, seed):
    return wl.randn_bf16(shape, torch.Generator().manual_seed(seed)).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_rotated(got, want, size, what):
    err = np.abs(f64(got) - want)
    # where nothing was rotated (size 0) the row was copied: it must be exact
    bound = np.where(size > 0, HALF_STEP * np.abs(want) + ANGLE * (1 + HALF_STEP) * size, 0.0)
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} components off, worst {float((err - bound).max()):.3g}"


def rotated(x, positions, w, interleaved, mscale=1.0):
    """[N][H][d] fp64 -> (rotated, |a| + |b|)."""
    both = [ref.rotate(x[n], int(positions[n]), w, interleaved, mscale) for n in range(len(x))]
    return np.stack([y for y, _ in both]), np.stack([s for _, s in both])


POSITIONS = [0, 1, 17, 4095, 131071, 2 ** 20 + 3, -5]


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,heads", [(128, 128, 8), (64, 32, 3), (64, 64, 5), (80, 24, 2), (96, 20, 7),
                                         (72, 10, 1), (8, 2, 4), (256, 64, 33), (1024, 1024, 1), (1024, 6, 2),
                                         (128, 126, 2)])
def test_rotate(pa, d, rot, heads, interleaved):
    w = ref.angular_frequencies(rot)
    freqs = cuda(pa.rotary_frequencies(rot))
    x = normal((len(POSITIONS), heads, d), seed=d + rot)
    want, size = rotated(f64(x), POSITIONS, w, interleaved, 1.25)
    out = torch.full_like(x, float("nan"))
    pa.rotate(out, x, cuda(np.asarray(POSITIONS)), freqs, interleaved=interleaved, mscale=1.25)
    check_rotated(out, want, size, f"d={d} rot={rot}")
    # in place, and a strided view of a wider row, give the same bits
    wide = normal((len(POSITIONS), heads + 3, d), seed=1)
    wide[:, 2:2 + heads] = x
    view_out = torch.empty_like(x)
    pa.rotate(view_out, wide[:, 2:2 + heads], cuda(np.asarray(POSITIONS)), freqs, interleaved=interleaved, mscale=1.25)
    pa.rotate(x, x, cuda(np.asarray(POSITIONS)), freqs, interleaved=interleaved, mscale=1.25)
    assert np.array_equal(bits(x), bits(out)) and np.array_equal(bits(view_out), bits(out))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192, high=4.0),
                                dict(scaling="parts_index", factor=16.0, original_len=4096)])
def test_rotate_scaled_and_far(pa, kw):
    """Scaled frequencies at far positions.  The frequencies themselves may
    differ by some 2^-47 between the two fp64 evaluations: 2^-24 at 2^23."""
    x = normal((4, 2, 64), seed=5)
    positions = [3, 98304, 2 ** 22 + 1, 2 ** 23]
    want, size = rotated(f64(x), positions, ref.angular_frequencies(64, **kw), False)
    out = torch.empty_like(x)
    pa.rotate(out, x, cuda(np.asarray(positions)), cuda(pa.rotary_frequencies(64, **kw)))
    check_rotated(out, want, size, str(kw))


def test_rotate_positions_beyond_32_bits(pa):
    """Frequencies that are binary fractions of a turn make the fp64 angle of a
    position of 2^40 exact: only the kernel's reduction is tested."""
    turns = [2.0 ** -3, 2.0 ** -43, 3 * 2.0 ** -42, 1 - 2.0 ** -20]
    freqs = cuda(np.asarray([int(t * 2 ** 64) for t in turns], dtype=np.uint64).view(np.int64))
    positions = [2 ** 40 + 5, -(2 ** 41) + 1, 2 ** 32 - 1]
    x = normal((3, 2, 8), seed=6)
    want, size = np.zeros((3, 2, 8)), np.zeros((3, 2, 8))
    for n, pos in enumerate(positions):
        w = [2 * math.pi * float((pos * int(t * 2 ** 64)) % 2 ** 64) / 2.0 ** 64 for t in turns]
        want[n], size[n] = ref.rotate(f64(x)[n], 1, w, True)
    out = torch.empty_like(x)
    pa.rotate(out, x, cuda(np.asarray(positions)), freqs, interleaved=True)
    check_rotated(out, want, size, "2^40")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_inverse_is_the_gradient(pa, interleaved):
    """y = R x is linear: the gradient of <g, y> is R^T g.  The inverse call
    against the formula, and against differences (the forward call on x and on
    x plus each unit vector: columns of R, each bf16)."""
    d, rot, pos = 32, 24, 1234
    w = ref.angular_frequencies(rot)
    freqs = cuda(pa.rotary_frequencies(rot))
    g = normal((1, 1, d), seed=8)
    back = torch.empty_like(g)
    pa.rotate(back, g, cuda(np.asarray([pos])), freqs, interleaved=interleaved, mscale=1.5, inverse=True)
    want, size = ref.rotate(f64(g)[0, 0], -pos, w, interleaved, 1.5)
    check_rotated(back, want[None, None], size[None, None], "inverse")
    units = torch.eye(d, dtype=torch.bfloat16, device="cuda").reshape(d, 1, d)
    columns = torch.empty_like(units)
    pa.rotate(columns, units, cuda(np.full(d, pos)), freqs, interleaved=interleaved, mscale=1.5)
    cols = f64(columns)[:, 0]                          # row i: R e_i - R 0
    slope = cols @ f64(g)[0, 0]
    # each entry of R rounded once, two entries a column; then the inverse call's own bound
    bound = (HALF_STEP * np.abs(cols) + 1.5 * ANGLE * (cols != 0)) @ np.abs(f64(g)[0, 0]) + \
        HALF_STEP * np.abs(want) + ANGLE * 1.01 * size
    assert (np.abs(f64(back)[0, 0] - slope) <= bound * 1.01).all()


def _cached(pa, n, hq, hkv, d, b, rot, interleaved, seed, pad=0.2, layers=1, layer=0, fused=True, mscale=1.0):
    rng = np.random.default_rng(seed)
    nb = -(-n // b) + 3
    shape = (nb, 2, hkv, b, d) if layers == 1 else (nb, 2, layers, hkv, b, d)
    pool = normal(shape, seed)
    if fused:
        qkv = normal((n, hq + 2 * hkv, d), seed + 1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = normal((n, hq, d), seed + 1), normal((n, hkv, d), seed + 2), normal((n, hkv, d), seed + 3)
    slots = rng.permutation(nb * b)[:n].astype(np.int64)
    slots[rng.random(n) < pad] = -1
    positions = rng.integers(0, 200000, size=n)
    w, freqs = ref.angular_frequencies(rot), cuda(pa.rotary_frequencies(rot))
    want = f64(pool)
    view = want if layers == 1 else want[:, :, layer]
    size = np.zeros_like(want)
    sview = size if layers == 1 else size[:, :, layer]
    rk, sk = rotated(f64(k), positions, w, interleaved, mscale)
    for i in range(n):
        if slots[i] >= 0:
            blk, off = slots[i] // b, slots[i] % b
            view[blk, 0, :, off], sview[blk, 0, :, off] = rk[i], sk[i]
            view[blk, 1, :, off] = f64(v)[i]
    q_want, q_size = rotated(f64(q), positions, w, interleaved, mscale)
    q_out = torch.full((n, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pa.rotate_and_cache(pool, q_out if hq else None, q if hq else None, k, v, cuda(positions), cuda(slots), freqs,
                        interleaved=interleaved, mscale=mscale, layer=layer if layers > 1 else None)
    assert pa.get_device_error() == 0
    what = f"n={n} {hq}/{hkv} d={d} b={b} rot={rot}"
    check_rotated(q_out, q_want, q_size, what + " q")
    check_rotated(pool, want, size, what + " pool")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,b,rot", [(1, 4, 2, 64, 16, 64), (64, 64, 8, 128, 16, 128), (37, 28, 4, 64, 32, 32),
                                              (130, 8, 1, 128, 8, 48), (9, 3, 3, 80, 5, 20), (5, 0, 2, 128, 64, 128),
                                              (3, 71, 1, 64, 4, 6), (700, 6, 2, 64, 16, 64)])
def test_rotate_and_cache(pa, n, hq, hkv, d, b, rot, interleaved):
    _cached(pa, n, hq, hkv, d, b, rot, interleaved, seed=n + d, mscale=1.0 if n % 2 else 0.875)


def test_rotate_and_cache_layer_of_a_layered_pool(pa):
    _cached(pa, 33, 8, 2, 64, 16, 64, False, seed=3, layers=3, layer=1, fused=False)


def test_rotate_and_cache_equals_rotate_then_slot_writer(pa):
    """Full-size prefill chunk: the fused call's bits are those of the two calls."""
    w = wl.prefill_chunk(batch=4, ctx=1000, chunk=300, num_blocks=512)
    t = wl.make_tensors(w, "cuda")
    n = w.batch * w.chunk
    q, k, v = t["q"].reshape(n, 64, 128), t["new_k"], t["new_v"]
    slots = cuda(pa.slot_mapping(w.tables, w.new_seq_idx, w.new_positions, 16, w.num_blocks))
    positions, freqs = cuda(w.new_positions), cuda(pa.rotary_frequencies(128))
    pool_a, pool_b = t["pool"], t["pool"].clone()
    qa, qb, kb = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    pa.rotate_and_cache(pool_a, qa, q, k, v, positions, slots, freqs)
    pa.rotate(qb, q, positions, freqs)
    pa.rotate(kb, k, positions, freqs)
    pa.reshape_and_cache(pool_b, kb, v, slots)
    assert torch.equal(qa.view(torch.int16), qb.view(torch.int16))
    assert torch.equal(pool_a.view(torch.int16), pool_b.view(torch.int16))


def test_rotate_and_cache_bad_slot(pa):
    """A slot past the pool raises the bit; its token's q is rotated all the same."""
    pool = normal((4, 2, 2, 16, 64), 1)
    before = bits(pool).copy()
    q, k, v = normal((3, 4, 64), 2), normal((3, 2, 64), 3), normal((3, 2, 64), 4)
    q_out, q_ref = torch.empty_like(q), torch.empty_like(q)
    freqs, positions = cuda(pa.rotary_frequencies(64)), cuda(np.asarray([1, 2, 3]))
    pa.rotate_and_cache(pool, q_out, q, k, v, positions, cuda(np.asarray([64, -1, 2 ** 40])), freqs)
    assert pa.get_device_error() == 2
    pa.rotate(q_ref, q, positions, freqs)
    assert np.array_equal(bits(pool), before) and np.array_equal(bits(q_out), bits(q_ref))


# ---------------------------------------------------------------------------
# compaction
# ---------------------------------------------------------------------------

def _tables(rng, counts, nb, width):
    ids = iter(rng.permutation(nb))
    t = np.full((len(counts), width), -1, np.int32)
    for s, c in enumerate(counts):
        t[s, :c] = [next(ids) for _ in range(c)]
    return t, ids


def _compaction(lens, keeps, b, seed, fork=False, starts=None, width=None):
    rng = np.random.default_rng(seed)
    counts = [-(-L // b) for L in lens]
    nb = sum(counts) * (2 if fork else 1) + 2
    width = width or max(max(counts), 1)
    src, ids = _tables(rng, counts, nb, width)
    dst = src
    if fork:
        dst = np.full_like(src, -1)
        for s, c in enumerate(counts):
            dst[s, :c] = [next(ids) for _ in range(c)]
    keep = np.zeros((len(lens), max(1, max(len(k) for k in keeps))), np.int32)
    for s, k in enumerate(keeps):
        keep[s, :len(k)] = k
    return nb, src, dst, keep, np.asarray([len(k) for k in keeps], np.int32)


def _run_compaction(pa, lens, keeps, hkv, d, b, rot=None, interleaved=False, fork=False, starts=None, seed=0,
                    layers=1, layer=0):
    nb, src, dst, keep, counts = _compaction(lens, keeps, b, seed, fork)
    pool = normal((nb, 2, hkv, b, d) if layers == 1 else (nb, 2, layers, hkv, b, d), seed)
    want = f64(pool)
    size = np.zeros_like(want)
    w = ref.angular_frequencies(rot) if rot else None
    view = want if layers == 1 else want[:, :, layer]
    moved, msize = ref.compact(view, src, dst, keep, counts, starts, w, interleaved)
    if layers == 1:
        want, size = moved, msize
    else:
        want[:, :, layer], size[:, :, layer] = moved, msize
    src_t = cuda(src)
    pa.compact_tokens(pool, src_t, cuda(dst) if fork else src_t, cuda(np.asarray(lens, np.int32)), cuda(keep),
                      cuda(counts), starts=None if starts is None else cuda(np.asarray(starts, np.int32)),
                      freqs=cuda(pa.rotary_frequencies(rot)) if rot else None, interleaved=interleaved,
                      layer=layer if layers > 1 else None)
    assert pa.get_device_error() == 0
    check_rotated(pool, want, size, f"lens={lens[:4]} d={d} b={b} rot={rot} fork={fork}")


def _scattered(rng, L, n):
    return np.sort(rng.permutation(L)[:n])


@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("d,b,rot,interleaved", [(128, 16, None, False), (128, 16, 128, False), (64, 32, 32, True),
                                                 (64, 8, 64, False), (80, 4, 24, True), (128, 64, 20, False),
                                                 (256, 16, 10, False), (72, 5, 6, True)])
def test_compact_subsets(pa, d, b, rot, interleaved, fork):
    """Ragged lengths with empty sequences, one token, everything kept, nothing
    kept, only the last token, scattered halves over several tiles."""
    rng = np.random.default_rng(d + b)
    lens = [0, 1, 40, 40, 65, 200, 331, 130]
    keeps = [np.arange(0), np.arange(1), np.arange(40), np.arange(0), np.asarray([64]), _scattered(rng, 200, 100),
             _scattered(rng, 331, 129), np.concatenate([np.arange(4), np.arange(66, 130)])]
    _run_compaction(pa, lens, keeps, 2, d, b, rot, interleaved, fork, seed=d)


@pytest.mark.parametrize("hkv", [1, 8])
@pytest.mark.parametrize("rot", [None, 64])
def test_compact_long_in_place(pa, hkv, rot):
    """Thousands of rows of one sequence moved by one position, by half the
    length and at random: every tile overwrites what a neighbour has just read."""
    rng = np.random.default_rng(4)
    for keep in (np.arange(1, 4097), np.concatenate([np.arange(4), np.arange(2049, 4097)]),
                 _scattered(rng, 4097, 3000)):
        _run_compaction(pa, [4097], [keep], hkv, 64, 16, rot, seed=9)


def test_compact_many_sequences(pa):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 90, size=150)]
    _run_compaction(pa, lens, [_scattered(rng, L, int(rng.integers(0, L + 1))) for L in lens], 4, 64, 16, 64, seed=2)


def test_compact_accepted_drafts(pa):
    """Rows move from a draft tree's positions to the end of the context."""
    lens, starts = [50, 33, 16, 100], [34, 17, 0, 84]
    keeps = [[34, 36, 41], [17], [3, 4, 15], [99]]
    _run_compaction(pa, lens, [np.asarray(k) for k in keeps], 8, 128, 16, None, starts=starts, seed=3)
    _run_compaction(pa, lens, [np.asarray(k) for k in keeps], 2, 128, 16, 128, starts=starts, seed=3, fork=True)


@pytest.mark.parametrize("d,rot,interleaved", [(80, 16, False), (24, 24, True), (200, 48, True), (256, 256, False),
                                               (8, 2, False), (256, 2, True), (40, 20, False), (72, 24, True),
                                               (256, 48, False)])
def test_compact_head_sizes_in_every_split(pa, d, rot, interleaved):
    """Head sizes whose vectors do not divide a CTA's threads, keys turned whole,
    in part or not, in each way the work is split: a warp a sequence, one CTA, the
    clusters of an ordered pass, and CTAs that share out-of-place tiles."""
    rng = np.random.default_rng(d + rot)
    splits = [([40, 9, 17, 64], [2, 0, 1, 2], 2), ([50 + i for i in range(90)], [25 + i // 3 for i in range(90)], 2),
              ([700, 333, 512], [350, 333, 200], 4), ([2600], [1300], 1), ([900] * 12, [450] * 12, 2)]
    for k, (lens, kept, hkv) in enumerate(splits):
        keeps = [_scattered(rng, L, n) for L, n in zip(lens, kept)]
        for r in (rot, None):
            for fork in (False, True):
                _run_compaction(pa, lens, keeps, hkv, d, 16, r, interleaved, fork, seed=d + k)


def test_compact_layer_of_a_layered_pool(pa):
    rng = np.random.default_rng(6)
    _run_compaction(pa, [100, 37], [_scattered(rng, 100, 50), _scattered(rng, 37, 20)], 2, 64, 16, 64, layers=3,
                    layer=2, seed=7)


def test_compact_bad_values(pa):
    """Bad positions, lengths and table entries raise their bits, touch nothing
    outside the sequence's blocks and leave other sequences right."""
    b, d, hkv = 16, 64, 2
    lens = [64, 64, 64]
    keeps = [np.asarray([5, 9, 30]), np.asarray([1, 8, 20]), np.asarray([2, 3, 50])]

    def run(change):
        nb, src, dst, keep, counts = _compaction(lens, keeps, b, 1)
        a = {"lens": np.asarray(lens, np.int32), "src": src.copy(), "keep": keep, "counts": counts,
             "starts": np.zeros(3, np.int32)}
        change(a)
        pool = normal((nb, 2, hkv, b, d), 11)
        good = ref.compact(f64(pool), src, src, keep * 0 + np.asarray([list(k) for k in keeps]), [0, 0, 3])[0]
        src_t = cuda(a["src"])
        before = f64(pool)
        pa.compact_tokens(pool, src_t, src_t, cuda(a["lens"]), cuda(a["keep"]), cuda(a["counts"]),
                          starts=cuda(a["starts"]))
        err = pa.get_device_error()
        after = f64(pool)
        own = set(src[:2].ravel().tolist())
        for blk in range(nb):
            if blk not in own:
                assert np.array_equal(after[blk], good[blk]), blk
        return err, before, after, src

    def keep(a, s, i, v):
        a["keep"][s, i] = v

    assert run(lambda a: keep(a, 0, 1, 5))[0] == 0x20            # twice the same
    assert run(lambda a: keep(a, 0, 2, 64))[0] == 0x20           # past the length
    assert run(lambda a: keep(a, 0, 0, -1))[0] == 0x20
    assert run(lambda a: a["starts"].__setitem__(0, 6))[0] == 0x20   # would move a row up
    assert run(lambda a: a["starts"].__setitem__(0, 2 ** 31 - 1))[0] == 0x20
    assert run(lambda a: a["starts"].__setitem__(0, -1))[0] == 0x4
    assert run(lambda a: a["lens"].__setitem__(0, 65))[0] == 0x4     # beyond the table
    assert run(lambda a: a["counts"].__setitem__(0, 4))[0] == 0x4    # beyond keep's width
    assert run(lambda a: a["counts"].__setitem__(0, -1))[0] == 0x4
    err, before, after, src = run(lambda a: a["src"].__setitem__((0, 0), 10 ** 6))
    assert err == 0x1
    assert run(lambda a: None)[0] == 0


# ---------------------------------------------------------------------------
# beam selection
# ---------------------------------------------------------------------------

def _score_bound(want, vocab):
    # The sum is an fp32 sum of at most k elements per thread, 256 threads a CTA,
    # slices of 4096 elements or more; a CTA never has more than the whole row.
    k = -(-vocab // 256) + 8
    return 2.0 ** -24 * np.abs(want) + 2.0 ** -22 + 2 * 24 * 2.0 ** -23 + k * 2.0 ** -24


def _select(pa, logits, scores, n, finished=None, end=0):
    G, J, V = logits.shape
    ws = torch.empty(max(1, pa.beam_select_workspace_size(G, J, V, n)), dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)                                       # its contents do not matter
    out = (torch.full((G, n), float("nan"), dtype=torch.float32, device="cuda"),
           torch.full((G, n), -7, dtype=torch.int32, device="cuda"),
           torch.full((G, n), -7, dtype=torch.int32, device="cuda"))
    pa.beam_select(*out, logits, scores, finished=finished, end_token=end, workspace=ws)
    return out


def _check_selection(out, logits, scores, n, finished=None, end=0, what=""):
    got, parents, tokens = (t.cpu().numpy() for t in out)
    G, J, V = logits.shape
    x, s = f64(logits), f64(scores)
    done = None if finished is None else finished.cpu().numpy()
    for g in range(G):
        y = ref.beam_scores(x[g], s[g], None if done is None else done[g], end)
        best, bp, bt = ref.best(y, n)
        bound = _score_bound(np.where(np.isfinite(best), best, 0.0), V)
        # the inputs leave no two neighbours of different beams nearer than the scores are exact
        near = [i for i in range(1, n) if np.isfinite(best[i]) and bp[i] != bp[i - 1] and
                0 < best[i - 1] - best[i] <= 2 * bound[i]]
        assert not near, f"{what}: the inputs themselves leave the order open at {near}"
        assert list(parents[g]) == bp and list(tokens[g]) == bt, f"{what} group {g}"
        inf = np.isinf(best)
        assert np.array_equal(np.isneginf(got[g]), inf), f"{what} group {g}"
        assert (np.abs(got[g][~inf] - best[~inf]) <= bound[~inf]).all(), f"{what} group {g}"


def _random_beams(G, J, V, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((G, J, V), generator=gen) * 3).to(dtype).cuda()
    s = (-20 * torch.rand((G, J), generator=gen)).cuda()
    return x, s


BEAM_CASES = [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 21), (1, 4, 1000, 8), (3, 5, 4097, 10), (2, 2, 8191, 4),
              (5, 1, 2049, 64), (1, 64, 300, 64), (2, 16, 9001, 32), (1, 2, 50257, 4)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,J,V,n", BEAM_CASES)
def test_beam_select(pa, G, J, V, n, dtype):
    x, s = _random_beams(G, J, V, seed=V + J, dtype=dtype)
    _check_selection(_select(pa, x, s, n), x, s, n, what=f"{G}x{J}x{V}")
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_select_ties_and_masks(pa, dtype):
    """Equal rows, rows of one value, of the type's lowest value, of -inf; unused
    and ended beams; fewer candidates than places."""
    V, n, low = 3001, 12, torch.finfo(dtype).min
    x, s = _random_beams(9, 3, V, seed=2, dtype=dtype)
    done = torch.zeros((9, 3), dtype=torch.bool, device="cuda")
    x[0] = 0.0                                           # all equal: by index
    s[0] = torch.tensor([-1.0, -1.0, -1.0])
    x[1, 1] = x[1, 0]                                    # twins
    s[1, 1] = s[1, 0]
    s[2, 1:] = -math.inf                                 # a prompt's first step
    x[3, 0] = low                                        # uniform, however low
    x[3, 1] = -math.inf                                  # nothing left
    x[4] = -math.inf                                     # nothing left at all
    x[5] = -math.inf
    x[5, 1, 77] = 1.0                                    # one candidate
    x[5, 2, [5, 3000]] = -2.0
    done[6, 0] = True                                    # ended
    x[6, 0] = float("nan")                               # and not read
    done[7] = True                                       # all ended
    x[8] = x[8].masked_fill(torch.arange(V, device="cuda") % 7 != 0, low)
    _check_selection(_select(pa, x, s, n, done, 13), x, s, n, done, 13, f"masks {dtype}")
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_select_nan_and_inf(pa, dtype):
    """A row with a NaN or +inf logit and a NaN or +inf beam score count as rows
    without candidates and raise the bit, one at a time."""
    for where in range(4):
        x, s = _random_beams(1, 3, 5000, seed=3, dtype=dtype)
        if where < 2:
            x[0, 1, 4321] = (float("nan"), float("inf"))[where]
        else:
            s[0, 1] = (float("nan"), float("inf"))[where - 2]
        out = _select(pa, x, s, 6)
        assert pa.get_device_error() == 0x40
        x[0, 1] = 0.0
        s[0, 1] = -math.inf
        _check_selection(out, x, s, 6, what=f"bad value {where}")
    x, s = _random_beams(1, 2, 100, seed=4, dtype=dtype)
    x[0, 1] = -math.inf
    x[0, 1, 5] = float("nan")                            # a NaN among -inf only
    _select(pa, x, s, 4)
    assert pa.get_device_error() == 0x40


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_select_crowded_threads(pa, dtype):
    """Large values all on the elements of a few threads, thousands of them: more
    than are ranked at once."""
    V = 131072
    x = torch.full((1, 1, V), -4.0, device="cuda")
    idx = torch.arange(V, device="cuda")
    period = 256 * (8 if dtype == torch.bfloat16 else 4)
    crowd = idx % period < 64
    x[0, 0, crowd] = ((idx[crowd] * 2654435761) % 97).float() / 16
    x = x.to(dtype)
    s = torch.zeros((1, 1), device="cuda")
    _check_selection(_select(pa, x, s, 64), x, s, 64, what="crowded")
    # ascending, descending, and all equal long rows
    ramp = torch.arange(V, dtype=torch.float32, device="cuda") / 4096
    x = torch.stack([ramp, ramp.flip(0), torch.ones_like(ramp)])[:, None].to(dtype)
    s = torch.zeros((3, 1), device="cuda")
    _check_selection(_select(pa, x, s, 16), x, s, 16, what="ramps")
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_select_extreme_values(pa, dtype):
    """Logits far beyond any model's, up to where fp32 steps exceed any score."""
    V = 6001
    x, _ = _random_beams(7, 2, V, seed=8, dtype=torch.float32)
    x[0] *= 1e9
    x[1] = torch.sign(x[1]) * 3e37
    x[2] = x[2] * 1e5 + 2e6
    x[3] = -3e38
    x[3, 0, ::3] = -1e30
    x[4, 0] = 2.0 ** 28
    x[4, 1] = -(2.0 ** 28)
    x[5] = x[5].round() + 2.0 ** 22                      # either side of 2^22, fp32 steps of 1/2
    x[6] = x[6].round() - 2.0 ** 22
    x = x.to(dtype)
    s = torch.zeros((7, 2), device="cuda")
    s[:, 1] = -0.5
    _check_selection(_select(pa, x, s, 9), x, s, 9, what=f"extreme {dtype}")
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("J,V,n", [(3, 20001, 12), (4, 32000, 8), (16, 5000, 64), (1, 70000, 1), (5, 4096, 33),
                                   (20, 70001, 24)])
def test_beam_select_few_groups_and_many(pa, J, V, n, dtype):
    """Few groups take one launch and many take two, with other slices: both are
    right, on rows of all kinds, and a group's place among the others is nothing
    to it."""
    x, s = _random_beams(4, J, V, seed=V, dtype=dtype)
    done = torch.zeros((4, J), dtype=torch.bool, device="cuda")
    x[1] = x[1].masked_fill(torch.arange(V, device="cuda") % 11 != 0, -math.inf)
    x[2, 0] = torch.finfo(dtype).min
    done[2, J - 1] = J > 1
    x[3, :, V // 2:] = x[3, :, :1]
    few = _select(pa, x, s, n, done, V - 1)
    _check_selection(few, x, s, n, done, V - 1, f"few {J}x{V}")
    many = _select(pa, x.repeat(30, 1, 1), s.repeat(30, 1), n, done.repeat(30, 1), V - 1)
    for a in many:
        assert torch.equal(a.view(30, 4, n), a.view(30, 4, n)[:1].expand(30, 4, n))
    _check_selection(tuple(a[:4] for a in many), x, s, n, done, V - 1, f"many {J}x{V}")
    assert torch.equal(few[1], many[1][:4]) and torch.equal(few[2], many[2][:4])
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("G,J,V,n", [(2, 4, 9000, 8), (50, 4, 9000, 8)])
def test_beam_select_captured_in_either_form(pa, G, J, V, n):
    """One launch or two, replayed on new logits in the same buffers."""
    x, s = _random_beams(G, J, V, seed=G, dtype=torch.bfloat16)
    ws = torch.empty(pa.beam_select_workspace_size(G, J, V, n), dtype=torch.uint8, device="cuda")
    out = tuple(torch.empty((G, n), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
    pa.beam_select(*out, x, s, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.beam_select(*out, x, s, workspace=ws)
        pa.beam_select(*out, x, s, workspace=ws)         # the second overtakes nothing of the first
    for seed in range(3):
        y, _ = _random_beams(G, J, V, seed=100 + seed, dtype=torch.bfloat16)
        x.copy_(y)
        graph.replay()
        want = _select(pa, y, s, n)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    _check_selection(out, x, s, n, what=f"replayed {G}x{J}")
    assert pa.get_device_error() == 0


def test_beam_select_equal_rows_at_any_alignment(pa):
    """Twin beams have equal sums, and so equal scores, wherever their rows
    begin: their candidates alternate, the lower beam first."""
    for dtype, V in ((torch.bfloat16, 5003), (torch.float32, 9997), (torch.bfloat16, 40001)):
        x, s = _random_beams(1, 8, V, seed=9, dtype=dtype)
        x[0, 1:] = x[0, 0]
        s.fill_(-3.0)
        out = _select(pa, x, s, 24)
        _check_selection(out, x, s, 24, what=f"twins {dtype} {V}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stride", [2050, 2051, 2500])
def test_beam_select_strided_rows(pa, stride, dtype):
    V = 2049
    wide, s = _random_beams(3, 4, stride, seed=6, dtype=dtype)
    wide[..., V:] = 1000.0                               # what lies behind a row is not read into it
    x = wide[..., :V]
    _check_selection(_select(pa, x, s, 8), x, s, 8, what=f"stride {stride}")


def test_beam_select_repeats_and_streams(pa):
    """Same bits call after call on one workspace, and on a side stream."""
    x, s = _random_beams(8, 4, 32000, seed=7, dtype=torch.bfloat16)
    first = [t.clone() for t in _select(pa, x, s, 8)]
    ws = torch.empty(pa.beam_select_workspace_size(8, 4, 32000, 8), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        out = [torch.empty_like(t) for t in first]
        pa.beam_select(*out, x, s, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in first]
    with torch.cuda.stream(side):
        pa.beam_select(*out, x, s, workspace=ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_binding_refusals(pa):
    pool = normal((4, 2, 2, 16, 64), 1)
    k = normal((2, 2, 64), 2)
    pos, slots, freqs = cuda(np.asarray([1, 2])), cuda(np.asarray([3, 4])), cuda(pa.rotary_frequencies(64))
    with pytest.raises(ValueError):
        pa.rotate_and_cache(pool, None, normal((2, 4, 64), 1), k, k, pos, slots, freqs)
    with pytest.raises(ValueError):
        pa.rotate_and_cache(pool, None, None, k.transpose(0, 1), k, pos, slots, freqs)
    with pytest.raises(ValueError):
        pa.rotate_and_cache(pool, None, None, k, k, pos[:1], slots, freqs)
    with pytest.raises(TypeError):
        pa.rotate_and_cache(pool, None, None, k.float(), k, pos, slots, freqs)
    with pytest.raises(TypeError):
        pa.rotate(k, k, pos.int(), freqs)
    with pytest.raises(pa.PagedAttentionError):
        pa.rotate(k, k, pos, cuda(pa.rotary_frequencies(128)))            # more than the head has
    table = cuda(np.zeros((1, 4), np.int32))
    one = cuda(np.ones(1, np.int32))
    with pytest.raises(ValueError):
        pa.compact_tokens(pool, table, table[:, :2].contiguous(), one, cuda(np.zeros((1, 1), np.int32)), one)
    with pytest.raises(ValueError):
        pa.compact_tokens(pool, table, table, one, cuda(np.zeros((2, 1), np.int32)), one)
    x, s = _random_beams(1, 2, 64, seed=1, dtype=torch.float32)
    with pytest.raises(TypeError):
        _select(pa, x.half(), s, 2)
    with pytest.raises(ValueError):
        _select(pa, x, s[:, :1], 2)
    with pytest.raises(ValueError):
        _select(pa, x.transpose(1, 2), s.new_zeros((1, 64)), 2)
    with pytest.raises(pa.PagedAttentionError):
        pa.beam_select(torch.empty((1, 2), device="cuda"), one.new_empty((1, 2)), one.new_empty((1, 2)), x, s)


def test_captured_and_replayed(pa):
    """All three in one graph, replayed on changed inputs."""
    x, s = _random_beams(2, 4, 5003, seed=9, dtype=torch.float32)
    pool = normal((12, 2, 2, 16, 64), 1)
    q, k, v = normal((8, 4, 64), 2), normal((8, 2, 64), 3), normal((8, 2, 64), 4)
    pos, slots = cuda(np.arange(8)), cuda(np.arange(8))
    freqs = cuda(pa.rotary_frequencies(64))
    table = cuda(np.arange(12, dtype=np.int32)[None])
    lens, counts = cuda(np.asarray([100], np.int32)), cuda(np.asarray([40], np.int32))
    keep = cuda(np.arange(20, 60, dtype=np.int32)[None])
    ws = torch.empty(pa.beam_select_workspace_size(2, 4, 5003, 8), dtype=torch.uint8, device="cuda")

    def run(q_out, p, out):
        pa.rotate_and_cache(p, q_out, q, k, v, pos, slots, freqs)
        pa.compact_tokens(p, table, table, lens, keep, counts, freqs=freqs)
        pa.beam_select(*out, x, s, workspace=ws)

    new = lambda: (torch.empty_like(q), pool.clone(), (torch.empty((2, 8), device="cuda"),  # noqa: E731
                   torch.empty((2, 8), dtype=torch.int32, device="cuda"),
                   torch.empty((2, 8), dtype=torch.int32, device="cuda")))
    run(*new())
    torch.cuda.synchronize()
    held = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*held)
    x.add_(torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    held[1].copy_(pool)
    graph.replay()
    eager = new()
    run(*eager)
    torch.cuda.synchronize()
    assert torch.equal(held[0], eager[0]) and torch.equal(held[1], eager[1])
    assert all(torch.equal(a, b) for a, b in zip(held[2], eager[2]))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("hkv,rot", [(8, None), (2, 64), (1, 10), (3, None)])
def test_compact_clusters_captured_and_beside_other_work(pa, hkv, rot):
    """Long in-place compactions that clusters of CTAs share, captured and
    replayed, while another stream copies memory: the same bits as an eager run
    of the out-of-place form into fresh blocks."""
    b, d, L = 16, 64, 20000
    rng = np.random.default_rng(hkv)
    keep = _scattered(rng, L, 12000)
    width = -(-L // b)
    ids = rng.permutation(2 * width).astype(np.int32)
    src, fresh = cuda(ids[None, :width].copy()), cuda(ids[None, width:].copy())
    start = normal((2 * width, 2, hkv, b, d), 5)
    lens, counts = cuda(np.asarray([L], np.int32)), cuda(np.asarray([len(keep)], np.int32))
    keep_t = cuda(keep.astype(np.int32)[None])
    freqs = cuda(pa.rotary_frequencies(rot)) if rot else None
    other = start.clone()
    pa.compact_tokens(other, src, fresh, lens, keep_t, counts, freqs=freqs)
    order = torch.as_tensor(ids.astype(np.int64), device="cuda")
    at = torch.arange(len(keep), device="cuda")
    want = other[order[width:][at // b], :, :, at % b]
    pool = start.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.compact_tokens(pool, src, src, lens, keep_t, counts, freqs=freqs)
    side, junk = torch.cuda.Stream(), torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    target = torch.empty_like(junk)
    for _ in range(6):
        pool.copy_(start)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            target.copy_(junk)
        graph.replay()
        torch.cuda.synchronize()
        got = pool[order[:width][at // b], :, :, at % b]
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        # rows behind the last one, and blocks of nobody, as they were
        rest = torch.arange(len(keep), L, device="cuda")
        assert torch.equal(pool[order[:width][rest // b], :, :, rest % b],
                           start[order[:width][rest // b], :, :, rest % b])
        assert torch.equal(pool[order[width:]], start[order[width:]])
    assert pa.get_device_error() == 0


def test_compact_fork_keeps_a_common_beginning_and_refuses_its_own_blocks(pa):
    """Equal table entries for unmoved rows are fine out of place; a row that
    would move into a block the sequence still reads is refused."""
    b, d, hkv, L = 16, 64, 2, 160
    rng = np.random.default_rng(8)
    ids = rng.permutation(24).astype(np.int32)
    src = ids[None, :10].copy()
    dst = np.concatenate([ids[:3], ids[10:17]])[None].copy()      # three shared blocks, then fresh ones
    keep = np.concatenate([np.arange(48), 48 + _scattered(rng, 112, 60)])
    pool = normal((24, 2, hkv, b, d), 9)
    want, size = ref.compact(f64(pool), src, dst, keep[None], [len(keep)], None, ref.angular_frequencies(64), False)
    args = (cuda(np.asarray([L], np.int32)), cuda(keep.astype(np.int32)[None]), cuda(np.asarray([len(keep)], np.int32)))
    pa.compact_tokens(pool, cuda(src), cuda(dst), *args, freqs=cuda(pa.rotary_frequencies(64)))
    assert pa.get_device_error() == 0
    check_rotated(pool, want, size, "common beginning")
    clone = pool.clone()
    pa.compact_tokens(pool, cuda(src), cuda(src.copy()), *args)      # another tensor of the same blocks
    assert pa.get_device_error() == 0x1
    moved = keep != np.arange(len(keep))
    assert moved.any() and torch.equal(pool, clone)


def test_offsets_beyond_32_bits(pa):
    """Slots and rows behind 2^32 bytes of one pool."""
    nb, hkv, b, d = 70000, 8, 16, 128                               # 4.6 GB
    pool = torch.zeros((nb, 2, hkv, b, d), dtype=torch.bfloat16, device="cuda")
    high = np.asarray([69999, 65537, 66000, 3], np.int32)
    n = 64
    k, v = normal((n, hkv, d), 1), normal((n, hkv, d), 2)
    slots = (high.astype(np.int64)[:, None] * b + np.arange(b)).ravel()
    w, freqs = ref.angular_frequencies(d), cuda(pa.rotary_frequencies(d))
    pa.rotate_and_cache(pool, None, None, k, v, cuda(np.arange(n)), cuda(slots), freqs)
    rows, sizes = rotated(f64(k), np.arange(n), w, False)
    at = torch.as_tensor(high.astype(np.int64), device="cuda")
    got = pool[at]                                                   # [4][2][Hkv][b][d]
    check_rotated(got[:, 0].transpose(1, 2).reshape(n, hkv, d), rows, sizes, "slots")
    assert torch.equal(got[:, 1].transpose(1, 2).reshape(n, hkv, d), v)
    keep = np.arange(1, 64, 2)
    table = cuda(high[None].copy())
    pa.compact_tokens(pool, table, table, cuda(np.asarray([n], np.int32)), cuda(keep.astype(np.int32)[None]),
                      cuda(np.asarray([len(keep)], np.int32)))
    after = pool[at]
    flat, old = after.transpose(2, 3).reshape(4, 2, b, hkv, d), got.transpose(2, 3).reshape(4, 2, b, hkv, d)
    for i, p in enumerate(keep):
        assert torch.equal(flat[i // b, :, i % b], old[p // b, :, p % b])
    assert pa.get_device_error() == 0
    pool[at] = 0
    assert int(torch.count_nonzero(pool.view(torch.int64).view(-1))) == 0   # nothing else was touched


def test_beam_select_offsets_beyond_32_bits(pa):
    """More than 2^31 logits: one spike a row, the last rows read right."""
    rows, V = 300, 7_500_001
    x = torch.zeros((rows, 1, V), dtype=torch.bfloat16, device="cuda")
    spike = (torch.arange(rows, device="cuda") * 24593 + 12345) % V
    x[torch.arange(rows, device="cuda"), 0, spike] = 20.0
    s = torch.zeros((rows, 1), device="cuda")
    scores, parents, tokens = _select(pa, x, s, 2)
    assert torch.equal(tokens[:, 0].long(), spike) and not parents.any()
    assert torch.equal(tokens[:, 1].long(), torch.where(spike == 0, 1, 0))
    want = -math.log1p((V - 1) * math.exp(-20.0))
    # the sum of equal small terms: 2^-22 each (the hardware's 2^x), and a thread's
    # additions, at most V / 256 of them, one half step each
    tol = 2.0 ** -22 + (V / 256 + 64) * 2.0 ** -24
    assert float((scores[:, 0] - want).abs().max()) <= tol
    assert float((scores[:, 1] - (want - 20.0)).abs().max()) <= tol + 2.0 ** -19
    assert pa.get_device_error() == 0


def test_two_streams_at_once(pa):
    """The same calls on two streams at the same time, each with its own buffers."""
    x, s = _random_beams(16, 4, 40000, seed=12, dtype=torch.bfloat16)
    pool0 = normal((300, 2, 4, 16, 64), 1)
    q, k, v = normal((512, 8, 64), 2), normal((512, 4, 64), 3), normal((512, 4, 64), 4)
    pos, slots = cuda(np.arange(512)), cuda(np.arange(512) + 7)
    freqs = cuda(pa.rotary_frequencies(64))
    table = cuda(np.arange(300, dtype=np.int32)[None])
    keep = cuda(np.arange(1000, 4000, dtype=np.int32)[None])
    lens, counts = cuda(np.asarray([4500], np.int32)), cuda(np.asarray([3000], np.int32))
    nbytes = pa.beam_select_workspace_size(16, 4, 40000, 8)

    def buffers():
        return (pool0.clone(), torch.empty_like(q), torch.empty(nbytes, dtype=torch.uint8, device="cuda"),
                (torch.empty((16, 8), device="cuda"), torch.empty((16, 8), dtype=torch.int32, device="cuda"),
                 torch.empty((16, 8), dtype=torch.int32, device="cuda")))

    def run(held, stream):
        pool, q_out, ws, out = held
        pa.rotate_and_cache(pool, q_out, q, k, v, pos, slots, freqs, stream=stream)
        pa.compact_tokens(pool, table, table, lens, keep, counts, freqs=freqs, stream=stream)
        pa.beam_select(*out, x, s, workspace=ws, stream=stream)

    alone = buffers()
    run(alone, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    held = [buffers() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for (pool, *_rest), stream in zip(held, streams):
            with torch.cuda.stream(stream):
                pool.copy_(pool0)
        for h, stream in zip(held, streams):
            run(h, stream)
    torch.cuda.synchronize()
    for pool, q_out, _, out in held:
        assert torch.equal(pool, alone[0]) and torch.equal(q_out, alone[1])
        assert all(torch.equal(a, b) for a, b in zip(out, alone[3]))
    assert pa.get_device_error() == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_beam_decode_with_rotary_and_a_sliding_window(pa):
    """Two prompts of three beams over several steps, as a serving loop runs them:
    rotary positions into the cache, decode, a stand-in projection to logits, the
    selection, the reordering with copy-on-write; once the contexts reach a limit
    each beam's cache slides to four first tokens and the latest ones with its
    keys turned back.  The cache of every beam is checked row by row against its
    history replayed in fp64, and decode against attention over it."""
    hq, hkv, d, b, V, beams, prompts, steps = 8, 2, 64, 16, 97, 3, 2, 14
    limit, kept = 44, 24
    nb, scale = 64, d ** -0.5
    gen = torch.Generator().manual_seed(21)
    embed_q, embed_k, embed_v = (torch.randn((V, h, d), generator=gen).to(torch.bfloat16) for h in (hq, hkv, hkv))
    head = (torch.randn((hq * d, V), generator=gen) * 0.2).cuda()
    w, freqs = ref.angular_frequencies(d), cuda(pa.rotary_frequencies(d))
    pool = torch.zeros((nb, 2, hkv, b, d), dtype=torch.bfloat16, device="cuda")
    bm = pa.BlockManager(nb, b)
    # a beam's state on the host: the tokens of its cached rows, in order, with fp64 key and value rows
    seqs, state = [], []
    for p in range(prompts):
        s = bm.add_seq()
        tokens = torch.randint(0, V, (31 + p,), generator=gen).numpy()
        slots, _ = bm.append_tokens(s, len(tokens))
        k, v = embed_k[tokens].cuda(), embed_v[tokens].cuda()
        pa.rotate_and_cache(pool, None, None, k, v, cuda(np.arange(len(tokens))), cuda(slots), freqs)
        rows = [(ref.rotate(f64(k)[i], i, w, False), f64(v)[i], 1) for i in range(len(tokens))]
        seqs.append([s] + [bm.fork(s) for _ in range(beams - 1)])
        state.append([list(rows) for _ in range(beams)])
    flat = [s for group in seqs for s in group]
    last = torch.randint(0, V, (prompts * beams,), generator=gen)
    scores = torch.full((prompts, beams), -math.inf)
    scores[:, 0] = 0.0
    scores = scores.cuda()
    ws = torch.empty(pa.beam_select_workspace_size(prompts, beams, V, beams), dtype=torch.uint8, device="cuda")
    slides = 0
    for step in range(steps):
        if max(bm.table(s)[1] for s in flat) >= limit:
            slides += 1
            pairs = [pair for s in flat for pair in bm.unshare(s)]
            if pairs:
                pa.copy_blocks(pool, cuda(np.asarray(pairs, np.int32)))
            info = [bm.table(s) for s in flat]
            width = max(len(t) for t, _ in info)
            tables = np.full((len(flat), width), -1, np.int32)
            for i, (t, _) in enumerate(info):
                tables[i, :len(t)] = t
            keeps = [np.concatenate([np.arange(4), np.arange(n - kept + 4, n)]).astype(np.int32) for _, n in info]
            t = cuda(tables)
            pa.compact_tokens(pool, t, t, cuda(np.asarray([n for _, n in info], np.int32)), cuda(np.stack(keeps)),
                              cuda(np.full(len(flat), kept, np.int32)), freqs=freqs)
            for i, s in enumerate(flat):
                bm.truncate(s, kept)
                rows = state[i // beams][i % beams]
                out = []
                for new, old in enumerate(keeps[i]):
                    (k, size), v, rounds = rows[old]
                    if new != old:
                        (k, more), rounds = ref.rotate(k, new - int(old), w, False), rounds + 1
                        size = np.maximum(size, more)
                    out.append(((k, size), v, rounds))
                state[i // beams][i % beams] = out
        # one step: every beam appends its last token
        positions, slots, pairs = [], [], []
        for s in flat:
            positions.append(bm.table(s)[1])
            slot, cow = bm.append_tokens(s, 1)
            slots.append(slot[0])
            if cow:
                pairs.append(cow)
        if pairs:
            pa.copy_blocks(pool, cuda(np.asarray(pairs, np.int32)))
        q, k, v = embed_q[last].cuda(), embed_k[last].cuda(), embed_v[last].cuda()
        q_rot = torch.empty_like(q)
        pa.rotate_and_cache(pool, q_rot, q, k, v, cuda(np.asarray(positions)), cuda(np.asarray(slots)), freqs)
        for i in range(len(flat)):
            state[i // beams][i % beams].append((ref.rotate(f64(k)[i], positions[i], w, False), f64(v)[i], 1))
        info = [bm.table(s) for s in flat]
        width = max(len(t) for t, _ in info)
        tables = np.full((len(flat), width), -1, np.int32)
        for i, (t, _) in enumerate(info):
            tables[i, :len(t)] = t
        lens = np.asarray([n for _, n in info], np.int32)
        out = torch.empty_like(q)
        nbytes = pa.decode_workspace_size(pool, len(flat), hq, int(lens.max()), 0)
        pa.decode(out, q_rot, pool, cuda(tables), cuda(lens), int(lens.max()), scale, 0,
                  torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda"))
        # the cache against the replayed history
        host = f64(pool)
        for i, (t, n) in enumerate(info):
            rows = state[i // beams][i % beams]
            assert len(rows) == n
            for pos, ((kr, size), vr, rounds) in enumerate(rows):
                got_k, got_v = host[t[pos // b], 0, :, pos % b], host[t[pos // b], 1, :, pos % b]
                # each rounding is off by half a step of its own value, at most 2^-8 of the pair's size,
                # and a later rotation mixes the pair's two errors
                tol = rounds * (2 * HALF_STEP + ANGLE) * size * 1.02
                assert (np.abs(got_k - kr) <= tol).all(), (step, i, pos)
                assert np.array_equal(got_v, vr)
            # decode over the cached rows themselves
            keys = np.stack([host[t[p // b], 0, :, p % b] for p in range(n)])
            vals = np.stack([host[t[p // b], 1, :, p % b] for p in range(n)])
            for h in range(hq):
                a = scale * keys[:, h * hkv // hq] @ f64(q_rot)[i, h]
                a = np.exp(a - a.max())
                want = (a / a.sum()) @ vals[:, h * hkv // hq]
                assert (np.abs(f64(out)[i, h] - want) <= np.maximum(4e-3, 1e-2 * np.abs(want))).all()
        logits = (out.reshape(len(flat), hq * d).float() @ head).reshape(prompts, beams, V)
        best = (torch.empty((prompts, beams), device="cuda"),
                torch.empty((prompts, beams), dtype=torch.int32, device="cuda"),
                torch.empty((prompts, beams), dtype=torch.int32, device="cuda"))
        pa.beam_select(*best, logits, scores, workspace=ws)
        _check_selection(best, logits, scores, beams, what=f"step {step}")
        parents = best[1].cpu().numpy()
        for p in range(prompts):
            bm.reorder(seqs[p], parents[p])
            state[p] = [list(state[p][int(j)]) for j in parents[p]]
        scores, last = best[0], best[2].cpu().reshape(-1).long()
    assert slides >= 1 and pa.get_device_error() == 0
