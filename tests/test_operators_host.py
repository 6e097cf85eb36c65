"""Rotary frequencies, the block manager's reorder / unshare / truncate, and the
host-side refusals of the rotary, compaction and beam-selection calls (no GPU)."""
import ctypes
import math
import random

import numpy as np
import pytest

from oracle import operators as ref


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from paged_kv_cache_167_gb300 import binding
    return binding


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192, low=1.0, high=4.0),
            dict(scaling="parts", factor=32.0, original_len=2048, low=1.0, high=32.0),
            dict(scaling="parts_index", factor=16.0, original_len=4096, low=1.0, high=32.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot", [2, 8, 24, 64, 128, 130])
def test_rotary_frequencies(B, kw, rot):
    """2^-64 turn fractions of the formula's frequencies.  Two fp64 evaluations of
    base^e with 0 >= e > -1 differ, in units of u = 2^-53, by 2 ln(base) (the
    exponents' roundings, each moved by the logarithm of the base), by 6 (the
    scaled base's own power, product and quotient) and by 10 for the remaining
    powers, products and quotients: R = 16 + 2 ln(base).  The mix of the by-parts
    form has g = (turns - low) / (high - low) with turns <= high wherever g is not
    clamped, so g is off by at most (R + 4) high / (high - low), and w' = w ((1 - g) / s + g)
    >= w / s by s times that, relative."""
    w = np.asarray(ref.angular_frequencies(rot, **kw))
    turns = B.rotary_frequencies(rot, **kw).view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert turns.shape == (rot // 2,)
    want = w / (2 * math.pi)
    base, s = kw.get("base", 10000.0), kw.get("factor", 1.0)
    if kw.get("scaling") == "base" and rot > 2:
        base *= s ** (rot / (rot - 2))
    bound = 16 + 2 * math.log(base)
    if kw.get("scaling") == "parts":
        bound += s * (bound + 4) * kw["high"] / (kw["high"] - kw["low"])
    assert (np.abs(turns - want) <= bound * 2.0 ** -53 * want + 2.0 ** -64).all()


def test_rotary_turns_wrap(B):
    """Whole turns drop out, negative frequencies wrap, an exact half is exact."""
    t = B.rotary_turns([0.0, math.pi, -math.pi / 2, 2 * math.pi * 5 + math.pi, -1e-300]).view(np.uint64)
    assert t[0] == 0 and t[1] == 2 ** 63 and t[2] == 3 * 2 ** 62 and t[4] == 0
    assert abs(float(t[3]) / 2.0 ** 64 - 0.5) <= 6 * 2.0 ** -52
    assert len(B.rotary_turns([])) == 0


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=math.nan),
                                dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.inf),
                                dict(scaling="parts", factor=2.0, original_len=0.0),
                                dict(scaling="parts", factor=2.0, original_len=4096, low=4.0, high=4.0),
                                dict(scaling="parts_index", factor=2.0, original_len=4096, low=0.0),
                                dict(scaling="base", factor=1e300, base=1e300)])
def test_rotary_refusals(B, kw):
    kw.setdefault("rot_dim", 64)
    with pytest.raises(B.PagedAttentionError) as e:
        B.rotary_frequencies(**kw)
    assert e.value.status == 1


def test_rotary_more_refusals(B):
    with pytest.raises(B.PagedAttentionError):
        B.rotary_turns([1.0, math.inf])
    with pytest.raises(ValueError):
        B.rotary_frequencies(64, scaling="none")
    assert B.lib().pa_rotary_frequencies(None, None) == 1
    assert B.lib().pa_rotary_turns(None, -1, None) == 1


def _pool(B, base=0x10000, nb=64, hkv=8, b=16, d=128, bstride=0, kvstride=0, dtype=0):
    return B.PaKvPool(base, nb, hkv, b, d, dtype, bstride, kvstride)


def test_device_call_refusals(B):
    """Bad arguments give a status on the host; nothing is launched (there is no
    GPU here, and the pointers are no memory)."""
    L, P = B.lib(), ctypes.c_void_p
    ok, null, odd = P(0x20000), P(0), P(0x20008)
    rot = lambda turns=0x30000, r=128, flags=0, m=1.0: ctypes.byref(B.PaRotary(turns, r, flags, m))  # noqa: E731

    def rotate(out=ok, x=ok, stride=0, pos=ok, n=4, heads=8, d=128, rotary=None):
        return L.pa_rotate(out, x, stride, pos, n, heads, d, rotary or rot(), null)

    assert rotate(n=0) == 0 and rotate(heads=0) == 0
    assert rotate(n=-1) == 1 and rotate(n=2 ** 31) == 1 and rotate(heads=65536) == 1 and rotate(d=0) == 1
    assert rotate(d=100) == 2 and rotate(d=2048) == 2
    assert rotate(out=null) == 1 and rotate(x=odd) == 1 and rotate(pos=null) == 1
    assert rotate(stride=8 * 128 - 8) == 1 and rotate(stride=8 * 128 + 4) == 1     # overlapping, not whole vectors
    for bad in (rot(turns=0), rot(turns=0x30004), rot(r=0), rot(r=65), rot(r=136), rot(flags=4), rot(m=math.nan),
                rot(m=math.inf)):
        assert rotate(rotary=bad) == 1
    assert L.pa_rotate(ok, ok, 0, ok, 4, 8, 128, None, null) == 1

    def cached(pool=None, qo=ok, q=ok, qs=0, k=ok, ks=0, v=ok, vs=0, pos=ok, slots=ok, n=4, hq=64, rotary=None):
        return L.pa_rotate_and_cache(ctypes.byref(pool or _pool(B)), qo, q, qs, k, ks, v, vs, pos, slots, n, hq,
                                     rotary or rot(), null)

    assert cached(n=0) == 0 and cached(n=0, hq=0, q=null, qo=null) == 0
    assert cached(pool=_pool(B, base=0x10001)) == 1 and cached(pool=_pool(B, dtype=1)) == 2
    assert cached(pool=_pool(B, d=2048)) == 2
    assert cached(n=-1) == 1 and cached(hq=-1) == 1 and cached(hq=65535) == 1
    assert cached(k=null) == 1 and cached(v=odd) == 1 and cached(pos=null) == 1 and cached(slots=null) == 1
    assert cached(q=null) == 1 and cached(qo=odd) == 1
    assert cached(ks=8 * 128 - 8) == 1 and cached(vs=1025) == 1 and cached(qs=64 * 128 - 8) == 1
    assert cached(rotary=rot(r=130)) == 1

    def compact(pool=None, src=ok, dst=ok, width=8, lens=ok, keep=ok, most=16, counts=ok, starts=null, n=2,
                rotary=None):
        return L.pa_compact_tokens(ctypes.byref(pool or _pool(B)), src, dst, width, lens, keep, most, counts, starts,
                                   n, rotary, null)

    assert compact(n=0) == 0 and compact(most=0) == 0
    assert compact(pool=_pool(B, d=264)) == 2 and compact(pool=_pool(B, nb=0)) == 1
    assert compact(n=-1) == 1 and compact(n=65536) == 1 and compact(most=-1) == 1 and compact(width=0) == 1
    for name in ("src", "dst", "lens", "keep", "counts"):
        assert compact(**{name: null}) == 1
    assert compact(rotary=rot(r=256)) == 1 and compact(rotary=rot(turns=0)) == 1

    size = L.pa_beam_select_workspace_size(4, 4, 32000, 8)
    assert size > 0 and size % 256 == 0

    def select(out=ok, logits=ok, dtype=0, stride=0, scores=ok, done=null, end=0, groups=4, beams=4, vocab=32000,
               n=8, ws=ok, ws_bytes=size):
        return L.pa_beam_select(out, ok, ok, logits, dtype, stride, scores, done, end, groups, beams, vocab, n, ws,
                                ws_bytes, null)

    assert select(groups=0) == 0
    assert select(groups=-1) == 1 and select(beams=0) == 1 and select(vocab=0) == 1 and select(n=0) == 1
    assert select(beams=1, vocab=7, n=8) == 1                     # more than there are
    assert select(beams=64, vocab=2 ** 26, n=8) == 1              # flat index beyond 31 bits
    assert select(groups=16384) == 1                              # rows beyond the grid
    assert select(beams=65) == 2 and select(n=65) == 2 and select(dtype=2) == 2
    assert select(stride=31999) == 1 and select(logits=odd) == 1 and select(out=null) == 1 and select(scores=null) == 1
    assert select(done=ok, end=-1) == 1 and select(done=ok, end=32000) == 1
    assert select(ws=null) == 3 and select(ws_bytes=size - 1) == 3 and select(ws=P(0x20010)) == 3
    for shape in ((-1, 4, 100, 8), (1, 65, 100, 8), (1, 4, 100, 65), (1, 1, 4, 8), (0, 4, 100, 8)):
        assert L.pa_beam_select_workspace_size(*shape) == 0


@pytest.fixture()
def bm(B):
    from paged_kv_cache_167_gb300 import BlockManager
    return BlockManager


def _check_counts(m, seqs, cached=()):
    """Every block's count is the number of tables (and cache entries) holding it."""
    count = {}
    for s in seqs:
        for blk in m.table(s)[0]:
            count[int(blk)] = count.get(int(blk), 0) + 1
    for blk in cached:
        count[int(blk)] = count.get(int(blk), 0) + 1
    for blk in range(m.num_blocks):
        assert m.refcount(blk) == count.get(blk, 0), blk
    assert m.num_free() == m.num_blocks - len(count)


def test_reorder(bm):
    m = bm(32, 4)
    seqs = []
    for n in (5, 9, 2):
        s = m.add_seq()
        m.append_tokens(s, n)
        seqs.append(s)
    old = [m.table(s) for s in seqs]
    m.reorder(seqs, [1, 1, 0])                       # beam 2's blocks go, beam 1 goes on twice
    for j, p in enumerate((1, 1, 0)):
        t, n = m.table(seqs[j])
        assert np.array_equal(t, old[p][0]) and n == old[p][1]
    _check_counts(m, seqs)
    # the shared partly filled block forks on the first append, and only then
    _, cow = m.append_tokens(seqs[0], 1)
    assert cow is not None and cow[0] == old[1][0][-1]
    _, cow = m.append_tokens(seqs[1], 1)
    assert cow is None
    _check_counts(m, seqs)
    m.reorder(seqs, [0, 1, 2])                       # nothing changes
    m.reorder([], [])
    _check_counts(m, seqs)


def test_reorder_refusals(B, bm):
    m = bm(16, 4)
    a, b = m.add_seq(), m.add_seq()
    m.append_tokens(a, 6)
    before = m.table(a)[0].copy()
    for seqs, parents, status in (([a, b], [0, 2], 1), ([a, b], [0, -1], 1), ([a, a], [0, 1], 1),
                                  ([a, 99], [0, 1], 7)):
        with pytest.raises(B.PagedAttentionError) as e:
            m.reorder(seqs, parents)
        assert e.value.status == status
    with pytest.raises(ValueError):
        m.reorder([a, b], [0])
    m.set_host_pool(4)
    m.swap_out(b)
    with pytest.raises(B.PagedAttentionError) as e:
        m.reorder([a, b], [0, 0])
    assert e.value.status == 8
    assert np.array_equal(m.table(a)[0], before)
    _check_counts(m, [a])


def test_truncate(B, bm):
    m = bm(16, 4)
    a = m.add_seq()
    m.append_tokens(a, 14)
    b = m.fork(a)
    m.truncate(a, 5)
    assert m.table(a)[1] == 5 and len(m.table(a)[0]) == 2 and len(m.table(b)[0]) == 4
    _check_counts(m, [a, b])
    _, cow = m.append_tokens(a, 1)                   # block 1 is shared and now partly filled here
    assert cow is not None
    _check_counts(m, [a, b])
    m.truncate(a, 0)
    assert len(m.table(a)[0]) == 0
    _check_counts(m, [a, b])
    for n, status in ((1, 1), (-1, 1)):
        with pytest.raises(B.PagedAttentionError) as e:
            m.truncate(a, n)
        assert e.value.status == status
    with pytest.raises(B.PagedAttentionError):
        m.truncate(77, 0)


def test_unshare(B, bm):
    m = bm(16, 4)
    a = m.add_seq()
    m.append_tokens(a, 14)
    b = m.fork(a)
    old = m.table(a)[0].copy()
    pairs = m.unshare(a, 7)                          # blocks 1, 2, 3
    new = m.table(a)[0]
    assert new[0] == old[0] and np.array_equal(pairs, np.stack([old[1:], new[1:]], axis=1))
    assert not set(new[1:]) & set(old)
    _check_counts(m, [a, b])
    assert len(m.unshare(b, 4)) == 0                 # nobody else holds them any more
    assert len(m.unshare(a, 100)) == 0
    for seq, first, status in ((a, -1, 1), (99, 0, 7)):
        with pytest.raises(B.PagedAttentionError) as e:
            m.unshare(seq, first)
        assert e.value.status == status
    small = bm(5, 4)
    c = small.add_seq()
    small.append_tokens(c, 12)
    small.fork(c)
    before = small.table(c)[0].copy()
    with pytest.raises(B.PagedAttentionError) as e:
        small.unshare(c)                             # three shared, two free
    assert e.value.status == 6
    n = ctypes.c_int32()
    assert B.lib().pa_bm_unshare(small._h, c, 8, None, 0, ctypes.byref(n)) == 1      # no room for the pair
    assert np.array_equal(small.table(c)[0], before)


def test_unshare_under_eviction_pairs_never_chain(bm):
    """All blocks of the pool in use or cached: the fresh blocks come from
    evicted cache entries, and no block is both a source and a destination."""
    m = bm(8, 4)
    a = m.add_seq()
    m.append_tokens(a, 16)
    assert m.cache_seq(a, np.arange(16)) == 4        # a's blocks: held by a and by the cache
    b = m.add_seq()
    m.append_tokens(b, 16)
    m.cache_seq(b, np.arange(100, 116))
    m.free_seq(b)                                    # four blocks only the cache holds; none is free
    assert m.num_free() == 0 and m.num_evictable() == 4
    pairs = m.unshare(a)
    assert len(pairs) == 4 and not set(pairs[:, 0]) & set(pairs[:, 1])
    assert np.array_equal(m.table(a)[0], pairs[:, 1]) and len(set(pairs[:, 1])) == 4


def test_random_operations_keep_the_counts(bm):
    rng = random.Random(3)
    m = bm(96, 4)
    seqs = []
    for _ in range(4):
        seqs.append(m.add_seq())
        m.append_tokens(seqs[-1], rng.randint(0, 20))
    for _ in range(400):
        op = rng.choice(["reorder", "append", "truncate", "unshare"])
        s = rng.choice(seqs)
        if op == "reorder":
            m.reorder(seqs, [rng.randrange(4) for _ in seqs])
        elif op == "append" and m.table(s)[1] < 60:
            m.append_tokens(s, rng.randint(1, 5))
        elif op == "truncate":
            m.truncate(s, rng.randint(0, m.table(s)[1]))
        elif op == "unshare":
            m.unshare(s, rng.randint(0, 30))
            assert all(m.refcount(int(x)) == 1 for x in m.table(s)[0][8:])
        _check_counts(m, seqs)
