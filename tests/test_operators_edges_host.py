"""Host-side edges of the rotary, compaction and beam-selection calls and of the
block manager calls that go with them (no GPU)."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import operators as ref
from tests.written import check_written


def test_an_unwritten_component_fails_the_check():
    """NaN, infinity and a stale value fail; what the formula gives, rounded, passes."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 16))
    want, size = ref.rotate(x, 77, ref.angular_frequencies(8), False)      # components 8 .. 15 pass unchanged
    check_written(want, want, size, "as it should be")
    for at in ((0, 0), (1, 7), (2, 8), (2, 15)):
        for bad in (math.nan, math.inf, -math.inf, want[at] + 1.0):
            got = want.copy()
            got[at] = bad
            with pytest.raises(AssertionError):
                check_written(got, want, size, "planted")
    with pytest.raises(AssertionError):
        check_written(np.full_like(want, math.nan), want, size, "nothing written")


# ---------------------------------------------------------------------------
# block manager
# ---------------------------------------------------------------------------

@pytest.fixture()
def bm():
    import __graft_entry__
    __graft_entry__.build()
    from paged_kv_cache_167_gb300 import BlockManager
    return BlockManager


def _cached_below_an_evictable_entry(bm):
    """A pool with nothing free.  b's second block is held by b and by the prefix
    cache, below an entry that only the cache holds: an allocation evicts both
    entries, and the block is b's alone.  c and d share a partly filled block."""
    m = bm(5, 4)
    a = m.add_seq()
    m.append_tokens(a, 4)
    assert m.cache_seq(a, np.arange(4)) == 1
    b = m.add_seq()
    m.append_tokens(b, 8)
    assert m.cache_seq(b, np.arange(8)) == 1             # the first is cached already, in a's block
    c = m.add_seq()
    m.append_tokens(c, 6)
    d = m.fork(c)
    m.free_seq(a)
    assert m.num_free() == 0 and m.num_evictable() == 1
    assert m.refcount(int(m.table(b)[0][1])) == 2
    return m, b, c, d


def test_unshare_keeps_a_block_that_eviction_made_private(bm):
    m, b, c, _ = _cached_below_an_evictable_entry(bm)
    before = m.table(b)[0].copy()
    pairs = m.unshare(b)
    assert len(pairs) == 0 and np.array_equal(m.table(b)[0], before)
    assert m.refcount(int(before[1])) == 1 and m.num_free() == 1 and m.num_cached() == 0
    more = m.unshare(c, 4)                               # one block is free for it, and it is not one of b's
    assert len(more) == 1 and more[0, 1] not in before
    assert m.num_free() == 0


def test_append_keeps_a_block_that_eviction_made_private(bm):
    m, b, c, _ = _cached_below_an_evictable_entry(bm)
    m.truncate(b, 6)                                     # its last block: partly filled, and cached
    before = m.table(b)[0].copy()
    slots, cow = m.append_tokens(b, 1)
    assert cow is None and np.array_equal(m.table(b)[0], before)
    assert slots[0] == before[1] * 4 + 2 and m.refcount(int(before[1])) == 1
    _, cow = m.append_tokens(c, 1)
    assert cow is not None and cow[1] not in before
    assert m.num_free() == 0


def test_block_manager_when_memory_runs_out(tmp_path):
    """Reorder, unshare and truncate with each of their allocations failing in turn."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    from paged_kv_cache_167_gb300 import build
    exe = tmp_path / "bm_out_of_memory"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I",
                    os.path.join(build._cuda_home(), "include"),
                    os.path.join(build.ROOT, "tests", "c", "bm_out_of_memory.cpp"),
                    os.path.join(build.CSRC, "pa_block_manager.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
