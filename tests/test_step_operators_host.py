"""Host side of a step's tables, of positions of several axes and of
differential attention: the axes' layouts and the refusals (no GPU: every call
here is refused, or has nothing to do, before anything is launched)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operators as ref


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from paged_kv_cache_167_gb300 import binding
    return binding


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


# ---------------------------------------------------------------------------
# axes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("order", ["blocks", "cycled"])
@pytest.mark.parametrize("sections", [[64], [16, 24, 24], [24, 20, 20], [32, 32], [2, 0, 6], [0, 0, 8], [1, 1, 1, 1],
                                      [0, 8], [8, 0], [5, 11, 1, 7], [1], [3, 29]])
def test_axes_of_pairs(B, sections, order):
    assert B.rotary_axes(sections, order).tolist() == ref.axis_of_pair(sections, order)


@pytest.mark.parametrize("sections", [[], [-1, 5], [0], [0, 0], [1, 1, 1, 1, 1]])
def test_axes_refusals(B, sections):
    with pytest.raises(B.PagedAttentionError) as e:
        B.rotary_axes(sections)
    assert e.value.status == INVALID


def test_axes_more_refusals(B):
    with pytest.raises(ValueError):
        B.rotary_axes([4, 4], order="striped")
    own, out = (ctypes.c_int32 * 2)(4, 4), (ctypes.c_uint8 * 8)()
    f = B.lib().pa_rotary_sections
    assert f(own, 2, 0, 8, out) == 0 and list(out) == [0] * 4 + [1] * 4
    assert f(own, 2, 2, 8, out) == INVALID and f(own, 2, 0, 9, out) == INVALID
    assert f(None, 2, 0, 8, out) == INVALID and f(own, 2, 0, 8, None) == INVALID


FAKE = 1 << 20      # an aligned address that no refused call reads


def _rotate_axes(B, axis=(0, 1, 2, 0), num_axes=3, stride=0, tokens=4, **kw):
    axis = (ctypes.c_uint8 * len(axis))(*axis)
    axes = B.PaRotaryAxes(ctypes.addressof(axis), num_axes, stride)
    rot = B.PaRotary(FAKE, 8, kw.get("flags", 0), 1.0)
    return B.lib().pa_rotate_axes(FAKE, FAKE, 0, kw.get("positions", FAKE), tokens, 2, kw.get("d", 16),
                                  ctypes.byref(rot), kw.get("axes", ctypes.byref(axes)), None)


def test_rotate_axes_refusals(B):
    assert _rotate_axes(B, tokens=0) == 0
    assert _rotate_axes(B, axis=(0, 1, 3, 0)) == INVALID            # an axis that is not there
    assert _rotate_axes(B, num_axes=0) == INVALID and _rotate_axes(B, num_axes=5) == INVALID
    assert _rotate_axes(B, stride=3) == INVALID                     # rows that overlap
    assert _rotate_axes(B, axes=None) == INVALID
    assert _rotate_axes(B, positions=None) == INVALID
    assert _rotate_axes(B, d=12) == UNSUPPORTED and _rotate_axes(B, flags=4) == INVALID
    null = B.PaRotaryAxes(None, 3, 0)
    assert _rotate_axes(B, axes=ctypes.byref(null)) == INVALID
    rot = B.PaRotary(FAKE, 8, 0, 1.0)
    pool = B.PaKvPool(FAKE, 4, 2, 16, 16, 0, 0, 0)
    f = B.lib().pa_rotate_and_cache_axes
    assert f(ctypes.byref(pool), None, None, 0, FAKE, 0, FAKE, 0, FAKE, FAKE, 4, 0, ctypes.byref(rot), None,
             None) == INVALID


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def _extend(B, **kw):
    """A call whose arrays lie 2^16 bytes apart (never read: it is refused)."""
    at = lambda i: FAKE + (i << 16)  # noqa: E731
    a = dict(tables=at(0), width=4, lens=at(1), starts=at(2), positions=at(3), slots=at(4), tokens=8, ctx=at(5),
             new=at(6), offsets=None, seqs=3, free=at(7), num_free=10, cursor=at(8), cursor_out=at(9), b=16, blocks=64)
    a.update(kw)
    return B.lib().pa_extend_tables(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(width=0), dict(tokens=-1), dict(seqs=-1), dict(seqs=(1 << 20) + 1), dict(b=0),
                                dict(blocks=0), dict(blocks=1 << 31), dict(num_free=-1)] +
                         [{k: None} for k in ("tables", "lens", "starts", "positions", "slots", "ctx", "new", "free",
                                              "cursor", "cursor_out")])
def test_extend_refusals(B, kw):
    assert _extend(B, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(lens=FAKE + (5 << 16)), dict(lens=FAKE + (6 << 16) + 8),
                                dict(starts=FAKE + (5 << 16)), dict(cursor_out=FAKE + (8 << 16)), dict(offsets=FAKE + (1 << 16)),
                                dict(free=FAKE + (3 << 16) + 60), dict(ctx=FAKE + 44), dict(new=FAKE + (4 << 16) + 60)])
def test_extend_refuses_overlap(B, kw):
    """Inputs that another CTA may still read while one writes them."""
    assert _extend(B, **kw) == INVALID


def test_extend_oracle_by_hand():
    """The restatement the GPU tests compare with, on a step worked out by hand: b = 4,
    sequences of 3 + 2, 8 + 1, 0 + 0 and 5 + 1 tokens, one block already taken."""
    got = ref.extend_tables([[9, -1, -1], [1, 2, -1], [-1] * 3, [4, 5, -1]], [3, 8, 0, 5], [2, 1, 0, 1],
                            [7, 8, 3, 6], 1, 4, 10, 6)
    assert got["tables"] == [[9, 8, -1], [1, 2, 3], [-1] * 3, [4, 5, -1]]
    assert got["lens"] == [5, 9, 0, 6] and got["starts"] == [0, 2, 3, 3, 4] and got["cursor"] == 3
    assert got["positions"] == [3, 4, 8, 5, 0, 0] and got["slots"] == [39, 32, 12, 21, -1, -1]
    short = ref.extend_tables([[9, -1, -1], [1, 2, -1], [-1] * 3, [4, 5, -1]], [3, 8, 0, 5], [2, 1, 0, 1],
                              [7, 8], 1, 4, 10, 6)
    assert short["lens"] == [5, 8, 0, 6] and short["cursor"] == 2 and short["errors"] == 0x80
    assert short["slots"] == [39, 32, -1, 21, -1, -1]


# ---------------------------------------------------------------------------
# differential attention
# ---------------------------------------------------------------------------

def _decode_diff(B, hkv=2, hq=4, d=64, b=16, seqs=3, seq_len=40, q=FAKE, lam=FAKE, weight=FAKE, eps=1e-5, scale=0.1,
                 out_scale=1.0, dflags=0, flags=0, ws=FAKE, ws_bytes=1 << 40, new_k=None, new_v=None, diff=True):
    pool = B.PaKvPool(FAKE, 64, hkv, b, d, 0, 0, 0)
    weights = B.PaDiff(lam, weight, eps, out_scale, dflags)
    return B.lib().pa_decode_diff(FAKE, q, ctypes.byref(pool), FAKE, 4, FAKE, seqs, hq, seq_len, scale,
                                  ctypes.byref(weights) if diff else None, ws, ws_bytes, new_k, new_v, flags, None)


@pytest.mark.parametrize("kw", [dict(hkv=3, hq=3), dict(hq=5), dict(seqs=-1), dict(seq_len=-1), dict(q=None),
                                dict(q=FAKE + 8), dict(lam=None), dict(lam=FAKE + 2), dict(weight=FAKE + 4),
                                dict(eps=0.0), dict(eps=float("nan")), dict(eps=-1.0), dict(scale=float("inf")),
                                dict(out_scale=float("nan")), dict(dflags=2), dict(flags=2), dict(new_k=FAKE),
                                dict(new_k=FAKE, new_v=FAKE + 8), dict(diff=False), dict(seqs=65536)])
def test_decode_diff_refusals(B, kw):
    assert _decode_diff(B, **kw) == INVALID


def test_decode_diff_more_refusals(B):
    assert _decode_diff(B, d=32) == UNSUPPORTED and _decode_diff(B, b=12) == UNSUPPORTED
    assert _decode_diff(B, hq=6) == UNSUPPORTED
    assert _decode_diff(B, ws=None) == WORKSPACE and _decode_diff(B, ws_bytes=64) == WORKSPACE
    assert _decode_diff(B, ws=FAKE + 16) == WORKSPACE
    assert _decode_diff(B, seqs=0) == 0 and _decode_diff(B, seqs=0, weight=None, eps=0.0) == 0
    pool = B.PaKvPool(FAKE, 64, 3, 16, 64, 0, 0, 0)
    assert B.lib().pa_decode_diff_workspace_size(ctypes.byref(pool), 4, 6, 100) == 0


@pytest.mark.parametrize("shape,strides,ok", [((3, 1), (1, 1), True), ((3, 1), (0, 1), False), ((3, 1), (7, 0), True),
                                              ((1, 1), (0, 0), True), ((2, 4), (4, 1), True), ((2, 4), (9, 1), True),
                                              ((2, 4), (0, 1), False), ((2, 4), (3, 1), False),
                                              ((2, 4), (8, 2), False), ((2, 4), (1, 2), False)])
def test_axes_positions_of_any_stride(B, shape, strides, ok):
    """What reaches the library is the distance of the axes' rows; rows that share their
    memory (one position for all axes, expanded) have none and are refused."""
    positions = torch.arange(64).as_strided(shape, strides)
    axes = B.rotary_axes([2] * shape[0])
    freqs = torch.zeros(2 * shape[0], dtype=torch.int64)
    if not ok:
        with pytest.raises(ValueError, match="dense"):
            B._axes(axes, positions, shape[1], freqs, -1)
        return
    desc, address = B._axes(axes, positions, shape[1], freqs, -1)
    assert address == positions.data_ptr() and desc.num_axes == shape[0]
    for a in range(1, shape[0]):     # 0: num_tokens
        assert (desc.position_stride or shape[1]) * a == positions.stride(0) * a


def _prefill_diff(B, hkv=2, hq=4, d=64, b=16, seqs=3, chunk=5, ctx=30, q=FAKE, lam=FAKE, eps=1e-5, scale=0.1,
                  out_scale=1.0, dflags=0, diff=True):
    pool = B.PaKvPool(FAKE, 64, hkv, b, d, 0, 0, 0)
    weights = B.PaDiff(lam, FAKE, eps, out_scale, dflags)
    return B.lib().pa_prefill_diff(FAKE, q, ctypes.byref(pool), FAKE, 4, FAKE, seqs, chunk, hq, ctx, scale,
                                   ctypes.byref(weights) if diff else None, None)


@pytest.mark.parametrize("kw", [dict(hkv=3, hq=3), dict(hq=5), dict(seqs=-1), dict(chunk=-1), dict(ctx=-1),
                                dict(ctx=60), dict(q=None), dict(q=FAKE + 8), dict(lam=None), dict(eps=0.0),
                                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(dflags=4),
                                dict(out_scale=float("inf")), dict(diff=False), dict(seqs=65536),
                                dict(hkv=-2, hq=4)])
def test_prefill_diff_refusals(B, kw):
    assert _prefill_diff(B, **kw) == INVALID


def test_prefill_diff_refuses_positions_that_pass_31_bits(B):
    pool = B.PaKvPool(FAKE, 1 << 28, 2, 16, 64, 0, 0, 0)
    weights = B.PaDiff(FAKE, FAKE, 1e-5, 1.0, 0)
    for chunk, ctx in [(5, 2 ** 31 - 10), (2 ** 31 - 1, 2 ** 31 - 1), (300, 2 ** 31 - 301)]:
        assert B.lib().pa_prefill_diff(FAKE, FAKE, ctypes.byref(pool), FAKE, 1 << 27, FAKE, 1, chunk, 4, ctx, 0.1,
                                       ctypes.byref(weights), None) == INVALID


def test_prefill_diff_more_refusals(B):
    assert _prefill_diff(B, d=32) == UNSUPPORTED and _prefill_diff(B, b=4) == UNSUPPORTED
    assert _prefill_diff(B, hq=6) == UNSUPPORTED and _prefill_diff(B, hq=32) == UNSUPPORTED
    assert _prefill_diff(B, seqs=0) == 0 and _prefill_diff(B, chunk=0) == 0
