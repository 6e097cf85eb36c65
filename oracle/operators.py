"""fp64 restatements of the rotary positions, the compaction of cached tokens,
beam search's selection, a step's tables and positions of several axes, for the
tests: plain numpy, one token or row at a time, sharing no code with the library."""
from __future__ import annotations

import math
from typing import Optional

import numpy as np


def angular_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                        original_len: float = 0.0, low: float = 1.0, high: float = 32.0) -> list:
    """Radians per position of each pair."""
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    out = []
    for i in range(rot_dim // 2):
        w = 1.0 / base ** (2 * i / rot_dim)
        if scaling == "linear":
            w = w / factor
        elif scaling == "parts":
            turns = original_len * w / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - low) / (high - low)))
            w = share * w + (1 - share) * w / factor
        elif scaling == "parts_index":
            index = lambda turns: rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
            first = max(0, math.floor(index(high)))
            last = min(rot_dim - 1, math.ceil(index(low)))
            ramp = min(1.0, max(0.0, (i - first) / max(last - first, 1e-3)))
            w = (1 - ramp) * w + ramp * w / factor
        out.append(w)
    return out


def rotate(x: np.ndarray, position: int, w, interleaved: bool, mscale: float = 1.0):
    """One head row (or rows [..., d]) at one position; returns the rotated row
    and, for each component, |a| + |b| of its pair (what an angle error scales)."""
    x = np.asarray(x, np.float64)
    y, size = x.copy(), np.zeros_like(x)
    half = len(w)
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        phi = math.fmod(position * w[i], 2 * math.pi)
        c, s = mscale * math.cos(phi), mscale * math.sin(phi)
        a, b = x[..., p], x[..., q]
        y[..., p], y[..., q] = a * c - b * s, b * c + a * s
        size[..., p] = size[..., q] = abs(mscale) * (np.abs(a) + np.abs(b))
    return y, size


def compact(pool: np.ndarray, src_tables, dst_tables, keep, keep_lens, starts=None, w=None,
            interleaved: bool = False):
    """pool [NB][2][Hkv][b][d] fp64 -> (pool after, |a| + |b| of rotated components)."""
    before, after, size = pool, pool.copy(), np.zeros_like(pool)
    b = pool.shape[3]
    for s in range(len(keep_lens)):
        first = 0 if starts is None else int(starts[s])
        for i in range(int(keep_lens[s])):
            old, new = int(keep[s][i]), first + i
            sb, db = int(src_tables[s][old // b]), int(dst_tables[s][new // b])
            if old == new and sb == db:
                continue
            k = before[sb, 0, :, old % b]
            scale = np.zeros_like(k)
            if w is not None:
                k, scale = rotate(k, new - old, w, interleaved)
            after[db, 0, :, new % b] = k
            size[db, 0, :, new % b] = scale
            after[db, 1, :, new % b] = before[sb, 1, :, old % b]
    return after, size


def log_softmax(x: np.ndarray) -> np.ndarray:
    """Of one row; all -inf where no entry is above it, or with a NaN or +inf.
    The maximum is subtracted first, so that a row of lowest values is uniform."""
    if np.isnan(x).any() or np.isposinf(x).any() or not (x > -math.inf).any():
        return np.full(x.shape, -math.inf)
    below = x - x.max()
    return below - math.log(math.fsum(np.exp(below)))


def beam_scores(logits: np.ndarray, scores, finished: Optional[np.ndarray] = None, end_token: int = 0) -> np.ndarray:
    """fp64 scores [beams][vocab] of one group."""
    J, V = logits.shape
    y = np.full((J, V), -math.inf)
    for j in range(J):
        s = float(scores[j])
        if not (-math.inf < s < math.inf):
            continue
        if finished is not None and finished[j]:
            y[j, end_token] = s
            continue
        y[j] = s + log_softmax(np.asarray(logits[j], np.float64))
    return y


def best(scores: np.ndarray, n: int):
    """The n best of [beams][vocab]: (scores, beams, tokens), ties to the lowest
    flat index."""
    flat = scores.ravel()
    order = sorted(range(flat.size), key=lambda f: (-flat[f], f))[:n]
    return flat[order], [f // scores.shape[1] for f in order], [f % scores.shape[1] for f in order]


def axis_of_pair(sections, order: str) -> list:
    """The axis that turns each pair."""
    if order == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    n = len(sections)
    return [i % n if i < n * sections[i % n] else 0 for i in range(sum(sections))]


def rotate_axes(x: np.ndarray, positions, axis, w, interleaved: bool, mscale: float = 1.0):
    """One token's rows at one position an axis: each axis's pairs turned alone."""
    y, size = np.asarray(x, np.float64).copy(), np.zeros_like(x, dtype=np.float64)
    for a in set(axis):
        mine = [wi if ax == a else 0.0 for wi, ax in zip(w, axis)]
        turned, s = rotate(x, int(positions[a]), mine, interleaved, mscale)
        for i, ax in enumerate(axis):
            if ax == a:
                for p in ((2 * i, 2 * i + 1) if interleaved else (i, i + len(w))):
                    y[..., p], size[..., p] = turned[..., p], s[..., p]
    return y, size


def extend_tables(tables, ctx, new, free, cursor: int, block_size: int, num_blocks: int, max_tokens: int,
                  offsets=None) -> dict:
    """A step's tables, positions and slots, one token at a time, and the error
    bits it raises (tables as after the step; entries written only where taken)."""
    tables = [list(map(int, row)) for row in tables]
    width = len(tables[0]) if tables else 0
    B, b = len(ctx), block_size
    out = {"tables": tables, "lens": [], "starts": [], "positions": [0] * max_tokens, "slots": [-1] * max_tokens,
           "errors": 0}
    left = len(free) - cursor if 0 <= cursor <= len(free) else 0
    if not 0 <= cursor <= len(free):
        out["errors"] |= 0x80
    tok = blk = taken = 0
    for s in range(B):
        c, n = int(ctx[s]), int(new[s])
        if c < 0 or n < 0 or c + n > min(width * b, 2 ** 31 - 1):
            out["errors"] |= 0x4
            n = 0
            have = need = 0
        else:
            have = -(-c // b)
            need = -(-(c + n) // b) - have
        out["starts"].append(min(tok, max_tokens))
        served = tok + n <= max_tokens and (need == 0 or blk + need <= left)
        out["lens"].append(c + n if served else c)
        if not served:
            out["errors"] |= 0x80
        for j in range(n):
            if tok + j >= max_tokens:
                break
            pos = c + j
            out["positions"][tok + j] = pos + (int(offsets[s]) if offsets is not None else 0)
            if not served:
                continue
            fresh = pos // b >= have
            block = int(free[cursor + blk + pos // b - have]) if fresh else tables[s][pos // b]
            if not 0 <= block < num_blocks:
                out["errors"] |= 0x1
                block = -1
            if fresh:
                tables[s][pos // b] = block
            out["slots"][tok + j] = block * b + pos % b if block >= 0 else -1
        if served:
            taken = max(taken, blk + need) if need else taken
        tok += n
        blk += need
    out["starts"].append(min(tok, max_tokens))
    out["cursor"] = cursor + taken
    return out
