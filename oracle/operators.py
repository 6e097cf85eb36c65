"""fp64 restatements of the rotary positions, the compaction of cached tokens
and beam search's selection, for the tests: plain numpy, one token or row at a
time, sharing no code with the library."""
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
