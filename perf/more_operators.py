"""Cases, plain forms and calls of operators for a serving step built on the GPU.

extend_tables  block tables, positions and slots of a step's new tokens from
               the requests' lengths and a list of free blocks
rotate_axes    rotary positions with several axes (time, height, width): of
               queries and keys with the slot writer, and of one tensor alone
decode_diff    differential attention of single tokens over the paged cache:
               the difference of two softmax maps with learned weights, and
               the norm of each head behind it
prefill_diff   the same for chunks of prompt tokens, causal

``run`` with ``own`` false computes them with elementary torch operations;
with ``own`` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _extend_case(kind, seqs, tokens, first, b, pad=0, short=False):
    return {"op": "extend_tables", "kind": kind, "seqs": seqs, "tokens": tokens, "first": first, "b": b, "pad": pad,
            "short": short}


def _axes_case(tokens, hq, hkv, d, b, rot, sections, order, interleaved, cache, fused=False):
    return {"op": "rotate_axes", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "b": b, "rot": rot,
            "sections": " ".join(str(n) for n in sections), "order": order, "interleaved": interleaved, "cache": cache,
            "fused": fused}


def _decode_case(seqs, low, high, hq, hkv, d, b, norm, by_head=False):
    return {"op": "decode_diff", "seqs": seqs, "low": low, "high": high, "hq": hq, "hkv": hkv, "d": d, "b": b,
            "norm": norm, "by_head": by_head}


def _prefill_case(seqs, chunk, low, high, hq, hkv, d, b, norm, by_head=False):
    return {"op": "prefill_diff", "seqs": seqs, "chunk": chunk, "low": low, "high": high, "hq": hq, "hkv": hkv,
            "d": d, "b": b, "norm": norm, "by_head": by_head}


def listed():
    return [
        # one decode step of 64 chats: a launch-bound call before the first layer
        _named("extend_decode_64", _extend_case("decode", 64, 1, 850, 16)),
        # a continuous batch of 4,096 requests: single tokens, chunks of prompts, requests that pause
        _named("extend_mixed_4096", _extend_case("mixed", 4096, 512, 2000, 16, pad=1000)),
        # one prompt of 131,071 tokens behind a few cached ones
        _named("extend_prompt_131071", _extend_case("prompt", 1, 131071, 37, 32)),
        # one decode step of 64 chats (64/8 heads), positions of three axes
        _named("axes_decode_64", _axes_case(64, 64, 8, 128, 16, 128, [16, 24, 24], "blocks", False, True)),
        # 8,192 tokens of images and text, axes dealt out pair by pair, q, k and v views of one projection
        _named("axes_prefill_8192", _axes_case(8192, 64, 8, 128, 16, 128, [24, 20, 20], "cycled", False, True, True)),
        # an image encoder's queries: two axes over a part of an 80-wide head, interleaved pairs, an odd count
        _named("axes_image_5001", _axes_case(5001, 16, 0, 80, 0, 48, [12, 12], "blocks", True, False)),
        # one decode step of 64 chats, 32 pairs of query heads over four pairs of key heads
        _named("diff_decode_64", _decode_case(64, 600, 850, 64, 8, 128, 16, True)),
        # four long contexts
        _named("diff_decode_4x32768", _decode_case(4, 32768, 32768, 32, 8, 128, 16, True)),
        # a ragged batch of 64-wide heads, one query pair per key pair, no norm behind
        _named("diff_decode_ragged_33", _decode_case(33, 1, 3000, 16, 16, 64, 32, False)),
        # 16 chunks of 512 prompt tokens at 4,096 cached ones
        _named("diff_prefill_16x512", _prefill_case(16, 512, 4096, 4096, 64, 8, 128, 16, True)),
        # the first 2,048 tokens of one prompt
        _named("diff_prefill_1x2048", _prefill_case(1, 2048, 0, 0, 32, 8, 128, 64, True)),
        # odd chunks at ragged contexts, 64-wide heads, keys by query head
        _named("diff_prefill_ragged_5", _prefill_case(5, 333, 0, 3000, 16, 8, 64, 32, True, by_head=True)),
    ]


def _room(c):
    """Tokens that a step's arrays hold: a fixed number, as a captured step has."""
    if c["kind"] == "mixed":
        return c["seqs"] + (c["seqs"] // 64 + 2) * c["tokens"] + c["pad"]
    return c["seqs"] * c["tokens"] + c["pad"]


def _named(name, case):
    return dict(case, name=name)


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["extend_tables", "rotate_axes", "decode_diff", "decode_diff", "prefill_diff", "prefill_diff"])
    if op == "extend_tables":
        kind = rng.choice(["decode", "mixed", "prompt"])
        b = rng.choice([4, 8, 16, 32, 64])
        short = rng.random() < 0.25
        if kind == "decode":
            return _extend_case(kind, _log(rng, 1, 16384), 1, _log(rng, 1, 4000), b, rng.choice([0, 7, 500]), short)
        if kind == "mixed":
            return _extend_case(kind, _log(rng, 2, 8192), _log(rng, 2, 700), _log(rng, 1, 4000), b,
                                rng.choice([0, 300]), short)
        return _extend_case(kind, rng.randint(1, 4), _log(rng, 1, 32768), _log(rng, 1, 3000), b, 0, short)
    if op == "rotate_axes":
        d = rng.choice([64, 80, 128])
        rot = rng.choice([d, d, d // 2])
        cache = d != 80 and rng.random() < 0.7
        axes = rng.choice([2, 3, 3, 4])
        rest = rot // 2
        sections = []
        for i in range(axes - 1):
            sections.append(rng.randint(1, max(1, rest // (axes - i))))
            rest -= sections[-1]
        # dealt out pair by pair, the first axis takes what the others leave
        sections = [rest] + sections
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        return _axes_case(_log(rng, 1, 8192), hq, hkv if cache else 0, d, rng.choice([8, 16, 32, 64]) if cache else 0,
                          rot, sections, rng.choice(["blocks", "cycled"]), rng.random() < 0.4, cache,
                          cache and rng.random() < 0.5)
    d = rng.choice([64, 128])
    hkv = rng.choice([2, 4, 8])
    per = rng.choice([1, 2, 4, 8])
    by_head = per > 1 and rng.random() < 0.25
    norm = rng.random() < 0.7
    if op == "decode_diff":
        high = _log(rng, 1, 32768)
        seqs = max(1, min(_log(rng, 1, 64), 131072 // high))
        return _decode_case(seqs, max(1, high // rng.choice([1, 2, 8])), high, hkv * per, hkv, d,
                            rng.choice([4, 8, 16, 32, 64]), norm, by_head)
    chunk = _log(rng, 1, 2048)
    high = rng.choice([0, _log(rng, 1, 4096)])
    seqs = max(1, min(_log(rng, 1, 16), 8192 // chunk))
    return _prefill_case(seqs, chunk, high // 2, high, hkv * per, hkv, d, rng.choice([8, 16, 32, 64]), norm, by_head)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(torch.bfloat16)


def _cuda(a):
    return torch.as_tensor(a, device="cuda")


def _extend_inputs(c, seed):
    rng = np.random.default_rng(seed)
    n, b, top = c["seqs"], c["b"], c["tokens"]
    ctx = rng.integers(0, c["first"] + 1, size=n).astype(np.int64)
    if c["kind"] == "prompt":
        ctx[:] = c["first"]
        new = np.full(n, top, np.int64)
    elif c["kind"] == "decode":
        new = np.ones(n, np.int64)
    else:   # most requests decode one token, one in 64 takes a chunk of its prompt, some pause
        new = np.ones(n, np.int64)
        pick = rng.random(n)
        new[pick < 0.1] = 0
        chunk = pick > 1.0 - 1.0 / 64
        chunk[rng.integers(n)] = True
        new[chunk] = rng.integers(1, top + 1, size=int(chunk.sum()))
    have, need = -(-ctx // b), -(-(ctx + new) // b)
    width = -(-(c["first"] + top) // b) + 1
    wanted = int((need - have).sum())
    blocks = int(need.sum()) + 64
    ids = rng.permutation(blocks).astype(np.int32)
    tables = np.full((n, width), -1, np.int32)
    column = np.arange(width)
    tables[column[None, :] < have[:, None]] = ids[:int(have.sum())]
    before = 5                      # blocks of the list that earlier steps took
    free = ids[int(have.sum()):]
    if c["short"]:                  # fewer free blocks than the step wants
        free = free[:before + wanted // 2]
    tokens = _room(c)
    i32 = torch.int32
    return {"tables": _cuda(tables), "ctx": _cuda(ctx.astype(np.int32)), "new": _cuda(new.astype(np.int32)),
            "free": _cuda(free.copy()), "cursor": _cuda(np.array([min(before, len(free))], np.int32)),
            "offsets": _cuda(rng.integers(-200, 1, size=n).astype(np.int32)), "num_blocks": blocks,
            "lens": torch.empty(n, dtype=i32, device="cuda"), "starts": torch.empty(n + 1, dtype=i32, device="cuda"),
            "cursor_out": torch.empty(1, dtype=i32, device="cuda"),
            "positions": torch.empty(tokens, dtype=torch.int64, device="cuda"),
            "slots": torch.empty(tokens, dtype=torch.int64, device="cuda")}


def _sections(c):
    return [int(n) for n in c["sections"].split()]


def _axis_of_pair(sections, order):
    """The axis whose position turns each pair: the sections one behind the
    other, or pair i by axis i mod n while that axis has pairs left, else by
    the first."""
    pairs, n = sum(sections), len(sections)
    if order == "blocks":
        return np.repeat(np.arange(n), sections)
    i = np.arange(pairs)
    turn = i % n
    return np.where(i < n * np.asarray(sections)[turn], turn, 0)


def _axes_inputs(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    n, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
    axes = len(_sections(c))
    # images of 24 x 32 patches after 40 words each, one after the other; a further axis counts along
    i = np.arange(n)
    image, at = i // (40 + 768), i % (40 + 768)
    base = image * (40 + 32)
    patch = np.maximum(at - 40, 0)
    word = at < 40
    rows = np.where(word, base + at, base + 40 + patch // 32)
    columns = np.where(word, base + at, base + 40 + patch % 32)
    times = np.where(word, base + at, base + 40)
    pos = np.stack([times, rows, columns, i][:axes] if axes > 2 else [rows, columns]).astype(np.int64)
    if n <= 512:    # a decode step: every axis goes on from each context's last position
        pos = np.broadcast_to(600 + rng.integers(0, 251, size=n), (axes, n)).astype(np.int64)
    w = 10000.0 ** (-2.0 * np.arange(c["rot"] // 2, dtype=np.float64) / c["rot"])
    axis = _axis_of_pair(_sections(c), c["order"])
    s = {"positions": _cuda(pos.copy()), "w": w, "angular": _cuda(w), "axis": axis, "axis_dev": _cuda(axis)}
    if c["fused"]:
        qkv = _normal((n, hq + 2 * hkv, d), g)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"] = _normal((n, hq, d), g)
        if c["cache"]:
            s["k"], s["v"] = _normal((n, hkv, d), g), _normal((n, hkv, d), g)
    s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    if c["cache"]:
        blocks = -(-n // c["b"]) + 5
        s["pool"] = _normal((blocks, 2, hkv, c["b"], d), g)
        s["slots"] = _cuda(rng.permutation(blocks * c["b"])[:n].astype(np.int64))
    return s


def _paged(c, totals, g, rng):
    """A pool whose keys and values are those of ``totals`` tokens, and tables."""
    b, hkv, d = c["b"], c["hkv"], c["d"]
    count = -(-totals // b)
    blocks = int(count.sum()) + 3
    width = max(int(count.max()), 1)
    ids = rng.permutation(blocks).astype(np.int32)
    tables = np.full((len(totals), width), -1, np.int32)
    tables[np.arange(width)[None, :] < count[:, None]] = ids[:int(count.sum())]
    pool = torch.empty((blocks, 2, hkv, b, d), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (2 * hkv * b * d))
    for i in range(0, blocks, step):
        pool[i:i + step] = _normal(tuple(pool[i:i + step].shape), g)
    return pool, _cuda(tables)


def _weights(c, g):
    pairs = c["hq"] // 2
    lam = 0.2 + 0.6 * torch.rand(pairs, generator=g, device="cuda", dtype=torch.float32)
    weight = 1.0 + 0.1 * torch.randn(2 * c["d"], generator=g, device="cuda", dtype=torch.float32)
    return {"lam": lam, "weight": weight if c["norm"] else None, "eps": 1e-5, "out_scale": 0.2 if c["norm"] else 1.0,
            "scale": c["d"] ** -0.5}


def _decode_inputs(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    lens = rng.integers(c["low"], c["high"] + 1, size=c["seqs"]).astype(np.int64)
    pool, tables = _paged(c, lens, g, rng)
    # keys and queries of trained heads line up more than noise does: logits of a standard deviation near 2
    q = _normal((c["seqs"], c["hq"], c["d"]), g, 2.0)
    s = {"pool": pool, "tables": tables, "lens": _cuda(lens.astype(np.int32)), "max_len": int(c["high"]), "q": q,
         "out": torch.empty((c["seqs"], c["hq"] // 2, 2 * c["d"]), dtype=torch.bfloat16, device="cuda")}
    s.update(_weights(c, g))
    s["max_len"] = min(s["max_len"], tables.shape[1] * c["b"])
    return s


def _prefill_inputs(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    ctx = rng.integers(c["low"], c["high"] + 1, size=c["seqs"]).astype(np.int64)
    pool, tables = _paged(c, ctx + c["chunk"], g, rng)
    q = _normal((c["seqs"], c["chunk"], c["hq"], c["d"]), g, 2.0)
    s = {"pool": pool, "tables": tables, "ctx": _cuda(ctx.astype(np.int32)), "max_ctx": int(ctx.max()), "q": q,
         "host_ctx": ctx.tolist(),
         "out": torch.empty((c["seqs"], c["chunk"], c["hq"] // 2, 2 * c["d"]), dtype=torch.bfloat16, device="cuda")}
    s.update(_weights(c, g))
    return s


INPUTS = {"extend_tables": _extend_inputs, "rotate_axes": _axes_inputs, "decode_diff": _decode_inputs,
          "prefill_diff": _prefill_inputs}


def prepare(case, seed):
    s = INPUTS[case["op"]](case, seed)
    s["case"] = case
    if own:   # what a serving program keeps: frequencies on the device, the axes' layout, the workspace
        import paged_kv_cache_167_gb300 as pa
        s["pa"] = pa
        if case["op"] == "rotate_axes":
            s["freqs"] = torch.as_tensor(pa.rotary_turns(s["w"]), device="cuda")
            s["axes"] = pa.rotary_axes(_sections(case), order=case["order"])
        elif case["op"] == "decode_diff":
            nbytes = pa.decode_diff_workspace_size(s["pool"], case["seqs"], case["hq"], s["max_len"])
            s["workspace"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _extend_plain(s, c):
    b, tables = c["b"], s["tables"]
    ctx, new = s["ctx"].to(torch.int64), s["new"].to(torch.int64)
    most = s["slots"].numel()
    have, end = (ctx + b - 1) // b, (ctx + new + b - 1) // b
    need = end - have
    tok, blk = torch.cumsum(new, 0) - new, torch.cumsum(need, 0) - need
    cursor = s["cursor"].to(torch.int64)
    left = s["free"].numel() - cursor
    served = (tok + new <= most) & ((need == 0) | (blk + need <= left))
    s["lens"].copy_(torch.where(served, ctx + new, ctx))
    s["starts"][:-1] = tok.clamp_max(most)
    s["starts"][-1:] = (tok[-1:] + new[-1:]).clamp_max(most)
    s["cursor_out"].copy_(cursor + torch.where(served & (need > 0), blk + need, 0).amax())
    # the new blocks of each table
    column = torch.arange(tables.shape[1], device=tables.device)[None, :]
    fresh = served[:, None] & (column >= have[:, None]) & (column < end[:, None])
    at = (cursor + blk[:, None] + column - have[:, None]).clamp(0, max(s["free"].numel() - 1, 0))
    if s["free"].numel():
        tables.copy_(torch.where(fresh, s["free"][at], tables))
    # the tokens
    i = torch.arange(most, device=tables.device)
    seq = torch.searchsorted(tok + new, i, right=True).clamp_max(c["seqs"] - 1)
    real = i < tok[-1] + new[-1]
    pos = ctx[seq] + i - tok[seq]
    block = tables[seq, (pos // b).clamp(0, tables.shape[1] - 1)].to(torch.int64)
    s["positions"].copy_(torch.where(real, pos + s["offsets"][seq], 0))
    s["slots"].copy_(torch.where(real & served[seq], block * b + pos % b, -1))
    return s["tables"], s["lens"], s["starts"], s["cursor_out"], s["positions"], s["slots"]


def _turned(x, phi, interleaved):
    """x [n][heads][d] in fp32, its first pairs rotated by phi [n][pairs] (fp64)."""
    r = 2 * phi.shape[1]
    cos, sin = torch.cos(phi).to(torch.float32)[:, None, :], torch.sin(phi).to(torch.float32)[:, None, :]
    part = x[..., :r]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., r:]], dim=-1)


def _axes_plain(s, c):
    phi = s["positions"].to(torch.float64)[s["axis_dev"]].T * s["angular"][None, :]
    s["q_out"].copy_(_turned(s["q"].float(), phi, c["interleaved"]))
    if not c["cache"]:
        return s["q_out"]
    block, off = s["slots"] // c["b"], s["slots"] % c["b"]
    s["pool"][block, 0, :, off] = _turned(s["k"].float(), phi, c["interleaved"]).to(torch.bfloat16)
    s["pool"][block, 1, :, off] = s["v"]
    return s["q_out"], s["pool"]


def _key_head(c):
    """The key head that each query head reads: its pair's group has two, one
    for each map, or (by head) query head i reads key head i / (hq / hkv)."""
    i = np.arange(c["hq"])
    per = c["hq"] // c["hkv"]
    return i // per if c["by_head"] else (i // (2 * per)) * 2 + i % 2


def _softmax_rows(x):
    top = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(dim=-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _difference(s, probs, values):
    """probs [.., hq, rows, keys], values [.., pairs, keys, 2 d] -> the normed difference."""
    o1, o2 = torch.matmul(probs[..., 0::2, :, :], values), torch.matmul(probs[..., 1::2, :, :], values)
    x = o1 - s["lam"][:, None, None] * o2
    if s["weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"]) * s["weight"]
    return x * s["out_scale"]


def _decode_plain(s, c):
    b, hkv, d, B = c["b"], c["hkv"], c["d"], c["seqs"]
    heads = torch.as_tensor(_key_head(c), device="cuda")
    groups = torch.arange(c["hq"] // 2, device="cuda") // (c["hq"] // hkv)
    tables = s["tables"].to(torch.int64).clamp_min(0)
    step = max(1, (1 << 28) // (tables.shape[1] * b * d * max(hkv, c["hq"])))
    for i in range(0, B, step):
        t = tables[i:i + step]
        keys = s["pool"][t, 0].float().permute(0, 2, 1, 3, 4).flatten(2, 3)          # [n][hkv][tokens][d]
        values = s["pool"][t, 1].float().permute(0, 2, 1, 3, 4).flatten(2, 3)
        values = torch.cat([values[:, 0::2], values[:, 1::2]], dim=-1)                # [n][hkv / 2][tokens][2 d]
        logits = torch.matmul(keys[:, heads], s["q"][i:i + step].float()[..., None])[..., 0] * s["scale"]
        seen = torch.arange(logits.shape[-1], device="cuda")[None, :] < s["lens"][i:i + step, None]
        logits = torch.where(seen[:, None, :], logits, torch.full_like(logits, -math.inf))
        probs = _softmax_rows(logits)[:, :, None, :]
        s["out"][i:i + step] = _difference(s, probs, values[:, groups])[:, :, 0]
    return s["out"]


def _prefill_plain(s, c):
    b, hkv, d, C = c["b"], c["hkv"], c["d"], c["chunk"]
    heads = torch.as_tensor(_key_head(c), device="cuda")
    groups = torch.arange(c["hq"] // 2, device="cuda") // (c["hq"] // hkv)
    for i, ctx in enumerate(s["host_ctx"]):
        n = ctx + C
        t = s["tables"][i, :-(-n // b)].to(torch.int64)
        keys = s["pool"][t, 0].float().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]       # [hkv][tokens][d]
        values = s["pool"][t, 1].float().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]
        values = torch.cat([values[0::2], values[1::2]], dim=-1)
        q = s["q"][i].float().permute(1, 0, 2)
        for h in range(0, c["hq"], 16):      # 16 query heads at a time: the maps of all would not fit
            h1 = min(h + 16, c["hq"])
            logits = torch.matmul(q[h:h1], keys[heads[h:h1]].transpose(1, 2)) * s["scale"]
            late = torch.arange(n, device="cuda")[None, :] > ctx + torch.arange(C, device="cuda")[:, None]
            probs = _softmax_rows(logits.masked_fill_(late, -math.inf))
            part = dict(s, lam=s["lam"][h // 2:h1 // 2])
            s["out"][i, :, h // 2:h1 // 2] = _difference(part, probs, values[groups[h // 2:h1 // 2]]).permute(1, 0, 2)
    return s["out"]


PLAIN = {"extend_tables": _extend_plain, "rotate_axes": _axes_plain, "decode_diff": _decode_plain,
         "prefill_diff": _prefill_plain}


def run(s):
    c = s["case"]
    if not own:
        return PLAIN[c["op"]](s, c)
    pa = s["pa"]
    if c["op"] == "extend_tables":
        pa.extend_tables(s["tables"], s["lens"], s["starts"], s["positions"], s["slots"], s["ctx"], s["new"],
                         s["free"], s["cursor"], s["cursor_out"], c["b"], s["num_blocks"],
                         position_offsets=s["offsets"])
        return s["tables"], s["lens"], s["starts"], s["cursor_out"], s["positions"], s["slots"]
    if c["op"] == "rotate_axes":
        if not c["cache"]:
            pa.rotate(s["q_out"], s["q"], s["positions"], s["freqs"], interleaved=c["interleaved"], axes=s["axes"])
            return s["q_out"]
        pa.rotate_and_cache(s["pool"], s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"],
                            interleaved=c["interleaved"], axes=s["axes"])
        return s["q_out"], s["pool"]
    keys = "head" if c["by_head"] else "map"
    if c["op"] == "decode_diff":
        pa.decode_diff(s["out"], s["q"], s["pool"], s["tables"], s["lens"], s["max_len"], s["scale"], s["lam"],
                       norm_weight=s["weight"], eps=s["eps"], out_scale=s["out_scale"], keys=keys,
                       workspace=s["workspace"])
        return s["out"]
    pa.prefill_diff(s["out"], s["q"], s["pool"], s["tables"], s["ctx"], s["max_ctx"], s["scale"], s["lam"],
                    norm_weight=s["weight"], eps=s["eps"], out_scale=s["out_scale"], keys=keys)
    return s["out"]


def work(case):
    c = case
    if c["op"] == "extend_tables":
        new = c["seqs"] * (0.9 + c["tokens"] / 2 / 64) if c["kind"] == "mixed" else c["seqs"] * c["tokens"]
        return {"bytes": 16 * _room(c) + 20 * c["seqs"] + 8 * new / c["b"], "flops": 4.0 * _room(c)}
    if c["op"] == "rotate_axes":
        row = 2 * c["d"]
        axes = len(_sections(c))
        per = 2 * c["hq"] * row + 8 * axes + (4 * c["hkv"] * row + 8 if c["cache"] else 0)
        return {"bytes": c["tokens"] * per, "flops": c["tokens"] * (c["hq"] + c["hkv"]) * 3.0 * c["rot"]}
    row = 2 * c["d"]
    if c["op"] == "decode_diff":
        keys = c["seqs"] * (c["low"] + c["high"]) / 2
        return {"bytes": keys * 2 * c["hkv"] * row + 2 * c["seqs"] * c["hq"] * row, "flops": keys * c["hq"] * 6.0 * c["d"]}
    tokens = c["seqs"] * c["chunk"]
    cached = (c["low"] + c["high"]) / 2
    keys = c["seqs"] * (cached + c["chunk"])
    # a query sees the cached keys and half of the chunk's: a product with d and one with 2 d each
    seen = tokens * (cached + (c["chunk"] + 1) / 2)
    return {"bytes": keys * 2 * c["hkv"] * row + 2 * tokens * c["hq"] * row, "flops": seen * c["hq"] * 6.0 * c["d"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_axes(c, seed):
    s = _axes_inputs(c, seed)
    r, n = c["rot"], c["tokens"]
    phase = torch.stack([s["positions"][int(a)].double() * float(w) for a, w in zip(s["axis"], s["w"])], dim=1)
    factor = torch.polar(torch.ones_like(phase), phase).unsqueeze(1)

    def turn(x):
        x = x.double().clone()
        if c["interleaved"]:
            z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * factor
            x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * factor
            x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
        return x

    if not c["cache"]:
        return turn(s["q"])
    pool = s["pool"].double()
    flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, c["hkv"], c["d"])     # by slot
    flat[s["slots"], 0] = turn(s["k"])
    flat[s["slots"], 1] = s["v"].double()
    pool = flat.reshape(pool.shape[0], c["b"], 2, c["hkv"], c["d"]).permute(0, 2, 3, 1, 4).contiguous()
    return turn(s["q"]), pool


def _exact_pairs(s, c, q, rows, n_seen):
    """q [m][hq][d]; rows: slots of the keys; n_seen [m] keys each query sees -> [m][pairs][2 d]."""
    b, d, per = c["b"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty((q.shape[0], c["hq"] // 2, 2 * d), dtype=torch.float64, device="cuda")
    blocks, offs = rows // b, rows % b
    hidden = torch.arange(rows.numel(), device="cuda")[None, :] >= n_seen[:, None]
    for h in range(c["hq"] // 2):
        group = h // per
        v = torch.cat([s["pool"][blocks, 1, 2 * group, offs], s["pool"][blocks, 1, 2 * group + 1, offs]], 1).double()
        maps = []
        for j in (0, 1):
            head = (2 * h + j) // per if c["by_head"] else 2 * group + j
            k = s["pool"][blocks, 0, head, offs].double()
            logit = (q[:, 2 * h + j].double() @ k.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
            maps.append(torch.softmax(logit, dim=1) @ v)
        x = maps[0] - float(s["lam"][h]) * maps[1]
        if s["weight"] is not None:
            x = x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + s["eps"]) * s["weight"].double()
        out[:, h] = x * s["out_scale"]
    return out


def _slots(s, c, i, n):
    t = torch.arange(n, device="cuda")
    return s["tables"][i].to(torch.int64)[t // c["b"]] * c["b"] + t % c["b"]


def exact(case, seed):
    c = case
    if c["op"] == "extend_tables":
        return None       # whole numbers: nothing is rounded
    if c["op"] == "rotate_axes":
        return _exact_axes(c, seed)
    if c["op"] == "decode_diff":
        s = _decode_inputs(c, seed)
        outs = []
        for i, n in enumerate(s["lens"].tolist()):
            outs.append(_exact_pairs(s, c, s["q"][i:i + 1], _slots(s, c, i, n), torch.tensor([n], device="cuda")))
        return torch.cat(outs)
    s = _prefill_inputs(c, seed)
    outs = []
    for i, ctx in enumerate(s["host_ctx"]):
        seen = ctx + 1 + torch.arange(c["chunk"], device="cuda")
        outs.append(_exact_pairs(s, c, s["q"][i], _slots(s, c, i, ctx + c["chunk"]), seen))
    return torch.stack(outs)
