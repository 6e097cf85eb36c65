"""Cases, plain forms and calls of three operators around paged decode.

rotate_and_cache  rotary positions of a step's queries and keys, the keys and
                  values stored at their slots of the paged pool
compact_tokens    the kept tokens of a sequence moved to the front of its
                  blocks (or into other blocks), keys re-rotated when their
                  positions change
beam_select       the best continuations over every beam and the vocabulary

``run`` with ``own`` false computes them with elementary torch operations;
with ``own`` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

TWO_PI = 2.0 * math.pi


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rotate_case(tokens, hq, hkv, d, b, rot, interleaved, scaling, first, pad=0.0, fused=False):
    return {"op": "rotate_and_cache", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "b": b, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "first": first, "pad": pad, "fused": fused}


def _compact_case(kind, seqs, length, hkv, d, b, rot, interleaved, fork):
    return {"op": "compact_tokens", "kind": kind, "seqs": seqs, "length": length, "hkv": hkv, "d": d, "b": b,
            "rot": rot, "interleaved": interleaved, "fork": fork}


def _beam_case(groups, beams, vocab, n, dtype, state):
    return {"op": "beam_select", "groups": groups, "beams": beams, "vocab": vocab, "n": n, "dtype": dtype,
            "state": state}


def listed():
    return [
        # one decode step of 64 chats (64/8 heads): a launch-bound call between projection and attention
        dict(_rotate_case(64, 64, 8, 128, 16, 128, False, "plain", 600), name="rotate_decode_64"),
        # 16 chunks of 512 prompt tokens at 4,096 cached ones, as one prefill call takes them
        dict(_rotate_case(8192, 64, 8, 128, 16, 128, False, "plain", 4096), name="rotate_prefill_8192"),
        # half of a 64-wide head in the interleaved layout, odd batch with padding tokens, scaled by the pair index
        dict(_rotate_case(1001, 28, 4, 64, 32, 32, True, "parts_index", 0, pad=0.1), name="rotate_partial_1001"),
        # a long prompt near 131,072 positions, q, k and v views of one fused projection, scaled by parts
        dict(_rotate_case(32000, 64, 8, 128, 16, 128, False, "parts", 98304, fused=True), name="rotate_long_32000"),
        # accepted draft tokens of 64 chats moved up to the end of each context (a few rows: latency)
        dict(_compact_case("accept", 64, 850, 8, 128, 16, 0, False, False), name="compact_accept_64"),
        # 8 contexts of 8,192 slide to four first tokens and the last half, keys rotated back
        dict(_compact_case("window", 8, 8192, 8, 128, 16, 128, False, False), name="compact_window_8x8192"),
        # one long context keeps a scattered half of its tokens at their own angles
        dict(_compact_case("subset", 1, 131072, 8, 128, 16, 0, False, False), name="compact_subset_131072"),
        # ragged contexts forked into compacted private blocks, 64-wide heads, partial interleaved rotation
        dict(_compact_case("subset", 33, 3000, 4, 64, 32, 32, True, True), name="compact_fork_33"),
        # one prompt's four beams, a small vocabulary: a latency-bound call
        dict(_beam_case(1, 4, 32000, 8, "bf16", "running"), name="beam_1x4_v32000"),
        # 32 prompts of four beams, the batch of the grouped decode
        dict(_beam_case(32, 4, 128256, 8, "bf16", "running"), name="beam_32x4_v128256"),
        # an odd vocabulary in fp32, first step (only beam 0 lives), finished beams and banned tokens among the groups
        dict(_beam_case(9, 5, 50257, 10, "fp32", "mixed"), name="beam_9x5_v50257"),
        # 64 prompts of eight beams, fp32 logits, 16 continuations each
        dict(_beam_case(64, 8, 128256, 16, "fp32", "running"), name="beam_64x8_v128256"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotate_and_cache", "compact_tokens", "beam_select"])
    d = rng.choice([64, 128])
    b = rng.choice([8, 16, 32, 64])
    if op == "rotate_and_cache":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
        rot = rng.choice([16, d // 4, d // 2, d, d])
        scaling = rng.choice(["plain", "linear", "base", "parts", "parts_index"])
        return _rotate_case(_log(rng, 1, 32000), hq, hkv, d, b, rot, rng.random() < 0.4, scaling,
                            rng.choice([0, 17, 4096, 98304]), rng.choice([0.0, 0.0, 0.2]), rng.random() < 0.5)
    if op == "compact_tokens":
        kind = rng.choice(["accept", "window", "subset"])
        length = _log(rng, 40, 65536)
        seqs = max(1, min(_log(rng, 1, 64), 65536 // length))
        rot = 0 if kind == "accept" else rng.choice([0, d // 2, d])
        return _compact_case(kind, seqs, length, rng.choice([1, 2, 4, 8]), d, b, rot, rng.random() < 0.4,
                             rng.random() < 0.3)
    vocab = _log(rng, 500, 150000)
    beams = rng.randint(1, 16)
    groups = max(1, min(_log(rng, 1, 64), 60_000_000 // (beams * vocab)))
    return _beam_case(groups, beams, vocab, rng.choice([beams, 2 * beams, 2 * beams]), rng.choice(["bf16", "fp32"]),
                      rng.choice(["running", "running", "mixed"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

# scaling of the angular frequencies for a context longer than the trained one
SCALING = {"plain": (10000.0, 1.0, 0, 0.0, 0.0), "linear": (10000.0, 4.0, 0, 0.0, 0.0),
           "base": (10000.0, 8.0, 0, 0.0, 0.0), "parts": (500000.0, 8.0, 8192, 1.0, 4.0),
           "parts_index": (10000.0, 16.0, 4096, 1.0, 32.0)}


def _mscale(scaling):
    # the by-index form lengthens q and k so that the logits grow by (0.1 ln s + 1)^2
    return 0.1 * math.log(SCALING[scaling][1]) + 1.0 if scaling == "parts_index" else 1.0


def _angular(rot, scaling):
    """Radians per position of each pair, float64."""
    base, s, length, low, high = SCALING[scaling]
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base" and rot > 2:
        base = base * s ** (rot / (rot - 2))
    w = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return w / s
    if scaling == "parts":
        g = np.clip((length * w / TWO_PI - low) / (high - low), 0.0, 1.0)
        return (1.0 - g) * w / s + g * w
    if scaling == "parts_index":
        def at(turns):   # the (real) pair index that makes `turns` turns over the trained length
            return rot * math.log(length / (turns * TWO_PI)) / (2.0 * math.log(base))
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        ramp = np.clip((i - first) / max(last - first, 1e-3), 0.0, 1.0)
        return ramp * w / s + (1.0 - ramp) * w
    return w


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rotate_inputs(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    n, hq, hkv, d, b = c["tokens"], c["hq"], c["hkv"], c["d"], c["b"]
    if c["fused"]:
        qkv = _normal((n, hq + 2 * hkv, d), g)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = _normal((n, hq, d), g), _normal((n, hkv, d), g), _normal((n, hkv, d), g)
    blocks = -(-n // b) * 2 + 3
    # chunks of up to 512 tokens of consecutive positions, each in blocks of its own anywhere in the pool
    at = rng.permutation(blocks)[: -(-n // b)].astype(np.int64)
    slots = (at[:, None] * b + np.arange(b, dtype=np.int64)[None, :]).ravel()[:n]
    if n <= 512:   # a decode step: one token of each of n sequences, anywhere in its last block
        positions = c["first"] + rng.integers(0, 251, size=n).astype(np.int64)
        slots = rng.permutation(blocks * b)[:n].astype(np.int64)
    else:
        positions = c["first"] + np.arange(n, dtype=np.int64) % (512 if n <= 8192 else n)
    slots[rng.random(n) < c["pad"]] = -1
    rows = np.nonzero(slots >= 0)[0].astype(np.int64)
    cuda = lambda a: torch.as_tensor(a, device="cuda")  # noqa: E731
    return {"q": q, "k": k, "v": v, "pool": _normal((blocks, 2, hkv, b, d), g), "positions": cuda(positions),
            "slots": cuda(slots), "rows": cuda(rows), "angular": cuda(_angular(c["rot"], c["scaling"])),
            "mscale": _mscale(c["scaling"])}


def _compact_inputs(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    B, hkv, d, b = c["seqs"], c["hkv"], c["d"], c["b"]
    top = c["length"]
    lens = np.full(B, top, np.int64)
    if B > 1 and c["kind"] != "window":
        lens = rng.integers(max(20, top // 3), top + 1, size=B).astype(np.int64)
    starts = np.zeros(B, np.int64)
    keeps = []
    for s in range(B):
        L = int(lens[s])
        if c["kind"] == "accept":      # 16 draft tokens at the end, a path of one to six of them accepted
            starts[s] = L - 16
            keeps.append(L - 16 + np.sort(rng.permutation(16)[:rng.integers(1, 7)]))
        elif c["kind"] == "window":    # four first tokens and the last half
            keeps.append(np.concatenate([np.arange(4), np.arange(L - L // 2, L)]))
        else:                          # a scattered half
            keeps.append(np.sort(rng.permutation(L)[:L // 2]))
    width = -(-top // b)
    count = [-(-int(L) // b) for L in lens]
    blocks = B * width * (2 if c["fork"] else 1) + 2
    ids = iter(rng.permutation(blocks).astype(np.int32))
    src = np.full((B, width), -1, np.int32)
    for s in range(B):
        src[s, :count[s]] = [next(ids) for _ in range(count[s])]
    dst = src
    if c["fork"]:
        dst = np.full((B, width), -1, np.int32)
        for s in range(B):
            dst[s, :count[s]] = [next(ids) for _ in range(count[s])]
    most = max(len(k) for k in keeps)
    keep = np.zeros((B, most), np.int32)
    for s, k in enumerate(keeps):
        keep[s, :len(k)] = k
    keep_lens = np.asarray([len(k) for k in keeps], np.int32)
    seq = np.repeat(np.arange(B, dtype=np.int64), keep_lens)
    col = np.concatenate([np.arange(n, dtype=np.int64) for n in keep_lens])
    cuda = lambda a: torch.as_tensor(a, device="cuda")  # noqa: E731
    src_t = cuda(src)
    return {"pool": _normal((blocks, 2, hkv, b, d), g), "src": src_t, "dst": cuda(dst) if c["fork"] else src_t,
            "keep": cuda(keep), "keep_lens": cuda(keep_lens), "starts": cuda(starts.astype(np.int32)),
            "lens": cuda(lens.astype(np.int32)), "seq": cuda(seq), "col": cuda(col),
            "angular": cuda(_angular(c["rot"], "plain")) if c["rot"] else None}


def _beam_inputs(c, seed):
    g = _generator(seed)
    G, J, V = c["groups"], c["beams"], c["vocab"]
    x = torch.randn((G, J, V), generator=g, device="cuda", dtype=torch.float32).mul_(3.0)
    scores = -20.0 * torch.rand((G, J), generator=g, device="cuda", dtype=torch.float32)
    finished = torch.zeros((G, J), dtype=torch.bool, device="cuda")
    if c["state"] == "mixed":
        kind = torch.arange(G, device="cuda") % 3
        scores[kind == 0, 1:] = -math.inf                                               # a prompt's first step
        finished[kind == 1, -1] = True                                                  # a beam that has ended
        banned = torch.rand((V,), generator=g, device="cuda") < 0.5
        x[kind == 2] = x[kind == 2].masked_fill(banned, -math.inf)                      # banned tokens
    return {"logits": x.to(torch.bfloat16) if c["dtype"] == "bf16" else x, "beam_scores": scores,
            "finished": finished, "end": 2}


def prepare(case, seed):
    make = {"rotate_and_cache": _rotate_inputs, "compact_tokens": _compact_inputs, "beam_select": _beam_inputs}
    s = make[case["op"]](case, seed)
    s["case"] = case
    if case["op"] == "rotate_and_cache":
        s["q_out"] = torch.empty((case["tokens"], case["hq"], case["d"]), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "beam_select":
        shape = (case["groups"], case["n"])
        s["out"] = (torch.empty(shape, dtype=torch.float32, device="cuda"),
                    torch.empty(shape, dtype=torch.int32, device="cuda"),
                    torch.empty(shape, dtype=torch.int32, device="cuda"))
    if own:   # the handles a serving program keeps: the frequencies' device copy, the workspace
        import paged_kv_cache_167_gb300 as pa
        s["pa"] = pa
        if case.get("rot"):
            base, factor, length, low, high = SCALING[case.get("scaling", "plain")]
            turns = pa.rotary_frequencies(case["rot"], base, scaling=case.get("scaling", "plain"), factor=factor,
                                          original_len=length, low=low, high=high)
            s["freqs"] = torch.as_tensor(turns, device="cuda")
        if case["op"] == "beam_select":
            nbytes = pa.beam_select_workspace_size(case["groups"], case["beams"], case["vocab"], case["n"])
            s["workspace"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _turned(x, positions, angular, interleaved, mscale):
    """x [n][heads][d] in fp32 with its first 2 * len(angular) components
    rotated; the angles in fp64, since fp32 holds none of a far position's."""
    r = 2 * angular.numel()
    phi = positions.to(torch.float64)[:, None] * angular[None, :]
    cos = (torch.cos(phi) * mscale).to(torch.float32)[:, None, :]
    sin = (torch.sin(phi) * mscale).to(torch.float32)[:, None, :]
    part = x[..., :r]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., r:]], dim=-1)


def _rotate_plain(s, c):
    turn = lambda x: _turned(x.float(), s["positions"], s["angular"], c["interleaved"], s["mscale"])  # noqa: E731
    s["q_out"].copy_(turn(s["q"]))
    rows = s["rows"]
    slots = s["slots"][rows]
    block, off = slots // c["b"], slots % c["b"]
    s["pool"][block, 0, :, off] = turn(s["k"])[rows].to(torch.bfloat16)
    s["pool"][block, 1, :, off] = s["v"][rows]
    return s["q_out"], s["pool"]


def _compact_plain(s, c):
    b, pool, seq = c["b"], s["pool"], s["seq"]
    old = s["keep"][seq, s["col"]].to(torch.int64)
    new = s["starts"][seq].to(torch.int64) + s["col"]
    from_block, to_block = s["src"][seq, old // b].to(torch.int64), s["dst"][seq, new // b].to(torch.int64)
    keys, values = pool[from_block, 0, :, old % b], pool[from_block, 1, :, old % b]
    if s["angular"] is not None:
        keys = _turned(keys.float(), new - old, s["angular"], c["interleaved"], 1.0).to(torch.bfloat16)
    pool[to_block, 0, :, new % b] = keys
    pool[to_block, 1, :, new % b] = values
    return pool


def _beam_plain(s, c):
    # fp64: neighbouring candidates of different beams are ordered by sums whose fp32 roundings may cross
    x, scores, done = s["logits"].double(), s["beam_scores"].double(), s["finished"]
    G, J, V = x.shape
    minus = torch.full((), -math.inf, dtype=torch.float64, device=x.device)
    top = x.amax(dim=-1, keepdim=True).clamp_min(-torch.finfo(torch.float64).max)
    total = top + torch.log(torch.exp(x - top).sum(dim=-1, keepdim=True))
    y = scores[..., None] + torch.where(torch.isinf(total), minus, x - total)
    end = torch.arange(V, device=x.device) == s["end"]
    y = torch.where(done[..., None], torch.where(end, scores[..., None], minus), y).reshape(G, J * V)
    # the n largest, ties to the lowest index: all above the n-th value, then the first ones equal to it
    last = torch.topk(y, c["n"], dim=-1).values[:, -1:]
    index = torch.arange(J * V, device=x.device)
    above, equal = y > last, y == last
    rank = torch.where(above, 2 * J * V - index, torch.where(equal, J * V - index, -1))
    chosen = torch.topk(rank, c["n"], dim=-1).values
    chosen = torch.where(chosen > J * V, 2 * J * V - chosen, J * V - chosen).sort(dim=-1).values
    best, order = torch.sort(torch.gather(y, 1, chosen), dim=-1, descending=True, stable=True)
    chosen = torch.gather(chosen, 1, order)
    s["out"][0].copy_(best)
    s["out"][1].copy_(chosen // V)
    s["out"][2].copy_(chosen % V)
    return s["out"]


def run(s):
    c = s["case"]
    if own:
        pa = s["pa"]
        if c["op"] == "rotate_and_cache":
            pa.rotate_and_cache(s["pool"], s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"],
                                interleaved=c["interleaved"], mscale=s["mscale"])
            return s["q_out"], s["pool"]
        if c["op"] == "compact_tokens":
            pa.compact_tokens(s["pool"], s["src"], s["dst"], s["lens"], s["keep"], s["keep_lens"],
                              starts=s["starts"], freqs=s.get("freqs"), interleaved=c["interleaved"])
            return s["pool"]
        pa.beam_select(*s["out"], s["logits"], s["beam_scores"], finished=s["finished"], end_token=s["end"],
                       workspace=s["workspace"])
        return s["out"]
    if c["op"] == "rotate_and_cache":
        return _rotate_plain(s, c)
    if c["op"] == "compact_tokens":
        return _compact_plain(s, c)
    return _beam_plain(s, c)


def work(case):
    c = case
    if c["op"] == "rotate_and_cache":
        row = 2 * c["d"]
        kept = c["tokens"] * (1.0 - c["pad"])
        nbytes = c["tokens"] * (2 * c["hq"] * row + 16) + kept * 4 * c["hkv"] * row
        return {"bytes": nbytes, "flops": (c["tokens"] * c["hq"] + kept * c["hkv"]) * 3 * c["rot"]}
    if c["op"] == "compact_tokens":
        kept = {"accept": 3.5, "window": c["length"] // 2 + 4, "subset": c["length"] / 2}[c["kind"]] * c["seqs"]
        if c["kind"] == "subset" and c["seqs"] > 1:
            kept *= 2 / 3          # lengths between a third of the longest and the longest
        rows = kept * c["hkv"]
        return {"bytes": rows * 2 * 2 * 2 * c["d"] + 4 * kept, "flops": rows * 3 * c["rot"]}
    rows = c["groups"] * c["beams"]
    return {"bytes": rows * c["vocab"] * (2 if c["dtype"] == "bf16" else 4) + 12 * c["groups"] * c["n"] + 5 * rows,
            "flops": 4.0 * rows * c["vocab"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(x, positions, angular, interleaved, mscale):
    # each pair as a complex number times m e^{i phi}
    r = 2 * angular.numel()
    phase = positions.double().unsqueeze(1) * angular
    factor = torch.polar(torch.full_like(phase, mscale), phase).unsqueeze(1)
    x = x.double().clone()
    if interleaved:
        z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * factor
        x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * factor
        x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
    return x


def exact(case, seed):
    c = case
    if c["op"] == "rotate_and_cache":
        s = _rotate_inputs(c, seed)
        pool = s["pool"].double()
        flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, c["hkv"], c["d"])     # by slot
        real = s["slots"] >= 0
        flat[s["slots"][real], 0] = _exact_rows(s["k"], s["positions"], s["angular"], c["interleaved"],
                                                s["mscale"])[real]
        flat[s["slots"][real], 1] = s["v"][real].double()
        pool = flat.reshape(pool.shape[0], c["b"], 2, c["hkv"], c["d"]).permute(0, 2, 3, 1, 4).contiguous()
        return _exact_rows(s["q"], s["positions"], s["angular"], c["interleaved"], s["mscale"]), pool
    if c["op"] == "compact_tokens":
        s = _compact_inputs(c, seed)
        pool = s["pool"].double()
        shape, b = pool.shape, c["b"]
        flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, c["hkv"], c["d"]).contiguous()
        before = flat.clone() if not c["fork"] and c["seqs"] > 1 else None
        starts, counts = s["starts"].tolist(), s["keep_lens"].tolist()
        for i, n in enumerate(counts):
            old = s["keep"][i, :n].long()
            new = starts[i] + torch.arange(n, device="cuda")
            moved = (before if before is not None else flat)[s["src"][i].long()[old // b] * b + old % b]
            if s["angular"] is not None:
                moved = torch.stack([_exact_rows(moved[:, 0], new - old, s["angular"], c["interleaved"], 1.0),
                                     moved[:, 1]], dim=1)
            flat[s["dst"][i].long()[new // b] * b + new % b] = moved
        return flat.reshape(shape[0], b, 2, c["hkv"], c["d"]).permute(0, 2, 3, 1, 4).contiguous()
    s = _beam_inputs(c, seed)
    G, J, V, n = c["groups"], c["beams"], c["vocab"], c["n"]
    best, parents, tokens = [], [], []
    for g in range(G):
        x = s["logits"][g].double().cpu().numpy()
        y = np.full((J, V), -np.inf)
        for j in range(J):
            score = float(s["beam_scores"][g, j])
            if bool(s["finished"][g, j]):
                y[j, s["end"]] = score
            elif np.isfinite(x[j].max()) and np.isfinite(score):
                top = x[j].max()
                y[j] = score + x[j] - (top + math.log(np.exp(x[j] - top).sum()))
        y = y.ravel()
        near = np.nonzero(y >= np.partition(y, y.size - n)[y.size - n])[0]
        at = near[np.lexsort((near, -y[near]))][:n]
        best.append(y[at])
        parents.append(at // V)
        tokens.append(at % V)
    return np.asarray(best), np.asarray(parents, np.int32), np.asarray(tokens, np.int32)
