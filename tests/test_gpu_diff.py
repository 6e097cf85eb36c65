"""Differential attention over the paged cache against its definition in 64 bits
(tests/diff_reference.py, which derives the tolerances).  Every slot of the pool
that holds no token of the batch is NaN: nothing masked may reach an output."""
import numpy as np
import pytest
import torch

import pa_workloads as wl
from tests import diff_reference as dr

pytestmark = pytest.mark.gpu

bits = wl.bf16_bits


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_167_gb300 as pa
    assert torch.cuda.is_available(), "a CUDA device is required"
    pa.get_device_error(clear=True)
    yield pa
    pa.set_stream_k_ctas(0)
    pa.set_prefill_ctas(0)


class Batch:
    """Sequences of `lens` cached tokens in a pool of NaN (layer 1 of `layers`)."""

    def __init__(self, lens, hq, hkv, d, b, seed=0, norm=True, layers=0, chunk=0, keys="map", spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.b, self.keys = list(lens), hq, hkv, d, b, keys
        B = len(self.lens)
        count = [-(-n // b) for n in self.lens]
        blocks = sum(count) + 3
        ids = rng.permutation(blocks).astype(np.int32)
        width = max(max(count, default=0), 1) + 1
        table = np.full((B, width), -1, np.int32)
        at = 0
        shape = (blocks, 2, layers, hkv, b, d) if layers else (blocks, 2, hkv, b, d)
        self.pool = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.layer = 1 if layers else None
        view = self.pool[:, :, 1] if layers else self.pool
        rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.k, self.v = [], []
        for s, n in enumerate(self.lens):
            own = ids[at:at + count[s]]
            at += count[s]
            table[s, :count[s]] = own
            k, v = rand(hkv, n, d), rand(hkv, n, d)
            self.k.append(k)
            self.v.append(v)
            pos = torch.arange(n, device="cuda")
            blk = torch.as_tensor(own, device="cuda").long()
            if n:
                view[blk[pos // b], 0, :, pos % b] = k.transpose(0, 1)
                view[blk[pos // b], 1, :, pos % b] = v.transpose(0, 1)
        self.tables = torch.as_tensor(table, device="cuda")
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.max_len = max(max(self.lens, default=0), 1)
        self.scale = d ** -0.5
        self.lam = 1.5 * torch.rand(hq // 2, generator=g, device="cuda") - 0.3
        self.weight = 1 + 0.2 * torch.randn(2 * d, generator=g, device="cuda") if norm else None
        self.eps, self.out_scale = 1e-5, (0.2 if norm else 1.0)
        self.chunk = chunk
        qs = (B, chunk, hq, d) if chunk else (B, hq, d)
        self.q = (torch.randn(qs, generator=g, device="cuda") * spread).to(torch.bfloat16)
        self.out = torch.full(qs[:-2] + (hq // 2, 2 * d), float("nan"), dtype=torch.bfloat16, device="cuda")

    def weights(self):
        return dict(lam=self.lam, norm_weight=self.weight, eps=self.eps, out_scale=self.out_scale, keys=self.keys)

    def workspace(self, pa):
        n = pa.decode_diff_workspace_size(self.pool, len(self.lens), self.hq, self.max_len, layer=self.layer)
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def decode(self, pa, out=None, workspace=None, **kw):
        out = self.out if out is None else out
        pa.decode_diff(out, self.q, self.pool, self.tables, self.lens_dev, self.max_len, self.scale,
                       workspace=self.workspace(pa) if workspace is None else workspace, layer=self.layer,
                       **self.weights(), **kw)
        return out

    def prefill(self, pa, **kw):
        """The last `chunk` tokens of each sequence as queries, the others as context."""
        ctx = [n - self.chunk for n in self.lens]
        self.ctx_dev = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        pa.prefill_diff(self.out, self.q, self.pool, self.tables, self.ctx_dev, max(ctx, default=0), self.scale,
                        layer=self.layer, **self.weights(), **kw)
        return self.out

    def check_prefill(self, pa, what="", only=None):
        for s in range(len(self.lens)) if only is None else only:
            seen = self.lens[s] - self.chunk + 1 + torch.arange(self.chunk, device="cuda")
            want, tol = self.want(s, seen)
            dr.check(self.out[s], want, tol, f"{what} sequence {s}, {self.chunk} of {self.lens[s]} tokens")
        assert pa.get_device_error() == 0

    def want(self, s, lens=None):
        """Of sequence s: the definition's output and the tolerance."""
        q = self.q[s] if self.chunk else self.q[s:s + 1]
        seen = torch.tensor([self.lens[s]], device="cuda") if lens is None else lens
        return dr.pairs(q, self.k[s], self.v[s], seen, self.scale, self.lam, self.weight, self.eps, self.out_scale,
                        self.keys == "head", terms=1 if self.chunk else 2)

    def check(self, pa, out=None, what=""):
        out = self.out if out is None else out
        for s in range(len(self.lens)):
            want, tol = self.want(s)
            dr.check(out[s:s + 1], want, tol, f"{what} sequence {s} of {self.lens[s]} tokens")
        assert pa.get_device_error() == 0


RAGGED = [1, 0, 15, 16, 17, 33, 64, 63, 200, 2, 129]


@pytest.mark.parametrize("b", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("per", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_diff(pa, d, per, b):
    x = Batch(RAGGED, 4 * per, 4, d, b, seed=b + per, norm=per != 2, keys="head" if b == 32 else "map")
    x.decode(pa)
    x.check(pa, what=f"d={d} R={per} b={b}")


@pytest.mark.parametrize("keys", ["map", "head"])
@pytest.mark.parametrize("per", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_diff_keys(pa, d, per, keys):
    """Either assignment of key heads, in a layer of a pool, two and six KV heads."""
    for hkv in (2, 6):
        x = Batch([70, 1, 31], hkv * per, hkv, d, 16, seed=per, layers=3, keys=keys)
        before = x.pool.clone()
        x.decode(pa)
        x.check(pa, what=keys)
        assert np.array_equal(bits(x.pool), bits(before))


@pytest.mark.parametrize("d,per,b", [(128, 8, 16), (64, 1, 32), (128, 1, 8), (64, 4, 4), (128, 4, 64)])
def test_decode_diff_cuts(pa, d, per, b):
    """Every way to cut units between CTAs, one CTA to one a stage: the merge's records."""
    x = Batch([300, 1, 0, 95, 17, 160], 2 * per, 2, d, b, seed=3)
    for ctas in (1, 2, 3, 5, 7, 16, 33, 152, 1000):
        pa.set_stream_k_ctas(ctas)
        x.out.fill_(float("nan"))
        x.decode(pa)
        x.check(pa, what=f"{ctas} CTAs")
    pa.set_stream_k_ctas(0)


@pytest.mark.parametrize("d,per,lens", [(128, 8, [9000, 3, 4097]), (64, 1, [20000]), (128, 1, [5000] * 3),
                                        (64, 2, list(range(1, 400, 3))), (128, 2, [40] * 300)])
def test_decode_diff_long_and_many(pa, d, per, lens):
    x = Batch(lens, 2 * per, 2, d, 16, seed=11)
    x.decode(pa)
    x.check(pa)


@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_decode_diff_flat_and_sharp(pa, spread):
    """Equal logits, and maps that a single key takes."""
    x = Batch([500, 3, 77], 8, 2, 128, 16, seed=5, spread=spread)
    x.decode(pa)
    x.check(pa)


@pytest.mark.parametrize("norm", [False, True])
def test_decode_diff_nothing_cached(pa, norm):
    """No sequence has a token: zeros, with a bound of 0 tokens and with a larger one."""
    for max_len in (0, 1, 5000):
        x = Batch([0] * 5, 8, 2, 64, 16, seed=1, norm=norm)
        x.max_len = max_len
        x.decode(pa)
        assert torch.equal(x.out, torch.zeros_like(x.out)) and pa.get_device_error() == 0


@pytest.mark.parametrize("scale", [0.0, -0.09, 1.5])
def test_decode_diff_scales(pa, scale):
    """Any finite scale; a negative one is the positive one of negated queries."""
    x = Batch([200, 3, 65], 16, 2, 128, 16, seed=4)
    x.scale = scale
    x.decode(pa)
    if scale < 0:
        x.scale, x.q = -scale, -x.q
    x.check(pa, what=f"scale {scale}")


def test_decode_diff_equal_maps_cancel(pa):
    """The same query and key heads in both maps, lambda 1: nothing is left, whatever a
    unit's cuts; the norm of zeros is zero."""
    x = Batch([333, 20], 4, 2, 64, 16, seed=6, keys="head")
    x.q[:, 1::2] = x.q[:, 0::2]
    x.lam.fill_(1.0)
    x.decode(pa)
    assert torch.equal(x.out, torch.zeros_like(x.out)) and pa.get_device_error() == 0


def test_decode_diff_of_zero_lambda_is_decode(pa):
    """lambda 0 without a norm: map 1 alone, which plain decode computes for keys by head
    (each half of a value row one head's)."""
    x = Batch([100, 257, 5], 8, 4, 128, 16, seed=7, norm=False, keys="map")
    x.lam.zero_()
    x.decode(pa)
    x.check(pa)
    # plain decode of the first maps: query heads 2h against key head 2g, value heads 2g and 2g + 1
    ws = torch.empty(max(pa.decode_workspace_size(x.pool, 3, 8, x.max_len), 1), dtype=torch.uint8, device="cuda")
    q, plain = torch.zeros_like(x.q), torch.empty_like(x.q)
    q[:, 0::4] = x.q[:, 0::4]          # pairs 0, 2: R = 2, so heads 0, 4 read key head 0, 2
    pa.decode(plain, q, x.pool, x.tables, x.lens_dev, x.max_len, x.scale, 0, ws)
    # two kernels' outputs, each within the definition's bound of the same value
    for s in range(3):
        _, tol = x.want(s)
        for pair, head in ((0, 0), (2, 4)):
            diff = (x.out[s, pair, :128].double() - plain[s, head].double()).abs()
            assert (diff <= 2 * tol[0, pair, :128]).all()


@pytest.mark.parametrize("d,per,b", [(128, 4, 16), (64, 8, 32), (64, 1, 4), (128, 8, 64), (128, 2, 8)])
@pytest.mark.parametrize("flags", [0, 1])
def test_decode_diff_stores_new_tokens(pa, d, per, b, flags):
    """The call stores each sequence's last token itself, bit for bit, and nothing else."""
    x = Batch([1, 16, 17, 0, 95, 64, 200], 2 * per, 2, d, b, seed=8, layers=2)
    stored = x.pool.clone()
    new_k = torch.zeros((7, 2, d), dtype=torch.bfloat16, device="cuda")
    new_v = torch.zeros_like(new_k)
    for s, n in enumerate(x.lens):
        if n:
            blk = int(x.tables[s, (n - 1) // b])
            new_k[s], new_v[s] = x.k[s][:, -1], x.v[s][:, -1]
            x.pool[blk, :, 1, :, (n - 1) % b] = float("nan")      # not there before the call
    x.decode(pa, flags=flags, new_k=new_k, new_v=new_v)
    x.check(pa)
    assert np.array_equal(bits(x.pool), bits(stored))


def test_decode_diff_captured_and_concurrent(pa):
    x = Batch([700, 40, 333], 16, 4, 128, 16, seed=9)
    ws = x.workspace(pa)
    x.decode(pa, workspace=ws)
    first = x.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.decode(pa, workspace=ws)
    x.q.neg_()                    # new inputs in the same buffers
    graph.replay()
    torch.cuda.synchronize()
    x.check(pa, what="replayed")
    assert not torch.equal(first, x.out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs, spaces = [torch.empty_like(x.out) for _ in streams], [x.workspace(pa) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, w, stream in zip(outs, spaces, streams):
            x.decode(pa, out=o, workspace=w, stream=stream)
    torch.cuda.synchronize()
    for o in outs:
        x.check(pa, out=o, what="two streams")


def test_decode_diff_bad_pages(pa):
    """Lengths and table entries out of range are reported and not followed."""
    x = Batch([100, 50, 20, 7], 4, 2, 64, 16, seed=10)
    x.tables[0, 2] = 10 ** 6
    x.tables[1, 0] = -3
    x.lens_dev[2] = 5000
    x.decode(pa)
    assert pa.get_device_error(clear=True) == 0x1 | 0x4
    want, tol = x.want(3)
    dr.check(x.out[3:4], want, tol, "the sequence without a fault")
    x.lens_dev[2] = -1
    x.decode(pa)
    assert pa.get_device_error(clear=True) == 0x1 | 0x4
    assert torch.equal(x.out[2], torch.zeros_like(x.out[2]))


def test_decode_diff_refusals_of_the_binding(pa):
    x = Batch([20, 3], 4, 2, 64, 16, seed=12)
    ws = x.workspace(pa)
    good = dict(out=x.out, q=x.q, pool=x.pool, block_tables=x.tables, seq_lens=x.lens_dev, max_seq_len=20,
                scale=0.125, workspace=ws, **x.weights())
    for kw in (dict(out=x.out[:, :1]), dict(q=x.q[:, :3]), dict(lam=x.lam[:1]), dict(norm_weight=x.weight[:64]),
               dict(keys="both"), dict(seq_lens=x.lens_dev[:1])):
        with pytest.raises(ValueError):
            pa.decode_diff(**{**good, **kw})
    for kw in (dict(lam=x.lam.double()), dict(norm_weight=x.weight.bfloat16()), dict(q=x.q.float()),
               dict(lam=x.lam.cpu())):
        with pytest.raises((TypeError, ValueError)):
            pa.decode_diff(**{**good, **kw})
    for kw, status in ((dict(workspace=ws[:100]), 3), (dict(workspace=None), 3), (dict(eps=0.0), 1),
                       (dict(out_scale=float("inf")), 1), (dict(flags=2), 1)):
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.decode_diff(**{**good, **kw})
        assert e.value.status == status
    assert pa.get_device_error() == 0


# ---------------------------------------------------------------------------
# chunks of prompt tokens
# ---------------------------------------------------------------------------

def chunked(ctx, chunk, *args, **kw):
    return Batch([c + chunk for c in ctx], *args, chunk=chunk, **kw)


@pytest.mark.parametrize("b", [8, 16, 32, 64])
@pytest.mark.parametrize("per", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_diff(pa, d, per, b):
    x = chunked([0, 1, 127, 300], 40, 2 * per, 2, d, b, seed=b + per, norm=per != 2)
    x.prefill(pa)
    x.check_prefill(pa, f"d={d} R={per} b={b}")


@pytest.mark.parametrize("chunk", [1, 2, 15, 16, 17, 31, 64, 128, 129, 200, 333])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_diff_chunks(pa, d, chunk):
    """Chunks from one token on, whole and partial tiles of queries."""
    x = chunked([0, 63, 64, 65, 200], chunk, 8, 2, d, 16, seed=chunk)
    x.prefill(pa)
    x.check_prefill(pa)


@pytest.mark.parametrize("per", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_diff_keys_by_head(pa, d, per):
    for hkv in (2, 4):
        x = chunked([0, 77], 150, hkv * per, hkv, d, 32, seed=per, layers=2, keys="head")
        before = x.pool.clone()
        x.prefill(pa)
        x.check_prefill(pa)
        assert np.array_equal(bits(x.pool), bits(before))


@pytest.mark.parametrize("ctas", [1, 2, 4, 6, 20, 152])
def test_prefill_diff_hand_overs(pa, ctas):
    """One cluster walking every unit, up to one a pair of SMs: units of one tile and of
    many behind one another, with and without the norm's exchange."""
    pa.set_prefill_ctas(ctas)
    for d, per, norm in ((128, 4, True), (64, 1, True), (128, 1, False)):
        x = chunked([0, 500, 3, 100], 70, 2 * per, 2, d, 16, seed=ctas, norm=norm)
        x.prefill(pa)
        x.check_prefill(pa, f"{ctas} CTAs")
    pa.set_prefill_ctas(0)


@pytest.mark.parametrize("d,per,ctx,chunk", [(128, 8, [4000, 17], 256), (64, 2, [9000], 100), (128, 1, [0], 3100),
                                             (128, 4, [0] * 40, 33)])
def test_prefill_diff_long_and_many(pa, d, per, ctx, chunk):
    x = chunked(ctx, chunk, 2 * per, 2, d, 16, seed=21)
    x.prefill(pa)
    x.check_prefill(pa)


@pytest.mark.parametrize("spread", [0.0, 25.0])
def test_prefill_diff_flat_and_sharp(pa, spread):
    """Equal logits, and maps that move their maximum often."""
    x = chunked([700, 0], 130, 8, 2, 128, 16, seed=22, spread=spread)
    x.prefill(pa)
    x.check_prefill(pa)


@pytest.mark.parametrize("d,norm", [(64, True), (128, True), (128, False)])
def test_prefill_diff_equal_maps_cancel(pa, d, norm):
    """As in decode: the maps meet as the same bits, so nothing is left."""
    x = Batch([300, 77, 150], 8, 4, d, 16, seed=6, keys="head", chunk=70, norm=norm)
    x.q[:, :, 1::2] = x.q[:, :, 0::2]
    x.lam.fill_(1.0)
    x.prefill(pa)
    assert torch.equal(x.out, torch.zeros_like(x.out)) and pa.get_device_error() == 0


def test_prefill_diff_agrees_with_decode(pa):
    """A chunk of one token is a decode step: both within the definition's bounds."""
    x = chunked([300, 64, 0], 1, 16, 4, 128, 16, seed=23)
    x.prefill(pa)
    x.check_prefill(pa)
    out = torch.empty((3, 8, 256), dtype=torch.bfloat16, device="cuda")
    pa.decode_diff(out, x.q[:, 0].contiguous(), x.pool, x.tables, x.lens_dev, x.max_len, x.scale,
                   workspace=x.workspace(pa), **x.weights())
    for s in range(3):
        want, tol = x.want(s, torch.tensor([x.lens[s]], device="cuda"))
        dr.check(out[s:s + 1], want, tol, "decode")


def test_prefill_diff_captured_and_concurrent(pa):
    x, y = (chunked([200, 40], 130, 8, 2, 128, 16, seed=24 + i) for i in range(2))
    x.prefill(pa)
    graph = torch.cuda.CUDAGraph()
    ctx = x.ctx_dev
    with torch.cuda.graph(graph):
        pa.prefill_diff(x.out, x.q, x.pool, x.tables, ctx, 200, x.scale, **x.weights())
    x.q.neg_()
    graph.replay()
    torch.cuda.synchronize()
    x.check_prefill(pa, "replayed")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    x.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(4):
        for one, stream in zip((x, y), streams):
            pa.prefill_diff(one.out, one.q, one.pool, one.tables, ctx, 200, one.scale, stream=stream,
                            **one.weights())
    torch.cuda.synchronize()
    x.check_prefill(pa, "two streams")
    y.check_prefill(pa, "two streams")


def test_prefill_diff_bad_pages(pa):
    x = chunked([100, 50, 20], 30, 4, 2, 64, 16, seed=26)
    x.tables[0, 2] = 10 ** 6
    x.tables[0, 3] = -3
    x.ctx_dev = torch.tensor([100, 5000, 20], dtype=torch.int32, device="cuda")
    pa.prefill_diff(x.out, x.q, x.pool, x.tables, x.ctx_dev, 100, x.scale, **x.weights())
    assert pa.get_device_error(clear=True) == 0x1 | 0x4
    x.check_prefill(pa, only=[2])


def test_prefill_diff_refusals_of_the_binding(pa):
    x = chunked([20, 3], 5, 4, 2, 64, 16, seed=27)
    x.prefill(pa)
    good = dict(out=x.out, q=x.q, pool=x.pool, block_tables=x.tables, ctx_lens=x.ctx_dev, max_ctx_len=20,
                scale=0.125, **x.weights())
    for kw in (dict(out=x.out[:, :1]), dict(q=x.q[:, :, :3]), dict(lam=x.lam[:1]), dict(keys="both"),
               dict(ctx_lens=x.ctx_dev[:1])):
        with pytest.raises(ValueError):
            pa.prefill_diff(**{**good, **kw})
    for kw in (dict(lam=x.lam.double()), dict(q=x.q.float()), dict(ctx_lens=x.ctx_dev.cpu())):
        with pytest.raises((TypeError, ValueError)):
            pa.prefill_diff(**{**good, **kw})
    for kw in (dict(eps=-1.0), dict(scale=0.0), dict(max_ctx_len=4000)):
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.prefill_diff(**{**good, **kw})
        assert e.value.status == 1
    assert pa.get_device_error() == 0
