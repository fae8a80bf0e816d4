"""kv_rope and kv_rope_append against their definition in 64 bits (tests/more_util.py, which
derives the tolerance): types, layouts, parts of the head, positions far and negative, chunks
of one token and of many, every page size, the page index, and how a program uses them."""
import pytest
import torch

from chunk_util import D, TORCH, Problem
from more_util import frequencies, near_2pi, turned, turned_tolerance
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


def near(got, want, tol):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    over = (got - want).nan_to_num().abs() - tol.nan_to_num()
    assert float(over.max()) <= 0, float(over.max())


class Chunk:
    """A batch whose chunks are turned, and appended to a cache of its type that holds
    random tokens before them."""

    def __init__(self, dtype, hq, hkv, ps, before, news, rot=128, inter=False, scale=1.0,
                 given=None, loc="hbm", seed=0, max_new=None, base=10000.0, freq=None):
        lens = [a + n for a, n in zip(before, news)]
        self.p = p = Problem(dtype, hq, hkv, ps, lens, news, seed=seed, loc=loc)
        p.k.nan_to_num_(nan=3.0)
        p.v.nan_to_num_(nan=-3.0)
        p.upload(max_new=max_new)
        g = torch.Generator().manual_seed(seed + 1)
        t = TORCH[dtype]
        self.before = list(before)
        self.q = torch.randn(p.total, hq, D, generator=g).to(t)
        self.k = torch.randn(p.total, hkv, D, generator=g).to(t)
        self.v = torch.randn(p.total, hkv, D, generator=g).to(t)
        self.freq = frequencies(rot, base) if freq is None else freq
        self.inter, self.scale, self.rot = inter, scale, rot
        at = torch.zeros(p.total, dtype=torch.int64)
        for b, n in enumerate(news):
            at[p.start[b]:p.start[b] + n] = torch.arange(before[b], before[b] + n)
        self.at = at if given is None else given
        self.d_at = None if given is None else given.to(torch.int32).cuda()
        self.d_freq = self.freq.cuda()
        self.plan = kv.make_rope(self.d_freq, rot, inter, scale, self.d_at)
        self.d = {n: getattr(self, n).cuda() for n in "qkv"}
        self.ctx = torch.tensor(before, dtype=torch.int32, device="cuda")
        self.q_out = torch.full_like(self.d["q"], 7.0)
        self.k_out = torch.full_like(self.d["k"], 7.0)
        self.mine = torch.zeros(p.total, dtype=torch.bool)
        self.mine[:p.start[-1]] = True

    def rows(self, x):
        """The definition of x's rows, 7 where no sequence owns one, and the tolerance."""
        want = turned(x, self.at, self.freq, self.inter, self.scale)
        tol = turned_tolerance(x, self.p.dtype, self.rot // 2, self.inter, self.scale, self.at, self.freq)
        want[~self.mine], tol[~self.mine] = 7.0, 0.0
        return want, tol

    def turn(self, q=True, k=True, in_place=False, stream=None):
        st = torch.cuda.current_stream() if stream is None else stream
        p, d = self.p, self.d
        q_out = d["q"] if in_place else self.q_out
        k_out = d["k"] if in_place else self.k_out
        kv.kv_rope(p.shape, p.chunk, self.plan, d["q"] if q else None, q_out if q else None,
                   d["k"] if k else None, k_out if k else None,
                   self.ctx if self.d_at is None else None, st)
        return q_out, k_out

    def put(self, ctx_out=None, mm=None, rope=True, q=True, stream=None):
        st = torch.cuda.current_stream() if stream is None else stream
        p, d = self.p, self.d
        q = q and rope
        kv.kv_rope_append(p.shape, p.chunk, self.plan if rope else None, d["q"] if q else None,
                          self.q_out if q else None, d["k"], d["v"], p.d_k, p.d_v, p.d_table, self.ctx,
                          ctx_out, mm, st)
        torch.cuda.synchronize()

    def check_cache(self, rope=True, skip=()):
        p = self.p
        want_k, tol_k = p.k.double(), torch.zeros_like(p.k, dtype=torch.float64)
        want_v = p.v.double()
        k, tol = self.rows(self.k) if rope else (self.k.double(), torch.zeros(self.k.shape).double())
        for b, n in enumerate(p.news):
            for i in range(n):
                pos = self.before[b] + i
                ph = int(p.table[b, pos // p.ps])
                if b in skip or not 0 <= ph < p.pages:
                    continue
                want_k[ph, :, pos % p.ps] = k[p.start[b] + i]
                tol_k[ph, :, pos % p.ps] = tol[p.start[b] + i]
                want_v[ph, :, pos % p.ps] = self.v[p.start[b] + i].double()
        near(p.d_k, want_k, tol_k)
        assert torch.equal(p.d_v.double().cpu(), want_v)

    def index(self):
        """What the index holds before the append (5 where a page has no token)."""
        p = self.p
        mm = torch.full((p.pages, p.hkv, 2, D), 5.0, dtype=TORCH[p.dtype], device="cuda")
        self.build(mm, self.ctx)
        kv.kv_device_status()  # (the build takes lengths from 1 on, and records the others)
        return mm

    def build(self, mm, ctx):
        p = self.p
        kv.kv_page_minmax_build(p.shape, p.d_k, p.d_table, ctx, mm, torch.cuda.current_stream())


SHAPES = [
    (8, 2, 16, [0, 15, 16, 100, 33], [1, 1, 1, 0, 1]),
    (4, 4, 32, [0, 31, 7], [70, 1, 33]),
    (7, 1, 64, [63, 0], [2, 129]),
    (6, 3, 128, [5], [300]),
    (32, 32, 16, [17, 0, 1], [5, 16, 40]),
    (64, 2, 16, [3, 50], [9, 3]),
]
ROTS = [(128, False), (128, True), (64, False), (96, True), (24, False), (8, True), (8, False)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rot,inter", ROTS)
def test_rows(dtype, rot, inter):
    for i, (hq, hkv, ps, before, news) in enumerate(SHAPES):
        c = Chunk(dtype, hq, hkv, ps, before, news, rot, inter, seed=i, scale=1.0 if i % 2 else 1.25)
        c.turn()
        torch.cuda.synchronize()
        near(c.q_out, *c.rows(c.q))
        near(c.k_out, *c.rows(c.k))
        # channels behind the turned ones keep their bits
        x, y = c.q_out[c.mine][..., rot:], c.d["q"][c.mine][..., rot:]
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_one_kind_and_in_place(dtype):
    c = Chunk(dtype, 8, 2, 16, [3, 40], [20, 7], 64)
    for kind, other in (("q", "k"), ("k", "q")):
        c.turn(**{other: False})
        out, left = getattr(c, kind + "_out"), getattr(c, other + "_out")
        near(out, *c.rows(getattr(c, kind)))
        assert (left == 7).all()
        out.fill_(7)
    c.turn()
    q, k = c.turn(in_place=True)
    assert torch.equal(q[c.mine], c.q_out[c.mine]) and torch.equal(k[c.mine], c.k_out[c.mine])
    assert torch.equal(q[~c.mine].cpu(), c.q[~c.mine])  # rows no sequence owns


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("inter", [False, True])
def test_given_positions(dtype, inter):
    """Far, negative and repeated ones; turning by -t undoes turning by t."""
    g = torch.Generator().manual_seed(2)
    c0 = Chunk(dtype, 4, 2, 16, [0, 9], [40, 11])
    at = torch.randint(-(1 << 31), 1 << 31, (c0.p.total,), generator=g)
    at[:9] = torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), 1 << 20, 1 << 20, 131071, -131072])
    c = Chunk(dtype, 4, 2, 16, [0, 9], [40, 11], 64, inter, given=at)
    c.turn()
    # the angles by integers: 64 bits lose those of such positions
    angle = near_2pi(c.freq, at)
    want = c.q.double().clone()
    half = 32
    j = torch.arange(half)
    a, b = (2 * j, 2 * j + 1) if inter else (j, j + half)
    u, v = want[..., a].clone(), want[..., b].clone()
    cs, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    want[..., a], want[..., b] = u * cs - v * sn, u * sn + v * cs
    want[~c.mine] = 7.0
    tol = c.rows(c.q)[1]
    # (the frequency is kept to 2^-63 turns: times 2^31 positions, 2^-29 radians at most)
    near(c.q_out, want, tol + 2.0 ** -29 * c.q.double().abs().max())
    ok = torch.arange(c.p.total) != 4  # (-2^31 has no opposite)
    back = Chunk(dtype, 4, 2, 16, [0, 9], [40, 11], 64, inter, given=torch.where(ok, -at, 0))
    back.d["q"].copy_(c.q_out)
    back.turn()
    size = c.q.double().abs().max()
    eps = torch.finfo(TORCH[dtype]).eps / 2
    lim = 2 * (2 * eps + 2.0 ** -20) * 2 * size  # two roundings and two turnings
    rows = c.mine & ok
    assert float((back.q_out[rows].double().cpu() - c.q[rows].double()).abs().max()) <= lim


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_frequencies(dtype):
    """Zero, tiny, negative, above a turn per position, powers of two."""
    freq = torch.tensor([0.0, 1e-300, 2.0 ** -70, 2.0 ** -64, 1e-19, 1e-9, -0.5, 1.0, -3.0, 6.283185307179586,
                         7.0, 100.0, 1e6, 2.0 ** 40, 2.0 ** 53, 3e-5], dtype=torch.float64)
    c = Chunk(dtype, 2, 1, 16, [0], [33], 32, freq=freq)
    c.turn()
    angle = near_2pi(freq, c.at)
    want = c.q.double().clone()
    u, v = want[..., :16].clone(), want[..., 16:32].clone()
    cs, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    want[..., :16], want[..., 16:32] = u * cs - v * sn, u * sn + v * cs
    want[~c.mine] = 7.0
    tol = turned_tolerance(c.q, dtype, 16)
    # (1 / 2 pi is kept to 66 bits: an angle a to a * 2^-63, 32 positions on; the others far finer)
    loose = torch.where(freq.abs() >= 2.0 ** 40, 32 * freq.abs() * 2.0 ** -63, 0.0)
    tol[..., :16] += 4 * loose
    tol[..., 16:32] += 4 * loose
    tol[~c.mine] = 0.0
    near(c.q_out, want, tol)


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_append(dtype, loc):
    for i, (hq, hkv, ps, before, news) in enumerate(SHAPES):
        rot, inter = ROTS[i]
        c = Chunk(dtype, hq, hkv, ps, before, news, rot, inter, loc=loc, seed=i)
        out = torch.full((len(news),), -9, dtype=torch.int32, device="cuda")
        c.put(out)
        c.check_cache()
        near(c.q_out, *c.rows(c.q))
        assert out.tolist() == c.p.lens and c.ctx.tolist() == before
        # the same bits as the rows turned by themselves
        c.turn()
        q = c.q_out.clone()
        c.put(out)
        assert torch.equal(q, c.q_out)
        for b, n in enumerate(news):
            for r in range(n):
                pos = before[b] + r
                at = int(c.p.table[b, pos // ps])
                assert torch.equal(c.p.d_k[at, :, pos % ps].cpu(), c.k_out[c.p.start[b] + r].cpu())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_without_turning(dtype):
    """Keys with NaN of any bits, infinities and zeros of both signs are stored as they are."""
    for hq, hkv, ps, before, news in SHAPES[:4]:
        c = Chunk(dtype, hq, hkv, ps, before, news)
        bits = torch.int32 if dtype == "f32" else torch.int16
        g = torch.Generator().manual_seed(4)
        info = torch.iinfo(bits)
        for n in "kv":
            raw = torch.randint(info.min, info.max, c.d[n].shape, generator=g, dtype=bits)
            c.d[n] = raw.view(TORCH[dtype]).cuda()
        c.put(rope=False)
        for name, cache in (("k", c.p.d_k), ("v", c.p.d_v)):
            for b, n in enumerate(news):
                for r in range(n):
                    pos = before[b] + r
                    at = int(c.p.table[b, pos // ps])
                    assert torch.equal(cache[at, :, pos % ps].view(bits), c.d[name][c.p.start[b] + r].view(bits))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_index(dtype):
    """Bit-identical to the build on the new lengths, in pages opened and continued, of every size."""
    bits = torch.int32 if dtype == "f32" else torch.int16
    for i, (hq, hkv, ps, before, news) in enumerate(SHAPES):
        for rope in (True, False):
            c = Chunk(dtype, hq, hkv, ps, before, news, seed=i)
            c.k[:, :, ::5] = 0.0
            c.k[:, :, 1::10] = -0.0
            c.d["k"].copy_(c.k)
            mm = c.index()
            untouched = mm.clone()
            out = torch.zeros(len(news), dtype=torch.int32, device="cuda")
            c.put(out, mm, rope)
            c.build(untouched, out)
            torch.cuda.synchronize()
            assert torch.equal(mm.view(bits), untouched.view(bits))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,ps,rot,inter", [(32, 8, 16, 128, False), (14, 7, 32, 64, True), (32, 8, 64, 72, False),
                                                 (24, 12, 128, 128, True), (8, 8, 16, 8, False)])
def test_many_sequences(dtype, hq, hkv, ps, rot, inter):
    """Enough blocks for several kv heads to share one: rows, the append, its index."""
    bits = torch.int32 if dtype == "f32" else torch.int16
    g = torch.Generator().manual_seed(hq + ps)
    before = torch.randint(0, 140, (270,), generator=g).tolist()
    news = torch.randint(0, 41, (270,), generator=g).tolist()
    c = Chunk(dtype, hq, hkv, ps, before, news, rot, inter, max_new=40)
    mm = c.index()
    anew = mm.clone()
    out = torch.zeros(len(news), dtype=torch.int32, device="cuda")
    c.put(out, mm)
    c.check_cache()
    near(c.q_out, *c.rows(c.q))
    c.build(anew, out)
    torch.cuda.synchronize()
    assert torch.equal(mm.view(bits), anew.view(bits)) and out.tolist() == c.p.lens
    q = c.q_out.clone()
    c.q_out.fill_(7.0)
    c.put(out)  # without an index the tiles are of 16 tokens
    assert torch.equal(q, c.q_out)
    c.check_cache()
    c.turn()
    torch.cuda.synchronize()
    near(c.k_out, *c.rows(c.k))
    assert torch.equal(q, c.q_out)


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 0, 7], [1000, 3, 64], [0, 0, 0]])
@pytest.mark.parametrize("index", [False, True])
@pytest.mark.parametrize("hq,hkv", [(8, 4), (10, 5), (3, 1)])
def test_lengths_in_place(news, index, hq, hkv):
    before = [5, 9, 0]
    c = Chunk("bf16", hq, hkv, 16, before, news)
    c.put(c.ctx, c.index() if index else None)
    c.check_cache()
    assert c.ctx.tolist() == [x + n for x, n in zip(before, news)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("index", [False, True])
def test_skips_what_is_out_of_range(index, in_place):
    """A bad page drops its tokens and keeps the length; a bad length or chunk skips the sequence."""
    news, before = [40, 20, 6, 5], [0, 3, 2, 4]
    c = Chunk("f16", 4, 2, 16, before, news)
    p = c.p
    mm = c.index() if index else None
    p.table[0, 1] = p.pages
    p.d_table.copy_(p.table)
    c.ctx[2] = p.max_pages * 16 - 5  # six tokens do not fit
    out = c.ctx if in_place else torch.full((4,), -9, dtype=torch.int32, device="cuda")
    c.put(out, mm)
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    c.check_cache(skip=(2,))
    assert out.tolist() == [0, 23, p.max_pages * 16 - 5, 9]
    want, tol = c.rows(c.q)
    want[p.start[2]:p.start[3]], tol[p.start[2]:p.start[3]] = 7.0, 0.0
    near(c.q_out, want, tol)
    # a chunk longer than the launch was sized for, and starts out of order
    for start in ([0, 41, 45, 50, 55], [0, 40, 30, 50, 71], [-1, 40, 60, 66, 71]):
        c = Chunk("f16", 2, 2, 16, before, news, max_new=40)
        c.p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        c.put(out, mm)
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
        c.turn()
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    c = Chunk("f16", 2, 2, 16, before, news)
    for bad in (-1, (1 << 31) - 10):
        c.ctx[1] = bad
        c.turn()
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
        want, tol = c.rows(c.q)
        want[40:60], tol[40:60] = 7.0, 0.0
        near(c.q_out, want, tol)


def test_a_graph_and_another_stream():
    c = Chunk("bf16", 8, 2, 16, [5, 30], [1, 1])
    # (the third replay opens a page: one that nobody has)
    c.p.table[1, 2] = next(i for i in range(c.p.pages) if i not in c.p.table)
    c.p.d_table.copy_(c.p.table)
    mm = c.index()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    kv_call = lambda: kv.kv_rope_append(  # noqa: E731
        c.p.shape, c.p.chunk, c.plan, c.d["q"], c.q_out, c.d["k"], c.d["v"], c.p.d_k, c.p.d_v,
        c.p.d_table, c.ctx, c.ctx, mm, st)
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            kv_call()
        for _ in range(3):
            graph.replay()
    st.synchronize()
    assert c.ctx.tolist() == [8, 33]
    for b, pos0 in enumerate((5, 30)):
        for step in range(3):
            pos = pos0 + step
            at = torch.full((c.p.total,), pos)
            want = turned(c.k, at, c.freq)[b]
            tol = turned_tolerance(c.k, "bf16", 64)[b]
            near(c.p.d_k[int(c.p.table[b, pos // 16]), :, pos % 16], want, tol)
    want = mm.clone()
    c.build(want, c.ctx)
    assert torch.equal(want, mm)


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_path_together(dtype, loc):
    """DecodeLayer: prompts, a few proposed tokens, single tokens appended with their
    positions; the chunk attention over them, and the sparse step through the index kept."""
    from offloaded_kv_cache_gb300 import workloads as W
    from offloaded_kv_cache_gb300.pipeline import DecodeLayer, Rotary
    spec = W.tiny_spec(dtype=dtype, batch=2, hq=8, hkv=2, context=200, ps=16, topk=4, index=5)
    layer = DecodeLayer(W.generate(spec, context_lens=[200, 170]), kv_loc=loc)
    layer.context_lens.zero_()
    rotary = Rotary(64, base=500000.0, stretch=4.0)
    t, g = TORCH[dtype], torch.Generator().manual_seed(1)
    for n in ([150, 120], [5, 0], [1, 1], [1, 1]):
        start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        k, v = (torch.randn(sum(n), 2, D, generator=g).to(t).cuda() for _ in "kv")
        q = torch.randn(sum(n), 8, D, generator=g).to(t).cuda()
        old = layer.context_lens.tolist()
        got = layer.append_chunk(k, v, start, max(n), rotary, q)
        at = torch.cat([torch.arange(o, o + m) for o, m in zip(old, n)])
        near(got, turned(q.cpu(), at, rotary.freq.cpu(), False, rotary.scale),
             turned_tolerance(q.cpu(), dtype, 32, False, rotary.scale, at, rotary.freq.cpu()))
        assert layer.context_lens.tolist() == [o + m for o, m in zip(old, n)]
        out = layer.chunk_attn(got, start, max(n))
    kept = layer.minmax.clone()
    layer.build_index()
    assert torch.equal(kept, layer.minmax)
    # every page selected: the sparse step is the chunk attention of the last token
    layer.q.copy_(got)
    layer.topk = spec.max_pages
    layer.indices = torch.empty((2, 8, spec.max_pages), dtype=torch.int32, device="cuda")
    layer.workspace = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    layer.sparse_step()
    torch.cuda.synchronize()
    # both compute the same sums, each within 2^-8 (2^-11, 2^-24) of weights and result
    tol = {"f32": 1e-5, "f16": 2.0 ** -9, "bf16": 2.0 ** -6}[dtype]
    assert float((layer.out - out.float()).abs().max()) <= tol * 6


def test_q8_cache_with_a_rotary():
    """Q8Cache.append turns its keys first: the bits of kv_rope and then kv_q8_append."""
    from offloaded_kv_cache_gb300.pipeline import Q8Cache, Rotary
    c = Chunk("bf16", 8, 2, 16, [0, 0], [40, 7], 64)
    rotary = Rotary(64)
    caches = []
    for turn_first in (False, True):
        ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
        cache = Q8Cache(c.p.shape, c.p.d_table, ctx)
        start = c.p.d_start
        if turn_first:
            c.turn()
            cache.append(c.k_out, c.d["v"], start, 40)
        else:
            q = cache.append(c.d["k"], c.d["v"], start, 40, rotary=rotary, q=c.d["q"])
        assert ctx.tolist() == [40, 7]
        caches.append(cache)
    assert torch.equal(q[c.mine], c.q_out[c.mine])
    assert torch.equal(caches[0].k_codes, caches[1].k_codes)
    assert torch.equal(caches[0].k_scale, caches[1].k_scale)
