"""kv_chunk_attn and kv_q8_chunk_attn against their definition in 64 bits
(tests/chunk_util.py, which also derives the tolerance): types, head groups,
page sizes, ragged lengths, windows, empty rows, bad pages, what unseen tokens
hold, and how a program uses the calls (graphs, streams, the whole path)."""
import math

import pytest
import torch

from chunk_util import D, TORCH, Problem, check
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


def run(p):
    p.upload()
    p.attend()
    torch.cuda.synchronize()
    check(p.d_out, *p.expected())
    return p


# lengths (with the chunk's own tokens) and chunk sizes
RAGGED = [
    ([1], [1]),
    ([17], [17]),
    ([300, 1, 64, 129], [1, 1, 1, 1]),
    ([200, 5, 131, 64, 0], [7, 0, 131, 3, 0]),
    ([513, 128], [257, 128]),
    ([1025, 40], [3, 40]),
]


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,news", RAGGED, ids=[str(i) for i in range(len(RAGGED))])
def test_ragged(dtype, lens, news, q8):
    run(Problem(dtype, 4, 2, 16, lens, news, q8=q8, seed=len(lens)))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (8, 1), (14, 2), (3, 3), (96, 1)])
@pytest.mark.parametrize("n", [1, 9, 50])
def test_head_groups(dtype, hq, hkv, n, q8):
    run(Problem(dtype, hq, hkv, 32, [150, 61], [n, 1], q8=q8, seed=hq))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,window", [("f16", 0), ("bf16", 100), ("f32", 33)])
def test_page_sizes(dtype, ps, window, q8):
    run(Problem(dtype, 8, 2, ps, [ps * 3 + 1, ps - 1, 401], [40, ps - 1, 5], window, q8=q8, seed=ps))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300])
def test_windows(dtype, window, q8):
    run(Problem(dtype, 2, 1, 16, [420, 90], [140, 90], window, q8=q8, seed=window))


# few rows per kv head: units of 8, 16, 64 and 128 packed rows
FEW = [(8, 2, 2), (8, 1, 1), (7, 1, 2), (16, 1, 1), (4, 1, 4), (6, 2, 11), (8, 1, 8), (8, 1, 16)]


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,n", FEW)
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("ps", [16, 128])
def test_few_rows(dtype, hq, hkv, n, window, ps, q8):
    run(Problem(dtype, hq, hkv, ps, [n + 120, n, 390, 5], [n, n, 1, 0], window, q8=q8, seed=n))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [2, 20])
def test_few_rows_with_vectors_of_very_different_size(dtype, n):
    """Keys and values of the 8-bit cache whose scales differ by up to 2^20, queries
    whose rows do; scores reach tens either way."""
    p = Problem(dtype, 4, 2, 16, [300, 64], [n, 1], q8=True, seed=n)
    g = torch.Generator().manual_seed(5)
    for name in "kv":
        scale = p.scale8[name]
        lo = 127 - (15 if dtype == "f16" else 20)
        new = torch.randint(lo, 121, scale.shape, generator=g).to(torch.uint8)
        p.scale8[name] = torch.where(scale == 255, scale, new)
    p.q = (p.q.float() * torch.exp2(torch.randint(-12, 3, (p.total, 4, 1), generator=g).float())
           ).to(TORCH[dtype])
    run(p)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing(dtype, q8):
    """Fewer cached tokens than the chunk has rows: the first rows see none and are 0."""
    run(Problem(dtype, 4, 2, 16, [3, 0, 140], [10, 5, 200], q8=q8))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype,scale,q_size", [
    ("f32", -0.2, 1.0), ("bf16", -0.2, 1.0), ("f16", 0.0, 1.0), ("bf16", 1.0, 16.0),
    ("f16", 0.5, 8.0), ("f32", 1.0, 8.0)])
@pytest.mark.parametrize("n", [3, 20, 150])
def test_scales(dtype, scale, q_size, n, q8):
    """Negative and zero scales, and scores in the hundreds (one weight near 1)."""
    run(Problem(dtype, 4, 2, 16, [260, 30], [n, 1], scale=scale, q_size=q_size, q8=q8))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("n", [4, 30, 150])
def test_running_maximum_moves(dtype, order, n, q8):
    """Scores that rise (fall) by 20 powers of two from tile to tile."""
    p = Problem(dtype, 2, 1, 16, [700], [n], q8=False, scale=1.0)
    ramp = order * torch.linspace(-100, 100, 700)
    p.q = torch.zeros_like(p.q)
    p.q[:, :, 0] = 1
    for j in range(700):
        p.k[p.table[0, j // 16], :, j % 16, 0] = ramp[j]
    if q8:
        from chunk_util import quantise
        p.q8, p.code, p.scale8 = True, {}, {}
        for n in "kv":
            c, s = quantise(getattr(p, n).double().numpy(), dtype)
            p.code[n], p.scale8[n] = torch.from_numpy(c), torch.from_numpy(s)
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_unseen_tokens_do_not_reach_a_row(dtype, window, what):
    """Non-finite values in one token's K and V, in the middle of the chunk:
    rows that see it are NaN in its channels, the others untouched."""
    p = Problem(dtype, 4, 2, 16, [300, 40], [160, 10], window)
    for j, c in ((200, 3), (290, 99), (145, 64)):
        p.v[p.table[0, j // 16], 1, j % 16, c] = what
    p.upload()
    p.attend()
    want, tol = p.expected()
    got = p.d_out.double().cpu()
    # a row that sees an infinite value may hold the infinity instead of NaN
    got[torch.isinf(got)] = math.nan
    check(got, want, tol)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_unseen_keys_do_not_reach_a_row(dtype):
    p = Problem(dtype, 2, 1, 16, [200], [100])
    p.k[p.table[0, 150 // 16], :, 150 % 16] = math.nan
    run(p)


@pytest.mark.parametrize("n", [100, 51, 20, 7])
def test_unseen_8_bit_vectors_do_not_reach_a_row(n):
    for name in "kv":
        for dtype in ("f16", "bf16", "f32"):
            p = Problem(dtype, 2, 1, 16, [160, 33], [n, 1], q8=True)
            p.code[name][p.table[0, 155 // 16], :, 155 % 16] = 0x7F
            p.scale8[name][p.table[0, 155 // 16], :, 155 % 16] = 255
            run(p)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_bad_pages_are_skipped(dtype, q8):
    p = Problem(dtype, 4, 2, 16, [150, 40, 300], [30, 1, 2], q8=q8)
    p.table[0, 3] = p.pages
    p.table[2, 0] = -1
    p.table[2, 18] = 1 << 30
    p.upload()
    p.attend()
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_sequences_are_skipped(dtype, q8):
    p = Problem(dtype, 4, 2, 16, [150, 40, 300], [30, 1, 20], q8=q8)
    p.upload(max_new=25)
    p.d_lens[1] = p.max_pages * 16 + 1
    p.attend()
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    want, tol = p.expected()
    want[:31], tol[:31] = 7, 0
    check(p.d_out, want, tol)
    p.d_lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
    p.d_out.fill_(7)
    for start in ([0, 30, 20, 40], [0, 30, 31, 1 << 20], [-5, 0, 1, 21]):
        p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        p.attend()
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("lens,news", [([150, 40], [30, 1]), ([900, 20], [1, 1])])
def test_host_resident_cache(dtype, lens, news, q8):
    run(Problem(dtype, 8, 2, 16, lens, news, q8=q8, loc="host"))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype,hq,hkv,lens,news", [
    ("bf16", 32, 8, [5000, 3000], [1, 1]),
    ("f16", 8, 1, [9000], [70]),
    ("bf16", 4, 4, [257] * 40, [33] * 40),
    ("f32", 2, 1, [4097], [65])])
def test_longer_and_many(dtype, hq, hkv, lens, news, q8):
    """Units that many CTAs share, and many units per CTA."""
    run(Problem(dtype, hq, hkv, 64, lens, news, q8=q8))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,most,n", [(33, 300, 1), (33, 300, 90), (70, 200, 5), (600, 60, 3),
                                          (1100, 17, 1)])
def test_many_sequences(dtype, batch, most, n, q8):
    """More sequences than a CTA has warps, lanes of a warp, threads; some empty."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, most, (batch,), generator=g).tolist()
    news = [min(x, int(torch.randint(0, n + 1, (1,), generator=g))) for x in lens]
    run(Problem(dtype, 4, 2, 16, lens, news, q8=q8, seed=n))


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype,hq,hkv,ps,lens,news,window", [
    ("bf16", 8, 2, 16, [2600, 1300, 1101], [150, 90, 40], 1100),
    ("f16", 2, 2, 128, [1500, 1400], [300, 1], 1030),
    ("f16", 4, 1, 64, [9000, 4300], [20, 25], 4200),
    ("bf16", 6, 1, 32, [4500], [9], 4097)])
def test_long_windows(dtype, hq, hkv, ps, lens, news, window, q8):
    """Windows that end in long contexts, and vectors that are not finite before, at and
    in them."""
    p = Problem(dtype, hq, hkv, ps, lens, news, window, q8=q8)
    if not q8:
        first = lens[0] - news[0]  # the first row's token
        for j, c in ((first - window, 5), (first - window + 3, 77), (first - 40, 20)):
            p.v[p.table[0, j // ps], 0, j % ps, c] = math.nan
    run(p)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("hq,n", [(130, 1), (130, 3), (200, 2), (256, 1)])
def test_more_heads_per_kv_head_than_a_tile_has_rows(hq, n, q8):
    run(Problem("bf16", hq, 1, 16, [150, 33], [n, 1], 0, q8=q8))


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("dtype,pages,q8", [("bf16", 140_000, False), ("f32", 70_000, False),
                                            ("f16", 270_000, True)])
def test_offsets_past_32_bits(dtype, pages, n, q8):
    """Pages at the end of caches of more than 4 GiB each."""
    p = Problem(dtype, 16, 8, 16, [150, 40], [n, 1], q8=q8).upload()
    small = p.pages
    p.shape.num_phys_pages = pages
    p.d_table.copy_(torch.where(p.table >= 0, p.table + (pages - small), -1))
    big = {}

    def grow(name, x):
        big[name] = torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
        big[name][pages - small:] = x
        return big[name]

    if q8:
        c, s = p.d_code, p.d_scale
        p.cache = kv.make_q8_cache(grow("k", c["k"]), grow("v", c["v"]), grow("ks", s["k"]),
                                   grow("vs", s["v"]))
        p.ws = torch.empty(kv.kv_q8_chunk_workspace_bytes(p.shape, p.chunk), dtype=torch.uint8,
                           device="cuda")
    else:
        p.d_k, p.d_v = grow("k", p.d_k), grow("v", p.d_v)
    p.attend()
    torch.cuda.synchronize()
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows_at_all(dtype, q8):
    """A batch none of whose sequences brings a token: nothing is written."""
    p = Problem(dtype, 4, 2, 16, [30, 0], [0, 0], q8=q8).upload()
    p.attend()
    torch.cuda.synchronize()
    assert (p.d_out == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_pages_shared_by_sequences(dtype):
    """A common prefix held once; the rest of each sequence in pages of its own."""
    for q8 in (False, True):
        for loc in ("hbm", "host"):
            p = Problem(dtype, 4, 2, 16, [100, 90, 80], [4, 1, 30], q8=q8, loc=loc)
            p.table[1, :3] = p.table[0, :3]
            p.table[2, :3] = p.table[0, :3]
            run(p)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("n", [1, 20, 300])
def test_a_workspace_too_small_is_refused(n, q8):
    p = Problem("bf16", 8, 2, 16, [400], [n], q8=q8).upload()
    for ws in (p.ws[:-256], p.ws[:16]):
        assert p.attend(ws=ws, check=False) == kv.KV_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert (p.d_out == 7).all()


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
def test_cache_memory_of_the_wrong_kind_is_refused(q8):
    p = Problem("bf16", 8, 2, 16, [40], [2], q8=q8, loc="host").upload()
    p.shape.kv_loc = kv.KV_LOC_HBM
    assert p.attend(check=False) == kv.KV_ERR_LOCATION
    p = Problem("bf16", 8, 2, 16, [40], [2], q8=q8).upload()
    p.shape.kv_loc = kv.KV_LOC_HOST_PINNED
    assert p.attend(check=False) in (kv.KV_ERR_LOCATION, kv.KV_ERR_WORKSPACE)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_chunk_in_pieces_equals_the_chunk(dtype):
    """60 tokens at once, and as 25 + 1 + 34 on the cache as it stood then."""
    for q8 in (False, True):
        p = run(Problem(dtype, 4, 2, 16, [200], [60], q8=q8))
        whole, (want, tol) = p.d_out.clone(), p.expected()
        q = p.d_q.clone()
        at = 0
        for n in (25, 1, 34):
            p.d_q[:n] = q[at:at + n]
            p.d_start.copy_(torch.tensor([0, n], dtype=torch.int32))
            p.d_lens.fill_(140 + at + n)
            p.d_out.fill_(7)
            p.attend()
            check(p.d_out[:n], want[at:at + n], tol[at:at + n])
            assert (p.d_out[n:] == 7).all()
            at += n
        check(whole, want, tol)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_bit_for_bit_and_in_a_graph(dtype, q8):
    p = run(Problem(dtype, 8, 2, 16, [700, 333, 12], [40, 1, 12], q8=q8))
    first = p.d_out.clone()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            p.attend(stream=st)
        for _ in range(3):
            p.d_out.fill_(7)
            graph.replay()
        st.synchronize()
    assert torch.equal(first, p.d_out)
    # new lengths and queries under the same graph
    p.lens, p.news = [650, 200, 9], [40, 1, 12]
    p.d_lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
    p.q = torch.flip(p.q, [2])
    p.d_q.copy_(p.q)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        graph.replay()
    st.synchronize()
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_two_streams_at_once(dtype):
    ps = [Problem(dtype, 8, 2, 16, [2000 + i, 100], [60, 1], seed=i, q8=i == 1).upload()
          for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, st in zip(ps, streams):
            p.attend(stream=st)
    torch.cuda.synchronize()
    for p in ps:
        check(p.d_out, *p.expected())


@pytest.mark.parametrize("dtype,ps", [("f32", 16), ("f16", 16), ("bf16", 64)])
def test_one_token_chunks_agree_with_dense_decode(dtype, ps):
    p = run(Problem(dtype, 8, 2, ps, [300, 77, 1], [1, 1, 1]))
    out = torch.empty(3, 8, D, dtype=torch.float32, device="cuda")
    ws = torch.empty(max(16, kv.kv_attn_workspace_bytes(p.shape, 0)), dtype=torch.uint8,
                     device="cuda")
    for x in (p.d_k, p.d_v):  # the decode call reads whole pages
        x.nan_to_num_(nan=0.0)
    kv.kv_dense_decode_attn(p.shape, p.d_q, p.d_k, p.d_v, p.d_table, p.d_lens, p.scale, out, ws,
                            ws.numel(), torch.cuda.current_stream())
    want, tol = p.expected()
    check(p.d_out[:3], out.double().cpu(), 2 * tol[:3] + 2e-5)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_path_together(dtype):
    """A prompt and then single tokens through the 8-bit cache: append, attend in
    place; the same cache read back into the type's own form gives the same
    attention, and the calls that were there before take it."""
    hq, hkv, ps, prompt, steps = 8, 2, 16, [70, 33], 3
    lens = [n + steps for n in prompt]
    p = Problem(dtype, hq, hkv, ps, lens, prompt, q8=True, seed=4).upload()
    t = TORCH[dtype]
    g = torch.Generator().manual_seed(11)
    code = {n: torch.zeros_like(p.d_code[n]) for n in "kv"}
    scale = {n: torch.zeros_like(p.d_scale[n]) for n in "kv"}
    cache = kv.make_q8_cache(code["k"], code["v"], scale["k"], scale["v"])
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream()
    for step in range(1 + steps):
        news = prompt if step == 0 else [1, 1]
        start = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device="cuda")
        chunk = kv.make_chunk(start, sum(news), max(news))
        kn, vn = (torch.randn(sum(news), hkv, D, generator=g).to(t).cuda() for _ in "kv")
        q = torch.randn(sum(news), hq, D, generator=g).to(t)
        kv.kv_q8_append(p.shape, chunk, kn, vn, cache, p.d_table, ctx, ctx, st)
        got = torch.empty(sum(news), hq, D, dtype=t, device="cuda")
        ws = torch.empty(max(16, kv.kv_q8_chunk_workspace_bytes(p.shape, chunk)), dtype=torch.uint8,
                         device="cuda")
        kv.kv_q8_chunk_attn(p.shape, chunk, q.cuda(), cache, p.d_table, ctx, p.scale, got, ws,
                            ws.numel(), st)
        # read back
        back = [torch.zeros(p.pages, hkv, ps, D, dtype=t, device="cuda") for _ in "kv"]
        kv.kv_q8_read(p.shape, cache, p.d_table, ctx, p.d_table, p.pages, back[0], back[1], st)
        again = torch.empty_like(got)
        ws = torch.empty(max(16, kv.kv_chunk_workspace_bytes(p.shape, chunk)), dtype=torch.uint8,
                         device="cuda")
        kv.kv_chunk_attn(p.shape, chunk, q.cuda(), back[0], back[1], p.d_table, ctx, p.scale, again,
                         ws, ws.numel(), st)
        # the definition
        p.lens, p.news, p.start, p.total = ctx.tolist(), news, start.tolist(), sum(news)
        p.q = q
        p.code = {n: code[n].cpu() for n in "kv"}
        p.scale8 = {n: scale[n].cpu() for n in "kv"}
        want, tol = p.expected()
        check(got, want, tol)
        check(again, want, tol)
    # an index over the pages read back, and decode attention on it
    minmax = torch.zeros(p.pages, hkv, 2, D, dtype=t, device="cuda")
    kv.kv_page_minmax_build(p.shape, back[0], p.d_table, ctx, minmax, st)
    out = torch.empty(2, hq, D, dtype=torch.float32, device="cuda")
    ws = torch.empty(max(16, kv.kv_attn_workspace_bytes(p.shape, 0)), dtype=torch.uint8,
                     device="cuda")
    kv.kv_dense_decode_attn(p.shape, q.cuda(), back[0], back[1], p.d_table, ctx, p.scale, out, ws,
                            ws.numel(), st)
    check(out, want, tol + 2e-5)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("news", [[1, 1], [13, 1], [90, 200]])
def test_a_wait_that_runs_out_is_reported(news, q8):
    """A K/V tile that is never filled (the testing hook): the bounded waits give
    up, the status says so, and the next call is exact."""
    p = Problem("bf16", 8, 2, 16, [700, 300], news, q8=q8).upload()
    kv.kv_debug_config(0, 2_000_000)
    try:
        p.attend()
        assert kv.kv_device_status() == kv.KV_ERR_DEVICE_TIMEOUT
    finally:
        kv.kv_debug_config(-1, 2_000_000_000)
    p.d_out.fill_(7)
    p.attend()
    torch.cuda.synchronize()
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_pipeline_classes(dtype, loc):
    """DecodeLayer.chunk_attn and Q8Cache run the calls and keep the lengths."""
    from offloaded_kv_cache_gb300 import workloads as W
    from offloaded_kv_cache_gb300.pipeline import DecodeLayer, Q8Cache
    spec = W.tiny_spec(dtype=dtype, batch=2, hq=8, hkv=2, context=90, ps=16, topk=2, index=5)
    layer = DecodeLayer(W.generate(spec, context_lens=[90, 41]), kv_loc=loc)
    t = TORCH[dtype]
    q8 = Q8Cache(layer.shape, layer.block_table, torch.zeros(2, dtype=torch.int32, device="cuda"),
                 kv_loc=loc)
    g = torch.Generator().manual_seed(1)
    for n in ([50, 12], [1, 1], [0, 3]):
        start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        k, v = (torch.randn(sum(n), 2, D, generator=g).to(t).cuda() for _ in "kv")
        q = torch.randn(sum(n), 8, D, generator=g).to(t).cuda()
        q8.append(k, v, start, max(n))
        got = q8.attend(q, start, max(n), layer.scale)
    assert q8.context_lens.tolist() == [51, 16]
    back = [torch.zeros(spec.num_phys_pages, 2, 16, D, dtype=t, device="cuda") for _ in "kv"]
    q8.read_back(*back)
    layer.context_lens.copy_(q8.context_lens)
    torch.cuda.synchronize()
    layer.k_cache.copy_(back[0])
    layer.v_cache.copy_(back[1])
    again = layer.chunk_attn(q, start, max(n))
    torch.cuda.synchronize()
    # both compute the same sums, each within 2^-8 (2^-11, 2^-24) of weights and result
    tol = {"f32": 1e-5, "f16": 2.0 ** -9, "bf16": 2.0 ** -6}[dtype]
    assert float((got.float() - again.float()).abs().max()) <= tol * (1 + float(back[1].abs().max()))


def _small_layer(dtype="bf16"):
    from offloaded_kv_cache_gb300 import workloads as W
    from offloaded_kv_cache_gb300.pipeline import DecodeLayer
    spec = W.tiny_spec(dtype=dtype, batch=2, hq=8, hkv=2, context=600, ps=16, topk=5, index=7)
    layer = DecodeLayer(W.generate(spec, context_lens=[600, 333]))
    g = torch.Generator().manual_seed(3)

    def rows(*n):
        start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        return torch.randn(sum(n), 8, D, generator=g).to(TORCH[dtype]).cuda(), start, max(n)
    return layer, rows


def test_pipeline_chunk_leaves_the_selected_pages():
    """The page lists of select_fused stay in the layer's workspace over a chunk."""
    layer, rows = _small_layer()
    layer.build_index()
    layer.sparse_step_fused()
    want = layer.out.clone()
    layer.select_fused()
    layer.chunk_attn(*rows(200, 300))
    layer.sparse_attn_selected()
    assert torch.equal(layer.out, want)


def test_pipeline_chunk_in_graphs():
    """Two captured calls replay together, and after larger eager ones, as they ran alone."""
    layer, rows = _small_layer()
    calls = [rows(1, 1), rows(40, 60)]
    want = [layer.chunk_attn(*c) for c in calls]
    graphs, got, streams = [], [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(layer.chunk_attn(*c))
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    big = rows(500, 333)
    alone = layer.chunk_attn(*big)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        assert torch.equal(layer.chunk_attn(*big), alone)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_pipeline_chunk_refusals():
    layer, rows = _small_layer()
    q, start, most = rows(3, 4)
    for bad in (q.half(), q[:, :4], q.transpose(0, 1).contiguous().transpose(0, 1),
                torch.zeros(7, 8, D, dtype=q.dtype)):
        with pytest.raises(ValueError, match="q: a contiguous"):
            layer.chunk_attn(bad, start, most)
    with pytest.raises(ValueError, match="q_start"):
        layer.chunk_attn(q, start[:2], most)
    with pytest.raises(ValueError, match="out"):
        layer.chunk_attn(q, start, most, out=torch.empty_like(q, dtype=torch.float32))
