"""The 4-bit cache: kv_q4_append and kv_q4_read bit for bit what the format's definition
gives in 64 bits, kv_q4_chunk_attn against its definition on those values (tests/more_util.py,
chunk_util.py, which derives the tolerance), at the sizes and masks where each can go wrong."""
import os
import random

import numpy as np
import pytest
import torch

from chunk_util import D, TORCH, Problem, check
from more_util import STEPS, Problem4, quantise4, restore4, turned, turned_tolerance
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu

CASES = int(os.environ.get("KV_Q4_FUZZ_CASES", "60"))


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    kv.kv_debug_config(-1, 2_000_000_000)
    assert kv.kv_device_status() == kv.KV_OK


# --- append ------------------------------------------------------------------------------
class Append:
    """A batch whose chunks go into an empty 4-bit cache."""

    def __init__(self, dtype, hkv, ps, before, news, loc="hbm", seed=0, rows=None, max_new=None):
        lens = [a + n for a, n in zip(before, news)]
        self.p = p = Problem(dtype, hkv, hkv, ps, lens, news, seed=seed, loc=loc)
        g = torch.Generator().manual_seed(seed + 1)
        mag = torch.exp2(torch.randint(-9, 9, (p.total, hkv, 1), generator=g).float())
        self.new = {}
        for name in ("k", "v"):
            x = torch.randn(p.total, hkv, D, generator=g) * mag
            x[..., 5::37] *= 12
            if rows is not None:
                x[:rows.shape[0]] = rows[:, None]
            self.new[name] = x.to(TORCH[dtype])
        self.before = torch.tensor(before, dtype=torch.int32, device="cuda")
        p.upload(max_new=max_new)
        shape = (p.pages, hkv, ps)
        fill = lambda v, *row: p.put(torch.full((*shape, *row), v, dtype=torch.uint8), True)  # noqa: E731
        self.got = {n: (fill(0xAB, D // 2), fill(0xCD, D // 16), fill(0xEF)) for n in "kv"}
        (kc, ks, kp), (vc, vs, vp) = self.got["k"], self.got["v"]
        self.cache = kv.make_q4_cache(kc, vc, ks, vs, kp, vp)
        self.d_new = {n: x.cuda() for n, x in self.new.items()}

    def run(self, out=None, stream=None):
        p = self.p
        kv.kv_q4_append(p.shape, p.chunk, self.d_new["k"], self.d_new["v"], self.cache, p.d_table,
                        self.before, out, torch.cuda.current_stream() if stream is None else stream)
        torch.cuda.synchronize()

    def check(self):
        p = self.p
        for n in "kv":
            want = [np.full(x.shape, f, dtype=np.uint8) for x, f in zip(self.got[n], (0xAB, 0xCD, 0xEF))]
            new = quantise4(self.new[n].double().numpy(), p.dtype)
            for b, k in enumerate(p.news):
                for i in range(k):
                    pos = p.lens[b] - k + i
                    ph = int(p.table[b, pos // p.ps])
                    if 0 <= ph < p.pages:
                        for w, x in zip(want, new):
                            w[ph, :, pos % p.ps] = x[p.start[b] + i]
            for x, w in zip(reversed(self.got[n]), reversed(want)):
                assert np.array_equal(x.cpu().numpy(), w)


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype,hkv,ps,before,news", [
    ("bf16", 8, 16, [0, 15, 16, 100, 33], [1, 1, 1, 0, 1]),
    ("f16", 4, 32, [0, 31, 7], [70, 1, 33]),
    ("f32", 1, 64, [63, 0], [2, 129]),
    ("bf16", 3, 128, [5], [300]),
    ("f16", 32, 16, [17, 0, 1], [5, 16, 40]),
    ("f32", 8, 16, [3, 40], [200, 31]),
])
def test_append(dtype, hkv, ps, before, news, loc):
    a = Append(dtype, hkv, ps, before, news, loc)
    out = torch.full((len(news),), -9, dtype=torch.int32, device="cuda")
    a.run(out)
    a.check()
    assert out.tolist() == a.p.lens and a.before.tolist() == before


def difficult(t):
    """Zeros of both signs, one large element, maxima at and beside every border of the power
    and of the scale, ties and their neighbours, subnormals, the saturated range, infinities, NaN."""
    big = torch.finfo(t).max
    rows = [torch.zeros(D, dtype=torch.float64), -torch.zeros(D, dtype=torch.float64)]
    up = lambda x: torch.nextafter(torch.tensor(x).to(t), torch.tensor(float("inf")).to(t)).double().item()  # noqa: E731
    for top in (3136.0, up(3136.0), 1568.0, up(1568.0), 12.25, up(12.25), 1.75, 50176.0, 50200.0, 60000.0,
                big, 2.0 ** -15, 2.0 ** -24, 2.0 ** -110, 2.0 ** -126, 1e-30, 2.0 ** -133, 2.0 ** -149):
        x = torch.linspace(-1, 1, D, dtype=torch.float64) * top
        rows.append(x)
        y = torch.zeros(D, dtype=torch.float64)
        y[77] = -top
        rows.append(y)
    # groups whose maxima are 7 s and its neighbours, for every s, under a maximum of 3136
    for k in range(0, 126, 7):
        x = torch.zeros(D, dtype=torch.float64)
        for g in range(7):
            s = float(7 * STEPS[k + g])
            x[16 * g] = (s, up(s), -s)[g % 3]
            x[16 * g + 3] = s / 2
        x[127] = 3136.0
        rows.append(x)
    # every tie c + 1/2 under many scales, and the type's values beside it
    for s in (1.0, 1.125, 0.6875, 13.0, 448.0, 0.001953125, 0.009765625):
        tie = torch.arange(-6.5, 7.0) * s
        x = torch.zeros(D, dtype=torch.float64)
        x[:14], x[14], x[15] = tie, 7 * s, -7 * s
        d = tie.to(t)
        above = torch.nextafter(d, torch.full_like(d, float("inf"))).double()
        below = torch.nextafter(d, torch.full_like(d, -float("inf"))).double()
        x[16:30], x[30] = above, 7 * s
        x[32:46], x[46] = below, 7 * s
        x[127] = 3136.0
        rows.append(x)
    for bad in (float("inf"), -float("inf"), float("nan")):
        x = torch.randn(D, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
        x[5] = bad
        rows.append(x)
    return torch.stack(rows)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_append_difficult_vectors(dtype):
    rows = difficult(TORCH[dtype]).float()
    a = Append(dtype, 2, 16, [3], [len(rows)], rows=rows)
    a.run()
    a.check()


def test_append_beside_ties():
    """fp32: elements at (c + 1/2) s (1 +- 2^-k) for every c, many s and k from 6 to 23."""
    groups = []
    for i, s in enumerate(STEPS[1:127]):
        for k in range(6 + i % 3, 24, 3):
            tie = torch.arange(-6.5, 7.0).double() * float(s)
            side = (-1.0) ** torch.arange(14)
            groups.append(torch.cat([tie * (1 + side * 2.0 ** -k), torch.tensor([7.0, -7.0]).double() * float(s)]))
    groups = groups[:len(groups) // 7 * 7]
    x = torch.stack(groups).reshape(-1, 7 * 16)
    last = torch.zeros(len(x), 16, dtype=torch.float64)
    last[:, 5] = 3136.0  # the power is 0
    rows = torch.cat([x, last], 1).float()
    a = Append("f32", 2, 16, [5], [len(rows)], rows=rows)
    a.run()
    a.check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_every_value(dtype):
    """Every finite value of the type as an element, beside group maxima of many sizes."""
    t = TORCH[dtype]
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(t)
    v = v[torch.isfinite(v)]
    v = v[torch.argsort(v.float().abs())]
    pad = -len(v) % 15
    v = torch.cat([v, v[-pad:]]) if pad else v
    groups = v.reshape(-1, 15)
    g = torch.Generator().manual_seed(8)
    lead = groups.float().abs().amax(-1) * torch.exp2(3 * torch.rand(len(groups), generator=g))
    lead = lead.clamp(max=float(torch.finfo(t).max)).to(t)
    groups = torch.cat([groups, lead[:, None]], 1)
    more = -len(groups) % 8
    rows = torch.cat([groups, groups[:more]]).reshape(-1, D).float()
    a = Append(dtype, 1, 16, [0], [len(rows)], rows=rows)
    a.run()
    a.check()


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 0, 7], [1000, 3, 64], [0, 0, 0]])
def test_append_lengths_in_place(news):
    before = [5, 9, 0]
    a = Append("bf16", 4, 16, before, news)
    a.run(a.before)
    a.check()
    assert a.before.tolist() == [x + n for x, n in zip(before, news)]


def test_append_skips_what_is_out_of_range():
    a = Append("f16", 2, 16, [0, 3, 2, 4], [40, 20, 6, 5])
    p = a.p
    p.table[0, 1] = p.pages
    p.d_table.copy_(p.table)
    out = torch.full((4,), -9, dtype=torch.int32, device="cuda")
    a.before[2] = p.max_pages * 16 - 5  # six tokens do not fit
    p.news[2] = 0
    a.run(out)
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    a.check()
    assert out.tolist() == [0, 23, p.max_pages * 16 - 5, 9]
    for start in ([0, 41, 45, 50, 55], [0, 40, 30, 50, 71], [-1, 40, 60, 66, 71]):
        a = Append("f16", 2, 16, [0, 3, 2, 4], [40, 20, 6, 5])
        a.p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        a.run(out)
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS


# --- read back ---------------------------------------------------------------------------
@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype,hkv,ps,lens", [
    ("bf16", 8, 16, [1, 16, 17, 0, 300]),
    ("f16", 4, 32, [95, 700]),
    ("f32", 1, 64, [129, 64, 1]),
    ("bf16", 3, 128, [1000]),
])
def test_read(dtype, hkv, ps, lens, loc):
    p = Problem4(dtype, hkv, hkv, ps, lens, [0] * len(lens), loc=loc).upload()
    out_pages = p.pages + 3
    # pages of its own order; one page of the longest row stays out
    table = torch.full_like(p.table, -1)
    order = torch.randperm(out_pages, generator=torch.Generator().manual_seed(9))
    at = 0
    for b, n in enumerate(lens):
        for i in range(-(-n // ps)):
            if not (i == 1 and n == max(lens)):
                table[b, i] = order[at]
            at += 1
    want = {}
    for n in "kv":
        x = np.full((out_pages, hkv, ps, D), 7.0)
        value = restore4(*(t.numpy() for t in p.four[n]))
        for b, length in enumerate(lens):
            for j in range(length):
                to = int(table[b, j // ps])
                if to >= 0:
                    x[to, :, j % ps] = value[int(p.table[b, j // ps]), :, j % ps]
        want[n] = torch.from_numpy(x)
    got = {n: torch.full((out_pages, hkv, ps, D), 7.0, dtype=TORCH[dtype], device="cuda")
           for n in "kv"}
    kv.kv_q4_read(p.shape, p.cache, p.d_table, p.d_lens, table.cuda(), out_pages, got["k"],
                  got["v"], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for n in "kv":
        assert torch.equal(got[n].double().cpu(), want[n])


@pytest.mark.parametrize("dtype,powers", [("f16", range(112, 132)), ("bf16", range(17, 132)),
                                          ("f32", range(17, 132))])
def test_read_every_code_scale_and_power(dtype, powers):
    """All integers a writer may leave (and -8) under every scale and power, and NaN."""
    powers = list(powers) + [255]
    n = len(powers) * 16
    p = Problem4(dtype, 1, 1, 128, [n], [0])
    code = torch.arange(256, dtype=torch.uint8)[torch.arange(D // 2) % 16 * 17]
    for j in range(n):
        ph, slot = int(p.table[0, j // 128]), j % 128
        for name in "kv":
            c, s, w = p.four[name]
            c[ph, 0, slot] = code
            s[ph, 0, slot] = torch.clamp(torch.arange(8) + 8 * (j % 16), max=126).to(torch.uint8)
            w[ph, 0, slot] = powers[j // 16]
    p.upload()
    out = [torch.zeros(p.pages, 1, 128, D, dtype=TORCH[dtype], device="cuda") for _ in "kv"]
    kv.kv_q4_read(p.shape, p.cache, p.d_table, p.d_lens, p.d_table, p.pages, out[0], out[1],
                  torch.cuda.current_stream())
    for name, x in zip("kv", out):
        want = torch.from_numpy(restore4(*(t.numpy() for t in p.four[name])))
        want = want.to(TORCH[dtype]).double()  # (-8 * 448 * 2^4 is more than f16 holds)
        for j in range(n):
            ph, slot = int(p.table[0, j // 128]), j % 128
            assert torch.equal(x[ph, 0, slot].double().cpu().nan_to_num(nan=1e9),
                               want[ph, 0, slot].nan_to_num(nan=1e9))


def test_read_out_of_range():
    p = Problem4("bf16", 2, 2, 16, [50, 20], [0, 0])
    p.table[0, 2] = -5
    p.upload()
    out = [torch.full((p.pages, 2, 16, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    to = p.table.clone()
    to[0, 2] = p.pages - 1
    to[1, 1] = p.pages
    kv.kv_q4_read(p.shape, p.cache, p.d_table, p.d_lens, to.cuda(), p.pages, out[0], out[1],
                  torch.cuda.current_stream())
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    assert not torch.isnan(out[0]).any()
    p.d_lens[0] = p.max_pages * 16 + 1
    kv.kv_q4_read(p.shape, p.cache, p.d_table, p.d_lens, p.d_table, p.pages, out[0], out[1],
                  torch.cuda.current_stream())
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS


# --- attention ---------------------------------------------------------------------------
def run(p):
    p.upload()
    p.attend()
    torch.cuda.synchronize()
    check(p.d_out, *p.expected())
    return p


RAGGED = [
    ([1], [1]),
    ([17], [17]),
    ([300, 1, 64, 129], [1, 1, 1, 1]),
    ([200, 5, 131, 64, 0], [7, 0, 131, 3, 0]),
    ([513, 128], [257, 128]),
    ([1025, 40], [3, 40]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,news", RAGGED, ids=[str(i) for i in range(len(RAGGED))])
def test_ragged(dtype, lens, news):
    run(Problem4(dtype, 4, 2, 16, lens, news, seed=len(lens)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (8, 1), (14, 2), (3, 3), (96, 1)])
@pytest.mark.parametrize("n", [1, 9, 50])
def test_head_groups(dtype, hq, hkv, n):
    run(Problem4(dtype, hq, hkv, 32, [150, 61], [n, 1], seed=hq))


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,window", [("f16", 0), ("bf16", 100), ("f32", 33)])
def test_page_sizes(dtype, ps, window):
    run(Problem4(dtype, 8, 2, ps, [ps * 3 + 1, ps - 1, 401], [40, ps - 1, 5], window, seed=ps))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300])
def test_windows(dtype, window):
    run(Problem4(dtype, 2, 1, 16, [420, 90], [140, 90], window, seed=window))


FEW = [(8, 2, 2), (8, 1, 1), (7, 1, 2), (16, 1, 1), (4, 1, 4), (6, 2, 11), (8, 1, 8), (8, 1, 16)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,n", FEW)
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("ps", [16, 128])
def test_few_rows(dtype, hq, hkv, n, window, ps):
    run(Problem4(dtype, hq, hkv, ps, [n + 120, n, 390, 5], [n, n, 1, 0], window, seed=n))


# A table for long contexts takes the form of twice as many warps.
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,n", FEW)
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("ps", [16, 128])
def test_few_rows_of_a_wide_table(dtype, hq, hkv, n, window, ps):
    run(Problem4(dtype, hq, hkv, ps, [n + 120, n, 390, 5, 1100], [n, n, 1, 0, 1], window, seed=n,
                 extra_pages=6000 // ps))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 9])
def test_odd_values_under_a_wide_table(dtype, n):
    """Scores that rise from tile to tile, vectors of all sizes, one of NaN, and bad pages."""
    p = Problem4(dtype, 2, 1, 16, [700, 1300, 600], [n, n, 1], scale=1.0, extra_pages=400)
    p.q = torch.zeros_like(p.q)
    p.q[:, :, 0] = 1
    for j in range(700):
        p.k[p.table[0, j // 16], :, j % 16, 0] = -100 + j / 3.5
    x = p.k.double().nan_to_num(nan=0.0).numpy()
    p.four["k"] = [torch.from_numpy(t) for t in quantise4(x, dtype)]
    c, s, w = p.four["v"]
    g = torch.Generator().manual_seed(6)
    p.four["v"][2] = torch.where(w == 255, w, torch.randint(112, 124, w.shape, generator=g).to(torch.uint8))
    p.set_nan("v", p.table[1, 1290 // 16], slice(None), 1290 % 16)
    p.table[1, 7] = p.pages
    p.table[2, 30] = -1
    p.upload()
    p.attend()
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [2, 20, 150])
def test_vectors_of_very_different_size(dtype, n):
    """Keys and values whose powers differ by up to 2^20, groups whose scales do by 2^17,
    queries whose rows do; scores reach tens either way."""
    p = Problem4(dtype, 4, 2, 16, [300, 64], [n, 1], seed=n)
    g = torch.Generator().manual_seed(5)
    for name in "kv":
        c, s, w = p.four[name]
        lo = 127 - (15 if dtype == "f16" else 28)
        new = torch.randint(lo, 118, w.shape, generator=g).to(torch.uint8)
        p.four[name][2] = torch.where(w == 255, w, new)
        some = torch.randint(0, 127, s.shape, generator=g).to(torch.uint8)
        p.four[name][1] = torch.where((w == 255)[..., None], s, some)
    p.q = (p.q.float() * torch.exp2(torch.randint(-12, 3, (p.total, 4, 1), generator=g).float())
           ).to(TORCH[dtype])
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing(dtype):
    run(Problem4(dtype, 4, 2, 16, [3, 0, 140], [10, 5, 200]))


@pytest.mark.parametrize("dtype,scale,q_size", [
    ("f32", -0.2, 1.0), ("bf16", -0.2, 1.0), ("f16", 0.0, 1.0), ("bf16", 1.0, 16.0),
    ("f16", 0.5, 8.0), ("f32", 1.0, 8.0)])
@pytest.mark.parametrize("n", [3, 20, 150])
def test_scales(dtype, scale, q_size, n):
    run(Problem4(dtype, 4, 2, 16, [260, 30], [n, 1], scale=scale, q_size=q_size))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("n", [4, 30, 150])
def test_running_maximum_moves(dtype, order, n):
    """Scores that rise (fall) by 20 powers of two from tile to tile."""
    p = Problem4(dtype, 2, 1, 16, [700], [n], scale=1.0)
    ramp = order * torch.linspace(-100, 100, 700)
    p.q = torch.zeros_like(p.q)
    p.q[:, :, 0] = 1
    for j in range(700):
        p.k[p.table[0, j // 16], :, j % 16, 0] = ramp[j]
    x = p.k.double().nan_to_num(nan=0.0).numpy()
    p.four["k"] = [torch.from_numpy(t) for t in quantise4(x, dtype)]
    run(p)


@pytest.mark.parametrize("n", [100, 51, 20, 7])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ["k", "v"])
def test_vectors_that_are_nan(name, dtype, n):
    """Rows that see one are NaN, the others untouched."""
    p = Problem4(dtype, 2, 1, 16, [160, 33], [n, 1])
    p.set_nan(name, p.table[0, 155 // 16], slice(None), 155 % 16)
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("news", [[30, 1, 2], [1, 1, 1], [150, 40, 200]])
def test_bad_pages_are_skipped(dtype, news):
    p = Problem4(dtype, 4, 2, 16, [150, 40, 300], news)
    p.table[0, 3] = p.pages
    p.table[2, 0] = -1
    p.table[2, 18] = 1 << 30
    p.upload()
    p.attend()
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 30])
def test_pages_behind_every_window_may_be_gone(dtype, n):
    p = Problem4(dtype, 4, 2, 16, [500], [n], window=60).upload()
    p.attend()
    want = p.d_out.clone()
    p.d_table[0, :(500 - n - 60 + 1) // 16] = -1
    p.d_out.fill_(7)
    p.attend()
    torch.cuda.synchronize()
    assert torch.equal(want, p.d_out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_sequences_are_skipped(dtype):
    p = Problem4(dtype, 4, 2, 16, [150, 40, 300], [30, 1, 20])
    p.upload(max_new=25)
    p.d_lens[1] = p.max_pages * 16 + 1
    p.attend()
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    want, tol = p.expected()
    want[:31], tol[:31] = 7, 0
    check(p.d_out, want, tol)
    p.d_lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
    for start in ([0, 30, 20, 40], [0, 30, 31, 1 << 20], [-5, 0, 1, 21]):
        p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        p.attend()
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,news", [([150, 40], [30, 1]), ([900, 20], [1, 1]), ([700, 300], [250, 300])])
def test_host_resident_cache(dtype, lens, news):
    run(Problem4(dtype, 8, 2, 16, lens, news, loc="host"))


@pytest.mark.parametrize("dtype,hq,hkv,lens,news", [
    ("bf16", 32, 8, [5000, 3001], [1, 1]),
    ("f16", 8, 1, [9000], [70]),
    ("bf16", 4, 4, [257] * 40, [33] * 40),
    ("f32", 2, 1, [4097], [65]),
    ("f16", 16, 2, [2500], [200])])
def test_longer_and_many(dtype, hq, hkv, lens, news):
    """Units that many CTAs share, and many units per CTA."""
    run(Problem4(dtype, hq, hkv, 64, lens, news))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,most,n", [(33, 300, 1), (33, 300, 90), (600, 60, 3), (1100, 17, 1)])
def test_many_sequences(dtype, batch, most, n):
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, most, (batch,), generator=g).tolist()
    news = [min(x, int(torch.randint(0, n + 1, (1,), generator=g))) for x in lens]
    run(Problem4(dtype, 4, 2, 16, lens, news, seed=n))


@pytest.mark.parametrize("hq,n", [(130, 1), (130, 3), (256, 1)])
def test_more_heads_per_kv_head_than_a_tile_has_rows(hq, n):
    run(Problem4("bf16", hq, 1, 16, [150, 33], [n, 1]))


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_offsets_past_32_bits(dtype, n):
    """Pages at the end of caches whose codes are more than 4 GiB each."""
    pages = 540_000
    p = Problem4(dtype, 16, 8, 16, [150, 40], [n, 1]).upload()
    small = p.pages
    p.shape.num_phys_pages = pages
    p.d_table.copy_(torch.where(p.table >= 0, p.table + (pages - small), -1))
    big = {n: [] for n in "kv"}
    for n in "kv":
        for x in p.d_four[n]:
            y = torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
            y[pages - small:] = x
            big[n].append(y)
    p.use(big)
    p.attend()
    torch.cuda.synchronize()
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("heads", [8, 32])
def test_as_many_tokens_as_an_int_counts(heads):
    """One page, 2^27 - 1 times in the table: the attention over its 16 tokens.

    8 rows: a warp takes 2^31 / 32 / 2432 = 27594 steps of two products (cut by 2^-23 of the sum
    at most) and eight weights a lane (2^-24): 2 * 27594 * 2^-23 + 8 * 27594 * 2^-24 = 2%.  32
    rows: a CTA takes 2^31 / 128 / 152 = 110377 tiles of eight products, cut by half of that on
    average and of a sum half as large on average: 8 * 110377 * 2^-25 = 2.6%, and as much at most
    for the weights.  A twentieth of the largest value."""
    p = Problem4("bf16", heads, 1, 16, [16], [1], seed=5).upload()
    want, tol = p.expected()
    pages = 2 ** 27 - 1
    p.shape.max_pages_per_seq = pages
    p.d_table = torch.full((1, pages), int(p.table[0, 0]), dtype=torch.int32, device="cuda")
    p.d_lens = torch.tensor([16 * pages], dtype=torch.int32, device="cuda")
    p.use(p.d_four)
    p.attend()
    torch.cuda.synchronize()
    top = float(p.tokens("v", 0, 0)[0].abs().max())
    off = (p.d_out.cpu().double() - want).abs()
    assert bool((off <= tol + top / 20).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows_at_all(dtype):
    p = Problem4(dtype, 4, 2, 16, [30, 0], [0, 0]).upload()
    p.attend()
    torch.cuda.synchronize()
    assert (p.d_out == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("loc", ["hbm", "host"])
def test_pages_shared_by_sequences(dtype, loc):
    p = Problem4(dtype, 4, 2, 16, [100, 90, 80], [4, 1, 30], loc=loc)
    p.table[1, :3] = p.table[0, :3]
    p.table[2, :3] = p.table[0, :3]
    run(p)


@pytest.mark.parametrize("n", [1, 20, 300])
def test_a_workspace_too_small_is_refused(n):
    p = Problem4("bf16", 8, 2, 16, [400], [n]).upload()
    for ws in (p.ws[:-256], p.ws[:16]):
        assert p.attend(ws=ws, check=False) == kv.KV_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert (p.d_out == 7).all()


def test_cache_memory_of_the_wrong_kind_is_refused():
    p = Problem4("bf16", 8, 2, 16, [40], [2], loc="host").upload()
    p.shape.kv_loc = kv.KV_LOC_HBM
    assert p.attend(check=False) == kv.KV_ERR_LOCATION
    p = Problem4("bf16", 8, 2, 16, [40], [2]).upload()
    p.shape.kv_loc = kv.KV_LOC_HOST_PINNED
    assert p.attend(check=False) in (kv.KV_ERR_LOCATION, kv.KV_ERR_WORKSPACE)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_chunk_in_pieces_equals_the_chunk(dtype):
    p = run(Problem4(dtype, 4, 2, 16, [200], [60]))
    want, tol = p.expected()
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", [([700, 333, 12], [40, 1, 12]), ([900, 33], [1, 1])])
def test_repeats_bit_for_bit_and_in_a_graph(dtype, lens, news):
    p = run(Problem4(dtype, 8, 2, 16, lens, news))
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
    p.lens = [x - 3 for x in lens]
    p.d_lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
    p.q = torch.flip(p.q, [2])
    p.d_q.copy_(p.q)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        graph.replay()
    st.synchronize()
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n", [1, 60])
def test_two_streams_at_once(dtype, n):
    ps = [Problem4(dtype, 8, 2, 16, [2000 + i, 100], [n, 1], seed=i).upload() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, st in zip(ps, streams):
            p.attend(stream=st)
    torch.cuda.synchronize()
    for p in ps:
        check(p.d_out, *p.expected())


@pytest.mark.parametrize("news", [[1, 1], [13, 1], [90, 200]])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_wait_that_runs_out_is_reported(news, dtype):
    """A tile that is never filled (the testing hook): the bounded waits give up, the status
    says so, and the next call is exact.  (The kernel for few rows, and for fp32, has no waits
    but those for its own copies.)"""
    waits = dtype != "f32" and max(news) > 1
    p = Problem4(dtype, 8, 2, 16, [700, 300], news).upload()
    for limit in (2_000_000, 500, 1):
        kv.kv_debug_config(0, limit)
        p.attend()
        kv.kv_debug_config(-1, 2_000_000_000)
        p.d_out.fill_(7)
        p.attend()  # right behind it
        assert kv.kv_device_status() == (kv.KV_ERR_DEVICE_TIMEOUT if waits else kv.KV_OK)
        check(p.d_out, *p.expected())


# --- as a program uses them --------------------------------------------------------------
@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_path_together(dtype, loc):
    """Prompts, proposed tokens and single tokens turned to their positions, quantised and
    attended in place; the cache read back gives the same attention."""
    from offloaded_kv_cache_gb300 import workloads as W
    from offloaded_kv_cache_gb300.pipeline import DecodeLayer, Q4Cache, Rotary
    spec = W.tiny_spec(dtype=dtype, batch=2, hq=8, hkv=2, context=200, ps=16, topk=2, index=5)
    layer = DecodeLayer(W.generate(spec, context_lens=[200, 170]), kv_loc=loc)
    t = TORCH[dtype]
    q4 = Q4Cache(layer.shape, layer.block_table, torch.zeros(2, dtype=torch.int32, device="cuda"),
                 kv_loc=loc)
    rotary = Rotary(128, base=500000.0, interleaved=True)
    g = torch.Generator().manual_seed(1)
    for n in ([150, 120], [0, 5], [1, 1], [3, 1]):
        start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        k, v = (torch.randn(sum(n), 2, D, generator=g).to(t).cuda() for _ in "kv")
        q = torch.randn(sum(n), 8, D, generator=g).to(t).cuda()
        old = q4.context_lens.tolist()
        q = q4.append(k, v, start, max(n), rotary=rotary, q=q)
        got = q4.attend(q, start, max(n), layer.scale)
        torch.cuda.synchronize()
        # what was stored: keys turned, then quantised
        at = torch.cat([torch.arange(o, o + m) for o, m in zip(old, n)])
        want = turned(k.cpu(), at, rotary.freq.cpu(), True)
        slack = turned_tolerance(k.cpu(), dtype, 64, True)
        for b, m in enumerate(n):
            for i in range(m):
                pos, row = old[b] + i, int(start[b]) + i
                ph = int(layer.block_table[b, pos // 16])
                stored = [x[ph, :, pos % 16].cpu().numpy() for x in (q4.k_codes, q4.k_scale, q4.k_power)]
                step = np.repeat(STEPS[stored[1]] * 2.0 ** (stored[2].astype(float) - 127)[..., None], 16, -1)
                off = np.abs(restore4(*stored) - want[row].numpy())
                assert (off <= 0.5 * step + slack[row].numpy()).all()
    assert q4.context_lens.tolist() == [154, 127]
    back = [torch.zeros(spec.num_phys_pages, 2, 16, D, dtype=t, device="cuda") for _ in "kv"]
    q4.read_back(*back)
    layer.context_lens.copy_(q4.context_lens)
    torch.cuda.synchronize()
    layer.k_cache.copy_(back[0])
    layer.v_cache.copy_(back[1])
    again = layer.chunk_attn(q, start, max(n))
    torch.cuda.synchronize()
    # both compute the same sums, each within 2^-8 (2^-11, 2^-24) of weights and result
    tol = {"f32": 1e-5, "f16": 2.0 ** -9, "bf16": 2.0 ** -6}[dtype]
    assert float((got.float() - again.float()).abs().max()) <= tol * (1 + float(back[1].abs().max()))


# --- random batches ----------------------------------------------------------------------
def draw(seed):
    r = random.Random(seed)
    dtype = r.choice(["f16", "bf16", "bf16", "f32"])
    hq, hkv = r.choice([(1, 1), (8, 2), (4, 4), (7, 1), (32, 8), (10, 2), (48, 4), (66, 1), (160, 1)])
    ps = r.choice([16, 32, 64, 128])
    near = lambda: max(0, r.choice([16, 64, 128, 256, 384, 640]) + r.randint(-2, 2))  # noqa: E731
    lens, news = [], []
    for _ in range(r.randint(1, 6)):
        length = near() if r.random() < 0.5 else r.randint(0, 900)
        n = r.choice([0, 1, 1, 2, 5, r.randint(0, 40), r.randint(0, 300)])
        n = min(n, 6000 // hq)
        if r.random() < 0.9:
            n = min(n, length)
        lens.append(length)
        news.append(n)
    p = Problem4(dtype, hq, hkv, ps, lens, news, r.choice([0, 0, 0, 1, 17, 128, r.randint(1, 700)]),
                 seed=seed, scale=r.choice([None, None, None, 0.5, -0.1, 0.0]),
                 q_size=r.choice([1.0, 1.0, 4.0]), loc=r.choice(["hbm", "hbm", "host"]),
                 extra_rows=r.randint(0 if sum(news) else 1, 3),  # (a call has a row)
                 # (a wide block table takes the forms for long contexts)
                 extra_pages=random.Random(-1 - seed).choice([1, 1500 // ps, 6000 // ps]))
    pages = [(b, i) for b in range(len(lens)) for i in range(-(-lens[b] // ps))]
    bad = bool(pages) and r.random() < 0.25
    if bad:
        for b, i in r.sample(pages, min(len(pages), 2)):
            p.table[b, i] = r.choice([-1, p.pages, 1 << 30])
    if pages and r.random() < 0.25:
        b, i = r.choice(pages)
        ph, h, slot = int(p.table[b, i]), r.randrange(hkv), r.randrange(ps)
        if 0 <= ph < p.pages and p.owned[ph, slot]:
            p.set_nan(r.choice("kv"), ph, h, slot)
    return p, bad


@pytest.mark.parametrize("seed", range(CASES))
def test_random_batch(seed):
    p, bad = draw(seed)
    p.upload()
    p.attend()
    status = kv.kv_device_status()
    assert status == kv.KV_OK or (bad and status == kv.KV_ERR_BOUNDS)
    want, tol = p.expected()
    check(p.d_out, want, tol)
