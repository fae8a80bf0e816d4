"""kv_q8_append and kv_q8_read: bit for bit what the format's definition gives
in 64 bits (tests/chunk_util.py), at ragged lengths, every type, page size
and location, with the vectors where a quantiser goes wrong."""
import numpy as np
import pytest
import torch

from chunk_util import D, E4M3, TORCH, Problem, quantise, restore
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


class Append:
    """A batch whose chunks go into an empty 8-bit cache."""

    def __init__(self, dtype, hkv, ps, before, news, loc="hbm", seed=0, rows=None, max_new=None):
        lens = [a + n for a, n in zip(before, news)]
        self.p = p = Problem(dtype, hkv, hkv, ps, lens, news, seed=seed, loc=loc)
        g = torch.Generator().manual_seed(seed + 1)
        mag = torch.exp2(torch.randint(-9, 9, (p.total, hkv, 1), generator=g).float())
        self.new = {}
        for name in ("k", "v"):
            x = torch.randn(p.total, hkv, D, generator=g) * mag
            if rows is not None:
                x[:rows.shape[0]] = rows[:, None]
            self.new[name] = x.to(TORCH[dtype])
        self.before = torch.tensor(before, dtype=torch.int32, device="cuda")
        p.upload(max_new=max_new)
        shape = (p.pages, hkv, ps, D)
        self.code = {n: p.put(torch.full(shape, 0xAB, dtype=torch.uint8), True) for n in "kv"}
        self.scale = {n: p.put(torch.full(shape[:3], 0xCD, dtype=torch.uint8), True) for n in "kv"}
        self.cache = kv.make_q8_cache(self.code["k"], self.code["v"], self.scale["k"],
                                      self.scale["v"])
        self.d_new = {n: x.cuda() for n, x in self.new.items()}

    def run(self, out=None, stream=None):
        p = self.p
        kv.kv_q8_append(p.shape, p.chunk, self.d_new["k"], self.d_new["v"], self.cache, p.d_table,
                        self.before, out, torch.cuda.current_stream() if stream is None else stream)
        torch.cuda.synchronize()

    def check(self):
        p = self.p
        for n in "kv":
            code = np.full((p.pages, p.hkv, p.ps, D), 0xAB, dtype=np.uint8)
            scale = np.full((p.pages, p.hkv, p.ps), 0xCD, dtype=np.uint8)
            c, s = quantise(self.new[n].double().numpy(), p.dtype)
            for b, k in enumerate(p.news):
                for i in range(k):
                    pos = p.lens[b] - k + i
                    ph = int(p.table[b, pos // p.ps])
                    if 0 <= ph < p.pages:
                        code[ph, :, pos % p.ps] = c[p.start[b] + i]
                        scale[ph, :, pos % p.ps] = s[p.start[b] + i]
            assert np.array_equal(self.scale[n].cpu().numpy(), scale)
            assert np.array_equal(self.code[n].cpu().numpy(), code)


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype,hkv,ps,before,news", [
    ("bf16", 8, 16, [0, 15, 16, 100, 33], [1, 1, 1, 0, 1]),
    ("f16", 4, 32, [0, 31, 7], [70, 1, 33]),
    ("f32", 1, 64, [63, 0], [2, 129]),
    ("bf16", 3, 128, [5], [300]),
    ("f16", 32, 16, [17, 0, 1], [5, 16, 40]),
])
def test_append(dtype, hkv, ps, before, news, loc):
    a = Append(dtype, hkv, ps, before, news, loc)
    out = torch.full((len(news),), -9, dtype=torch.int32, device="cuda")
    a.run(out)
    a.check()
    assert out.tolist() == a.p.lens and a.before.tolist() == before


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_append_difficult_vectors(dtype):
    """Zeros of both signs, one large element, maxima on both sides of 448 * 2^e,
    ties, subnormals, the saturated range, infinities and NaN."""
    t = TORCH[dtype]
    big = torch.finfo(t).max
    rows = [torch.zeros(D), -torch.zeros(D)]
    for top in (448.0, 449.0, 447.0, 1.75, 1.7500001, 57344.0, 57345.0, 60000.0, big, 2.0 ** -15,
                2.0 ** -24, 2.0 ** -110, 2.0 ** -126, 1e-30, 2.0 ** -133, 2.0 ** -149):
        x = torch.linspace(-1, 1, D, dtype=torch.float64) * top
        rows.append(x.float())
        y = torch.zeros(D)
        y[77] = -top
        rows.append(y)
    # every midpoint of two neighbouring codes, under a maximum of 448
    mid = torch.from_numpy((E4M3[:126] + E4M3[1:127]) / 2).float()
    rows.append(torch.cat([mid, torch.tensor([448.0, -448.0])]))
    rows.append(-rows[-1] / 64)
    for bad in (float("inf"), -float("inf"), float("nan")):
        x = torch.randn(D, generator=torch.Generator().manual_seed(3))
        x[5] = bad
        rows.append(x)
    rows = torch.stack(rows)
    a = Append(dtype, 2, 16, [3], [len(rows)], rows=rows)
    a.run()
    a.check()


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 0, 7], [1000, 3, 64]])
def test_append_lengths_in_place(news):
    before = [5, 9, 0]
    a = Append("bf16", 4, 16, before, news)
    a.run(a.before)
    a.check()
    assert a.before.tolist() == [x + n for x, n in zip(before, news)]


def test_append_skips_what_is_out_of_range():
    """A bad page drops its tokens and keeps the length; a bad length or chunk skips the sequence."""
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
    # a chunk longer than the launch was sized for, and starts out of order
    for start in ([0, 41, 45, 50, 55], [0, 40, 30, 50, 71], [-1, 40, 60, 66, 71]):
        a = Append("f16", 2, 16, [0, 3, 2, 4], [40, 20, 6, 5])
        a.p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        a.run(out)
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype,hkv,ps,lens", [
    ("bf16", 8, 16, [1, 16, 17, 0, 300]),
    ("f16", 4, 32, [95, 700]),
    ("f32", 1, 64, [129, 64, 1]),
    ("bf16", 3, 128, [1000]),
])
def test_read(dtype, hkv, ps, lens, loc):
    p = Problem(dtype, hkv, hkv, ps, lens, [0] * len(lens), q8=True, loc=loc).upload()
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
        value = restore(p.code[n].numpy(), p.scale8[n].numpy())
        for b, length in enumerate(lens):
            for j in range(length):
                to = int(table[b, j // ps])
                if to >= 0:
                    x[to, :, j % ps] = value[int(p.table[b, j // ps]), :, j % ps]
        want[n] = torch.from_numpy(x)
    got = {n: torch.full((out_pages, hkv, ps, D), 7.0, dtype=TORCH[dtype], device="cuda")
           for n in "kv"}
    kv.kv_q8_read(p.shape, p.cache, p.d_table, p.d_lens, table.cuda(), out_pages, got["k"],
                  got["v"], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for n in "kv":
        assert torch.equal(got[n].double().cpu(), want[n])


def test_read_every_code_and_scale():
    """All 256 codes under every scale byte a writer of the type leaves, and NaN."""
    for dtype, scales in (("f16", range(112, 135)), ("bf16", range(17, 135)), ("f32", range(17, 135))):
        scales = list(scales) + [255]
        p = Problem(dtype, 1, 1, 128, [2 * len(scales)], [0], q8=True)
        code = torch.arange(256, dtype=torch.uint8).reshape(2, D).repeat(len(scales), 1)
        byte = torch.tensor(scales, dtype=torch.uint8).repeat_interleave(2)
        for j in range(2 * len(scales)):
            ph = int(p.table[0, j // 128])
            for n in "kv":
                p.code[n][ph, 0, j % 128] = code[j]
                p.scale8[n][ph, 0, j % 128] = byte[j]
        p.upload()
        out = [torch.zeros(p.pages, 1, 128, D, dtype=TORCH[dtype], device="cuda") for _ in "kv"]
        kv.kv_q8_read(p.shape, p.cache, p.d_table, p.d_lens, p.d_table, p.pages, out[0], out[1],
                      torch.cuda.current_stream())
        want = torch.from_numpy(restore(code.numpy(), byte.numpy()))
        rows = [(int(p.table[0, j // 128]), j % 128) for j in range(2 * len(scales))]
        for x in out:
            got = torch.stack([x[a, 0, b] for a, b in rows]).double().cpu()
            assert torch.equal(got.nan_to_num(nan=1e9), want.nan_to_num(nan=1e9))


def test_read_out_of_range():
    p = Problem("bf16", 2, 2, 16, [50, 20], [0, 0], q8=True)
    p.table[0, 2] = -5
    p.upload()
    out = [torch.full((p.pages, 2, 16, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    to = p.table.clone()
    to[0, 2] = p.pages - 1
    to[1, 1] = p.pages
    kv.kv_q8_read(p.shape, p.cache, p.d_table, p.d_lens, to.cuda(), p.pages, out[0], out[1],
                  torch.cuda.current_stream())
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    assert not torch.isnan(out[0]).any()
    p.d_lens[0] = p.max_pages * 16 + 1
    kv.kv_q8_read(p.shape, p.cache, p.d_table, p.d_lens, p.d_table, p.pages, out[0], out[1],
                  torch.cuda.current_stream())
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
