"""Rows with infinities, NaN and the type's largest values, turned and appended: what is not
finite is what the formula gives in the pair's two channels and nowhere else, and the index is
bit for bit the one built anew over such keys."""
import pytest
import torch

from chunk_util import D, TORCH
from more_util import turned, turned_tolerance
from offloaded_kv_cache_gb300 import kvsparse as kv
from test_gpu_rope import Chunk, ROTS, SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


def special(c, seed):
    """Strews infinities, NaN and large values over q, k and v."""
    g = torch.Generator().manual_seed(seed)
    t = TORCH[c.p.dtype]
    big = torch.finfo(t).max
    values = torch.tensor([float("inf"), -float("inf"), float("nan"), big / 4, -big / 4, 0.0, -0.0]).to(t)
    for n in "qkv":
        x = getattr(c, n)
        which = torch.randint(0, 60, x.shape, generator=g)
        for i, v in enumerate(values):
            x[which == i] = v
        c.d[n].copy_(x)


def same(got, want, tol, dtype):
    """NaN and infinities where the formula has them; elsewhere within the tolerance.  A result
    at the type's border may be either (its tolerance reaches over it)."""
    got = got.double().cpu()
    border = torch.finfo(TORCH[dtype]).max
    near = (want.abs() + tol >= border) & torch.isfinite(want)
    assert torch.equal(torch.isnan(got) & ~near, torch.isnan(want) & ~near)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    rest = torch.isfinite(want) & ~near
    assert (got[rest] - want[rest]).abs().le(tol[rest]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rot,inter", ROTS)
def test_rows(dtype, rot, inter):
    for i, (hq, hkv, ps, before, news) in enumerate(SHAPES[:4]):
        # (no position 0, and no frequency whose sine is 0: infinity * 0 would hang on a sign)
        c = Chunk(dtype, hq, hkv, ps, [n + 1 for n in before], news, rot, inter, seed=i)
        special(c, i)
        c.turn()
        torch.cuda.synchronize()
        for n, out in (("q", c.q_out), ("k", c.k_out)):
            x = getattr(c, n)
            want = turned(x, c.at, c.freq, inter)
            # the tolerance of what is finite in both channels of a pair
            tol = turned_tolerance(x.nan_to_num(nan=0.0, posinf=0.0, neginf=0.0), dtype, rot // 2, inter,
                                   1.0, c.at, c.freq)
            want[~c.mine], tol[~c.mine] = 7.0, 0.0
            same(out, want, tol, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rope", [True, False])
def test_index(dtype, rope):
    bits = torch.int32 if dtype == "f32" else torch.int16
    for i, (hq, hkv, ps, before, news) in enumerate(SHAPES):
        rot, inter = ROTS[i]
        c = Chunk(dtype, hq, hkv, ps, before, news, rot, inter, seed=i)
        special(c, 50 + i)
        mm = c.index()
        anew = mm.clone()
        out = torch.zeros(len(news), dtype=torch.int32, device="cuda")
        c.put(out, mm, rope)
        c.build(anew, out)
        torch.cuda.synchronize()
        assert torch.equal(mm.view(bits), anew.view(bits))
        # the keys in the cache are the rows turned by themselves, values the rows
        c.turn()
        torch.cuda.synchronize()
        keys = c.k_out if rope else c.d["k"]
        for b, n in enumerate(news):
            for r in range(n):
                pos = before[b] + r
                at = int(c.p.table[b, pos // ps])
                for cache, rows in ((c.p.d_k, keys), (c.p.d_v, c.d["v"])):
                    assert torch.equal(cache[at, :, pos % ps].view(bits).cpu(),
                                       rows[c.p.start[b] + r].view(bits).cpu())
