"""kv_rope_append refuses rows that lie in the cache or the index it writes, and takes those
beside them."""
import pytest
import torch

from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu

B, HQ, HKV, PS, PAGES, MAXP, TOTAL = 2, 4, 2, 16, 6, 3, 10
CACHE, INDEX = PAGES * HKV * PS * 128 * 2, PAGES * HKV * 2 * 128 * 2
BYTES_Q, BYTES_K = TOTAL * HQ * 128 * 2, TOTAL * HKV * 128 * 2


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


@pytest.mark.parametrize("loc", ["hbm", "host"])
def test_overlaps_are_refused(loc):
    # one device buffer of bf16 1.0, parts of which the calls are given; the caches apart from it
    # where they are in host memory
    one = torch.full((1 << 21,), 1.0, dtype=torch.bfloat16, device="cuda")
    base = one.data_ptr()
    cache = torch.zeros(2 * CACHE // 2, dtype=torch.bfloat16).pin_memory() if loc == "host" else None
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, start = ints(*range(PAGES)).view(B, MAXP), ints(3, 20), ints(0, 4, 9)
    freq = torch.ones(64, dtype=torch.float64, device="cuda")
    rope = kv.make_rope(freq, 128)
    shape = kv.make_shape(B, HQ, HKV, 128, PS, MAXP, PAGES, "bf16", loc)
    chunk = kv.make_chunk(start, TOTAL, 5)
    at = dict(k=0, v=CACHE, mm=2 * CACHE, q=2 * CACHE + INDEX)
    at["q_out"] = at["q"] + BYTES_Q
    at["k_new"] = at["q_out"] + BYTES_Q
    at["v_new"] = at["k_new"] + BYTES_K
    assert at["v_new"] + BYTES_K <= one.numel() * 2

    def call(**kw):
        a = {n: base + x for n, x in {**at, **kw}.items()}
        if cache is not None:
            a["k"], a["v"] = cache.data_ptr() + kw.get("k", 0), cache.data_ptr() + kw.get("v", CACHE)
        return kv.kv_rope_append(shape, chunk, rope, a["q"], a["q_out"], a["k_new"], a["v_new"], a["k"],
                                 a["v"], table, lens, None, a["mm"], check=False)

    good = [dict(), dict(q_out=at["q"]), dict(v_new=at["k_new"]), dict(q=at["k_new"] - 16 - BYTES_Q, q_out=at["v_new"] + BYTES_K)]
    bad = [dict(mm=at["q"]), dict(mm=at["k_new"] + 16), dict(q_out=at["mm"] + INDEX - 16), dict(v=CACHE - 16),
           dict(v=0), dict(q=at["mm"]), dict(k_new=at["mm"] + 16), dict(v_new=at["mm"] + INDEX - 16)]
    if loc == "hbm":
        bad += [dict(q_out=0), dict(q_out=CACHE - 16), dict(q=CACHE + 32), dict(k_new=0), dict(k_new=CACHE - 16),
                dict(v_new=2 * CACHE - 16), dict(mm=CACHE - 16), dict(mm=0)]
    for kw in bad:
        assert call(**kw) == kv.KV_ERR_INVALID_ARG, kw
    torch.cuda.synchronize()
    assert bool((one == 1).all())  # nothing ran
    for kw in good:
        assert call(**kw) == kv.KV_OK, kw
    torch.cuda.synchronize()
