"""Random ragged batches through kv_chunk_attn and kv_q8_chunk_attn against the
definition in 64 bits: every type, head grouping, page size, location, window,
lengths on and around the tile sizes, rows that see nothing, out-of-range pages
and vectors that are not finite."""
import os
import random

import pytest
import torch

from chunk_util import Problem, check
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu

CASES = int(os.environ.get("KV_CHUNK_FUZZ_CASES", "60"))


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield


def draw(seed):
    r = random.Random(seed)
    dtype, q8 = r.choice(["f16", "bf16", "bf16", "f32"]), r.random() < 0.5
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
    p = Problem(dtype, hq, hkv, ps, lens, news, r.choice([0, 0, 0, 1, 17, 128, r.randint(1, 700)]),
                q8=q8, seed=seed, scale=r.choice([None, None, None, 0.5, -0.1, 0.0]),
                q_size=r.choice([1.0, 1.0, 4.0]), loc=r.choice(["hbm", "hbm", "host"]),
                extra_rows=r.randint(0 if sum(news) else 1, 3),  # (a call has a row)
                # (a wide block table takes the forms for long contexts)
                extra_pages=random.Random(-1 - seed).choice([1, 1500 // ps, 6000 // ps]))
    pages = [(b, i) for b in range(len(lens)) for i in range(-(-lens[b] // ps))]
    bad = bool(pages) and r.random() < 0.25
    if bad:
        for b, i in r.sample(pages, min(len(pages), 2)):
            p.table[b, i] = r.choice([-1, p.pages, 1 << 30])
    if pages and r.random() < 0.25:  # a vector that is not finite
        b, i = r.choice(pages)
        ph, h, slot = int(p.table[b, i]), r.randrange(hkv), r.randrange(ps)
        if 0 <= ph < p.pages and p.owned[ph, slot]:
            name = r.choice("kv")
            if q8:
                p.code[name][ph, h, slot], p.scale8[name][ph, h, slot] = 0x7F, 255
            elif name == "k":
                p.k[ph, h, slot] = float("nan")
            else:
                p.v[ph, h, slot, r.randrange(128)] = r.choice([float("nan"), float("inf")])
    return p, bad


@pytest.mark.parametrize("seed", range(CASES))
def test_random_batch(seed):
    p, bad = draw(seed)
    p.upload()
    p.attend()
    status = kv.kv_device_status()
    assert status == kv.KV_OK or (bad and status == kv.KV_ERR_BOUNDS)
    want, tol = p.expected()
    got = p.d_out.double().cpu()
    if not p.q8:  # a row that sees an infinite value may hold the infinity instead of NaN
        got[torch.isinf(got) & torch.isnan(want)] = float("nan")
    check(got, want, tol)
