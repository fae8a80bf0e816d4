"""Infinities and NaN among the values that a row sees: a channel is what the sum of
positive weights times values makes of them in exact arithmetic (an infinity where all
are of one sign, else NaN), wherever tiles, units and the CTAs' shares are cut and
however small a weight is."""
import math

import pytest
import torch

from chunk_util import Problem, check
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


def put(p, b, j, h, c, x):
    p.v[p.table[b, j // p.ps], h, j % p.ps, c] = x


def expected(p):
    """The definition's outputs: Problem.expected() has NaN wherever a row sees a value that
    is not finite; here the sum of those values."""
    want, tol = p.expected()
    G = p.hq // p.hkv
    for b, length in enumerate(p.lens):
        for h in range(p.hkv):
            v, ok = p.tokens("v", b, h)
            k, _ = p.tokens("k", b, h)
            for i in range(p.news[b]):
                t = length - p.news[b] + i
                lo = max(0, t - p.window + 1) if p.window else 0
                seen = torch.zeros(length, dtype=torch.bool)
                seen[lo:max(t + 1, lo)] = True
                seen &= ok
                if torch.isnan(k[seen]).any():
                    continue  # the weights are NaN
                x = v[seen]
                odd = torch.where(torch.isfinite(x), 0.0, x).sum(0)
                some = ~torch.isfinite(x).all(0)
                row = want[p.start[b] + i, h * G:(h + 1) * G]
                row[:, some] = odd[some]
    return want, tol


def same(got, want, tol):
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])
    zero = torch.zeros(())
    check(torch.where(inf, zero, got), torch.where(inf, zero, want), tol)


def run(p):
    p.upload()
    p.attend()
    torch.cuda.synchronize()
    same(p.d_out, *expected(p))


def scatter(p, seed):
    """Values that are not finite at tokens spread over sequence 0, channels of every group of lanes."""
    g = torch.Generator().manual_seed(seed)
    for k in range(24):
        j = int(torch.randint(0, p.lens[0], (1,), generator=g))
        c = int(torch.randint(0, 128, (1,), generator=g))
        put(p, 0, j, k % p.hkv, c, (INF, -INF, INF, NAN)[k % 4])
    last = p.lens[0] - 1
    for j, c, x in ((0, 3, INF), (last, 3, -INF), (0, 70, INF), (last, 70, INF), (0, 127, -INF),
                    (last - p.news[0] // 2, 9, INF)):
        put(p, 0, j, 0, c, x)


# chunk sizes for every kernel and form; extra pages for those that the table's width chooses
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 13, 30, 90, 150])
@pytest.mark.parametrize("extra", [1, 90, 300])
def test_scattered(dtype, n, extra):
    p = Problem(dtype, 4, 2, 16, [700, 40], [n, 10], extra_pages=extra, seed=n)
    scatter(p, n)
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 13, 150])
@pytest.mark.parametrize("window", [1, 90, 400])
def test_windows(dtype, n, window):
    p = Problem(dtype, 4, 2, 32, [700, 40], [n, 10], window, extra_pages=40, seed=n)
    scatter(p, n)
    run(p)


@pytest.mark.parametrize("dtype,hq,hkv,n", [("f32", 1, 1, 33), ("f32", 2, 1, 150), ("bf16", 8, 1, 1),
                                            ("f16", 8, 1, 10), ("bf16", 2, 1, 300)])
def test_units_that_many_ctas_share(dtype, hq, hkv, n):
    p = Problem(dtype, hq, hkv, 64, [6000], [n], seed=n)
    for j, c, x in ((5, 1, INF), (3000, 1, INF), (5, 64, INF), (4000, 64, -INF), (5990, 100, -INF)):
        put(p, 0, j, 0, c, x)
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 30, 150, 300])
@pytest.mark.parametrize("order", [1, -1])
def test_weights_that_round_to_zero(dtype, n, order):
    """Scores from -100 to 100 along the context, rising or falling, as exponents of e: most
    weights are below every type's range, none is 0."""
    p = Problem(dtype, 2, 1, 16, [1500], [n], scale=1.0)
    p.q = torch.zeros_like(p.q)
    p.q[:, :, 0] = 1
    ramp = order * torch.linspace(-100, 100, 1500)
    for j in range(1500):
        p.k[p.table[0, j // 16], :, j % 16, 0] = ramp[j]
    for j, c, x in ((2, 4, INF), (700, 5, -INF), (1498, 6, INF), (1499 - n // 2, 7, -INF), (2, 8, NAN),
                    (2, 60, INF), (1400, 60, -INF), (700, 127, INF)):
        put(p, 0, j, 0, c, x)
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 30, 300])
def test_keys_that_are_nan_beside_them(dtype, n):
    p = Problem(dtype, 4, 2, 16, [700], [n])
    scatter(p, n)
    p.k[p.table[0, 690 // 16], 1, 690 % 16] = NAN
    run(p)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 150])
def test_host_resident_cache(dtype, n):
    p = Problem(dtype, 4, 2, 16, [400], [n], loc="host")
    scatter(p, n)
    run(p)


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 30, 90, 200])
@pytest.mark.parametrize("window,extra", [(1, 1), (1, 90), (2, 300)])
def test_rows_that_see_nan_keys_alone(dtype, n, window, extra, q8):
    p = Problem(dtype, 4, 2, 16, [700, 40], [n, 10], window, extra_pages=extra, q8=q8, seed=n)
    for j in (699, 698, 699 - n // 2, 700 - n):
        if q8:
            p.code["k"][p.table[0, j // 16], 1, j % 16] = 0x7F
            p.scale8["k"][p.table[0, j // 16], 1, j % 16] = 255
        else:
            p.k[p.table[0, j // 16], 1, j % 16, 9] = NAN
    p.upload()
    p.attend()
    torch.cuda.synchronize()
    check(p.d_out, *p.expected())
