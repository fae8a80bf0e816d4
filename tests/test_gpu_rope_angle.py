"""Turned unit vectors are the cosine and the sine of the angle, off by no more than the header's
bound beside what fp32 sines are."""
import math
import random

import pytest
import torch

from chunk_util import D
from more_util import near_2pi
from offloaded_kv_cache_gb300 import kvsparse as kv
from test_gpu_rope import Chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("lo,hi", [(-70, -9), (-8, 0), (1, 20), (20, 53)])
def test_bound(kvlib, lo, hi, inter):
    rng = random.Random(lo)
    freq = torch.tensor([math.ldexp(rng.uniform(1, 2) * rng.choice([-1, 1]), rng.randint(lo, hi))
                         for _ in range(64)], dtype=torch.float64)
    at = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31] +
                      [rng.randint(-2 ** 31, 2 ** 31 - 1) for _ in range(20)] +
                      [rng.randint(0, 1 << 20) for _ in range(7)])
    c = Chunk("f32", 1, 1, 16, [0], [30], 128, inter, freq=freq, given=at)
    j = torch.arange(64)
    a, b = (2 * j, 2 * j + 1) if inter else (j, j + 64)
    x = torch.zeros(c.p.total, 1, D)
    x[..., a] = 1.0
    c.d["q"].copy_(x)
    c.turn()
    got = c.q_out.double().cpu()[:30, 0]
    angle = near_2pi(freq, at)[:30]
    t = at[:30, None].double().abs()
    turns = t * (2.0 ** -64 + freq.abs() * 2.0 ** -66) + 2.0 ** -33
    # sine and cosine of at most an eighth of a turn rounded to 24 bits (2^-24 * pi / 4), within
    # two units in the last place (2^-23): below 2^-21
    tol = 2 * math.pi * turns + 2.0 ** -21
    assert ((got[:, a] - torch.cos(angle)).abs() <= tol).all()
    assert ((got[:, b] - torch.sin(angle)).abs() <= tol).all()
    assert kv.kv_device_status() == kv.KV_OK
