"""Frequencies that the device finds unfit: the pair is multiplied by the scale alone, the
others turn, and the status word says so; without turning none is read."""
import math

import pytest
import torch

from more_util import frequencies, turned, turned_tolerance
from offloaded_kv_cache_gb300 import kvsparse as kv
from test_gpu_rope import Chunk, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [math.nan, -math.nan, math.inf, -math.inf, 2.0 ** 54, -1e300])
def test_unfit(kvlib, dtype, inter, bad):
    kv.kv_device_status()
    for at in (0, 15, 31):
        freq = frequencies(64)
        freq[at] = bad
        c = Chunk(dtype, 4, 2, 16, [3, 0, 70], [20, 1, 0], 64, inter, scale=1.25, freq=freq)
        still = freq.clone()
        still[at] = 0.0
        for call in (c.turn, lambda: c.put(torch.zeros(3, dtype=torch.int32, device="cuda"))):
            c.q_out.fill_(7.0)
            call()
            torch.cuda.synchronize()
            assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
            want = turned(c.q, c.at, still, inter, 1.25)
            tol = turned_tolerance(c.q, dtype, 32, inter, 1.25, c.at, still)
            want[~c.mine], tol[~c.mine] = 7.0, 0.0
            near(c.q_out, want, tol)
        c.put(rope=False)
        assert kv.kv_device_status() == kv.KV_OK


def test_the_largest_that_fit(kvlib):
    kv.kv_device_status()
    freq = frequencies(64)
    freq[3], freq[4] = math.nextafter(2.0 ** 54, 0), -math.nextafter(2.0 ** 54, 0)
    c = Chunk("f32", 4, 2, 16, [3], [20], 64, freq=freq)
    c.turn()
    torch.cuda.synchronize()
    assert kv.kv_device_status() == kv.KV_OK
