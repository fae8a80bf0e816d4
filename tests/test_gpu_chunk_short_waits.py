"""Bounded waits of chunk attention that run out while other copies and products are in
flight: a tile that is never filled (the testing hook), under limits shorter than a
tile's way from memory.  The call ends, the status says so, and the calls behind it, in
the same stream and on the same SMs, are exact: nothing that was in flight lands in them."""
import pytest
import torch

from chunk_util import Problem, check
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    kv.kv_debug_config(-1, 2_000_000_000)
    assert kv.kv_device_status() == kv.KV_OK


# chunk sizes for every kernel with such waits; extra pages for the forms that the table's width chooses
@pytest.mark.parametrize("q8,dtype,news", [
    (q8, *c) for q8 in (False, True) for c in (("bf16", [1, 1]), ("f16", [13, 1]), ("bf16", [90, 200]))
] + [(True, "f32", [2, 1])])
@pytest.mark.parametrize("extra", [1, 90, 300])
@pytest.mark.parametrize("limit", [1, 500, 3000])
def test_short_limits(dtype, news, extra, limit, q8):
    p = Problem(dtype, 8, 2, 16, [700, 300], news, q8=q8, extra_pages=extra).upload()
    want, tol = p.expected()
    seen = []
    for skip in (0, 8, 0, -1):  # (the first tile of a share is there, the second may not be)
        kv.kv_debug_config(skip, limit)
        p.attend()
        kv.kv_debug_config(-1, 2_000_000_000)
        p.d_out.fill_(7)
        p.attend()  # right behind it
        seen.append(kv.kv_device_status())
        check(p.d_out, want, tol)
    assert set(seen) <= {kv.KV_OK, kv.KV_ERR_DEVICE_TIMEOUT}
    assert seen[0] == seen[2] == kv.KV_ERR_DEVICE_TIMEOUT
