"""Chunk attention with a sliding window over a block table whose pages behind every
window have been given back: their entries are out of range (or another sequence's),
which is no error; an entry that some row needs still is one."""
import pytest
import torch

from chunk_util import Problem, check
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


def first_needed(p, b):
    """The first token that a row of sequence b sees."""
    return max(0, p.lens[b] - p.news[b] - p.window + 1)


def free(p, b, upto):
    """Gives back sequence b's pages that lie wholly before token `upto`."""
    count = upto // p.ps
    p.table[b, :count] = torch.tensor([-1, p.pages, 1 << 30], dtype=torch.int32).repeat(count)[:count]
    return count


# chunk sizes for every kernel and form; extra pages for those that the table's width chooses
@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 13, 90, 200])
@pytest.mark.parametrize("ps,window,extra", [(16, 40, 1), (16, 150, 300), (128, 100, 40), (32, 1, 1)])
def test_freed_pages(dtype, n, ps, window, extra, q8):
    p = Problem(dtype, 4, 2, ps, [700, 431, 90, 30], [n, 1, min(n, 90), 0], window, q8=q8, seed=n,
                extra_pages=extra)
    assert sum(free(p, b, first_needed(p, b)) for b in range(3)) > 3
    p.table[3, :2] = -1  # (no row, so no page is needed)
    p.upload()
    p.attend()
    assert kv.kv_device_status() == kv.KV_OK
    check(p.d_out, *p.expected())
    # one page more, which the first row needs
    assert free(p, 0, first_needed(p, 0) + ps) > 0
    p.d_table.copy_(p.table)
    p.attend()
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    check(p.d_out, *p.expected())


@pytest.mark.parametrize("q8", [False, True], ids=["own", "q8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 200])
def test_freed_pages_of_a_cache_in_host_memory(dtype, n, q8):
    p = Problem(dtype, 4, 2, 16, [700, 431], [n, 1], 100, q8=q8, loc="host")
    assert sum(free(p, b, first_needed(p, b)) for b in range(2)) > 5
    p.upload()
    p.attend()
    assert kv.kv_device_status() == kv.KV_OK
    check(p.d_out, *p.expected())
