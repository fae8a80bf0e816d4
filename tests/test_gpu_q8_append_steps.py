"""kv_q8_append where a block takes several steps (a sequence has more steps of 32 vectors
than blocks: 2432 blocks over the batch): the pages, positions and data that a block
carries from step to step, a ragged last step, sequences of other lengths and none, and
what only a later step meets."""
import pytest
import torch

from offloaded_kv_cache_gb300 import kvsparse as kv
from test_gpu_q8 import Append, _lib  # noqa: F401  (the fixture is used)

pytestmark = pytest.mark.gpu


def batch(n, most, seed):
    g = torch.Generator().manual_seed(seed)
    news = torch.randint(0, 4, (n,), generator=g).tolist()
    news[0], news[n // 2], news[n - 1] = most, most - 1, most - 3  # a few long ones
    before = torch.randint(0, 50, (n,), generator=g).tolist()
    return before, news


# (tokens x heads / 32 steps against 2432 / sequences blocks: 70 / 38, 73 / 38, 41 / 25, 102 / 19)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,most,hkv,ps", [(64, 70, 32, 16), (64, 71, 33, 16), (100, 185, 7, 32),
                                           (128, 65, 50, 64)])
def test_several_steps(dtype, n, most, hkv, ps, in_place):
    before, news = batch(n, most, n + most)
    assert -(-most * hkv // 32) > -(-2432 // n)
    a = Append(dtype, hkv, ps, before, news, seed=most)
    out = a.before if in_place else torch.full((n,), -9, dtype=torch.int32, device="cuda")
    a.run(out)
    a.check()
    assert out.tolist() == a.p.lens


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bad_page_in_a_later_step(dtype, in_place):
    """Tokens of one page are dropped, the sequence keeps its length, the others go in."""
    before, news = batch(64, 70, 5)
    before[0] = 3
    a = Append(dtype, 32, 16, before, news, seed=5)
    a.p.table[0, 4] = a.p.pages  # tokens 61 .. 72 of the chunk; step 38 and later ones are second steps
    a.p.d_table.copy_(a.p.table)
    out = a.before if in_place else torch.full((64,), -9, dtype=torch.int32, device="cuda")
    a.run(out)
    assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
    a.check()
    assert out.tolist() == [before[0]] + a.p.lens[1:]
