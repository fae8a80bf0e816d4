"""Calls whose units of 8 rows the host could not count in 32 bits (it goes by the table's
width and the rows that the arrays have), computed by the kernels with larger units."""
import pytest

from chunk_util import Problem, check
from more_util import Problem4
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


@pytest.mark.parametrize("form", [4, 8])
@pytest.mark.parametrize("window", [0, 50])
def test_fp32_of_many_rows(form, window):
    # 4096 rows of 8 heads: units of 8 rows and tiles of 64 tokens are 4098 x 8 x 66004 > 2^31
    kw = dict(extra_rows=4096 - 45, extra_pages=33000, window=window, seed=form)
    lens, news = [300, 77], [40, 5]
    p = Problem4("f32", 64, 8, 128, lens, news, **kw) if form == 4 else \
        Problem("f32", 64, 8, 128, lens, news, q8=True, **kw)
    p.upload(max_new=4096)
    p.attend()
    check(p.d_out, *p.expected())
    once = p.d_out.clone()
    p.d_out.fill_(7.0)
    p.attend()
    assert bool((p.d_out == once).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_rows_of_a_very_wide_table(dtype):
    # 24 rows a kv head: three units of 8 rows and tiles of 64 tokens are 3 x 96 x 8 x 2^20 > 2^31
    lens = [200, 130] + [5] * 94
    p = Problem4(dtype, 192, 8, 128, lens, [1] * 96, extra_pages=(1 << 19) - 4, seed=3)
    p.upload()
    p.attend()
    check(p.d_out, *p.expected())
