"""Calls whose units of few rows would be too many to count in 32 bits take the kernels with
larger units; only what those cannot count is refused."""
import pytest

from offloaded_kv_cache_gb300 import kvsparse as kv

FAKE = 0x10000  # 16-byte aligned address that is never dereferenced


def shape(batch, hq, hkv, pages, dtype, loc="hbm", ps=16, phys=None):
    return kv.make_shape(batch, hq, hkv, 128, ps, pages, phys or batch * pages, dtype, loc)


SIZES = [kv.kv_chunk_workspace_bytes, kv.kv_q8_chunk_workspace_bytes, kv.kv_q4_chunk_workspace_bytes]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("loc", ["hbm", "host"])
def test_a_long_fp32_prompt(kvlib, size, loc):
    s = shape(1, 64, 8, 131072 // 16, "f32", loc)
    assert size(s, kv.make_chunk(FAKE, 131072, 131072)) > 0


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_rows_of_very_many_tokens(kvlib, size, dtype):
    """24 rows a kv head over 4096 sequences of 2^21 tokens: three units of 8, or one of 128."""
    s = shape(4096, 64 * 3, 8, 1 << 14, dtype, ps=128, phys=1000)
    assert size(s, kv.make_chunk(FAKE, 4096, 1)) > 0


@pytest.mark.parametrize("size", SIZES)
def test_what_the_largest_units_cannot_count_is_refused(kvlib, size):
    for dtype in ("f32", "f16", "bf16"):
        s = shape(4096, 64, 8, 1 << 19, dtype, ps=128, phys=1000)
        assert size(s, kv.make_chunk(FAKE, 1 << 20, 256)) == 0


def test_calls_that_count_keep_their_plan(kvlib):
    """(8 rows a unit: no pages in the workspace)"""
    s = shape(4, 32, 8, 2048, "f32")
    assert kv.kv_q4_chunk_workspace_bytes(s, kv.make_chunk(FAKE, 8192, 2048)) < 1 << 24
    assert kv.kv_q8_chunk_workspace_bytes(s, kv.make_chunk(FAKE, 8192, 2048)) < 1 << 24
