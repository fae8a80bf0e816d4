"""Shapes whose launches would pass 2^31 blocks are refused as unsupported before anything
runs, by the calls and by the workspace sizes."""
import pytest

from offloaded_kv_cache_gb300 import kvsparse as kv

FAKE = 0x10000  # 16-byte aligned address that is never dereferenced
CACHE = kv.make_q8_cache(FAKE, FAKE, FAKE, FAKE)


def shape(batch, loc, dtype="bf16"):
    """Tables for 2^24 tokens a sequence, 8 kv heads: 2^22 blocks of the read back a sequence."""
    return kv.make_shape(batch, 8, 8, 128, 16, 1 << 20, 1000, dtype, loc)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("loc", ["hbm", "host"])
def test_read(kvlib, loc, dtype):
    assert kv.kv_q8_read(shape(512, loc, dtype), CACHE, FAKE, FAKE, FAKE, 1000, FAKE, FAKE,
                         check=False) == kv.KV_ERR_UNSUPPORTED
    # (no device here, or no such memory there)
    assert kv.kv_q8_read(shape(511, loc, dtype), CACHE, FAKE, FAKE, FAKE, 1000, FAKE, FAKE,
                         check=False) in (kv.KV_ERR_CUDA, kv.KV_ERR_LOCATION)


@pytest.mark.parametrize("n", [1, 1000])
def test_attention_through_the_workspace(kvlib, n):
    """A cache in host memory, and many rows over the 8-bit cache, are staged."""
    chunk = kv.make_chunk(FAKE, 1000, n)
    for batch, fits in ((512, False), (300, True)):
        s = shape(batch, "host")
        for size, call in (
                (kv.kv_chunk_workspace_bytes, lambda: kv.kv_chunk_attn(
                    s, chunk, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, FAKE, 1 << 40, check=False)),
                (kv.kv_q8_chunk_workspace_bytes, lambda: kv.kv_q8_chunk_attn(
                    s, chunk, FAKE, CACHE, FAKE, FAKE, 0.1, FAKE, FAKE, 1 << 40, check=False))):
            assert (size(s, chunk) > 0) == fits
            assert (call() == kv.KV_ERR_UNSUPPORTED) == (not fits)
    chunk = kv.make_chunk(FAKE, 1000, 1000)
    assert kv.kv_q8_chunk_workspace_bytes(shape(512, "hbm"), chunk) == 0
    assert kv.kv_chunk_workspace_bytes(shape(512, "hbm"), chunk) > 0  # (reads pages where they are)
