"""The chunk operators' boundary without a GPU: struct layouts, workspace
sizes, refused arguments; and the 8-bit format's definition used by the GPU
tests, against torch's own conversion."""
import ctypes

import numpy as np
import pytest
import torch

from chunk_util import E4M3, quantise, restore
from offloaded_kv_cache_gb300 import kvsparse as kv

FAKE = 0x10000  # 16-byte aligned address that is never dereferenced


def shape(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                max_pages_per_seq=4, num_phys_pages=8, dtype="bf16", kv_loc="hbm")
    base.update(kw)
    return kv.make_shape(**base)


def chunk(**kw):
    base = dict(q_start=FAKE, total_q=10, max_q_len=5, window=0)
    base.update(kw)
    return kv.make_chunk(**base)


CACHE = kv.make_q8_cache(FAKE, FAKE, FAKE, FAKE)


def calls(s, c, **kw):
    """Status of every chunk entry point, in a fixed order."""
    a = dict(q=FAKE, k=FAKE, v=FAKE, cache=CACHE, bt=FAKE, ctx=FAKE, scale=0.1, out=FAKE, ws=FAKE,
             nws=1 << 40)
    a.update(kw)
    return (kv.kv_chunk_attn(s, c, a["q"], a["k"], a["v"], a["bt"], a["ctx"], a["scale"], a["out"],
                             a["ws"], a["nws"], check=False),
            kv.kv_q8_chunk_attn(s, c, a["q"], a["cache"], a["bt"], a["ctx"], a["scale"], a["out"],
                                a["ws"], a["nws"], check=False),
            kv.kv_q8_append(s, c, a["q"], a["out"], a["cache"], a["bt"], a["ctx"], None,
                            check=False))


def test_struct_layouts():
    assert ctypes.sizeof(kv.kv_chunk) == 24 and kv.kv_chunk.window.offset == 16
    assert ctypes.sizeof(kv.kv_q8_cache) == 32


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), kv.KV_ERR_UNSUPPORTED), (dict(page_size=48), kv.KV_ERR_UNSUPPORTED),
    (dict(dtype=7), kv.KV_ERR_UNSUPPORTED), (dict(num_q_heads=7), kv.KV_ERR_INVALID_ARG),
    (dict(batch=0), kv.KV_ERR_INVALID_ARG), (dict(kv_loc=5), kv.KV_ERR_INVALID_ARG)])
def test_bad_shapes_are_refused(kvlib, kw, code):
    s, c = shape(**kw), chunk()
    assert calls(s, c) == (code,) * 3
    assert kv.kv_q8_read(s, CACHE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, check=False) == code
    assert kv.kv_chunk_workspace_bytes(s, c) == 0
    assert kv.kv_q8_chunk_workspace_bytes(s, c) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q_start=None), kv.KV_ERR_INVALID_ARG), (dict(q_start=FAKE + 2), kv.KV_ERR_INVALID_ARG),
    (dict(total_q=0), kv.KV_ERR_INVALID_ARG), (dict(max_q_len=0), kv.KV_ERR_INVALID_ARG),
    (dict(window=-1), kv.KV_ERR_INVALID_ARG),
    (dict(total_q=1 << 30), kv.KV_ERR_UNSUPPORTED)])
def test_bad_chunks_are_refused(kvlib, kw, code):
    s, c = shape(), chunk(**kw)
    assert calls(s, c) == (code,) * 3
    assert kv.kv_chunk_workspace_bytes(s, c) == 0
    c = chunk()
    c.reserved = 1
    assert calls(s, c) == (kv.KV_ERR_INVALID_ARG,) * 3
    assert calls(s, None) == (kv.KV_ERR_INVALID_ARG,) * 3


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=FAKE + 8), dict(out=None), dict(bt=FAKE + 2),
                                dict(ctx=None)])
def test_bad_pointers_are_refused(kvlib, kw):
    assert calls(shape(), chunk(), **kw) == (kv.KV_ERR_INVALID_ARG,) * 3


def test_lengths_that_overlap_in_part_are_refused(kvlib):
    for d in (4, -4):
        assert kv.kv_q8_append(shape(), chunk(), FAKE, FAKE, CACHE, FAKE, FAKE, FAKE + d,
                               check=False) == kv.KV_ERR_INVALID_ARG


def test_more_tiles_than_an_int_are_refused(kvlib):
    s = shape(batch=1, num_q_heads=8, num_kv_heads=8, page_size=128, num_phys_pages=1 << 20,
              max_pages_per_seq=1 << 20)
    assert kv.kv_chunk_workspace_bytes(s, chunk(total_q=1 << 27, max_q_len=1 << 27)) == 0
    assert calls(s, chunk(total_q=1 << 27, max_q_len=1 << 27))[0] == kv.KV_ERR_UNSUPPORTED


def test_bad_scales_and_outputs_are_refused(kvlib):
    for scale in (float("nan"), float("inf")):
        assert calls(shape(), chunk(), scale=scale)[:2] == (kv.KV_ERR_INVALID_ARG,) * 2
    read = lambda **kw: kv.kv_q8_read(*[kw.get(k, v) for k, v in dict(  # noqa: E731
        shape=shape(), cache=CACHE, bt=FAKE, ctx=FAKE, to=FAKE, pages=4, k=FAKE, v=FAKE).items()],
        check=False)
    for kw in (dict(k=None), dict(v=FAKE + 4), dict(to=None), dict(pages=0), dict(ctx=FAKE + 1)):
        assert read(**kw) == kv.KV_ERR_INVALID_ARG
    assert read(pages=1 << 40) == kv.KV_ERR_UNSUPPORTED


def test_workspace_sizes(kvlib):
    """Bounded by the GPU's size, not by the batch, and enough for a smaller one."""
    small = kv.kv_chunk_workspace_bytes(shape(), chunk())
    assert 0 < small < 1 << 24
    for dtype in ("f32", "f16", "bf16"):
        big = shape(batch=512, num_q_heads=64, num_kv_heads=8, max_pages_per_seq=4096,
                    num_phys_pages=1 << 20, dtype=dtype)
        assert kv.kv_chunk_workspace_bytes(big, chunk(total_q=1 << 20, max_q_len=1 << 15)) < 1 << 27


def test_e4m3_definition():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3, want, equal_nan=True)


@pytest.mark.parametrize("dtype,least", [("f32", -110), ("bf16", -110), ("f16", -15)])
def test_quantiser_definition(dtype, least):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 128)) * 2.0 ** rng.integers(-30, 18, (200, 1))
    x[0] = 0
    c, s = quantise(x, dtype)
    e = s.astype(int) - 127
    top = np.abs(x).max(-1)
    assert (e >= least).all() and (e <= 7).all() and e[0] == least
    free = (e > least) & (e < 7)
    assert (top[free] <= 448 * 2.0 ** e[free]).all() and (top[free] > 224 * 2.0 ** e[free]).all()
    y = torch.from_numpy(np.clip(x * 2.0 ** -e[:, None], -448, 448)).float()
    t = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # float rounds the quotient first: compare where that is exact
    same = y.double().numpy() == np.clip(x * 2.0 ** -e[:, None], -448, 448)
    assert np.array_equal(c[same], t[same])
    err = np.abs(restore(c, s) - np.clip(x, -57344, 57344))
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * 2.0 ** e[:, None])).all()


def test_pipeline_refuses_tensors_the_kernels_would_misread():
    """A bare address says nothing of type, shape, order or place."""
    from offloaded_kv_cache_gb300 import pipeline
    x = torch.zeros(3, 2, 128)
    for got, shape, dtype in ((x, (3, 2, 128), torch.float32),      # not on the device
                              (x, (3, 2, 128), torch.float16),
                              (x, (3, 4, 128), torch.float32)):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            pipeline._need(got, "q", shape, dtype)
    table = torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    q8 = pipeline.Q8Cache(kv.make_shape(1, 4, 2, 128, 16, 2, 2, "f32", "hbm"), table, lens,
                          device="cpu")
    start = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="q_start"):
        q8.append(x, x, start, 3, stream=0)
    with pytest.raises(ValueError, match="q_start"):
        q8.attend(torch.zeros(3, 4, 128), start, 3, 1.0, stream=0)
    with pytest.raises(ValueError, match="k_out"):
        q8.read_back(torch.zeros(2, 2, 16, 128), torch.zeros(2, 2, 16, 128), stream=0)
