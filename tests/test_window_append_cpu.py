"""kv_window_trim's refusals, and that every append of a layer with a window runs it first,
on the lengths before, without a GPU."""
import types

import pytest
import torch

from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import pipeline

FAKE = 0x10000  # 16-byte aligned address that is never dereferenced


def shape(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                max_pages_per_seq=4, num_phys_pages=8, dtype="bf16", kv_loc="hbm")
    base.update(kw)
    return kv.make_shape(**base)


SHAPE = shape()


def trim(s=None, ctx=FAKE, **kw):
    base = dict(cache_pages=8, cache_k=FAKE, cache_v=FAKE, slot_page=FAKE, page_slot=FAKE)
    base.update(kw)
    return kv.kv_window_trim(s or shape(), kv.make_window(**base), ctx, check=False)


@pytest.mark.parametrize("kw", [dict(cache_pages=0), dict(cache_pages=-1), dict(slot_page=None),
                                dict(page_slot=None), dict(slot_page=FAKE + 2), dict(ctx=None),
                                dict(ctx=FAKE + 1), dict(s=shape(batch=0))])
def test_bad_arguments_are_refused(kvlib, kw):
    assert trim(**kw) == kv.KV_ERR_INVALID_ARG


def test_shapes_are_checked(kvlib):
    assert trim(shape(head_dim=64)) == kv.KV_ERR_UNSUPPORTED
    wide = shape(batch=1 << 20, num_q_heads=1 << 12, num_kv_heads=1 << 12, num_phys_pages=1)
    assert trim(wide) == kv.KV_ERR_UNSUPPORTED


def test_good_arguments_are_taken(kvlib):
    if torch.cuda.is_available():
        pytest.skip("a call with made-up addresses that every check lets pass")
    assert trim() == kv.KV_ERR_CUDA


def layer(calls, window, monkeypatch):
    for name in ("kv_window_trim", "kv_append_token", "kv_rope_append"):
        monkeypatch.setattr(kv, name, lambda *a, _n=name, **k: calls.append((_n, a)))
    monkeypatch.setattr(pipeline, "_chunk_inputs", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x = types.SimpleNamespace(shape=SHAPE, window=window, context_lens="lens", k_cache=None,
                              v_cache=None, block_table=None, minmax=None, _st=lambda s: s, _unmeant=0, _replayed=False)
    x.trim_window = lambda stream=None: pipeline.DecodeLayer.trim_window(x, stream)
    return x


@pytest.mark.parametrize("window", [None, "window"])
@pytest.mark.parametrize("advance", [True, False])
def test_appends_trim_an_enabled_window_first(monkeypatch, window, advance):
    calls = []
    x = layer(calls, window, monkeypatch)
    new = torch.zeros(3, 2, 128)
    pipeline.DecodeLayer.append(x, new, new, advance=advance, stream="st")
    pipeline.DecodeLayer.append_chunk(x, new, new, torch.zeros(3, dtype=torch.int32), 3,
                                      advance=advance, stream="st")
    names = [n for n, _ in calls]
    if window is None:
        assert names == ["kv_append_token", "kv_rope_append"]
    else:
        assert names == ["kv_window_trim", "kv_append_token", "kv_window_trim", "kv_rope_append"]
        assert calls[0][1] == calls[2][1] == (SHAPE, "window", "lens", "st")
