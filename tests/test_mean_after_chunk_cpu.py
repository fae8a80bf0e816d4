"""What a layer's build_mean_index(last_only=True) rebuilds: the last pages after one append,
every page after a chunk or several appends, without a GPU."""
import types

import pytest
import torch

from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import pipeline

SHAPE = kv.make_shape(2, 8, 2, 128, 16, 4, 8, "bf16", "hbm")
NEW = torch.zeros(3, 2, 128)


@pytest.fixture
def layer(monkeypatch):
    calls = []
    for name in ("kv_page_mean_build", "kv_page_mean_refresh"):
        monkeypatch.setattr(kv, name, lambda *a, _n=name: calls.append(_n))
    for name in ("kv_append_token", "kv_rope_append"):
        monkeypatch.setattr(kv, name, lambda *a: None)
    monkeypatch.setattr(pipeline, "_chunk_inputs", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x = pipeline.DecodeLayer.__new__(pipeline.DecodeLayer)
    x.spec = types.SimpleNamespace(num_phys_pages=8, num_kv_heads=2, head_dim=128, dtype="bf16")
    x.shape, x.device, x.calls = SHAPE, "cpu", calls
    x.mean = x.window = x.context_lens = x.k_cache = x.v_cache = x.block_table = x.minmax = None
    x._unmeant, x._replayed = 0, False
    return x


def chunk(layer):
    layer.append_chunk(NEW, NEW, torch.zeros(3, dtype=torch.int32), 3, stream=0)


def built(layer, **kw):
    layer.calls.clear()
    layer.build_mean_index(stream=0, **kw)
    assert len(layer.calls) == 1
    return layer.calls[0] == "kv_page_mean_build"


def test_the_first_build_is_whole(layer):
    assert built(layer, last_only=True) and not built(layer, last_only=True)


def test_after_each_append_the_last_pages(layer):
    assert built(layer)
    for _ in range(3):
        layer.append(NEW, NEW, stream=0)
        assert not built(layer, last_only=True)
    assert built(layer)


def test_after_several_appends_every_page(layer):
    built(layer)
    layer.append(NEW, NEW, stream=0)
    layer.append(NEW, NEW, stream=0)
    assert built(layer, last_only=True)
    layer.append(NEW, NEW, stream=0)
    assert not built(layer, last_only=True)


def test_after_a_chunk_every_page(layer):
    built(layer)
    chunk(layer)
    assert built(layer, last_only=True) and not built(layer, last_only=True)
    chunk(layer)
    layer.append(NEW, NEW, stream=0)
    assert built(layer, last_only=True) and not built(layer, last_only=True)


def test_once_a_graph_holds_a_chunk_every_page(layer, monkeypatch):
    built(layer)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    chunk(layer)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for _ in range(3):
        assert built(layer, last_only=True)
