"""DecodeLayer.chunk_attn and Q8Cache refuse, before any call into the library, block
tables and lengths that the kernels would misread: they take bare addresses.  Without a
GPU: the tensors are stand-ins that only say what a tensor on one would."""
import types

import pytest
import torch

from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import pipeline

B, HQ, HKV, PS, PAGES = 2, 8, 2, 16, 6


class Stand:
    """What _need() looks at of a tensor."""

    def __init__(self, shape, dtype, device="cuda:0", contiguous=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.is_cuda, self._contiguous = self.device.type == "cuda", contiguous

    def is_contiguous(self):
        return self._contiguous


@pytest.fixture(autouse=True)
def _no_call(monkeypatch):
    def called(*_args, **_kw):
        raise AssertionError("the library was called")

    for name in ("kv_q8_append", "kv_q8_chunk_attn", "kv_q8_read", "kv_chunk_attn",
                 "kv_chunk_workspace_bytes", "kv_q8_chunk_workspace_bytes", "make_chunk"):
        monkeypatch.setattr(kv, name, called)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def good():
    return dict(block_table=Stand((B, PAGES), torch.int32), context_lens=Stand((B,), torch.int32))


BAD = [
    ("context_lens", Stand((B,), torch.int64)), ("context_lens", Stand((B, 1), torch.int32)),
    ("context_lens", Stand((B + 1,), torch.int32)), ("context_lens", torch.zeros(B, dtype=torch.int32)),
    ("context_lens", Stand((B,), torch.int32, "cuda:1")),
    ("context_lens", Stand((B,), torch.int32, contiguous=False)),
    ("block_table", Stand((B, PAGES), torch.int64)), ("block_table", Stand((B, PAGES - 1), torch.int32)),
    ("block_table", Stand((PAGES, B), torch.int32)), ("block_table", Stand((B * PAGES,), torch.int32)),
    ("block_table", torch.zeros(B, PAGES, dtype=torch.int32)),
    ("block_table", Stand((B, PAGES), torch.int32, "cuda:1")),
    ("block_table", Stand((B, PAGES), torch.int32, contiguous=False)),
]
SHAPE = kv.make_shape(B, HQ, HKV, 128, PS, PAGES, 9, "bf16", "hbm")
START = Stand((B + 1,), torch.int32)
Q, NEW = Stand((3, HQ, 128), torch.bfloat16), Stand((3, HKV, 128), torch.bfloat16)
BACK = Stand((9, HKV, PS, 128), torch.bfloat16)


def q8_calls(cache):
    return [lambda: cache.append(NEW, NEW, START, 3, stream=0),
            lambda: cache.attend(Q, START, 3, 1.0, stream=0),
            lambda: cache.read_back(BACK, BACK, stream=0),
            lambda: cache.read_back(BACK, BACK, Stand((B, PAGES), torch.int32), stream=0)]


@pytest.mark.parametrize("name,bad", BAD)
def test_q8_cache(name, bad):
    """Each call looks: the attributes can be set after the constructor has run."""
    cache = pipeline.Q8Cache(SHAPE, device="cpu", **good())
    setattr(cache, name, bad)
    for call in q8_calls(cache):
        with pytest.raises(ValueError, match=name + ": a contiguous"):
            call()


def test_q8_cache_takes_good_ones():
    for call in q8_calls(pipeline.Q8Cache(SHAPE, device="cpu", **good())):
        with pytest.raises(AssertionError, match="the library was called"):
            call()


@pytest.mark.parametrize("name,bad", BAD)
def test_layer(name, bad):
    layer = types.SimpleNamespace(shape=SHAPE, _st=lambda s: s, **good())
    with pytest.raises(AssertionError, match="the library was called"):
        pipeline.DecodeLayer.chunk_attn(layer, Q, START, 3, stream=0)
    setattr(layer, name, bad)
    with pytest.raises(ValueError, match=name + ": a contiguous"):
        pipeline.DecodeLayer.chunk_attn(layer, Q, START, 3, stream=0)


def test_tensors_of_another_device():
    """The kernels run on the current device."""
    away = Stand((3, HQ, 128), torch.bfloat16, "cuda:1")
    with pytest.raises(ValueError, match="q: a contiguous"):
        pipeline.Q8Cache(SHAPE, device="cpu", **good()).attend(away, START, 3, 1.0, stream=0)
