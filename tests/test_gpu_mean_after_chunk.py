"""The mean-key index after chunks and after several appends: bit for bit the index built
anew, scores and all."""
import pytest
import torch

from chunk_util import D
from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import workloads as W
from offloaded_kv_cache_gb300.pipeline import TORCH_DTYPE, DecodeLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("how", ["chunk", "tokens", "graph"])
def test_index_follows(dtype, how):
    ps = 16
    spec = W.tiny_spec(dtype=dtype, batch=2, hq=8, hkv=2, context=ps * 20, ps=ps, index=140)
    layer = DecodeLayer(W.generate(spec, context_lens=[ps * 20] * 2))
    layer.context_lens.copy_(torch.tensor([5 * ps + 10, 3 * ps]))
    layer.build_mean_index()
    g = torch.Generator().manual_seed(3)
    new = lambda n: torch.randn(n, 2, D, generator=g).to(TORCH_DTYPE[dtype]).cuda()  # noqa: E731
    start = torch.tensor([0, 10, 50], dtype=torch.int32, device="cuda")
    if how == "chunk":
        layer.append_chunk(new(50), new(50), start, 40)
    elif how == "tokens":
        for _ in range(ps):
            layer.append(new(2), new(2))
    else:
        k, v, st = new(50), new(50), torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            layer.append_chunk(k, v, start, 40)
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            layer.build_mean_index(last_only=True)
    layer.build_mean_index(last_only=True)
    got = layer.mean.clone()
    layer.mean.zero_()
    layer.build_mean_index()
    used = layer.mean != 0
    assert torch.equal(got[used], layer.mean[used]) and used.any()
