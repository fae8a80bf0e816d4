"""A layer's chunks and single tokens, turned and appended, against the fp64 oracle over the
cache that they leave: the chunk attention of the last tokens and the sparse step over every
page through the index kept, with tolerances from the arithmetic."""
import numpy as np
import pytest
import torch

import oracle
from chunk_util import D, TORCH
from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import workloads as W
from offloaded_kv_cache_gb300.pipeline import DecodeLayer, Rotary, torch_to_bits
from parity_util import ATOL

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_debug_config(-1, 2_000_000_000)
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


@pytest.mark.parametrize("loc", ["hbm", "host"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_against_the_oracle(dtype, loc):
    spec = W.tiny_spec(dtype=dtype, batch=2, hq=8, hkv=2, context=208, ps=16, topk=13, index=6)
    wl = W.generate(spec, context_lens=[208, 208])
    layer = DecodeLayer(wl, kv_loc=loc)
    layer.context_lens.zero_()
    rotary = Rotary(64, base=500000.0, stretch=4.0)
    t, g = TORCH[dtype], torch.Generator().manual_seed(1)
    for n in ([150, 120], [5, 0], [40, 31], [1, 1], [1, 1]):
        start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        k, v = (torch.randn(sum(n), 2, D, generator=g).to(t).cuda() for _ in "kv")
        q = torch.randn(sum(n), 8, D, generator=g).to(t).cuda()
        q = layer.append_chunk(k, v, start, max(n), rotary, q)
        out = layer.chunk_attn(q, start, max(n))
    layer.q.copy_(q)
    layer.sparse_step()
    torch.cuda.synchronize()
    bits = lambda x: torch_to_bits(x).view(wl.q.dtype)  # noqa: E731
    kc, vc = (bits(x).reshape(wl.k_cache.shape) for x in (layer.k_cache, layer.v_cache))
    lens = layer.context_lens.cpu().numpy()
    assert lens.tolist() == [197, 153]
    want = oracle.attention(dtype, bits(q).reshape(wl.q.shape), kc, vc, wl.block_table, lens, wl.scale)
    assert np.abs(layer.out.cpu().numpy() - want).max() <= ATOL[dtype]
    # the chunk's, as in chunk_util.expected(): the result rounded once; of sum w |v| <= max |v|,
    # half a step of dtype for the weights (16-bit types; f16 ones below its range after a shift of
    # 2^7 by 2^-32 each), and the fp32 arithmetic: scores of 128 terms, scaled in fp32, ex2, the sums
    half = torch.finfo(t).eps / 2
    used = [int(p) for b in range(2) for p in wl.block_table[b, :-(-int(lens[b]) // 16)]]
    top = max(float(layer.v_cache[p].float().abs().max()) for p in used)
    most = max(float(layer.k_cache[p].double().abs().sum(-1).max()) for p in used)
    dz = float(q.double().abs().max()) * most * wl.scale
    rel = (half if dtype != "f32" else 0) + dz * (2 * D * 2.0 ** -24 + 2.0 ** -21) + 2.0 ** -21 \
        + 208 * (2.0 ** -24 + 2.0 ** -32)
    assert (np.abs(out.double().cpu().numpy() - want) <= half * np.abs(want) + rel * top).all()
