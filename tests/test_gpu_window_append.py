"""The page window while the cache behind it grows: tokens appended by chunks across page
borders, one by one while the last page is not selected, after lengths were taken back, and
in a captured graph.  The window's output is the sparse attention's over the same selection
(ATOL of the fp64 oracle), its slots hold the cache's tokens bit for bit, and kv_window_trim's
maps are those of its definition."""
import numpy as np
import pytest
import torch

import oracle
from chunk_util import D
from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import workloads as W
from offloaded_kv_cache_gb300.pipeline import TORCH_DTYPE, DecodeLayer, torch_to_bits
from parity_util import ATOL

pytestmark = pytest.mark.gpu

PS, K = 16, 3


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_debug_config(-1, 2_000_000_000)
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


class Growing:
    """A layer with a window, and what its steps have to give."""

    def __init__(self, dtype="bf16", loc="host", lens=(5 * PS + 10, 3 * PS + 1), hq=8, seed=0):
        spec = W.tiny_spec(dtype=dtype, batch=2, hq=hq, hkv=2, context=PS * 20, ps=PS, index=130 + seed)
        self.wl = W.generate(spec, context_lens=[PS * 20] * 2)  # (every page has an entry)
        self.layer = DecodeLayer(self.wl, kv_loc=loc, topk=K)
        self.layer.context_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.layer.enable_window(4 * (hq // 2) * K)
        self.g = torch.Generator().manual_seed(seed)
        self.dtype, self.spec = dtype, spec

    def rows(self, n):
        return torch.randn(n, self.spec.num_kv_heads, D, generator=self.g).to(TORCH_DTYPE[self.dtype]).cuda()

    def chunk(self, *news):
        start = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device="cuda")
        self.layer.append_chunk(self.rows(sum(news)), self.rows(sum(news)), start, max(news))

    def token(self):
        self.layer.append(self.rows(2), self.rows(2))

    def step(self, *pages):
        """A window step whose heads select the given pages of each sequence."""
        layer, s = self.layer, self.spec
        idx = np.full((s.batch, s.num_q_heads, K), -1, dtype=np.int32)
        for b, p in enumerate(pages):
            idx[b, :, :len(p)] = sorted(p)
        scores = torch.randn(s.batch, s.num_q_heads, s.max_pages, generator=self.g).cuda()
        layer.window_attn(indices=torch.from_numpy(idx).cuda(), scores=scores)
        torch.cuda.synchronize()
        lens = layer.context_lens.cpu().numpy()
        kc, vc = (torch_to_bits(x).view(self.wl.k_cache.dtype) for x in (layer.k_cache, layer.v_cache))
        want = oracle.attention(self.dtype, self.wl.q, kc, vc, self.wl.block_table, lens,
                                self.wl.scale, indices=idx)
        assert np.abs(layer.out.cpu().numpy() - want).max() <= ATOL[self.dtype]
        # every page the step needed is in its slot, token by token
        wk, wv = torch_to_bits(layer.win_k), torch_to_bits(layer.win_v)
        kc, vc = kc.view(wk.dtype), vc.view(wv.dtype)
        at, C = layer.win_page_slot.cpu().numpy(), layer.window.cache_pages
        for b, p in enumerate(pages):
            for kvh in range(s.num_kv_heads):
                for page in p:
                    n, slot = min(PS, lens[b] - page * PS), at[b, kvh, page]
                    ph = self.wl.block_table[b, page]
                    assert slot >= 0 and np.array_equal(wk[b * C + slot, kvh, :n], kc[ph, kvh, :n])
                    assert np.array_equal(wv[b * C + slot, kvh, :n], vc[ph, kvh, :n])


@pytest.mark.parametrize("loc", ["host", "hbm"])
@pytest.mark.parametrize("dtype,hq", [("bf16", 8), ("f16", 4), ("f32", 2), ("bf16", 32)])
def test_a_chunk_across_a_page_border(dtype, hq, loc):
    """The page that was partly filled when it was copied is an inner page afterwards."""
    w = Growing(dtype, loc, hq=hq)
    w.step([0, 2, 5], [0, 3])
    w.chunk(10, 40)
    w.step([0, 5, 6], [3, 4, 5])
    w.chunk(1, 33)
    w.step([4, 5, 6], [4, 5, 6])


def test_single_tokens_while_the_last_page_is_not_selected():
    w = Growing()
    w.step([1, 5], [2, 3])
    for _ in range(2 * PS):
        w.token()
        w.step([0, 1, 2], [0, 1])
    w.step([5, 6, 7], [3, 4, 5])


def test_several_tokens_between_two_steps():
    w = Growing()
    w.step([5], [3])
    for _ in range(PS + 2):
        w.token()
    w.step([4, 5, 6], [2, 3, 4])


def test_lengths_taken_back():
    """Proposed tokens that were not taken: others follow at their positions, pages on."""
    w = Growing(lens=(5 * PS + 3, 4 * PS))
    w.chunk(40, 33)
    w.step([5, 6, 7], [4, 5, 6])
    w.layer.context_lens.copy_(torch.tensor([5 * PS + 5, 4 * PS], dtype=torch.int32))
    w.chunk(60, 60)
    w.step([5, 6, 7], [4, 5, 6])


def test_a_captured_graph():
    w = Growing(lens=(5 * PS + 10, 3 * PS))
    w.step([4, 5], [2])
    k, v = w.rows(2), w.rows(2)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        w.layer.append(k, v, stream=st)
    for i in range(PS):
        k.copy_(w.rows(2))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        if i % 3 == 0:
            w.step([0, 1, 4], [0, 2])
    assert w.layer.context_lens.tolist() == [6 * PS + 10, 4 * PS]
    w.step([4, 5, 6], [2, 3])


def test_trim_is_its_definition():
    w = Growing()
    layer, s, C = w.layer, w.spec, 24
    rng = np.random.default_rng(5)
    for lens in ([0, PS], [PS - 1, 20 * PS], [7 * PS, 7 * PS + 1], [-1, 5], [3 * PS, 20 * PS + 1]):
        slot = np.full((2, 2, C), -1, dtype=np.int32)
        page = np.full((2, 2, s.max_pages), -1, dtype=np.int32)
        for g in np.ndindex(2, 2):
            slots = rng.permutation(C)[:12]
            pages = rng.permutation(20)[:12]
            slot[g][slots], page[g][pages] = pages, slots
        d_slot, d_page = torch.from_numpy(slot).cuda(), torch.from_numpy(page).cuda()
        ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
        win = kv.make_window(C, layer.win_k, layer.win_v, d_slot, d_page)
        kv.kv_window_trim(layer.shape, win, ctx, torch.cuda.current_stream())
        bad = [not 0 <= n <= s.max_pages * PS for n in lens]
        assert kv.kv_device_status() == (kv.KV_ERR_BOUNDS if any(bad) else kv.KV_OK)
        for b in range(2):
            if bad[b]:
                continue
            for h in range(2):
                for p in range(s.max_pages):
                    if (p + 1) * PS > lens[b] and page[b, h, p] >= 0:
                        slot[b, h, page[b, h, p]] = -1
                        page[b, h, p] = -1
        assert np.array_equal(d_slot.cpu().numpy(), slot) and np.array_equal(d_page.cpu().numpy(), page)
