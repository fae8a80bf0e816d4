"""Rotary positions and the 4-bit cache without a GPU: struct layouts, refused arguments,
workspace sizes, the pipeline's checks, and the definitions that the GPU tests use."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

from chunk_util import TORCH
from more_util import STEPS, frequencies, near_2pi, quantise4, restore4, turned
from offloaded_kv_cache_gb300 import kvsparse as kv
from offloaded_kv_cache_gb300 import pipeline
from test_chunk_pipeline_cpu import BACK, BAD, NEW, Q, SHAPE, START, Stand, good

FAKE = 0x10000  # 16-byte aligned address that is never dereferenced
FAR = 1 << 24   # apart from FAKE by more than any array below
CACHE = kv.make_q4_cache(*[FAKE] * 6)


def shape(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                max_pages_per_seq=4, num_phys_pages=8, dtype="bf16", kv_loc="hbm")
    base.update(kw)
    return kv.make_shape(**base)


def chunk(**kw):
    base = dict(q_start=FAKE, total_q=10, max_q_len=5, window=0)
    base.update(kw)
    return kv.make_chunk(**base)


def rope(**kw):
    base = dict(freq=FAKE, rotary_dim=128, interleaved=False, scale=1.0, positions=None)
    base.update(kw)
    return kv.make_rope(**base)


# the arguments were taken (no device here, or no such memory there)
NO_DEVICE = (kv.KV_ERR_CUDA, kv.KV_ERR_LOCATION)


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("calls with made-up addresses that every check lets pass")


def turn(s=None, c=None, r=None, **kw):
    a = dict(q=FAKE, q_out=FAKE, k=FAKE + FAR, k_out=FAKE + 2 * FAR, ctx=FAKE)
    a.update(kw)
    return kv.kv_rope(s or shape(), c or chunk(), r or rope(), a["q"], a["q_out"], a["k"], a["k_out"],
                      a["ctx"], check=False)


def put(s=None, c=None, r=0, **kw):
    a = dict(q=FAKE, q_out=FAKE, k=FAKE + FAR, v=FAKE + 2 * FAR, kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE,
             ctx_out=None, mm=None)
    a.update(kw)
    return kv.kv_rope_append(s or shape(), c or chunk(), rope() if r == 0 else r, a["q"], a["q_out"],
                             a["k"], a["v"], a["kc"], a["vc"], a["bt"], a["ctx"], a["ctx_out"], a["mm"],
                             check=False)


def four(s, c, **kw):
    """Status of every call over the 4-bit cache, in a fixed order."""
    a = dict(q=FAKE, cache=CACHE, bt=FAKE, ctx=FAKE, scale=0.1, out=FAKE, ws=FAKE, nws=1 << 40)
    a.update(kw)
    return (kv.kv_q4_chunk_attn(s, c, a["q"], a["cache"], a["bt"], a["ctx"], a["scale"], a["out"],
                                a["ws"], a["nws"], check=False),
            kv.kv_q4_append(s, c, a["q"], a["out"], a["cache"], a["bt"], a["ctx"], None, check=False))


def test_struct_layouts():
    assert ctypes.sizeof(kv.kv_rope_plan) == 32 and kv.kv_rope_plan.scale.offset == 24
    assert ctypes.sizeof(kv.kv_q4_cache) == 48


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), kv.KV_ERR_UNSUPPORTED), (dict(page_size=48), kv.KV_ERR_UNSUPPORTED),
    (dict(dtype=7), kv.KV_ERR_UNSUPPORTED), (dict(num_q_heads=7), kv.KV_ERR_INVALID_ARG),
    (dict(batch=0), kv.KV_ERR_INVALID_ARG), (dict(kv_loc=5), kv.KV_ERR_INVALID_ARG)])
def test_bad_shapes_are_refused(kvlib, kw, code):
    s, c = shape(**kw), chunk()
    assert turn(s) == put(s) == code and four(s, c) == (code,) * 2
    assert kv.kv_q4_read(s, CACHE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, check=False) == code
    assert kv.kv_q4_chunk_workspace_bytes(s, c) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q_start=None), kv.KV_ERR_INVALID_ARG), (dict(q_start=FAKE + 2), kv.KV_ERR_INVALID_ARG),
    (dict(total_q=0), kv.KV_ERR_INVALID_ARG), (dict(max_q_len=0), kv.KV_ERR_INVALID_ARG),
    (dict(window=-1), kv.KV_ERR_INVALID_ARG), (dict(total_q=1 << 30), kv.KV_ERR_UNSUPPORTED)])
def test_bad_chunks_are_refused(kvlib, kw, code):
    c = chunk(**kw)
    assert turn(c=c) == put(c=c) == code and four(shape(), c) == (code,) * 2
    assert kv.kv_q4_chunk_workspace_bytes(shape(), c) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(freq=None), kv.KV_ERR_INVALID_ARG), (dict(freq=FAKE + 4), kv.KV_ERR_INVALID_ARG),
    (dict(positions=FAKE + 2), kv.KV_ERR_INVALID_ARG), (dict(scale=math.nan), kv.KV_ERR_INVALID_ARG),
    (dict(scale=math.inf), kv.KV_ERR_INVALID_ARG), (dict(interleaved=2), kv.KV_ERR_INVALID_ARG),
    (dict(rotary_dim=0), kv.KV_ERR_UNSUPPORTED), (dict(rotary_dim=12), kv.KV_ERR_UNSUPPORTED),
    (dict(rotary_dim=136), kv.KV_ERR_UNSUPPORTED), (dict(rotary_dim=-8), kv.KV_ERR_UNSUPPORTED)])
def test_bad_rotary_plans_are_refused(kvlib, kw, code):
    r = rope(**kw)
    assert turn(r=r) == put(r=r) == code
    r = rope()
    r.reserved = 1
    assert turn(r=r) == put(r=r) == kv.KV_ERR_INVALID_ARG


BYTES_Q, BYTES_K = 10 * 8 * 128 * 2, 10 * 2 * 128 * 2


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q_out=None), dict(q=FAKE + 8), dict(q_out=FAKE + BYTES_Q - 16),
    dict(k=FAKE + 4 + FAR), dict(k_out=None), dict(k_out=FAKE + FAR + 16),
    dict(q=None, q_out=None, k=None, k_out=None), dict(k_out=FAKE), dict(q_out=FAKE + FAR),
    dict(ctx=FAKE + 2), dict(ctx=None)])
def test_rows_that_do_not_fit_are_refused(kvlib, kw):
    assert turn(**kw) == kv.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(), dict(k=None, k_out=None), dict(q=None, q_out=None), dict(k_out=FAKE + FAR),
    dict(q_out=FAKE + BYTES_Q), dict(k_out=FAKE + FAR - BYTES_K),
    dict(r=rope(positions=FAKE), ctx=None)])
def test_rows_that_fit_are_taken(kvlib, no_gpu, kw):
    assert turn(**kw) in NO_DEVICE


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q_out=None), dict(r=None), dict(k=None), dict(v=FAKE + 8), dict(bt=None),
    dict(ctx=FAKE + 1), dict(ctx_out=FAKE + 4), dict(ctx_out=FAKE + 2), dict(mm=FAKE + 8),
    dict(q_out=FAKE + FAR), dict(q_out=FAKE + 2 * FAR - 16), dict(q_out=FAKE + 16)])
def test_appends_that_do_not_fit_are_refused(kvlib, kw):
    assert put(**kw) == kv.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(), dict(q=None, q_out=None), dict(r=None, q=None, q_out=None), dict(ctx_out=FAKE),
    dict(ctx_out=FAKE + 8), dict(mm=FAKE)])
def test_appends_that_fit_are_taken(kvlib, no_gpu, kw):
    assert put(**kw) in NO_DEVICE


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=FAKE + 8), dict(out=None), dict(bt=FAKE + 2),
                                dict(ctx=None)])
def test_bad_pointers_are_refused(kvlib, kw):
    assert four(shape(), chunk(), **kw) == (kv.KV_ERR_INVALID_ARG,) * 2


def test_bad_reads_are_refused(kvlib):
    read = lambda **kw: kv.kv_q4_read(*[kw.get(k, v) for k, v in dict(  # noqa: E731
        shape=shape(), cache=CACHE, bt=FAKE, ctx=FAKE, to=FAKE, pages=4, k=FAKE, v=FAKE).items()],
        check=False)
    for kw in (dict(k=None), dict(v=FAKE + 4), dict(to=None), dict(pages=0), dict(ctx=FAKE + 1)):
        assert read(**kw) == kv.KV_ERR_INVALID_ARG
    assert read(pages=1 << 40) == kv.KV_ERR_UNSUPPORTED
    wide = shape(batch=512, num_q_heads=8, num_kv_heads=8, max_pages_per_seq=1 << 20)
    assert read(shape=wide) == kv.KV_ERR_UNSUPPORTED
    for scale in (math.nan, math.inf):
        assert four(shape(), chunk(), scale=scale)[0] == kv.KV_ERR_INVALID_ARG


def test_launches_that_do_not_count_in_an_int_are_refused(kvlib):
    s = shape(batch=1 << 16, num_q_heads=64, num_kv_heads=64, max_pages_per_seq=1 << 12)
    c = chunk(total_q=1 << 24, max_q_len=1 << 24)
    q = dict(q=FAKE, q_out=FAKE, k=None, k_out=None)
    assert turn(s, c, **q) == kv.KV_ERR_UNSUPPORTED
    assert put(s, c, r=None, q=None, q_out=None, v=FAKE + (1 << 50)) == kv.KV_ERR_UNSUPPORTED


def test_workspace_sizes(kvlib):
    """Enough for the call, and bounded by the cache that passes through it."""
    assert 0 < kv.kv_q4_chunk_workspace_bytes(shape(), chunk()) < 1 << 24


# --- the definitions -----------------------------------------------------------------------
@pytest.mark.parametrize("dtype,least", [("f32", -110), ("bf16", -110), ("f16", -15)])
def test_quantiser_definition(dtype, least):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 128)) * 2.0 ** rng.integers(-30, 18, (200, 1))
    x = torch.from_numpy(x).to(TORCH[dtype]).double().numpy()
    x[0] = 0
    code, scale, power = quantise4(x, dtype)
    # (some are beyond f16: those vectors are NaN)
    finite = np.isfinite(x).all(-1)
    assert ((power == 255) == ~finite).all()
    x, code, scale, power = x[finite], code[finite], scale[finite], power[finite]
    e = power.astype(int) - 127
    assert (e >= least).all() and (e <= 4).all() and e[0] == least
    top = np.abs(x).max(-1)
    free = (e > least) & (e < 4)
    assert (top[free] <= 3136 * 2.0 ** e[free]).all() and (top[free] > 1568 * 2.0 ** e[free]).all()
    y = (x * 2.0 ** -e[:, None].astype(float)).reshape(-1, 8, 16)
    most, s = np.abs(y).max(-1), STEPS[scale]
    fits = most <= 3136
    assert (7 * s[fits] >= most[fits]).all()
    assert (7 * STEPS[np.maximum(scale, 1) - 1][fits & (scale > 0)] < most[fits & (scale > 0)]).all()
    # half a step of the group's scale
    err = np.abs(restore4(code, scale, power) - np.clip(x, -50176, 50176)).reshape(-1, 8, 16)
    assert (err <= 0.5 * s[..., None] * 2.0 ** e[:, None, None]).all()
    # the values are the type's own
    value = torch.from_numpy(restore4(code, scale, power))
    assert torch.equal(value.to(TORCH[dtype]).double(), value)


def test_ties_go_up():
    x = np.zeros((1, 128))
    x[0, :16] = [7, -7, 0.5, -0.5, 1.5, -1.5, 6.5, -6.5, 2.5, -2.5, 3.5, -3.5, 4.5, -4.5, 5.5, -5.5]
    code, scale, power = quantise4(x, "f32")
    got = restore4(code, scale, power)[0, :16]
    assert got.tolist() == [7, -7, 1, 0, 2, -1, 7, -6, 3, -2, 4, -3, 5, -4, 6, -5]


def test_turning_definition():
    x = torch.randn(3, 2, 128, dtype=torch.float64)
    f = frequencies(64)
    y = turned(x, torch.tensor([0, 5, 900]), f)
    assert torch.equal(y[0], x[0]) and torch.equal(y[..., 64:], x[..., 64:])
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
    back = turned(y, -torch.tensor([0, 5, 900]), f)
    assert torch.allclose(back, x)
    angle = near_2pi(f, torch.tensor([0, 5, 900]))
    want = (torch.tensor([0, 5, 900])[:, None] * f) % (2 * math.pi)
    assert torch.allclose(torch.cos(angle), torch.cos(want), atol=1e-12)
    assert torch.allclose(torch.sin(angle), torch.sin(want), atol=1e-12)


# --- the pipeline's checks -------------------------------------------------------------------
@pytest.fixture
def no_call(monkeypatch):
    def called(*_args, **_kw):
        raise AssertionError("the library was called")

    for name in ("kv_q4_append", "kv_q4_chunk_attn", "kv_q4_read", "kv_q4_chunk_workspace_bytes",
                 "kv_rope", "kv_rope_append", "make_chunk"):
        monkeypatch.setattr(kv, name, called)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def q4_calls(cache):
    return [lambda: cache.append(NEW, NEW, START, 3, stream=0),
            lambda: cache.attend(Q, START, 3, 1.0, stream=0),
            lambda: cache.read_back(BACK, BACK, stream=0),
            lambda: cache.read_back(BACK, BACK, Stand((2, 6), torch.int32), stream=0)]


@pytest.mark.parametrize("name,bad", BAD)
def test_q4_cache_looks_at_its_tensors(no_call, name, bad):
    cache = pipeline.Q4Cache(SHAPE, device="cpu", **good())
    for call in q4_calls(cache):
        with pytest.raises(AssertionError, match="the library was called"):
            call()
    setattr(cache, name, bad)
    for call in q4_calls(cache):
        with pytest.raises(ValueError, match=name + ": a contiguous"):
            call()


@pytest.mark.parametrize("kind", [pipeline.Q8Cache, pipeline.Q4Cache])
def test_caches_look_at_q_and_positions(no_call, kind):
    cache = kind(SHAPE, device="cpu", **good())
    for kw in (dict(q=Q), dict(positions=Stand((3,), torch.int32))):
        with pytest.raises(ValueError, match="rotary"):
            cache.append(NEW, NEW, START, 3, stream=0, **kw)
    with pytest.raises(ValueError, match="q: a contiguous"):
        cache.append(NEW, NEW, START, 3, stream=0, rotary=pipeline.Rotary(device="cpu"), q=NEW)


@pytest.mark.parametrize("name,bad", BAD)
def test_append_chunk_looks_at_its_tensors(no_call, name, bad):
    layer = types.SimpleNamespace(shape=SHAPE, _st=lambda s: s, **good())
    append = lambda **kw: pipeline.DecodeLayer.append_chunk(layer, NEW, NEW, START, 3, stream=0, **kw)  # noqa: E731
    with pytest.raises(AssertionError, match="the library was called"):
        append()
    for kw in (dict(q=Q), dict(positions=Stand((3,), torch.int32))):
        with pytest.raises(ValueError, match="rotary"):
            append(**kw)
    rotary = pipeline.Rotary(device="cpu")
    with pytest.raises(ValueError, match="q: a contiguous"):
        append(rotary=rotary, q=Stand((3, 8, 128), torch.float16))
    setattr(layer, name, bad)
    with pytest.raises(ValueError, match=name + ": a contiguous"):
        append()


def test_rotary_plan_looks_at_its_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    rotary = pipeline.Rotary(device="cpu")
    with pytest.raises(ValueError, match="freq: a contiguous CUDA"):
        rotary.plan(3)
    rotary.freq = Stand((64,), torch.float64)
    for bad in (Stand((3,), torch.int64), Stand((4,), torch.int32), Stand((3,), torch.int32, "cuda:1")):
        with pytest.raises(ValueError, match="positions: a contiguous CUDA"):
            rotary.plan(3, bad)


def test_rotary_frequencies():
    plain = pipeline.Rotary(64, base=500000.0, device="cpu")
    assert torch.equal(plain.freq, frequencies(64, 500000.0)) and plain.scale == 1.0
    far = pipeline.Rotary(64, base=500000.0, stretch=8.0, device="cpu")
    turns = plain.freq * 8192 / (2 * math.pi)
    assert torch.equal(far.freq[turns >= 32], plain.freq[turns >= 32])
    assert torch.allclose(far.freq[turns <= 1], plain.freq[turns <= 1] / 8)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (far.freq[between] < plain.freq[between]).all()
    assert (far.freq[between] > plain.freq[between] / 8).all()
    assert far.scale == pytest.approx(0.1 * math.log(8) + 1)
    even = pipeline.Rotary(64, stretch=4.0, fast=1.0, slow=1.0, scale=1.0, device="cpu")
    assert torch.allclose(even.freq, frequencies(64) / 4) and even.scale == 1.0
    own = pipeline.Rotary(16, freq=torch.arange(8), device="cpu")
    assert own.freq.dtype == torch.float64 and own.freq.tolist() == list(range(8))
    for kw in (dict(rotary_dim=12), dict(rotary_dim=0), dict(rotary_dim=256), dict(stretch=0.5),
               dict(base=0.0), dict(fast=1.0, slow=2.0), dict(freq=torch.zeros(3))):
        with pytest.raises(ValueError):
            pipeline.Rotary(**{"device": "cpu", **kw})
