"""Appends whose q_start is out of order, out of range or longer than the launch was sized for:
the sequences that it spoils are left whole (cache, rows, lengths, index), the others are stored,
turned and advanced; every byte of every output is looked at."""
import numpy as np
import pytest
import torch

import test_gpu_q4
import test_gpu_q8
from chunk_util import quantise
from more_util import quantise4, turned, turned_tolerance
from offloaded_kv_cache_gb300 import kvsparse as kv
from test_gpu_rope import Chunk, near

pytestmark = pytest.mark.gpu

BEFORE, NEWS, MOST = [0, 3, 2, 4], [45, 45, 45, 45], 40
STARTS = [[0, 41, 45, 50, 55], [0, 40, 30, 50, 71], [-1, 40, 60, 66, 71], [0, 40, 60, 66, 183],
          [7, 7, 47, 48, 182], [0, 1 << 30, 40, 41, 42], [-(1 << 31), -1, 0, 40, 41], [182, 182, 182, 182, 183],
          [-40, 0, 0, 1, (1 << 31) - 1]]


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


def taken(start, total, cap):
    """(row, sequence, position) of every token that is stored, and the lengths after."""
    rows, lens = [], list(BEFORE)
    for b, (q0, q1) in enumerate(zip(start, start[1:])):
        if q0 < 0 or q1 < q0 or q1 > total or q1 - q0 > MOST or BEFORE[b] + q1 - q0 > cap:
            continue
        rows += [(r, b, BEFORE[b] + r - q0) for r in range(q0, q1)]
        lens[b] += q1 - q0
    return rows, lens


@pytest.mark.parametrize("index", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_append(dtype, in_place, index):
    for start in STARTS:
        c = Chunk(dtype, 4, 2, 16, BEFORE, NEWS, 64, max_new=MOST)
        p = c.p
        rows, lens = taken(start, p.total, p.max_pages * 16)
        mm = c.index() if index else None
        anew = mm.clone() if index else None
        p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        out = c.ctx if in_place else torch.full((4,), -9, dtype=torch.int32, device="cuda")
        c.put(out, mm)
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
        assert out.tolist() == lens
        # (behind a start out of order two sequences may own a row: each stores its key where it
        # is, and the row of q is turned for one of them)
        owners = np.bincount([r for r, _, _ in rows], minlength=p.total)
        mine, once = torch.from_numpy(owners > 0), torch.from_numpy(owners < 2)

        def check_rows(x, out, lens):
            at = torch.zeros(p.total, dtype=torch.int64)
            for r, b, pos in rows:
                at[r] = pos - BEFORE[b] + lens[b]
            want, tol = turned(x, at, c.freq), turned_tolerance(x, dtype, 32, False, 1.0, at, c.freq)
            want[~mine], tol[~mine] = 7.0, 0.0
            near(out[once], want[once], tol[once])

        check_rows(c.q, c.q_out, BEFORE)
        row, seq, pos = (torch.tensor(x, dtype=torch.int64) for x in (zip(*rows) if rows else ((), (), ())))
        page = p.table[seq, pos // 16].long()
        want_k, tol_k, want_v = p.k.double(), torch.zeros_like(p.k, dtype=torch.float64), p.v.double()
        want_k[page, :, pos % 16] = turned(c.k[row], pos, c.freq)
        tol_k[page, :, pos % 16] = turned_tolerance(c.k[row], dtype, 32, False, 1.0, pos, c.freq)
        want_v[page, :, pos % 16] = c.v[row].double()
        near(p.d_k, want_k, tol_k)
        assert torch.equal(p.d_v.double().cpu(), want_v)
        if index:
            c.build(anew, torch.tensor(lens, dtype=torch.int32, device="cuda"))
            kv.kv_device_status()  # (the build takes lengths from 1 on)
            assert torch.equal(mm, anew)
        # the rows alone, at the positions behind the lengths now
        c.turn()
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
        for x, got in ((c.q, c.q_out), (c.k, c.k_out)):
            check_rows(x, got, lens if in_place else BEFORE)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_quantised_appends(dtype, in_place, bits):
    for start in STARTS:
        a = (test_gpu_q4 if bits == 4 else test_gpu_q8).Append(dtype, 2, 16, BEFORE, NEWS, max_new=MOST)
        p = a.p
        rows, lens = taken(start, p.total, p.max_pages * 16)
        p.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        out = a.before if in_place else torch.full((4,), -9, dtype=torch.int32, device="cuda")
        got = a.got if bits == 4 else {n: (a.code[n], a.scale[n]) for n in "kv"}
        want = {n: [x.cpu().numpy().copy() for x in got[n]] for n in "kv"}
        a.run(out)
        assert kv.kv_device_status() == kv.KV_ERR_BOUNDS
        assert out.tolist() == lens
        for n in "kv":
            new = (quantise4 if bits == 4 else quantise)(a.new[n].double().numpy(), dtype)
            for r, b, pos in rows:
                ph = int(p.table[b, pos // 16])
                for w, x in zip(want[n], new):
                    w[ph, :, pos % 16] = x[r]
            for x, w in zip(got[n], want[n]):
                assert np.array_equal(x.cpu().numpy(), w)
