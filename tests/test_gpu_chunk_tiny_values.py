"""Values of the 8-bit cache near the least that its format holds: their scales enter the
few-row kernel's weights, and what a sequence's tokens add up to must not depend on which
warp had the largest score."""
import pytest
import torch

from chunk_util import Problem, check
from offloaded_kv_cache_gb300 import kvsparse as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(kvlib):
    kv.kv_device_status()
    yield
    assert kv.kv_device_status() == kv.KV_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("byte", [17, 20, 60])
@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("length", [700, 9000])
def test_tiny_values(dtype, byte, n, length):
    """One token with a weight e^7.5 times every other's, up to thousands of those."""
    p = Problem(dtype, 4, 1, 16, [length], [n], q8=True, scale=1.0, seed=n)
    p.q = torch.zeros_like(p.q)
    p.q[:, :, 0] = 1
    # keys: 0 but for one of 7.5; values: equal scales, codes as drawn
    zero, tall = 0x00, int((torch.tensor([7.5]).to(torch.float8_e4m3fn).view(torch.uint8))[0])
    for j in range(length):
        ph, at = p.table[0, j // 16], j % 16
        p.code["k"][ph, :, at] = zero
        p.scale8["k"][ph, :, at] = 127
        p.scale8["v"][ph, :, at] = byte
    p.code["k"][p.table[0, 3 // 16], :, 3, 0] = tall
    p.upload()
    p.attend()
    torch.cuda.synchronize()
    want, tol = p.expected()
    # (a subnormal bf16 or fp32 result is off by half its last place)
    check(p.d_out, want, tol + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -149) * (want != 7))
