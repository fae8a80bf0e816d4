"""Rotary refuses frequencies that the kernels do not turn by."""
import math

import pytest
import torch

from offloaded_kv_cache_gb300.pipeline import Rotary


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 2.0 ** 54, -2.0 ** 54, 1e300])
@pytest.mark.parametrize("at", [0, 7])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_refused(bad, at, dtype):
    if dtype == torch.float32 and bad == 1e300:
        bad = 1e38
    freq = torch.ones(8, dtype=dtype)
    freq[at] = bad
    with pytest.raises(ValueError, match="2\\^54"):
        Rotary(16, freq=freq, device="cpu")


def test_taken():
    freq = torch.tensor([0.0, -0.0, 1e-300, math.nextafter(2.0 ** 54, 0), -math.nextafter(2.0 ** 54, 0), 1, 2, 3],
                        dtype=torch.float64)
    assert torch.equal(Rotary(16, freq=freq, device="cpu").freq, freq)
    assert Rotary(16, base=1e-9, stretch=1e9, device="cpu").freq.isfinite().all()
