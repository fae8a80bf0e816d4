"""Rotary positions and the 4-bit format from their definitions in 64 bits (numpy and
torch on the CPU; nothing of the library's own), and batches over a 4-bit cache."""
import math

import numpy as np
import torch

from chunk_util import D, E4M3, LEAST, TORCH, Problem
from offloaded_kv_cache_gb300 import kvsparse as kv

STEPS = E4M3[:127]  # 0 .. 448


# --- rotary positions ----------------------------------------------------------------
def turned(x, positions, freq, interleaved=False, scale=1.0):
    """x [rows, heads, 128] in 64 bits, turned; freq [rotary_dim / 2], positions [rows]."""
    y = x.double().clone()
    half = len(freq)
    j = torch.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    angle = positions.double()[:, None, None] * freq
    c, s = scale * torch.cos(angle), scale * torch.sin(angle)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    return y


def turned_tolerance(x, dtype, half, interleaved=False, scale=1.0, positions=None, freq=None):
    """What the arithmetic may be off by: the result is rounded once (half an eps of it);
    sine and cosine are fp32 values of an angle rounded in fp32 within an eighth of a
    turn (2^-24 of it and 2^-33 turns; their own error is 2 ulp, 2^-22), multiplied by the
    scale and summed in fp32 (3 * 2^-24): 2^-21 of |a| + |b| in all.  The definition above
    multiplies position and frequency in 64 bits, 2^-53 of the angle, as the fraction of a
    turn is kept."""
    y = x.double().abs()
    j = torch.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    far = 0.0
    if positions is not None:
        far = 2.0 ** -51 * (positions.double().abs()[:, None, None] * freq.abs())
    size = y[..., a] + y[..., b]
    tol = torch.zeros_like(y)
    t = abs(scale) * size * (2.0 ** -21 + far)
    tol[..., a], tol[..., b] = t, t
    eps = torch.finfo(TORCH[dtype]).eps / 2
    least = 2.0 ** -25 if dtype == "f16" else 0.0  # half of the least f16
    turned_up = torch.zeros_like(y)
    turned_up[..., a], turned_up[..., b] = abs(scale) * size, abs(scale) * size
    return tol + eps * (turned_up + tol) + least * (turned_up > 0)


# --- the 4-bit format -------------------------------------------------------------------
def quantise4(x, dtype):
    """(bytes [..., 64], scale codes [..., 8], power bytes [...]) of vectors x [..., 128]
    (numpy, any float type), in 64 bits, by comparisons."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(-1)
    x0 = np.where(finite[..., None], x, 0.0)
    top = np.abs(x0).max(-1)
    e = np.full(top.shape, LEAST[dtype])
    for _ in range(4 - LEAST[dtype]):
        e = np.where((top > 3136.0 * 2.0 ** e) & (e < 4), e + 1, e)
    y = (x0 * 2.0 ** -e[..., None].astype(np.float64)).reshape(*x.shape[:-1], 8, 16)
    scale = np.minimum(np.searchsorted(7 * STEPS, np.abs(y).max(-1), side="left"), 126)
    s = STEPS[scale][..., None]
    # floor(y / s + 1/2): the largest c with (2 c - 1) s <= 2 y
    c = np.full(y.shape, -8)
    for k in range(-7, 8):
        c = np.where((2 * k - 1) * s <= 2 * y, k, c)
    c = np.where(s == 0, 0, np.clip(c, -7, 7)).reshape(x.shape) + 8
    c = np.where(finite[..., None], c, 8).astype(np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4),
            np.where(finite[..., None], scale, 0).astype(np.uint8),
            np.where(finite, e + 127, 255).astype(np.uint8))


def restore4(code, scale, power):
    c = np.stack([code & 15, code >> 4], -1).reshape(*code.shape[:-1], D).astype(np.float64) - 8
    up = np.where(power == 255, np.nan, 2.0 ** (power.astype(np.float64) - 127))
    return c * np.repeat(E4M3[scale] * up[..., None], 16, -1)


class Problem4(Problem):
    """A batch over a 4-bit cache.  Slots no token owns hold NaN (power 255, scales NaN)."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.four = {}
        hole = ~self.owned[:, None].expand(-1, self.hkv, -1).numpy()
        for name in "kv":
            x = getattr(self, name).double().nan_to_num(nan=0.0).numpy()
            c, s, p = quantise4(x, self.dtype)
            c[hole], s[hole], p[hole] = 0xFF, 0x7F, 255
            self.four[name] = [torch.from_numpy(t) for t in (c, s, p)]

    def upload(self, total=None, max_new=None):
        super().upload(total, max_new)
        self.d_four = {n: [self.put(t, True) for t in self.four[n]] for n in "kv"}
        self.use(self.d_four)
        return self

    def use(self, four):
        (kc, ks, kp), (vc, vs, vp) = four["k"], four["v"]
        self.cache = kv.make_q4_cache(kc, vc, ks, vs, kp, vp)
        self.ws = torch.full((max(16, kv.kv_q4_chunk_workspace_bytes(self.shape, self.chunk)),), 255,
                             dtype=torch.uint8, device=self.device)  # NaN patterns

    def attend(self, stream=None, out=None, ws=None, check=True):
        out = self.d_out if out is None else out
        ws = self.ws if ws is None else ws
        st = torch.cuda.current_stream() if stream is None else stream
        return kv.kv_q4_chunk_attn(self.shape, self.chunk, self.d_q, self.cache, self.d_table,
                                   self.d_lens, self.scale, out, ws, ws.numel(), st, check=check)

    def tokens(self, name, b, h):
        at = torch.arange(self.lens[b])
        page = self.table[b].long()[at // self.ps]
        ok = (page >= 0) & (page < self.pages)
        page = torch.where(ok, page, 0)
        x = restore4(*(t[page, h, at % self.ps].numpy() for t in self.four[name]))
        return torch.from_numpy(x), ok

    def expected(self):
        """Problem.expected(), whose tolerance is relative to the sum of w |v|: here a channel
        may be 0 in every vector that weighs anything, and what is left is below the weights'
        own range.  Weights are at most 1 beside a sum of at least 1.  In fp32 those below
        2^-126 are 0; those that enter a product as f16 (as one or two terms, 2^7 up, times
        the vector's power 2^e relative to the row's largest w 2^e) are off by half of the
        least f16, 2^-25, so by 2^-32 of it, times |c s| <= 3136: 2^-32 * 3136 * 2^e a token."""
        want, tol = super().expected()
        power = self.four["v"][2]
        used = power[power != 255]
        top = 2.0 ** (int(used.max()) - 127) if used.numel() else 0.0
        more = max(self.lens) * (2.0 ** -32 + 2.0 ** -126) * 3136 * top
        owned = torch.zeros(self.total, dtype=torch.bool)
        for b, n in enumerate(self.news):
            owned[self.start[b]:self.start[b] + n] = True
        return want, tol + more * owned[:, None, None]

    def set_nan(self, name, page, h, slot):
        c, s, p = self.four[name]
        c[page, h, slot], s[page, h, slot], p[page, h, slot] = 0x88, 0, 255


def frequencies(rotary_dim, base=10000.0):
    return base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)


def near_2pi(freq, positions):
    """Angles of positions * freq within one turn, by integers: for positions so far that
    64 bits lose the product's fraction."""
    from fractions import Fraction
    # 2 pi by Machin's formula
    one = 1 << 260

    def arctan_inverse(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (term if k % 2 == 0 else -term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total

    two_pi = Fraction(2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)
    out = torch.empty(len(positions), len(freq), dtype=torch.float64)
    for i, t in enumerate(positions):
        for j, f in enumerate(freq):
            turns = Fraction(float(f)) * int(t) / two_pi
            out[i, j] = float((turns - math.floor(turns)) * two_pi)
    return out
