"""Problems for the chunk operators and their definitions in 64 bits (numpy
and torch on the CPU; nothing of the library's own)."""
import math

import numpy as np
import torch

from offloaded_kv_cache_gb300 import kvsparse as kv

D = 128
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LEAST = {"f32": -110, "f16": -15, "bf16": -110}


# --- the 8-bit format ---------------------------------------------------------
def e4m3_values():
    """The value of each of the 256 codes, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if s else x)
    return v


E4M3 = e4m3_values()


def quantise(x, dtype):
    """(codes, scale bytes) of vectors x [..., 128] (numpy, any float type), in
    64 bits: the exponent by comparison, the code by nearest value, ties to the
    code with an even mantissa."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(-1)
    x0 = np.where(finite[..., None], x, 0.0)
    top = np.abs(x0).max(-1)
    e = np.full(top.shape, LEAST[dtype])
    for _ in range(7 - LEAST[dtype]):
        e = np.where((top > 448.0 * 2.0 ** e) & (e < 7), e + 1, e)
    y = np.clip(x0 * 2.0 ** -e[..., None].astype(np.float64), -448, 448)
    pos = E4M3[:127]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code | (np.signbit(y).astype(np.int64) << 7)
    code = np.where(finite[..., None], code, 0x7F).astype(np.uint8)
    return code, np.where(finite, e + 127, 255).astype(np.uint8)


def restore(code, scale):
    up = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return E4M3[code] * up[..., None]


# --- a ragged batch over a paged cache ----------------------------------------
class Problem:
    """lens: cached tokens of each sequence, its new ones included; news: new
    tokens.  Slots no token owns hold NaN (codes 0x7f under scale 255)."""

    def __init__(self, dtype, hq, hkv, ps, lens, news, window=0, q8=False, seed=0, scale=None,
                 extra_rows=2, extra_pages=1, q_size=1.0, loc="hbm", device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.hq, self.hkv, self.ps, self.window = dtype, hq, hkv, ps, window
        self.lens, self.news, self.q8, self.loc = list(lens), list(news), q8, loc
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        B = len(lens)
        self.max_pages = max(1, max(-(-n // ps) for n in lens)) + extra_pages
        need = [-(-n // ps) for n in lens]
        self.pages = sum(need) + 2
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.start = [0]
        for n in news:
            self.start.append(self.start[-1] + n)
        self.total = self.start[-1] + extra_rows
        t = TORCH[dtype]
        self.q = (q_size * torch.randn(self.total, hq, D, generator=g)).to(t)
        shape = (self.pages, hkv, ps, D)
        self.k, self.v = torch.randn(shape, generator=g).to(t), torch.randn(shape, generator=g).to(t)
        owned = torch.zeros(self.pages, ps, dtype=torch.bool)
        for b in range(B):
            for p in range(need[b]):
                owned[self.table[b, p], :min(ps, lens[b] - p * ps)] = True
        self.owned = owned
        if q8:
            self.code, self.scale8 = {}, {}
            for name in ("k", "v"):
                c, s = quantise(getattr(self, name).double().numpy(), dtype)
                hole = ~owned[:, None].expand(-1, hkv, -1).numpy()
                c[hole], s[hole] = 0x7F, 255
                self.code[name], self.scale8[name] = torch.from_numpy(c), torch.from_numpy(s)
        else:
            for x in (self.k, self.v):
                x[~owned[:, None].expand(-1, hkv, -1)] = math.nan
        self.device = device

    # --- device side
    def put(self, x, host=False):
        if host and self.loc == "host":
            return x.contiguous().pin_memory()
        return x.contiguous().to(self.device)

    def upload(self, total=None, max_new=None):
        self.d_table = self.put(self.table)
        self.d_lens = self.put(torch.tensor(self.lens, dtype=torch.int32))
        self.d_start = self.put(torch.tensor(self.start, dtype=torch.int32))
        self.shape = kv.make_shape(len(self.lens), self.hq, self.hkv, D, self.ps, self.max_pages,
                                   self.pages, self.dtype, self.loc)
        self.chunk = kv.make_chunk(self.d_start, total or self.total,
                                   max_new or max(1, max(self.news)), self.window)
        self.d_q = self.put(self.q)
        if self.q8:
            self.d_code = {n: self.put(self.code[n], True) for n in ("k", "v")}
            self.d_scale = {n: self.put(self.scale8[n], True) for n in ("k", "v")}
            self.cache = kv.make_q8_cache(self.d_code["k"], self.d_code["v"], self.d_scale["k"],
                                          self.d_scale["v"])
        else:
            self.d_k, self.d_v = self.put(self.k, True), self.put(self.v, True)
        # rows no sequence owns keep this
        self.d_out = torch.full((self.total, self.hq, D), 7.0, dtype=TORCH[self.dtype],
                                device=self.device)
        need = kv.kv_q8_chunk_workspace_bytes if self.q8 else kv.kv_chunk_workspace_bytes
        self.ws = torch.full((max(16, need(self.shape, self.chunk)),), 255, dtype=torch.uint8,
                             device=self.device)  # NaN patterns
        return self

    def attend(self, stream=None, out=None, ws=None, check=True):
        out = self.d_out if out is None else out
        ws = self.ws if ws is None else ws
        st = torch.cuda.current_stream() if stream is None else stream
        if self.q8:
            return kv.kv_q8_chunk_attn(self.shape, self.chunk, self.d_q, self.cache, self.d_table,
                                       self.d_lens, self.scale, out, ws, ws.numel(), st,
                                       check=check)
        return kv.kv_chunk_attn(self.shape, self.chunk, self.d_q, self.d_k, self.d_v, self.d_table,
                                self.d_lens, self.scale, out, ws, ws.numel(), st, check=check)

    # --- the definition
    def tokens(self, name, b, h):
        """fp64 vectors of sequence b's cached tokens, and which of their pages are in range."""
        at = torch.arange(self.lens[b])
        page = self.table[b].long()[at // self.ps]
        ok = (page >= 0) & (page < self.pages)
        page = torch.where(ok, page, 0)
        if self.q8:
            x = torch.from_numpy(restore(self.code[name][page, h, at % self.ps].numpy(),
                                         self.scale8[name][page, h, at % self.ps].numpy()))
        else:
            x = getattr(self, name)[page, h, at % self.ps].double()
        return x, ok

    def expected(self):
        """(out, tolerance) in 64 bits; rows no sequence owns are 7, tolerance 0.

        Tolerance, from the arithmetic the header states: the result is
        rounded once (half an eps of it); the weights enter the value product
        in dtype (half an eps of sum w |v|, 16-bit types); scores are fp32 dot
        products of 128 terms (128 * 2^-24 of sum |q k|, as an exponent's
        error), scaled in fp32 (2^-22 of the largest exponent); ex2 is within
        2^-21; sums of `len` fp32 terms, and f16 weights below its range."""
        out = torch.full((self.total, self.hq, D), 7.0, dtype=torch.float64)
        tol = torch.zeros_like(out)
        half = torch.finfo(TORCH[self.dtype]).eps / 2
        G = self.hq // self.hkv
        for b in range(len(self.lens)):
            n, length = self.news[b], self.lens[b]
            if n == 0:
                continue
            rows = slice(self.start[b], self.start[b] + n)
            t = torch.arange(length - n, length)[:, None]
            j = torch.arange(length)[None]
            for h in range(self.hkv):
                k, ok = self.tokens("k", b, h)
                v, _ = self.tokens("v", b, h)
                seen = (j <= t) & ok[None]
                if self.window:
                    seen &= j > t - self.window
                for head in range(h * G, (h + 1) * G):
                    q = self.q[rows, head].double()
                    z = (q @ torch.nan_to_num(k).T) * self.scale
                    nan = torch.isnan(k).any(-1)[None] & seen
                    z = z.masked_fill(~seen, -math.inf)
                    top = z.amax(-1, keepdim=True) if length else torch.zeros(n, 1)
                    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top).double())
                    s = p.sum(-1, keepdim=True)
                    w = p / torch.where(s == 0, 1.0, s)
                    vz = torch.where(torch.isfinite(v), v, 0.0)
                    o = w @ vz
                    # a token that is seen and not finite makes its channels NaN
                    bad = (~torch.isfinite(v)).double()
                    o[(seen.double() @ bad) > 0] = math.nan
                    o[nan.any(-1)] = math.nan
                    out[rows, head] = o
                    dz = (q.abs() @ torch.nan_to_num(k).abs().T).max() * abs(self.scale) \
                        if length else torch.tensor(0.0)
                    rel = (half if self.dtype != "f32" else 0) + 2 * float(dz) * D * 2.0 ** -24 \
                        + float(dz) * 2.0 ** -21 + 2.0 ** -21 + length * 2.0 ** -24
                    size = w @ vz.abs()
                    small = 2.0 ** -25 if self.dtype == "f16" else 0
                    tol[rows, head] = half * o.nan_to_num().abs() + rel * size + small * (
                        1 + length * 2.0 ** -7 * (vz.abs().max() if length else 0))
        return out, tol


def check(got, want, tol):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    err = (got - want).nan_to_num().abs()
    over = err - tol
    assert float(over.max()) <= 0, (float(err.max()), float(over.max()))
