"""Rotary positions on the way into a paged cache, and a paged cache held in 4 bits, case by case.

Each case has a plain form in elementary torch operations and the library's own calls beside it; `own`
says which of the two `run` takes.  Formulas, for sequence b with n_b new tokens, row i of which is at
position t (len_b + i, len_b being its length before them, or a given one), and vectors x of 128 channels:

  rope    the first r channels are r / 2 pairs (x_j, x_{j + r/2}) or, interleaved, (x_2j, x_2j+1), turned by
          the angle t * freq_j:  (a, b) -> m (a cos - b sin, a sin + b cos); the other channels stay.
          Rounded once, to the type of x
  append  (rope_append) q and the new keys turned, keys and values stored behind the sequence's cached
          tokens, the channel-wise minimum and maximum of the keys of every page brought up to date
  q4      x is held as 128 integers c of 4 bits, a scale s (e4m3) for each 16 channels, and a power of two:
          e = the smallest integer with max |x| <= 7 * 448 * 2^e, kept in [-15, 4] for f16, [-110, 4] for
          bf16 and f32; s = the smallest e4m3 value with max |x| <= 7 s 2^e over its 16 channels, at most
          448; c = floor(x / (s 2^e) + 1/2), limited to +-7 (0 where s is 0).  Stands for c s 2^e.
          Byte j of a vector holds c + 8 of channels 2j (low half) and 2j + 1; e is kept as e + 127
  q4_read the values that a 4-bit cache stands for, in the model's type
  q4_chunk  row i of the chunk is token t = len_b - n_b + i of the 4-bit cache, which holds the chunk too;
          out = sum_j softmax_j(scale * q . k_j) v_j  over  max(0, t - window + 1) <= j <= t
"""
import math

import torch

own = False

D = 128
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
ROW4 = D // 2 + D // 16 + 1  # bytes of a vector in 4 bits
GOLDEN = 0.6180339887498949
BASES = {"rope": dict(rot=D, inter=False, base=10000.0, stretch=1.0, given=False, index=False),
         "rope_append": dict(rot=D, inter=False, base=10000.0, stretch=1.0, given=False, index=True),
         "q4_append": {}, "q4_read": {}, "q4_chunk": dict(window=0)}


def listed():
    def case(name, op, dtype, batch, hq, hkv, ps, ctx, new, **more):
        return {"name": name, "op": op, "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "ps": ps,
                "ctx": ctx, "new": new, **BASES[op], **more}

    return [
        # q and k of one token of 32 running sequences, on their way into a cache of another form
        case("rope_decode", "rope", "bf16", 32, 32, 8, 16, 4000, 1, base=500000.0),
        # prompts of a batch, half of the channels turned, as many kv heads as query heads
        case("rope_prompts", "rope", "f16", 32, 32, 32, 16, 513, 513, rot=64, inter=True),
        # the whole append of a decode step: q and k turned, k and v stored, page index kept
        case("rope_append_decode", "rope_append", "bf16", 32, 32, 8, 16, 4000, 1, base=500000.0),
        # a prefill step's ragged chunks of a batch of four, frequencies stretched for long contexts
        case("rope_append_chunk", "rope_append", "bf16", 4, 32, 8, 16, 4099, 2048, base=500000.0, stretch=8.0),
        # single precision, a few proposed tokens far into long documents
        case("rope_append_far", "rope_append", "f32", 4, 14, 2, 32, 131072, 7, rot=96, inter=True, stretch=4.0),
        # one new token of 32 running sequences into the 4-bit cache
        case("q4_append_decode", "q4_append", "bf16", 32, 32, 8, 16, 4000, 1),
        # the whole prompts of a batch with as many kv heads as query heads
        case("q4_append_prompts", "q4_append", "f16", 32, 32, 32, 16, 513, 513),
        # a short conversation brought back from the 4-bit cache
        case("q4_read_short", "q4_read", "f16", 2, 32, 32, 16, 544, 1),
        # a long-context batch brought back from the 4-bit cache
        case("q4_read_long", "q4_read", "bf16", 4, 32, 8, 16, 32768, 1),
        # one token per sequence over the 4-bit cache, short contexts: latency
        case("q4_decode_short", "q4_chunk", "f16", 4, 32, 8, 16, 700, 1),
        # one token per sequence over the 4-bit cache, long contexts: bandwidth
        case("q4_decode_long", "q4_chunk", "bf16", 8, 64, 8, 64, 65536, 1),
        # chunked prefill over the 4-bit cache with a sliding window
        case("q4_prefill", "q4_chunk", "bf16", 2, 32, 8, 32, 16001, 1000, window=8192),
    ]


HEADS = [(1, 1), (4, 4), (32, 32), (32, 8), (64, 8), (14, 2), (40, 8), (6, 6), (12, 4), (32, 2)]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["rope", "rope_append", "rope_append", "q4_append", "q4_read", "q4_chunk", "q4_chunk"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        hq, hkv = rng.choice(HEADS)
        ctx = spread(1, 131072 if op in ("rope", "rope_append") else 65536)
        new = 1 if rng.random() < 0.25 else min(ctx, spread(1, 2048))
        c = {"op": op, "dtype": dtype, "batch": spread(1, 32), "hq": hq, "hkv": hkv,
             "ps": rng.choice([16, 32, 64, 128]), "ctx": ctx, "new": new, **BASES[op]}
        if op in ("rope", "rope_append"):
            c.update(rot=rng.choice([8, 24, 32, 64, 96, 128, 128]), inter=rng.random() < 0.5,
                     base=rng.choice([10000.0, 500000.0, 1000000.0]), stretch=rng.choice([1.0, 1.0, 4.0, 32.0]),
                     given=rng.random() < 0.3, index=op == "rope_append" and rng.random() < 0.6)
        if op == "q4_chunk":
            c["window"] = spread(1, 65536) if rng.random() < 0.3 else 0
        w = work(c)
        cache = 2 * c["batch"] * ctx * hkv * D * SIZE[dtype]
        scores = 4 * c["batch"] * hq * new * ctx
        # no dearer than the largest listed cases: bytes, operations, and the plain form's memory
        if w["bytes"] > 5.6e8 or w["flops"] > (5e10 if dtype == "f32" else 1.8e11) or cache > 2.2e9:
            continue
        if op == "q4_chunk" and scores > 6e9:
            continue
        return c


def lengths(case):
    """(context length, chunk length) of every sequence: the first at the full sizes, the others ragged, every fifth without new tokens."""
    n, ctx = [], []
    for b in range(case["batch"]):
        f, g = (0.37 + b * GOLDEN) % 1.0, (0.71 + b * GOLDEN * GOLDEN) % 1.0
        length = case["ctx"] if b == 0 else max(1, round(case["ctx"] * (0.4 + 0.6 * f)))
        new = case["new"] if b == 0 else max(1, round(case["new"] * (0.3 + 0.7 * g)))
        if b % 5 == 3 and case["new"] > 1:
            new = 0
        ctx.append(length)
        n.append(min(new, length))
    return ctx, n


def pairs(length, n, window):
    """(query, key) pairs of one sequence, and the keys that any of its rows sees."""
    if n == 0:
        return 0, 0
    first = length - n
    if window <= 0:
        window = length
    full = max(0, min(n, window - first))  # rows that see everything before them
    total = full * first + full * (full + 1) // 2 + (n - full) * window
    return total, length - max(0, first - window + 1)


def work(case):
    ctx, n = lengths(case)
    size, hq, hkv, ps, op = SIZE[case["dtype"]], case["hq"], case["hkv"], case["ps"], case["op"]
    new = sum(n)
    if op == "rope":
        return {"bytes": new * (hq + hkv) * 2 * D * size, "flops": new * (hq + hkv) * 3 * case["rot"]}
    if op == "rope_append":
        # index entries of the pages touched are written, those of pages begun before are read too
        entries = sum(-(-a // ps) - (a - k) // ps + ((a - k) % ps > 0) for a, k in zip(ctx, n) if k) if case["index"] else 0
        return {"bytes": new * (hq + 2 * hkv) * 2 * D * size + entries * hkv * 2 * D * size,
                "flops": new * (hq + hkv) * 3 * case["rot"]}
    if op == "q4_append":
        return {"bytes": new * hkv * 2 * (D * size + ROW4), "flops": 0}
    if op == "q4_read":
        return {"bytes": sum(ctx) * hkv * 2 * (D * size + ROW4), "flops": 0}
    got = [pairs(a, b, case["window"]) for a, b in zip(ctx, n)]
    return {"bytes": sum(k for _, k in got) * hkv * 2 * ROW4 + 2 * new * hq * D * size,
            "flops": 4 * D * hq * sum(p for p, _ in got)}


def frequencies(case):
    """Radians per position of every pair, in 64 bits, and the factor of the turned channels.  Stretched by a
    factor f: pairs that turn 32 times or more over 8192 positions stay, those that turn once or less are
    slowed by f, those between in proportion; the factor is 0.1 log f + 1."""
    r, f = case["rot"], case["stretch"]
    freq = case["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    keep = ((freq * 8192 / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return freq * (keep + (1 - keep) / f), (0.1 * math.log(f) + 1 if f > 1 else 1.0)


# --- the 4-bit form of vectors x [..., 128]
def e4m3_steps(device):
    """The e4m3 values from 0 to 448 in their codes' order, in 32 bits."""
    return torch.arange(127, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn).float()


def packed(x, dtype):
    """(bytes [..., 64], scale codes [..., 8], power bytes [...]) of x."""
    x = x.float()
    m, p = torch.frexp(x.abs().amax(-1))
    # 7 * 448 = 0.765625 * 2^12
    e = torch.where(m <= 0.765625, p - 12, p - 11)
    e = torch.where(m == 0, -1000, e).clamp(-15 if dtype == "f16" else -110, 4)
    down = ((127 - e) << 23).to(torch.int32).view(torch.float32)
    y = (x * down[..., None]).unflatten(-1, (8, 16))
    steps = e4m3_steps(x.device)
    scale = torch.searchsorted(7 * steps, y.abs().amax(-1)).clamp(max=126)
    s = steps[scale]
    # (in 64 bits: values next to a border)
    c = torch.floor(y.double() / torch.where(s == 0, 1.0, s)[..., None].double() + 0.5).clamp(-7, 7)
    c = (torch.where(s[..., None] == 0, 0, c).to(torch.int32) + 8).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale.to(torch.uint8), (e + 127).to(torch.uint8)


def unpacked(code, scale, power):
    """The fp32 values of bytes [..., 64] with scale codes [..., 8] and power bytes [...]."""
    c = torch.stack([code & 15, code >> 4], -1).flatten(-2).float() - 8
    s = scale.view(torch.float8_e4m3fn).float() * (power.to(torch.int32) << 23).view(torch.float32)[..., None]
    return (c.unflatten(-1, (8, 16)) * s[..., None]).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype, op = TORCH[case["dtype"]], case["op"]
    B, hq, hkv, ps = case["batch"], case["hq"], case["hkv"], case["ps"]
    ctx, n = lengths(case)
    max_pages = -(-case["ctx"] // ps) + 1
    need = [-(-c // ps) for c in ctx]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table, at = torch.full((B, max_pages), -1, dtype=torch.int32), 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    total = sum(n) + 2  # two rows behind the last sequence, as in a padded batch
    start = [0]
    for k in n:
        start.append(start[-1] + k)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": dict(case), "table": table.to(dev), "start": ints(start), "total": total, "max_new": max(max(n), 1),
         "pages": pages, "max_pages": max_pages, "scale": 1.0 / math.sqrt(D)}

    def rows(count, heads):
        return torch.randn((count, heads, D), generator=g, device=dev, dtype=torch.float32).to(dtype)

    def cache():
        return torch.randn((pages, hkv, ps, D), generator=g, device=dev, dtype=torch.float32).to(dtype)

    # keys carry a few large channels; values do not
    wide = torch.where(torch.arange(D, device=dev) % 37 == 5, 12.0, 1.0)
    s["lens"] = ints([c - k for c, k in zip(ctx, n)] if "append" in op or op == "rope" else ctx)
    if "append" in op:
        s["lens_out"] = ints([0] * B)
    if op in ("rope", "rope_append"):
        freq, s["factor"] = frequencies(case)
        s["freq"], s["given"] = freq.to(dev), None
        if case["given"]:  # positions that are not the cache's: tokens were dropped from it before
            s["given"] = torch.randint(0, 1 << 20, (total,), generator=g, device=dev, dtype=torch.int32)
        s["q"], s["k_new"] = rows(total, hq), (rows(total, hkv).float() * wide).to(dtype)
        s["q_out"] = torch.zeros_like(s["q"])
        if op == "rope":
            s["k_out"] = torch.zeros_like(s["k_new"])
            return s
        s["v_new"], s["k"], s["v"] = rows(total, hkv), cache(), cache()
        s["minmax"] = None
        if case["index"]:  # of the tokens cached before; pages without any hold zeros
            owner = torch.zeros(pages, dtype=torch.int32)
            for b in range(B):
                owner[table[b, :need[b]].long()] = (ctx[b] - n[b] - ps * torch.arange(need[b], dtype=torch.int32)).clamp(0, ps)
            there = torch.arange(ps, device=dev) < owner.to(dev)[:, None]
            hole = ~there[:, None, :, None]
            lo, hi = s["k"].masked_fill(hole, math.inf).amin(2), s["k"].masked_fill(hole, -math.inf).amax(2)
            s["minmax"] = torch.stack([lo, hi], 2).masked_fill(~there.any(-1)[:, None, None, None], 0.0)
        return s
    if op == "q4_append":
        s["k_new"], s["v_new"] = (rows(total, hkv).float() * wide).to(dtype), rows(total, hkv)
        for name in ("k", "v"):
            s[name + "_code"] = torch.zeros((pages, hkv, ps, D // 2), dtype=torch.uint8, device=dev)
            s[name + "_scale"] = torch.zeros((pages, hkv, ps, D // 16), dtype=torch.uint8, device=dev)
            s[name + "_power"] = torch.zeros((pages, hkv, ps), dtype=torch.uint8, device=dev)
        return s
    for name in ("k", "v"):
        x = cache()
        got = []
        for part in x.split(max(1, (1 << 26) // (hkv * ps * D))):
            got.append(packed(part, case["dtype"]))
        s[name + "_code"], s[name + "_scale"], s[name + "_power"] = (torch.cat(t) for t in zip(*got))
    if op == "q4_read":
        s["k_out"], s["v_out"] = (torch.zeros((pages, hkv, ps, D), dtype=dtype, device=dev) for _ in range(2))
        return s
    s["q"] = rows(total, hq)
    s["out"] = torch.zeros((total, hq, D), dtype=dtype, device=dev)
    return s


def slots(s, lens, count, most):
    """For the tokens lens[b] .. lens[b] + count[b] - 1 of every sequence: (which are tokens, page, slot), [B, most] each."""
    t = lens[:, None].long() + torch.arange(most, device=lens.device)
    there = torch.arange(most, device=lens.device) < count[:, None]
    t = torch.where(there, t, 0)
    ps = s["case"]["ps"]
    page = torch.gather(s["table"].long(), 1, t // ps)
    return there, page, t % ps


def new_rows(s):
    """The chunk's rows [m], and the sequence and the position in it of each."""
    count = s["start"][1:] - s["start"][:-1]
    i = torch.arange(s["max_new"], device=count.device)
    there = i < count[:, None]
    row = (s["start"][:-1, None] + i)[there].long()
    seq = torch.arange(count.numel(), device=count.device)[:, None].expand_as(there)[there]
    return row, seq, (s["lens"][:, None] + i)[there].long()


def turned(s, x, cos, sin):
    """x [m, heads, 128] with its first rot channels turned; cos, sin: [m, 1, rot / 2]."""
    rot, y = s["case"]["rot"], x.float()
    head = y[..., :rot]
    if s["case"]["inter"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([head, y[..., rot:]], -1).to(x.dtype)


def plain_rope(s):
    case = s["case"]
    row, seq, pos = new_rows(s)
    at = pos if s["given"] is None else s["given"][row].long()
    # (angles in 64 bits: those of far positions lose their fraction in 32)
    angle = at[:, None, None].double() * s["freq"]
    cos, sin = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()
    s["q_out"][row] = turned(s, s["q"][row], cos, sin)
    k = turned(s, s["k_new"][row], cos, sin)
    if case["op"] == "rope":
        s["k_out"][row] = k
        return
    page, slot = s["table"].long()[seq, pos // case["ps"]], pos % case["ps"]
    s["k"][page, :, slot] = k
    s["v"][page, :, slot] = s["v_new"][row]
    s["lens_out"] = s["lens"] + (s["start"][1:] - s["start"][:-1])
    if s["minmax"] is not None:
        mm = s["minmax"]
        begun = page[slot == 0]  # pages that this chunk opens
        mm[begun, :, 0], mm[begun, :, 1] = math.inf, -math.inf
        for at, how in ((0, "amin"), (1, "amax")):
            part = mm[:, :, at].float().index_reduce(0, page, k.float(), how)
            mm[:, :, at] = part.to(mm.dtype)


def plain_append(s):
    row, seq, pos = new_rows(s)
    page, slot = s["table"].long()[seq, pos // s["case"]["ps"]], pos % s["case"]["ps"]
    for name in ("k", "v"):
        code, scale, power = packed(s[name + "_new"][row], s["case"]["dtype"])
        s[name + "_code"][page, :, slot] = code
        s[name + "_scale"][page, :, slot] = scale
        s[name + "_power"][page, :, slot] = power
    s["lens_out"] = s["lens"] + (s["start"][1:] - s["start"][:-1])


def values(s, name, *at):
    return unpacked(*(s[name + part][at] for part in ("_code", "_scale", "_power")))


def plain_read(s):
    there, page, slot = slots(s, torch.zeros_like(s["lens"]), s["lens"], s["case"]["ctx"])
    page, slot = page[there], slot[there]
    for name in ("k", "v"):
        x = unpacked(*(s[name + part][page, :, slot] for part in ("_code", "_scale", "_power")))
        s[name + "_out"][page, :, slot] = x.to(s[name + "_out"].dtype)


def plain_chunk(s):
    case = s["case"]
    B, hq, hkv, most = case["batch"], case["hq"], case["hkv"], s["max_new"]
    dev, count = s["lens"].device, s["start"][1:] - s["start"][:-1]
    page = s["table"].long().clamp(min=0)
    k, v = (values(s, name, page).transpose(1, 2).reshape(B, hkv, -1, D)[:, :, :case["ctx"]] for name in ("k", "v"))
    there = torch.arange(most, device=dev) < count[:, None]
    row = torch.where(there, s["start"][:-1, None] + torch.arange(most, device=dev), 0).long()
    q = s["q"][row].float().reshape(B, most, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(B, hkv, -1, D)
    t = (s["lens"] - count)[:, None] + torch.arange(most, device=dev)
    j = torch.arange(case["ctx"], device=dev)
    seen = (j <= t[..., None]) & (j < s["lens"][:, None, None]) & there[..., None]
    if case["window"]:
        seen &= j > t[..., None] - case["window"]
    score = (q @ k.transpose(-1, -2)).reshape(B, hq, most, -1) * s["scale"]
    score.masked_fill_(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = p.reshape(B, hkv, -1, p.shape[-1]) @ v
    o = o.reshape(B, hq, most, D) / torch.where(total == 0, 1.0, total)
    s["out"][row[there]] = o.transpose(1, 2)[there].to(s["out"].dtype)


def own_call(s):
    from offloaded_kv_cache_gb300 import kvsparse as kv

    case, op = s["case"], s["case"]["op"]
    st = torch.cuda.current_stream()
    if "shape" not in s:  # what a program sets up once beside its buffers
        s["shape"] = kv.make_shape(case["batch"], case["hq"], case["hkv"], D, case["ps"], s["max_pages"], s["pages"], case["dtype"])
        s["chunk"] = kv.make_chunk(s["start"], s["total"], s["max_new"], case.get("window", 0))
        if op.startswith("q4"):
            s["q4"] = kv.make_q4_cache(s["k_code"], s["v_code"], s["k_scale"], s["v_scale"], s["k_power"], s["v_power"])
        else:
            s["turn"] = kv.make_rope(s["freq"], case["rot"], case["inter"], s["factor"], s["given"])
        s["bytes"] = kv.kv_q4_chunk_workspace_bytes(s["shape"], s["chunk"]) if op == "q4_chunk" else 0
        s["space"] = torch.empty(max(16, s["bytes"]), dtype=torch.uint8, device=s["table"].device)
    if op == "rope":
        kv.kv_rope(s["shape"], s["chunk"], s["turn"], s["q"], s["q_out"], s["k_new"], s["k_out"], s["lens"], st)
    elif op == "rope_append":
        kv.kv_rope_append(s["shape"], s["chunk"], s["turn"], s["q"], s["q_out"], s["k_new"], s["v_new"], s["k"], s["v"],
                          s["table"], s["lens"], s["lens_out"], s["minmax"], st)
    elif op == "q4_append":
        kv.kv_q4_append(s["shape"], s["chunk"], s["k_new"], s["v_new"], s["q4"], s["table"], s["lens"], s["lens_out"], st)
    elif op == "q4_read":
        kv.kv_q4_read(s["shape"], s["q4"], s["table"], s["lens"], s["table"], s["pages"], s["k_out"], s["v_out"], st)
    else:
        kv.kv_q4_chunk_attn(s["shape"], s["chunk"], s["q"], s["q4"], s["table"], s["lens"], s["scale"], s["out"], s["space"], s["bytes"], st)


def run(state):
    op = state["case"]["op"]
    if own:
        own_call(state)
    else:
        {"rope": plain_rope, "rope_append": plain_rope, "q4_append": plain_append, "q4_read": plain_read}.get(op, plain_chunk)(state)
    if op == "rope":
        return {"q": state["q_out"], "k": state["k_out"]}
    if op == "rope_append":
        return {"q": state["q_out"], "k": state["k"], "v": state["v"], "lens": state["lens_out"], "minmax": state["minmax"]}
    if op == "q4_append":  # the codes two to a byte, as whole numbers
        out = {name + part: state[name + part] for name in ("k", "v") for part in ("_code", "_power")}
        out.update({name + "_scale": state[name + "_scale"].view(torch.float8_e4m3fn) for name in ("k", "v")})
        return {**out, "lens": state["lens_out"]}
    if op == "q4_read":
        return {"k": state["k_out"], "v": state["v_out"]}
    return {"out": state["out"]}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    dev, ps, op = s["table"].device, case["ps"], case["op"]
    ctx, n = lengths(case)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    pages = lambda b, t: (s["table"][b, t // ps].long(), t % ps)  # noqa: E731
    two = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    steps = torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()

    def value(name, p, h, o):
        code = s[name + "_code"][p, h, o].long()
        c = torch.zeros((*code.shape[:-1], D), dtype=torch.float64, device=dev)
        c[..., 0::2], c[..., 1::2] = (code % 16).double() - 8, (code // 16).double() - 8
        scale = steps[s[name + "_scale"][p, h, o].long()] * two(s[name + "_power"][p, h, o].int() - 127)[..., None]
        return c * scale.repeat_interleave(16, -1)

    if op in ("rope", "rope_append"):
        rot, half = case["rot"], case["rot"] // 2
        j = torch.arange(half, device=dev)
        first, second = (2 * j, 2 * j + 1) if case["inter"] else (j, j + half)

        def turn(x, at):
            y = x.double()
            z = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=dev), at.double()[:, None, None] * s["freq"])
            w = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = w.real, w.imag
            return y

        out = {"q": torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)}
        if op == "rope":
            out["k"] = torch.zeros(s["k_new"].shape, dtype=torch.float64, device=dev)
        else:
            out["k"], out["v"] = s["k"].double(), s["v"].double()
            out["minmax"] = None if s["minmax"] is None else s["minmax"].double()
            out["lens"] = torch.tensor([a + b for a, b in zip(lens, n)], dtype=torch.int32, device=dev)
        for b in range(case["batch"]):
            if n[b] == 0:
                continue
            rows, t = slice(start[b], start[b] + n[b]), torch.arange(lens[b], lens[b] + n[b], device=dev)
            at = t if s["given"] is None else s["given"][rows]
            out["q"][rows] = turn(s["q"][rows], at)
            k = turn(s["k_new"][rows], at)
            if op == "rope":
                out["k"][rows] = k
                continue
            p, o = pages(b, t)
            out["k"][p, :, o], out["v"][p, :, o] = k, s["v_new"][rows].double()
            if s["minmax"] is not None:
                for page in range(lens[b] // ps, (lens[b] + n[b] - 1) // ps + 1):
                    at = s["table"][b, page].long()
                    seen = out["k"][at, :, :min(ps, lens[b] + n[b] - page * ps)]
                    out["minmax"][at, :, 0], out["minmax"][at, :, 1] = seen.amin(1), seen.amax(1)
        return out
    if op == "q4_append":
        out = {"lens": torch.tensor([a + b for a, b in zip(lens, n)], dtype=torch.int32, device=dev)}
        least = -15 if case["dtype"] == "f16" else -110
        for name in ("k", "v"):
            for part in ("_code", "_power"):
                out[name + part] = torch.zeros_like(s[name + part])
            out[name + "_scale"] = torch.zeros(s[name + "_scale"].shape, dtype=torch.float64, device=dev)
            for b in range(case["batch"]):
                p, o = pages(b, torch.arange(lens[b], lens[b] + n[b], device=dev))
                x = s[name + "_new"][start[b]:start[b] + n[b]].double()
                top = x.abs().amax(-1)
                # the smallest e with top <= 3136 * 2^e: a guess from the logarithm, put right by comparing
                e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0) / 3136.0)) - 1
                for _ in range(3):
                    e = torch.where(top > 3136.0 * two(e), e + 1, e)
                e = torch.where(top > 0, e, -1000).clamp(least, 4)
                y = (x * two(-e)[..., None]).unflatten(-1, (8, 16))
                # the smallest step that reaches: as many as do not
                scale = steps[(7 * steps < y.abs().amax(-1, keepdim=True)).sum(-1).clamp(max=126)]
                c = torch.floor((2 * y + scale[..., None]) / (2 * torch.where(scale > 0, scale, 1.0)[..., None]))
                c = torch.where(scale[..., None] > 0, c.clamp(-7, 7), 0.0).flatten(-2).long() + 8
                out[name + "_code"][p, :, o] = (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)
                out[name + "_scale"][p, :, o] = scale
                out[name + "_power"][p, :, o] = (e + 127).to(torch.uint8)
        return out
    if op == "q4_read":
        out = {name: torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=dev) for name in ("k", "v")}
        heads = torch.arange(case["hkv"], device=dev)[None]
        for b in range(case["batch"]):
            p, o = pages(b, torch.arange(ctx[b], device=dev))
            for name in ("k", "v"):
                out[name][p, :, o] = value(name, p[:, None], heads, o[:, None])
        return out
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    group = case["hq"] // case["hkv"]
    for b in range(case["batch"]):
        if n[b] == 0:
            continue
        i = torch.arange(ctx[b] - n[b], ctx[b], device=dev)
        lo = max(0, ctx[b] - n[b] - case["window"] + 1) if case["window"] else 0
        j = torch.arange(lo, ctx[b], device=dev)
        hidden = j[None] > i[:, None]
        if case["window"]:
            hidden |= j[None] <= i[:, None] - case["window"]
        p, o = pages(b, j)
        for h in range(case["hkv"]):
            k, v = (value(name, p, h, o) for name in ("k", "v"))
            for head in range(h * group, (h + 1) * group):
                q = s["q"][start[b]:start[b] + n[b], head].double()
                z = ((q @ k.T) * s["scale"]).masked_fill(hidden, -math.inf)
                out[start[b]:start[b] + n[b], head] = torch.softmax(z, -1) @ v
    return {"out": out}
