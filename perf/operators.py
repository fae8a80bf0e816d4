"""The chunk operators over a paged cache, case by case: 8-bit append, 8-bit read back, and the attention
of a chunk of new tokens over a cache of the model's own type or of 8 bits.

Each case has a plain form in elementary torch operations and the library's own calls beside it; `own`
says which of the two `run` takes.  Formulas, for sequence b with len_b cached tokens of which the last
n_b are the chunk's:

  append  every key and value vector x (128 elements) is held as e4m3 codes c and one power of two 2^e:
          e = the smallest integer with max|x| <= 448 * 2^e, kept in [-15, 7] for f16 and [-110, 7] for
          bf16 and f32; c = e4m3(x * 2^-e), ties to even, limited to +-448; the scale is kept as the
          byte e + 127
  read    x' = c * 2^e
  chunk   row i of the chunk is token t = len_b - n_b + i;
          out = sum_j softmax_j(scale * q . k_j) v_j  over  max(0, t - window + 1) <= j <= t
"""
import math

import torch

own = False

D = 128
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
GOLDEN = 0.6180339887498949


def listed():
    def case(name, op, dtype, batch, hq, hkv, ps, ctx, new, window=0):
        return {"name": name, "op": op, "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "ps": ps,
                "ctx": ctx, "new": new, "window": window}

    return [
        # one new token of 32 running sequences: the append of every decode step
        case("append_decode", "append", "bf16", 32, 32, 8, 16, 4000, 1),
        # a prefill step's ragged chunks of a batch of four
        case("append_chunk", "append", "bf16", 4, 32, 8, 16, 4099, 2048),
        # the whole prompts of a batch with as many kv heads as query heads
        case("append_prompts", "append", "f16", 32, 32, 32, 16, 513, 513),
        # a short conversation brought back from the 8-bit cache
        case("read_short", "read", "f16", 2, 32, 32, 16, 544, 1),
        # a long-context batch brought back from the 8-bit cache
        case("read_long", "read", "bf16", 4, 32, 8, 16, 32768, 1),
        # single precision, one head: the smallest configuration, a short chunk behind a long context
        case("chunk_f32", "chunk", "f32", 1, 1, 1, 16, 4096, 33),
        # whole prompts, no cached context before them
        case("chunk_prompts", "chunk", "f16", 32, 32, 32, 16, 512, 512),
        # chunked prefill of a long document: the arithmetic-bound end
        case("chunk_prefill", "chunk", "bf16", 1, 32, 8, 16, 32768, 2048),
        # a few proposed tokens per sequence checked against long contexts: the bandwidth-bound end
        case("chunk_verify", "chunk", "bf16", 8, 64, 8, 64, 65536, 5),
        # one token per sequence over the 8-bit cache, short contexts: latency
        case("q8_decode_short", "q8_chunk", "f16", 4, 32, 8, 16, 700, 1),
        # one token per sequence over the 8-bit cache, long contexts: bandwidth
        case("q8_decode_long", "q8_chunk", "bf16", 8, 64, 8, 64, 65536, 1),
        # chunked prefill over the 8-bit cache with a sliding window
        case("q8_prefill", "q8_chunk", "bf16", 2, 32, 8, 32, 16001, 1000, 8192),
    ]


HEADS = [(1, 1), (4, 4), (32, 32), (32, 8), (64, 8), (14, 2), (40, 8), (6, 6), (12, 4), (32, 2)]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["append", "read", "chunk", "chunk", "q8_chunk", "q8_chunk"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        hq, hkv = rng.choice(HEADS)
        ctx = spread(1, 65536)
        new = 1 if rng.random() < 0.25 else min(ctx, spread(1, 2048))
        c = {"op": op, "dtype": dtype, "batch": spread(1, 32), "hq": hq, "hkv": hkv,
             "ps": rng.choice([16, 32, 64, 128]), "ctx": ctx, "new": new,
             "window": spread(1, 65536) if rng.random() < 0.3 else 0}
        if op in ("append", "read"):
            c["window"] = 0
        w = work(c)
        cache = 2 * c["batch"] * ctx * hkv * D * SIZE[dtype]
        scores = 4 * c["batch"] * hq * new * ctx
        # no dearer than the largest listed cases: bytes, operations, and the plain form's memory
        if w["bytes"] > 2.1e9 or w["flops"] > (5e10 if dtype == "f32" else 1e12) or cache > 2.2e9:
            continue
        if op in ("chunk", "q8_chunk") and scores > 9e9:
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
    size, hq, hkv = SIZE[case["dtype"]], case["hq"], case["hkv"]
    if case["op"] == "append":
        return {"bytes": sum(n) * hkv * 2 * (D * size + D + 1), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(ctx) * hkv * 2 * (D * size + D + 1), "flops": 0}
    got = [pairs(a, b, case["window"]) for a, b in zip(ctx, n)]
    row = D + 1 if case["op"] == "q8_chunk" else D * size
    return {"bytes": sum(k for _, k in got) * hkv * 2 * row + 2 * sum(n) * hq * D * size,
            "flops": 4 * D * hq * sum(p for p, _ in got)}


def quantised(x, dtype):
    """Codes (uint8, e4m3 bits) and scale bytes of vectors x [..., 128]."""
    x = x.float()
    m, p = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(-15 if dtype == "f16" else -110, 7)
    down = ((127 - e) << 23).to(torch.int32).view(torch.float32)
    code = (x * down[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return code.view(torch.uint8), (e + 127).to(torch.uint8)


def restored(code, scale):
    """The fp32 values of codes [..., 128] with scale bytes [...]."""
    up = (scale.to(torch.int32) << 23).view(torch.float32)
    return code.view(torch.float8_e4m3fn).float() * up[..., None]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype, B, hq, hkv, ps = TORCH[case["dtype"]], case["batch"], case["hq"], case["hkv"], case["ps"]
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

    if case["op"] == "append":
        before = [c - k for c, k in zip(ctx, n)]
        s["lens"], s["lens_out"] = ints(before), ints([0] * B)
        # keys carry a few large channels, as after rotary positions; values do not
        wide = torch.where(torch.arange(D, device=dev) % 37 == 5, 12.0, 1.0)
        s["k_new"], s["v_new"] = (rows(total, hkv).float() * wide).to(dtype), rows(total, hkv)
        for name in ("k", "v"):
            s[name + "_code"] = torch.zeros((pages, hkv, ps, D), dtype=torch.uint8, device=dev)
            s[name + "_scale"] = torch.zeros((pages, hkv, ps), dtype=torch.uint8, device=dev)
        return s
    s["lens"] = ints(ctx)
    if case["op"] in ("read", "q8_chunk"):
        for name in ("k", "v"):
            s[name + "_code"], s[name + "_scale"] = quantised(cache(), case["dtype"])
    if case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros((pages, hkv, ps, D), dtype=dtype, device=dev) for _ in range(2))
        return s
    if case["op"] == "chunk":
        s["k"], s["v"] = cache(), cache()
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


def plain_append(s):
    count = s["start"][1:] - s["start"][:-1]
    there, page, slot = slots(s, s["lens"], count, s["max_new"])
    row = (s["start"][:-1, None] + torch.arange(s["max_new"], device=count.device))[there].long()
    page, slot = page[there], slot[there]
    for name in ("k", "v"):
        code, scale = quantised(s[name + "_new"][row], s["case"]["dtype"])
        s[name + "_code"][page, :, slot] = code
        s[name + "_scale"][page, :, slot] = scale
    s["lens_out"] = s["lens"] + count


def plain_read(s):
    there, page, slot = slots(s, torch.zeros_like(s["lens"]), s["lens"], s["case"]["ctx"])
    page, slot = page[there], slot[there]
    for name in ("k", "v"):
        x = restored(s[name + "_code"][page, :, slot], s[name + "_scale"][page, :, slot])
        s[name + "_out"][page, :, slot] = x.to(s[name + "_out"].dtype)


def plain_chunk(s):
    case = s["case"]
    B, hq, hkv, most = case["batch"], case["hq"], case["hkv"], s["max_new"]
    dev, count = s["lens"].device, s["start"][1:] - s["start"][:-1]
    page = s["table"].long().clamp(min=0)
    if case["op"] == "chunk":
        k, v = s["k"][page].float(), s["v"][page].float()
    else:
        k, v = (restored(s[name + "_code"][page], s[name + "_scale"][page]) for name in ("k", "v"))
    k, v = (x.transpose(1, 2).reshape(B, hkv, -1, D)[:, :, :case["ctx"]] for x in (k, v))
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
        s["chunk"] = kv.make_chunk(s["start"], s["total"], s["max_new"], case["window"])
        if op != "chunk":
            s["q8"] = kv.make_q8_cache(s["k_code"], s["v_code"], s["k_scale"], s["v_scale"])
        need = {"chunk": kv.kv_chunk_workspace_bytes, "q8_chunk": kv.kv_q8_chunk_workspace_bytes}.get(op)
        s["bytes"] = need(s["shape"], s["chunk"]) if need else 0
        s["space"] = torch.empty(max(16, s["bytes"]), dtype=torch.uint8, device=s["table"].device)
    if op == "append":
        kv.kv_q8_append(s["shape"], s["chunk"], s["k_new"], s["v_new"], s["q8"], s["table"], s["lens"], s["lens_out"], st)
    elif op == "read":
        kv.kv_q8_read(s["shape"], s["q8"], s["table"], s["lens"], s["table"], s["pages"], s["k_out"], s["v_out"], st)
    elif op == "chunk":
        kv.kv_chunk_attn(s["shape"], s["chunk"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], s["out"], s["space"], s["bytes"], st)
    else:
        kv.kv_q8_chunk_attn(s["shape"], s["chunk"], s["q"], s["q8"], s["table"], s["lens"], s["scale"], s["out"], s["space"], s["bytes"], st)


def run(state):
    op = state["case"]["op"]
    if own:
        own_call(state)
    else:
        {"append": plain_append, "read": plain_read}.get(op, plain_chunk)(state)
    if op == "append":
        code = {k: state[k + "_code"].view(torch.float8_e4m3fn) for k in ("k", "v")}
        return {"k_code": code["k"], "v_code": code["v"], "k_scale": state["k_scale"], "v_scale": state["v_scale"],
                "lens": state["lens_out"]}
    if op == "read":
        return {"k": state["k_out"], "v": state["v_out"]}
    return {"out": state["out"]}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, one sequence and one head at a time."""
    s = prepare(case, seed)
    dev, ps, op = s["table"].device, case["ps"], case["op"]
    ctx, n = lengths(case)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    pages = lambda b, t: (s["table"][b, t // ps].long(), t % ps)  # noqa: E731
    two = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    value = lambda name, p, h, o: (s[name + "_code"][p, h, o].view(torch.float8_e4m3fn).double()  # noqa: E731
                                   * two(s[name + "_scale"][p, h, o].int() - 127)[..., None])
    if op == "append":
        out = {"lens": torch.tensor([a + b for a, b in zip(lens, n)], dtype=torch.int32, device=dev)}
        least = -15 if case["dtype"] == "f16" else -110
        for name in ("k", "v"):
            code = torch.zeros(s[name + "_code"].shape, dtype=torch.float64, device=dev)
            scale = torch.zeros_like(s[name + "_scale"])
            for b in range(case["batch"]):
                p, o = pages(b, torch.arange(lens[b], lens[b] + n[b], device=dev))
                x = s[name + "_new"][start[b]:start[b] + n[b]].double()
                top = x.abs().amax(-1)
                # the smallest e with top <= 448 * 2^e: a guess from the logarithm, put right by comparing
                e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0) / 448.0)) - 1
                for _ in range(3):
                    e = torch.where(top > 448.0 * two(e), e + 1, e)
                e = torch.where(top > 0, e, -1000).clamp(least, 7)
                y = (x * two(-e)[..., None]).clamp(-448, 448)
                grid = two(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
                code[p, :, o] = torch.round(y / grid) * grid
                scale[p, :, o] = (e + 127).to(torch.uint8)
            out[name + "_code"], out[name + "_scale"] = code, scale
        return out
    if op == "read":
        out = {name: torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=dev) for name in ("k", "v")}
        for b in range(case["batch"]):
            p, o = pages(b, torch.arange(ctx[b], device=dev))
            for name in ("k", "v"):
                out[name][p, :, o] = value(name, p[:, None], torch.arange(case["hkv"], device=dev)[None], o[:, None])
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
            k, v = (s[name][p, h, o].double() if op == "chunk" else value(name, p, h, o) for name in ("k", "v"))
            for head in range(h * group, (h + 1) * group):
                q = s["q"][start[b]:start[b] + n[b], head].double()
                z = ((q @ k.T) * s["scale"]).masked_fill(hidden, -math.inf)
                out[start[b]:start[b] + n[b], head] = torch.softmax(z, -1) @ v
    return {"out": out}
