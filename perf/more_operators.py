"""The operators around an 8-bit cache as a serving program runs them: cases, inputs, one pass, and the work of a pass.

Operators: rotary positions of queries and keys; keys and values written into cache pages as e4m3 codes with a power-of-two scale for each block of
tokens and head; such pages read back as packed 16-bit rows; and attention of single tokens over them. ``own`` false computes them with elementary torch
operations in fp32 (angles in fp64), ``own`` true calls the library."""

import math

import torch

own = False

LN2 = math.log(2.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = torch.float8_e4m3fn
LARGEST = 448.0


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(map(str, values))


def _lens(count, most):
    """Lengths spread over 1..most."""
    return [1 + (i * 7919 + 13) * 104729 % most for i in range(count)]


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decode step of a handful of sequences: latency.
        {"name": "rotary_tokens", "op": "rotary", "tokens": 8, "heads": 8, "kv_heads": 2, "dim": 64, "turning": 64, "far": 8192, "stretch": 1.0,
         "interleaved": False, "transpose": False, "dtype": "bf16"},
        # A packed prefill chunk, whole heads turned.
        {"name": "rotary_chunk", "op": "rotary", "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "turning": 128, "far": 16384, "stretch": 1.0,
         "interleaved": False, "transpose": False, "dtype": "bf16"},
        # The gradient in fp32: neighbours paired, part of the head, a context stretched 16 times, far positions.
        {"name": "rotary_gradient", "op": "rotary", "tokens": 4099, "heads": 12, "kv_heads": 4, "dim": 96, "turning": 40, "far": 1000000, "stretch": 16.0,
         "interleaved": True, "transpose": True, "dtype": "fp32"},
        # One new token for each sequence of a chat batch: latency.
        {"name": "write_tokens", "op": "write", "new": _text([1] * 64), "held": _text(_lens(64, 9215)), "kv_heads": 8, "dim": 128, "page": 64, "block": 64,
         "dtype": "bf16"},
        # A ragged batch of prompts, some behind cached tokens that end inside a block.
        {"name": "write_ragged", "op": "write", "new": "37,1900,512,1,255,1024,129,700", "held": "1000,0,1536,776,31,476,0,2801", "kv_heads": 4, "dim": 96,
         "page": 32, "block": 16, "dtype": "fp16"},
        # One long prompt.
        {"name": "write_prompt", "op": "write", "new": "16389", "held": "0", "kv_heads": 8, "dim": 128, "page": 128, "block": 128, "dtype": "bf16"},
        # Short sequences read back for a prompt's attention: latency.
        {"name": "read_short", "op": "read", "lens": "160,200,33", "kv_heads": 2, "dim": 64, "page": 16, "block": 16, "dtype": "fp16"},
        # The keys and values that a packed prefill chunk attends to.
        {"name": "read_chunk", "op": "read", "lens": "8192,6201,2048,4100", "kv_heads": 8, "dim": 128, "page": 64, "block": 32, "dtype": "bf16"},
        # A few short sequences: latency.
        {"name": "attend_short", "op": "attend", "lens": "200,161,183", "kv_heads": 2, "group": 4, "dim": 64, "page": 16, "block": 16, "dtype": "bf16"},
        # Ragged lengths, odd group and head dim.
        {"name": "attend_ragged", "op": "attend", "lens": _text(_lens(33, 8000)), "kv_heads": 8, "group": 5, "dim": 80, "page": 32, "block": 16, "dtype": "fp16"},
        # A chat batch.
        {"name": "attend_chat", "op": "attend", "lens": _text(_lens(64, 9216)), "kv_heads": 8, "group": 4, "dim": 128, "page": 64, "block": 64, "dtype": "bf16"},
        # Two long documents: little but the long axis to split.
        {"name": "attend_documents", "op": "attend", "lens": "262143,196613", "kv_heads": 4, "group": 8, "dim": 128, "page": 128, "block": 32, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "attend", "attend"])
    if op == "rotary":
        dim = rng.choice([64, 96, 128, 128, 2 * rng.randint(8, 64)])
        c = {"op": op, "tokens": _log(rng, 1, 8192), "heads": rng.choice([4, 8, 12, 16, 32]), "kv_heads": rng.choice([1, 2, 4, 8]), "dim": dim,
             "turning": dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2), "far": _log(rng, 1000, 1000000), "stretch": rng.choice([1.0, 1.0, 4.0, 16.0]),
             "interleaved": rng.random() < 0.5, "transpose": rng.random() < 0.3, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
        while c["tokens"] * (c["heads"] + c["kv_heads"]) * dim > 8192 * 40 * 64:
            c["tokens"] //= 2
        return c
    page = rng.choice([16, 32, 64, 128])
    c = {"op": op, "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128, 128, 16 * rng.randint(2, 8)]), "page": page,
         "block": rng.choice([b for b in (16, 32, 64, 128) if b <= page]), "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op == "write":
        count = _log(rng, 1, 128)
        new = [1] * count if rng.random() < 0.4 else [_log(rng, 1, max(1, 16000 // count)) for _ in range(count)]
        return {**c, "new": _text(new), "held": _text([0 if rng.random() < 0.3 else _log(rng, 1, 9000) for _ in new])}
    if op == "read":
        count = _log(rng, 1, 64)
        return {**c, "lens": _text([_log(rng, 1, max(1, 20000 // count)) for _ in range(count)])}
    count = _log(rng, 1, 128)
    most = min(200000, 400000 // count)
    return {**c, "group": rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), "lens": _text([_log(rng, 1, most) for _ in range(count)])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _dev(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """Radians per token of every pair, in fp64: those that turn less than once in 8192 tokens slowed down by `stretch`, those that turn more than 32 times
    kept, the others in between."""
    f = 10000.0 ** (-torch.arange(c["turning"] // 2, dtype=torch.float64) * 2 / c["turning"])
    w = ((f * 8192 / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f * (w + (1 - w) / c["stretch"])


def _factor(c):
    return 1.0 + 0.1 * math.log(c["stretch"])


def _paged(c, g, lens, room):
    """Pages of held tokens, with room for `room` tokens in each sequence."""
    page = c["page"]
    need = [-(-n // page) for n in room]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    tables, at = [], 0
    for n in need:
        tables.append(ids[at:at + n] + [-1] * (max(need) - n))
        at += n
    codes = torch.randn((2, pages, page, c["kv_heads"], c["dim"]), generator=g, device="cuda", dtype=torch.float32)
    cache = codes.mul_(80.0).clamp_(-LARGEST, LARGEST).to(CODES)
    power = torch.randint(-7, -4, (2, pages, page // c["block"], c["kv_heads"]), generator=g, device="cuda")
    return {"cache": cache, "scales": torch.exp2(power.float()), "tables": _dev(tables), "lens": _dev(lens)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dt = case, DTYPES[case["dtype"]]
    if c["op"] == "rotary":
        s = {"q": _randn(g, (c["tokens"], c["heads"], c["dim"]), dt), "k": _randn(g, (c["tokens"], c["kv_heads"], c["dim"]), dt),
             "positions": torch.randint(0, c["far"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32),
             "frequencies": _frequencies(c).cuda(), "interleaved": c["interleaved"], "transpose": c["transpose"], "factor": _factor(c)}
        # what a program lays out once for a model: turns per token in fixed point, 2^64 to a turn
        turns = s["frequencies"].cpu() / (2 * math.pi)
        s["turns"] = torch.tensor([(int(round(x * 2.0 ** 64)) + 2 ** 63) % 2 ** 64 - 2 ** 63 for x in turns.tolist()], dtype=torch.int64, device="cuda")
    elif c["op"] == "write":
        new, held = _ints(c["new"]), _ints(c["held"])
        s = _paged(c, g, held, [a + b for a, b in zip(new, held)])
        shape = (sum(new), c["kv_heads"], c["dim"])
        # tokens of other magnitudes, now and then one that its block's scale does not hold
        s["k"], s["v"] = ((torch.randn(shape, generator=g, device="cuda") * torch.randn((shape[0], 1, 1), generator=g, device="cuda").mul_(0.7).exp_()).to(dt)
                          for _ in range(2))
        s["cu"] = _dev([sum(new[:i]) for i in range(len(new) + 1)])
    elif c["op"] == "read":
        lens = _ints(c["lens"])
        s = _paged(c, g, lens, lens)
        s["cu"] = _dev([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["total"], s["dtype"] = sum(lens), dt
    else:
        lens = _ints(c["lens"])
        s = _paged(c, g, lens, lens)
        s["q"] = _randn(g, (len(lens), c["kv_heads"] * c["group"], c["dim"]), dt, 1.5)
    s["op"] = c["op"]
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _turned(x, cos, sin, interleaved):
    """x [T, heads, dim] with its first 2 * cos.shape[-1] elements turned."""
    n = 2 * cos.shape[-1]
    y = x.float()
    cos, sin = cos[:, None], sin[:, None]
    a, b = (y[..., 0:n:2], y[..., 1:n:2]) if interleaved else (y[..., :n // 2], y[..., n // 2:n])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((turned, y[..., n:]), -1).to(x.dtype)


def _plain_rotary(s):
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()
    if s["transpose"]:
        sin = -sin
    return _turned(s["q"], cos, sin, s["interleaved"]), _turned(s["k"], cos, sin, s["interleaved"])


def _power(x):
    """The smallest power of two from 2^-126 on that is not below x."""
    m, e = torch.frexp(x)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
    return torch.ldexp(torch.ones_like(x), e)


def _plain_write(s):
    (_, pages, page, heads, dim), cu, lens, tables = s["cache"].shape, s["cu"], s["lens"].long(), s["tables"].long()
    per = s["scales"].shape[2]
    block = page // per
    x = torch.stack((s["k"], s["v"])).float()
    tok = torch.arange(x.shape[1], device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = lens[seq] + tok - cu[seq]
    at = tables[seq, pos // page] * page + pos % page
    # the largest value of every block's new tokens, and the scale that it needs
    top = torch.zeros((2, pages * per, heads), device=x.device)
    where = (at // block)[None, :, None].expand(2, -1, heads)
    top.scatter_reduce_(1, where, x.abs().amax(-1), "amax")
    need = _power(top / LARGEST)  # exact in fp32 but for the last bit, which no 16-bit input reaches
    scales = s["scales"].view(2, pages * per, heads)
    # a block that holds tokens already keeps its scale, or has them rounded to the new one
    first = lens // block * block
    has = (lens % block > 0) & (cu[1:] > cu[:-1])
    old = tables.gather(1, (first // page)[:, None].clamp(max=tables.shape[1] - 1))[:, 0] * per + first % page // block
    held = torch.zeros(pages * per, dtype=torch.bool, device=x.device)
    held[old[has]] = True
    fits = torch.where(held[None, :, None], torch.maximum(need, scales), need)
    mine, was = old[has], (torch.arange(block, device=x.device) < (lens % block)[has, None])[None, :, :, None, None]
    codes = s["cache"].view(2, pages * per, block, heads, dim)
    kept = codes.view(torch.uint8)[:, mine].view(CODES).float()
    ratio = (scales[:, mine] / fits[:, mine])[:, :, None, :, None]
    again = torch.where(was, (kept * ratio).to(CODES).float(), kept).to(CODES)
    codes.view(torch.uint8)[:, mine] = again.view(torch.uint8)
    fresh = torch.zeros(pages * per, dtype=torch.bool, device=x.device)
    fresh[at // block] = True
    scales.copy_(torch.where(fresh[None, :, None], fits, scales))
    rows = (x / fits[:, at // block][..., None]).to(CODES)
    s["cache"].view(2, pages * page, heads, dim).view(torch.uint8)[:, at] = rows.view(torch.uint8)


def _plain_read(s):
    pages, page, heads, dim = s["cache"].shape[1:]
    cu, tables = s["cu"], s["tables"].long()
    block = page // s["scales"].shape[2]
    tok = torch.arange(s["total"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = tok - cu[seq]
    at = tables[seq, pos // page] * page + pos % page
    codes = s["cache"].view(2, pages * page, heads, dim).view(torch.uint8)[:, at].view(CODES).float()
    return tuple((codes * s["scales"].view(2, -1, heads)[:, at // block][..., None]).to(s["dtype"]))


def _plain_attend(s):
    q, lens, tables = s["q"], s["lens"], s["tables"].long().clamp(min=0)
    pages, page, kv_heads, dim = s["cache"].shape[1:]
    per = s["scales"].shape[2]
    batch, heads = q.shape[:2]
    n = tables.shape[1] * page
    codes = s["cache"].view(torch.uint8)

    def rows(i):
        """[kv head, batch, token, dim] of keys or values."""
        x = codes[i][tables].view(CODES).float().view(batch, n // page * per, page // per, kv_heads, dim)
        x.mul_(s["scales"][i][tables].view(batch, n // page * per, 1, kv_heads, 1))
        return x.view(batch, n, kv_heads, dim).permute(2, 0, 1, 3)

    x = torch.matmul(q.float().view(batch, kv_heads, -1, dim).transpose(0, 1), rows(0).transpose(-1, -2)).mul_(1.0 / (math.sqrt(dim) * LN2))
    x.masked_fill_((torch.arange(n, device=q.device) >= lens[:, None])[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp2_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows(1)) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log2(l)).squeeze(-1)
    return out.transpose(0, 1).reshape(batch, heads, dim).to(q.dtype), lse.transpose(0, 1).reshape(batch, heads)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        import deepseek_sparse_attention_row_gb300 as dsa
    if s["op"] == "rotary":
        if own:
            return dsa.dsa_rotary(s["q"], s["k"], s["positions"], s["turns"], interleaved=s["interleaved"], factor=s["factor"], transpose=s["transpose"])
        return _plain_rotary(s)
    if s["op"] == "write":
        if own:
            dsa.dsa_quant_cache_write(s["k"], s["v"], s["cu"], s["cache"][0], s["cache"][1], s["scales"][0], s["scales"][1], s["tables"], s["lens"])
        else:
            _plain_write(s)
        return {"cache": s["cache"], "scales": s["scales"]}
    if s["op"] == "read":
        if own:
            return dsa.dsa_quant_cache_read(s["cache"][0], s["cache"][1], s["scales"][0], s["scales"][1], s["tables"], s["cu"], total=s["total"], dtype=s["dtype"])
        return _plain_read(s)
    if own:
        return dsa.dsa_quant_attention(s["q"], s["cache"][0], s["cache"][1], s["scales"][0], s["scales"][1], s["tables"], s["lens"])
    return _plain_attend(s)


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": n * c["dim"] * 2 * (4 if c["dtype"] == "fp32" else 2) + 4 * c["tokens"] + 4 * c["turning"], "flops": 3 * n * c["turning"]}
    row = 2 * c["kv_heads"] * c["dim"]  # elements of a token's key and value
    scale = 8 * c["kv_heads"]
    if c["op"] == "write":
        new, held = _ints(c["new"]), _ints(c["held"])
        blocks = sum((a + b - 1) // c["block"] - a // c["block"] + 1 for a, b in zip(held, new))
        return {"bytes": sum(new) * row * 3 + blocks * scale + 12 * len(new), "flops": 2 * sum(new) * row}
    lens = _ints(c["lens"])
    blocks = sum(-(-n // c["block"]) for n in lens)
    ints = 8 * len(lens) + 4 * sum(-(-n // c["page"]) for n in lens)
    if c["op"] == "read":
        return {"bytes": sum(lens) * row * 3 + blocks * scale + ints, "flops": sum(lens) * row}
    heads = len(lens) * c["kv_heads"] * c["group"]
    return {"bytes": sum(lens) * row + blocks * scale + ints + heads * (4 * c["dim"] + 4), "flops": 2 * row * c["group"] * sum(lens)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _nearest(y):
    """The e4m3 value next to y (|y| up to 448), the even one of two: four significant bits, steps of 2^-9 at the least."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -9))).clamp(min=-6.0) - 3)
    return torch.round(y / step) * step


def _least_power(x):
    """The least power of two not below x, from 2^-126 on."""
    e = torch.ceil(torch.log2(x.clamp(min=2.0 ** -126)))
    e = torch.where(torch.exp2(e - 1) >= x, e - 1, torch.where(torch.exp2(e) < x, e + 1, e))
    return torch.exp2(e.clamp(min=-126.0))


def _exact_rotary(s):
    n = 2 * len(s["frequencies"])
    angle = s["positions"].double()[:, None, None] * s["frequencies"] * (-1 if s["transpose"] else 1)
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle)
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double()
        first, second = (slice(0, n, 2), slice(1, n, 2)) if s["interleaved"] else (slice(0, n // 2), slice(n // 2, n))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rotary":
        return _exact_rotary(s)
    cache, scales = s["cache"].double(), s["scales"].double()
    page, block, tables = c["page"], c["block"], s["tables"].tolist()
    if c["op"] == "write":
        start = 0
        for i, (n, a) in enumerate(zip(_ints(c["new"]), _ints(c["held"]))):
            for b in range(a // block, (a + n - 1) // block + 1):
                lo, hi = max(a, b * block), min(a + n, (b + 1) * block)
                p, at = tables[i][b * block // page], b * block % page
                x = torch.stack([s[t][start + lo - a:start + hi - a] for t in "kv"]).double()
                fits = _least_power(x.abs().amax((1, 3)) / LARGEST)
                held = cache[:, p, at:at + lo - b * block]
                if lo > b * block:
                    was = scales[:, p, at // block].clone()
                    fits = torch.maximum(fits, was)
                    held.copy_(_nearest(held * (was / fits)[:, None, :, None]))
                scales[:, p, at // block] = fits
                cache[:, p, at + lo - b * block:at + hi - b * block] = _nearest(x / fits[:, None, :, None])
            start += n
        return {"cache": cache, "scales": scales}
    lens = _ints(c["lens"])
    if c["op"] == "attend" and sum(lens) * c["kv_heads"] * c["group"] * c["dim"] > 4e9:
        return None
    out, lses = [], []
    for i, n in enumerate(lens):
        ids = s["tables"][i, :-(-n // page)].long()
        k, v = ((cache[t][ids] * scales[t][ids].repeat_interleave(block, 1)[..., None]).reshape(-1, c["kv_heads"], c["dim"])[:n] for t in (0, 1))
        if c["op"] == "read":
            out.append(torch.stack((k, v)))
            continue
        x = torch.einsum("hgd,nhd->hgn", s["q"][i].double().view(c["kv_heads"], c["group"], c["dim"]), k) / math.sqrt(c["dim"])
        out.append(torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).flatten(0, 1))
        lses.append(torch.logsumexp(x, -1).flatten() / LN2)
    if c["op"] == "read":
        return tuple(torch.cat(out, 1))
    return torch.stack(out), torch.stack(lses)
