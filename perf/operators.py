"""The attention and cache operators as a serving program runs them: cases, inputs, one pass, and the work of a pass.

Operators: attention over whole packed prompts, decode attention for a batch that shares a long prefix on a paged cache, and the forking, freeing
and compacting of that cache's pages. ``own`` false computes them with elementary torch operations in fp32, ``own`` true calls the library."""

import math

import torch

own = False

LN2 = math.log(2.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _ints(text):
    return [int(x) for x in text.split(",")]


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A handful of short prompts, one of them a single token: latency.
        {"name": "prompt_short", "op": "prompt", "q": "1,33,7", "k": "1,33,20", "kv_heads": 2, "group": 4, "dim": 64, "dtype": "bf16", "causal": True},
        # A ragged batch attending in full to keys of other lengths (an earlier context shard, merged by LSE later); odd group and head dim.
        {"name": "prompt_ragged", "op": "prompt", "q": "37,1900,512,1,255,1024,129,700", "k": "1037,1900,2048,777,31,1500,129,3500", "kv_heads": 4, "group": 3,
         "dim": 96, "dtype": "fp16", "causal": False},
        # The packed prefill chunk: 4 requests of 2048 query tokens behind cached prefixes.
        {"name": "prompt_chunk", "op": "prompt", "q": "2048,2048,2048,2048", "k": "8192,6201,2048,4100", "kv_heads": 8, "group": 4, "dim": 128, "dtype": "bf16",
         "causal": True},
        # One long prompt.
        {"name": "prompt_long", "op": "prompt", "q": "16389", "k": "16389", "kv_heads": 2, "group": 8, "dim": 128, "dtype": "bf16", "causal": True},
        # A few sequences behind a short system prompt: latency.
        {"name": "shared_small", "op": "shared", "batch": 3, "prefix": 160, "own": 40, "page": 16, "kv_heads": 2, "group": 4, "dim": 64, "dtype": "bf16"},
        # Nothing shared: plain paged decode; odd group and head dim.
        {"name": "shared_none", "op": "shared", "batch": 33, "prefix": 0, "own": 8000, "page": 32, "kv_heads": 8, "group": 5, "dim": 80, "dtype": "fp16"},
        # A chat batch behind a long system prompt.
        {"name": "shared_chat", "op": "shared", "batch": 64, "prefix": 8192, "own": 1024, "page": 64, "kv_heads": 8, "group": 4, "dim": 128, "dtype": "bf16"},
        # Many samples from one long document.
        {"name": "shared_document", "op": "shared", "batch": 128, "prefix": 32768, "own": 2048, "page": 128, "kv_heads": 4, "group": 8, "dim": 128,
         "dtype": "bf16"},
        # Beams dropped and forked anew, a small cache: latency of the bookkeeping.
        {"name": "fork_small", "op": "fork", "parents": 4, "children": 4, "length": 90, "page": 16, "planes": 4, "kv_heads": 2, "dim": 64},
        # The same for a serving cache (8 layers of keys and values).
        {"name": "fork_beams", "op": "fork", "parents": 64, "children": 256, "length": 1000, "page": 64, "planes": 16, "kv_heads": 8, "dim": 128},
        # A beam step whose dropped beams leave holes, then a compaction.
        {"name": "compact_small", "op": "compact", "parents": 4, "children": 4, "length": 90, "page": 16, "planes": 4, "kv_heads": 2, "dim": 64},
        {"name": "compact_beams", "op": "compact", "parents": 64, "children": 128, "length": 1000, "page": 64, "planes": 16, "kv_heads": 8, "dim": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "shared", "shared", "shared", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim = rng.choice([64, 128, 128, 8 * rng.randint(4, 16)])
    if op == "prompt":
        causal = rng.random() < 0.7
        count = _log(rng, 1, 9)
        q = [_log(rng, 1, 16000 // count) for _ in range(count)]
        k = [n + (0 if rng.random() < 0.5 else _log(rng, 1, 4000)) for n in q] if causal else [_log(rng, 1, 16000 // count) for _ in range(count)]
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        kv_heads = rng.choice([1, 2, 4, 8])
        while kv_heads * group * max(q) * max(k) * count > 8 * 2 ** 30 or kv_heads * group * sum(a * b for a, b in zip(q, k)) * dim > 16 * 128 * 16389 ** 2 // 2:
            q, k = [max(1, n // 2) for n in q], [max(1, n // 2) for n in k]
            if causal:
                k = [max(a, b) for a, b in zip(q, k)]
        return {"op": op, "q": ",".join(map(str, q)), "k": ",".join(map(str, k)), "kv_heads": kv_heads, "group": group, "dim": dim, "dtype": dtype,
                "causal": causal}
    if op == "shared":
        page = rng.choice([16, 32, 64, 128])
        return {"op": op, "batch": _log(rng, 1, 128), "prefix": 0 if rng.random() < 0.15 else page * max(1, _log(rng, 64, 32768) // page), "own": _log(rng, 2, 2048),
                "page": page, "kv_heads": rng.choice([1, 2, 4]), "group": rng.choice([1, 2, 3, 4, 6, 8]), "dim": dim, "dtype": dtype}
    parents = _log(rng, 1, 64)
    return {"op": op, "parents": parents, "children": _log(rng, 1, 128), "length": _log(rng, 20, 1000), "page": rng.choice([16, 32, 64]), "planes": 2 * rng.randint(1, 8),
            "kv_heads": rng.choice([1, 2, 4, 8]), "dim": dim}


def _own_lens(c):
    """Own tokens of every sequence: spread over 1..own."""
    return [1 + (i * 7919 + 13) % c["own"] for i in range(c["batch"])]


def _parent_lens(c):
    """Lengths around `length`, nearly all ending inside a page."""
    return [max(1, c["length"] - (i * 37) % (1 + c["length"] // 2)) for i in range(c["parents"])]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _dev(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = case
    s = {"op": c["op"]}
    if c["op"] == "prompt":
        ql, kl = _ints(c["q"]), _ints(c["k"])
        heads, dt = c["kv_heads"] * c["group"], DTYPES[c["dtype"]]
        s["q"] = _randn(g, (sum(ql), heads, c["dim"]), dt, 1.5)
        s["k"] = _randn(g, (sum(kl), c["kv_heads"], c["dim"]), dt)
        s["v"] = _randn(g, (sum(kl), c["kv_heads"], c["dim"]), dt)
        s["cu_q"] = _dev([sum(ql[:i]) for i in range(len(ql) + 1)])
        s["cu_k"] = _dev([sum(kl[:i]) for i in range(len(kl) + 1)])
        s["max_q"], s["max_k"], s["causal"] = max(ql), max(kl), c["causal"]
        return s
    if c["op"] == "shared":
        dt, page, batch = DTYPES[c["dtype"]], c["page"], c["batch"]
        own_lens = _own_lens(c)
        pre, most = c["prefix"] // page, -(-c["own"] // page)
        pages = pre + sum(-(-n // page) for n in own_lens)
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
        tables, at = [], pre
        for n in own_lens:
            need = -(-n // page)
            tables.append(ids[:pre] + ids[at:at + need] + [-1] * (most - need))
            at += need
        s["cache"] = _randn(g, (2, pages, page, c["kv_heads"], c["dim"]), dt)
        s["tables"] = _dev(tables)
        s["lens"] = _dev([c["prefix"] + n for n in own_lens])
        s["q"] = _randn(g, (batch, c["kv_heads"] * c["group"], c["dim"]), dt, 1.5)
        s["prefix"] = c["prefix"]
        return s
    # fork and compact: parents on scattered pages, empty slots for the children
    page, lens = c["page"], _parent_lens(c)
    slots = c["parents"] + (1 if c["op"] == "fork" else 2) * c["children"]
    width = -(-max(lens) // page) + 1
    used = sum(-(-n // page) for n in lens)
    pages = used + 2 * c["children"] + 5
    # the parents' pages leave holes of random places among the low ids
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    tables, at = [], 0
    for n in lens:
        need = -(-n // page)
        tables.append(ids[at:at + need] + [-1] * (width - need))
        at += need
    tables += [[-1] * width] * (slots - c["parents"])
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[torch.tensor(ids[:used], device="cuda")] = 1
    s["cache"] = torch.randn((c["planes"], pages, page, c["kv_heads"], c["dim"]), generator=g, device="cuda", dtype=torch.bfloat16)
    s["refs"], s["tables"] = refs, _dev(tables)
    s["lens"] = _dev(lens + [0] * (slots - c["parents"]))
    pick = torch.randint(0, c["parents"], (2, c["children"]), generator=g, device="cuda", dtype=torch.int32)
    s["parents"], s["others"] = pick[0].contiguous(), pick[1].contiguous()
    first = c["parents"] + c["children"]
    s["first"] = torch.arange(c["parents"], first, dtype=torch.int32, device="cuda")
    s["second"] = torch.arange(first, first + c["children"], dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _attend(q, k, v, see, scale):
    """q [..., m, D], k and v [..., n, D] fp32, see broadcasts to [..., m, n]: output, and the base-2 log-sum-exp."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale / LN2)
    x.masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp2_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    return out, (m + torch.log2(l)).squeeze(-1)


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    (tq, heads, dim), kv_heads = q.shape, k.shape[1]
    group = heads // kv_heads
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    ql, kl, count = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1], len(cu_q) - 1
    at_q, at_k = torch.arange(s["max_q"], device=q.device), torch.arange(s["max_k"], device=q.device)
    iq = (cu_q[:-1, None] + at_q).clamp_(max=tq - 1)
    ik = (cu_k[:-1, None] + at_k).clamp_(max=k.shape[0] - 1)
    # [seq, kv head, group * token, dim]
    pq = q.float()[iq].view(count, s["max_q"], kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(count, kv_heads, group * s["max_q"], dim)
    pk, pv = (t.float()[ik].permute(0, 2, 1, 3).contiguous() for t in (k, v))
    lim = kl[:, None].expand(-1, s["max_q"])
    if s["causal"]:
        lim = at_q + 1 + (kl - ql)[:, None]
    see = (at_k < torch.minimum(lim, kl[:, None])[..., None])[:, None].repeat(1, 1, group, 1)
    out, lse = _attend(pq, pk, pv, see, 1.0 / math.sqrt(dim))
    out = out.view(count, kv_heads, group, s["max_q"], dim)
    lse = lse.view(count, kv_heads, group, s["max_q"])
    tok = torch.arange(tq, device=q.device)
    seq = torch.searchsorted(cu_q[1:], tok, right=True)
    pos = tok - cu_q[seq]
    return out[seq, :, :, pos].reshape(tq, heads, dim).to(q.dtype), lse[seq, :, :, pos].reshape(tq, heads)


def _plain_shared(s):
    q, (k_pages, v_pages) = s["q"], s["cache"]
    batch, heads, dim = q.shape
    _, page, kv_heads, _ = k_pages.shape
    group, pre = heads // kv_heads, s["prefix"] // page
    scale = 1.0 / math.sqrt(dim)
    rows = q.float().view(batch, kv_heads, group, dim).transpose(0, 1)
    parts = []
    if pre:
        ids = s["tables"][0, :pre].long()
        k, v = (t[ids].float().reshape(pre * page, kv_heads, dim).transpose(0, 1).contiguous() for t in (k_pages, v_pages))
        see = torch.arange(pre * page, device=q.device) < s["lens"][:, None]
        out, lse = _attend(rows.reshape(kv_heads, batch * group, dim), k, v, see.repeat_interleave(group, 0), scale)
        parts.append((out.view(kv_heads, batch, group, dim), lse.view(kv_heads, batch, group)))
    ids = s["tables"][:, pre:].long().clamp(min=0)
    n = ids.shape[1] * page
    k, v = (t[ids].float().reshape(batch, n, kv_heads, dim).permute(2, 0, 1, 3).contiguous() for t in (k_pages, v_pages))
    see = torch.arange(n, device=q.device) < (s["lens"] - s["prefix"])[:, None]
    parts.append(_attend(rows, k, v, see[:, None], scale))
    lses = torch.stack([p[1] for p in parts])
    m = lses.amax(0)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    shares = torch.exp2(lses - m)
    total = shares.sum(0)
    out = (torch.stack([p[0] for p in parts]) * (shares / total.clamp(min=1e-38))[..., None]).sum(0)
    lse = m + torch.log2(total)
    return out.transpose(0, 1).reshape(batch, heads, dim).to(q.dtype), lse.transpose(0, 1).reshape(batch, heads)


def _plain_free(s, seqs):
    refs, tables, lens = s["refs"], s["tables"], s["lens"]
    go = torch.zeros(len(lens), dtype=torch.bool, device=refs.device)
    go[seqs.long()] = True
    ids = torch.where(go[:, None] & (tables >= 0), tables, len(refs)).long().flatten()
    gone = torch.zeros(len(refs) + 1, dtype=torch.int32, device=refs.device)
    gone.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    refs.sub_(gone[:-1]).clamp_(min=0)
    tables.masked_fill_(go[:, None], -1)
    lens.masked_fill_(go, 0)


def _plain_fork(s, parents, children):
    """Status of every child: 0 forked, 1 no page left, 2 refused."""
    cache, refs, tables, lens = s["cache"], s["refs"], s["tables"], s["lens"]
    page, p, c = cache.shape[2], parents.long(), children.long()
    ok = (lens[c] == 0) & (tables[c, 0] < 0)
    whole, rest = lens[p] // page, lens[p] % page
    src = tables[p].gather(1, whole.long()[:, None].clamp(max=tables.shape[1] - 1))[:, 0]
    need = ok & (rest > 0)
    rank = need.int().cumsum(0) - need.int()
    free = torch.argsort((refs != 0).int(), stable=True)
    full = need & (rank >= (refs == 0).sum())
    status = torch.where(ok, full.int(), 2).int()
    done, need = status == 0, need & ~full
    at = torch.arange(tables.shape[1], device=refs.device)
    row = torch.where(at < whole[:, None], tables[p], -1)
    fresh = free[rank.long()].int()
    row = torch.where((at == whole[:, None]) & need[:, None], fresh[:, None], row)
    ids = torch.where(done[:, None] & (row >= 0), row, len(refs)).long().flatten()
    more = torch.zeros(len(refs) + 1, dtype=torch.int32, device=refs.device)
    more.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    refs.add_(more[:-1])
    tables[c[done]] = row[done]
    lens[c[done]] = lens[p[done]]
    to, of, n = fresh[need].long(), src[need].long(), rest[need]
    old = cache[:, to]
    used = (torch.arange(page, device=refs.device) < n[:, None])[None, :, :, None, None]
    cache[:, to] = torch.where(used, cache[:, of], old)
    return status


def _plain_compact(s):
    cache, refs, tables = s["cache"], s["refs"], s["tables"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(len(refs), device=refs.device)
    movers, holes = (live & (at >= count)).nonzero()[:, 0], (~live & (at < count)).nonzero()[:, 0]
    remap = torch.where(live, at, -1).int()
    remap[movers] = holes.int()
    cache[:, holes] = cache[:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    tables.copy_(torch.where(tables >= 0, remap[tables.clamp(min=0).long()], tables))
    return remap, count.int().view(1)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        import deepseek_sparse_attention_row_gb300 as dsa
    if s["op"] == "prompt":
        if own:
            return dsa.dsa_prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"])
        return _plain_prompt(s)
    if s["op"] == "shared":
        if own:
            return dsa.dsa_shared_prefix_attention(s["q"], s["cache"][0], s["cache"][1], s["tables"], s["lens"], s["prefix"])
        return _plain_shared(s)
    if own:
        def free(seqs):
            dsa.dsa_cache_free(s["refs"], s["tables"], s["lens"], seqs)

        def fork(parents, children):
            return dsa.dsa_cache_fork(s["cache"], s["refs"], s["tables"], s["lens"], parents, children)
    else:
        def free(seqs):
            _plain_free(s, seqs)

        def fork(parents, children):
            return _plain_fork(s, parents, children)
    if s["op"] == "fork":
        # a beam step: the last step's children are dropped, new ones forked
        free(s["first"])
        status = fork(s["parents"], s["first"])
        return {"status": status, "refs": s["refs"], "tables": s["tables"], "lens": s["lens"], "cache": s["cache"]}
    # the same with two sets of children, the first of which is dropped again and leaves holes below the second's pages
    free(s["second"])
    one = fork(s["parents"], s["first"])
    two = fork(s["others"], s["second"])
    free(s["first"])
    remap, live = dsa.dsa_cache_compact(s["cache"], s["refs"], s["tables"]) if own else _plain_compact(s)
    return {"one": one, "two": two, "remap": remap, "live": live, "refs": s["refs"], "tables": s["tables"], "lens": s["lens"], "cache": s["cache"]}


def work(case):
    c = case
    if c["op"] == "prompt":
        ql, kl, heads = _ints(c["q"]), _ints(c["k"]), c["kv_heads"] * c["group"]
        pairs = sum(sum(max(0, min(b, i + 1 + b - a)) for i in range(a)) if c["causal"] else a * b for a, b in zip(ql, kl))
        return {"bytes": 4 * c["dim"] * (heads * sum(ql) + c["kv_heads"] * sum(kl)) + 4 * heads * sum(ql), "flops": 4 * c["dim"] * heads * pairs}
    if c["op"] == "shared":
        lens, heads = _own_lens(c), c["kv_heads"] * c["group"]
        return {"bytes": 4 * c["dim"] * (c["kv_heads"] * (c["prefix"] + sum(lens)) + heads * c["batch"]) + 4 * heads * c["batch"],
                "flops": 4 * c["dim"] * heads * (c["batch"] * c["prefix"] + sum(lens))}
    # Copied bytes, read and written. Each child gets the used tokens of a page (on average half a page); a compaction also moves whole pages: about
    # one for each of the second set of children. Page counts and the tables of the children are read and written.
    token = 2 * c["kv_heads"] * c["dim"] * c["planes"]
    part = sum(n % c["page"] for n in _parent_lens(c)) / c["parents"]
    pages = sum(-(-n // c["page"]) for n in _parent_lens(c)) + 2 * c["children"] + 5
    ints = 8 * pages + 8 * c["children"] * (2 + -(-c["length"] // c["page"]))
    copied = c["children"] * part if c["op"] == "fork" else c["children"] * (2 * part + c["page"])
    return {"bytes": 2 * token * copied + ints, "flops": 0}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _softmax64(q, k, v, seen):
    """Rows of one head against its keys: row i attends to the first seen[i] keys. Natural exponentials; the LSE is turned to base 2 at the end."""
    out = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    for a in range(0, q.shape[0], 4096):
        n = seen[a:a + 4096]
        top = int(n.max())
        if top <= 0:
            continue
        x = q[a:a + 4096] @ k[:top].T / math.sqrt(q.shape[1])
        x[torch.arange(top, device=q.device)[None, :] >= n[:, None]] = -math.inf
        z = torch.logsumexp(x, 1)
        some = n > 0
        w = torch.exp(x - torch.where(some, z, torch.zeros_like(z))[:, None])
        out[a:a + 4096] = w @ v[:top]
        lse[a:a + 4096] = torch.where(some, z / LN2, lse[a:a + 4096])
    return out, lse


def exact(case, seed):
    c = case
    if c["op"] not in ("prompt", "shared"):
        return None
    s = prepare(c, seed)
    q = s["q"].double()
    heads, group = q.shape[1], c["group"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    if c["op"] == "prompt":
        if work(c)["flops"] > 6e12:
            return None
        a = b = 0
        for nq, nk in zip(_ints(c["q"]), _ints(c["k"])):
            seen = torch.full((nq,), nk, device=q.device)
            if c["causal"]:
                seen = (torch.arange(nq, device=q.device) + 1 + nk - nq).clamp(0, nk)
            for h in range(heads):
                k, v = (s[t][b:b + nk, h // group].double() for t in ("k", "v"))
                out[a:a + nq, h], lse[a:a + nq, h] = _softmax64(q[a:a + nq, h], k, v, seen)
            a, b = a + nq, b + nk
        return out, lse
    lens = [c["prefix"] + n for n in _own_lens(c)]
    for i, n in enumerate(lens):
        ids = s["tables"][i, :-(-n // c["page"])].long()
        k, v = (t[ids].reshape(-1, c["kv_heads"], c["dim"])[:n].double() for t in s["cache"])
        x = torch.einsum("hgd,nhd->hgn", q[i].view(-1, group, c["dim"]), k) / math.sqrt(c["dim"])
        out[i] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(heads, -1)
        lse[i] = torch.logsumexp(x, -1).reshape(heads) / LN2
    return out, lse
