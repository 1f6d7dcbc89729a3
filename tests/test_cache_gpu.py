"""Forking, freeing and compacting cache pages against a plain sequential
model, entry by entry and byte by byte; and the whole serving round of prompt
attention, fork, decode and compaction."""

import math
import random

import numpy as np
import pytest

import attention_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_row_gb300 as dsa

    assert torch.cuda.is_available(), "these tests need a CUDA device"
    return torch, dsa


class Model:
    """The cache's state in numpy, changed one pair and one page at a time."""

    def __init__(self, cache, refs, tables, lens):
        self.cache, self.refs, self.tables, self.lens = cache, refs, tables, lens
        self.planes, self.pages, self.page = cache.shape[:3]

    def good(self, n):
        return 0 <= n < self.pages

    def fork(self, parents, children):
        old_tables, old_lens = self.tables.copy(), self.lens.copy()
        free = [n for n in range(self.pages) if self.refs[n] == 0]
        status, named, slots = [], set(), len(old_lens)
        for p, c in zip(parents, children):
            if not (0 <= p < slots and 0 <= c < slots) or c in named \
                    or old_lens[c] != 0 or old_tables[c, 0] >= 0:
                named.add(c)
                status.append(2)
                continue
            named.add(c)
            n = min(max(int(old_lens[p]), 0), old_tables.shape[1] * self.page)
            whole, rest = divmod(n, self.page)
            row = [-1] * old_tables.shape[1]
            row[:whole] = old_tables[p, :whole]
            if rest:
                src = old_tables[p, whole]
                if not self.good(src):
                    status.append(2)
                    continue
                if not free:
                    status.append(1)
                    continue
                row[whole] = free.pop(0)
                self.cache[:, row[whole], :rest] = self.cache[:, src, :rest]
            for x in row:
                if self.good(x):
                    self.refs[x] += 1
            self.tables[c] = row
            self.lens[c] = n
            status.append(0)
        return status

    def free(self, seqs):
        for s in set(seqs):
            if 0 <= s < len(self.lens):
                for x in self.tables[s]:
                    if self.good(x):
                        self.refs[x] = max(0, self.refs[x] - 1)
                self.tables[s] = -1
                self.lens[s] = 0

    def compact(self):
        used = [n for n in range(self.pages) if self.refs[n] > 0]
        holes = [n for n in range(len(used)) if self.refs[n] == 0]
        remap = np.full(self.pages, -1, np.int32)
        remap[used] = used
        for src, dst in zip([n for n in used if n >= len(used)], holes):
            remap[src] = dst
            self.cache[:, dst] = self.cache[:, src]
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for row in self.tables:
            for j, x in enumerate(row):
                if self.good(x):
                    row[j] = remap[x]
        return remap, len(used)


def build(torch, seed, planes=2, pages=40, page=4, slots=12, width=6, filled=6, token=(2, 8),
          dtype="int16"):
    """A state with `filled` sequences on random pages, and its model."""
    rng = np.random.default_rng(seed)
    cache = rng.integers(-30000, 30000, (planes, pages, page, *token)).astype(dtype)
    refs, lens = np.zeros(pages, np.int32), np.zeros(slots, np.int32)
    tables = np.full((slots, width), -1, np.int32)
    ids = list(rng.permutation(pages))
    for s in range(filled):
        lens[s] = rng.integers(0, width * page + 1)
        for j in range(-(-int(lens[s]) // page)):
            if not ids:
                lens[s] = j * page
                break
            tables[s, j] = ids.pop()
            refs[tables[s, j]] = 1
    return Model(cache, refs, tables, lens), [torch.from_numpy(x.copy()).cuda()
                                              for x in (cache, refs, tables, lens)]


def same(torch, m, t, what=""):
    torch.cuda.synchronize()
    for name, x, y in zip(("cache", "refs", "tables", "lens"), t,
                          (m.cache, m.refs, m.tables, m.lens)):
        np.testing.assert_array_equal(x.cpu().numpy(), y, err_msg=f"{what} {name}")


def ints(torch, values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def fork(env, m, t, parents, children):
    torch, dsa = env
    status = dsa.dsa_cache_fork(*t, ints(torch, parents), ints(torch, children))
    want = m.fork(parents, children)
    torch.cuda.synchronize()
    assert status.tolist() == want
    return want


def free(env, m, t, seqs):
    torch, dsa = env
    dsa.dsa_cache_free(*t[1:], ints(torch, seqs))
    m.free(seqs)


def compact(env, m, t):
    torch, dsa = env
    remap, live = dsa.dsa_cache_compact(*t[:3])
    want, n = m.compact()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(remap.cpu().numpy(), want)
    assert live.tolist() == [n]


@pytest.mark.parametrize("seed", range(12))
def test_random_rounds(env, seed):
    """Forks, frees and compactions in random order, with lists that name
    slots twice, out of range, full ones and empty parents."""
    torch, _ = env
    rng = random.Random(seed)
    slots = rng.choice([3, 12, 40])
    m, t = build(torch, seed, planes=rng.choice([1, 2, 5]), pages=rng.choice([1, 17, 40, 1500]),
                 page=rng.choice([1, 4, 16, 5]), slots=slots, width=rng.choice([1, 6, 300]),
                 filled=rng.randint(0, slots), token=rng.choice([(8,), (2, 8), (3, 1, 24)]))
    for i in range(15):
        n = rng.choice([0, 1, 3, 10])
        what = rng.choice(["fork", "fork", "free", "compact"])
        if what == "fork":
            fork(env, m, t, [rng.randint(-1, slots) for _ in range(n)],
                 [rng.randint(-1, slots) for _ in range(n)])
        elif what == "free":
            free(env, m, t, [rng.randint(-2, slots + 1) for _ in range(n)])
        else:
            compact(env, m, t)
        same(torch, m, t, f"step {i} {what}")


def test_fork_shares_whole_pages_and_copies_the_used_tokens(env):
    torch, _ = env
    m, t = build(torch, 1, filled=0)
    for x, y in ((m.tables, t[2]), (m.lens, t[3]), (m.refs, t[1])):
        if x is m.tables:
            x[0, :3] = [7, 30, 11]
        elif x is m.lens:
            x[0] = 10
        else:
            x[[7, 30, 11]] = 1
        y.copy_(torch.from_numpy(x))
    assert fork(env, m, t, [0, 0], [4, 2]) == [0, 0]
    same(torch, m, t)
    assert m.tables[4, :4].tolist() == [7, 30, 0, -1] and m.tables[2, :4].tolist() == [7, 30, 1, -1]
    assert m.refs[[7, 30, 11, 0, 1]].tolist() == [3, 3, 1, 1, 1]


def test_fork_runs_out_of_pages(env):
    torch, _ = env
    m, t = build(torch, 2, pages=9, page=4, slots=20, width=6, filled=0)
    m.tables[0, :3], m.lens[0] = [0, 4, 8], 9       # partly filled
    m.tables[1, :2], m.lens[1] = [1, 5], 8          # whole pages only
    m.refs[[0, 4, 8, 1, 5]] = 1
    for x, y in zip((m.refs, m.tables, m.lens), t[1:]):
        y.copy_(torch.from_numpy(x))
    got = fork(env, m, t, [0, 0, 1, 0, 0, 0, 1], [10, 11, 12, 13, 14, 15, 16])
    assert got == [0, 0, 0, 0, 0, 1, 0]
    same(torch, m, t)


def test_fork_many_pairs(env):
    """More pairs than a CTA has threads, more pages than one pass scans."""
    torch, _ = env
    m, t = build(torch, 3, planes=1, pages=9000, page=4, slots=5000, width=5, filled=300)
    rng = random.Random(3)
    parents = [rng.randrange(300) for _ in range(3000)]
    children = rng.sample(range(290, 5000), 3000)
    fork(env, m, t, parents, children)
    same(torch, m, t, "fork")
    free(env, m, t, list(range(0, 5000, 3)))
    same(torch, m, t, "free")
    compact(env, m, t)
    same(torch, m, t, "compact")


def test_tables_with_entries_out_of_range(env):
    """Never followed: shared and cleared like -1, and a parent whose partial
    page is missing is refused."""
    torch, _ = env
    m, t = build(torch, 4, pages=20, page=4, slots=8, width=6, filled=0)
    m.tables[0, :4], m.lens[0] = [20, 3, -5, 6], 14
    m.tables[1, :2], m.lens[1] = [2 ** 31 - 1, 99], 6
    m.tables[2, :1], m.lens[2] = [9], 10 ** 6       # longer than its table
    m.refs[[3, 6, 9]] = 1
    for x, y in zip((m.refs, m.tables, m.lens), t[1:]):
        y.copy_(torch.from_numpy(x))
    assert fork(env, m, t, [0, 1, 2], [5, 6, 7]) == [0, 2, 0]
    same(torch, m, t, "fork")
    compact(env, m, t)
    same(torch, m, t, "compact")
    free(env, m, t, [0, 5, 1, 7, 2, 2])
    same(torch, m, t, "free")
    assert m.refs.sum() == 0


def test_strided_state(env):
    """Planes and pages with gaps, tables as a slice of a wider tensor."""
    torch, _ = env
    m, t = build(torch, 5, planes=3, pages=30, slots=10, filled=5)
    planes, pages, page = m.cache.shape[:3]
    pool = torch.full((planes + 1, pages + 2, 2 * page, 2, 8), 77, dtype=torch.int16, device="cuda")
    view = pool[1:, 2:, :page]
    view.copy_(t[0])
    wide = torch.full((10, 11), -9, dtype=torch.int32, device="cuda")
    wide[:, 3:9] = t[2]
    s = [view, t[1], wide[:, 3:9], t[3]]
    fork(env, m, s, [0, 1, 2, 3], [5, 6, 7, 8])
    free(env, m, s, [1, 3])
    compact(env, m, s)
    same(torch, m, s)
    assert (wide[:, :3] == -9).all() and (wide[:, 9:] == -9).all()
    assert (pool[0] == 77).all() and (pool[:, :2] == 77).all() and (pool[:, :, page:] == 77).all()


@pytest.mark.parametrize("dtype", ["float32", "uint8", "bfloat16"])
def test_element_types(env, dtype):
    torch, _ = env
    m, t = build(torch, 6, token=(4, 8), dtype="int32")
    bits = t[0].view(torch.uint8).view(getattr(torch, dtype))
    s = [bits, *t[1:]]
    fork(env, m, s, [0, 1, 2, 3, 4], [7, 8, 9, 10, 11])
    free(env, m, s, [0, 2, 8])
    compact(env, m, s)
    same(torch, m, t)


def test_captured_round(env):
    """A captured round of free, fork and compaction, replayed."""
    torch, dsa = env
    m, t = build(torch, 7, planes=2, pages=60, slots=14, filled=6)
    parents, children, gone = [0, 1, 2, 3, 4], [6, 7, 8, 9, 10], [6, 7, 8, 9, 10]
    dev = [ints(torch, x) for x in (parents, children, gone)]
    fork(env, m, t, parents, children)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_cache_free(*t[1:], dev[2])
        status = dsa.dsa_cache_fork(*t, dev[0], dev[1])
        remap, live = dsa.dsa_cache_compact(*t[:3])
    for _ in range(3):
        g.replay()
        m.free(gone)
        want = m.fork(parents, children)
        moved = m.compact()
        torch.cuda.synchronize()
        assert status.tolist() == want and live.tolist() == [moved[1]]
        np.testing.assert_array_equal(remap.cpu().numpy(), moved[0])
        same(torch, m, t)
        # other parents of the same length, through the same addresses
        parents.reverse()
        dev[0].copy_(ints(torch, parents))


def test_other_stream(env):
    torch, dsa = env
    m, t = build(torch, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    parents, children = ints(torch, [0, 1, 2]), ints(torch, [7, 8, 9])
    s.wait_stream(torch.cuda.current_stream())
    status = dsa.dsa_cache_fork(*t, parents, children, stream=s)
    dsa.dsa_cache_free(*t[1:], parents, stream=s)
    dsa.dsa_cache_compact(*t[:3], stream=s)
    s.synchronize()
    assert status.tolist() == m.fork([0, 1, 2], [7, 8, 9])
    m.free([0, 1, 2])
    m.compact()
    same(torch, m, t)


def test_nothing_to_do(env):
    torch, dsa = env
    m, t = build(torch, 9)
    none = ints(torch, [])
    assert dsa.dsa_cache_fork(*t, none, none).shape == (0,)
    dsa.dsa_cache_free(*t[1:], none)
    same(torch, m, t)
    cache = torch.zeros((2, 0, 4, 8), dtype=torch.int16, device="cuda")
    tables = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    remap, live = dsa.dsa_cache_compact(cache, none, tables)
    torch.cuda.synchronize()
    assert remap.shape == (0,) and live.tolist() == [0] and (tables == -1).all()


def test_serving_round(env):
    """Prompts of two requests run through prompt attention and go into the
    cache; the first is forked into samples that share its whole pages; each
    sample appends a token and decodes; a sample is dropped, the cache is
    compacted, and decoding gives the same bits from the moved pages."""
    torch, dsa = env
    H, Hkv, D, page, N, slots, width = 8, 2, 64, 16, 40, 8, 8
    g = torch.Generator().manual_seed(3)
    ql = [75, 40]
    T = sum(ql)
    q = (torch.randn(T, H, D, generator=g) * 1.5).bfloat16().cuda()
    k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    cu = ints(torch, [0, 75, 115])
    out, lse = dsa.dsa_prompt_attention(q, k, v, cu, cu)
    want = ref.prompt(q, k, v, [0, 75, 115], [0, 75, 115], True)
    torch.cuda.synchronize()
    ref.check(out, want[0], want[2], "prompt out")
    ref.check(lse, want[1], want[3], "prompt lse")

    cache = torch.full((2, N, page, Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda")
    refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    tables = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
    at = 0
    for s, ids in ((0, [31, 4, 22, 9, 17]), (1, [5, 38, 0])):
        tables[s, :len(ids)] = ints(torch, ids)
        refs[torch.tensor(ids, device="cuda")] = 1
        lens[s] = ql[s]
        for t in range(ql[s]):
            cache[0, ids[t // page], t % page] = k[at + t]
            cache[1, ids[t // page], t % page] = v[at + t]
        at += ql[s]
    # the last query of each prompt, decoded from the cache: the same attention
    last = torch.tensor([74, 114], device="cuda")
    dec, dec_lse = dsa.dsa_shared_prefix_attention(q[last], cache[0], cache[1], tables[:2],
                                                   lens[:2])
    torch.cuda.synchronize()
    ref.check(dec, want[0][last.cpu()], want[2][last.cpu()], "decode out")
    ref.check(dec_lse, want[1][last.cpu()], want[3][last.cpu()], "decode lse")

    kids = [2, 3, 4, 5]
    status = dsa.dsa_cache_fork(cache, refs, tables, lens, ints(torch, [0] * 4),
                                ints(torch, kids))
    assert status.tolist() == [0] * 4
    new = torch.randn(2, 4, Hkv, D, generator=g).bfloat16().cuda()
    rows = torch.tensor(kids, device="cuda")
    cache[:, tables[rows, 75 // page].long(), 75 % page] = new
    lens[rows] += 1
    tok = (torch.randn(4, H, D, generator=g) * 1.5).bfloat16().cuda()

    def decode(slots):
        i = torch.tensor(slots, device="cuda")
        pick = torch.tensor([kids.index(s) for s in slots], device="cuda")
        got = dsa.dsa_shared_prefix_attention(tok[pick], cache[0], cache[1], tables[i], lens[i],
                                              64)
        torch.cuda.synchronize()
        w = ref.paged(tok[pick], cache[0], cache[1], tables[i], lens[i], tables[i[0]], 64)
        ref.check(got[0], w[0], w[2], "sample out")
        ref.check(got[1], w[1], w[3], "sample lse")
        return got

    first = decode(kids)
    dsa.dsa_cache_free(refs, tables, lens, ints(torch, [0, 3]))
    left = decode([2, 4, 5])
    assert torch.equal(left[0], first[0][[0, 2, 3]])
    remap, live = dsa.dsa_cache_compact(cache, refs, tables)
    torch.cuda.synchronize()
    assert live.tolist() == [4 + 3 + 3]      # shared pages, own pages, the second prompt's
    assert int(tables.max()) == 9
    moved = decode([2, 4, 5])
    assert torch.equal(left[0], moved[0]) and torch.equal(left[1], moved[1])
