"""Prompt attention and shared-prefix decode attention against their
definition in 64 bits, within the bound of tests/attention_reference.py."""

import math

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
    yield torch, dsa
    torch.cuda.synchronize()
    assert dsa.attention_error() == 0, "a kernel's wait gave up"


def ints(torch, values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def make(torch, seed, tokens, keys, heads, kv_heads, dim, dtype, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(tokens, heads, dim, generator=g) * spread).to(dtype).cuda()
    k, v = (torch.randn(keys, kv_heads, dim, generator=g).to(dtype).cuda() for _ in range(2))
    return q, k, v


def check_prompt(env, q, k, v, ql, kl, causal, scale=None, **kw):
    torch, dsa = env
    cu_q, cu_k = offsets(ql), offsets(kl)
    out, lse = dsa.dsa_prompt_attention(q, k, v, ints(torch, cu_q), ints(torch, cu_k),
                                        causal=causal, scale=scale, **kw)
    torch.cuda.synchronize()
    want = ref.prompt(q, k, v, cu_q, cu_k, causal, scale)
    n = cu_q[-1]
    ref.check(out[:n], want[0][:n], want[2][:n], "out")
    ref.check(lse[:n], want[1][:n], want[3][:n], "lse")
    return out, lse


LENGTHS = [  # queries, keys
    ([1], [1]),
    ([5, 0, 1, 33], [5, 7, 1, 33]),
    ([127, 128, 129], [127, 128, 129]),
    ([64, 130], [400, 131]),
    ([257, 1, 300], [300, 513, 17]),      # the last sequence's first rows see nothing
    ([40, 3, 0, 9], [0, 200, 0, 4]),      # a sequence without keys
]
SHAPES = [  # heads, kv heads, head dim
    (4, 4, 64), (8, 2, 128), (6, 2, 96), (5, 1, 40), (16, 1, 8), (7, 1, 120), (24, 2, 72),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", LENGTHS, ids=[str(x) for x in LENGTHS])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(x) for x in SHAPES])
def test_prompt_sweep(env, shape, lengths, causal, dtype):
    torch, _ = env
    ql, kl = lengths
    q, k, v = make(torch, 7 * sum(ql) + shape[2], sum(ql), sum(kl), *shape, getattr(torch, dtype))
    check_prompt(env, q, k, v, ql, kl, causal)


@pytest.mark.parametrize("heads,kv_heads,dim", [(64, 1, 64), (128, 1, 16), (100, 1, 128),
                                                (33, 1, 64)])
def test_prompt_wide_groups(env, heads, kv_heads, dim):
    torch, _ = env
    q, k, v = make(torch, heads, 23, 150, heads, kv_heads, dim, torch.bfloat16)
    check_prompt(env, q, k, v, [20, 3], [147, 3], True)


def test_prompt_runs_of_sequences_without_keys(env):
    """More of them in a row than a CTA plans ahead, between others."""
    torch, _ = env
    ql = [40] + [9] * 4000 + [130] + [1] * 30 + [20]
    kl = [40] + [0] * 4000 + [130] + [0] * 30 + [25]
    q, k, v = make(torch, 21, sum(ql), sum(kl), 2, 1, 64, torch.bfloat16)
    check_prompt(env, q, k, v, ql, kl, True)
    check_prompt(env, q, k, v, ql, kl, False)


def test_prompt_longer_keys(env):
    """Many key tiles per row, so that the running maximum moves often."""
    torch, _ = env
    q, k, v = make(torch, 3, 70, 5000, 4, 2, 128, torch.bfloat16)
    k *= torch.linspace(0.2, 2.5, 5000, device="cuda").to(k.dtype)[:, None, None]
    check_prompt(env, q, k, v, [70], [5000], True)
    check_prompt(env, q, k, v, [69, 1], [1500, 3500], False)


@pytest.mark.parametrize("scale", [1e-3, 0.125, 3.0])
def test_prompt_scale(env, scale):
    torch, _ = env
    q, k, v = make(torch, 11, 150, 150, 4, 2, 64, torch.bfloat16, spread=1.0)
    check_prompt(env, q, k, v, [150], [150], True, scale)


@pytest.mark.parametrize("scale", [2e-38, 1e-30])
def test_scales_that_make_all_keys_equal(env, scale):
    """8 / (scale log2 e) overflows for the first: the base has to move all the
    same, and the sums are those of equal weights."""
    torch, _ = env
    q, k, v = make(torch, 36, 40, 300, 4, 2, 64, torch.bfloat16)
    check_prompt(env, q, k, v, [40], [300], True, scale)
    p = make_paged(torch, 37, 3, 4, 2, 64, 16, 32, [20, 0, 150], torch.bfloat16)
    check_paged(env, *p, 32, scale=scale)


def test_prompt_strided(env):
    """Views: a fused [T, H + 2 Hkv, D] projection, head-major tensors, padded
    heads; outputs into views, the bytes around them untouched."""
    torch, dsa = env
    T, H, Hkv, D = 140, 6, 2, 64
    g = torch.Generator().manual_seed(5)
    fused = torch.randn(T, H + 2 * Hkv, D, generator=g).bfloat16().cuda()
    q, k, v = fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]
    want, want_lse = check_prompt(env, q, k, v, [100, 40], [100, 40], True)
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    wide = torch.full((T, H, D + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    lses = torch.full((H, T + 3), 5.0, device="cuda")
    dsa.dsa_prompt_attention(*hm, ints(torch, [0, 100, 140]), ints(torch, [0, 100, 140]),
                             out=wide[..., 8:8 + D], lse_out=lses[:, :T].t())
    torch.cuda.synchronize()
    assert torch.equal(wide[..., 8:8 + D], want)
    assert (wide[..., :8] == 7).all() and (wide[..., 8 + D:] == 7).all()
    assert torch.equal(lses[:, :T].t(), want_lse) and (lses[:, T:] == 5).all()


def test_prompt_one_token_views(env):
    """Dimensions of one element may have any stride."""
    torch, _ = env
    q, k, v = make(torch, 6, 1, 9, 1, 1, 64, torch.bfloat16)
    odd = torch.as_strided(q, (1, 1, 64), (3, 5, 1))
    check_prompt(env, odd, k, v, [1], [9], True)


def test_broadcast_heads(env):
    """One key/value head expanded to several (a stride of 0)."""
    torch, dsa = env
    q, k, v = make(torch, 33, 90, 150, 4, 1, 64, torch.bfloat16)
    ke, ve = k.expand(-1, 2, -1), v.expand(-1, 2, -1)
    want, want_lse = check_prompt(env, q, k.repeat(1, 2, 1), v.repeat(1, 2, 1), [90], [150], True)
    out, lse = dsa.dsa_prompt_attention(q, ke, ve, ints(torch, [0, 90]), ints(torch, [0, 150]))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_attention_gpu as t
import deepseek_sparse_attention_row_gb300 as dsa
q, k, v = t.make(torch, 40, 100, 3000, 8, 2, 128, torch.bfloat16)
cu_q, cu_k = t.ints(torch, [0, 100]), t.ints(torch, [0, 3000])
p = t.make_paged(torch, 41, 5, 8, 2, 64, 16, 32, [3, 0, 40, 17, 90], torch.bfloat16)
c = torch.zeros(2, 9, 16, 8, dtype=torch.bfloat16, device="cuda")
refs = t.ints(torch, [1] + [0] * 8)
tables, lens = t.ints(torch, [[0, -1], [-1, -1]]), t.ints(torch, [5, 0])
who, kid = t.ints(torch, [0]), t.ints(torch, [1])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = dsa.dsa_prompt_attention(q, k, v, cu_q, cu_k)
    b = dsa.dsa_shared_prefix_attention(*p, 32)
    dsa.dsa_cache_free(refs, tables, lens, kid)
    st = dsa.dsa_cache_fork(c, refs, tables, lens, who, kid)
    m = dsa.dsa_cache_compact(c, refs, tables)
g.replay()
torch.cuda.synchronize()
t.check_prompt((torch, dsa), q, k, v, [100], [3000], True)
t.check_paged((torch, dsa), *p, 32)
assert torch.equal(a[0], dsa.dsa_prompt_attention(q, k, v, cu_q, cu_k)[0])
assert torch.equal(b[0], dsa.dsa_shared_prefix_attention(*p, 32)[0])
assert st.tolist() == [0] and tables.tolist() == [[0, -1], [1, -1]] and m[1].tolist() == [2]
"""


def test_first_calls_of_a_process_may_be_captured(env):
    import os
    import subprocess
    import sys

    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr


def test_prompt_rows_of_no_sequence(env):
    """Rows before the first and behind the last sequence stay as they were,
    and what lies there is not read into any result."""
    torch, dsa = env
    q, k, v = make(torch, 8, 300, 300, 4, 2, 64, torch.bfloat16)
    q[:10] = math.nan
    q[200:] = math.nan
    k[:5], v[:5], k[222:], v[222:] = math.nan, math.inf, math.nan, math.inf
    out = torch.full_like(q, 3.0)
    lse = torch.full((300, 4), 4.0, device="cuda")
    dsa.dsa_prompt_attention(q, k, v, ints(torch, [10, 150, 200]), ints(torch, [5, 145, 222]),
                             out=out, lse_out=lse)
    torch.cuda.synchronize()
    want = ref.prompt(q[10:200], k[5:222], v[5:222], [0, 140, 190], [0, 140, 217], True)
    ref.check(out[10:200], want[0], want[2], "out")
    ref.check(lse[10:200], want[1], want[3], "lse")
    for t, x in ((out, 3.0), (lse, 4.0)):
        assert (t[:10] == x).all() and (t[200:] == x).all()


def test_prompt_offsets_are_clamped(env):
    torch, dsa = env
    q, k, v = make(torch, 9, 40, 50, 4, 2, 64, torch.bfloat16)
    out, lse = dsa.dsa_prompt_attention(q, k, v, ints(torch, [-7, 25, 1000]),
                                        ints(torch, [-3, 30, 2 ** 31 - 1]), causal=False)
    want = ref.prompt(q, k, v, [0, 25, 40], [0, 30, 50], False)
    torch.cuda.synchronize()
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("total_k", [120, 9000])
def test_prompt_offsets_that_decrease(env, total_k):
    """Rows are unspecified then, and nothing else is: the call ends, writes
    only rows of out and lse, and leaves the next call alone."""
    torch, dsa = env
    q, k, v = make(torch, 38, 90, total_k, 4, 2, 64, torch.bfloat16)
    out = torch.full((94, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((94, 4), 4.0, device="cuda")
    for a, b in (([60, 10, 90, 0, 80], [0, total_k, 50, 100, 7]),
                 ([2 ** 31 - 1, -2 ** 31, 45, 44, 90], [total_k, 0, total_k, 0, total_k])):
        dsa.dsa_prompt_attention(q, k, v, ints(torch, a), ints(torch, b), out=out[2:92],
                                 lse_out=lse[2:92])
        torch.cuda.synchronize()
        for t, x in ((out, 3.0), (lse, 4.0)):
            assert (t[:2] == x).all() and (t[92:] == x).all()
    check_prompt(env, q, k, v, [50, 40], [60, total_k - 60], True)


@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_prompt_masked_places_hold_anything(env, what, dtype):
    """Keys and values behind a row's last key (in the same tile, and in the
    next sequence's rows) never reach it."""
    torch, _ = env
    x = float(what)
    ql, kl = [130, 70, 200], [190, 70, 290]
    q, k, v = make(torch, 12, 400, 550, 4, 2, 64, getattr(torch, dtype))
    clean = [t.clone() for t in (q, k, v)]
    k[259, 0], v[259, 1] = x, x          # the second sequence's last key
    v[260 + 284, 0, 3] = x               # seen by the third one's last rows alone
    k[260 + 288, 1] = x
    out, _ = check_prompt(env, q, k, v, ql, kl, True)
    base, _ = check_prompt(env, *clean, ql, kl, True)
    _, _, tol, _ = ref.prompt(*clean, offsets(ql), offsets(kl), True)
    seen = torch.zeros(400, dtype=torch.bool, device="cuda")
    seen[199] = True
    seen[200 + 194:] = True
    # The other rows' definition is the same in both runs and each run is
    # within tol of it (checked above), so they differ by 2 tol at most: equal
    # bits are not promised, rows next to such values are summed in another
    # order.
    off = (out[~seen].double() - base[~seen].double()).abs().cpu()
    assert (off <= 2 * tol[~seen.cpu()]).all()


def test_prompt_merges_over_key_shards(env):
    """Runs over disjoint parts of the keys merge into the run over all."""
    torch, dsa = env
    T, H, D = 150, 4, 128
    q, k, v = make(torch, 13, T, 350, H, 2, D, torch.bfloat16)
    one = ints(torch, [0, T])
    parts = [dsa.dsa_prompt_attention(q, k[:200], v[:200], one, ints(torch, [0, 200]),
                                      causal=False),
             dsa.dsa_prompt_attention(q, k[200:], v[200:], one, ints(torch, [0, 150]),
                                      causal=True)]
    merged, lse = dsa.dsa_merge_attn_out(torch.stack([p[0] for p in parts]),
                                         torch.stack([p[1] for p in parts]))
    torch.cuda.synchronize()
    want = ref.prompt(q, k, v, [0, T], [0, 350], True)
    # each part and the merged sum carry a rounding of their own
    h = ref.half_step(torch.bfloat16)
    size = sum(p[0].double().cpu().abs() * torch.exp2(p[1].double().cpu() - want[1])[..., None]
               for p in parts)
    ref.check(merged.transpose(0, 1), want[0], 2 * want[2] + 2 * h * size + h * want[0].abs(),
              "out")
    ref.check(lse, want[1], 3 * want[3] + 8 * ref.U, "lse")


def make_paged(torch, seed, batch, heads, kv_heads, dim, page, prefix, own, dtype, extra=0):
    """Sequences of prefix + own[i] tokens on scattered pages, the rest NaN."""
    g = torch.Generator().manual_seed(seed)
    pre = prefix // page
    width = pre + max([-(-n // page) for n in own] + [0]) + extra
    need = pre + sum(-(-n // page) for n in own)
    pages = need + 3
    ids = torch.randperm(pages, generator=g).tolist()
    k, v = (torch.full((pages, page, kv_heads, dim), math.nan, dtype=dtype) for _ in range(2))
    at = pre
    tables = []

    def fill(ids, tokens):
        for t in range(0, tokens, page):
            n = min(page, tokens - t)
            for x in (k, v):
                x[ids[t // page], :n] = torch.randn(n, kv_heads, dim, generator=g).to(dtype)

    fill(ids[:pre], prefix)
    for n in own:
        mine = ids[at:at + -(-n // page)]
        at += len(mine)
        fill(mine, n)
        tables.append(ids[:pre] + mine + [-1] * (width - pre - len(mine)))
    q = (torch.randn(batch, heads, dim, generator=g) * 1.5).to(dtype)
    lens = [prefix + n for n in own]
    tables = torch.tensor(tables, dtype=torch.int32).view(batch, width)
    return q.cuda(), k.cuda(), v.cuda(), tables.cuda(), ints(torch, lens)


def check_paged(env, q, k, v, tables, lens, prefix, prefix_pages=None, scale=None, **kw):
    torch, dsa = env
    out, lse = dsa.dsa_shared_prefix_attention(q, k, v, tables, lens, prefix, scale=scale,
                                               prefix_pages=prefix_pages, **kw)
    torch.cuda.synchronize()
    shared = tables[0] if prefix_pages is None else prefix_pages
    want = ref.paged(q, k, v, tables, lens, shared, prefix, scale)
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")
    return out, lse


PAGED = [  # batch, heads, kv heads, dim, page, prefix, own tokens
    (1, 4, 4, 64, 16, 0, [1]),
    (3, 8, 2, 128, 16, 48, [1, 16, 17]),
    (5, 6, 2, 96, 32, 320, [31, 0, 64, 5, 200]),
    (2, 5, 1, 40, 64, 64, [0, 0]),
    (40, 8, 2, 64, 16, 144, [1 + (i * 13) % 50 for i in range(40)]),
    (33, 12, 4, 80, 64, 128, [(i * 37) % 130 for i in range(33)]),
    (17, 16, 1, 128, 128, 256, [(i * 111) % 700 for i in range(17)]),
    (2, 128, 1, 64, 256, 512, [300, 7]),
    (1, 2, 2, 128, 64, 0, [2500]),
    (9, 7, 1, 120, 1024, 1024, [i * 5 for i in range(9)]),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", PAGED, ids=[str(c[:6]) for c in PAGED])
def test_shared_sweep(env, case, dtype):
    torch, _ = env
    batch, heads, kv_heads, dim, page, prefix, own = case
    t = make_paged(torch, dim + page, *case, getattr(torch, dtype))
    check_paged(env, *t, prefix)


def test_shared_many_short_sequences(env):
    """Several segments per CTA, most of one tile, every third one empty."""
    torch, _ = env
    own = [0 if i % 3 == 0 else 1 + (i * 53) % 260 for i in range(700)]
    t = make_paged(torch, 24, 700, 4, 2, 64, 16, 32, own, torch.bfloat16)
    check_paged(env, *t, 32)
    check_paged(env, *t, 0)


def test_shared_prefix_is_only_a_matter_of_speed(env):
    """With and without the shared part named: the same attention."""
    torch, dsa = env
    own = [(i * 29) % 90 for i in range(12)]
    t = make_paged(torch, 4, 12, 8, 2, 64, 16, 160, own, torch.bfloat16)
    for prefix in (160, 96, 16, 0):
        check_paged(env, *t, prefix)


def test_shared_lengths_below_the_prefix(env):
    """Empty rows (padding), rows that end inside the prefix, lengths out of
    range; the first row's table is all -1, the prefix is given apart."""
    torch, _ = env
    q, k, v, tables, lens = make_paged(torch, 5, 6, 4, 2, 64, 16, 96, [20, 3, 40, 0, 9, 33],
                                       torch.bfloat16, extra=1)
    prefix = tables[0, :6].clone()
    tables[0] = -1
    lens.copy_(ints(torch, [0, 50, 136, -4, 97, 10 ** 6]))
    # the last length is clamped to the table's width: its row of pages ends
    # in -1, and the NaN behind its own tokens lies on a page that it has
    k[tables[5, 8].item()] = 0.5
    v[tables[5, 8].item()] = 0.25
    check_paged(env, q, k, v, tables, lens, 96, prefix)


def test_shared_bad_pages_are_not_seen(env):
    torch, _ = env
    q, k, v, tables, lens = make_paged(torch, 6, 5, 8, 2, 128, 16, 320, [100, 300, 40, 64, 1],
                                       torch.bfloat16)
    n = k.shape[0]
    tables[:, 3] = -1
    tables[:, 18] = n
    tables[1, 24] = -2 ** 31
    tables[1, 30] = 2 ** 31 - 1
    tables[2, 20] = n + 7
    tables[4, 20] = -1
    check_paged(env, q, k, v, tables, lens, 320)
    check_paged(env, q, k, v, tables, lens, 0)
    tables[:, :20] = -1     # nothing of the prefix is left
    check_paged(env, q, k, v, tables, lens, 320)


def test_shared_strided(env):
    """Head-major pages inside a larger pool, strided tables and outputs."""
    torch, dsa = env
    t = make_paged(torch, 7, 7, 6, 2, 64, 32, 64, [10, 0, 77, 32, 5, 31, 1], torch.float16)
    q, k, v, tables, lens = t
    want, want_lse = check_paged(env, *t, 64)
    pool = torch.zeros((k.shape[0], 3, 2, 32, 64), dtype=k.dtype, device="cuda")
    pool[:, 0], pool[:, 2] = k.transpose(1, 2), v.transpose(1, 2)
    wide = torch.full((7, tables.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + tables.shape[1]] = tables
    out = torch.full((6, 7, 72), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((6, 9), 5.0, device="cuda")
    dsa.dsa_shared_prefix_attention(q, pool[:, 0].transpose(1, 2), pool[:, 2].transpose(1, 2),
                                    wide[:, 2:2 + tables.shape[1]], lens, 64,
                                    out=out[:, :, :64].transpose(0, 1), lse_out=lse[:, :7].t())
    torch.cuda.synchronize()
    assert torch.equal(out[:, :, :64].transpose(0, 1), want) and (out[:, :, 64:] == 7).all()
    assert torch.equal(lse[:, :7].t(), want_lse) and (lse[:, 7:] == 5).all()


@pytest.mark.parametrize("what", ["nan", "inf"])
def test_shared_special_values_that_are_seen(env, what):
    """An infinite or NaN value of one sequence stays with its own rows."""
    torch, _ = env
    q, k, v, tables, lens = make_paged(torch, 9, 4, 4, 2, 64, 16, 32, [20, 40, 3, 18],
                                       torch.bfloat16)
    v[tables[1, 2].item(), 3, 0, 5] = float(what)
    k[tables[3, 2].item(), 1, 1] = math.nan
    check_paged(env, q, k, v, tables, lens, 32)


def test_shared_equals_prompt_attention(env):
    """Single tokens on pages and a packed batch of one query each."""
    torch, dsa = env
    own = [70, 1, 33]
    q, k, v, tables, lens = make_paged(torch, 10, 3, 8, 4, 64, 16, 64, own, torch.bfloat16)
    out, lse = check_paged(env, q, k, v, tables, lens, 64)
    rows = [tables[b, :-(-(64 + n) // 16)].long() for b, n in enumerate(own)]
    pk, pv = (torch.cat([t[i].reshape(-1, 4, 64)[:64 + n] for i, n in zip(rows, own)])
              for t in (k, v))
    check_prompt(env, q, pk, pv, [1, 1, 1], [64 + n for n in own], True)


def test_streams_and_graphs(env):
    """Calls on another stream, captured, and replayed on new contents; two
    graphs of the same call in flight at once do not disturb each other."""
    torch, dsa = env
    q, k, v = make(torch, 14, 200, 200, 8, 2, 128, torch.bfloat16)
    cu = ints(torch, [0, 60, 200])
    p = make_paged(torch, 15, 20, 8, 2, 128, 16, 320, [3 * i for i in range(20)], torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, la = dsa.dsa_prompt_attention(q, k, v, cu, cu, stream=side)
    b, lb = dsa.dsa_shared_prefix_attention(*p, 320, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want_a, want_b = check_prompt(env, q, k, v, [60, 140], [60, 140], True), \
        check_paged(env, *p, 320)
    assert torch.equal(a, want_a[0]) and torch.equal(la, want_a[1])
    assert torch.equal(b, want_b[0]) and torch.equal(lb, want_b[1])
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x = dsa.dsa_prompt_attention(q, k, v, cu, cu)
            y = dsa.dsa_shared_prefix_attention(*p, 320)
        graphs.append(g)
        outs.append((x, y))
    for n in range(2):
        if n:       # other contents and lengths, the same graphs
            q.mul_(0.5)
            p[0].mul_(0.5)
            p[4].sub_(1).clamp_(min=0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        wa, wb = check_prompt(env, q, k, v, [60, 140], [60, 140], True), check_paged(env, *p, 320)
        for x, y in outs:
            assert torch.equal(x[0], wa[0]) and torch.equal(x[1], wa[1])
            assert torch.equal(y[0], wb[0]) and torch.equal(y[1], wb[1])


def test_calls_repeat_bit_for_bit(env):
    torch, dsa = env
    q, k, v = make(torch, 16, 500, 900, 8, 2, 128, torch.bfloat16)
    cu_q, cu_k = ints(torch, [0, 500]), ints(torch, [0, 900])
    p = make_paged(torch, 17, 30, 8, 2, 64, 16, 1600, [40 * i for i in range(30)], torch.bfloat16)
    first = (*dsa.dsa_prompt_attention(q, k, v, cu_q, cu_k),
             *dsa.dsa_shared_prefix_attention(*p, 1600))
    for _ in range(20):
        again = (*dsa.dsa_prompt_attention(q, k, v, cu_q, cu_k),
                 *dsa.dsa_shared_prefix_attention(*p, 1600))
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_own_workspace(env):
    torch, dsa = env
    p = make_paged(torch, 18, 10, 8, 2, 64, 16, 320, [9 * i for i in range(10)], torch.bfloat16)
    q, k, _, tables, _ = p
    want = check_paged(env, *p, 320)
    need = dsa.shared_prefix_workspace_bytes(10, 8, 2, 64, 320, tables.shape[1], 16)
    buf = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = dsa.dsa_shared_prefix_attention(*p, 320, workspace=buf[:need])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (buf[need:] == 255).all()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_shared_prefix_attention(*p, 320, workspace=buf[:need - 1])
    q, k, v = make(torch, 32, 300, 5000, 4, 2, 64, torch.bfloat16)
    want = check_prompt(env, q, k, v, [300], [5000], True)
    need = dsa.prompt_workspace_bytes(300, 5000, 4, 2, 64, 1)
    buf = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    cu = ints(torch, [0, 300]), ints(torch, [0, 5000])
    got = dsa.dsa_prompt_attention(q, k, v, *cu, workspace=buf[:need])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (buf[need:] == 255).all()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_prompt_attention(q, k, v, *cu, workspace=buf[:need - 1])


def test_calls_at_the_same_time(env):
    """Threads that call on one stream and on streams of their own, and a
    replayed graph beside them: no call disturbs another."""
    import threading

    torch, dsa = env
    q, k, v = make(torch, 34, 300, 6000, 8, 2, 64, torch.bfloat16)
    cu = ints(torch, [0, 300]), ints(torch, [0, 6000])
    p = make_paged(torch, 35, 20, 8, 2, 64, 16, 160, [7 * i for i in range(20)], torch.bfloat16)
    want = (*check_prompt(env, q, k, v, [300], [6000], True), *check_paged(env, *p, 160))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed = (*dsa.dsa_prompt_attention(q, k, v, *cu),
                   *dsa.dsa_shared_prefix_attention(*p, 160))
    main, bad = torch.cuda.current_stream(), []

    def work(stream):
        with torch.cuda.stream(stream):
            got = [(*dsa.dsa_prompt_attention(q, k, v, *cu),
                    *dsa.dsa_shared_prefix_attention(*p, 160)) for _ in range(15)]
        stream.synchronize()
        bad.extend(1 for r in got if not all(torch.equal(x, y) for x, y in zip(r, want)))

    streams = [main, main, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(s,)) for s in streams]
    for t in threads:
        t.start()
    beside = torch.cuda.Stream()
    with torch.cuda.stream(beside):
        for _ in range(15):
            g.replay()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    assert all(torch.equal(x, y) for x, y in zip(graphed, want))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl", [
    ([1, 1], [9000, 3]),                     # one block across many CTAs
    ([2], [40000]),
    ([700, 0, 33, 300], [2500, 10, 0, 900]),
    ([2100, 5], [1500, 3000]),               # rows without keys, then few with many
    ([9] * 300, [40] * 300),
], ids=["one block", "long and alone", "mixed", "few queries", "many"])
def test_prompt_blocks_cut_between_ctas(env, ql, kl, causal):
    """More keys than the kernel leaves whole: blocks are cut between CTAs and
    their parts joined, at odd places."""
    torch, dsa = env
    for heads, kv_heads, dim in ((6, 2, 64), (4, 4, 128), (5, 1, 72)):
        q, k, v = make(torch, sum(ql) + dim, sum(ql), sum(kl), heads, kv_heads, dim,
                       torch.bfloat16)
        assert dsa.prompt_workspace_bytes(sum(ql), sum(kl), heads, kv_heads, dim, len(ql)) > 0
        check_prompt(env, q, k, v, ql, kl, causal)


def test_prompt_cut_blocks_with_values_that_are_not_finite(env):
    """Hidden infinities and NaN beside a cut, and seen ones behind it."""
    torch, _ = env
    ql, kl = [300, 40], [5000, 700]
    q, k, v = make(torch, 31, 340, 5700, 4, 2, 64, torch.bfloat16)
    v[4999, 0], k[4999, 1] = math.nan, math.inf     # the last query's own key
    v[4800, 1, 7] = math.inf
    v[5000 + 650, 0, 2] = -math.inf
    check_prompt(env, q, k, v, ql, kl, True)


def test_nothing_to_do(env):
    torch, dsa = env
    q, k, v = make(torch, 19, 4, 4, 4, 2, 64, torch.bfloat16)
    none = ints(torch, [0])
    out = torch.full_like(q, 2.0)
    dsa.dsa_prompt_attention(q, k, v, none, none, out=out)
    assert (out == 2).all()
    out, lse = dsa.dsa_prompt_attention(q[:0], k, v, ints(torch, [0, 0]), ints(torch, [0, 4]))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = dsa.dsa_prompt_attention(q, k[:0], v[:0], ints(torch, [0, 4]), ints(torch, [0, 0]))
    assert (out == 0).all() and (lse == -math.inf).all()
    pages = torch.zeros((0, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.dsa_shared_prefix_attention(q, pages, pages, torch.full((4, 3), 0,
                                               dtype=torch.int32, device="cuda"),
                                               ints(torch, [5, 0, 48, 7]))
    assert (out == 0).all() and (lse == -math.inf).all()
    empty = torch.zeros((4, 0), dtype=torch.int32, device="cuda")
    kp = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.dsa_shared_prefix_attention(q, kp, kp, empty, ints(torch, [5, 0, 48, 7]))
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = dsa.dsa_shared_prefix_attention(q[:0], kp, kp, empty[:0], none[:0])
    assert out.shape == (0, 4, 64)


@pytest.mark.slow
def test_prompt_long(env):
    """A long packed batch, sampled rows against the definition."""
    torch, dsa = env
    ql, kl = [4100, 1000, 2048], [4100, 5000, 2048]
    q, k, v = make(torch, 20, sum(ql), sum(kl), 8, 2, 128, torch.bfloat16)
    cu_q, cu_k = offsets(ql), offsets(kl)
    out, lse = dsa.dsa_prompt_attention(q, k, v, ints(torch, cu_q), ints(torch, cu_k))
    torch.cuda.synchronize()
    for i, (a, c) in enumerate(zip(cu_q[:-1], cu_k[:-1])):
        for t in (0, 1, 127, 128, 500, ql[i] // 2 + 3, ql[i] - 1):
            n = kl[i] - ql[i] + t + 1
            want = ref.prompt(q[a + t:a + t + 1], k[c:c + n], v[c:c + n], [0, 1], [0, n], False)
            ref.check(out[a + t:a + t + 1], want[0], want[2], f"out {i} {t}")
            ref.check(lse[a + t:a + t + 1], want[1], want[3], f"lse {i} {t}")


def test_prompt_that_takes_longer_than_a_wait_may_stand_still(env):
    """About 16 seconds on the device, with no value behind the sequence's end
    (whole key tiles): the warp that clears those waits all along."""
    torch, dsa = env
    tokens, heads, dim, keys = 65536, 128, 8, 1 << 17
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q = rand(tokens, heads, dim)
    cu_q = ints(torch, [0, tokens])

    def run(n):
        k, v = rand(n, 1, dim), rand(n, 1, dim)
        first, last = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        first.record()
        out, lse = dsa.dsa_prompt_attention(q, k, v, cu_q, ints(torch, [0, n]), causal=False)
        last.record()
        torch.cuda.synchronize()
        return k, v, out, lse, first.elapsed_time(last) / 1e3

    run(keys)
    keys *= int(16 / run(keys)[-1]) + 1
    k, v, out, lse, seconds = run(keys)
    assert dsa.attention_error() == 0, f"a wait gave up in a call of {seconds:.1f} s"
    # Some rows in 64 bits. Weights rounded to bf16 (half a step: 2^-9 each
    # way of the fraction line's upper part) move an output by at most
    # 2^-9 sum w |v|, about 0.8 of that here; fp32 sums of key tiles, each
    # rounded twice 2^-24 at most of a sum that stays within five deviations,
    # 5 sqrt(keys) of values around 0, add 2^-12. l is a sum over keys / 128
    # tiles, 2^-24 of it lost at each: below 2^-8 of l for 2^23 keys, and
    # 1 / ln 2 of that in the base-2 logarithm.
    for t in (0, tokens // 2 + 1, tokens - 1):
        for h in (0, 77, heads - 1):
            x = (k[:, 0].double() * q[t, h].double()).sum(1) / math.sqrt(dim)
            w = torch.exp(x - torch.logsumexp(x, 0))
            want = (w[:, None] * v[:, 0].double()).sum(0)
            assert (out[t, h].double() - want).abs().max() < 2.0 ** -8, (t, h)
            assert abs(lse[t, h].double() - torch.logsumexp(x, 0) / math.log(2.0)) < 2.0 ** -7


@pytest.mark.parametrize("page", [16, 64])
def test_shared_tables_of_the_longest_length(env, page):
    """A row of pages for all lengths below 2^31, of which the first and the
    last are there: the sequence's last key tile ends at 2^31."""
    torch, dsa = env
    width = (2 ** 31 - 1) // page
    g = torch.Generator().manual_seed(6)
    q = torch.randn(1, 4, 64, generator=g).bfloat16().cuda()
    k, v = (torch.randn(2, page, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    tables = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    tables[0, 0], tables[0, -1] = 1, 0
    for lens in (width * page, 2 ** 31 - 1):
        out, lse = dsa.dsa_shared_prefix_attention(q, k, v, tables, ints(torch, [lens]))
        want = ref.paged(q, k, v, ints(torch, [[1, 0]]), ints(torch, [2 * page]), None, 0)
        ref.check(out, want[0], want[2], "out")
        ref.check(lse, want[1], want[3], "lse")


def test_the_error_flag_is_read_behind_all_streams(env):
    """A call on a stream that the default stream does not wait for."""
    torch, dsa = env
    side = torch.cuda.Stream()
    q, k, v = make(torch, 41, 4096, 262144, 8, 1, 128, torch.bfloat16)
    cu_q, cu_k = ints(torch, [0, 4096]), ints(torch, [0, 262144])
    torch.cuda.synchronize()
    for _ in range(20):  # some 3 ms each
        dsa.dsa_prompt_attention(q, k, v, cu_q, cu_k, causal=False, stream=side)
    assert not side.query(), "the calls ended before the flag was read: nothing is shown"
    assert dsa.attention_error() == 0
    assert side.query(), "the flag was read before the calls ended"


@pytest.mark.parametrize("empty", [[0], [0, 1, 2], list(range(40)), list(range(45))])
def test_shared_default_prefix_passes_over_empty_slots(env, empty):
    """Slots that dsa_cache_free emptied, in front of the live ones."""
    torch, dsa = env
    q, k, v, tables, lens = make_paged(torch, 43, 45, 8, 2, 64, 16, 96, [20 + i for i in range(45)],
                                       torch.bfloat16)
    pages = tables[-1, :6].clone()
    refs = torch.full((k.shape[0],), 50, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_free(refs, tables, lens, ints(torch, empty))
    out, lse = dsa.dsa_shared_prefix_attention(q, k, v, tables, lens, 96)
    want = ref.paged(q, k, v, tables, lens, pages, 96)
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")
    # a row that is named is taken as it is
    last = dsa.dsa_shared_prefix_attention(q, k, v, tables, lens, 96, prefix_pages=pages)
    assert torch.equal(out, last[0]) and torch.equal(lse, last[1])


def test_shared_default_prefix_of_a_slot_without_tokens(env):
    """A row with pages counts although its sequence sees none of them yet; an
    empty slot whose entries behind the first are stale does not."""
    torch, dsa = env
    q, k, v, tables, lens = make_paged(torch, 44, 3, 4, 2, 64, 16, 64, [9, 30, 17], torch.float16)
    lens[0] = 0
    tables[1, :4] = 99999  # not there
    check_paged(env, q, k, v, tables, lens, 64)
    tables[0, 0] = -1
    tables[1, :4] = tables[2, :4]
    out, lse = dsa.dsa_shared_prefix_attention(q, k, v, tables, lens, 64)
    want = ref.paged(q, k, v, tables, lens, tables[1, :4], 64)
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")


def test_fp16_parts_merge_in_fp32(env):
    """The merge takes no fp16; widened parts lose nothing on the way."""
    torch, dsa = env
    T, H, D = 150, 4, 96
    q, k, v = make(torch, 45, T, 350, H, 2, D, torch.float16)
    one = ints(torch, [0, T])
    parts = [dsa.dsa_prompt_attention(q, k[:200], v[:200], one, ints(torch, [0, 200]),
                                      causal=False),
             dsa.dsa_prompt_attention(q, k[200:], v[200:], one, ints(torch, [0, 150]),
                                      causal=True)]
    outs, lses = (torch.stack([p[i] for p in parts]) for i in range(2))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        dsa.dsa_merge_attn_out(outs, lses)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        dsa.dsa_correct_attn_out(outs[0], lses, 0)
    merged, lse = dsa.dsa_merge_attn_out(outs.float(), lses)
    torch.cuda.synchronize()
    want = ref.prompt(q, k, v, [0, T], [0, 350], True)
    # each part carries a rounding of its own, the merged sum none but fp32's
    h = ref.half_step(torch.float16)
    size = sum(p[0].double().cpu().abs() * torch.exp2(p[1].double().cpu() - want[1])[..., None]
               for p in parts)
    ref.check(merged.transpose(0, 1), want[0], 2 * want[2] + 2 * h * size + 2.0 ** -24, "out")
    ref.check(lse, want[1], 3 * want[3] + 8 * ref.U, "lse")


def test_kept_workspaces_are_bounded_and_released(env):
    """Streams and threads without end keep no more than the bound."""
    import threading

    torch, dsa = env
    q, k, v = make(torch, 46, 300, 6000, 8, 2, 128, torch.bfloat16)
    cu = ints(torch, [0, 300]), ints(torch, [0, 6000])
    need = dsa.prompt_workspace_bytes(300, 6000, 8, 2, 128, 1)
    assert dsa._KEEP_ALL_BYTES < 12 * need and need <= dsa._KEEP_BYTES
    want = check_prompt(env, q, k, v, [300], [6000], True)
    dsa.release_workspaces()
    got = []

    def work(stream):
        got.append(dsa.dsa_prompt_attention(q, k, v, *cu, stream=stream))
        kept = sum(x[2] for x in list(dsa._scratch_cache.values()))
        got[-1] += (kept,)

    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(12)]:
        work(s)
    for _ in range(12):
        t = threading.Thread(target=work, args=(torch.cuda.current_stream(),))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 24
    for out, lse, kept in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert need <= kept <= dsa._KEEP_ALL_BYTES
    before = torch.cuda.memory_allocated()
    dsa.release_workspaces()
    assert not dsa._scratch_cache and torch.cuda.memory_allocated() <= before - need


def test_a_stream_with_another_ones_handle_gets_a_workspace_of_its_own(env):
    """Streams that are not PyTorch's: one is destroyed, the next may get its
    handle."""
    import ctypes

    torch, dsa = env
    rt = ctypes.CDLL("libcudart.so." + torch.version.cuda.split(".")[0])
    p = make_paged(torch, 47, 4, 4, 2, 64, 16, 32, [5, 60, 0, 9], torch.bfloat16)
    want = check_paged(env, *p, 32)
    dsa.release_workspaces()
    ids, handles = set(), set()
    for _ in range(5):
        handle = ctypes.c_void_p()
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(handle), 1) == 0
        stream = torch.cuda.ExternalStream(handle.value)
        ids.add(dsa.library().dsa_stream_id(handle.value))
        handles.add(handle.value)
        for _ in range(2):
            got = dsa.dsa_shared_prefix_attention(*p, 32, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert rt.cudaStreamDestroy(handle) == 0
    assert len(ids) == 5 and 2 ** 64 - 1 not in ids
    assert len(dsa._scratch_cache) == 5, f"{len(handles)} handles"
    dsa.release_workspaces()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 64), (8, 1, 128), (6, 2, 40), (2, 2, 104)])
@pytest.mark.parametrize("ql,kl", [([130, 70, 200], [190, 70, 290]), ([300, 40], [5000, 700]),
                                   ([128], [128]), ([700], [700])])
def test_prompt_values_that_are_not_seen_leave_no_trace(env, ql, kl, heads, kv_heads, dim, dtype):
    """Rows in front of infinities and NaN: the same bits as with any other
    values there. Rows behind them: what their definition says."""
    torch, _ = env
    tq, tk = sum(ql), sum(kl)
    q, k, v = make(torch, 48, tq, tk, heads, kv_heads, dim, getattr(torch, dtype))
    clean = check_prompt(env, q, k, v, ql, kl, True)
    first = kl[0] - ql[0] + ql[0] // 2       # seen by the first sequence's second half
    v[first, 0, 3] = math.inf
    v[first + 9, 0, 3] = -math.inf
    v[first + 5, kv_heads - 1, dim - 1] = math.nan
    v[first + 20, :, 17] = math.inf
    v[tk - 1] = math.nan                     # seen by the last query alone
    k[first + 31, 0] = math.nan              # its rows are NaN from there on
    out, lse = check_prompt(env, q, k, v, ql, kl, True)
    for t in (slice(0, ql[0] // 2), slice(ql[0], tq - 1)):
        assert torch.equal(out[t], clean[0][t]) and torch.equal(lse[t], clean[1][t])


@pytest.mark.parametrize("batch,heads,kv_heads,dim,page", [
    (3, 4, 2, 64, 16), (9, 8, 2, 128, 64), (150, 4, 1, 64, 16), (40, 16, 2, 80, 256)])
def test_shared_prefix_values_that_are_not_seen_leave_no_trace(env, batch, heads, kv_heads, dim,
                                                               page):
    """The same for sequences that end inside the prefix."""
    torch, _ = env
    prefix = 768
    t = make_paged(torch, 49, batch, heads, kv_heads, dim, page, prefix,
                   [(i * 31) % 90 for i in range(batch)], torch.bfloat16)
    q, k, v, tables, lens = t
    short = [(i * 97) % 700 for i in range(batch)]
    for i in range(0, batch, 2):
        lens[i] = short[i]
    clean = check_paged(env, *t, prefix)

    def at(pos):
        return tables[0, pos // page].item(), pos % page

    v[at(420)][0, 3] = math.inf
    v[at(421)][kv_heads - 1, 5] = math.nan
    v[at(767)][:] = math.nan
    v[at(300)][0, 7], v[at(650)][0, 7] = math.inf, -math.inf
    out, lse = check_paged(env, *t, prefix)
    front = (lens <= 300)
    assert front.any() and torch.equal(out[front], clean[0][front])
    assert torch.equal(lse, clean[1])


def test_a_hidden_infinity_does_not_hold_up_a_long_prompt(env):
    """One infinite value at the end of 262144 tokens; 11 ms without it."""
    torch, dsa = env
    n = 262144
    g = torch.Generator(device="cuda").manual_seed(50)
    q, k, v = (torch.randn(n, 1, 128, generator=g, device="cuda").bfloat16() for _ in range(3))
    cu = ints(torch, [0, n])
    want = dsa.dsa_prompt_attention(q, k, v, cu, cu)
    v[-1, 0, 77] = math.inf
    for _ in range(2):
        first, last = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        first.record()
        got = dsa.dsa_prompt_attention(q, k, v, cu, cu)
        last.record()
        torch.cuda.synchronize()
    assert dsa.attention_error() == 0
    assert torch.equal(got[0][:-1], want[0][:-1]) and torch.equal(got[1], want[1])
    assert got[0][-1].isinf().nonzero().tolist() == [[0, 77]]
    assert first.elapsed_time(last) < 500, "ms"
