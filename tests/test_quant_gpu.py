"""Writing, reading and attending to pages of 8-bit codes against their
definition in 64 bits (tests/quant_reference.py)."""

import math
import threading

import numpy as np
import pytest

import attention_reference as ref
import quant_reference as quant

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


def ints(torch, values):
    return torch.tensor(np.asarray(values, np.int32), device="cuda")


def offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


class Pool:
    """Random codes and power-of-two scales on scattered pages, with the CPU's
    copy of them."""

    def __init__(self, torch, seed, room, heads, dim, page, block, spare=3, low=-9, high=-4):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in room]
        pages = sum(need) + spare
        width = max(need + [1])
        ids = rng.permutation(pages).astype(np.int32)
        self.tables = np.full((len(room), width), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.codes = rng.integers(0, 256, (2, pages, page, heads, dim)).astype(np.uint8)
        self.codes[(self.codes & 127) == 127] = 0x34
        self.scales = np.exp2(rng.integers(low, high, (2, pages, page // block, heads))).astype(
            np.float32)
        self.torch = torch

    def gpu(self):
        t = self.torch
        cache = t.from_numpy(self.codes.copy()).cuda().view(t.float8_e4m3fn)
        scales = t.from_numpy(self.scales.copy()).cuda()
        return cache, scales, ints(t, self.tables)


def rows(torch, seed, total, heads, dim, dtype):
    """Tokens of magnitudes that are spread over some powers of two."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(total, heads, dim, generator=g) *
             torch.exp(1.5 * torch.randn(total, heads, 1, generator=g))).to(dtype).cuda()
            for _ in range(2)]


def check_write(env, pool, k, v, cu, lens, gpu=None, **kw):
    torch, dsa = env
    cache, scales, tables = gpu or pool.gpu()
    dsa.dsa_quant_cache_write(k, v, ints(torch, cu), cache[0], cache[1], scales[0], scales[1],
                              tables, ints(torch, lens), **kw)
    torch.cuda.synchronize()
    codes, want = pool.codes.copy(), pool.scales.astype(np.float64)
    quant.write(k.double().cpu().numpy(), v.double().cpu().numpy(), cu, codes, want, pool.tables,
                lens)
    got = scales.cpu().numpy()
    np.testing.assert_array_equal(got, want.astype(np.float32))
    quant.same_codes(cache.view(torch.uint8).cpu().numpy(), codes, "codes")
    return cache, scales, tables


WRITES = [  # new tokens, held tokens
    ([1], [0]),
    ([1, 1, 1, 1], [0, 1, 15, 16]),
    ([1] * 9, [63, 64, 65, 127, 128, 129, 2, 30, 31]),
    ([5, 0, 33, 17], [3, 9, 0, 40]),
    ([300, 1, 129], [0, 255, 100]),
    ([0, 0], [4, 0]),
    ([40, 200, 3], [5, 11, 0]),
]
POOLS = [  # heads, head dim, page, block
    (2, 64, 16, 16), (8, 128, 64, 64), (3, 80, 32, 8), (1, 16, 16, 1), (5, 112, 128, 32),
    (4, 96, 256, 256), (2, 48, 64, 2), (1, 128, 512, 256),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("lengths", WRITES, ids=[str(x) for x in WRITES])
@pytest.mark.parametrize("shape", POOLS, ids=[str(x) for x in POOLS])
def test_write_sweep(env, shape, lengths, dtype):
    torch, _ = env
    new, held = lengths
    heads, dim, page, block = shape
    pool = Pool(torch, sum(held) + dim, [a + b for a, b in zip(new, held)], heads, dim, page,
                block)
    k, v = rows(torch, dim + sum(new), sum(new), heads, dim, getattr(torch, dtype))
    check_write(env, pool, k, v, offsets(new), held)


def test_write_token_by_token(env):
    """Scales grow as tokens come; every step is the model's."""
    torch, _ = env
    pool = Pool(torch, 1, [50, 40], 2, 32, 16, 16)
    gpu, held = None, [0, 7]
    for i in range(20):
        k, v = rows(torch, 100 + i, 2, 2, 32, torch.bfloat16)
        gpu = check_write(env, pool, k * (1.3 ** i), v, [0, 1, 2], held, gpu)
        pool.codes = gpu[0].view(torch.uint8).cpu().numpy()
        pool.scales = gpu[1].cpu().numpy()
        held = [n + 1 for n in held]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_write_special_values(env, dtype):
    """NaN, infinities, zeros of both signs, the largest and the smallest
    numbers: codes of what is not finite are NaN, and scales ignore them."""
    torch, _ = env
    dt = getattr(torch, dtype)
    pool = Pool(torch, 2, [70, 20, 33], 2, 32, 16, 8)
    k, v = rows(torch, 3, 90, 2, 32, dt)
    most = torch.finfo(dt).max
    k[3, 0, 5], k[4, 1, 6], k[5, 0, 7], v[2, 0, 0] = math.nan, math.inf, -math.inf, -0.0
    k[8:16] = 0.0
    v[8:16] = -0.0
    k[16:24, 0] = most
    v[16:24, 1, 3] = -most
    k[24:32] = torch.finfo(dt).smallest_normal / 8
    v[24:32] = math.nan
    v[32:40] = math.inf
    v[40:48, :, ::2] = 448.0
    v[40:48, :, 1::2] = 449.0 if dtype == "float16" else 450.0
    k[40:48] = 448.0
    check_write(env, pool, k, v, [0, 55, 60, 90], [9, 15, 3])


def test_write_rounds_to_even(env):
    """Every midpoint between two codes, and its neighbours in fp16."""
    torch, _ = env
    mids = (quant.VALUES[:126] + quant.VALUES[1:127]) / 2
    x = torch.from_numpy(np.concatenate([mids, -mids, [448.0] * 4])).half()
    x = torch.cat([x, torch.nextafter(x, torch.tensor(500.0).half()),
                   torch.nextafter(x, torch.tensor(-500.0).half())])
    x = torch.cat([x, x.new_full((-len(x) % 128,), 448.0)]).clamp(-448, 448).view(-1, 1, 128)
    x = torch.cat([x, x.new_full((16 - len(x), 1, 128), 448.0)]).cuda()
    pool = Pool(torch, 5, [16], 1, 128, 16, 16)
    _, scales, tables = check_write(env, pool, x, -x, [0, 16], [0])
    assert scales[:, tables[0, 0]].flatten().tolist() == [1.0, 1.0]


@pytest.mark.parametrize("old", [0.0, -1.0, math.nan, math.inf, 3e38, 1e-45, 1e-40, 0.7, 3.0,
                                 2.0 ** -5])
def test_write_next_to_any_old_scale(env, old):
    torch, _ = env
    pool = Pool(torch, 6, [40, 40], 2, 64, 16, 16)
    pool.scales[:] = old
    k, v = rows(torch, 7, 7, 2, 64, torch.bfloat16)
    if math.isfinite(old) and old > 1e30:
        k, v = k * 1e38, v * 1e37
    check_write(env, pool, k, v, [0, 3, 7], [9, 30])


def test_write_without_a_page(env):
    """Missing and bad pages, and tokens behind the table, are dropped."""
    torch, _ = env
    pool = Pool(torch, 8, [100, 90, 64], 2, 64, 16, 16)
    pool.tables[0, 2], pool.tables[0, 4], pool.tables[1, 5] = -1, 9999, -(2 ** 31)
    pool.tables[2, :] = -1
    k, v = rows(torch, 9, 290, 2, 64, torch.bfloat16)
    check_write(env, pool, k, v, [0, 150, 230, 290], [10, 20, 4])
    check_write(env, pool, k, v, [0, 150, 230, 290], [2 ** 31 - 1, 112, 111])
    check_write(env, pool, k, v, [0, 150, 230, 290], [-5, -(2 ** 31), 0])


def test_write_rows_of_no_sequence(env):
    """In front of the first offset, behind the last one, offsets past the end."""
    torch, _ = env
    pool = Pool(torch, 10, [100, 90, 64], 2, 64, 32, 16)
    k, v = rows(torch, 11, 120, 2, 64, torch.float16)
    check_write(env, pool, k, v, [40, 60, 60, 80], [3, 9, 0])
    check_write(env, pool, k, v, [0, 50, 100, 500], [3, 9, 0])
    check_write(env, pool, k, v, [-7, 50, 100, 120], [3, 9, 0])


def test_write_offsets_that_decrease(env):
    """Only the blocks of these sequences are touched, if any."""
    torch, dsa = env
    pool = Pool(torch, 12, [100, 90, 64], 2, 64, 16, 16)
    k, v = rows(torch, 13, 60, 2, 64, torch.bfloat16)
    cache, scales, tables = pool.gpu()
    dsa.dsa_quant_cache_write(k, v, ints(torch, [50, 10, 60, 0]), cache[0], cache[1], scales[0],
                              scales[1], tables, ints(torch, [3, 9, 0]))
    torch.cuda.synchronize()
    mine = set(pool.tables[pool.tables >= 0].tolist())
    rest = [n for n in range(pool.codes.shape[1]) if n not in mine]
    np.testing.assert_array_equal(cache.view(torch.uint8).cpu().numpy()[:, rest],
                                  pool.codes[:, rest])


def test_write_strided(env):
    """Heads of a fused projection, token-major pools of several layers, heads
    in front of tokens."""
    torch, dsa = env
    H, D, page, block = 3, 48, 32, 16
    pool = Pool(torch, 14, [70, 40], H, D, page, block)
    both = torch.randn(60, 2 * H + 4, D + 8, device="cuda").bfloat16()
    k, v = both[:, :H, :D], both[:, H + 2:2 * H + 2, :D]
    codes = torch.from_numpy(pool.codes).cuda()
    N = codes.shape[1]
    wide = torch.zeros((2, H, N, page, 64), dtype=torch.uint8, device="cuda")
    view = wide[..., :D].permute(0, 2, 3, 1, 4)
    view.copy_(codes)
    scales = torch.zeros((2, N, 5, page // block, H), device="cuda")
    scales[:, :, 2] = torch.from_numpy(pool.scales).cuda()
    gpu = view.view(torch.float8_e4m3fn), scales[:, :, 2], ints(torch, pool.tables)
    check_write(env, pool, k, v, [0, 45, 60], [20, 17], gpu)
    assert int(wide[..., D:].max()) == 0
    lone = torch.randn(60, 1, D, device="cuda").bfloat16().expand(60, H, D)   # one head for all
    check_write(env, pool, lone, lone, [0, 45, 60], [20, 17])


READS = [[1], [16, 1, 0, 33], [200, 127, 128, 129], [0, 0], [3] * 40]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("lens", READS, ids=[str(x) for x in READS])
@pytest.mark.parametrize("shape", POOLS, ids=[str(x) for x in POOLS])
def test_read_sweep(env, shape, lens, dtype):
    torch, dsa = env
    heads, dim, page, block = shape
    pool = Pool(torch, sum(lens) + dim, lens, heads, dim, page, block)
    cache, scales, tables = pool.gpu()
    dt = getattr(torch, dtype)
    k, v = dsa.dsa_quant_cache_read(cache[0], cache[1], scales[0], scales[1], tables,
                                    ints(torch, offsets(lens)), total=sum(lens), dtype=dt)
    torch.cuda.synchronize()
    want = np.concatenate([quant.read(pool.codes, pool.scales, pool.tables, s, n)
                           for s, n in enumerate(lens)], 1)
    for got, w in ((k, want[0]), (v, want[1])):
        # four bits times a power of two: exact in both types, but for fp16's range
        assert torch.equal(got.cpu(), torch.from_numpy(w).to(dt))


def test_read_any_scale_and_code(env):
    """Scales that are no powers of two, NaN codes and scales; one rounding."""
    torch, dsa = env
    pool = Pool(torch, 20, [60], 2, 64, 16, 8)
    rng = np.random.default_rng(1)
    pool.scales = rng.uniform(0.01, 3, pool.scales.shape).astype(np.float32)
    pool.codes[0, pool.tables[0, 1], 3, 0, 9], pool.codes[1, pool.tables[0, 0], 0, 1, 0] = 127, 255
    pool.scales[0, pool.tables[0, 2], 1, 1] = math.nan
    cache, scales, tables = pool.gpu()
    for dt in (torch.bfloat16, torch.float16):
        got = dsa.dsa_quant_cache_read(cache[0], cache[1], scales[0], scales[1], tables,
                                       ints(torch, [0, 60]), total=60, dtype=dt)
        want = quant.read(pool.codes, pool.scales, pool.tables, 0, 60)
        for g, w in zip(got, want):
            # the product to fp32 and then to 16 bits: half a step, and 2^-24 of it
            h = torch.finfo(dt).eps / 2
            w = torch.from_numpy(w)
            low = 2.0 ** -25 if dt == torch.float16 else 0.0
            ref.check(g, w, (h * (1 + 2.0 ** -10) + 2.0 ** -24) * w.abs().nan_to_num() + low,
                      "read")


def test_read_rows_of_no_sequence_and_without_a_page(env):
    torch, dsa = env
    pool = Pool(torch, 21, [60, 40], 2, 64, 16, 16)
    pool.tables[0, 1], pool.tables[1, 0] = -1, 7777
    cache, scales, tables = pool.gpu()
    outs = [torch.full((150, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = dsa.dsa_quant_cache_read(cache[0], cache[1], scales[0], scales[1], tables,
                                   ints(torch, [10, 90, 130]), k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    assert got[0] is outs[0] and got[1] is outs[1]
    for i, o in enumerate(outs):
        o = o.double().cpu()
        assert (o[:10] == 7).all() and (o[130:] == 7).all()
        for s, (a, b) in enumerate(((10, 90), (90, 130))):
            w = quant.read(pool.codes, pool.scales, pool.tables, s, b - a)[i]
            assert torch.equal(o[a:b], torch.from_numpy(w).bfloat16().double())
    # past the end of the output, and decreasing: nothing outside is written
    room = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_quant_cache_read(cache[0], cache[1], scales[0], scales[1], tables,
                             ints(torch, [0, 20, 500]), k_out=room[10:50], v_out=outs[1][:40])
    dsa.dsa_quant_cache_read(cache[0], cache[1], scales[0], scales[1], tables,
                             ints(torch, [30, 2, 9]), k_out=room[10:50], v_out=outs[1][:40])
    torch.cuda.synchronize()
    assert (room[:10] == 7).all() and (room[50:] == 7).all()


@pytest.mark.parametrize("which", ["k_out", "v_out"])
def test_read_into_one_given_output(env, which):
    torch, dsa = env
    pool = Pool(torch, 24, [40, 3], 3, 16, 16, 16)
    cache, scales, tables = pool.gpu()
    c = (cache[0], cache[1], scales[0], scales[1])
    cu = ints(torch, [0, 40, 43])
    want = dsa.dsa_quant_cache_read(*c, tables, cu, total=43, dtype=torch.float16)
    mine = torch.zeros(43, 3, 16, dtype=torch.float16, device="cuda")
    got = dsa.dsa_quant_cache_read(*c, tables, cu, **{which: mine})
    torch.cuda.synchronize()
    assert got[which == "v_out"] is mine
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError, match="total is 42"):
        dsa.dsa_quant_cache_read(*c, tables, cu, total=42, **{which: mine})
    with pytest.raises(TypeError, match="bfloat16"):
        dsa.dsa_quant_cache_read(*c, tables, cu, dtype=torch.bfloat16, **{which: mine})
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dsa.dsa_quant_cache_read(*c, tables, cu, **{which: mine.float()})
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dsa.dsa_quant_cache_read(*c, tables, cu, total=43, dtype=torch.float32)
    with pytest.raises(ValueError, match="total"):
        dsa.dsa_quant_cache_read(*c, tables, cu)


def test_binding_refusals(env):
    """Tensors that do not belong together."""
    torch, dsa = env
    pool = Pool(torch, 25, [40, 3], 2, 64, 16, 8)
    cache, scales, tables = pool.gpu()
    c = dict(k_pages=cache[0], v_pages=cache[1], k_scales=scales[0], v_scales=scales[1],
             tables=tables)
    q, lens = queries(torch, 26, 2, 4, 64, torch.bfloat16), ints(torch, [40, 3])
    k = queries(torch, 27, 5, 2, 64, torch.bfloat16)
    cu = ints(torch, [0, 2, 5])
    bad = [  # changed, the error, what it says
        (dict(k_pages=cache[0].view(torch.uint8)), TypeError, "float8"),
        (dict(v_pages=cache[1][:-1]), ValueError, "do not match"),
        (dict(k_pages=cache[0].permute(0, 1, 3, 2)), ValueError, "k_pages|do not match"),
        (dict(k_scales=scales[0].half()), TypeError, "float32"),
        (dict(k_scales=scales[0][:, :1].expand(-1, 3, -1)), ValueError, "k_scales must be"),
        (dict(v_scales=scales[1][:, :1].contiguous()), ValueError, "do not match"),
        (dict(v_scales=scales[1].transpose(1, 2).contiguous().transpose(1, 2)), ValueError,
         "contiguous"),
        (dict(tables=tables.long()), TypeError, "int32"),
        (dict(tables=tables[0]), ValueError, "2 dimensions"),
        (dict(tables=tables.cpu()), ValueError, "CUDA"),
        (dict(tables=tables.repeat(1, 2)[:, ::2]), ValueError, "unit stride"),
    ]
    for kw, error, match in bad:
        with pytest.raises(error, match=match):
            dsa.dsa_quant_attention(q, lens=lens, **{**c, **kw})
        with pytest.raises(error, match=match):
            dsa.dsa_quant_cache_write(k, k, cu, lens=lens, **{**c, **kw})
    for kw, match in ((dict(q=q[:1]), "do not match"), (dict(q=q[..., :32]), "do not match"),
                      (dict(lens=lens[:1]), "do not match"), (dict(q=q[0]), "3 dimensions"),
                      (dict(out=q[:, :2]), "out must be"), (dict(q=q[:, :3]), "invalid argument")):
        with pytest.raises((ValueError, dsa.DsaError), match=match):
            dsa.dsa_quant_attention(**{**dict(q=q, lens=lens), **c, **kw})
    for kw, match in ((dict(v=k[:4]), "do not match"), (dict(k=k[:, :1], v=k[:, :1]), "match"),
                      (dict(cu=cu[:2]), "cu holds"), (dict(lens=lens[:1]), "cu holds")):
        with pytest.raises(ValueError, match=match):
            dsa.dsa_quant_cache_write(**{**dict(k=k, v=k, cu=cu, lens=lens), **c, **kw})


def test_read_strided(env):
    torch, dsa = env
    pool = Pool(torch, 22, [50, 21], 3, 48, 16, 4)
    cache, scales, tables = pool.gpu()
    wide = torch.full((2, 3, 71, 64), 7.0, dtype=torch.float16, device="cuda")
    outs = [w[..., 8:56].permute(1, 0, 2) for w in wide]
    dsa.dsa_quant_cache_read(cache[0], cache[1], scales[0], scales[1], tables,
                             ints(torch, [0, 50, 71]), k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    for i in (0, 1):
        want = np.concatenate([quant.read(pool.codes, pool.scales, pool.tables, s, n)[i]
                               for s, n in ((0, 50), (1, 21))])
        assert torch.equal(outs[i].cpu(), torch.from_numpy(want).half())
    assert (wide[..., :8] == 7).all() and (wide[..., 56:] == 7).all()


def check_attend(env, pool, q, lens, scale=None, gpu=None, **kw):
    torch, dsa = env
    cache, scales, tables = gpu or pool.gpu()
    out, lse = dsa.dsa_quant_attention(q, cache[0], cache[1], scales[0], scales[1], tables,
                                       ints(torch, lens), scale=scale, **kw)
    torch.cuda.synchronize()
    want = quant.attend(q, pool.codes, pool.scales, pool.tables, lens, scale)
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")
    return out, lse


def queries(torch, seed, batch, heads, dim, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(batch, heads, dim, generator=g) * spread).to(dtype).cuda()


ATTENDS = [[1], [1, 0, 31, 32, 33], [15, 16, 17, 300], [2000, 7, 129], [64] * 20, [0, 0],
           [1025, 511, 513]]
GROUPS = [  # query heads, kv heads, head dim, page, block
    (2, 2, 64, 16, 16), (8, 2, 128, 64, 64), (15, 3, 80, 32, 8), (16, 1, 16, 16, 1),
    (10, 5, 112, 128, 32), (12, 4, 96, 256, 128), (7, 1, 48, 64, 2), (24, 2, 128, 32, 32),
    (8, 1, 32, 32, 16), (17, 1, 64, 16, 16), (9, 1, 128, 16, 4),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("lens", ATTENDS, ids=[str(x) for x in ATTENDS])
@pytest.mark.parametrize("shape", GROUPS, ids=[str(x) for x in GROUPS])
def test_attention_sweep(env, shape, lens, dtype):
    torch, _ = env
    heads, kv_heads, dim, page, block = shape
    pool = Pool(torch, sum(lens) + dim, lens, kv_heads, dim, page, block)
    q = queries(torch, dim, len(lens), heads, dim, getattr(torch, dtype))
    check_attend(env, pool, q, lens)


@pytest.mark.parametrize("heads,kv_heads,dim", [(64, 1, 64), (128, 1, 128), (100, 1, 16),
                                                (66, 2, 80)])
def test_attention_wide_groups(env, heads, kv_heads, dim):
    torch, _ = env
    lens = [400, 33]
    pool = Pool(torch, heads, lens, kv_heads, dim, 32, 16)
    check_attend(env, pool, queries(torch, 1, 2, heads, dim, torch.bfloat16), lens)


@pytest.mark.parametrize("heads,kv_heads", [(3, 3), (15, 3), (27, 3), (16, 1), (40, 2)])
@pytest.mark.parametrize("lens", [[1, 31, 32, 33], [3000, 0, 577]], ids=["short", "long"])
@pytest.mark.parametrize("dim", [80, 96, 112])
def test_attention_heads_between_64_and_128(env, dim, lens, heads, kv_heads):
    torch, _ = env
    pool = Pool(torch, 51, lens, kv_heads, dim, 32, 16)
    check_attend(env, pool, queries(torch, 52, len(lens), heads, dim, torch.float16), lens)


@pytest.mark.parametrize("lens", [[9000], [5000, 1, 0, 12345], [40] * 300, [3000] * 7])
def test_attention_long_and_many(env, lens):
    torch, _ = env
    pool = Pool(torch, 5, lens, 2, 64, 64, 16)
    check_attend(env, pool, queries(torch, 2, len(lens), 6, 64, torch.float16), lens)


def test_attention_moving_maximum(env):
    """Scores that grow along the context, and keys of very different scales."""
    torch, _ = env
    lens = [6000, 4000]
    pool = Pool(torch, 6, lens, 1, 128, 16, 16, low=-10, high=-9)
    for s, n in enumerate(lens):
        for i, p in enumerate(pool.tables[s, :n // 16]):
            pool.scales[0, p] = 2.0 ** (-12 + 8 * i * 16 / n)
            pool.scales[1, p] = 2.0 ** (8 - 12 * i * 16 / n)
    check_attend(env, pool, queries(torch, 3, 2, 8, 128, torch.bfloat16, 0.1), lens)


@pytest.mark.parametrize("scale", [1e-3, 0.125, 3.0, 2e-38])
def test_attention_scale(env, scale):
    torch, _ = env
    pool = Pool(torch, 7, [150], 2, 64, 16, 16)
    check_attend(env, pool, queries(torch, 4, 1, 4, 64, torch.bfloat16, 0.2), [150], scale)


def test_attention_any_scales(env):
    """Scales that are no powers of two, of all sizes, and zeros."""
    torch, _ = env
    rng = np.random.default_rng(8)
    for lo, hi in ((-8, -3), (-40, -20)):
        pool = Pool(torch, 8, [150, 300], 2, 64, 16, 8)
        pool.scales = np.exp2(rng.uniform(lo, hi, pool.scales.shape)).astype(np.float32)
        pool.scales[1, ::3] = 0.0
        check_attend(env, pool, queries(torch, 9, 2, 4, 64, torch.bfloat16, 0.3), [150, 300])
    pool.scales[1] = 0.0
    out, _ = check_attend(env, pool, queries(torch, 9, 2, 4, 64, torch.bfloat16, 0.3), [150, 300])
    assert not out.any()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("size", [1e-3, 1e3, 3e4])
def test_attention_query_sizes(env, dtype, size):
    """Queries whose elements differ by many powers of two from each other."""
    torch, _ = env
    pool = Pool(torch, 10, [90], 1, 64, 16, 16, low=-30, high=-29)
    g = torch.Generator().manual_seed(1)
    q = torch.exp2(torch.randint(-24, 1, (1, 8, 64), generator=g).float()) * size
    q = (q * torch.randn(1, 8, 64, generator=g).clamp(-2, 2)).to(getattr(torch, dtype)).cuda()
    check_attend(env, pool, q, [90])


def test_attention_extreme_queries(env):
    """bf16 queries at both ends of the type's range, brought back by the
    scales of the keys."""
    torch, _ = env
    for e, ks in ((100, -108), (-120, 105), (-132, 115)):
        pool = Pool(torch, 11, [90], 1, 64, 16, 16)
        pool.scales[0] = 2.0 ** ks
        q = torch.randint(1, 3, (1, 4, 64), generator=torch.Generator().manual_seed(2)).double()
        q = (q * 2.0 ** e).to(torch.bfloat16).cuda()
        check_attend(env, pool, q, [90])


@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_attention_special_queries(env, what):
    torch, _ = env
    pool = Pool(torch, 12, [40, 70], 1, 64, 16, 16)
    pool.codes[(pool.codes & 127) == 0] = 1      # infinity times zero is another test's
    q = queries(torch, 5, 2, 4, 64, torch.bfloat16)
    q[1, 2, 3] = float(what)
    check_attend(env, pool, q, [40, 70])


def test_attention_rows_of_infinitely_low_scores(env):
    """All scores -inf: 0 and -inf, as where nothing is seen."""
    torch, _ = env
    pool = Pool(torch, 13, [40], 1, 64, 16, 16)
    pool.codes[0, ..., 0] = 0x38                 # 1
    q = queries(torch, 6, 1, 4, 64, torch.bfloat16)
    q[0, 1, 0] = -math.inf
    out, lse = check_attend(env, pool, q, [40])
    assert not out[0, 1].any() and lse[0, 1] == -math.inf


def test_attention_special_codes_that_are_seen(env):
    torch, _ = env
    pool = Pool(torch, 14, [40, 70, 90], 2, 64, 16, 8)
    at = pool.tables
    pool.codes[0, at[0, 1], 3, 0, 9] = 127                 # a key's: its rows
    pool.codes[1, at[1, 2], 1, 1, 5] = 255                 # a value's: that dimension
    pool.scales[1, at[2, 0], 1, 0] = math.nan
    out, _ = check_attend(env, pool, queries(torch, 7, 3, 6, 64, torch.bfloat16), [40, 70, 90])
    assert out[0, :3].isnan().all() and out[1, 3:, 5].isnan().all()
    assert int(out[1].isnan().sum()) == 3


@pytest.mark.parametrize("dim,page,block", [(64, 16, 16), (128, 64, 4), (80, 32, 32)])
def test_attention_places_that_are_not_seen_hold_anything(env, dim, page, block):
    """NaN codes and scales behind the ends, on pages of no table and of missing
    entries leave the bits as they are."""
    torch, _ = env
    lens = [40, 1, 0, 700, 33]
    pool = Pool(torch, 15, [n + 200 for n in lens], 2, dim, page, block)
    pool.tables[3, 2] = -1
    q = queries(torch, 8, 5, 8, dim, torch.bfloat16)
    out, lse = check_attend(env, pool, q, lens)
    seen = np.zeros(pool.codes.shape[1:3], bool)
    for s, n in enumerate(lens):
        for t in range(n):
            if pool.tables[s, t // page] >= 0:
                seen[pool.tables[s, t // page], t % page] = True
    pool.codes[:, ~seen] = 127
    blocks = seen.reshape(seen.shape[0], page // block, block).any(2)
    pool.scales[:, ~blocks] = math.nan
    again = check_attend(env, pool, q, lens)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    pool.scales[:, ~blocks] = math.inf
    again = check_attend(env, pool, q, lens)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_attention_missing_pages(env):
    torch, _ = env
    lens = [100, 300, 64]
    pool = Pool(torch, 16, lens, 2, 64, 16, 16)
    pool.tables[0, 0], pool.tables[0, 6], pool.tables[1, 3:9] = -1, 9999, -(2 ** 31)
    pool.tables[2, :] = -1
    out, lse = check_attend(env, pool, queries(torch, 9, 3, 4, 64, torch.bfloat16), lens)
    assert not out[2].any() and (lse[2] == -math.inf).all()


def test_attention_lengths_are_clamped(env):
    torch, _ = env
    pool = Pool(torch, 17, [64, 64], 2, 64, 16, 16)
    q = queries(torch, 10, 2, 4, 64, torch.bfloat16)
    check_attend(env, pool, q, [2 ** 31 - 1, -(2 ** 31)])
    check_attend(env, pool, q, [65, -1])


@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (16, 128)])
def test_attention_tables_of_the_longest_length(env, page, dim):
    """A row of pages for all lengths below 2^31, of which the first and the last
    are there: the last tile ends at 2^31, or a page before it."""
    torch, dsa = env
    pool = Pool(torch, 44, [2 * page], 2, dim, page, 16, spare=0)
    cache, scales, _ = pool.gpu()
    c = (cache[0], cache[1], scales[0], scales[1])
    width = (2 ** 31 - 1) // page
    tables = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    tables[0, 0], tables[0, -1] = int(pool.tables[0, 0]), int(pool.tables[0, 1])
    q = queries(torch, 45, 1, 4, dim, torch.bfloat16)
    want = quant.attend(q, pool.codes, pool.scales, pool.tables, [2 * page])
    for n in (width * page, 2 ** 31 - 1):
        out, lse = dsa.dsa_quant_attention(q, *c, tables, ints(torch, [n]))
        ref.check(out, want[0], want[2], "out")
        ref.check(lse, want[1], want[3], "lse")
    # the last page's tokens, written and (its first row's) read back
    k, v = rows(torch, 46, 3, 2, dim, torch.bfloat16)
    held = width * page - 3
    pool.scales[:, pool.tables[0, 1]] = 2.0 ** -9
    scales.copy_(torch.from_numpy(pool.scales))
    dsa.dsa_quant_cache_write(k, v, ints(torch, [0, 3]), *c, tables, ints(torch, [held]))
    model = pool.scales.astype(np.float64)
    quant.write(k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 3], pool.codes, model,
                pool.tables, [2 * page - 3])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(scales.cpu().numpy(), model.astype(np.float32))
    quant.same_codes(cache.view(torch.uint8).cpu().numpy(), pool.codes, "codes")


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch, quant_reference as quant, test_quant_gpu as t
import deepseek_sparse_attention_row_gb300 as dsa

for lens in ([60, 30], [3000, 30]):     # a launch, and two
    pool = t.Pool(torch, 1, [n + 2 for n in lens], 2, 64, 16, 16)
    cache, scales, tables = pool.gpu()
    c = (cache[0], cache[1], scales[0], scales[1])
    q, at = t.queries(torch, 2, 2, 4, 64, torch.bfloat16), t.ints(torch, lens)
    k = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, turns = t.ints(torch, [0, 2, 4]), dsa.rotary_turns([1.0] * 32)
    pos = t.ints(torch, [0, 1, 2, 3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        turned, _ = dsa.dsa_rotary(k, None, pos, turns)
        back = dsa.dsa_quant_cache_read(*c, tables, cu, total=4)
        out, lse = dsa.dsa_quant_attention(q, *c, tables, at)
        dsa.dsa_quant_cache_write(turned, k, cu, *c, tables, at)
    g.replay()
    torch.cuda.synchronize()
    want = quant.attend(q, pool.codes, pool.scales, pool.tables, lens)
    assert ((out.double().cpu() - want[0]).abs() <= want[2]).all()
    assert torch.equal(back[0].double().cpu()[:2],
                       torch.from_numpy(quant.read(pool.codes, pool.scales, pool.tables, 0, 2)[0]))
"""


def test_first_calls_of_a_process_may_be_captured(env):
    import os
    import subprocess
    import sys

    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr


@pytest.mark.parametrize("kv_heads,group", [(40, 1), (7, 40), (2000, 1)])
def test_attention_many_rows(env, kv_heads, group):
    """Rows that do not divide the warps, parts of a group, and more rows than
    warps."""
    torch, _ = env
    lens = [700, 33]
    pool = Pool(torch, 47, lens, kv_heads, 16, 16, 16)
    check_attend(env, pool, queries(torch, 48, 2, kv_heads * group, 16, torch.bfloat16), lens)


@pytest.mark.parametrize("batch", [160, 901, 1823, 5000])
@pytest.mark.parametrize("lens", [[1], [1, 0, 0, 33], [0, 0, 16, 0, 31, 700], [32, 64, 0]],
                         ids=["ones", "some", "one longer", "whole tiles"])
def test_attention_shares_about_a_tile_long(env, batch, lens):
    """About as many short sequences as warps, which then have a tile, or parts of a
    sequence, or nothing at all to do."""
    torch, _ = env
    lens = (lens * batch)[:batch]
    pool = Pool(torch, 49, lens, 1, 16, 16, 16)
    check_attend(env, pool, queries(torch, 50, batch, 1, 16, torch.bfloat16), lens)


def test_attention_strided(env):
    torch, dsa = env
    H, Hkv, D, page, block = 6, 3, 48, 32, 16
    lens = [70, 300]
    pool = Pool(torch, 18, lens, Hkv, D, page, block)
    N = pool.codes.shape[1]
    wide = torch.full((2, Hkv, N, page, 64), 127, dtype=torch.uint8, device="cuda")
    view = wide[..., :D].permute(0, 2, 3, 1, 4)
    view.copy_(torch.from_numpy(pool.codes).cuda())
    scales = torch.full((2, N, 5, page // block, Hkv), math.nan, device="cuda")
    scales[:, :, 2] = torch.from_numpy(pool.scales).cuda()
    table = torch.full((2, 40), 5, dtype=torch.int32, device="cuda")
    table[:, :pool.tables.shape[1]] = ints(torch, pool.tables)
    gpu = (view.view(torch.float8_e4m3fn), scales[:, :, 2], table[:, :pool.tables.shape[1]])
    q = torch.randn(H, 2, D + 8, device="cuda").half()[..., :D].transpose(0, 1)
    out = torch.full((2, H + 2, D + 8), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((H, 2), 7.0, device="cuda").t()
    got = check_attend(env, pool, q, lens, gpu=gpu, out=out[:, 1:H + 1, :D], lse_out=lse)
    assert got[0].data_ptr() == out[:, 1:].data_ptr()
    assert (out[:, 0] == 7).all() and (out[:, -1] == 7).all() and (out[..., D:] == 7).all()


def test_nothing_to_do(env):
    torch, dsa = env
    pool = Pool(torch, 19, [20], 2, 64, 16, 16)
    cache, scales, tables = pool.gpu()
    c = (cache[0], cache[1], scales[0], scales[1])
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_quant_cache_write(k, k, ints(torch, [0, 0]), *c, tables, ints(torch, [3]))
    dsa.dsa_quant_cache_write(k, k, ints(torch, [0]), *c, tables[:0], ints(torch, []))
    got = dsa.dsa_quant_cache_read(*c, tables, ints(torch, [0, 0]), total=0)
    assert got[0].shape == (0, 2, 64)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.dsa_quant_attention(q, *c, tables[:0], ints(torch, []))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # no pages at all, and tables without columns
    empty = [t[:0] for t in c]
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for pages, t in ((empty, ints(torch, [[0, 1], [2, -1]])), (c, ints(torch, [[], []]))):
        out, lse = dsa.dsa_quant_attention(q, *pages, t, ints(torch, [9, 3]))
        got = dsa.dsa_quant_cache_read(*pages, t, ints(torch, [0, 2, 5]), total=5)
        dsa.dsa_quant_cache_write(torch.ones_like(got[0]), got[1], ints(torch, [0, 2, 5]), *pages,
                                  t, ints(torch, [0, 0]))
        torch.cuda.synchronize()
        assert not out.any() and (lse == -math.inf).all() and not got[0].any()
    quant.same_codes(cache.view(torch.uint8).cpu().numpy(), pool.codes, "codes")


def test_streams_and_graphs(env):
    """On another stream, captured and replayed on changed inputs, and two
    graphs whose replays overlap."""
    torch, dsa = env
    lens = [700, 90, 1500]
    pool = Pool(torch, 23, [n + 20 for n in lens], 2, 64, 16, 16)
    cache, scales, tables = pool.gpu()
    c = (cache[0], cache[1], scales[0], scales[1])
    k, v = rows(torch, 24, 6, 2, 64, torch.bfloat16)
    cu, held, after = (ints(torch, x) for x in ([0, 2, 4, 6], lens, [n + 2 for n in lens]))
    q = queries(torch, 25, 3, 8, 64, torch.bfloat16)

    def step():
        dsa.dsa_quant_cache_write(k, v, cu, *c, tables, held)
        back = dsa.dsa_quant_cache_read(*c, tables, cu, total=6)
        return (*back, *dsa.dsa_quant_attention(q, *c, tables, after))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_quant_attention(q, *c, tables, after, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[2]) and torch.equal(got[1], want[3])
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    q.mul_(-0.5)
    graphs[0].replay()
    again = dsa.dsa_quant_attention(q, *c, tables, after)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][2], again[0]) and not torch.equal(again[0], want[2])


def test_calls_at_the_same_time(env):
    """Four threads on streams of their own; and every call repeats bit for bit."""
    torch, dsa = env
    jobs = []
    for i in range(4):
        lens = [900 * i + 40, 200, 3000 - 500 * i]
        pool = Pool(torch, 30 + i, lens, 2, 64, 32, 16)
        cache, scales, tables = pool.gpu()
        args = (queries(torch, i, 3, 8, 64, torch.bfloat16), cache[0], cache[1], scales[0],
                scales[1], tables, ints(torch, lens))
        jobs.append((args, [t.clone() for t in dsa.dsa_quant_attention(*args)]))
    torch.cuda.synchronize()
    bad = []

    def work(args, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = dsa.dsa_quant_attention(*args)
                if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                    bad.append(1)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_own_workspace(env):
    torch, dsa = env
    lens = [3000, 10]
    pool = Pool(torch, 40, lens, 2, 64, 16, 16)
    cache, scales, tables = pool.gpu()
    q = queries(torch, 41, 2, 8, 64, torch.bfloat16)
    args = (q, cache[0], cache[1], scales[0], scales[1], tables, ints(torch, lens))
    want = dsa.dsa_quant_attention(*args)
    need = dsa.quant_attention_workspace_bytes(2, 8, 2, 64, tables.shape[1], 16)
    ws = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")
    got = dsa.dsa_quant_attention(*args, workspace=ws[:need] if need else None)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (ws[need:] == 0xff).all()
    if need:
        with pytest.raises(dsa.DsaError):
            dsa.dsa_quant_attention(*args, workspace=ws[:need - 1])
        with pytest.raises(dsa.DsaError):
            dsa.dsa_quant_attention(*args, workspace=ws[16:16 + need])


def test_parts_merge(env):
    """Two ranges of a context, merged by their log-sum-exps, give the whole."""
    torch, dsa = env
    pool = Pool(torch, 42, [320], 2, 64, 16, 16)
    q = queries(torch, 43, 1, 8, 64, torch.bfloat16)
    cache, scales, tables = pool.gpu()
    c = (cache[0], cache[1], scales[0], scales[1])
    parts = [dsa.dsa_quant_attention(q, *c, t, ints(torch, [n]))
             for t, n in ((tables[:, :7], 112), (tables[:, 7:], 208))]
    merged, lse = dsa.dsa_merge_attn_out(torch.stack([p[0] for p in parts]),
                                         torch.stack([p[1] for p in parts]))
    torch.cuda.synchronize()
    want = quant.attend(q, pool.codes, pool.scales, pool.tables, [320])
    # each part's own rounding and the merge's
    ref.check(merged.transpose(0, 1), want[0], 3 * want[2] + 2.0 ** -7 * want[0].abs().amax(),
              "merged")
    ref.check(lse, want[1], 3 * want[3] + 2.0 ** -20, "merged lse")


@pytest.mark.parametrize("planes,per", [(2, 3), (6, 40), (1, 700)])
def test_fork_and_compaction_carry_scales(env, planes, per):
    """Byte for byte: a copied partial page brings all of its scales, moved pages
    theirs, and nothing else changes. (Pages and tables are the plain calls'.)"""
    torch, dsa = env
    N, page, slots, width = 40, 4, 12, 6
    rng = np.random.default_rng(per)
    cache = rng.integers(-30000, 30000, (planes, N, page, 2, 8)).astype(np.int16)
    wide = rng.standard_normal((planes, N, 2, per)).astype(np.float32)  # [:, :, 1]: another layer's
    refs, lens = np.zeros(N, np.int32), np.zeros(slots, np.int32)
    tables = np.full((slots, width), -1, np.int32)
    ids = list(rng.permutation(N))
    for s in range(6):
        lens[s] = (5, 8, 0, 23, 1, 14)[s]
        for j in range(-(-int(lens[s]) // page)):
            tables[s, j] = ids.pop()
            refs[tables[s, j]] = 1
    state = [[torch.from_numpy(x.copy()).cuda() for x in (cache, refs, tables, lens)]
             for _ in range(2)]
    scales = torch.from_numpy(wide.copy()).cuda()
    pairs = ints(torch, [0, 1, 2, 3, 3, 99]), ints(torch, [6, 7, 8, 9, 10, 11])
    a = dsa.dsa_cache_fork(*state[0], *pairs)
    b = dsa.dsa_cache_fork(*state[1], *pairs, scales=scales[:, :, 0])
    torch.cuda.synchronize()
    assert torch.equal(a, b) and a.tolist() == [0, 0, 0, 0, 0, 2]
    for x, y in zip(*state):
        assert torch.equal(x, y)
    after = state[0][2].cpu().numpy()
    for p, c in ((0, 6), (3, 9), (3, 10)):      # these end inside a page
        j = lens[p] // page
        assert after[c, j] != tables[p, j]
        wide[:, after[c, j], 0] = wide[:, tables[p, j], 0]
    np.testing.assert_array_equal(scales.cpu().numpy(), wide)
    for st in state:
        dsa.dsa_cache_free(*st[1:], ints(torch, [1, 5, 6]))
    used = state[0][1].cpu().numpy() > 0
    a = dsa.dsa_cache_compact(*state[0][:3])
    b = dsa.dsa_cache_compact(*state[1][:3], scales=scales[:, :, 0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for x, y in zip(*state):
        assert torch.equal(x, y)
    moved = 0
    for src, dst in enumerate(a[0].tolist()):
        if used[src] and dst != src:
            wide[:, dst, 0] = wide[:, src, 0]
            moved += 1
    assert moved > 0
    np.testing.assert_array_equal(scales.cpu().numpy(), wide)


def test_forked_samples_of_an_8_bit_cache(env):
    """A sample forked from a prompt attends to the same bits; it grows, its block's
    scale with it, the prompt stays as it was; compaction changes no bit."""
    torch, dsa = env
    Hkv, D, page, block, N = 2, 64, 32, 16, 20
    pool = Pool(torch, 60, [75] + [0] * 3, Hkv, D, page, block, spare=N - 3)
    N = pool.codes.shape[1]
    pool.tables = np.concatenate([pool.tables, np.full((4, 1), -1, np.int32)], 1)
    cache, scales, tables = pool.gpu()
    refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    refs[tables[0, :3].long()] = 1
    lens = ints(torch, [75, 0, 0, 0])
    q = queries(torch, 61, 4, 8, D, torch.bfloat16)
    q[1:] = q[0]
    c = (cache[0], cache[1], scales[0], scales[1])
    first = dsa.dsa_quant_attention(q, *c, tables, lens)
    status = dsa.dsa_cache_fork(cache, refs, tables, lens, ints(torch, [0, 0]),
                                ints(torch, [2, 3]), scales=scales)
    assert status.tolist() == [0, 0]
    got = dsa.dsa_quant_attention(q, *c, tables, lens)
    for i in (0, 2, 3):
        assert torch.equal(got[0][i], first[0][0]) and torch.equal(got[1][i], first[1][0])
    k, v = rows(torch, 62, 1, Hkv, D, torch.bfloat16)
    dsa.dsa_quant_cache_write(k * 100, v * 100, ints(torch, [0, 0, 0, 1, 1]), *c, tables, lens)
    lens[2] += 1
    grown = dsa.dsa_quant_attention(q, *c, tables, lens)
    for i in (0, 3):
        assert torch.equal(grown[0][i], first[0][0]) and torch.equal(grown[1][i], first[1][0])
    assert not torch.equal(grown[0][2], first[0][0])
    host = (cache.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), tables.cpu().numpy())
    want = quant.attend(q, *host, lens.cpu().numpy())
    ref.check(grown[0], want[0], want[2], "out")
    dsa.dsa_cache_free(refs, tables, lens, ints(torch, [0]))
    dsa.dsa_cache_compact(cache, refs, tables, scales=scales)
    moved = dsa.dsa_quant_attention(q, *c, tables, lens)
    torch.cuda.synchronize()
    assert int(tables.max()) == 3               # two shared pages, two of their own
    assert torch.equal(moved[0][2:], grown[0][2:]) and torch.equal(moved[1][2:], grown[1][2:])


def test_serving_round(env):
    """Two prompts turned by their positions and written, chunk by chunk; the
    second chunk attends to the cache read back; then decode steps, each written
    and attended to."""
    torch, dsa = env
    H, Hkv, D, page, N, block = 8, 2, 64, 16, 24, 16
    g = torch.Generator().manual_seed(50)
    turns = dsa.rotary_turns(dsa.rotary_frequencies(D))
    plans = [[75, 30], [20, 44], [1, 1], [1, 1]]            # tokens of each step and sequence
    total = [sum(p[s] for p in plans) for s in (0, 1)]
    q, k, v = ([torch.randn(n, h, D, generator=g).bfloat16().cuda() for n in total]
               for h in (H, Hkv, Hkv))
    cache = torch.zeros((2, N, page, Hkv, D), dtype=torch.uint8, device="cuda")
    cache = cache.fill_(127).view(torch.float8_e4m3fn)
    scales = torch.full((2, N, page // block, Hkv), math.nan, device="cuda")
    c = (cache[0], cache[1], scales[0], scales[1])
    tables = ints(torch, np.random.default_rng(0).permutation(N)[:16].reshape(2, 8))
    held = [0, 0]
    codes = cache.view(torch.uint8).cpu().numpy()
    model = scales.cpu().numpy().astype(np.float64)
    for plan in plans:
        cut = [slice(a, a + n) for a, n in zip(held, plan)]
        qs, ks, vs = (torch.cat([t[s][cut[s]] for s in (0, 1)]) for t in (q, k, v))
        pos = ints(torch, [i for s in (0, 1) for i in range(held[s], held[s] + plan[s])])
        qs, ks = dsa.dsa_rotary(qs, ks, pos, turns)
        dsa.dsa_quant_cache_write(ks, vs, ints(torch, offsets(plan)), *c, tables,
                                  ints(torch, held))
        quant.write(ks.double().cpu().numpy(), vs.double().cpu().numpy(), offsets(plan), codes,
                    model, tables.cpu().numpy(), held)
        held = [a + n for a, n in zip(held, plan)]
        args = codes, model.astype(np.float32), tables.cpu().numpy()
        if max(plan) > 1:
            kk, vv = dsa.dsa_quant_cache_read(*c, tables, ints(torch, offsets(held)),
                                              total=sum(held))
            out, lse = dsa.dsa_prompt_attention(qs, kk, vv, ints(torch, offsets(plan)),
                                                ints(torch, offsets(held)))
            want = ref.prompt(qs, kk, vv, offsets(plan), offsets(held), True)
            plain = np.concatenate([quant.read(*args, s, held[s]) for s in (0, 1)], 1)
            assert np.array_equal(kk.double().cpu().numpy(), plain[0])
            assert np.array_equal(vv.double().cpu().numpy(), plain[1])
        else:
            out, lse = dsa.dsa_quant_attention(qs, *c, tables, ints(torch, held))
            want = quant.attend(qs, *args, held)
        torch.cuda.synchronize()
        ref.check(out, want[0], want[2], "out")
        ref.check(lse, want[1], want[3], "lse")
