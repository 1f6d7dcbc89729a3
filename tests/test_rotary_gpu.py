"""Rotary positions against their definition in 64 bits.

The bound of an output, with u = 2^-24 and h half a step of its type: cosine and
sine are off by at most 2^-23 (an ulp, and the rounding of the angle's rest, at
most an eighth of a turn, to fp32), times factor in fp32 u more, two products and
a sum 2u: (2^-23 + 4u) factor (|a| + |b|), and h of the result (below fp16's
normal range 2^-25, below bf16's and fp32's nothing that is tested)."""

import math

import numpy as np
import pytest

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


def turned(torch, x, pos, freq, interleaved, factor, transpose):
    """(outputs, sizes |a| + |b| of what is turned) in fp64."""
    y = x.double().cpu()
    n = 2 * len(freq)
    # the angle's fraction of a turn, exact: integers of any size
    turns = [round(float(f) / (2 * math.pi) * 2.0 ** 64) for f in freq]
    t = np.array([[(int(p) * f) % 2 ** 64 / 2 ** 64 for f in turns] for p in pos])
    t = torch.from_numpy(2 * math.pi * t.reshape(len(pos), len(turns)))[:, None]
    if transpose:
        t = -t
    one, two = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2),
                                                                      slice(n // 2, n))
    a, b = y[..., one].clone(), y[..., two].clone()
    size = torch.zeros_like(y)
    size[..., one] = size[..., two] = abs(factor) * (a.abs() + b.abs())
    y[..., one] = factor * (a * t.cos() - b * t.sin())
    y[..., two] = factor * (b * t.cos() + a * t.sin())
    return y, size


def check(torch, got, want, size, what):
    h = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu()
    tol = (2.0 ** -23 + 4 * 2.0 ** -24) * size
    tol = tol + h * (want.abs() + tol) * (size > 0) + (2.0 ** -25 if h == 2.0 ** -11 else 0)
    bad = (got - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def make(torch, seed, tokens, heads, kv_heads, dim, dtype, far=5000):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(tokens, heads, dim, generator=g).to(dtype).cuda()
    k = torch.randn(tokens, kv_heads, dim, generator=g).to(dtype).cuda()
    pos = torch.randint(-far, far, (tokens,), generator=g, dtype=torch.int32)
    return q, k, pos


def run(env, q, k, pos, freq, interleaved=False, factor=1.0, transpose=False, **kw):
    torch, dsa = env
    was = q.clone(), None if k is None else k.clone()
    got = dsa.dsa_rotary(q, k, pos.cuda(), dsa.rotary_turns(freq), interleaved=interleaved,
                         factor=factor, transpose=transpose, **kw)
    torch.cuda.synchronize()
    for x, y, what in zip(was, got, "qk"):
        if x is not None:
            want, size = turned(torch, x, pos.tolist(), freq, interleaved, factor, transpose)
            check(torch, y, want, size, what)
    return got


SHAPES = [  # tokens, heads, kv heads, head dim, turned elements
    (1, 1, 1, 2, 2), (7, 8, 2, 64, 64), (33, 5, 1, 128, 128), (3, 4, 4, 96, 40), (9, 3, 2, 44, 12),
    (5, 2, 1, 33, 18), (130, 32, 8, 128, 64), (2, 1, 3, 122, 122), (4, 2, 2, 64, 0),
    (300, 2, 2, 66, 34),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(x) for x in SHAPES])
def test_sweep(env, shape, transpose, interleaved, dtype):
    torch, dsa = env
    *sizes, n = shape
    q, k, pos = make(torch, sum(shape), *sizes, getattr(torch, dtype))
    freq = dsa.rotary_frequencies(n).tolist() if n else []
    run(env, q, k, pos, freq, interleaved, 1.0 if n % 4 else 1.375, transpose)


@pytest.mark.parametrize("far", [2 ** 31 - 1, -(2 ** 31), 10 ** 6, 0])
def test_far_positions(env, far):
    """The angle is as good at 2^31 as at 0."""
    torch, dsa = env
    q, k, _ = make(torch, 1, 4, 2, 1, 64, torch.float32)
    pos = torch.tensor([far, max(far - 1, -(2 ** 31)), 1, -1], dtype=torch.int32)
    run(env, q, k, pos, dsa.rotary_frequencies(64).tolist())


def test_quarter_turns(env):
    """Frequencies that are fractions of a turn: cosines of exactly 0 and 1."""
    torch, dsa = env
    q = torch.randn(9, 1, 8, device="cuda")
    pos = torch.arange(9, dtype=torch.int32)
    freq = [2 * math.pi / 4, 2 * math.pi / 2, 2 * math.pi, -2 * math.pi / 4]
    out, _ = run(env, q, None, pos, freq)
    a, b = q[..., :4], q[..., 4:]
    assert torch.equal(out[1, 0, 0], -b[1, 0, 0]) and torch.equal(out[1, 0, 4], a[1, 0, 0])
    assert torch.equal(out[2, 0, 0], -a[2, 0, 0]) and torch.equal(out[4, 0, 0], a[4, 0, 0])
    assert torch.equal(out[..., 2], a[..., 2]) and torch.equal(out[1, 0, 3], b[1, 0, 3])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,n", [(64, 64), (96, 40), (30, 14)])
def test_in_place(env, dim, n, interleaved):
    torch, dsa = env
    q, k, pos = make(torch, 5, 50, 6, 2, dim, torch.bfloat16)
    freq = dsa.rotary_frequencies(n).tolist()
    want = run(env, q, k, pos, freq, interleaved)
    got = run(env, q, k, pos, freq, interleaved, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_strided(env, shift, interleaved):
    """Parts of a fused projection, at addresses of every alignment, to heads in
    front of tokens; what lies between is left as it was."""
    torch, dsa = env
    T, H, Hkv, D, n = 21, 4, 2, 40, 24
    both = torch.randn(T, H + Hkv + 1, D + 8, device="cuda").half()
    q, k = both[:, :H, shift:D + shift], both[:, H + 1:, shift:D + shift]
    wide = torch.full((H + Hkv, T, D + 8), 7.0, dtype=torch.float16, device="cuda")
    outs = wide[:H, :, 8 - shift:D + 8 - shift], wide[H:, :, 8 - shift:D + 8 - shift]
    pos = torch.arange(T, dtype=torch.int32)
    run(env, q, k, pos, dsa.rotary_frequencies(n).tolist(), interleaved,
        q_out=outs[0].transpose(0, 1), k_out=outs[1].transpose(0, 1))
    assert (wide[..., :8 - shift] == 7).all() and (wide[..., D + 8 - shift:] == 7).all()


def test_broadcast_and_single(env):
    """A head for all heads, one token's view of any stride, no k, no heads."""
    torch, dsa = env
    freq = dsa.rotary_frequencies(64).tolist()
    q = torch.randn(12, 1, 64, device="cuda").bfloat16().expand(12, 5, 64)
    run(env, q, None, torch.arange(12, dtype=torch.int32), freq)
    one = torch.as_strided(torch.randn(500, device="cuda"), (1, 3, 64), (7, 64, 1))
    run(env, one, one[:, :1], torch.tensor([9], dtype=torch.int32), freq)
    none = torch.zeros(4, 0, 64, device="cuda")
    got = dsa.dsa_rotary(none, torch.ones(4, 2, 64, device="cuda"),
                         torch.zeros(4, dtype=torch.int32, device="cuda"), dsa.rotary_turns(freq))
    assert got[0].shape == (4, 0, 64) and (got[1] == 1).all()
    empty = torch.zeros(0, 3, 64, device="cuda")
    got = dsa.dsa_rotary(empty, None, torch.zeros(0, dtype=torch.int32, device="cuda"),
                         dsa.rotary_turns(freq))
    assert got[0].shape == (0, 3, 64) and got[1] is None


def test_transpose_is_the_gradient(env):
    """<g, R x> = <R^T g, x>, against differences in fp64 of the definition;
    and with factor 1 it turns back."""
    torch, dsa = env
    freq = dsa.rotary_frequencies(48, stretch=4.0, method="parts").tolist()
    q, k, pos = make(torch, 6, 17, 3, 2, 64, torch.float32)
    turns = dsa.rotary_turns(freq)
    for interleaved in (False, True):
        g = torch.randn(17, 3, 64, device="cuda")
        grad, _ = dsa.dsa_rotary(g, None, pos.cuda(), turns, interleaved=interleaved, factor=1.25,
                                 transpose=True)
        g64, x64 = g.double().cpu(), q.double().cpu()
        step = 2.0 ** -20
        for t, h, d in ((0, 0, 0), (3, 1, 23), (16, 2, 24), (9, 0, 47), (5, 1, 60)):
            up, down = x64.clone(), x64.clone()
            up[t, h, d] += step
            down[t, h, d] -= step
            f = [(turned(torch, x, pos.tolist(), freq, interleaved, 1.25, False)[0] * g64).sum()
                 for x in (up, down)]
            # linear: the difference quotient is exact but for fp64's rounding of f (2^-53 * |f|
            # / step, |f| < 2^12: 2^-21); the kernel is held to 2^-20 of the gradients' size
            want = float((f[0] - f[1]) / (2 * step))
            assert abs(float(grad[t, h, d]) - want) < 2.0 ** -20 * 8 + 2.0 ** -20 * 8
        there, _ = dsa.dsa_rotary(q, None, pos.cuda(), turns, interleaved=interleaved)
        back, _ = dsa.dsa_rotary(there, None, pos.cuda(), turns, interleaved=interleaved,
                                 transpose=True)
        # two turns, each within (2^-23 + 4u + u) of the pair's size, at most 2^(1/2) |(a, b)|
        assert (back - q).abs().max() < 4 * 6 * 2.0 ** -24 * 2 * q.abs().max()


def test_infinities_stay_in_their_pairs(env):
    torch, dsa = env
    q, _, pos = make(torch, 7, 3, 2, 1, 64, torch.bfloat16)
    q[1, 0, 5], q[2, 1, 33] = math.inf, math.nan
    out, _ = dsa.dsa_rotary(q, None, pos.cuda(), dsa.rotary_turns(dsa.rotary_frequencies(64)))
    bad = ~out.isfinite()
    want = torch.zeros_like(bad)
    want[1, 0, [5, 37]] = want[2, 1, [1, 33]] = True
    assert torch.equal(bad, want)


def test_long(env):
    """More than 2^31 elements between the first token and the last."""
    torch, dsa = env
    T, step = 3, 2 ** 30 + 64
    big = torch.zeros(2 * step + 256, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(big, (T, 2, 64), (step, 64, 1))
    q.copy_(torch.randn(T, 2, 64, device="cuda"))
    freq = dsa.rotary_frequencies(64).tolist()
    run(env, q, None, torch.tensor([1, 2, 3], dtype=torch.int32), freq, q_out=q)


def test_streams_and_graphs(env):
    torch, dsa = env
    q, k, pos = make(torch, 8, 40, 8, 2, 64, torch.bfloat16)
    turns, at = dsa.rotary_turns(dsa.rotary_frequencies(64)), pos.cuda()
    want = dsa.dsa_rotary(q, k, at, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_rotary(q, k, at, turns, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = dsa.dsa_rotary(q, k, at, turns)
    at.add_(1)
    g.replay()
    want = dsa.dsa_rotary(q, k, at, turns)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refusals(env):
    torch, dsa = env
    q, k, pos = make(torch, 9, 4, 2, 1, 64, torch.bfloat16)
    at, turns = pos.cuda(), dsa.rotary_turns(dsa.rotary_frequencies(64))
    for kw, match in ((dict(k=k[:3]), "k must be"), (dict(k=k[..., :32]), "k must be"),
                      (dict(positions=at[:3]), "positions holds"),
                      (dict(turns=torch.cat([turns, turns])), "do not fit"),
                      (dict(turns=turns.view(2, 16)), "1 dimensions"),
                      (dict(turns=torch.cat([turns, turns])[::2]), "contiguous"),
                      (dict(positions=pos), "CUDA"), (dict(q_out=k), "q_out must be"),
                      (dict(k=None, k_out=k), "without k"),
                      (dict(q_out=q.view(2, 4, 64).transpose(0, 1)), "itself")):
        with pytest.raises(ValueError, match=match):
            dsa.dsa_rotary(**{**dict(q=q, k=k, positions=at, turns=turns), **kw})
    for kw in (dict(k=k.half()), dict(turns=turns.int()), dict(q=q.double())):
        with pytest.raises(TypeError):
            dsa.dsa_rotary(**{**dict(q=q, k=k, positions=at, turns=turns), **kw})
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rotary(q, k, at, turns, factor=math.inf)
