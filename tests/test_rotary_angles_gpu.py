"""Small angles of the rotary positions against their definition in 64 bits, where one
element of each pair is 0, so that an output is a cosine or a sine times the other.

The bound, with u = 2^-24: the rest of the angle is rounded to fp32, u of itself, which
moves a sine by no more than u of itself and a cosine (at most an eighth of a turn away)
by less; sincospi is good to an ulp, 2u; factor is rounded to fp32 (u) and multiplied
(u); the product is rounded once (u): 6u of the output, 7u with second-order terms. 16-bit
outputs are rounded once more, h = eps / 2 of themselves (none here is subnormal)."""

import math

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


def frequencies(dsa, which):
    if which == "near quarters":  # cosines, too, get small
        return [(n + x) * math.pi / 2 for n in (1, 2, 3, 4)
                for x in (1e-3, -1e-3, 1e-5, -1e-6, 1e-7, -1e-8)]
    base, stretch = which
    return dsa.rotary_frequencies(128, base, stretch=stretch).tolist()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("which", [(1e4, 1.0), (5e5, 8.0), (1e7, 4.0), "near quarters"], ids=str)
def test_small_angles(env, which, interleaved, transpose, dtype):
    torch, dsa = env
    freq = frequencies(dsa, which)
    pairs, factor = len(freq), 1.1
    positions = [0, 1, -1, 2, 3, 5, -17, 100]
    turns = dsa.rotary_turns(freq)
    # signed fractions of a turn from whole numbers; (p F) mod 2^64 is exact
    whole = [[(p * int(f) + 2 ** 63) % 2 ** 64 - 2 ** 63 for f in turns.tolist()]
             for p in positions]
    t = torch.tensor([[x / 2.0 ** 64 * 2 * math.pi for x in row] for row in whole],
                     dtype=torch.float64)[:, None] * (-1 if transpose else 1)
    g = torch.Generator().manual_seed(3)
    dt = getattr(torch, dtype)
    h = torch.finfo(dt).eps / 2 if dt is not torch.float32 else 0.0
    for first in (True, False):  # which element of a pair is not 0
        x = (torch.rand(len(positions), 2, pairs, generator=g) + 1).to(dt)
        y = torch.zeros_like(x)
        parts = (x, y) if first else (y, x)
        q = torch.stack(parts, -1).flatten(-2) if interleaved else torch.cat(parts, -1)
        got, _ = dsa.dsa_rotary(q.cuda(), None, torch.tensor(positions, dtype=torch.int32).cuda(),
                                turns, interleaved=interleaved, factor=factor,
                                transpose=transpose)
        got = got.double().cpu()
        a, b = ((got[..., 0::2], got[..., 1::2]) if interleaved
                else (got[..., :pairs], got[..., pairs:]))
        x = x.double() * factor
        want = (x * t.cos(), x * t.sin()) if first else (-x * t.sin(), x * t.cos())
        for z, w in zip((a, b), want):
            # what is 0 by definition (position 0, whole quarters) is to be 0
            w = torch.where(w.abs() < 1e-15, 0.0, w)
            tol = 7 * 2.0 ** -24 * w.abs()
            tol = tol + h * (w.abs() + tol)
            bad = (z - w).abs() > tol
            assert not bad.any(), (first, int(bad.sum()), bad.nonzero()[0].tolist(),
                                   float(((z - w).abs() / w.abs().clamp(min=1e-30)).max()))
