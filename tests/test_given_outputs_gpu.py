"""Outputs that the caller gives to the rotary and 8-bit cache operators: where they may
lie, and what autograd learns of their being written."""

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


T, H, HKV, D = 12, 4, 2, 32


def turning(torch, dsa):
    return (torch.arange(T, dtype=torch.int32, device="cuda"),
            dsa.rotary_turns(dsa.rotary_frequencies(D)))


def flat(torch, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).cuda()


def at(torch, x, offset, heads, token, head):
    return torch.as_strided(x, (T, heads, D), (token, head, 1), offset)


ROW = H * D
OVERLAPS = [  # q, k, q_out, k_out as (offset, heads, token stride, head stride) of one buffer
    ((0, H, ROW, D), None, (D, H, ROW, D), None),               # a head further
    ((0, H, ROW, D), None, (ROW, H, ROW, D), None),             # a token further
    ((ROW, H, ROW, D), None, (0, H, ROW, D), None),             # a token in front
    ((0, H, ROW, D), None, (3, H, ROW, D), None),               # some elements further
    ((0, H, ROW, D), None, (T * ROW - 1, H, ROW, D), None),     # one element in common
    ((0, H, ROW, D), None, (0, H, D, T * D), None),             # heads in front of tokens
    ((0, H, ROW, D), None, (40 * ROW, H, 16, D * T), None),     # rows of the output overlap
    ((0, H, ROW, D), None, (40 * ROW, H, ROW, 0), None),
    ((0, 2, ROW, D), (0, 2, ROW, D), (9000, 2, ROW, D), (0, 2, ROW, D)),   # q is read, too
    ((0, 2, ROW, D), (2 * D, 2, ROW, D), (2 * D, 2, ROW, D), (9000, 2, ROW, D)),
    ((0, 2, ROW, D), (2 * D, 2, ROW, D), (2 * D, 2, ROW, D), (0, 2, ROW, D)),  # exchanged
    ((0, 2, ROW, D), (2 * D, 2, ROW, D), (4096, 2, ROW, D), (4096, 2, ROW, D)),
    ((0, 2, ROW, D), (2 * D, 2, ROW, D), (4096, 2, ROW, D), (4096 + D, 2, ROW, D)),
    ((0, 2, 3 * D, D), None, (2 * D, 2, 5 * D, D), None),       # steps of another length
]


@pytest.mark.parametrize("where", OVERLAPS, ids=str)
def test_rotary_refuses_outputs_that_overlap(env, where):
    torch, dsa = env
    x = flat(torch, 20000)
    was = x.clone()
    q, k, qo, ko = (None if w is None else at(torch, x, *w) for w in where)
    positions, turns = turning(torch, dsa)
    with pytest.raises(ValueError, match="overlap|apart"):
        dsa.dsa_rotary(q, k, positions, turns, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert torch.equal(x, was)


APART = [
    ((0, H, ROW, D), None, (T * ROW, H, ROW, D), None),                      # one behind the other
    ((0, 2, ROW, D), (2 * D, 2, ROW, D), (0, 2, ROW, D), (2 * D, 2, ROW, D)),   # a fused row in place
    ((0, 1, ROW, D), (2 * D, 1, ROW, D), (D, 1, ROW, D), (3 * D, 1, ROW, D)),   # gaps of a fused row
    ((0, H, 2 * ROW, 2 * D), None, (D, H, 2 * ROW, 2 * D), None),              # halves of wider heads
    ((D, H, 2 * ROW, 2 * D), None, (0, H, 2 * ROW, 2 * D), None),
    ((0, 2, 2 * D, T * 2 * D), (D, 2, 2 * D, T * 2 * D),
     (0, 2, 2 * D, T * 2 * D), (D, 2, 2 * D, T * 2 * D)),                      # heads first, in place
    ((0, 2, 6 * D, D), None, (3 * D, 2, 6 * D, 2 * D), None),                  # other steps
    ((0, 1, 4 * D, D), None, (2 * D, 2, 8 * D, 8 * D * T), None),
]


@pytest.mark.parametrize("where", APART, ids=str)
def test_rotary_takes_interleaved_outputs(env, where):
    torch, dsa = env
    x = flat(torch, 20000, 1)
    q, k, qo, ko = (None if w is None else at(torch, x, *w) for w in where)
    if qo.shape != q.shape:
        q = q.expand(qo.shape)
    positions, turns = turning(torch, dsa)
    want = dsa.dsa_rotary(q, k, positions, turns)
    got = dsa.dsa_rotary(q, k, positions, turns, q_out=qo, k_out=ko)
    for a, b in zip(got, want):
        assert b is None or torch.equal(a, b)


def cache(torch):
    codes = torch.zeros(2, 5, 16, HKV, D, dtype=torch.uint8, device="cuda").view(
        torch.float8_e4m3fn)
    scales = torch.ones(2, 5, 1, HKV, device="cuda")
    tables = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32, device="cuda")
    return codes, scales, tables, torch.tensor([20, 9], dtype=torch.int32, device="cuda")


def test_read_refuses_outputs_that_overlap(env):
    torch, dsa = env
    codes, scales, tables, _ = cache(torch)
    cu = torch.tensor([0, 7, 12], dtype=torch.int32, device="cuda")
    x = torch.zeros(T, 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    args = codes[0], codes[1], scales[0], scales[1], tables, cu
    for k, v in ((x[:, :2], x[:, :2]), (x[:, :2], x[:, 1:3]),
                 (x[:1, :2].expand(T, 2, D), x[:, 2:])):
        with pytest.raises(ValueError, match="overlap|apart"):
            dsa.dsa_quant_cache_read(*args, k_out=k, v_out=v)
    dsa.dsa_quant_cache_read(*args, k_out=x[:, :2], v_out=x[:, 2:])


def counted(tensors, call):
    was = [t._version for t in tensors]
    call()
    assert all(t._version > v for t, v in zip(tensors, was))


def test_writing_is_counted(env):
    """Version counters move, so that a backward pass finds that what it kept is gone."""
    torch, dsa = env
    positions, turns = turning(torch, dsa)
    q, k = (flat(torch, T * n * D, n).view(T, n, D) for n in (H, HKV))
    counted((q, k), lambda: dsa.dsa_rotary(q, k, positions, turns, q_out=q, k_out=k))
    counted((q,), lambda: dsa.dsa_rotary(q, k, positions, turns, q_out=q))
    codes, scales, tables, lens = cache(torch)
    pages = codes[0], codes[1], scales[0], scales[1], tables
    x = torch.randn(3, HKV, D, device="cuda").bfloat16()
    cu = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    counted((codes, scales), lambda: dsa.dsa_quant_cache_write(x, x, cu, *pages, lens))
    y, z = torch.empty_like(x), torch.empty_like(x)
    counted((y, z), lambda: dsa.dsa_quant_cache_read(*pages, cu, k_out=y, v_out=z))
    q1 = torch.randn(2, H, D, device="cuda").bfloat16()
    out, lse = torch.empty_like(q1), torch.empty(2, H, device="cuda")
    counted((out, lse), lambda: dsa.dsa_quant_attention(q1, *pages, lens, out=out, lse_out=lse))
    with torch.inference_mode():  # such tensors have no counter
        y = torch.empty_like(x)
        dsa.dsa_quant_cache_read(*pages, cu, k_out=y, v_out=z)
    dsa.dsa_quant_cache_read(*pages, cu, k_out=y, v_out=z)


def test_a_gradient_through_what_was_turned_in_place_is_refused(env):
    torch, dsa = env
    positions, turns = turning(torch, dsa)
    w = torch.ones(T, H, D, device="cuda", requires_grad=True)
    q = flat(torch, T * H * D).view(T, H, D)
    loss = (q * w).sum()  # keeps q
    dsa.dsa_rotary(q, None, positions, turns, q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_that_require_a_gradient_are_refused(env):
    """Their graphs would not know of the call: the gradient of what was turned in place
    would come back without the turn."""
    torch, dsa = env
    positions, turns = turning(torch, dsa)
    x = flat(torch, T * H * D).view(T, H, D).requires_grad_()
    k = flat(torch, T * HKV * D).view(T, HKV, D)
    q = x * 2
    for kw in (dict(q_out=q), dict(q_out=torch.empty_like(q, requires_grad=True)),
               dict(k_out=torch.empty_like(k, requires_grad=True))):
        with pytest.raises(ValueError, match="requires a gradient"):
            dsa.dsa_rotary(q, k, positions, turns, **kw)
    want = dsa.dsa_rotary(q, k, positions, turns)
    with torch.no_grad():
        got = dsa.dsa_rotary(q, k, positions, turns, q_out=q)
    assert got[0] is q and torch.equal(q, want[0])
    y = (x * 2).detach()
    assert torch.equal(dsa.dsa_rotary(y, k, positions, turns, q_out=y)[0], want[0])
    codes, scales, tables, lens = cache(torch)
    pages = codes[0], codes[1], scales[0], scales[1], tables
    cu = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    z = torch.empty(3, HKV, D, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="v_out requires"):
        dsa.dsa_quant_cache_read(*pages, cu, k_out=z.detach(), v_out=z)
    q1 = torch.zeros(2, H, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="lse_out requires"):
        dsa.dsa_quant_attention(q1, *pages, lens, lse_out=torch.empty(
            2, H, device="cuda", requires_grad=True))
