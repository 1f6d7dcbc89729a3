"""How exact attention on 8-bit pages is, where its error shows: values that cancel, and
scales at the lowest end of fp32.

The bound is that of quant_reference.attend but for the weights, which are two fp16
numbers, the nearest one and what is left of it: H = 2^-22 of a weight instead of 2^-11
(the rest is exact in fp32 and at most 2^-11 of the weight), or 2^-32 of the largest one.
With n tokens of one scale, D dimensions, u = 2^-24:
  E = (2 D + 12) u max_j |x_j|' + 3 u   (|x|' with absolute values in the product)
  L = 6 u (2 max_j |x_j|' + 2 |log2 sv|)
  A = 2 (H + 2 (ln2 (E + L) + 3 2^-22 + 4 n u))
  tol = A sum_j w_j |v_j| + 2 2^-32 max_j(w_j sv) sum_j |code_j| + h |out|, h = eps / 2,
of which the last one is not doubled, and 2^-25 more for fp16 results below 2^-14."""

import math

import numpy as np
import pytest

import quant_reference as quant

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_row_gb300 as dsa

    assert torch.cuda.is_available(), "these tests need a CUDA device"
    yield torch, dsa
    torch.cuda.synchronize()


def check(torch, got, q, k, v, sv, scale):
    """got [heads, D] against q [heads, D] over keys and value codes [n, D] (fp64)."""
    n, dim = k.shape
    c = scale / math.log(2.0)
    x, size = c * (q @ k.T), c * (q.abs() @ k.abs().T).max()
    w = torch.softmax(x * math.log(2.0), -1)
    want = w @ v * sv
    e = (2 * dim + 12) * U * size + 3 * U
    d = 6 * U * (2 * size + 2 * abs(math.log2(sv)))
    a = 2 * (2.0 ** -22 + 2 * (math.log(2.0) * (e + d) + 3 * 2.0 ** -22 + 4 * n * U))
    tol = a * (w @ v.abs()) * sv + torch.finfo(got.dtype).eps / 2 * want.abs()
    tol += 2.0 ** -31 * w.amax(-1, keepdim=True) * sv * v.abs().sum(0)
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = (got.double().cpu() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(),
                           float(((got.double().cpu() - want).abs() / tol).max()))


# heads of a group, head dim, tokens of a sequence, sequences: one launch and two, eight
# columns and sixteen, whole products and tails
CANCEL = [(3, 64, 2, 1), (1, 16, 96, 3), (8, 128, 2, 40), (16, 128, 64, 5), (12, 80, 34, 3),
          (5, 80, 2, 300), (16, 96, 32, 2), (9, 64, 200, 200), (40, 48, 6, 1), (4, 112, 700, 9)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("shape", CANCEL, ids=str)
def test_values_that_cancel(env, shape, dtype):
    """Keys in pairs that are almost alike, whose values are opposite: outputs are the
    differences of weights, which fp16 alone would not hold."""
    torch, dsa = env
    group, dim, n, batch = shape
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(sum(shape))
    page = 32
    pages = -(-n // page)
    codes = np.zeros((2, pages * page, 1, dim), np.uint8)
    codes[0, :n:2, 0] = quant.encode(rng.normal(size=(len(range(0, n, 2)), dim)))
    codes[0, 1:n:2] = codes[0, :n:2][:len(range(1, n, 2))]
    codes[0, 1:n:2, 0, 0] ^= 1  # the last bit of one element
    codes[1, :n:2, 0] = quant.encode(rng.uniform(1, 2, size=(len(range(0, n, 2)), dim)))
    codes[1, 1:n:2] = codes[1, :n:2][:len(range(1, n, 2))] ^ 128
    scales = np.ones((2, pages, 1, 1), np.float32)
    cache = torch.from_numpy(codes.reshape(2, pages, page, 1, dim)).cuda().view(
        torch.float8_e4m3fn)
    s = torch.from_numpy(scales).cuda()
    q = torch.from_numpy(rng.normal(size=(batch, group, dim)) * 2.0 ** -4).to(dt)
    tables = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out, _ = dsa.dsa_quant_attention(q.cuda(), cache[0], cache[1], s[0], s[1], tables, lens,
                                     scale=0.25)
    k, v = (torch.from_numpy(quant.VALUES[codes[i, :n, 0]]) for i in (0, 1))
    for b in range(batch):
        check(torch, out[b], q[b].double(), k, v, 1.0, 0.25)


@pytest.mark.parametrize("power", [-100, -119, -123, -126])
@pytest.mark.parametrize("n,batch,kv_heads", [(9001, 300, 8), (901, 3, 1), (60, 2, 2)])
def test_the_smallest_scales_of_values(env, n, batch, kv_heads, power):
    """Even weights of many tokens under scales near 2^-126: what the sum is divided by may
    not go through fp32's subnormal numbers. (The sequences share their pages.)"""
    torch, dsa = env
    dim, page = 64, 128
    rng = np.random.default_rng(n)
    pages = -(-n // page)
    codes = rng.integers(0x38, 0x7f, (2, pages * page, 1, dim)).astype(np.uint8)  # 1 to 448
    codes = np.repeat(codes, kv_heads, 2)
    cache = torch.from_numpy(codes.reshape(2, pages, page, kv_heads, dim)).cuda().view(
        torch.float8_e4m3fn)
    s = torch.ones(2, pages, 1, kv_heads, device="cuda")
    s[1] = 2.0 ** power
    q = torch.zeros(batch, kv_heads, dim, dtype=torch.bfloat16)
    tables = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out, _ = dsa.dsa_quant_attention(q.cuda(), cache[0], cache[1], s[0], s[1], tables, lens)
    k, v = (torch.from_numpy(quant.VALUES[codes[i, :n, 0]]) for i in (0, 1))
    got = out.reshape(batch * kv_heads, dim)
    check(torch, got, torch.zeros(1, dim, dtype=torch.float64), k, v, 2.0 ** power, 0.125)
