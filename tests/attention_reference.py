"""Attention from its definition in 64 bits, and the bound that a kernel's
results are held to (plain torch on the CPU, no code of the library).

The bound of one output value, for a row over n keys of head dimension D with
c = scale * log2 e, weights w_j (normalised) and the operands' rounding
h = eps / 2 (2^-8 for bf16, 2^-11 for fp16), u = 2^-24:

* x_j = c <q, k_j>: the products of bf16 or fp16 operands are exact in fp32;
  the sum of D of them is off by at most 2 D u sum_d |q_d k_jd| (2u for a sum
  that need not round to nearest at each step), scaling and the subtraction of
  the maximum add 3u (|x_j| + |m|). E = the largest such error over the keys.
* A weight 2^(x_j - m) then is off by ln2 * E relative to it, exp2 adds 2^-22,
  its rounding for the product with V adds h. Weights appear above and below
  the fraction line: A = h + 2 (ln2 * E + 2^-22 + 2 n u) + h^2, the last
  term for what these do to each other.
* The n products with V are summed in fp32: covered by the 2 n u of A.
* One more rounding of the result: h |out|.
  tol = A sum_j w_j |v_j| + h |out|
* fp16 weights below 2^-14 have an absolute rounding of 2^-25 each. They are
  relative to a maximum that is at least 1 and so is l: 2^-25 sum_j |v_j|.
  fp16 results below 2^-14: 2^-25.
* lse: E + (2^-22 + 2 n u) / ln2 + 3u |lse|.
E and A are doubled for what second-order terms leave out.
"""

import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, see, scale, dtype):
    """q [m, D], k and v [n, D] fp64, see bool [m, n]: (out, lse, tolerance of
    out, tolerance of lse), each key that a row does not see left out of it."""
    m, n, dim = q.shape[0], k.shape[0], q.shape[1]
    out = torch.zeros((m, v.shape[1]), dtype=torch.float64)
    lse = torch.full((m,), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    h, c = half_step(dtype), scale / math.log(2.0)
    special = not (torch.isfinite(k).all() and torch.isfinite(v).all())
    if n == 0 or m == 0:
        return out, lse, tol, tol_lse
    groups = [(torch.arange(m), torch.arange(n), see)]
    if special:  # row by row over its own keys alone
        groups = [(torch.tensor([i]), see[i].nonzero()[:, 0], None) for i in range(m)]
    for rows, keys, mask in groups:
        if len(keys) == 0:
            continue
        kk, vv = k[keys], v[keys]
        x = c * (q[rows] @ kk.T)
        size = abs(c) * (q[rows].abs() @ kk.abs().T)
        if mask is not None:
            x = torch.where(mask, x, -math.inf)
            size = torch.where(mask, size, 0.0)
        some = torch.ones(len(rows), dtype=torch.bool) if mask is None else mask.any(1)
        top = x.amax(1)
        top = torch.where(some, top, 0.0)
        p = torch.exp2(x - top[:, None])
        l = torch.where(some, p.sum(1), 1.0)
        w = p / l[:, None]
        o = w @ vv
        out[rows] = torch.where(some[:, None], o, 0.0)
        lse[rows] = torch.where(some, top + torch.log2(l), -math.inf)
        e = 2 * ((2 * dim + 6) * U * size.amax(1) + 3 * U)
        a = h + 2 * (math.log(2.0) * e + 2.0 ** -22 + 2 * n * U) + h * h
        t = a[:, None] * (w @ vv.abs()) + h * o.abs()
        if dtype == torch.float16:
            seen = torch.ones_like(p) if mask is None else mask.double()
            t = t + 2.0 ** -25 * (seen @ vv.abs()) + 2.0 ** -25
        tol[rows] = 2 * t
        tol_lse[rows] = 2 * (e + (2.0 ** -22 + 2 * n * U) / math.log(2.0)) + \
            3 * U * lse[rows].abs().nan_to_num(0.0, 0.0, 0.0)
    return out, lse, tol, tol_lse


def check(got, want, tol, what):
    got, want = got.double().cpu(), want.cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN positions differ"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = want.isfinite()
    assert got[fine].isfinite().all(), f"{what}: unexpected infinity"
    off = (got - want).abs()
    bad = fine & (off > tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first "
                             f"at {i}: got {got[i]:.9g} want {want[i]:.9g} tol {tol[i]:.3g}")


def prompt(q, k, v, cu_q, cu_k, causal, scale=None):
    """The packed form: (out, lse, tolerances); rows of no sequence are NaN."""
    dtype = q.dtype
    q, k, v = (t.double().cpu() for t in (q, k, v))
    tq, heads, dim = q.shape
    group = heads // k.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    out = torch.full_like(q, math.nan)
    lse = torch.full((tq, heads), math.nan, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(len(cu_q) - 1):
        a, b, c, d = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
        nq, nk = b - a, d - c
        see = torch.ones((nq, nk), dtype=torch.bool)
        if causal:
            see = torch.arange(nk)[None, :] < torch.arange(nq)[:, None] + 1 + nk - nq
        for h in range(heads):
            r = attend(q[a:b, h], k[c:d, h // group], v[c:d, h // group], see, scale, dtype)
            out[a:b, h], lse[a:b, h], tol[a:b, h], tol_lse[a:b, h] = r
    return out, lse, tol, tol_lse


def paged(q, k_pages, v_pages, tables, lens, prefix_pages, prefix_len, scale=None):
    """One token per sequence on pages; bad pages are not seen."""
    dtype = q.dtype
    q, k_pages, v_pages = (t.double().cpu() for t in (q, k_pages, v_pages))
    tables, lens = tables.cpu(), lens.cpu()
    batch, heads, dim = q.shape
    pages, page, kv_heads, _ = k_pages.shape
    group = heads // kv_heads
    scale = dim ** -0.5 if scale is None else scale
    out, lse = torch.zeros_like(q), torch.zeros((batch, heads), dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(batch):
        ids = tables[b].tolist()
        if prefix_len:
            ids[:prefix_len // page] = prefix_pages.cpu().tolist()[:prefix_len // page]
        n = max(0, min(int(lens[b]), len(ids) * page))
        at = [(ids[t // page], t % page) for t in range(n) if 0 <= ids[t // page] < pages]
        i, j = (torch.tensor([x[y] for x in at], dtype=torch.long) for y in (0, 1))
        for g in range(kv_heads):
            k, v = k_pages[i, j, g], v_pages[i, j, g]
            rows = slice(g * group, (g + 1) * group)
            see = torch.ones((group, len(at)), dtype=torch.bool)
            r = attend(q[b, rows], k, v, see, scale, dtype)
            out[b, rows], lse[b, rows], tol[b, rows], tol_lse[b, rows] = r
    return out, lse, tol, tol_lse
