"""The 8-bit cache from its definition in 64 bits (numpy and plain torch on the
CPU, no code of the library).

Codes: e4m3, by a table of the 256 values. Writing is compared byte by byte:
scales are powers of two, so that x / scale is exact in fp32 and the code is the
nearest one, the even one of two.

The bound of an attention output, for a row over n tokens, h = eps / 2 of the
output's type, u = 2^-24, x_j = c sk_j <q, code_j>, w_j the normalised weights:

* q (16 bits) times a power of two, times a code (4 bits): exact in fp32. The sum
  of D products: 2 D u sum_d |q_d k_jd| (2u for a sum that need not round to
  nearest at each step). Multiplying by c and sk, and subtracting the maximum:
  12 u of the same. E = the largest such error over the tokens, and 3u.
* The weight with its value's scale is 2^(x_j + log2 sv_j - M): log2 (2 u of
  itself), the sum and the difference add L = 6 u (|x_j| + |log2 sv_j| + |M|).
* exp2 adds 2^-22, the rounding to fp16 H = 2^-11 (or 2^-32 of the largest
  weight). The products with codes are exact; sums over n: 2 n u.
* Parts are joined by their log-sum-exps: each at most 2^-22 + E + 6 u log2 n off.
  tol = A sum_j w_j |v_j| + 2^-32 max_j(w_j sv_j) sum_j |code_j| + h |out|
  A = H + 2 (ln2 (E + L) + 3 2^-22 + 4 n u) + H^2
* fp16 results below 2^-14: 2^-25 more.
* lse: E + (3 2^-22 + 4 n u) / ln2 + 6 u (|lse| + log2 n).
E and A are doubled for what second-order terms leave out.
"""

import math

import numpy as np
import torch

U = 2.0 ** -24
LARGEST = 448.0


def _values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        v[c] = math.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


VALUES = _values()


def encode(x):
    """The codes next to x (fp64 numpy), to even; what passes 448 becomes 448; NaN 127."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=LARGEST, neginf=LARGEST)), LARGEST)
    hi = np.searchsorted(VALUES[:127], a)              # first code not below a
    hi = np.minimum(hi, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUES[hi] - a, a - VALUES[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (VALUES[hi] == a), hi, lo)
    c = np.where(np.signbit(x), c + 128, c)
    return np.where(np.isnan(x), 127, c).astype(np.uint8)


def least_power(x):
    """The least power of two from 2^-126 to 2^126 that is not below x."""
    if not x > 0:
        return 2.0 ** -126
    m, e = math.frexp(min(x, 2.0 ** 126))
    return 2.0 ** min(max(e - 1 if m == 0.5 else e, -126), 126)


def write(k, v, cu, codes, scales, tables, lens):
    """In place: codes uint8 [2, N, page, H, D], scales float64 [2, N, page / block, H]; k, v
    float64 [T, H, D]."""
    _, pages, page, heads, _ = codes.shape
    block = page // scales.shape[2]
    total = k.shape[0]
    for s in range(len(lens)):
        r0, r1 = (min(max(int(c), 0), total) for c in cu[s:s + 2])
        held = max(int(lens[s]), 0)
        end = held + r1 - r0
        for start in range(held // block * block, end, block):
            if start >= tables.shape[1] * page or r1 <= r0:
                break
            n = tables[s, start // page]
            if not 0 <= n < pages:
                continue
            lo, hi = max(start, held), min(end, start + block)
            at, b = start % page, start % page // block
            for kv, x in enumerate((k, v)):
                for h in range(heads):
                    rows = x[r0 + lo - held:r0 + hi - held, h]
                    rows = np.where(np.isfinite(rows), rows, math.nan)
                    new = least_power(np.nanmax(np.abs(rows), initial=0.0) / LARGEST)
                    old = scales[kv, n, b, h]
                    if lo > start:
                        new = max(new, least_power(old))
                        if new != old:
                            # the product is rounded to fp32 before the power divides it
                            part = codes[kv, n, at:at + lo - start, h]
                            with np.errstate(all="ignore"):
                                z = (VALUES[part].astype(np.float32) * np.float32(old))
                            part[...] = encode(z.astype(np.float64) / new)
                    scales[kv, n, b, h] = new
                    codes[kv, n, at + lo - start:at + hi - start, h] = encode(rows / new)


def same_codes(got, want, what):
    got, want = np.asarray(got), np.asarray(want)
    nan = (want & 127) == 127
    assert np.array_equal((got & 127) == 127, nan), f"{what}: NaN codes differ"
    bad = (got != want) & ~nan
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4],
                           want[bad][:4])


def read(codes, scales, tables, s, n):
    """Values of the first n tokens of sequence s: fp64 [2, n, H, D]; 0 for no page."""
    _, pages, page, heads, dim = codes.shape
    block = page // scales.shape[2]
    out = np.zeros((2, n, heads, dim))
    for t in range(n):
        p = tables[s, t // page] if t // page < tables.shape[1] else -1
        if 0 <= p < pages:
            out[:, t] = VALUES[codes[:, p, t % page]] * \
                scales[:, p, t % page // block][..., None].astype(np.float64)
    return out


def attend(q, codes, scales, tables, lens, scale=None):
    """(out, lse, tolerances) in fp64; q torch [B, H, D], codes uint8 and scales
    float32 numpy, tables and lens numpy."""
    dtype, q = q.dtype, q.double().cpu()
    batch, heads, dim = q.shape
    _, pages, page, kv_heads, _ = codes.shape
    block, group = page // scales.shape[2], heads // kv_heads
    c = (dim ** -0.5 if scale is None else scale) / math.log(2.0)
    out, lse = torch.zeros_like(q), torch.full((batch, heads), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    h, H = torch.finfo(dtype).eps / 2, 2.0 ** -11
    values = torch.from_numpy(VALUES)
    for b in range(batch):
        t = np.arange(max(0, min(int(lens[b]), tables.shape[1] * page)))
        p = tables[b, t // page]
        t, p = t[(p >= 0) & (p < pages)], p[(p >= 0) & (p < pages)]
        n = len(t)
        if n == 0:
            continue
        for g in range(kv_heads):
            kc, vc = (values[torch.from_numpy(codes[i, p, t % page, g].astype(np.int64))]
                      for i in (0, 1))
            sk, sv = (torch.from_numpy(scales[i, p, t % page // block, g].astype(np.float64))
                      for i in (0, 1))
            rows = slice(g * group, (g + 1) * group)
            x = c * (q[b, rows] @ (kc * sk[:, None]).T)
            size = c * (q[b, rows].abs() @ (kc * sk[:, None]).abs().T)
            top = x.amax(1, keepdim=True)
            base = torch.where(top == -math.inf, 0.0, top)
            w = torch.exp2(x - base)
            l = w.sum(1, keepdim=True)
            none = l == 0
            w = w / torch.where(none, 1.0, l)
            v = vc * sv[:, None]
            o = w @ v
            out[b, rows] = torch.where(none, 0.0, o)
            lse[b, rows] = torch.where(none, -math.inf, base + torch.log2(l))[:, 0]
            big = size.nan_to_num(0.0, 0.0, 0.0).amax(1, keepdim=True)
            lg = torch.log2(sv).nan_to_num(0.0, 0.0, 0.0).abs().max()
            e = 2 * ((2 * dim + 12) * U * big + 3 * U)
            d = 6 * U * (2 * big + 2 * lg)
            a = H + 2 * (math.log(2.0) * (e + d) + 3 * 2.0 ** -22 + 4 * n * U) + H * H
            r = a * (w.nan_to_num() @ v.abs().nan_to_num()) + h * o.abs().nan_to_num(0, 0, 0)
            r += 2.0 ** -32 * (w * sv).nan_to_num().amax(1, keepdim=True) * \
                vc.abs().nan_to_num().sum(0)
            if dtype == torch.float16:
                r = r + 2.0 ** -25
            tol[b, rows] = 2 * r
            near = lse[b, rows].abs().nan_to_num(0.0, 0.0, 0.0)
            tol_lse[b, rows] = 2 * (e[:, 0] + (3 * 2.0 ** -22 + 4 * n * U) / math.log(2.0)) + \
                6 * U * (near + math.log2(n + 1))
    return out, lse, tol, tol_lse
