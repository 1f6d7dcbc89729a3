"""The rotary and 8-bit cache operators without a GPU: refusals of the C ABI (no
call below reaches a CUDA API) and of the binding, the angles' layout, and the
reference's codes."""

import ctypes
import math

import numpy as np
import pytest

import quant_reference as quant

torch = pytest.importorskip("torch")

DSA_OK, DSA_EINVAL, DSA_EUNSUPPORTED = 0, -1, -3
F32, BF16, F16 = 0, 1, 2
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call fails before a launch
ODD = ctypes.c_void_p(0x1008)
ONE = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def dsa():
    from deepseek_sparse_attention_row_gb300 import _build_lib

    _build_lib.build()
    import deepseek_sparse_attention_row_gb300 as dsa

    return dsa


def call(fn, a, kw):
    assert set(kw) <= set(a), set(kw) - set(a)
    return fn(*{**a, **kw}.values())


def rotary(lib, **kw):
    return call(lib.dsa_rotary, dict(
        q=FAKE, q_out=FAKE, heads=4, q_st=256, q_sh=64, qo_st=256, qo_sh=64, k=FAKE, k_out=FAKE,
        kv_heads=2, k_st=128, k_sh=64, ko_st=128, ko_sh=64, dtype=BF16, tokens=10, head_dim=64,
        positions=FAKE, turns=FAKE, pairs=32, interleaved=0, factor=1.0, transpose=0,
        stream=None), kw)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DSA_EINVAL), (dict(dtype=-1), DSA_EINVAL), (dict(heads=-1), DSA_EINVAL),
    (dict(kv_heads=-1), DSA_EINVAL), (dict(tokens=-1), DSA_EINVAL),
    (dict(head_dim=-1), DSA_EINVAL), (dict(pairs=-1), DSA_EINVAL), (dict(pairs=33), DSA_EINVAL),
    (dict(factor=math.nan), DSA_EINVAL), (dict(factor=-math.inf), DSA_EINVAL),
    (dict(q_st=-1), DSA_EINVAL), (dict(ko_sh=-64), DSA_EINVAL),
    (dict(q=None), DSA_EINVAL), (dict(q_out=None), DSA_EINVAL), (dict(k=None), DSA_EINVAL),
    (dict(k_out=None), DSA_EINVAL), (dict(positions=None), DSA_EINVAL),
    (dict(turns=None), DSA_EINVAL), (dict(q=ONE), DSA_EINVAL), (dict(k_out=ONE), DSA_EINVAL),
    (dict(q=ctypes.c_void_p(0x1002), dtype=F32), DSA_EINVAL),
    (dict(tokens=2 ** 31), DSA_EUNSUPPORTED), (dict(head_dim=4097), DSA_EUNSUPPORTED),
    (dict(heads=2 ** 30, kv_heads=2 ** 30), DSA_EUNSUPPORTED),
    (dict(tokens=0, q=None, positions=None), DSA_OK), (dict(head_dim=0, pairs=0), DSA_OK),
    (dict(heads=0, kv_heads=0, q=None, q_st=-1), DSA_OK),
], ids=str)
def test_rotary_refusals(dsa, kw, want):
    assert rotary(dsa.library(), **kw) == want


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] + \
        [(n, ctypes.c_int64) for n in ("num_pages", "kc_sn", "kc_st", "kc_sh", "vc_sn", "vc_st",
                                       "vc_sh", "ks_sn", "vs_sn")] + \
        [("tables", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
         ("ld_tables", ctypes.c_int64)] + \
        [(n, ctypes.c_int32) for n in ("page_size", "block", "kv_heads", "head_dim")]


PAGES = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, num_pages=20, kc_sn=2048,
             kc_st=128, kc_sh=64, vc_sn=2048, vc_st=128, vc_sh=64, ks_sn=4, vs_sn=4, tables=FAKE,
             max_pages=6, ld_tables=6, page_size=16, block=8, kv_heads=2, head_dim=64)


def on_pages(fn, a, kw):
    """fn with the keywords of PAGES in its first argument, or as that argument."""
    pages = {**PAGES, **{n: v for n, v in kw.items() if n in PAGES}}
    pages = ctypes.byref(Pages(*pages.values())) if kw.get("pages", 1) else None
    return call(fn, dict(pages=pages, **a), {n: v for n, v in kw.items()
                                             if n not in PAGES and n != "pages"})


def write(lib, **kw):
    return on_pages(lib.dsa_quant_cache_write, dict(
        k=FAKE, v=FAKE, dtype=BF16, total=10, k_st=128, k_sh=64, v_st=128, v_sh=64, cu=FAKE,
        seqs=3, lens=FAKE, stream=None), kw)


def read(lib, **kw):
    return on_pages(lib.dsa_quant_cache_read, dict(
        cu=FAKE, seqs=3, total=10, dtype=BF16, k=FAKE, k_st=128, k_sh=64, v=FAKE, v_st=128,
        v_sh=64, stream=None), kw)


def attend(lib, **kw):
    return on_pages(lib.dsa_quant_attention, dict(
        q=FAKE, dtype=BF16, batch=3, heads=8, q_sb=512, q_sh=64, lens=FAKE, scale=0.125, out=FAKE,
        o_sb=512, o_sh=64, lse=None, l_sb=8, l_sh=1, workspace=FAKE, workspace_bytes=1 << 40,
        stream=None), kw)


def test_the_binding_packs_the_struct(dsa):
    assert dsa._QUANT_PAGES.size == ctypes.sizeof(Pages) == 144


COMMON = [
    (dict(pages=0), DSA_EINVAL),
    (dict(num_pages=-1), DSA_EINVAL), (dict(page_size=0), DSA_EINVAL), (dict(block=0), DSA_EINVAL),
    (dict(block=32), DSA_EINVAL), (dict(head_dim=0), DSA_EINVAL), (dict(max_pages=-1), DSA_EINVAL),
    (dict(ld_tables=5), DSA_EINVAL), (dict(ks_sn=-1), DSA_EINVAL),
    (dict(page_size=8), DSA_EUNSUPPORTED), (dict(page_size=48), DSA_EUNSUPPORTED),
    (dict(page_size=48, block=3), DSA_EUNSUPPORTED),
    (dict(num_pages=2 ** 31), DSA_EUNSUPPORTED),
    (dict(max_pages=2 ** 30, ld_tables=2 ** 30), DSA_EUNSUPPORTED),
    (dict(head_dim=72), DSA_EUNSUPPORTED), (dict(head_dim=144), DSA_EUNSUPPORTED),
    (dict(k_codes=None), DSA_EINVAL), (dict(v_codes=None), DSA_EINVAL),
    (dict(k_scales=None), DSA_EINVAL), (dict(v_scales=None), DSA_EINVAL),
    (dict(tables=None), DSA_EINVAL), (dict(k_codes=ODD), DSA_EUNSUPPORTED),
    (dict(v_codes=ODD), DSA_EUNSUPPORTED), (dict(k_scales=ONE), DSA_EUNSUPPORTED),
    (dict(kc_sn=2056), DSA_EUNSUPPORTED), (dict(kc_st=-128), DSA_EUNSUPPORTED),
    (dict(vc_sh=8), DSA_EUNSUPPORTED), (dict(dtype=9), DSA_EINVAL),
    (dict(dtype=F32), DSA_EUNSUPPORTED),
]
ROWS = [
    (dict(kv_heads=-1), DSA_EINVAL), (dict(kv_heads=2 ** 20 + 1), DSA_EUNSUPPORTED),
    (dict(total=-1), DSA_EINVAL), (dict(seqs=-1), DSA_EINVAL),
    (dict(total=2 ** 31), DSA_EUNSUPPORTED), (dict(seqs=2 ** 28), DSA_EUNSUPPORTED),
    (dict(k=None), DSA_EINVAL), (dict(v=None), DSA_EINVAL), (dict(cu=None), DSA_EINVAL),
    (dict(k=ODD), DSA_EUNSUPPORTED), (dict(v=ODD), DSA_EUNSUPPORTED),
    (dict(k_st=132), DSA_EUNSUPPORTED), (dict(v_sh=-64), DSA_EUNSUPPORTED),
    (dict(total=0, k=None, cu=None), DSA_OK), (dict(seqs=0, v=None), DSA_OK),
    (dict(kv_heads=0, k=None), DSA_OK),
]


@pytest.mark.parametrize("kw,want", COMMON + ROWS + [
    (dict(lens=None), DSA_EINVAL), (dict(page_size=512, block=512), DSA_EUNSUPPORTED),
    (dict(num_pages=0, k_codes=None, k_scales=None), DSA_OK),
    (dict(max_pages=0, ld_tables=0, tables=None), DSA_OK),
], ids=str)
def test_write_refusals(dsa, kw, want):
    assert write(dsa.library(), **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + ROWS, ids=str)
def test_read_refusals(dsa, kw, want):
    assert read(dsa.library(), **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(batch=-1), DSA_EINVAL), (dict(heads=-1), DSA_EINVAL), (dict(kv_heads=0), DSA_EINVAL),
    (dict(heads=7), DSA_EINVAL), (dict(heads=258), DSA_EUNSUPPORTED),
    (dict(batch=2 ** 31), DSA_EUNSUPPORTED), (dict(batch=2 ** 30), DSA_EUNSUPPORTED),
    (dict(scale=0.0), DSA_EINVAL), (dict(scale=-1.0), DSA_EINVAL),
    (dict(scale=math.nan), DSA_EINVAL), (dict(scale=2.4e38), DSA_EINVAL),
    (dict(q=None), DSA_EINVAL), (dict(out=None), DSA_EINVAL), (dict(lens=None), DSA_EINVAL),
    (dict(q=ODD), DSA_EUNSUPPORTED), (dict(out=ODD), DSA_EUNSUPPORTED),
    (dict(q_sh=68), DSA_EUNSUPPORTED), (dict(o_sb=-8), DSA_EUNSUPPORTED),
    (dict(batch=0, q=None, lens=None), DSA_OK), (dict(heads=0, out=None), DSA_OK),
], ids=str)
def test_attention_refusals(dsa, kw, want):
    assert attend(dsa.library(), **kw) == want


def scaled(**kw):
    a = dict(cache=FAKE, planes=2, plane_stride=2560, num_pages=10, page_stride=256, page_size=4,
             token_bytes=64, scales=FAKE, scale_plane=160, scale_page=16, scale_bytes=16,
             refs=FAKE, tables=FAKE, seqs=5, max_pages=6, ld_tables=6)
    a.update({n: v for n, v in kw.items() if n in a})
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(scales=None), DSA_EINVAL), (dict(scale_bytes=-4), DSA_EINVAL),
    (dict(scale_plane=-4), DSA_EINVAL), (dict(scale_page=-4), DSA_EINVAL),
    (dict(scales=ONE), DSA_EUNSUPPORTED), (dict(scale_bytes=6), DSA_EUNSUPPORTED),
    (dict(scale_page=18), DSA_EUNSUPPORTED), (dict(scale_plane=161), DSA_EUNSUPPORTED),
    (dict(scale_bytes=2 ** 31), DSA_EUNSUPPORTED), (dict(cache=ODD), DSA_EUNSUPPORTED),
    (dict(refs=None), DSA_EINVAL), (dict(tables=None), DSA_EINVAL),
    (dict(ld_tables=5), DSA_EINVAL), (dict(workspace=None), DSA_EINVAL),
    (dict(workspace_bytes=8), DSA_EINVAL),
], ids=str)
def test_scaled_cache_refusals(dsa, kw, want):
    lib, ws = dsa.library(), dict(workspace=FAKE, workspace_bytes=1 << 20, stream=None)
    ws.update({n: v for n, v in kw.items() if n in ws})
    assert set(kw) <= set(scaled()) | set(ws)
    assert lib.dsa_cache_fork_scaled(*scaled(**kw).values(), FAKE, FAKE, FAKE, 3, FAKE,
                                     *ws.values()) == want
    assert lib.dsa_cache_compact_scaled(*scaled(**kw).values(), FAKE, FAKE, *ws.values()) == want


def test_scales_in_the_binding(dsa):
    x = torch.zeros(2, 5, 3)
    with pytest.raises(ValueError, match="expected cuda:0"):
        dsa._page_scales(x, 2, 5, 0)


def test_workspace_sizes(dsa):
    size = dsa.quant_attention_workspace_bytes
    assert size(0, 8, 2, 64, 100, 16) == 0 and size(3, 8, 3, 64, 100, 16) == 0
    assert size(-1, 8, 2, 64, 100, 16) == 0 and size(3, 8, 2, 60, 100, 16) == 0
    assert size(3, 8, 2, 64, -1, 16) == 0 and size(3, 8, 2, 64, 100, 24) == 0


def test_binding_refusals(dsa):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    p = torch.zeros(3, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(3, 2, 2)
    t = torch.zeros(4, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_rotary(x, None, i, i)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        dsa.dsa_rotary(x.double(), None, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_quant_cache_write(x, x, i, p, p, s, s, t, i)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dsa.dsa_quant_cache_write(x.float(), x, i, p, p, s, s, t, i)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_quant_cache_read(p, p, s, s, t, i, total=3)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_quant_attention(x, p, p, s, s, t, i)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dsa.dsa_quant_attention(x.float(), p, p, s, s, t, i)


def test_turns(dsa):
    two = 2 * math.pi
    got = dsa.rotary_turns([0.0, two / 4, two / 2, two, -two / 4, 3 * two / 4, 1.0], device="cpu")
    assert got.dtype == torch.int64
    assert got.tolist()[:6] == [0, 2 ** 62, -2 ** 63, 0, -2 ** 62, -2 ** 62]
    assert abs(got[6].item() / 2.0 ** 64 * two - 1) < 2.0 ** -52
    f = dsa.rotary_frequencies(64)
    assert torch.equal(dsa.rotary_turns(f, "cpu"), dsa.rotary_turns(f.tolist(), "cpu"))
    with pytest.raises(ValueError, match="finite"):
        dsa.rotary_turns([math.nan], "cpu")
    with pytest.raises(ValueError, match="vector"):
        dsa.rotary_turns(f[None], "cpu")


def test_frequencies(dsa):
    f = dsa.rotary_frequencies(64, 500000.0)
    want = [500000.0 ** (-2 * i / 64) for i in range(32)]
    assert f.dtype == torch.float64 and np.allclose(f, want, rtol=1e-14, atol=0)
    assert torch.equal(dsa.rotary_frequencies(64, 500000.0, stretch=4.0), f / 4)
    b = dsa.rotary_frequencies(64, 500000.0, stretch=4.0, method="base")
    assert b[0] == 1 and abs(b[-1] / f[-1] * 4 - 1) < 1e-13
    p = dsa.rotary_frequencies(64, stretch=8.0, method="parts", trained=4096, slow=1.0, fast=32.0)
    f = dsa.rotary_frequencies(64)
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(p[turns >= 32], f[turns >= 32])
    assert torch.allclose(p[turns <= 1], f[turns <= 1] / 8, rtol=1e-15, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (p[mid] < f[mid]).all() and (p[mid] > f[mid] / 8).all()
    for kw in (dict(rotary_dim=5), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0),
               dict(rotary_dim=8, stretch=-1.0), dict(rotary_dim=8, method="other"),
               dict(rotary_dim=2, method="base", stretch=2.0),
               dict(rotary_dim=8, method="parts", slow=3.0, fast=3.0)):
        with pytest.raises(ValueError):
            dsa.rotary_frequencies(**kw)


def test_reference_codes():
    """The table's rounding against torch's cast, at codes, midpoints and beside them."""
    v = quant.VALUES[:127]
    mids = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mids, np.nextafter(mids, 0), np.nextafter(mids, 500.0), [math.nan]])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    quant.same_codes(quant.encode(x), want, "codes")
    assert quant.encode([1e9, -math.inf]).tolist() == [126, 254]
    for x, p in ((0.0, 2.0 ** -126), (1.0, 1.0), (1.5, 2.0), (2.0 ** -130, 2.0 ** -126),
                 (3e38, 2.0 ** 126), (math.nan, 2.0 ** -126), (-1.0, 2.0 ** -126)):
        assert quant.least_power(x) == p
