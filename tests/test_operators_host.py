"""Refusals of the attention and cache operators without a GPU: the binding's
own checks, and the C ABI's (no call below reaches a CUDA API)."""

import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

DSA_OK, DSA_EINVAL, DSA_EUNSUPPORTED = 0, -1, -3
F32, BF16, F16 = 0, 1, 2
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call fails before a launch
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def dsa():
    from deepseek_sparse_attention_row_gb300 import _build_lib

    _build_lib.build()
    import deepseek_sparse_attention_row_gb300 as dsa

    return dsa


def prompt(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=BF16, total_q=10, total_k=10, heads=4, kv_heads=2,
             head_dim=64, q_st=256, q_sh=64, k_st=128, k_sh=64, v_st=128, v_sh=64, cu_q=FAKE,
             cu_k=FAKE, seqs=1, causal=1, scale=0.125, out=FAKE, o_st=256, o_sh=64, lse=None,
             l_st=4, l_sh=1, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dsa_prompt_attention(*a.values())


COMMON = [
    (dict(dtype=7), DSA_EINVAL),
    (dict(dtype=-1), DSA_EINVAL),
    (dict(dtype=F32), DSA_EUNSUPPORTED),
    (dict(heads=-1), DSA_EINVAL),
    (dict(kv_heads=0), DSA_EINVAL),
    (dict(heads=5), DSA_EINVAL),
    (dict(heads=258, kv_heads=2), DSA_EUNSUPPORTED),
    (dict(head_dim=0), DSA_EINVAL),
    (dict(head_dim=60), DSA_EUNSUPPORTED),
    (dict(head_dim=136), DSA_EUNSUPPORTED),
    (dict(scale=0.0), DSA_EINVAL),
    (dict(scale=-1.0), DSA_EINVAL),
    (dict(scale=math.nan), DSA_EINVAL),
    (dict(scale=math.inf), DSA_EINVAL),
    (dict(q=None), DSA_EINVAL),
    (dict(out=None), DSA_EINVAL),
    (dict(q=ODD), DSA_EUNSUPPORTED),
    (dict(out=ODD), DSA_EUNSUPPORTED),
    (dict(q_sh=68), DSA_EUNSUPPORTED),
    (dict(k_st=132), DSA_EUNSUPPORTED),
    (dict(v_sh=60), DSA_EUNSUPPORTED),
    (dict(o_sh=65), DSA_EUNSUPPORTED),
    (dict(k_sh=-64), DSA_EUNSUPPORTED),
    (dict(heads=0), DSA_OK),
]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(total_q=-1), DSA_EINVAL),
    (dict(total_k=-1), DSA_EINVAL),
    (dict(seqs=-1), DSA_EINVAL),
    (dict(total_q=2 ** 31), DSA_EUNSUPPORTED),
    (dict(total_k=2 ** 31), DSA_EUNSUPPORTED),
    (dict(cu_q=None), DSA_EINVAL),
    (dict(cu_k=None), DSA_EINVAL),
    (dict(k=None), DSA_EINVAL),
    (dict(v=None), DSA_EINVAL),
    (dict(k=ODD), DSA_EUNSUPPORTED),
    (dict(v=ODD), DSA_EUNSUPPORTED),
    (dict(total_q=0, q=None, out=None), DSA_OK),
    (dict(seqs=0, q=None, out=None, cu_q=None), DSA_OK),
    (dict(total_k=100000, workspace=None), DSA_EINVAL),
    (dict(total_k=100000, workspace=ODD), DSA_EINVAL),
    (dict(total_k=100000, workspace_bytes=4096), DSA_EINVAL),
], ids=str)
def test_prompt_refusals(dsa, kw, want):
    assert prompt(dsa.library(), **kw) == want


def shared(lib, **kw):
    a = dict(q=FAKE, k_pages=FAKE, v_pages=FAKE, dtype=BF16, batch=3, heads=4, kv_heads=2,
             head_dim=64, num_pages=20, page_size=16, q_sb=256, q_sh=64, k_sn=2048, k_st=128,
             k_sh=64, v_sn=2048, v_st=128, v_sh=64, prefix_pages=FAKE, prefix_len=32, tables=FAKE,
             max_pages=8, ld_tables=8, lens=FAKE, scale=0.125, out=FAKE, o_sb=256, o_sh=64,
             lse=None, l_sb=4, l_sh=1, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dsa_shared_prefix_attention(*a.values())


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(batch=-1), DSA_EINVAL),
    (dict(batch=2 ** 31), DSA_EUNSUPPORTED),
    (dict(num_pages=-1), DSA_EINVAL),
    (dict(num_pages=2 ** 31), DSA_EUNSUPPORTED),
    (dict(page_size=0), DSA_EINVAL),
    (dict(page_size=8), DSA_EUNSUPPORTED),
    (dict(page_size=48, prefix_len=48), DSA_EUNSUPPORTED),
    (dict(max_pages=-1), DSA_EINVAL),
    (dict(ld_tables=7), DSA_EINVAL),
    (dict(max_pages=2 ** 30, ld_tables=2 ** 30), DSA_EUNSUPPORTED),
    (dict(prefix_len=-16), DSA_EINVAL),
    (dict(prefix_len=40), DSA_EINVAL),
    (dict(prefix_len=144), DSA_EINVAL),
    (dict(prefix_pages=None), DSA_EINVAL),
    (dict(tables=None), DSA_EINVAL),
    (dict(lens=None), DSA_EINVAL),
    (dict(k_pages=None), DSA_EINVAL),
    (dict(v_pages=None), DSA_EINVAL),
    (dict(k_pages=ODD), DSA_EUNSUPPORTED),
    (dict(v_pages=ODD), DSA_EUNSUPPORTED),
    (dict(k_sn=2052), DSA_EUNSUPPORTED),
    (dict(v_sn=2049), DSA_EUNSUPPORTED),
    (dict(batch=0, q=None, out=None, lens=None), DSA_OK),
], ids=str)
def test_shared_refusals(dsa, kw, want):
    assert shared(dsa.library(), **kw) == want


def state(**kw):
    a = dict(cache=FAKE, planes=2, plane_stride=20 * 256, num_pages=20, page_stride=256,
             page_size=4, token_bytes=64, refs=FAKE, tables=FAKE, seqs=5, max_pages=6,
             ld_tables=6)
    return a


def fork(lib, **kw):
    a = state()
    a.update(lens=FAKE, parents=FAKE, children=FAKE, pairs=3, status=FAKE, workspace=FAKE,
             workspace_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dsa_cache_fork(*a.values())


def compact(lib, **kw):
    a = state()
    a.update(remap=FAKE, live=FAKE, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.dsa_cache_compact(*a.values())


STATE = [
    (dict(cache=None), DSA_EINVAL),
    (dict(cache=ODD), DSA_EUNSUPPORTED),
    (dict(planes=-1), DSA_EINVAL),
    (dict(plane_stride=1001), DSA_EUNSUPPORTED),
    (dict(page_stride=264), DSA_EUNSUPPORTED),
    (dict(token_bytes=24), DSA_EUNSUPPORTED),
    (dict(token_bytes=-16), DSA_EINVAL),
    (dict(page_size=0), DSA_EINVAL),
    (dict(num_pages=-1), DSA_EINVAL),
    (dict(num_pages=2 ** 31), DSA_EUNSUPPORTED),
    (dict(seqs=-1), DSA_EINVAL),
    (dict(seqs=2 ** 31), DSA_EUNSUPPORTED),
    (dict(max_pages=-1), DSA_EINVAL),
    (dict(ld_tables=5), DSA_EINVAL),
    (dict(max_pages=2 ** 30, ld_tables=2 ** 30), DSA_EUNSUPPORTED),
    (dict(refs=None), DSA_EINVAL),
    (dict(tables=None), DSA_EINVAL),
    (dict(workspace=None), DSA_EINVAL),
    (dict(workspace=ODD), DSA_EINVAL),
    (dict(workspace_bytes=8), DSA_EINVAL),
]


@pytest.mark.parametrize("kw,want", STATE + [
    (dict(pairs=-1), DSA_EINVAL),
    (dict(pairs=2 ** 16), DSA_EUNSUPPORTED),
    (dict(parents=None), DSA_EINVAL),
    (dict(children=None), DSA_EINVAL),
    (dict(status=None), DSA_EINVAL),
    (dict(lens=None), DSA_EINVAL),
    (dict(max_pages=0), DSA_EINVAL),
    (dict(pairs=0, parents=None, status=None, workspace=None), DSA_OK),
], ids=str)
def test_fork_refusals(dsa, kw, want):
    assert fork(dsa.library(), **kw) == want


@pytest.mark.parametrize("kw,want", STATE + [
    (dict(remap=None), DSA_EINVAL),
    (dict(live=None), DSA_EINVAL),
], ids=str)
def test_compact_refusals(dsa, kw, want):
    assert compact(dsa.library(), **kw) == want


def test_free_refusals(dsa):
    lib = dsa.library()

    def call(refs=FAKE, num_pages=20, tables=FAKE, seqs=5, max_pages=6, ld=6, lens=FAKE,
             which=FAKE, count=2):
        return lib.dsa_cache_free(refs, num_pages, tables, seqs, max_pages, ld, lens, which, count,
                                  None)

    for kw in (dict(refs=None), dict(tables=None), dict(lens=None), dict(which=None),
               dict(num_pages=-1), dict(seqs=-1), dict(max_pages=-1), dict(ld=5), dict(count=-1)):
        assert call(**kw) == DSA_EINVAL, kw
    for kw in (dict(num_pages=2 ** 31), dict(seqs=2 ** 31), dict(count=2 ** 31)):
        assert call(**kw) == DSA_EUNSUPPORTED, kw
    assert call(count=0, which=None) == DSA_OK


def test_workspace_sizes(dsa):
    assert dsa.cache_workspace_bytes(-1, 5) == 0 and dsa.cache_workspace_bytes(1, -1) == 0
    assert dsa.cache_workspace_bytes(0, 1000) >= 8000
    assert dsa.shared_prefix_workspace_bytes(0, 8, 2, 64, 0, 5, 16) == 0
    assert dsa.shared_prefix_workspace_bytes(-1, 8, 2, 64, 0, 5, 16) == 0
    assert dsa.shared_prefix_workspace_bytes(4, 8, 3, 64, 0, 5, 16) == 0
    assert dsa.prompt_workspace_bytes(0, 100000, 8, 2, 64, 1) == 0
    assert dsa.prompt_workspace_bytes(100, 100, 8, 2, 64, 1) == 0
    assert dsa.prompt_workspace_bytes(100, -1, 8, 2, 64, 1) == 0
    assert dsa.prompt_workspace_bytes(100, 100000, 8, 2, 64, 1) > 256 * 64 * 4


def test_binding_takes_cuda_tensors_only(dsa):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dsa.dsa_prompt_attention(x, x, x, i, i)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dsa.dsa_prompt_attention(x.float(), x, x, i, i)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dsa.dsa_shared_prefix_attention(x.double(), x, x, i, i)
    t = torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="tables must be a CUDA tensor"):
        dsa.dsa_cache_free(i, t, torch.zeros(3, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="cache must be a CUDA tensor"):
        dsa._cache_planes(torch.zeros(2, 3, 4, 8), 3, 0)


def test_binding_strides(dsa):
    x = torch.zeros(5, 4, 64)

    def rows(t):
        return dsa._row_strides(t.shape, t.stride(), "q")

    assert rows(x) == (256, 64)
    assert rows(x[:, ::2]) == (256, 128)
    assert rows(torch.as_strided(x, (1, 4, 64), (3, 64, 1))) == (64, 64)
    with pytest.raises(ValueError, match="unit stride"):
        rows(x.transpose(1, 2))


@pytest.mark.parametrize("scale,want", [(2.4e38, DSA_EINVAL), (3.4e38, DSA_EINVAL),
                                        (2.3e38, DSA_OK), (1e-38, DSA_OK)])
def test_scales_whose_product_with_log2_e_overflows(dsa, scale, want):
    """Accepted ones fall through to the next check (no heads: nothing to do)."""
    assert prompt(dsa.library(), scale=scale, heads=0) == want
    assert shared(dsa.library(), scale=scale, heads=0) == want


def test_the_merge_takes_no_fp16(dsa):
    """As dsa_attention.h says of the outputs that go to it."""
    lib = dsa.library()
    assert lib.dsa_merge_attn_out(FAKE, F16, 2, 3, 4, 64, 768, 256, 64, 1, FAKE, 12, 4, 1, FAKE,
                                  192, 64, 1, None, 4, 1, None) == DSA_EINVAL
    assert lib.dsa_correct_attn_out(FAKE, F16, 3, 4, 64, 256, 64, 1, FAKE, 2, 12, 4, 1, 0, FAKE,
                                    192, 64, 1, None, 4, 1, None) == DSA_EINVAL


@pytest.mark.parametrize("batch,want", [(2 ** 31 - 1, DSA_EUNSUPPORTED), (2 ** 26 - 1, DSA_EINVAL)])
def test_batches_whose_join_has_too_many_ctas(dsa, batch, want):
    """Refused before a launch; the one below the limit gets as far as its
    missing workspace. (No pages: the rows alone count.)"""
    assert shared(dsa.library(), batch=batch, heads=128, kv_heads=1, prefix_len=0,
                  prefix_pages=None, max_pages=0, num_pages=0, workspace=None) == want
