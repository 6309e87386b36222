"""The calls around a drafted block on a machine without a GPU: refusals before any launch, sizes."""
import ctypes

import pytest

from jacobi_speculative_decode_gb300 import build as B
from jacobi_speculative_decode_gb300 import xp


@pytest.fixture(scope="module")
def lib():
    B.build()
    return xp.lib()


def desc(**kw):
    d = dict(pages=100, page_size=16, layers=2, kv_heads=8, head_dim=128, max_seqs=32, dtype=xp.XP_BF16,
             stride_layer=100 * 16 * 8 * 128, stride_page=16 * 8 * 128, stride_token=8 * 128, stride_head=128,
             k=4096, v=4096)
    d.update(kw)
    return xp.xp_cache_desc(**d)


def test_no_handle(lib):
    no = xp.XP_ENOTPREPARED
    assert lib.xp_verify_drafts(None, 1, 0, 0, None, 0, 1, None, 1, 4, 9, 0, None, 1, 1, 9, 1, 1, None, 1, 1,
                                None) == no
    assert lib.xp_cache_append(None, 0, 1, 1, 0, 0, 0, 8, 128, 0, 1, 1, 1, 1, 1, None) == no
    assert lib.xp_cache_copy(None, 1, 1, 1, None) == no
    assert lib.xp_cache_resize(None, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, None) == no
    assert lib.xp_cache_fork(None, 1, 1, 1, 1, 1, None, 1, 1, 1, 1, 1, 1, 1, 1, None) == no
    assert lib.xp_cache_compact(None, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, None, None, None) == no
    assert lib.xp_cache_get_error(None, None) == no
    a = xp.xp_attn(0, 1, 1, 8, 128, 0, 0, 16, 1.0, 0, 0, 0, 0, 0, 0)
    assert lib.xp_prefix_attention(None, ctypes.byref(a), 1, None, 0, 1, 1, 1, 1, 1, None, 1, 1, None) == no
    assert lib.xp_attention_workspace_bytes(None, ctypes.byref(a)) == 0
    assert lib.xp_verify_workspace_bytes(None, 1) == 0
    lib.xp_cache_destroy(None)


@pytest.mark.parametrize("bad", [
    dict(pages=0), dict(page_size=0), dict(layers=0), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=257),
    dict(max_seqs=0), dict(dtype=7), dict(stride_page=16 * 8 * 128 - 1), dict(stride_token=8 * 128 + 8),
    dict(stride_head=64), dict(stride_layer=-1)], ids=str)
def test_cache_descriptors_refused(lib, bad):
    d = desc(**bad)
    out = ctypes.c_void_p()
    assert xp.xp_cache_prep_bytes(d) == 0
    assert lib.xp_cache_create(ctypes.byref(d), 4096, 1 << 30, None, ctypes.byref(out)) == xp.XP_EINVAL
    assert out.value is None


def test_cache_create_refused(lib):
    out = ctypes.c_void_p()
    d = desc()
    need = xp.xp_cache_prep_bytes(d)
    # the error word, five arrays over pages at most, three over rows
    assert 4 * (4 * 100 + 3 * 32) <= need <= 4 * (4 * 100 + 3 * 32) + 9 * 256
    for args, code in (((None, need), xp.XP_EINVAL), ((4097, need), xp.XP_EINVAL),
                       ((4096, need - 1), xp.XP_ECAPACITY)):
        assert lib.xp_cache_create(ctypes.byref(d), *args, None, ctypes.byref(out)) == code
    for bad in (dict(k=None), dict(v=None), dict(k=4097)):
        assert lib.xp_cache_create(ctypes.byref(desc(**bad)), 4096, need, None,
                                   ctypes.byref(out)) == xp.XP_EINVAL
    assert lib.xp_cache_create(ctypes.byref(d), 4096, need, None, None) == xp.XP_EINVAL


def test_page_orders(lib):
    heads_outside = dict(stride_head=16 * 128, stride_token=128)
    assert xp.xp_cache_prep_bytes(desc(**heads_outside)) > 0
    # one head, or one token a page: the other stride does not matter
    assert xp.xp_cache_prep_bytes(desc(kv_heads=1, stride_token=128, stride_head=5)) > 0
    assert xp.xp_cache_prep_bytes(desc(page_size=1, stride_token=3)) > 0


def test_new_status_strings(lib):
    for code in range(9, 14):
        assert xp.status_str(code) != "unknown status" and code in xp.STATUS


def test_pages_whose_size_passes_64_bits_are_refused(lib):
    huge = dict(page_size=1 << 30, kv_heads=1 << 30, head_dim=16, stride_token=1 << 34, stride_head=16)
    assert xp.xp_cache_prep_bytes(desc(**huge)) == 0          # 2^64 elements
    assert xp.xp_cache_prep_bytes(desc(page_size=1 << 21, stride_page=1 << 40)) == 0          # 2^31
