"""Quantised caches and log probabilities on a machine without a GPU: sizes, descriptors and arguments that
are refused before any launch, and what the binding passes on."""
import ctypes

import pytest
import torch

from jacobi_speculative_decode_gb300 import build as B
from jacobi_speculative_decode_gb300 import xp
from oracle import quant_oracle as Q
from test_step_checks_cpu import Recorder, gpu, i32


@pytest.fixture(scope="module")
def lib():
    B.build()
    return xp.lib()


@pytest.mark.parametrize("ps", [1, 5, 16, 20, 64])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 208, 256])
@pytest.mark.parametrize("bits", [4, 8])
def test_bytes_of_a_head(lib, ps, dim, bits):
    assert xp.xp_quant_head_bytes(ps, dim, bits) == Q.sizes(ps, dim, bits)[2]


def test_bytes_refused(lib):
    for ps, dim, dtype in ((0, 64, xp.XP_Q4), (-1, 64, xp.XP_Q8), (16, 0, xp.XP_Q4), (16, 8, xp.XP_Q4),
                           (16, 100, xp.XP_Q8), (16, 272, xp.XP_Q8), (16, 64, xp.XP_BF16), (16, 64, xp.XP_F32),
                           (16, 64, 4)):
        assert lib.xp_quant_head_bytes(ps, dim, dtype) == 0
    with pytest.raises(ValueError, match="bits"):
        xp.xp_quant_head_bytes(16, 64, 6)


def desc(bits=4, **kw):
    ps, heads, dim = kw.get("page_size", 16), kw.get("kv_heads", 8), kw.get("head_dim", 128)
    code, _, size = Q.sizes(ps, dim, bits)
    d = dict(pages=100, page_size=ps, layers=2, kv_heads=heads, head_dim=dim, max_seqs=32,
             dtype=xp.XP_Q4 if bits == 4 else xp.XP_Q8, stride_layer=100 * heads * size,
             stride_page=heads * size, stride_token=code, stride_head=size, k=4096, v=4096)
    d.update(kw)
    return xp.xp_cache_desc(**d)


@pytest.mark.parametrize("bits", [4, 8])
def test_descriptors(lib, bits):
    size = Q.sizes(16, 128, bits)[2]
    assert xp.xp_cache_prep_bytes(desc(bits)) > 0
    assert xp.xp_cache_prep_bytes(desc(bits, stride_page=8 * size + 16)) > 0
    assert xp.xp_cache_prep_bytes(desc(bits, kv_heads=1, stride_head=3)) > 0       # never used
    assert xp.xp_cache_prep_bytes(desc(bits, page_size=1, stride_token=3)) > 0
    assert xp.xp_cache_prep_bytes(desc(bits, pages=1, stride_page=8 * size + 1)) > 0
    assert xp.xp_cache_prep_bytes(desc(bits, layers=1, stride_layer=5)) > 0


BAD = [dict(pages=0), dict(page_size=0), dict(layers=0), dict(kv_heads=0), dict(max_seqs=0), dict(head_dim=72),
       dict(head_dim=272), dict(stride_head=16), dict(stride_token=128 * 8), dict(stride_page=64),
       dict(stride_layer=-16), dict(stride_layer=100 * 8 * 4096 + 8), dict(stride_page=8 * 4096 + 8),
       dict(dtype=5)]


@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("bits", [4, 8])
def test_descriptors_refused(lib, bits, bad):
    kw = dict(bad)
    if "head_dim" in bad:
        kw.update(stride_head=10 ** 6, stride_token=10 ** 3)
    d = desc(bits)
    for name, value in kw.items():
        setattr(d, name, value)
    out = ctypes.c_void_p()
    assert xp.xp_cache_prep_bytes(d) == 0
    assert lib.xp_cache_create(ctypes.byref(d), 4096, 1 << 30, None, ctypes.byref(out)) == xp.XP_EINVAL


def test_sizes_that_pass_31_bits_are_refused(lib):
    for kw in (dict(page_size=1 << 30), dict(kv_heads=1 << 24), dict(page_size=1 << 20, kv_heads=1 << 20)):
        d = desc(4)
        for name, value in kw.items():
            setattr(d, name, value)
        d.stride_head, d.stride_page = 1 << 40, 1 << 62
        assert xp.xp_cache_prep_bytes(d) == 0


def test_create_refused(lib):
    out = ctypes.c_void_p()
    need = xp.xp_cache_prep_bytes(desc())
    for bad in (dict(k=None), dict(v=None), dict(k=4104), dict(v=4097)):      # 16-byte boundaries
        assert lib.xp_cache_create(ctypes.byref(desc(**bad)), 4096, need, None,
                                   ctypes.byref(out)) == xp.XP_EINVAL


def test_no_handle(lib):
    no = xp.XP_ENOTPREPARED
    assert lib.xp_cache_read(None, 0, 1, 1, 1, 1, None, 1, 1, 1, 1, 0, 0, 0, 8, 128, 0, None) == no
    assert lib.xp_token_logprobs(None, 1, 0, 0, 1, 1, 1, 9, 0, None, 0, None, None, None, None, None, 1, 1,
                                 None) == no
    assert lib.xp_logprobs_workspace_bytes(None, 1, 1) == 0


@pytest.mark.parametrize("dtype", [xp.XP_Q8, xp.XP_Q4])
def test_heads_are_not_of_a_cache_type(lib, dtype):
    w = xp.make_weights(64, 8, 8, 8, 4, 2, dtype)
    assert xp.xp_head_prep_bytes(w) == 0
    assert lib.xp_fold_mix(4096, 4096, 8, 4, dtype, None) == xp.XP_EINVAL


@pytest.fixture
def calls(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(xp, "_lib", rec)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return rec.calls


def read_args():
    return dict(layer=0, table=i32(2, 3), lens=i32(2), first=i32(2), k=gpu(2, 3, 1, 16), v=gpu(2, 3, 1, 16))


def logprobs_args():
    i64 = torch.int64
    return dict(logits=gpu(2, 4, 64), tokens=gpu(2, 4, dtype=i64), temperature=gpu(2), logprob=gpu(2, 4),
                entropy=gpu(2, 4), rank=i32(2, 4), top_ids=gpu(2, 4, 3, dtype=i64), top_logprobs=gpu(2, 4, 3),
                ws=gpu(256, dtype=torch.uint8))


CALLS = {"xp_cache_read": (xp.xp_cache_read, read_args), "xp_token_logprobs": (xp.xp_token_logprobs, logprobs_args)}


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, args) in CALLS.items() for a, t in args().items()
                                      if isinstance(t, torch.Tensor)])
def test_every_tensor_has_to_be_on_the_current_device(calls, name, arg):
    call, args = CALLS[name]
    args = args()
    call(1, stream=0, **args)
    assert [c[0] for c in calls] == [name]
    with pytest.raises(ValueError, match="%s: not on the current" % arg):
        call(1, stream=0, **{**args, arg: args[arg].as_subclass(torch.Tensor)})
    assert len(calls) == 1


@pytest.mark.parametrize("arg,bad", [
    ("k", gpu(2, 3, 1, 8)), ("v", gpu(2, 3, 1, 16, dtype=torch.bfloat16)), ("lens", i32(1)),
    ("first", gpu(2)), ("table", i32(1, 3)), ("table", gpu(2, 3)), ("k", gpu(2, 3, 1, 16, 1))], ids=str)
def test_read_arguments_refused(calls, arg, bad):
    with pytest.raises(ValueError):
        xp.xp_cache_read(1, stream=0, **{**read_args(), arg: bad})
    with pytest.raises(ValueError, match="bf16 or fp32"):
        xp.xp_cache_read(1, stream=0, **{**read_args(), "k": i32(2, 3, 1, 16), "v": i32(2, 3, 1, 16)})
    assert not calls


@pytest.mark.parametrize("arg,bad", [
    ("logits", gpu(2, 64, 4).transpose(1, 2)), ("logits", i32(2, 4, 64)), ("tokens", i32(2, 4)),
    ("tokens", gpu(2, 3, dtype=torch.int64)), ("temperature", gpu(1)), ("logprob", gpu(2, 3)),
    ("rank", gpu(2, 4)), ("top_ids", gpu(2, 4, 2, dtype=torch.int64)), ("top_logprobs", gpu(4, 2, 3)),
    ("top_logprobs", gpu(2, 4, 3, dtype=torch.float64)), ("entropy", gpu(4, 2).t())], ids=str)
def test_logprobs_arguments_refused(calls, arg, bad):
    with pytest.raises(ValueError):
        xp.xp_token_logprobs(1, stream=0, **{**logprobs_args(), arg: bad})
    assert not calls


def test_the_number_of_alternatives_is_their_last_size(calls):
    args = logprobs_args()
    xp.xp_token_logprobs(1, stream=0, **args)
    xp.xp_token_logprobs(1, stream=0, **{**args, "top_ids": None})
    xp.xp_token_logprobs(1, stream=0, **{**args, "top_ids": None, "top_logprobs": None})
    assert [c[1][10] for c in calls] == [3, 3, 0]


def test_pools_of_a_quantised_cache(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    size = xp.xp_quant_head_bytes(16, 64, 4)
    u8 = torch.uint8
    k, v = gpu(2, 5, 3, size, dtype=u8), gpu(2, 5, 3, size, dtype=u8)
    d = xp.make_quant_cache_desc(k, v, 16, 64, 4)
    assert (d.pages, d.page_size, d.layers, d.kv_heads, d.head_dim) == (5, 16, 2, 3, 64)
    assert (d.stride_layer, d.stride_page, d.stride_token, d.stride_head) == (15 * size, 3 * size, 32, size)
    wide = gpu(2, 5, 6, size, dtype=u8)
    for bad in ((k, gpu(2, 5, 3, size)), (k, gpu(2, 4, 3, size, dtype=u8)), (wide[:, :, ::2], wide[:, :, ::2]),
                (k[0], v[0])):
        with pytest.raises(ValueError):
            xp.make_quant_cache_desc(*bad, 16, 64, 4)
    for ps, dim, bits in ((16, 72, 4), (0, 64, 4), (16, 64, 8), (17, 64, 4), (16, 64, 5)):
        with pytest.raises(ValueError):
            xp.make_quant_cache_desc(k, v, ps, dim, bits)
