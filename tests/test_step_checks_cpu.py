"""What the binding passes on and refuses, without a GPU: tensors that say they are on one, and a
library that records its calls."""
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(xp, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib.calls


def test_append_passes_the_columns_of_its_table(calls):
    wide = gpu(3, 10, dtype=torch.int32)
    k = gpu(3, 2, 4, 8)
    xp.xp_cache_append(1, 0, k, k, wide[:, 4:8], gpu(3, dtype=torch.int32), stream=0)
    (_, args), = calls
    assert args[11:13] == (10, 4)          # rows 10 apart, 4 columns


def i32(*shape):
    return gpu(*shape, dtype=torch.int32)


def verify_args():
    i64 = torch.int64
    return dict(target=gpu(2, 4, 64), draft=gpu(6, 64), blk=gpu(2, 4, dtype=i64), n_draft=i32(2),
                temperature=gpu(2), u=gpu(2, 3), noise=gpu(2, 64), tokens=gpu(2, 4, dtype=i64),
                counts=i32(2), prob=gpu(2, 3), ws=gpu(256, dtype=torch.uint8))


def attention_args():
    q, out = gpu(2, 3, 4, 64), gpu(2, 3, 4, 64)
    return dict(attn=xp.make_attn(q, out, 0, 20, 40, 0.1), q=q, prefix_table=i32(2), table=i32(2, 3),
                lens=i32(2), out=out, lse=gpu(2, 3, 4), ws=gpu(256, dtype=torch.uint8))


CALLS = {
    "xp_verify_drafts": (xp.xp_verify_drafts, verify_args),
    "xp_prefix_attention": (xp.xp_prefix_attention, attention_args),
    "xp_cache_append": (xp.xp_cache_append, lambda: dict(
        layer=0, k=gpu(2, 3, 1, 8), v=gpu(2, 3, 1, 8), table=i32(2, 3), lens=i32(2))),
    "xp_cache_copy": (xp.xp_cache_copy, lambda: dict(src=i32(2), dst=i32(2))),
    "xp_cache_resize": (xp.xp_cache_resize, lambda: dict(
        table=i32(2, 3), lens=i32(2), new_lens=i32(2), refs=i32(9), table_out=i32(2, 3), lens_out=i32(2),
        refs_out=i32(9))),
    "xp_cache_fork": (xp.xp_cache_fork, lambda: dict(
        table=i32(2, 3), lens=i32(2), parent=i32(4), cut=i32(4), refs=i32(9), child_table=i32(4, 3),
        child_lens=i32(4), refs_out=i32(9))),
    "xp_cache_compact": (xp.xp_cache_compact, lambda: dict(
        table=i32(2, 3), lens=i32(2), refs=i32(9), table_out=i32(2, 3), refs_out=i32(9), map=i32(9),
        live=i32(1))),
}
TENSORS = [(name, arg) for name, (_, args) in CALLS.items() for arg, t in args().items()
           if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name,arg", TENSORS, ids=lambda x: x)
def test_every_tensor_has_to_be_on_the_current_device(calls, monkeypatch, name, arg):
    call, args = CALLS[name]
    args = args()
    call(1, stream=0, **args)
    assert [c[0] for c in calls] == [name if name != "xp_cache_append" else "xp_cache_append_columns"]
    calls.clear()
    host = args[arg].as_subclass(torch.Tensor)
    with pytest.raises(ValueError, match="%s: not on the current" % arg):
        call(1, stream=0, **{**args, arg: host})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="not on the current"):
        call(1, stream=0, **args)
    assert not calls


def test_pools_and_scratch_have_to_be_on_the_current_device(calls):
    k, v = gpu(1, 4, 4, 1, 8), gpu(1, 4, 4, 1, 8)
    d = xp.make_cache_desc(k, v)
    xp.xp_cache_create(d, gpu(256, dtype=torch.uint8), stream=0)
    calls.clear()
    for bad in (lambda: xp.make_cache_desc(k.as_subclass(torch.Tensor), v),
                lambda: xp.make_cache_desc(k, v.as_subclass(torch.Tensor)),
                lambda: xp.xp_cache_create(d, torch.zeros(256, dtype=torch.uint8), stream=0)):
        with pytest.raises(ValueError, match="not on the current"):
            bad()
    assert not calls


def test_lse_is_fp32(calls):
    args = attention_args()
    with pytest.raises(ValueError, match="lse"):
        xp.xp_prefix_attention(1, stream=0, **{**args, "lse": i32(2, 3, 4)})
    assert not calls


@pytest.mark.parametrize("has_raw", [True, False])
def test_the_current_stream_with_and_without_the_private_call(monkeypatch, has_raw):
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    if has_raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 77 + device, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert xp._stream(None) == (80 if has_raw else 1234)
    assert xp._stream(5) == 5 and xp._stream(Stream) == 1234
