"""Which tensors the scored attention calls look at before they launch on the
current device, and where the stream comes from, without a GPU: stand-ins for
tensors and for the library."""

import pytest

from paged_kv_cache_hkv_gb300 import binding

torch = pytest.importorskip("torch")

T, HQ, HKV, D, R, BLOCKS, WIDTH = 5, 4, 2, 64, 3, 8, 4


class Stand:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return self.shape[i + 1:].numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


def tensors():
    bf, i32 = torch.bfloat16, torch.int32
    return dict(out=Stand(bf, T, HQ, D), q=Stand(bf, T, HQ, D), kv_cache=Stand(bf, BLOCKS, 2, 16, HKV, D),
                key=Stand(bf, T, HKV, D), value=Stand(bf, T, HKV, D),
                block_table=Stand(i32, R, WIDTH), seq_lens=Stand(i32, R),
                query_start_loc=Stand(i32, R + 1), num_computed_tokens=Stand(i32, R),
                workspace=Stand(torch.uint8, 512), slot_mapping=Stand(torch.int64, T),
                alibi_slopes=Stand(torch.float32, HQ), key_begin=Stand(i32, T), key_end=Stand(i32, T))


SCORES = ("alibi_slopes", "key_begin", "key_end")
WRITE = ("key", "value", "slot_mapping")
CALLS = {"pkv_paged_attention": (binding.pkv_paged_attention, WRITE),
         "pkv_paged_attention_with_write": (binding.pkv_paged_attention_with_write, ()),
         "pkv_paged_attention_static_workspace": (binding.pkv_paged_attention_static_workspace,
                                                  WRITE + ("workspace",)),
         "StepCalls": (lambda **kw: binding.StepCalls(**kw).attend(), ())}


@pytest.fixture
def library(monkeypatch):
    called = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(binding, "load", Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0x40, raising=False)
    return called


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_of_a_scored_call_is_on_one_device(library, name):
    call, without = CALLS[name]
    sizes = dict(max_query_len=4, max_seq_len=40, scale=0.125)

    def args(skip=()):
        return {k: t for k, t in tensors().items() if k not in without and k not in skip}

    call(**args(), **sizes)
    assert len(library) == 1
    for moved in args():
        a = args()
        a[moved].device = torch.device("cuda", 1)
        with pytest.raises(ValueError, match="cuda:"):
            call(**a, **sizes)
        # the cap alone makes a call a scored one
        if moved not in SCORES:
            a = args(SCORES)
            a[moved].device = torch.device("cuda", 1)
            with pytest.raises(ValueError, match="cuda:"):
                call(**a, softcap=30.0, **sizes)
    assert len(library) == 1
    # all on another device than the current one
    a = args()
    for t in a.values():
        t.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="current device"):
        call(**a, **sizes)
    # plain calls are checked no more than they were
    a = args(SCORES)
    a["kv_cache"].device = torch.device("cuda", 1)
    call(**a, **sizes)
    assert len(library) == 2


def test_the_current_stream_without_torchs_private_call(monkeypatch):
    from types import SimpleNamespace
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: SimpleNamespace(cuda_stream=0x70 + d))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0x40 + i, raising=False)
    assert binding._stream(None).value == 0x42
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert binding._stream(None).value == 0x72 and binding._stream(None, 2).value == 0x72
