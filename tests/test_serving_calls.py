"""The calls of serving.py around the library, without a GPU: tensors are stand-ins that say they lie on one, and the
library's entry points are replaced, so that nothing is launched."""
import os
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


class Fake:
    """What serving.py asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self._stride = torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        return self._stride if d is None else self._stride[d]

    def data_ptr(self):
        return 4096


@pytest.fixture
def sv():
    from bit_quantized_sparse_gb300 import _build
    if not os.path.exists(_build.LIB):
        _build.build()
    from bit_quantized_sparse_gb300 import serving
    return serving


@pytest.fixture
def calls(sv, monkeypatch):
    """The library's calls by name, with their arguments; every one succeeds.  GPU 0 is current."""
    made = []
    for name in ("moe_w4_kv_append", "moe_w4_attend_decode", "moe_w4_kv_evict", "moe_w4_token_logprobs",
                 "moe_w4_workspace_init"):
        monkeypatch.setattr(sv.mw, name, lambda *a, name=name: made.append((name, a)) or 0)
    monkeypatch.setattr(sv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(sv, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(sv, "_empty", lambda stream, shape, dtype, device: Fake(shape, dtype, device))
    monkeypatch.setattr(sv, "_ctrl", {})
    monkeypatch.setattr(sv, "_capturing", lambda stream: False, raising=False)
    return made


def cache(sv, device="cuda:0", seqs=2, pages=4, page=16, heads=2, dim=64, slots=None):
    kv = [Fake((8, heads, page, dim), torch.bfloat16, device) for _ in range(2)]
    shape = (seqs, heads, slots or pages * page)
    return sv.PagedKVCache(*kv, Fake((seqs, pages), torch.int32, device), Fake((seqs,), torch.int32, device),
                           Fake(shape, torch.float32, device), Fake(shape, torch.int32, device))


def every_call(sv, device="cuda:0", stream=None):
    """One call of each operator, as functions."""
    c = cache(sv, device)
    q = Fake((2, 4, 64), torch.bfloat16, device)
    new = Fake((2, 2, 64), torch.bfloat16, device)
    seen = Fake((2,), torch.int32, device)
    x = Fake((3, 100), torch.float32, device)
    return c, [lambda: sv.kv_append(c, new, new, stream=stream), lambda: sv.attend_decode(c, q, stream=stream),
               lambda: sv.kv_evict(c, seen, 32, stream=stream), lambda: sv.token_logprobs(x, top=3, stream=stream)]


def test_calls_reach_the_library(sv, calls):
    for call in every_call(sv)[1]:
        call()
    assert [name for name, _ in calls if name != "moe_w4_workspace_init"] == [
        "moe_w4_kv_append", "moe_w4_attend_decode", "moe_w4_kv_evict", "moe_w4_token_logprobs"]


@pytest.mark.parametrize("device,stream", [
    ("cuda:1", None),                                                                     # tensors of a GPU that is not current
    ("cuda:1", SimpleNamespace(cuda_stream=7, device=torch.device("cuda:1"))),
    ("cuda:0", SimpleNamespace(cuda_stream=7, device=torch.device("cuda:1")))])           # a stream of another GPU
def test_other_gpus_are_refused(sv, calls, device, stream):
    """The library launches on the current GPU: tensors and streams of another one are refused, with nothing enqueued."""
    c, every = every_call(sv, device, stream)
    for call in every:
        with pytest.raises(ValueError, match="GPU"):
            call()
    assert not calls and not c._ws and not c._kept and not sv._ctrl


@pytest.mark.parametrize("which", range(4))
def test_first_call_in_a_capture_is_refused(sv, calls, monkeypatch, which):
    """A workspace made while its stream is captured would be cleared by the graph only, and taken for clear before."""
    stream = SimpleNamespace(cuda_stream=9, device=torch.device("cuda:0"))
    c, every = every_call(sv, stream=stream)
    monkeypatch.setattr(sv, "_capturing", lambda s: s is stream)
    with pytest.raises(RuntimeError, match="captur"):
        every[which]()
    assert not calls and not c._ws and not c._kept and not sv._ctrl
    monkeypatch.setattr(sv, "_capturing", lambda s: False)
    every[which]()                                             # the call outside
    made = len(calls)
    monkeypatch.setattr(sv, "_capturing", lambda s: True)
    every[which]()                                             # may be captured then
    assert len(calls) == made + 1 and calls[-1][0] != "moe_w4_workspace_init"


def test_larger_workspace_in_a_capture_is_refused(sv, calls, monkeypatch):
    c, (append, attend, _, _) = every_call(sv)
    append()
    monkeypatch.setattr(sv, "_capturing", lambda s: True)
    append()
    ws = dict(c._ws)
    with pytest.raises(RuntimeError, match="captur"):
        attend()                                               # needs a larger one than the append made
    assert c._ws == ws and len(c._kept) == 1


def test_reset_clears_every_workspace(sv, calls, monkeypatch):
    """All that graphs may hold, in place, with the GPU idle before and after."""
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: calls.append(("synchronize", ())))
    monkeypatch.setattr(Fake, "numel", lambda self: self.shape.numel(), raising=False)
    c, every = every_call(sv)
    for call in every:
        call()
    sizes = [t.numel() for t in c._kept]
    assert len(sizes) == 2                                     # the append's, and a larger one
    kept, ctrl = list(c._kept), dict(sv._ctrl)
    for reset, want in ((c.reset, sizes), (sv.logprobs_reset, [256])):
        del calls[:]
        reset()
        assert [a[1] for name, a in calls if name == "moe_w4_workspace_init"] == want
        assert calls[0][0] == calls[-1][0] == "synchronize"
    assert c._kept == kept and sv._ctrl == ctrl


def test_attention_of_a_cache_with_fewer_weights_than_places(sv, calls):
    """With weights the default bound is what they have room for: the library refuses a larger one."""
    c = cache(sv, slots=40)
    q = Fake((2, 4, 64), torch.bfloat16, "cuda:0")
    sv.attend_decode(c, q, weight_out=c.weight)
    sv.attend_decode(c, q)
    sv.attend_decode(c, q, max_len=7, weight_out=c.weight)
    assert [a[5] for name, a in calls if name == "moe_w4_attend_decode"] == [40, 64, 7]


@pytest.mark.parametrize("kw", [dict(budget=2 ** 32 + 8), dict(sink=2 ** 32), dict(recent=2 ** 32 + 1), dict(max_len=2 ** 32 + 40),
                                dict(budget=2 ** 31), dict(recent=-2 ** 32)])
def test_eviction_refuses_numbers_past_32_bits(sv, calls, kw):
    """The C ABI takes ints: cut to 32 bits, a budget of 2^32 + 8 would keep 8 tokens."""
    with pytest.raises(ValueError, match=next(iter(kw))):
        sv.kv_evict(cache(sv), Fake((2,), torch.int32, "cuda:0"), **{**dict(budget=32), **kw})
    assert not calls


def test_other_calls_refuse_numbers_past_32_bits(sv, calls):
    q = Fake((2, 4, 64), torch.bfloat16, "cuda:0")
    with pytest.raises(ValueError, match="max_len"):
        sv.attend_decode(cache(sv), q, max_len=2 ** 32 + 5)
    with pytest.raises(ValueError, match="top"):
        sv.token_logprobs(Fake((2, 100), torch.float32, "cuda:0"), top=2 ** 32 + 3)
    assert not calls


def test_growing_sequences_leave_nothing_behind(sv, calls):
    """A decode loop gives another bound every step: what the cache remembers of them does not grow."""
    c = cache(sv, pages=4096)
    q = Fake((2, 4, 64), torch.bfloat16, "cuda:0")
    seen = Fake((2,), torch.int32, "cuda:0")
    for n in range(1, 3000):
        sv.attend_decode(c, q, max_len=n)
        sv.kv_evict(c, seen, n, max_len=n + 1)
    assert len(c._sizes) <= 256 and len(c._kept) <= 8
    assert calls[-1][1][-2] >= sv.mw.moe_w4_evict_workspace_size(c._c, 2999, 3000)   # and the workspace still suffices
