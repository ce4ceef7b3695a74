"""The operators around the sparse-MoE layer in a decode step, on torch tensors.

Thin calls of include/moe_w4_serving.h (libmoe_w4.so): a paged key-value cache
(`PagedKVCache`, `kv_append`), the attention of one new token per sequence over
it (`attend_decode`), cutting it to a budget by accumulated attention weight
(`kv_evict`), and token log probabilities with entropy and the top alternatives
(`token_logprobs`).

Every call is enqueued on `stream` (default: the current stream) and returns at
once; what it allocates belongs to that stream, tensors given to it must be
ready there, and they and the stream belong to the current GPU.  Arguments are
checked here (ValueError) and in the library (moe_w4.MoeW4Error); indexes in
device memory are checked by the kernels, which leave out what is out of range
and set the sticky status word (`PagedKVCache.status` and `reset`,
`logprobs_status` and `logprobs_reset`).  For use in a CUDA graph make one call
of the same sizes on the capturing stream first, so that its workspace exists
(RuntimeError otherwise); the cache keeps every workspace that a graph may hold.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import moe_w4 as mw

_TYPES = {torch.bfloat16: mw.MOE_W4_TYPE_BF16, torch.float16: mw.MOE_W4_TYPE_FP16, torch.float32: mw.MOE_W4_TYPE_FP32}
_byref = ctypes.byref


def _need(ok, what):
    if not ok:
        raise ValueError(what)


_INT = 2 ** 31   # C ints: ctypes would cut larger numbers to 32 bits


# The current stream's handle without the Stream object around it, where torch offers that (a call saves 3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _handle(stream, device):
    """The handle to launch on.  The library takes the current GPU, so tensors and stream have to be its own."""
    if device.index != _current_device():
        raise ValueError("tensors on %s, which is not the current GPU" % device)
    if stream is None:
        return _raw_stream(device.index)
    if stream.device != device:
        raise ValueError("a stream of the tensors' GPU")
    return stream.cuda_stream


def _empty(stream, shape, dtype, device):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _capturing(stream):
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _new_workspace(nbytes, device, stream):
    """`nbytes` of device memory of the call's stream, cleared there: now, not whenever a graph runs."""
    if _capturing(stream):
        raise RuntimeError("the stream is being captured and has no workspace for this call: make one call of the same "
                           "sizes on it before the capture")
    ws = _empty(stream, (nbytes,), torch.uint8, device)
    mw._check(mw.moe_w4_workspace_init(ws.data_ptr(), nbytes, _handle(stream, device)), "workspace_init")
    return ws


def _clear(workspaces, device):
    """Clears workspaces in place (graphs may hold their addresses), with the GPU idle before and after."""
    torch.cuda.synchronize(device)
    for ws in workspaces:
        mw._check(mw.moe_w4_workspace_init(ws.data_ptr(), ws.numel(), _handle(None, device)), "workspace_init")
    torch.cuda.synchronize(device)


def _word(ws):
    off = mw.moe_w4_status_offset()
    return int(ws[off:off + 4].view(torch.int32).item())


def _stride(t, d):
    """Stride of a dimension that is walked; one of a single entry has none."""
    return t.stride(d) if t.shape[d] > 1 else 0


class PagedKVCache:
    """A paged cache made of the caller's tensors (none is copied).

    k, v         bf16 or fp16, [pages][kv heads][page slots][head dim] views, last
                 dimension contiguous; storage in the order
                 [pages][slots][heads][dim] is given as .permute(0, 2, 1, 3)
    block_table  int32 [sequences][pages per sequence]
    seq_lens     int32 [sequences], tokens held; a decode step raises it by one
                 before kv_append and attend_decode
    weight, pos  fp32 and int32 [sequences][kv heads][slots], or None: the
                 attention weight that each token has drawn, and its position;
                 attend_decode adds up the first, eviction goes by both
    """

    def __init__(self, k, v, block_table, seq_lens, weight=None, pos=None):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype, "k and v: equal 4-D tensors")
        _need(k.dtype in (torch.bfloat16, torch.float16), "k and v: bfloat16 or float16")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "k and v: a contiguous head dimension")
        _need(all(_stride(k, d) == _stride(v, d) for d in range(3)), "k and v: equal strides")
        _need(block_table.dtype == torch.int32 and block_table.dim() == 2, "block_table: int32 [sequences][pages]")
        _need(_stride(block_table, 1) in (0, 1), "block_table: contiguous rows")
        n_seqs = block_table.shape[0]
        _need(seq_lens.dtype == torch.int32 and tuple(seq_lens.shape) == (n_seqs,) and _stride(seq_lens, 0) in (0, 1),
              "seq_lens: contiguous int32 [sequences]")
        _need(pos is None or weight is not None, "pos goes with weight")
        tensors = [k, v, block_table, seq_lens] + [t for t in (weight, pos) if t is not None]
        _need(all(t.is_cuda and t.device == k.device for t in tensors), "all tensors on one GPU")
        self.k, self.v, self.block_table, self.seq_lens, self.weight, self.pos = k, v, block_table, seq_lens, weight, pos
        self.device, self.n_seqs, self.n_kv_heads, self.head_dim = k.device, n_seqs, k.shape[1], k.shape[3]
        self.page_size, self.dtype = k.shape[2], k.dtype
        self.capacity = block_table.shape[1] * k.shape[2]
        c = self.c = mw.MoeW4KvCache()
        c.dtype, c.n_kv_heads, c.head_dim = _TYPES[k.dtype], k.shape[1], k.shape[3]
        c.page_size, c.num_pages = k.shape[2], k.shape[0]
        c.page_stride, c.head_stride, c.slot_stride = (_stride(k, d) for d in range(3))
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.n_seqs, c.pages_per_seq, c.table_stride = n_seqs, block_table.shape[1], _stride(block_table, 0)
        c.block_table, c.seq_lens = block_table.data_ptr(), seq_lens.data_ptr()
        self._c = _byref(c)
        self.t = self._t = None
        if weight is not None:
            _need(weight.dtype == torch.float32 and weight.dim() == 3
                  and tuple(weight.shape[:2]) == (n_seqs, self.n_kv_heads) and _stride(weight, 2) in (0, 1),
                  "weight: float32 [sequences][kv heads][slots], contiguous slots")
            if pos is not None:
                self._check_like_weight(pos, torch.int32)
            t = self.t = mw.MoeW4KvTrack()
            t.weight, t.pos, t.slots = weight.data_ptr(), mw._ptr(pos), weight.shape[2]
            t.seq_stride, t.head_stride = _stride(weight, 0), _stride(weight, 1)
            self._t = _byref(t)
        self._ws, self._sizes, self._kept = {}, {}, []

    @classmethod
    def allocate(cls, num_pages, page_size, n_kv_heads, head_dim, block_table, seq_lens, dtype=torch.bfloat16,
                 layout="head", track=False):
        """A cache on the block table's GPU.  layout "head": [pages][heads][slots][dim], "slot":
        [pages][slots][heads][dim].  Cached keys and values start undefined."""
        _need(layout in ("head", "slot"), "layout: 'head' or 'slot'")
        dev = block_table.device
        shape = (num_pages, n_kv_heads, page_size, head_dim)
        if layout == "slot":
            shape = (num_pages, page_size, n_kv_heads, head_dim)
        kv = [torch.empty(shape, dtype=dtype, device=dev) for _ in range(2)]
        if layout == "slot":
            kv = [t.permute(0, 2, 1, 3) for t in kv]
        weight = pos = None
        if track:
            shape = (block_table.shape[0], n_kv_heads, block_table.shape[1] * page_size)
            weight = torch.zeros(shape, dtype=torch.float32, device=dev)
            pos = torch.zeros(shape, dtype=torch.int32, device=dev)
        return cls(*kv, block_table, seq_lens, weight, pos)

    def _check_like_weight(self, t, dtype):
        """An array beside the cache has the layout of the cache's own weights."""
        w = self.weight
        if not (t.dtype is dtype and t.shape == w.shape and t.device == self.device
                and (t.stride() == w.stride() or all(_stride(t, d) == _stride(w, d) for d in range(3)))):
            raise ValueError("expected %s with the shape and strides of the cache's weights" % dtype)

    def _workspace(self, nbytes, stream, handle):
        """(address, bytes) of the stream's workspace.  One that has become too small is kept, as a CUDA graph may
        hold its address; sizes double, so those kept are no more than the one in use."""
        ws = self._ws.get(handle)
        if ws is None or ws[1] < nbytes:
            if ws is not None:
                nbytes = max(nbytes, 2 * ws[1])
            t = _new_workspace(nbytes, self.device, stream)
            self._kept.append(t)
            ws = self._ws[handle] = (t.data_ptr(), nbytes, t)
        return ws

    def _remember(self, key, size):
        """Keeps a call's workspace size; a loop whose bound grows step by step asks for ever new ones."""
        if len(self._sizes) >= 256:
            self._sizes.clear()
        size = self._sizes[key] = max(size, mw.CTRL_BYTES)
        return size

    def status(self) -> int:
        """The device status of the calls on this cache, all streams together (synchronises)."""
        torch.cuda.synchronize(self.device)
        got = 0
        for ws in self._kept:
            got |= _word(ws)
        return got

    def reset(self) -> None:
        """Clears the device status and the workspaces of this cache, all streams together, as has to be done after a
        wait that ran out (synchronises).  Keys, values, lengths, weights and positions stay."""
        _clear(self._kept, self.device)


def _like(t, dtype, shape, device):
    return t.dtype is dtype and t.shape == shape and t.device == device


def _check_index(t, n, device, what):
    if not (_like(t, torch.int32, (n,), device) and (n <= 1 or t.stride(0) == 1)):
        raise ValueError(what + ": contiguous int32 of %d entries on %s" % (n, device))


def _token_stride(t, heads, dim):
    """Elements between tokens of a [tokens][heads][dim] view, or -1 if a token is not contiguous."""
    token, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1):
        return -1
    return token if t.shape[0] > 1 else 0


def kv_append(cache: PagedKVCache, k, v, seq=None, slot=None, pos=None, stream=None) -> None:
    """Writes tokens' keys and values, [tokens][kv heads][head dim] each, into the cache.

    seq, slot  int32 [tokens]: the sequence of each token (None: token i is sequence i's) and its index in it
               (None: the last one, seq_lens - 1)
    pos        int32 [tokens]: position noted for eviction (None: the index); a cache with weights notes it and
               starts the token's weight at 0
    """
    device, heads, dim, n = cache.device, cache.n_kv_heads, cache.head_dim, k.shape[0]
    shape = (n, heads, dim)
    if not (_like(k, cache.dtype, shape, device) and _like(v, cache.dtype, shape, device)):
        raise ValueError("k and v: [tokens][kv heads][head dim] of the cache's type on its GPU")
    k_stride, v_stride = _token_stride(k, heads, dim), _token_stride(v, heads, dim)
    if k_stride < 0 or v_stride < 0:
        raise ValueError("k and v: each token contiguous")
    if seq is not None:
        _check_index(seq, n, device, "seq")
    if slot is not None:
        _check_index(slot, n, device, "slot")
    if pos is not None:
        _check_index(pos, n, device, "pos")
    handle = _handle(stream, device)
    ws = cache._workspace(mw.CTRL_BYTES, stream, handle)
    status = mw.moe_w4_kv_append(cache._c, cache._t, n, k.data_ptr(), k_stride, v.data_ptr(), v_stride, mw._ptr(seq),
                                 mw._ptr(slot), mw._ptr(pos), ws[0], ws[1], handle)
    if status:
        mw._check(status, "moe_w4_kv_append")


def attend_decode(cache: PagedKVCache, q, scale: Optional[float] = None, max_len: Optional[int] = None, out=None,
                  return_lse=False, weight_out=None, stream=None):
    """Attention of one new token per sequence, q [sequences][query heads][head dim], over its cached tokens.

    scale       of the scores (default 1/sqrt(head dim))
    max_len     upper bound of seq_lens (default: what the block table, and the weights if they are added up, can
                hold); a small one saves work
    return_lse  also return the log sum of the exponentials, fp32 [sequences][query heads]
    weight_out  fp32 tensor like cache.weight (it may be cache.weight itself): gets cache.weight plus the
                probability that each token drew, summed over the kv head's query heads
    Returns out, or (out, lse).
    """
    device, dim, dtype = cache.device, cache.head_dim, cache.dtype
    shape = q.shape
    if not (len(shape) == 3 and shape[0] == cache.n_seqs and shape[2] == dim and q.dtype is dtype and q.device == device):
        raise ValueError("q: [sequences][query heads][head dim] of the cache's type on its GPU")
    heads = shape[1]
    q_stride = _token_stride(q, heads, dim)
    if out is None:
        out = _empty(stream, shape, dtype, device)
        out_stride = heads * dim
    else:
        if not _like(out, dtype, shape, device):
            raise ValueError("out: like q")
        out_stride = _token_stride(out, heads, dim)
    if q_stride < 0 or out_stride < 0:
        raise ValueError("q and out: contiguous heads")
    lse = _empty(stream, (shape[0], heads), torch.float32, device) if return_lse else None
    track = None
    if weight_out is not None:
        _need(cache.weight is not None, "weight_out needs a cache with weights")
        cache._check_like_weight(weight_out, torch.float32)
        track = cache._t
    if max_len is None:
        max_len = cache.capacity if track is None else min(cache.capacity, cache.weight.shape[2])
    else:
        max_len = int(max_len)
    if not -_INT <= max_len < _INT:
        raise ValueError("max_len: a 32-bit integer")
    handle = _handle(stream, device)
    key = (heads, max_len, weight_out is not None)
    size = cache._sizes.get(key)
    if size is None:
        size = cache._remember(key, mw.moe_w4_attend_workspace_size(cache._c, heads, max_len, key[2]))
    ws = cache._workspace(size, stream, handle)
    status = mw.moe_w4_attend_decode(cache._c, heads, q.data_ptr(), q_stride, dim ** -0.5 if scale is None else scale,
                                     max_len, out.data_ptr(), out_stride, mw._ptr(lse), track, mw._ptr(weight_out),
                                     ws[0], ws[1], handle)
    if status:
        mw._check(status, "moe_w4_attend_decode")
    return (out, lse) if return_lse else out


def kv_evict(cache: PagedKVCache, seen, budget: int, sink: int = 0, recent: int = 0, max_len: Optional[int] = None,
             lens_out=None, weight_out=None, pos_out=None, stream=None) -> None:
    """Cuts every sequence of more than `budget` tokens to `budget`, head by head, keeping the tokens at positions
    below `sink` or among the last `recent` of the `seen` (int32 [sequences]) tokens fed, then those with the larger
    accumulated weight.  Keys and values move inside the cache; lengths, weights and positions go to lens_out,
    weight_out and pos_out (default: cache.seq_lens, cache.weight and cache.pos, in place)."""
    _need(cache.pos is not None, "eviction needs a cache with weights and positions")
    device = cache.device
    _check_index(seen, cache.n_seqs, device, "seen")
    if lens_out is None:
        lens_out = cache.seq_lens
    else:
        _check_index(lens_out, cache.n_seqs, device, "lens_out")
    if weight_out is None:
        weight_out = cache.weight
    else:
        cache._check_like_weight(weight_out, torch.float32)
    if pos_out is None:
        pos_out = cache.pos
    else:
        cache._check_like_weight(pos_out, torch.int32)
    max_len = min(cache.capacity, cache.weight.shape[2]) if max_len is None else int(max_len)
    budget = int(budget)
    if not (-_INT <= budget < _INT and -_INT <= sink < _INT and -_INT <= recent < _INT and -_INT <= max_len < _INT):
        raise ValueError("budget, sink, recent and max_len: 32-bit integers")
    handle = _handle(stream, device)
    key = (budget, max_len)
    size = cache._sizes.get(key)
    if size is None:
        size = cache._remember(key, mw.moe_w4_evict_workspace_size(cache._c, *key))
    ws = cache._workspace(size, stream, handle)
    status = mw.moe_w4_kv_evict(cache._c, cache._t, seen.data_ptr(), budget, sink, recent, max_len, lens_out.data_ptr(),
                                weight_out.data_ptr(), pos_out.data_ptr(), ws[0], ws[1], handle)
    if status:
        mw._check(status, "moe_w4_kv_evict")


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]       # fp32 [rows], None without targets
    entropy: torch.Tensor                 # fp32 [rows]
    top_index: Optional[torch.Tensor]     # int32 [rows][top], None for top = 0
    top_logprob: Optional[torch.Tensor]   # fp32 [rows][top]


_ctrl = {}   # (device index, stream) -> control header of the log-probability calls there, and its address


def token_logprobs(logits, targets=None, top: int = 0, stream=None) -> TokenLogprobs:
    """Log probabilities under softmax(logits) of int32 `targets` [rows] (-1: none asked, 0 returned), the entropy
    (natural logarithms), and the `top` most likely tokens, best first, the lower index first among equals.

    logits: fp32, bf16 or fp16 [rows][vocabulary], contiguous rows."""
    kind = _TYPES.get(logits.dtype)
    if kind is None or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits: a 2-D fp32, bf16 or fp16 tensor on the GPU")
    n, vocab = logits.shape
    row, one = logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError("logits: contiguous rows")
    device = logits.device
    if targets is not None:
        _check_index(targets, n, device, "targets")
    if not -_INT <= top < _INT:
        raise ValueError("top: a 32-bit integer")
    handle = _handle(stream, device)
    key = (device.index, handle)
    ws = _ctrl.get(key)
    if ws is None:
        t = _new_workspace(mw.CTRL_BYTES, device, stream)
        ws = _ctrl[key] = (t.data_ptr(), t)
    logprob = index = value = None
    entropy = _empty(stream, (n,), torch.float32, device)
    if targets is not None:
        logprob = _empty(stream, (n,), torch.float32, device)
    if top:
        index = _empty(stream, (n, top), torch.int32, device)
        value = _empty(stream, (n, top), torch.float32, device)
    status = mw.moe_w4_token_logprobs(kind, n, vocab, logits.data_ptr(), row if n > 1 else 0, mw._ptr(targets), top,
                                      mw._ptr(logprob), entropy.data_ptr(), mw._ptr(index), mw._ptr(value), ws[0],
                                      mw.CTRL_BYTES, handle)
    if status:
        mw._check(status, "moe_w4_token_logprobs")
    return TokenLogprobs(logprob, entropy, index, value)


def logprobs_status() -> int:
    """The device status of token_logprobs calls, all streams together (synchronises)."""
    torch.cuda.synchronize()
    got = 0
    for ws in _ctrl.values():
        got |= _word(ws[1])
    return got


def logprobs_reset() -> None:
    """Clears the device status of token_logprobs calls on the current GPU, all streams together (synchronises)."""
    device = torch.device("cuda", _current_device())
    _clear([t for (index, _), (_, t) in _ctrl.items() if index == device.index], device)
