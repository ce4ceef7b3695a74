"""The operators around the sparse-MoE layer in a decode step, on torch tensors.

Thin calls of include/moe_w4_serving.h and include/moe_w4_longctx.h
(libmoe_w4.so): norms of queries and keys with the position rotation
(`qk_norm_rope`, `Rope`), a paged key-value cache of 16-bit values or of 8-bit
codes (`PagedKVCache`, `PagedKVCache8`, `kv_append`, `kv_read`), the attention of
one new token per sequence over it, with a sliding window where asked for
(`attend_decode`), cutting a 16-bit one to a budget by accumulated attention
weight (`kv_evict`), and token log probabilities with entropy and the top
alternatives (`token_logprobs`).

Every call is enqueued on `stream` (default: the current stream) and returns at
once; what it allocates belongs to that stream, tensors given to it must be
ready there, and they and the stream belong to the current GPU.  Arguments are
checked here (ValueError) and in the library (moe_w4.MoeW4Error); indexes in
device memory are checked by the kernels, which leave out what is out of range
and set the sticky status word (`PagedKVCache.status` and `reset`,
`logprobs_status` and `logprobs_reset`).  For use in a CUDA graph make one call
of the same sizes on the capturing stream first, so that its workspace exists
(RuntimeError otherwise); the cache keeps every workspace that a graph may hold.
A stream's calls and the graphs captured on it share its workspace: they run one
after the other.  Graphs that are to run at once are captured on streams of their
own.
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

    _c8 = None

    def __init__(self, k, v, block_table, seq_lens, weight=None, pos=None):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype, "k and v: equal 4-D tensors")
        _need(k.dtype in (torch.bfloat16, torch.float16), "k and v: bfloat16 or float16")
        self._describe(k, v, block_table, seq_lens, k.dtype, weight, pos)
        self.c = self._c_struct(mw.MoeW4KvCache())
        self._c, self._address = _byref(self.c), ctypes.addressof(self.c)
        n_seqs = self.n_seqs
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

    def _describe(self, k, v, block_table, seq_lens, dtype, weight=None, pos=None, *more):
        """Checks what every cache is made of, and keeps it."""
        _need(k.stride(3) == 1 and v.stride(3) == 1, "k and v: a contiguous head dimension")
        _need(all(_stride(k, d) == _stride(v, d) for d in range(3)), "k and v: equal strides")
        _need(block_table.dtype == torch.int32 and block_table.dim() == 2, "block_table: int32 [sequences][pages]")
        _need(_stride(block_table, 1) in (0, 1), "block_table: contiguous rows")
        n_seqs = block_table.shape[0]
        _need(seq_lens.dtype == torch.int32 and tuple(seq_lens.shape) == (n_seqs,) and _stride(seq_lens, 0) in (0, 1),
              "seq_lens: contiguous int32 [sequences]")
        _need(pos is None or weight is not None, "pos goes with weight")
        tensors = [k, v, block_table, seq_lens] + [t for t in (weight, pos) + more if t is not None]
        _need(all(t.is_cuda and t.device == k.device for t in tensors), "all tensors on one GPU")
        self.k, self.v, self.block_table, self.seq_lens, self.weight, self.pos = k, v, block_table, seq_lens, weight, pos
        self.device, self.n_seqs, self.n_kv_heads, self.head_dim = k.device, n_seqs, k.shape[1], k.shape[3]
        self.page_size, self.dtype = k.shape[2], dtype
        self.capacity = block_table.shape[1] * k.shape[2]
        self._ws, self._sizes, self._kept, self._plans = {}, {}, [], {}

    def _c_struct(self, c):
        k, v, block_table = self.k, self.v, self.block_table
        c.dtype, c.n_kv_heads, c.head_dim = _TYPES[self.dtype], k.shape[1], k.shape[3]
        c.page_size, c.num_pages = k.shape[2], k.shape[0]
        c.page_stride, c.head_stride, c.slot_stride = (_stride(k, d) for d in range(3))
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.n_seqs, c.pages_per_seq, c.table_stride = self.n_seqs, block_table.shape[1], _stride(block_table, 0)
        c.block_table, c.seq_lens = block_table.data_ptr(), self.seq_lens.data_ptr()
        return c

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

    def _plan(self, key, plan):
        """Keeps what the checks of tensors of such shapes and strides came to: most calls' are those of the last."""
        if len(self._plans) >= 256:
            self._plans.clear()
        self._plans[key] = plan
        return plan

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


_CODES = (torch.float8_e4m3fn, torch.uint8)


class PagedKVCache8(PagedKVCache):
    """A paged cache of 8-bit codes (E4M3) made of the caller's tensors: value = code * scale.

    k, v              torch.float8_e4m3fn (or uint8, the same bytes), [pages][kv heads][page slots][head dim] views as in
                      PagedKVCache
    k_scale, v_scale  fp32 [pages][kv heads][blocks], contiguous blocks: the scale of each run of page slots / blocks
                      tokens (1, 2, 4 ... 128) of a head
    dtype             bfloat16 or float16, of the tokens written and read and of queries and outputs
    block_table, seq_lens  as in PagedKVCache

    kv_append chooses the scales: powers of two, which lose no bits of a code.  Weights and positions are not kept, and
    kv_evict does not take it: tokens of one block share a scale and cannot move one by one.

    kv_append and kv_read take bfloat16 of any size.  attend_decode adds up in fp32: the values that it sees have to lie
    below 2^80 in magnitude, and so has the scale of the scores times a head's largest query times a key's scale; scales
    of the caller's own are finite and not negative.
    """

    def __init__(self, k, v, k_scale, v_scale, block_table, seq_lens, dtype=torch.bfloat16):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype, "k and v: equal 4-D tensors")
        _need(k.dtype in _CODES, "k and v: float8_e4m3fn or uint8")
        _need(dtype in (torch.bfloat16, torch.float16), "dtype: bfloat16 or float16")
        self._describe(k, v, block_table, seq_lens, dtype, None, None, k_scale, v_scale)
        shape = k_scale.shape
        _need(k_scale.dtype == v_scale.dtype == torch.float32 and len(shape) == 3 and shape == v_scale.shape
              and tuple(shape[:2]) == tuple(k.shape[:2]) and shape[2] >= 1 and self.page_size % shape[2] == 0,
              "k_scale and v_scale: float32 [pages][kv heads][blocks of a page]")
        _need(_stride(k_scale, 2) in (0, 1) and all(_stride(k_scale, d) == _stride(v_scale, d) for d in range(3)),
              "k_scale and v_scale: equal strides, contiguous blocks")
        self.k_scale, self.v_scale, self.block = k_scale, v_scale, self.page_size // shape[2]
        c = self.c = mw.MoeW4Kv8Cache()
        self._c_struct(c.c)
        c.k_scale, c.v_scale, c.block = k_scale.data_ptr(), v_scale.data_ptr(), self.block
        c.scale_page_stride, c.scale_head_stride = _stride(k_scale, 0), _stride(k_scale, 1)
        self._c8 = self._address = ctypes.addressof(c)
        self.t = self._t = None

    @classmethod
    def allocate(cls, num_pages, page_size, n_kv_heads, head_dim, block_table, seq_lens, dtype=torch.bfloat16,
                 layout="head", block=16):
        """A cache on the block table's GPU, in `layout` as in PagedKVCache.allocate, with a scale for each `block`
        tokens of a head.  Codes and scales start at zero."""
        _need(layout in ("head", "slot"), "layout: 'head' or 'slot'")
        _need(block >= 1 and page_size % block == 0, "block: divides the page size")
        dev = block_table.device
        shape = (num_pages, n_kv_heads, page_size, head_dim)
        if layout == "slot":
            shape = (num_pages, page_size, n_kv_heads, head_dim)
        kv = [torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
        if layout == "slot":
            kv = [t.permute(0, 2, 1, 3) for t in kv]
        scales = [torch.zeros((num_pages, n_kv_heads, page_size // block), dtype=torch.float32, device=dev)
                  for _ in range(2)]
        return cls(*kv, *scales, block_table, seq_lens, dtype)


_pack_qk, _pack_tokens, _pack_attend = (mw.packer(c) for c in (mw.MoeW4QkCall, mw.MoeW4KvTokens, mw.MoeW4AttendCall))


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

    Into a PagedKVCache8 they go as codes with a scale for each block of tokens (moe_w4_kv8_append says how it is
    chosen), and `pos` is not taken.  There the tokens of a block have to be consecutive rows with consecutive indexes:
    sequence after sequence, not step after step.  Otherwise the block's scale is not defined; the kernels do not ask
    (those of the debug build do, and set the status).
    """
    if cache._c8 is not None:
        _need(pos is None, "pos: a cache of 8-bit codes keeps no positions")
        return _tokens_call(mw.moe_w4_kv8_append, "moe_w4_kv8_append", cache, k, v, seq, slot, stream)
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


def _tokens_call(call, where, cache, k, v, seq, slot, stream):
    """A call on tokens k and v at seq and slot of a cache."""
    device, dtype = cache.device, cache.dtype
    key = (k.shape, k.stride(), v.shape, v.stride())
    plan = cache._plans.get(key)
    if plan is None:
        shape, heads, dim = tuple(k.shape), cache.n_kv_heads, cache.head_dim
        if not (len(shape) == 3 and shape[1:] == (heads, dim) and v.shape == shape):
            raise ValueError("k and v: [tokens][kv heads][head dim]")
        strides = _token_stride(k, heads, dim), _token_stride(v, heads, dim)
        if min(strides) < 0:
            raise ValueError("k and v: each token contiguous")
        plan = cache._plan(key, (shape[0], shape[:1]) + strides)
    n, rows, k_stride, v_stride = plan
    if k.dtype is not dtype or v.dtype is not dtype or k.device != device or v.device != device:
        raise ValueError("k and v: of the cache's type on its GPU")
    seq_at = slot_at = 0
    if seq is not None:
        if seq.dtype is not torch.int32 or seq.shape != rows or seq.device != device or (n > 1 and seq.stride(0) != 1):
            _check_index(seq, n, device, "seq")
        seq_at = seq.data_ptr()
    if slot is not None:
        if slot.dtype is not torch.int32 or slot.shape != rows or slot.device != device or (n > 1 and slot.stride(0) != 1):
            _check_index(slot, n, device, "slot")
        slot_at = slot.data_ptr()
    handle = _handle(stream, device)
    ws = cache._ws.get(handle) or cache._workspace(mw.CTRL_BYTES, stream, handle)
    status = call(cache._address, _pack_tokens(n, k.data_ptr(), v.data_ptr(), k_stride, v_stride, seq_at, slot_at, ws[0], ws[1]),
                  handle)
    if status:
        mw._check(status, where)


def kv_read(cache: PagedKVCache, seq=None, slot=None, k_out=None, v_out=None, stream=None):
    """Reads cached tokens' keys and values back, [tokens][kv heads][head dim] each of the cache's type.

    seq, slot     int32 [tokens], as in kv_append
    k_out, v_out  where they go (None: new tensors); each token contiguous
    A token that the cache does not have is zeros.  Returns (k, v).
    """
    if k_out is None or v_out is None:
        if seq is not None and len(seq.shape) != 1:
            raise ValueError("seq: int32 [tokens]")
        shape = (cache.n_seqs if seq is None else seq.shape[0], cache.n_kv_heads, cache.head_dim)
        if k_out is None:
            k_out = _empty(stream, shape, cache.dtype, cache.device)
        if v_out is None:
            v_out = _empty(stream, shape, cache.dtype, cache.device)
    if cache._c8 is None:
        _tokens_call(mw.moe_w4_kv_read, "moe_w4_kv_read", cache, k_out, v_out, seq, slot, stream)
    else:
        _tokens_call(mw.moe_w4_kv8_read, "moe_w4_kv8_read", cache, k_out, v_out, seq, slot, stream)
    return k_out, v_out


def attend_decode(cache: PagedKVCache, q, scale: Optional[float] = None, max_len: Optional[int] = None, out=None,
                  return_lse=False, weight_out=None, stream=None, window: Optional[int] = None, sink: int = 0):
    """Attention of one new token per sequence, q [sequences][query heads][head dim], over its cached tokens.

    scale       of the scores (default 1/sqrt(head dim))
    max_len     upper bound of seq_lens (default: what the block table, and the weights if they are added up, can
                hold); a small one saves work
    return_lse  also return the log sum of the exponentials, fp32 [sequences][query heads]
    weight_out  fp32 tensor like cache.weight (it may be cache.weight itself): gets cache.weight plus the
                probability that each token drew, summed over the kv head's query heads
    window      see only the last `window` tokens of a sequence, the new one among them, and its first `sink` (None:
                all); tokens that are not seen are not read, their pages may be gone.  Not with weight_out
    Returns out, or (out, lse).
    """
    if window is not None or cache._c8 is not None:
        return _attend_more(cache, q, scale, max_len, out, return_lse, weight_out, stream, window, sink)
    _need(not sink, "sink goes with a window")
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


def _attend_more(cache, q, scale, max_len, out, return_lse, weight_out, stream, window, sink):
    """attend_decode over 8-bit codes, or with a window."""
    device, dtype = cache.device, cache.dtype
    shape = q.shape
    key = (shape, q.stride())
    plan = cache._plans.get(key)
    if plan is None:
        if not (len(shape) == 3 and shape[0] == cache.n_seqs and shape[2] == cache.head_dim):
            raise ValueError("q: [sequences][query heads][head dim]")
        heads, dim = shape[1], shape[2]
        q_stride = _token_stride(q, heads, dim)
        if q_stride < 0:
            raise ValueError("q: contiguous heads")
        if cache._c8 is None:
            size = mw.moe_w4_attend_workspace_size(cache._c, heads, 0, 0)
        else:
            size = mw.moe_w4_kv8_attend_workspace_size(cache._address, heads, 0)
        plan = cache._plan(key, (heads, q_stride, heads * dim, tuple(shape[:2]), max(size, mw.CTRL_BYTES), dim ** -0.5))
    heads, q_stride, out_stride, rows, size, default_scale = plan
    if q.dtype is not dtype or q.device != device:
        raise ValueError("q: of the cache's type on its GPU")
    _need(weight_out is None, "weights are not added up with a window, nor over 8-bit codes")
    if out is None:
        out = _empty(stream, shape, dtype, device)
    else:
        if not _like(out, dtype, shape, device):
            raise ValueError("out: like q")
        out_stride = _token_stride(out, heads, shape[2])
        if out_stride < 0:
            raise ValueError("out: contiguous heads")
    lse, lse_at = None, 0
    if return_lse:
        lse = _empty(stream, rows, torch.float32, device)
        lse_at = lse.data_ptr()
    max_len = cache.capacity if max_len is None else int(max_len)
    if window is None:
        window = 0
        _need(not sink, "sink goes with a window")
    elif not (1 <= window < _INT and 0 <= sink < _INT):
        raise ValueError("window: 1 or more, sink: 0 or more, 32-bit integers")
    if not -_INT <= max_len < _INT:
        raise ValueError("max_len: a 32-bit integer")
    handle = _handle(stream, device)
    ws = cache._ws.get(handle)
    if ws is None or ws[1] < size:
        ws = cache._workspace(size, stream, handle)
    args = _pack_attend(heads, max_len, int(window), int(sink), default_scale if scale is None else scale, q.data_ptr(),
                        out.data_ptr(), q_stride, out_stride, lse_at, ws[0], ws[1])
    if cache._c8 is None:
        status = mw.moe_w4_attend_window(cache._address, args, handle)
    else:
        status = mw.moe_w4_kv8_attend(cache._address, args, handle)
    if status:
        mw._check(status, "moe_w4_attend_window" if cache._c8 is None else "moe_w4_kv8_attend")
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


# 2^256 / (2 pi), from 76 digits: frequencies in turns are exact to 64 bits and more.
_TURNS = (1591549430918953357688837633725143620344596457404564487476673440588967976342 << 256) // 10 ** 76


def _turns(f):
    """A frequency in radians as turns, mod 1, in 64 bits, rounded once."""
    num, den = f.as_integer_ratio()            # den is a power of two
    shift = 256 - 64 + den.bit_length() - 1
    return (num * _TURNS + (1 << shift - 1) >> shift) % 2 ** 64


class Rope:
    """How the heads of a model turn with a token's position: what qk_norm_rope goes by, made once.

    inv_freq     the angle per position of each pair of dimensions, in radians: numbers or a tensor, a multiple of 8
                 of them; the first 2 * len(inv_freq) dimensions of a head turn
    axis         which row of the positions each pair turns with, 0..7 (None: there is one)
    interleaved  pair i is dimensions 2 i and 2 i + 1 (else i and len(inv_freq) + i)
    scale        of cosine and sine (models with stretched positions have one)
    """

    def __init__(self, inv_freq, axis=None, interleaved=False, scale=1.0, device=None):
        freqs = [float(f) for f in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
        _need(freqs and len(freqs) % 8 == 0, "inv_freq: a multiple of 8 pairs")
        _need(all(abs(f) < float("inf") for f in freqs), "inv_freq: finite numbers")   # NaN is not below
        turns = [_turns(f) for f in freqs]
        if axis is not None:
            axis = [int(x) for x in (axis.tolist() if hasattr(axis, "tolist") else axis)]
            _need(len(axis) == len(freqs) and all(0 <= x < 8 for x in axis), "axis: one of 0..7 for each pair")
        device = torch.device("cuda", _current_device()) if device is None else torch.device(device)
        # the bits of unsigned numbers, as int64 holds them
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        self.axis = None if axis is None else torch.tensor(axis, dtype=torch.int32, device=device)
        self.pairs, self.axes, self.device = len(freqs), max(axis) + 1 if axis else 1, self.turns.device
        c = self.c = mw.MoeW4Rope()
        c.turns, c.axis, c.pairs, c.axes = self.turns.data_ptr(), mw._ptr(self.axis), self.pairs, self.axes
        c.interleaved, c.scale = int(bool(interleaved)), float(scale)
        self._address, self._plans = ctypes.addressof(c), {}

    @classmethod
    def from_base(cls, rot_dim, base=10000.0, sections=None, interleaved=False, scale=1.0, device=None):
        """Frequencies base ** (-2 i / rot_dim) of rot_dim / 2 pairs.  sections: how many pairs turn with each row of the
        positions, one after the other, as (time, height, width)."""
        axis = None if sections is None else [a for a, n in enumerate(sections) for _ in range(n)]
        return cls([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], axis, interleaved, scale, device)


def qk_norm_rope(q, k, positions, rope: Optional[Rope], q_weight=None, k_weight=None, eps: float = 1e-6,
                 unit_offset=False, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q and k, then the rotation of its first dimensions by the token's position, in one pass:
    fp32 throughout, rounded once.

    q, k          bf16 or fp16 [tokens][heads][head dim] views (of one projection's output, say); k may be None
    positions     int32 [tokens], or [rows][tokens] for a rope with several axes; None without a rope
    rope          None: no rotation
    q_weight, k_weight  [head dim] of q's type, multiplied in after the norm (plus 1 with unit_offset); None: no norm
    q_out, k_out  where results go: new tensors (None), or q and k themselves
    Returns (q, k).
    """
    shape, dtype, device = q.shape, q.dtype, q.device
    plans = _no_rope if rope is None else rope._plans
    key = (shape, q.stride(), dtype, None if k is None else (k.shape, k.stride()),
           None if positions is None else (positions.shape, positions.stride()))
    plan = plans.get(key)
    if plan is None:
        if len(plans) >= 256:
            plans.clear()
        plan = plans[key] = _rope_plan(q, k, positions, rope)
    n, dim, kind, heads, k_heads, q_stride, k_stride, pos_stride, width = plan
    if device.type != "cuda" or (k is not None and (k.dtype is not dtype or k.device != device)):
        raise ValueError("q and k: of one type on one GPU")
    at = k_at = ko_at = ko_stride = qw_at = kw_at = pos_at = 0
    if q_weight is not None:
        if q_weight.dtype is not dtype or q_weight.shape != width or q_weight.device != device or q_weight.stride(0) != 1:
            raise ValueError("q_weight: contiguous [head dim] of q's type")
        qw_at = q_weight.data_ptr()
    if k_weight is not None:
        if k_weight.dtype is not dtype or k_weight.shape != width or k_weight.device != device or k_weight.stride(0) != 1:
            raise ValueError("k_weight: contiguous [head dim] of q's type")
        kw_at = k_weight.data_ptr()
    if rope is not None:
        if positions.dtype is not torch.int32 or positions.device != device or rope.device != device:
            raise ValueError("positions: int32 on q's GPU, as the rope")
        at, pos_at = rope._address, positions.data_ptr()
    if q_out is None:
        q_out, qo_stride = _empty(stream, shape, dtype, device), heads * dim
    else:
        qo_stride = _place(q_out, shape, dtype, device, "q_out")
    if k is None:
        _need(k_out is None, "k_out goes with k")
    else:
        if k_out is None:
            k_out, ko_stride = _empty(stream, k.shape, dtype, device), k_heads * dim
        else:
            ko_stride = _place(k_out, k.shape, dtype, device, "k_out")
        k_at, ko_at = k.data_ptr(), k_out.data_ptr()
    status = mw.moe_w4_qk_norm_rope(
        _pack_qk(kind, n, dim, heads, k_heads, 1 if unit_offset else 0, eps, q.data_ptr(), q_out.data_ptr(), k_at, ko_at,
                 q_stride, qo_stride, k_stride, ko_stride, qw_at, kw_at, at, pos_at, pos_stride), _handle(stream, device))
    if status:
        mw._check(status, "moe_w4_qk_norm_rope")
    return q_out, k_out


_no_rope = {}


def _rope_plan(q, k, positions, rope):
    """What tensors of such shapes and strides come to: tokens, head dim, type, heads of q and k, strides, a head's shape."""
    shape = q.shape
    if len(shape) != 3 or q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q: a 3-D bfloat16 or float16 tensor")
    n, heads, dim = shape
    k_heads = k_stride = pos_stride = 0
    q_stride = _token_stride(q, heads, dim)
    if k is not None:
        if not (len(k.shape) == 3 and k.shape[0] == n and k.shape[2] == dim):
            raise ValueError("k: [tokens][heads][head dim], like q")
        k_heads = k.shape[1]
        k_stride = _token_stride(k, k_heads, dim)
    if q_stride < 0 or k_stride < 0:
        raise ValueError("q and k: each token contiguous")
    if rope is None:
        _need(positions is None, "positions go with a rope")
    else:
        _need(positions is not None, "a rope goes with positions")
        rows = tuple(positions.shape)
        if rows != (rope.axes, n) and not (rope.axes == 1 and rows == (n,)):
            raise ValueError("positions: [tokens], or [%d][tokens]" % rope.axes)
        _need(n <= 1 or positions.stride(-1) == 1, "positions: contiguous rows")
        pos_stride = _stride(positions, 0) if len(rows) == 2 else 0
    return n, dim, _TYPES[q.dtype], heads, k_heads, q_stride, k_stride, pos_stride, (dim,)


def _place(t, shape, dtype, device, what):
    """Elements between the tokens of an output that is given."""
    if not _like(t, dtype, shape, device):
        raise ValueError(what + ": like " + what[0])
    stride = _token_stride(t, shape[1], shape[2])
    if stride < 0:
        raise ValueError(what + ": each token contiguous")
    return stride


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
