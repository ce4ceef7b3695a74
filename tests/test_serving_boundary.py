"""Host-side checks of the C ABI in moe_w4_serving.h: exports, sizes and refusals, before any device work."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 12          # an aligned address that no refused call touches
BIG = 1 << 40


@pytest.fixture(scope="module")
def mw():
    from bit_quantized_sparse_gb300 import _build
    if not os.path.exists(_build.LIB):
        _build.build()
    from bit_quantized_sparse_gb300 import moe_w4
    return moe_w4


def cache(mw, **kw):
    c = mw.MoeW4KvCache()
    d = dict(dtype=mw.MOE_W4_TYPE_BF16, n_kv_heads=2, head_dim=128, page_size=16, num_pages=8, page_stride=4096,
             head_stride=2048, slot_stride=128, k=A, v=A, n_seqs=3, pages_per_seq=4, table_stride=4, block_table=A,
             seq_lens=A)
    for k, v in {**d, **kw}.items():
        setattr(c, k, v)
    return c


def track(mw, **kw):
    t = mw.MoeW4KvTrack()
    for k, v in {**dict(weight=A, pos=A, seq_stride=128, head_stride=64, slots=64), **kw}.items():
        setattr(t, k, v)
    return t


def append(mw, c, t=None, n=3, k=A, ks=256, v=A, vs=256, seq=A, slot=A, pos=None, ws=A, nws=256):
    return mw.moe_w4_kv_append(c and ctypes.byref(c), t and ctypes.byref(t), n, k, ks, v, vs, seq, slot, pos, ws, nws, None)


def attend(mw, c, heads=4, q=A, qs=512, max_len=64, out=A, os_=512, lse=None, t=None, w=None, ws=A, nws=BIG):
    return mw.moe_w4_attend_decode(c and ctypes.byref(c), heads, q, qs, 1.0, max_len, out, os_, lse,
                                   t and ctypes.byref(t), w, ws, nws, None)


def evict(mw, c, t, seen=A, budget=32, sink=1, recent=1, max_len=64, lens=A, w=A, p=A, ws=A, nws=BIG):
    return mw.moe_w4_kv_evict(c and ctypes.byref(c), t and ctypes.byref(t), seen, budget, sink, recent, max_len, lens, w,
                              p, ws, nws, None)


def logprobs(mw, dtype=2, n=2, vocab=100, x=A, rs=100, t=A, top=3, lp=A, e=A, ti=A, tl=A, ws=A, nws=256):
    return mw.moe_w4_token_logprobs(dtype, n, vocab, x, rs, t, top, lp, e, ti, tl, ws, nws, None)


def test_every_declared_symbol_is_exported(mw):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_w4_serving.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_w4_[a-z_]+)\s*\(", text))
    assert len(names) == 6 and names <= set(mw.EXPORTED)
    lib = ctypes.CDLL(mw.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


BAD_CACHES = [("dtype", 2, -2), ("dtype", -1, -2), ("head_dim", 96, -2), ("head_dim", 0, -2), ("n_kv_heads", 0, -1),
              ("n_kv_heads", 1025, -2), ("page_size", 0, -1), ("num_pages", 0, -1), ("pages_per_seq", 0, -1),
              ("n_seqs", -1, -1), ("n_seqs", 4097, -2), ("page_size", 1 << 29, -2), ("page_stride", 4, -6),
              ("head_stride", 4, -6), ("slot_stride", 4, -6), ("page_stride", -8, -1), ("k", None, -1), ("v", None, -1),
              ("k", A + 8, -6), ("v", A + 2, -6), ("block_table", None, -1), ("block_table", A + 2, -6),
              ("table_stride", -1, -1)]


@pytest.mark.parametrize("field,value,code", BAD_CACHES)
def test_bad_caches_are_refused(mw, field, value, code):
    c = cache(mw, **{field: value})
    t = track(mw)
    assert append(mw, c) == code
    assert evict(mw, c, t) == code
    assert attend(mw, c, heads=4 if field != "n_kv_heads" else 1025 * 4) == code


def test_lengths_are_needed_where_they_are_read(mw):
    c = cache(mw, seq_lens=None)
    assert append(mw, c, slot=None) == mw.MOE_W4_ERR_INVALID
    assert attend(mw, c) == mw.MOE_W4_ERR_INVALID
    assert evict(mw, c, track(mw)) == mw.MOE_W4_ERR_INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(ks=-8), -1), (dict(ks=12), -6), (dict(vs=4), -6),
    (dict(k=A + 4), -6), (dict(v=A + 8), -6), (dict(seq=A + 2), -6), (dict(slot=A + 1), -6), (dict(pos=A + 2), -6),
    (dict(seq=None, n=2), -1), (dict(ws=None), -3), (dict(nws=255), -3), (dict(ws=A + 16), -3), (dict(n=0, k=None), 0)])
def test_append_refusals(mw, kw, code):
    assert append(mw, cache(mw), **kw) == code
    assert append(mw, None) == mw.MOE_W4_ERR_INVALID
    assert append(mw, cache(mw, n_seqs=0), n=0) == 0


def test_append_refuses_bad_tracks(mw):
    for kw, code in ((dict(weight=None), -1), (dict(slots=-1), -1), (dict(seq_stride=-1), -1), (dict(weight=A + 2), -6),
                     (dict(pos=A + 3), -6)):
        assert append(mw, cache(mw), track(mw, **kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), -1), (dict(heads=3), -1), (dict(heads=258), -2), (dict(q=None), -1), (dict(out=None), -1),
    (dict(max_len=-1), -1), (dict(max_len=65), -1), (dict(qs=-8), -1), (dict(os_=504), -1), (dict(qs=516), -6),
    (dict(os_=516), -6), (dict(q=A + 8), -6), (dict(out=A + 2), -6), (dict(lse=A + 2), -6), (dict(w=A), -1),
    (dict(ws=None), -3), (dict(ws=A + 128), -3), (dict(nws=1024), -3)])
def test_attend_refusals(mw, kw, code):
    assert attend(mw, cache(mw), **kw) == code
    assert attend(mw, None) == mw.MOE_W4_ERR_INVALID


def test_attend_refuses_bad_tracks(mw):
    c = cache(mw)
    assert attend(mw, c, t=track(mw)) == mw.MOE_W4_ERR_INVALID                    # no weight_out
    assert attend(mw, c, t=track(mw, slots=63), w=A) == mw.MOE_W4_ERR_INVALID     # fewer slots than max_len
    assert attend(mw, c, t=track(mw, weight=None), w=A) == mw.MOE_W4_ERR_INVALID
    assert attend(mw, c, t=track(mw), w=A + 2) == mw.MOE_W4_ERR_ALIGN


@pytest.mark.parametrize("kw,code", [
    (dict(t=None), -1), (dict(budget=0), -1), (dict(sink=-1), -1), (dict(recent=-1), -1), (dict(sink=20, recent=13), -1),
    (dict(max_len=-1), -1), (dict(max_len=65), -1), (dict(seen=None), -1), (dict(lens=None), -1), (dict(w=None), -1),
    (dict(p=None), -1), (dict(seen=A + 2), -6), (dict(lens=A + 2), -6), (dict(w=A + 1), -6), (dict(p=A + 2), -6),
    (dict(ws=None), -3), (dict(nws=512), -3), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), -1)])
def test_evict_refusals(mw, kw, code):
    assert evict(mw, cache(mw), **{"t": track(mw), **kw}) == code
    assert evict(mw, None, track(mw)) == mw.MOE_W4_ERR_INVALID


def test_evict_refuses_bad_tracks(mw):
    for kw in (dict(pos=None), dict(slots=63)):
        assert evict(mw, cache(mw), track(mw, **kw)) == mw.MOE_W4_ERR_INVALID
    assert evict(mw, cache(mw, n_seqs=4096, n_kv_heads=64), track(mw)) == mw.MOE_W4_ERR_UNSUPPORTED   # 262144 rows


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(vocab=0), -1), (dict(rs=-1), -1), (dict(rs=99), -1), (dict(top=-1), -1), (dict(top=101), -1),
    (dict(top=33), -2), (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(vocab=(1 << 20) + 1, rs=1 << 21), -2),
    (dict(x=None), -1), (dict(t=None), -1), (dict(lp=None), -1), (dict(ti=None), -1), (dict(tl=None), -1),
    (dict(x=A + 2), -6), (dict(x=A + 1, dtype=0), -6), (dict(t=A + 2), -6), (dict(e=A + 2), -6), (dict(ti=A + 2), -6),
    (dict(ws=None), -3), (dict(nws=255), -3), (dict(ws=A + 64), -3), (dict(n=0, x=None), 0)])
def test_logprobs_refusals(mw, kw, code):
    assert logprobs(mw, **kw) == code


def test_workspace_sizes(mw):
    c = cache(mw)
    p = ctypes.byref(c)
    sizes = [mw.moe_w4_attend_workspace_size(p, 4, n, 1) for n in (0, 1, 16, 17, 64)]
    assert sizes[0] >= 256 and all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert mw.moe_w4_attend_workspace_size(p, 4, 64, 0) <= sizes[-1]
    assert sizes[-1] - mw.moe_w4_attend_workspace_size(p, 4, 64, 0) >= 3 * 4 * 64 * 4   # a score per head and token
    assert mw.moe_w4_attend_workspace_size(p, 3, 64, 0) == 0 and mw.moe_w4_attend_workspace_size(None, 4, 64, 0) == 0
    assert mw.moe_w4_evict_workspace_size(p, 32, 64) >= 3 * 2 * 32 * 4
    assert mw.moe_w4_evict_workspace_size(p, 0, 64) == 0 and mw.moe_w4_evict_workspace_size(None, 1, 64) == 0
    # a budget past the longest sequence needs no more than that sequence
    assert mw.moe_w4_evict_workspace_size(p, 1 << 30, 64) == mw.moe_w4_evict_workspace_size(p, 64, 64)


def test_serving_module_checks_tensors(mw):
    torch = pytest.importorskip("torch")
    from bit_quantized_sparse_gb300 import serving as sv
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(k=k.float(), v=k.float()), dict(v=k[:, :, :, ::2]), dict(block_table=table.long()),
                dict(seq_lens=lens.repeat(2)), dict(pos=torch.zeros(1, 2, 64, dtype=torch.int32)), {}):   # {}: not on a GPU
        with pytest.raises(ValueError):
            sv.PagedKVCache(**{**dict(k=k, v=k, block_table=table, seq_lens=lens), **bad})
    with pytest.raises(ValueError):
        sv.token_logprobs(torch.zeros(2, 8))
