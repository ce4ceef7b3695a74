"""Calls of the operators for long contexts at the ends of what their arguments allow, on a GPU."""
import ctypes

import pytest

from .test_debug_build import _debug_lib
from .test_longctx_gpu import Setup8, ragged, sv, torch   # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", [False, True])
def test_read_from_a_cache_of_no_sequences(torch, sv, codes):
    """Rows are zeros and the status says so, as for any token that a cache does not have."""
    table, lens = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    cache = (sv.PagedKVCache8 if codes else sv.PagedKVCache).allocate(4, 16, 2, 64, table, lens)
    rows = torch.arange(5, dtype=torch.int32, device="cuda")
    out = torch.full((5, 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = sv.kv_read(cache, rows, rows, k_out=out[:, 0], v_out=out[:, 1])
    assert (out == 0).all() and cache.status() == 2
    cache.reset()
    assert sv.kv_read(cache)[0].shape == (0, 2, 64) and cache.status() == 0


@pytest.fixture(scope="module")
def debug_append(torch, sv):
    """kv_append of the debug build into a cache of codes; returns the status word it leaves."""
    mw = sv.mw
    lib = ctypes.CDLL(_debug_lib())
    f = lib.moe_w4_kv8_append
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_void_p] * 3
    stream = torch.cuda.current_stream().cuda_stream

    def append(cache, k, v, seq, slot):
        ws = torch.zeros(mw.CTRL_BYTES, dtype=torch.uint8, device="cuda")
        t = mw.MoeW4KvTokens(k.shape[0], k.data_ptr(), v.data_ptr(), k.stride(0), v.stride(0), seq.data_ptr(), slot.data_ptr(),
                             ws.data_ptr(), mw.CTRL_BYTES)
        assert f(cache._address, ctypes.addressof(t), stream) == 0
        torch.cuda.synchronize()
        at = mw.moe_w4_status_offset()
        return int(ws[at:at + 4].view(torch.int32).item())
    return append


@pytest.mark.parametrize("page,block", [(1, 1), (16, 2), (16, 16), (64, 32), (128, 128)])
def test_debug_build_refuses_rows_in_a_wrong_order(torch, sv, debug_append, page, block):
    """Sequence after sequence is taken, with the product's bytes; a block's rows apart, out of order, or one twice are
    refused, and nothing is written."""
    starts, counts = [5, 0, 130], [70, 40, 33]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    seq, slot = ragged(starts, counts)
    rows = list(zip(seq, slot))
    kv = torch.randn((len(rows) + 1, 2, 2, 64), device="cuda").to(torch.bfloat16)

    def caches():
        for _ in range(2):
            yield Setup8(torch, sv, starts, 2, 64, page, block, seed=page, room=80)
    product, debug = caches()
    n = len(rows)
    sv.kv_append(product.cache, kv[:n, 0], kv[:n, 1], seq=ints(seq), slot=ints(slot))
    assert product.cache.status() == 0
    assert debug_append(debug.cache, kv[:n, 0], kv[:n, 1], ints(seq), ints(slot)) == 0
    assert torch.equal(product.k, debug.k) and torch.equal(product.v, debug.v)
    for x, y in zip(product.scales, debug.scales):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
    by_step = sorted(rows, key=lambda r: (r[1] - starts[r[0]], r[0]))
    swapped = [rows[1], rows[0]] + rows[2:]
    bad = [rows + [rows[3]], rows[:9] + [rows[2]] + rows[9:]]
    if block > 1:
        bad += [by_step, swapped]
    before = [x.clone() for x in (debug.k, debug.v, *debug.scales)]
    for order in bad:
        m = len(order)
        assert debug_append(debug.cache, kv[:m, 0], kv[:m, 1], ints([b for b, _ in order]), ints([t for _, t in order])) == 2
        for x, y in zip(before, (debug.k, debug.v, *debug.scales)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
