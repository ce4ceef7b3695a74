"""Calls of the operators for long contexts at the ends of what their arguments allow, on a GPU."""
import pytest

from .test_longctx_gpu import sv, torch   # noqa: F401  (fixtures)

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
