"""Calls of the serving operators that were once answered wrongly, against the float64 oracle."""
import numpy as np
import pytest

from oracle import serving_oracle as SO
from tests.test_serving_gpu import Setup, check_evict, check_logprobs, f64, sv, torch  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


# ---- eviction: rows that are not cut, in calls whose moves are a kernel of their own ----
@pytest.mark.parametrize("dim,kv_heads", [(64, 1), (128, 3), (256, 2)])
@pytest.mark.parametrize("lens", [[2500, 100, 900, 0], [9000, 300]])
def test_evict_again_moves_nothing(torch, sv, dim, kv_heads, lens):
    """A second call finds every sequence within the budget: keys, values, weights and positions stay."""
    s = Setup(torch, sv, lens, kv_heads, dim, 16, seed=31, track=True)
    seen = s.lens + 7
    check_evict(torch, sv, s, seen, 300, 2, 5, True)
    assert s.lens.tolist() == [min(n, 300) for n in lens]
    before = [f64(t) for t in (s.k, s.v, s.weight, s.pos, s.lens)]
    for _ in range(2):
        sv.kv_evict(s.cache, seen, 300, 2, 5)
    for x, y in zip(before, (s.k, s.v, s.weight, s.pos, s.lens)):
        assert np.array_equal(x, f64(y), equal_nan=True)
    assert s.cache.status() == 0


def test_evict_of_other_sequences_than_before(torch, sv):
    """The rows that are cut change from call to call."""
    s = Setup(torch, sv, [700, 1500, 200, 1400], 2, 64, 16, seed=32, track=True)
    for lens in ([700, 1500, 200, 1400], [1, 280, 200, 1300], [699, 0, 200, 277], [250, 1400, 199, 3]):
        s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        check_evict(torch, sv, s, s.lens + 9, 280, 3, 20, False)


@pytest.mark.parametrize("track", [False, True])
def test_evict_after_attention_in_the_same_workspace(torch, sv, track):
    """The attention's partial results and scores lie where an eviction keeps its lists."""
    s = Setup(torch, sv, [9000, 20, 5000, 300], 2, 64, 16, seed=33, track=True)
    q = s.randn(4, 16, 64).to(s.dt)
    sv.attend_decode(s.cache, q, weight_out=torch.empty_like(s.weight) if track else None)
    assert len(s.cache._ws) == 1
    check_evict(torch, sv, s, s.lens + 9, 301, 3, 20, True)
    assert len(s.cache._kept) == 1   # one workspace served both
    sv.attend_decode(s.cache, q, weight_out=torch.empty_like(s.weight) if track else None)
    check_evict(torch, sv, s, s.lens + 9, 301, 3, 20, True)


# ---- log probabilities: clusters with the least to do before their parts meet ----
@pytest.mark.parametrize("dtype,vector", [("float32", 4), ("bfloat16", 8), ("float16", 8)])
@pytest.mark.parametrize("rows,ctas", [(1, 2), (1, 8), (7, 4), (57, 4), (57, 8), (114, 4), (228, 2)])
@pytest.mark.parametrize("top", [0, 20])
def test_logprobs_smallest_parts(torch, sv, dtype, vector, rows, ctas, top):
    """A vector a thread: the CTAs of a row start and finish almost together.  The same bytes every time."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + ctas)
    x = (torch.randn(rows, 256 * ctas * vector, device="cuda", generator=g) * 3).to(getattr(torch, dtype))
    t = torch.randint(0, x.shape[1], (rows,), device="cuda", generator=g).to(torch.int32)
    check_logprobs(torch, sv, x, t, top)
    first = sv.token_logprobs(x, t, top)
    for _ in range(50):
        for a, b in zip(first, sv.token_logprobs(x, t, top)):
            assert a is b is None or torch.equal(a, b)
