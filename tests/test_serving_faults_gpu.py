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


# ---- attention: tokens on pages outside the cache take no part ----
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim,kv_heads,group", [(64, 1, 4), (64, 2, 16), (64, 1, 24), (128, 2, 8), (128, 1, 12), (128, 1, 20),
                                                (256, 2, 8), (256, 1, 16)])
@pytest.mark.parametrize("page", [1, 7, 8, 16, 64])
def test_attention_leaves_bad_pages_out(torch, sv, dtype, dim, kv_heads, group, page):
    """Scores far below 0, where a token that scores 0 would take everything; a sequence without any page left."""
    lens = [100, 60, 1500, 0, 90, 33]
    s = Setup(torch, sv, lens, kv_heads, dim, page, "slot", dtype, seed=page, track=True)
    s.k.abs_()
    q = -s.randn(len(lens), kv_heads * group, dim).abs().to(s.dt)
    there = [torch.ones(n, dtype=torch.bool) for n in lens]
    for b, p, value in [(0, 1, s.k.shape[0]), (2, 0, -1), (2, 900 // page, 2 ** 31 - 1), (2, 901 // page, -2 ** 31),
                        (4, 89 // page, -7)] + [(5, p, -1) for p in range(-(-33 // page))]:
        s.table[b, p] = value
        there[b][p * page:(p + 1) * page] = False
    before = s.weight.clone()
    drawn = torch.full_like(s.weight, float("nan"))
    out, lse = sv.attend_decode(s.cache, q, scale=0.3, return_lse=True, max_len=1500, weight_out=drawn)
    assert s.cache.status() == 2
    u, bf = torch.finfo(s.dt).eps / 2, dtype == "bfloat16"
    pool_k, pool_v, table = f64(s.k), f64(s.v), s.table.cpu().numpy()
    for b, n in enumerate(lens):
        left = np.nonzero(there[b].numpy())[0]
        m = len(left)
        # the tokens left, a page each
        at = table[b, left // page], slice(None), left % page
        one = [x[at][:, :, None, :] if m else np.zeros((1, kv_heads, 1, dim)) for x in (pool_k, pool_v)]
        want = SO.attend(f64(q[b:b + 1]), *one, np.arange(max(m, 1))[None], [m], 0.3)
        for h, w in enumerate(want):
            mine = slice(h * group, (h + 1) * group)
            delta = (dim / 16 + 16 + 4) * 2.0 ** -24 * w["absqk"]
            rel = 2 * delta + 2.0 ** -20 + (2.0 ** -17 if bf else 2.0 ** -21) + (n / 64 + 64) * 2.0 ** -24
            tol = rel * w["absv"] + u * np.abs(w["out"]) + (0 if bf else 2.0 ** -38 * w["vsum"] / w["floor"]) + 2.0 ** -25
            assert np.all(np.abs(f64(out[b, mine]) - w["out"]) <= tol), (b, h)
            if m == 0:
                assert np.all(np.isneginf(f64(lse[b, mine])))
            else:
                assert np.all(np.abs(f64(lse[b, mine]) - w["lse"]) <= delta + 2.0 ** -20 + (n / 64 + 64) * 2.0 ** -24
                              + 8 * 2.0 ** -24 * (np.abs(w["lse"]) + w["absqk"]))
            more = f64(drawn[b, h, :n]) - f64(before[b, h, :n])
            assert np.all(more[~there[b].numpy()] == 0)
            assert np.all(np.abs(more[left] - w["drawn"]) <= (2 * delta + 2.0 ** -19 + 8 * 2.0 ** -24 * (w["absqk"] + np.abs(w["lse"]).max(initial=0, where=np.isfinite(w["lse"])))
                          + (n / 64 + 64) * 2.0 ** -24) * w["drawn"]
                          + (group + 4) * 2.0 ** -24 * (f64(before[b, h, left]) + w["drawn"]))


# ---- eviction: a move from or to a page outside the cache is left out as a whole ----
@pytest.mark.parametrize("lens,budget", [([400, 300, 90], 280), ([2000, 900, 90], 300)])   # moves by the selecting CTAs, and by a kernel
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_leaves_bad_pages_out(torch, sv, lens, budget, in_place):
    s = Setup(torch, sv, lens, 2, 64, 16, seed=41, track=True)
    for b, page, value in ((0, 0, -1), (0, 5, s.k.shape[0]), (0, budget // 16 + 2, 2 ** 31 - 1), (1, 3, -2 ** 31)):
        s.table[b, page] = value
    seen = s.lens + 5
    k, v, w, p = f64(s.k), f64(s.v), f64(s.weight), s.pos.cpu().numpy().copy()
    table, pages = s.table.cpu().numpy(), s.k.shape[0]
    left_out = 0
    for b, n in enumerate(lens):
        for h in range(2) if n > budget else ():
            kept = SO.kept_tokens(w[b, h, :n], p[b, h, :n], int(seen[b]), budget, 1, 9)
            holes = sorted(set(range(budget)) - set(kept))
            for to, frm in zip(holes, [j for j in kept if j >= budget]):
                if not all(0 <= table[b, j // 16] < pages for j in (to, frm)):
                    left_out += 1
                    continue
                for pool in (k, v):
                    pool[table[b, to // 16], h, to % 16] = pool[table[b, frm // 16], h, frm % 16]
                w[b, h, to], p[b, h, to] = w[b, h, frm], p[b, h, frm]
    assert left_out
    outs = {} if in_place else dict(lens_out=torch.zeros_like(s.lens), weight_out=torch.zeros_like(s.weight),
                                    pos_out=torch.zeros_like(s.pos))
    sv.kv_evict(s.cache, seen, budget, 1, 9, **outs)
    assert s.cache.status() == 2
    assert np.array_equal(f64(s.k), k, equal_nan=True) and np.array_equal(f64(s.v), v, equal_nan=True)
    got_w, got_p = f64(outs.get("weight_out", s.weight)), outs.get("pos_out", s.pos).cpu().numpy()
    for b, n in enumerate(lens):
        m = min(n, budget)
        assert np.array_equal(got_w[b, :, :m], w[b, :, :m]) and np.array_equal(got_p[b, :, :m], p[b, :, :m])
    assert outs.get("lens_out", s.lens).tolist() == [min(n, budget) for n in lens]


# ---- graphs: a stream's first call cannot be a captured one ----
def test_first_call_in_a_capture_is_refused(torch, sv):
    s = Setup(torch, sv, [100, 60], 2, 64, 16, seed=42, track=True)
    q = s.randn(2, 8, 64).to(s.dt)
    good = sv.attend_decode(s.cache, q)
    x = torch.randn(3, 1000, device="cuda")
    rows = sv.token_logprobs(x, top=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    known = len(sv._ctrl)
    new, seen = s.randn(2, 2, 64).to(s.dt), s.lens.clone()
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
        first = torch.zeros(1, device="cuda")   # something to capture
        for call in (lambda: sv.attend_decode(s.cache, q), lambda: sv.kv_append(s.cache, new, new),
                     lambda: sv.kv_evict(s.cache, seen, 50), lambda: sv.token_logprobs(x, top=4)):
            with pytest.raises(RuntimeError, match="captur"):
                call()
    del first
    assert len(s.cache._ws) == 1 and len(sv._ctrl) == known
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    out = torch.empty_like(q)
    with torch.cuda.stream(side):
        sv.attend_decode(s.cache, q)
        sv.token_logprobs(x, top=4)
        side.synchronize()
        for graph in graphs:                     # the second before the first has run
            with torch.cuda.graph(graph, stream=side):
                sv.attend_decode(s.cache, q, out=out)
                got = sv.token_logprobs(x, top=4)
    for graph in graphs[::-1]:
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, good)
    assert torch.equal(got.top_index, rows.top_index) and s.cache.status() == 0


# ---- status: cleared from Python ----
def test_cache_reset_clears_the_status(torch, sv):
    """After bad indexes, and after a wait that ran out (2 s), the cache is as new; its workspaces stay for graphs."""
    from bit_quantized_sparse_gb300 import moe_w4 as mw
    s = Setup(torch, sv, [4000, 70], 1, 64, 16, seed=43, track=True)
    q = s.randn(2, 4, 64).to(s.dt)
    good = sv.attend_decode(s.cache, q)
    page = int(s.table[1, 0])
    s.table[1, 0] = -1
    sv.attend_decode(s.cache, q)
    assert s.cache.status() == 2
    s.cache.reset()
    s.table[1, 0] = page
    assert s.cache.status() == 0 and torch.equal(sv.attend_decode(s.cache, q), good) and s.cache.status() == 0
    (ptr, size, _), = s.cache._ws.values()
    assert mw.moe_w4_test_skip_publish(ptr, size, 1, torch.cuda.current_stream().cuda_stream) == 0
    sv.attend_decode(s.cache, q)
    assert s.cache.status() == 1
    s.cache.reset()
    for _ in range(3):
        assert torch.equal(sv.attend_decode(s.cache, q), good) and s.cache.status() == 0
    assert [w[0] for w in s.cache._ws.values()] == [ptr]


def test_logprobs_reset_clears_the_status(torch, sv):
    sv.logprobs_reset()
    x = torch.randn(2, 500, device="cuda")
    side = torch.cuda.Stream()
    bad = torch.tensor([3, 500], dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    sv.token_logprobs(x, bad, stream=side)
    assert sv.logprobs_status() == 2
    sv.logprobs_reset()
    assert sv.logprobs_status() == 0
    again = sv.token_logprobs(x, bad, stream=side)
    assert sv.logprobs_status() == 2 and torch.isnan(again.logprob[1])
    sv.logprobs_reset()
    assert sv.logprobs_status() == 0
