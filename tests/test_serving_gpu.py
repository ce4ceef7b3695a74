"""GPU parity of the serving operators against the float64 oracle.

Tolerances count roundings (u = eps / 2 of a type):
  attention  a score is a D-term fp32 sum: its error is at most about
             delta = (D / 16 + 16) 2^-24 max sum |q k| scale (the tensor pipe adds 16 products
             at a time) plus the roundings of the score itself, 4 2^-24 |s|.  Each probability
             then is off by 2 delta + 2^-20 relative (its own and the sum's score errors, two
             exponentials of 2^-22, the sum), and by 2^-17 relative (bf16, two terms of 8 bits)
             or 2^-21 relative plus 2^-25 of the largest (fp16) from its split; adding n
             products in fp32 along chains of at most n / 64 tiles and 16 tokens adds
             (n / 64 + 64) 2^-24.  The output is rounded once more, u |out|.
  logprobs   Z adds vocab / 1024 + 64 terms or fewer in a chain, each exponential 2^-21 off.
"""
import numpy as np
import pytest

from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.fixture(scope="module")
def sv(torch):
    from bit_quantized_sparse_gb300 import _build
    _build.build()
    from bit_quantized_sparse_gb300 import serving
    return serving


def f64(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """A cache of random tokens; every slot that no token occupies holds NaN, table entries past a sequence are -1."""

    def __init__(self, torch, sv, lens, kv_heads=2, dim=64, page=16, layout="head", dtype="bfloat16", seed=0, track=False,
                 room=0, capacity=None, amp=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        self.dt, self.g, self.torch = getattr(torch, dtype), g, torch
        need = [-(-(n + room) // page) for n in lens]
        width = max(1, max(need), -(-(capacity or 1) // page))
        pages = sum(need) + 3
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = (pages, kv_heads, page, dim) if layout == "head" else (pages, page, kv_heads, dim)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=self.dt, device="cuda") for _ in range(2))
        if layout == "slot":
            self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        for b, n in enumerate(lens):
            if n:
                t = torch.arange(n, device="cuda")
                p = self.table[b, t // page].long()
                self.k[p, :, t % page] = (self.randn(n, kv_heads, dim) * amp).to(self.dt)
                self.v[p, :, t % page] = self.randn(n, kv_heads, dim).to(self.dt)
        self.weight = self.pos = None
        if track:
            self.weight = torch.rand((len(lens), kv_heads, width * page), device="cuda", generator=g) * 3
            self.pos = self.randn(len(lens), kv_heads, width * page).argsort(2).to(torch.int32)
        self.cache = sv.PagedKVCache(self.k, self.v, self.table, self.lens, self.weight, self.pos)

    def randn(self, *shape):
        return self.torch.randn(shape, device="cuda", generator=self.g)


def check_attention(s, q, out, lse, scale, drawn=None, before=None):
    got, glse = f64(out), f64(lse)
    lens = s.lens.tolist()
    heads, dim = s.cache.n_kv_heads, s.cache.head_dim
    group = q.shape[1] // heads
    want = SO.attend(f64(q), f64(s.k), f64(s.v), s.table.cpu().numpy(), lens, scale)
    bf = out.dtype == s.torch.bfloat16
    u = s.torch.finfo(out.dtype).eps / 2
    for i, w in enumerate(want):
        b, h = divmod(i, heads)
        n, mine = lens[b], slice(h * group, (h + 1) * group)
        delta = (dim / 16 + 16 + 4) * 2.0 ** -24 * w["absqk"]
        rel = 2 * delta + 2.0 ** -20 + (2.0 ** -17 if bf else 2.0 ** -21) + (n / 64 + 64) * 2.0 ** -24
        tol = rel * w["absv"] + u * np.abs(w["out"]) + (0 if bf else 2.0 ** -25 * w["vsum"] / w["floor"]) + 2.0 ** -25
        err = np.abs(got[b, mine] - w["out"])
        assert np.all(err <= tol), (i, n, float((err / tol).max()))
        if n == 0 or np.any(np.isneginf(w["lse"])):
            assert np.array_equal(glse[b, mine], w["lse"])
        else:
            assert np.all(np.abs(glse[b, mine] - w["lse"]) <= delta + 2.0 ** -20 + (n / 64 + 64) * 2.0 ** -24
                          + 8 * 2.0 ** -24 * (np.abs(w["lse"]) + w["absqk"]))
        if drawn is not None:
            more = f64(drawn[b, h, :n]) - f64(before[b, h, :n])
            assert np.all(np.abs(more - w["drawn"]) <= (2 * delta + 2.0 ** -19 + 8 * 2.0 ** -24 * w["absqk"] + (n / 64 + 64) * 2.0 ** -24)
                          * w["drawn"] + (group + 4) * 2.0 ** -24 * (f64(before[b, h, :n]) + w["drawn"]))
            # nothing past the length is written
            assert np.isnan(f64(drawn[b, h, n:])).all() or drawn.data_ptr() == s.weight.data_ptr()


LENS = [300, 0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 1000, 33, 448, 0]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("kv_heads,group,page,layout", [
    (2, 8, 16, "head"), (1, 1, 1, "slot"), (3, 5, 7, "head"), (2, 12, 64, "slot"), (1, 24, 128, "head"), (8, 4, 32, "slot"),
    (1, 16, 24, "slot"), (5, 1, 48, "head")])
def test_attention_lengths_heads_pages(torch, sv, dim, dtype, kv_heads, group, page, layout):
    s = Setup(torch, sv, LENS, kv_heads, dim, page, layout, dtype, seed=dim + group)
    q = s.randn(len(LENS), kv_heads * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True)
    assert s.cache.status() == 0
    check_attention(s, q, out, lse, dim ** -0.5)


@pytest.mark.parametrize("n", [1, 31, 64, 4097, 20011])
@pytest.mark.parametrize("dim,group", [(64, 3), (128, 8), (256, 8), (128, 16), (256, 10)])
def test_attention_one_sequence_split_over_the_gpu(torch, sv, n, dim, group):
    s = Setup(torch, sv, [n], 2, dim, 64, "head", seed=n)
    q = (s.randn(1, 2 * group, dim) * 2).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, scale=0.11, return_lse=True)
    check_attention(s, q, out, lse, 0.11)


@pytest.mark.parametrize("dim,group", [(64, 12), (64, 17), (64, 24), (64, 33), (128, 12), (128, 17), (128, 24), (128, 25),
                                       (128, 128), (256, 16), (256, 17), (256, 24)])
@pytest.mark.parametrize("kv_heads,page,layout", [(1, 16, "head"), (3, 7, "slot")])
def test_attention_large_groups(torch, sv, dim, group, kv_heads, page, layout):
    """Blocks of query heads of every size, rows that one CTA ends and rows that several share."""
    lens = [5000, 1, 0, 64, 65, 700, 129]
    s = Setup(torch, sv, lens, kv_heads, dim, page, layout, seed=24 + group)
    q = s.randn(len(lens), kv_heads * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True)
    check_attention(s, q, out, lse, dim ** -0.5)


@pytest.mark.parametrize("dim,group", [(64, 4), (64, 24), (128, 6), (128, 16), (256, 8), (256, 12)])
@pytest.mark.parametrize("page", [8, 24, 40])
@pytest.mark.parametrize("layout", ["head", "slot"])
def test_attention_pages_of_eights(torch, sv, dim, group, page, layout):
    """Pages of a multiple of 8 slots but not of 16: two runs to 16 tokens, often on two pages."""
    lens = [3000, 8, 9, 24, 511, 130]
    s = Setup(torch, sv, lens, 2, dim, page, layout, seed=page)
    q = s.randn(len(lens), 2 * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True)
    assert s.cache.status() == 0
    check_attention(s, q, out, lse, dim ** -0.5)


def test_attention_many_short_sequences(torch, sv):
    lens = [(i * 37) % 130 for i in range(700)]
    s = Setup(torch, sv, lens, 1, 64, 16, "head", seed=3)
    q = s.randn(len(lens), 4, 64).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True)
    check_attention(s, q, out, lse, 64 ** -0.5)


def test_attention_growing_and_large_scores(torch, sv):
    """Scores that rise through the sequence (the running maximum moves all the time) up to about +-2000."""
    s = Setup(torch, sv, [700, 64, 1500], 1, 64, 16, "head", "float16", seed=4)
    for b, n in enumerate(s.lens.tolist()):
        t = torch.arange(n, device="cuda")
        s.k[s.table[b, t // 16].long(), :, t % 16] *= (t * 0.05)[:, None, None].to(s.dt)
    q = (s.randn(3, 8, 64) * 4).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, scale=1.0, return_lse=True)
    check_attention(s, q, out, lse, 1.0)


def test_attention_rows_without_scores(torch, sv):
    """Scores that are all -inf give zeros and lse -inf; a NaN key gives NaN in its own row only."""
    s = Setup(torch, sv, [100, 40, 20], 1, 64, 16, seed=5)
    q = s.randn(3, 2, 64).abs().to(s.dt) + 0.1
    for b in (0, 1):
        n = int(s.lens[b])
        t = torch.arange(n, device="cuda")
        s.k[s.table[b, t // 16].long(), :, t % 16] = float("-inf")
    s.k[s.table[1, 0].long(), :, 3] = float("nan")
    out, lse = sv.attend_decode(s.cache, q, return_lse=True)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isfinite(out[2]).all()


@pytest.mark.parametrize("dim,kv_heads,group,page", [(256, 2, 8, 16), (64, 1, 20, 8), (128, 4, 1, 64)])
def test_attention_adds_up_weights(torch, sv, dim, kv_heads, group, page):
    lens = [513, 0, 1, 64, 1201, 90]
    s = Setup(torch, sv, lens, kv_heads, dim, page, "slot", seed=6, track=True)
    q = s.randn(len(lens), kv_heads * group, dim).to(s.dt)
    before = s.weight.clone()
    drawn = torch.full_like(s.weight, float("nan"))
    out, lse = sv.attend_decode(s.cache, q, return_lse=True, max_len=1201, weight_out=drawn)
    assert torch.equal(s.weight, before)
    check_attention(s, q, out, lse, dim ** -0.5, drawn, before)
    out2, lse2 = sv.attend_decode(s.cache, q, return_lse=True, max_len=1201, weight_out=s.weight)   # in place
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for b, n in enumerate(lens):
        assert torch.equal(s.weight[b, :, :n], drawn[b, :, :n]) and torch.equal(s.weight[b, :, n:], before[b, :, n:])


def test_attention_views_and_shared_pages(torch, sv):
    """q a slice of one projection's output, out with rows apart, two sequences that share their first pages."""
    s = Setup(torch, sv, [200, 200, 77], 2, 128, 16, "slot", "float16", seed=7)
    s.table[1, :12] = s.table[0, :12]
    proj = s.randn(3, 20, 128).to(s.dt)
    q = proj[:, 3:11]
    room = torch.full((3, 10, 128), 9.0, dtype=s.dt, device="cuda")
    out, lse = sv.attend_decode(s.cache, q, out=room[:, 1:9], return_lse=True)
    check_attention(s, q, out, lse, 128 ** -0.5)
    assert torch.all(room[:, 0] == 9) and torch.all(room[:, 9] == 9)


def test_attention_is_deterministic_on_any_stream_and_in_graphs(torch, sv):
    lens = [3000, 5, 0, 777]
    s = Setup(torch, sv, lens, 2, 128, 32, seed=8, track=True)
    q = s.randn(4, 16, 128).to(s.dt)
    w = torch.zeros_like(s.weight)
    first = sv.attend_decode(s.cache, q, return_lse=True, weight_out=w)
    w1 = w.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = sv.attend_decode(s.cache, q, return_lse=True, weight_out=w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1]) and torch.equal(w, w1)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sv.attend_decode(s.cache, q, out=out, weight_out=w)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            sv.attend_decode(s.cache, q, out=out, weight_out=w)
    out.zero_()
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(w, w1)
    # the lengths are read when the graph runs
    s.lens[0] = 40
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, sv.attend_decode(s.cache, q)) and not torch.equal(out[0], first[0][0])


def test_graph_outlives_a_larger_workspace(torch, sv):
    """A call that needs a larger workspace on the same stream leaves the one that a captured graph holds alone."""
    s = Setup(torch, sv, [3000, 70], 2, 64, 16, seed=22, track=True)
    q = s.randn(2, 8, 64).to(s.dt)
    out, w = torch.empty_like(q), torch.zeros_like(s.weight)
    good = sv.attend_decode(s.cache, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sv.attend_decode(s.cache, q, out=out)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            sv.attend_decode(s.cache, q, out=out)
        sv.attend_decode(s.cache, q, weight_out=w)
        waste = [torch.full((1 << 18,), -1, dtype=torch.int32, device="cuda") for _ in range(64)]   # takes what was freed
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, good) and s.cache.status() == 0 and len(waste) == 64


def test_attention_reports_bad_pages_and_lengths(torch, sv):
    """Pages outside the cache are left out, too long lengths are cut, and the status says so; the next cache is fine."""
    s = Setup(torch, sv, [100, 60], 1, 64, 16, seed=9)
    q = s.randn(2, 4, 64).to(s.dt)
    good = sv.attend_decode(s.cache, q)
    assert s.cache.status() == 0
    s.table[0, 2] = s.k.shape[0]
    got = sv.attend_decode(s.cache, q)
    assert torch.isfinite(got).all() and torch.equal(got[1], good[1])
    assert s.cache.status() == 2
    s2 = Setup(torch, sv, [100, 60], 1, 64, 16, seed=9)
    s2.lens[0], s2.lens[1] = 2 ** 31 - 1, -5
    got = sv.attend_decode(s2.cache, q, max_len=100)
    assert torch.equal(got[0], good[0]) and torch.all(got[1] == 0) and s2.cache.status() == 2


def test_attention_past_32_bit_offsets(torch, sv):
    """A pool of more than 2^31 elements; the tokens lie in its last pages."""
    if torch.cuda.mem_get_info()[0] < 24e9:
        pytest.skip("needs 24 GB")
    heads, dim, page, pages = 8, 256, 64, 16500
    k, v = (torch.empty((pages, heads, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    table = torch.arange(pages - 1, pages - 6, -1, device="cuda", dtype=torch.int32)[None].contiguous()
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    big = sv.PagedKVCache(k, v, table, lens)
    s = Setup(torch, sv, [300], heads, dim, page, seed=10)
    for i in range(5):
        k[table[0, i].long()], v[table[0, i].long()] = s.k[s.table[0, i].long()], s.v[s.table[0, i].long()]
    q = s.randn(1, 16, dim).to(s.dt)
    assert torch.equal(sv.attend_decode(big, q), sv.attend_decode(s.cache, q))
    new = s.randn(1, heads, dim).to(s.dt)
    sv.kv_append(big, new, new)
    assert torch.equal(k[table[0, 4].long(), :, 43], new[0]) and big.status() == 0


@pytest.mark.parametrize("dim,kv_heads,page,layout,dtype", [
    (64, 1, 1, "head", "bfloat16"), (128, 3, 7, "slot", "float16"), (256, 8, 64, "head", "bfloat16")])
@pytest.mark.parametrize("track", [False, True])
def test_append(torch, sv, dim, kv_heads, page, layout, dtype, track):
    s = Setup(torch, sv, [40, 0, 9], kv_heads, dim, page, layout, dtype, seed=11, track=track, room=30)
    seq = torch.tensor([2] * 13 + [0] * 30 + [1] * 1, dtype=torch.int32, device="cuda")
    slot = torch.cat([torch.arange(9, 22), torch.arange(40, 70), torch.arange(0, 1)]).to(torch.int32).cuda()
    mix = torch.randperm(len(seq), device="cuda")
    seq, slot = seq[mix].contiguous(), slot[mix].contiguous()
    kv = s.randn(len(seq), 3, kv_heads, dim).to(s.dt)
    want_k, want_v = SO.append(f64(s.k), f64(s.v), s.table.cpu().numpy(), f64(kv[:, 0]), f64(kv[:, 2]), seq.tolist(), slot.tolist())
    pos = (slot * 3 + 1).contiguous()
    w0 = None if not track else (s.weight.clone(), s.pos.clone())
    sv.kv_append(s.cache, kv[:, 0], kv[:, 2], seq=seq, slot=slot, pos=pos if track else None)
    assert s.cache.status() == 0
    assert np.array_equal(f64(s.k), want_k, equal_nan=True) and np.array_equal(f64(s.v), want_v, equal_nan=True)
    if track:
        w0[0][seq.long(), :, slot.long()] = 0
        w0[1][seq.long(), :, slot.long()] = pos[:, None].expand(-1, kv_heads)
        assert torch.equal(s.weight, w0[0]) and torch.equal(s.pos, w0[1])


def test_append_to_each_sequence_end(torch, sv):
    """Without seq and slot, token i becomes the last of sequence i; an idle sequence gets nothing."""
    s = Setup(torch, sv, [5, 0, 17], 2, 64, 4, seed=12, track=True, room=3)
    s.lens += torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    new = s.randn(3, 2, 64).to(s.dt)
    want = SO.append(f64(s.k), f64(s.v), s.table.cpu().numpy(), f64(new[[0, 2]]), f64(-new[[0, 2]]), [0, 2], [5, 17])
    sv.kv_append(s.cache, new, -new)
    assert np.array_equal(f64(s.k), want[0], equal_nan=True) and np.array_equal(f64(s.v), want[1], equal_nan=True)
    assert s.cache.status() == 0 and s.pos[2, :, 17].tolist() == [17, 17] and s.weight[0, :, 5].tolist() == [0, 0]
    sv.kv_append(s.cache, new[:0], new[:0], seq=s.lens[:0], slot=s.lens[:0])   # nothing to do


def test_append_reports_bad_places(torch, sv):
    s = Setup(torch, sv, [20, 20], 1, 64, 8, seed=13)
    before = s.k.clone()
    new = s.randn(6, 1, 64).to(s.dt)
    seq = torch.tensor([-1, 2, 0, 0, 1, 1], dtype=torch.int32, device="cuda")
    slot = torch.tensor([0, 0, -1, 24, 2 ** 30, 7], dtype=torch.int32, device="cuda")
    sv.kv_append(s.cache, new, new, seq=seq, slot=slot)
    assert s.cache.status() == 2
    before[s.table[1, 0].long(), :, 7] = new[5]
    assert torch.equal(s.k.nan_to_num(7), before.nan_to_num(7))


def check_evict(torch, sv, s, seen, budget, sink, recent, in_place, max_len=None):
    table, lens = s.table.cpu().numpy(), s.lens.tolist()
    want = SO.evict(f64(s.k), f64(s.v), table, lens, f64(s.weight), s.pos.cpu().numpy(), seen.tolist(), budget, sink, recent)
    w, p, n = s.weight, s.pos, s.lens
    if not in_place:
        w, p, n = torch.full_like(w, -7.0), torch.full_like(p, -7), torch.full_like(n, -7)
    sv.kv_evict(s.cache, seen, budget, sink, recent, max_len, **({} if in_place else dict(lens_out=n, weight_out=w, pos_out=p)))
    assert s.cache.status() == 0
    assert n.tolist() == want[4]
    assert np.array_equal(f64(s.k), want[0], equal_nan=True) and np.array_equal(f64(s.v), want[1], equal_nan=True)
    for b, m in enumerate(want[4]):
        assert np.array_equal(f64(w[b, :, :m]), want[2][b, :, :m], equal_nan=True)
        assert np.array_equal(p[b, :, :m].cpu().numpy(), want[3][b, :, :m])
        if not in_place:
            assert torch.all(w[b, :, m:] == -7) and torch.all(p[b, :, m:] == -7)


@pytest.mark.parametrize("dim,kv_heads,page,layout,dtype", [
    (64, 1, 1, "slot", "float16"), (128, 3, 7, "head", "bfloat16"), (256, 2, 64, "slot", "bfloat16")])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (33, 4, 9), (100, 0, 100), (700, 3, 0), (5000, 1, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(torch, sv, dim, kv_heads, page, layout, dtype, budget, sink, recent, in_place):
    lens = [100, 0, 1, 33, 34, 32, 2049, 701, 99]
    s = Setup(torch, sv, lens, kv_heads, dim, page, layout, dtype, seed=14 + budget, track=True)
    seen = s.lens + 40
    check_evict(torch, sv, s, seen, budget, sink, recent, in_place)


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "special", "negative"])
def test_evict_ties_and_odd_weights(torch, sv, kind):
    s = Setup(torch, sv, [1500, 1025, 130], 2, 64, 16, seed=15, track=True)
    w = s.weight
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "zeros":
        w.copy_(torch.where(w < 1.5, torch.zeros_like(w), -torch.zeros_like(w)))
    elif kind == "few":
        w.copy_((w * 1.3).floor())
    elif kind == "special":
        w[:, :, ::3], w[:, :, 1::7], w[:, :, 2::11] = float("nan"), float("inf"), float("-inf")
    else:
        w.neg_()
    check_evict(torch, sv, s, s.lens.clone(), 129, 2, 5, False)


def test_evict_long_rows(torch, sv):
    """More tokens than the selection holds in shared memory."""
    s = Setup(torch, sv, [60000, 40000], 1, 64, 256, seed=16, track=True)
    check_evict(torch, sv, s, s.lens.clone(), 20000, 4, 1000, False)


def test_evict_row_that_shared_memory_cannot_hold(torch, sv):
    s = Setup(torch, sv, [340001], 1, 64, 256, seed=18, track=True)
    check_evict(torch, sv, s, s.lens.clone(), 90000, 4, 1000, False)


@pytest.mark.parametrize("equal", [False, True])
@pytest.mark.parametrize("budget,sink,recent", [(64, 4, 9), (257, 0, 0)])
def test_evict_more_rows_than_sms(torch, sv, budget, sink, recent, equal):
    lens = [(37 * b) % 531 for b in range(60)] + [2500, 1024]
    s = Setup(torch, sv, lens, 4, 64, 16, seed=21, track=True)
    if equal:
        s.weight.fill_(0.5)
    check_evict(torch, sv, s, s.lens + 3, budget, sink, recent, equal)


def test_evict_more_protected_than_budget(torch, sv):
    """Positions that repeat can protect more tokens than fit: the first of them stay, still `budget` tokens."""
    s = Setup(torch, sv, [200], 1, 64, 16, seed=17, track=True)
    s.pos.zero_()
    check_evict(torch, sv, s, s.lens.clone(), 50, 1, 0, True)


def test_evict_reports_bad_pages_and_lengths(torch, sv):
    s = Setup(torch, sv, [200, 90], 1, 64, 16, seed=18, track=True)
    s.table[0, 0] = -3
    before = s.k[s.table[1, :6].long()].clone()
    sv.kv_evict(s.cache, s.lens.clone(), 100)
    assert s.cache.status() == 2 and s.lens.tolist() == [100, 90]
    assert torch.equal(s.k[s.table[1, :6].long()].nan_to_num(7), before.nan_to_num(7))
    s2 = Setup(torch, sv, [200, 90], 1, 64, 16, seed=18, track=True)
    s2.lens[0], s2.lens[1] = 2 ** 30, -1
    out = torch.zeros_like(s2.lens)
    sv.kv_evict(s2.cache, s2.lens, 100, max_len=200, lens_out=out)
    assert s2.cache.status() == 2 and out.tolist() == [100, 0]


def check_logprobs(torch, sv, x, targets, top):
    r = sv.token_logprobs(x, targets, top)
    lp, h, idx, val, spread = SO.token_logprobs(f64(x), targets.tolist(), top)
    sums = (x.shape[1] / 1024 + 64) * 2.0 ** -24 + 2.0 ** -21
    big = np.where(np.isfinite(f64(x)), np.abs(f64(x)), 0).max(axis=1, initial=0)
    tol = sums + 2.0 ** -22 * (1 + big)

    def near(got, want, tol):
        got = f64(got)
        same = np.isnan(want) & np.isnan(got) | (np.isinf(want) & (got == want))
        with np.errstate(invalid="ignore"):
            err = np.abs(got - want)
        assert np.all(same | (err <= tol + 2.0 ** -23 * np.abs(want))), (got, want)
    near(r.logprob, lp, tol)
    near(r.entropy, h, 2 * (sums + 2.0 ** -22) * (1 + spread))
    if top:
        assert np.array_equal(r.top_index.cpu().numpy(), idx)
        near(r.top_logprob, val, tol[:, None])
    else:
        assert r.top_index is None


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 31, 31), (2, 33, 32), (5, 257, 0), (7, 1000, 1), (3, 4097, 20),
                                            (2, 32000, 5), (4, 49999, 32), (1, 131071, 8), (1, 262144, 20)])
def test_logprobs_sizes(torch, sv, dtype, rows, vocab, top):
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    x = (torch.randn(rows, vocab, device="cuda", generator=g) * 3).to(getattr(torch, dtype))
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g).to(torch.int32)
    check_logprobs(torch, sv, x, t, top)
    assert sv.logprobs_status() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("offset", [1, 3, 8])
def test_logprobs_strided_rows(torch, sv, dtype, offset):
    """Rows apart and starting at any element."""
    room = torch.full((5, 9000 + 37), float("nan"), device="cuda").to(getattr(torch, dtype))
    x = room[:, offset:offset + 7001]
    x.copy_((torch.randn(5, 7001, device="cuda") * 5).to(x.dtype))
    check_logprobs(torch, sv, x, torch.tensor([0, 7000, 5, -1, 3500], dtype=torch.int32, device="cuda"), 13)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "masked", "lowest", "one", "peak", "two_values", "odd",
                                  "minus_zero", "periodic"])
@pytest.mark.parametrize("vocab", [200, 20003, 140001])
def test_logprobs_odd_rows(torch, sv, dtype, kind, vocab):
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    x = torch.randn(4, vocab, device="cuda", generator=g).to(dt)
    lin = torch.arange(vocab, device="cuda") * (8.0 / vocab)
    if kind == "equal":
        x.fill_(-3.25)
    elif kind == "ascending":
        x.copy_(lin.to(dt).expand(4, -1))
    elif kind == "descending":
        x.copy_((-lin).to(dt).expand(4, -1))
    elif kind == "masked":      # a grammar leaves a few tokens
        x[:, torch.arange(vocab, device="cuda") % 61 != 7] = float("-inf")
    elif kind == "lowest":
        x[:, torch.arange(vocab, device="cuda") % 61 != 7] = torch.finfo(dt).min
    elif kind == "one":         # one token is left, or none
        x.fill_(float("-inf"))
        x[0, vocab - 1], x[1, 0], x[2, vocab // 2] = 3.0, -5.0, 0.0
    elif kind == "peak":
        x[:, 17] = 90.0
    elif kind == "two_values":
        x.copy_((x > 1).to(dt))
    elif kind == "odd":
        x[0, 5], x[1, vocab - 3], x[2, 9] = float("nan"), float("inf"), float("-inf")
        x[3].fill_(float("nan"))
        x[3, 4] = 1.0
    elif kind == "periodic":    # a few threads of a block hold all the large logits
        x += torch.where(torch.arange(vocab, device="cuda") % (1024 if dtype == "float32" else 2048) < 120, 20, 0).to(dt)
    else:
        x.copy_(torch.where(x > 0, torch.zeros_like(x), -torch.zeros_like(x)))
    check_logprobs(torch, sv, x, torch.tensor([0, vocab - 1, vocab // 2, 17], dtype=torch.int32, device="cuda"), 20)


def test_logprobs_targets(torch, sv):
    """-1 asks for nothing; other targets outside the vocabulary give NaN and are reported."""
    x = torch.randn(4, 500, device="cuda")
    r = sv.token_logprobs(x, torch.tensor([-1, 499, 0, -1], dtype=torch.int32, device="cuda"))
    assert r.logprob[0] == 0 and r.logprob[3] == 0 and r.logprob[1] < 0 and sv.logprobs_status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = sv.token_logprobs(x, torch.tensor([-2, 500, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda"), stream=side)
    side.synchronize()
    assert torch.isnan(r.logprob[:3]).all() and torch.isfinite(r.logprob[3]) and sv.logprobs_status() == 2
    assert sv.token_logprobs(x).logprob is None
    sv._ctrl.clear()


def test_logprobs_deterministic_and_in_graphs(torch, sv):
    x = torch.randn(9, 70001, device="cuda").to(torch.bfloat16)
    t = torch.arange(9, device="cuda", dtype=torch.int32)
    first = sv.token_logprobs(x, t, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sv.token_logprobs(x, t, 7)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = sv.token_logprobs(x, t, 7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, got))


def test_empty_batches_and_bounds(torch, sv):
    """No sequences, no tokens, no rows, a bound of 0: nothing happens, or zeros and -inf."""
    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device="cuda")
    c = sv.PagedKVCache.allocate(4, 16, 2, 64, ints(0, 4), ints(0), track=True)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert sv.attend_decode(c, q, weight_out=c.weight).shape == q.shape
    sv.kv_append(c, q[:, :2], q[:, :2])
    sv.kv_evict(c, ints(0), 5)
    r = sv.token_logprobs(torch.zeros((0, 10), device="cuda"), ints(0), 3)
    assert r.logprob.shape == (0,) and r.top_index.shape == (0, 3)
    s = Setup(torch, sv, [0, 3], 2, 64, 16, seed=23, track=True)
    q, w = s.randn(2, 4, 64).to(s.dt), s.weight.clone()
    s.lens.zero_()
    out, lse = sv.attend_decode(s.cache, q, return_lse=True, weight_out=w, max_len=0)
    assert torch.all(out == 0) and torch.all(lse == float("-inf")) and torch.equal(w, s.weight)
    sv.kv_append(s.cache, q[:, :2], q[:, :2])       # idle sequences
    sv.kv_evict(s.cache, s.lens, 5, max_len=0)
    assert s.cache.status() == 0 and s.lens.tolist() == [0, 0]


def test_refusals_leave_no_work(torch, sv):
    from bit_quantized_sparse_gb300.moe_w4 import MoeW4Error
    s = Setup(torch, sv, [20, 20], 2, 64, 8, seed=19)
    q = s.randn(2, 4, 64).to(s.dt)
    for bad in (q.float(), q[:1], q[:, :, :32], q.cpu(), q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            sv.attend_decode(s.cache, bad)
    with pytest.raises(MoeW4Error):
        sv.attend_decode(s.cache, q[:, :3])           # heads that the kv heads do not divide
    with pytest.raises(MoeW4Error):
        sv.attend_decode(s.cache, q, max_len=25)      # more than the block table holds
    with pytest.raises(ValueError):
        sv.attend_decode(s.cache, q, weight_out=torch.zeros(2, 2, 24, device="cuda"))
    with pytest.raises(ValueError):
        sv.kv_evict(s.cache, s.lens, 5)
    with pytest.raises(ValueError):
        sv.kv_append(s.cache, q[:, :2], q[:, :2], seq=s.lens.long())
    with pytest.raises(ValueError):
        sv.token_logprobs(torch.zeros(2, 9, device="cuda").t())
    with pytest.raises(MoeW4Error):
        sv.token_logprobs(torch.zeros(2, 9, device="cuda"), top=10)


@pytest.mark.parametrize("rows,vocab,top,dtype", [(200, 5003, 9, "bfloat16"), (700, 5003, 9, "bfloat16"), (700, 7, 7, "float32"),
                                                  (2000, 1031, 32, "float16"), (3001, 257, 0, "bfloat16"), (950, 9001, 1, "float32")])
def test_logprobs_many_rows(torch, sv, rows, vocab, top, dtype):
    """More rows than the grid has places: CTAs take several in turn.  Some rows are odd: masked, equal, with NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x = (torch.randn(rows, vocab, device="cuda", generator=g) * 3).to(getattr(torch, dtype))
    x[5], x[6, 1:], x[7, 0], x[rows - 1, ::2] = 1.5, float("-inf"), float("nan"), float("-inf")
    x[8], x[9, -1] = float("-inf"), float("inf")
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g).to(torch.int32)
    check_logprobs(torch, sv, x, t, top)


def test_attention_wait_timeout_is_reported(torch, sv):
    """With the hook on, CTA 0 does not say that its partial result is there: the waits for it run out (2 s), the status
    says so, and after the workspace is cleared the next call is right."""
    from bit_quantized_sparse_gb300 import moe_w4 as mw
    s = Setup(torch, sv, [4000], 1, 64, 16, seed=20)
    q = s.randn(1, 4, 64).to(s.dt)
    good = sv.attend_decode(s.cache, q)
    (ptr, size, _), = s.cache._ws.values()
    stream = torch.cuda.current_stream().cuda_stream
    assert mw.moe_w4_test_skip_publish(ptr, size, 1, stream) == 0
    sv.attend_decode(s.cache, q)
    assert s.cache.status() == 1
    assert mw.moe_w4_workspace_init(ptr, size, stream) == 0
    assert torch.equal(sv.attend_decode(s.cache, q), good) and s.cache.status() == 0


def test_example_decodes_with_all_operators(torch, sv):
    """examples/decode_loop.py: the first step against a plain computation, the cache within its budget, no status, the
    same tokens every time."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_loop.py")
    spec = importlib.util.spec_from_file_location("decode_loop", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    (tokens, logprob, entropy), dec = ex.generate(70, seqs=3, budget=24, page=8)
    assert dec.cache.status() == 0 and dec.layer.status() == 0 and sv.logprobs_status() == 0
    n = dec.lens.tolist()
    assert n == [dec.length] * 3 and dec.length <= 32
    assert torch.isfinite(logprob).all() and torch.isfinite(entropy).all() and torch.all(logprob <= 0)
    held = dec.cache.pos[:, :, :n[0]]
    for b in range(3):
        for h in range(2):
            p = sorted(held[b, h].tolist())
            assert len(set(p)) == len(p) and p[:2] == [0, 1] and p[-6:] == list(range(64, 70))   # sinks, and the newest
    # every step hands out one unit of weight per query head: what is left is at most that
    assert torch.all(dec.cache.weight[:, :, :n[0]].sum(2) <= 70 * 4 * (1 + 1e-4))
    (again, _, _), _ = ex.generate(70, seqs=3, budget=24, page=8)
    assert torch.equal(tokens, again)
    # one token: attention returns its value vectors
    fresh = ex.Decoder(seqs=3)
    first = torch.arange(3, dtype=torch.int32, device="cuda")
    x = fresh.embed[first.long()]
    v = (fresh._normed(x) @ fresh.qkv).view(3, -1, 64)[:, -2:]
    x = x + v.repeat_interleave(4, 1).reshape(3, -1) @ fresh.proj
    from bit_quantized_sparse_gb300 import moe_w4 as mw
    x = x + mw.forward_decode(fresh.layer, fresh._normed(x).contiguous())
    logits = (fresh._normed(x) @ fresh.unembed).float()
    following, best = fresh.step(first)
    assert torch.equal(following.long(), logits.argmax(1))
    want = torch.log_softmax(logits, 1).amax(1)
    assert torch.allclose(best.top_logprob[:, 0], want, atol=1e-4)
