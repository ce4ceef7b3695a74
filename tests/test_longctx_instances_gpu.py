"""Instances of the long-context kernels by type, head size and blocks of query heads, and calls that only meet together.

Tolerances are those of test_longctx_accuracy_gpu.py (codes) and test_longctx_gpu.py (16 bits, rotation)."""
import numpy as np
import pytest

from oracle import longctx_oracle as LO

from .test_longctx_accuracy_gpu import worst
from .test_longctx_gpu import BOUNDS, Setup8, check_window16, sv, torch   # noqa: F401  (fixtures among them)
from .test_serving_gpu import Setup, f64

pytestmark = pytest.mark.gpu

# every count of blocks of 8 query heads that a head size has, and rows that are two of them
GROUPS = [(64, 3), (64, 16), (64, 24), (64, 33), (128, 8), (128, 12), (128, 24), (128, 40), (256, 1), (256, 12), (256, 20)]
LENS = [1700, 1, 0, 129, 640, 33]


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("window,sink", [(None, 0), (100, 20), (1000, 0), (1, 3)])
@pytest.mark.parametrize("dim,group", GROUPS)
def test_codes(torch, sv, capacity, dtype, window, sink, dim, group):
    s = Setup8(torch, sv, LENS, 2, dim, 16, 8, dtype=dtype, seed=dim + group, capacity=capacity)
    q = s.randn(len(LENS), 2 * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True, window=window, sink=sink)
    assert s.cache.status() == 0
    got = worst(s, q, out, lse, dim ** -0.5, window or 0, sink)
    assert max(got) <= 1, got


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("window,sink", [(100, 20), (1000, 0), (1, 3)])
@pytest.mark.parametrize("dim,group", GROUPS)
def test_window_of_16_bits(torch, sv, capacity, dtype, window, sink, dim, group):
    s = Setup(torch, sv, LENS, 2, dim, 16, "head", dtype, seed=dim + group, capacity=capacity)
    q = s.randn(len(LENS), 2 * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True, window=window, sink=sink)
    assert s.cache.status() == 0
    check_window16(s, q, out, lse, dim ** -0.5, window, sink)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("n", [3, 1500])
@pytest.mark.parametrize("dim,heads", [(64, (3, 2)), (128, (5, 1)), (256, (1, 1))])
@pytest.mark.parametrize("normed", ["q", "k"])
def test_norm_of_queries_or_keys_alone(torch, sv, dtype, n, dim, heads, normed):
    """One side has weights and a norm, the other none; heads of both lie in one warp."""
    dt, (hq, hk) = getattr(torch, dtype), heads
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    x = torch.randn((n, hq + hk, dim), device="cuda", generator=g).to(dt)
    w = (1 + 0.3 * torch.randn(dim, device="cuda", generator=g)).to(dt)
    pos = torch.randint(-9999, 9999, (n,), device="cuda", generator=g, dtype=torch.int32)
    freqs = [100.0 ** (-i / 16) for i in range(16)]
    got = sv.qk_norm_rope(x[:, :hq], x[:, hq:], pos, sv.Rope(freqs), **{normed + "_weight": w})
    u = torch.finfo(dt).eps / 2
    for name, y, xs in (("q", got[0], x[:, :hq]), ("k", got[1], x[:, hq:])):
        want, mag = LO.norm_rope(f64(xs), f64(w) if name == normed else None, 1e-6, 0.0, pos.cpu().numpy()[None], freqs, None, False, 1.0)
        assert np.all(np.abs(f64(y) - want) <= 2.0 ** -19 * mag + u * np.abs(want) + 2.0 ** -25)


@pytest.mark.parametrize("codes", [True, False])
def test_graphs_captured_on_two_streams_run_at_once(torch, sv, codes):
    """Graphs of one cache that were captured on streams of their own have workspaces of their own."""
    lens = [20000, 300]
    make = (lambda: Setup8(torch, sv, lens, 2, 128, 64, 16, seed=3, capacity=100000)) if codes else (
        lambda: Setup(torch, sv, lens, 2, 128, 64, seed=3, capacity=100000))
    s = make()
    qs = [s.randn(2, 16, 128).to(s.dt) for _ in range(2)]
    window = None if codes else 15000
    want = [sv.attend_decode(s.cache, q, window=window) for q in qs]
    torch.cuda.synchronize()
    streams, graphs, got = [torch.cuda.Stream() for _ in range(2)], [], []
    for q, stream in zip(qs, streams):
        sv.attend_decode(s.cache, q, window=window, stream=stream)
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs = [sv.attend_decode(s.cache, q, window=window) for _ in range(5)]
        graphs.append(g)
        got.append(outs)
    for _ in range(20):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    assert s.cache.status() == 0
    for outs, w in zip(got, want):
        assert all(torch.equal(x, w) for x in outs)
