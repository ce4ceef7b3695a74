"""Attention over 8-bit codes against the float64 oracle where rounded probabilities would show.

Tolerances count roundings (u = eps / 2 of the output's type).  delta is a score's error: the products of
the tensor pipe (dim / 16 sums of 16) and the scales' multiplications and the reduction to base 2, 22
roundings of 2^-24 more, and queries below 2^-29 of their head's largest by 2^-39 of it.  A probability has
twice that relative to it, 2^-20 for its exponential and those that bring it to other references; times the
values' scale it enters the product as two fp16 terms, off by 2^-21 relative.  What the tensor pipe and the
warps add up has n / 64 + 64 roundings of 2^-24.  The output is rounded once, u |out| or half of its type's
smallest step.
"""
import numpy as np
import pytest

from oracle import longctx_oracle as LO

from .test_longctx_gpu import BOUNDS, Setup8, sv, torch   # noqa: F401  (fixtures among them)
from .test_serving_gpu import f64

pytestmark = pytest.mark.gpu

# Half of the smallest step of the output's types.
SMALLEST = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}


def worst(s, q, out, lse, scale, window=0, sink=0):
    """The largest error in units of its tolerance, of outputs and of log sums."""
    got, glse = f64(out), f64(lse)
    heads, dim = s.cache.n_kv_heads, s.cache.head_dim
    group = q.shape[1] // heads
    k, v = s.values()
    want = LO.attend(f64(q), k, v, s.table.cpu().numpy(), s.lens.tolist(), scale, window, sink)
    u = s.torch.finfo(out.dtype).eps / 2
    small = SMALLEST[str(out.dtype).split(".")[1]]
    codes, vs = s.codes()[1], np.repeat(f64(s.scales[1]), s.cache.page_size // s.scales[1].shape[2], axis=2)
    most = [0.0, 0.0]
    for i, w in enumerate(want):
        b, h = divmod(i, heads)
        n, mine = len(w["slots"]), slice(h * group, (h + 1) * group)
        if n == 0:
            assert (got[b, mine] == 0).all() and np.isneginf(glse[b, mine]).all()
            continue
        delta = (dim / 16 + 22) * 2.0 ** -24 * w["absqk"]
        delta += 2.0 ** -39 * dim * abs(scale) * np.abs(f64(q[b, mine])).max() * np.abs(w["k"]).max()
        rel = 2 * delta + 2.0 ** -20 + 2.0 ** -21 + (n / 64 + 64) * 2.0 ** -24
        p = np.exp((f64(q[b, mine]) @ w["k"].T) * scale - w["lse"][:, None])
        vst = vs[w["pages"], h, w["slots"]]
        step = np.maximum(2.0 ** -49 * (p * vst).max(axis=1), 2.0 ** -125 * vst.max())
        tol = rel * w["absv"] + u * np.abs(w["out"]) + small + step[:, None] * np.abs(codes[w["pages"], h, w["slots"]]).sum(axis=0)
        off = np.abs(got[b, mine] - w["out"]) / tol
        ltol = delta + 2.0 ** -20 + (n / 64 + 64) * 2.0 ** -24 + 8 * 2.0 ** -24 * (np.abs(w["lse"]) + w["absqk"])
        loff = np.abs(glse[b, mine] - w["lse"]) / ltol
        assert np.isfinite(off).all() and np.isfinite(loff).all()
        most = [max(most[0], float(off.max())), max(most[1], float(loff.max()))]
    return most


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim,group,window", [(64, 3, 0), (128, 8, 0), (256, 12, 0), (128, 24, 0), (64, 20, 4), (256, 8, 3)])
def test_outputs_of_values_that_cancel(torch, sv, capacity, dtype, dim, group, window):
    """A few tokens, whose values nearly cancel in many dimensions: the probabilities' own rounding is what is left."""
    lens = [2, 3, 4, 5, 6, 9] * 3
    s = Setup8(torch, sv, lens, 2, dim, 16, 8, dtype=dtype, seed=dim + group, scales=(-7, -6), capacity=capacity)
    q = s.randn(len(lens), 2 * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, scale=0.02, return_lse=True, window=window or None)
    got = worst(s, q, out, lse, 0.02, window)
    assert max(got) <= 1, got


def e4m3(torch, x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def places(s, b):
    """Pages and slots of the tokens of sequence b."""
    t = s.torch.arange(int(s.lens[b]), device="cuda")
    return s.table[b, t // s.cache.page_size].long(), t % s.cache.page_size


def powers(s, lo, hi, shape):
    return s.torch.exp2(s.torch.randint(lo, hi, shape, device="cuda", generator=s.g).float())


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("depth", [0, 8, 14, 16, 18, 20, 22, 24, 26, 28, 30])
@pytest.mark.parametrize("lens,kv_heads,dim,group,block", [([200] * 20, 4, 64, 1, 16), ([3000, 20, 33], 2, 128, 8, 1),
                                                           ([20, 700], 1, 256, 12, 8), ([1000, 9], 1, 64, 24, 16)])
def test_first_token_that_takes_the_weight(torch, sv, capacity, dtype, depth, lens, kv_heads, dim, group, block):
    """The first token takes nearly all the weight and has values of 0; the others' scores lie `depth` nats below its own."""
    s = Setup8(torch, sv, lens, kv_heads, dim, 16, block, dtype=dtype, seed=depth, capacity=capacity)
    q = torch.zeros((len(lens), kv_heads * group, dim), dtype=s.dt, device="cuda")
    q[:, :, 0] = 1.0
    s.scales[0].fill_(1.0)
    s.scales[1].copy_(powers(s, 3, 8, s.scales[1].shape))
    for b in range(len(lens)):
        p, at = places(s, b)
        s.k[p, :, at, 0] = e4m3(torch, s.randn(len(p), kv_heads) * 0.25)
        s.v[p, :, at] = e4m3(torch, 100 * (1 + 0.25 * s.randn(len(p), kv_heads, dim)).abs())
        s.k[p[0], :, 0, 0], s.v[p[0], :, 0] = e4m3(torch, torch.tensor(float(depth), device="cuda")), 0
    out, lse = sv.attend_decode(s.cache, q, scale=1.0, return_lse=True)
    got = worst(s, q, out, lse, 1.0)
    assert max(got) <= 1, got


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("group,dim,window", [(1, 64, 0), (8, 128, 0), (12, 256, 0), (24, 64, 0), (8, 256, 64), (20, 128, 300)])
@pytest.mark.parametrize("dtype,scales", [("bfloat16", (-40, 10)), ("bfloat16", (-100, -90)), ("bfloat16", (-90, -80)),
                                          ("bfloat16", (30, 60)), ("float16", (-12, 7)), ("float16", (-40, 5)), ("bfloat16", (-126, -117))])
def test_scales_of_values_of_any_size(torch, sv, capacity, group, dim, window, dtype, scales):
    """Values' scales that differ by up to 2^50, and all small or large; the smallest ones are the caller's own.  Keys'
    scales are drawn apart from them."""
    lens = [1500, 257, 5, 40]
    s = Setup8(torch, sv, lens, 2, dim, 32, 8, dtype=dtype, seed=dim + group, scales=scales, capacity=capacity)
    s.scales[0].copy_(powers(s, -9, -5, s.scales[0].shape))
    q = s.randn(len(lens), 2 * group, dim).to(s.dt)
    out, lse = sv.attend_decode(s.cache, q, return_lse=True, window=window or None)
    got = worst(s, q, out, lse, dim ** -0.5, window)
    assert max(got) <= 1, got


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
@pytest.mark.parametrize("far,spread", [(20, 0), (60, 0), (60, 8), (75, 3), (300, 0)])
@pytest.mark.parametrize("group,dim", [(2, 64), (8, 128), (12, 256), (24, 64)])
def test_scales_that_undo_the_scores(torch, sv, capacity, order, far, spread, group, dim):
    """Scores over a range of `far` nats, values' scales that make up for them: every token counts alike though their
    probabilities lie 2^100 apart.  (At 300 nats scales end, and most probabilities are 0 in fp32.)"""
    lens = [1200, 300, 33, 6]
    s = Setup8(torch, sv, lens, 1, dim, 16, 1, seed=far + dim, capacity=capacity)
    q = torch.zeros((len(lens), group, dim), dtype=s.dt, device="cuda")
    q[:, :, 0] = 1.0
    for b, n in enumerate(lens):
        p, at = places(s, b)
        score = torch.rand(n, device="cuda", generator=s.g) * far
        score = score if order == "mixed" else score.sort(descending=order == "falling").values
        s.scales[0][p, :, at] = 1.0
        s.k[p, 0, at, 0] = e4m3(torch, score)
        held = s.k[p, 0, at, 0].view(torch.float8_e4m3fn).float()
        e = torch.round(-held / 0.6931) + torch.randint(-spread, spread + 1, (n,), device="cuda", generator=s.g)
        s.scales[1][p, 0, at] = torch.exp2(e.clamp(-100, 70)).float()
    out, lse = sv.attend_decode(s.cache, q, scale=1.0, return_lse=True)
    got = worst(s, q, out, lse, 1.0)
    assert max(got) <= 1, got


@pytest.mark.parametrize("capacity", BOUNDS)
@pytest.mark.parametrize("power", [4, 12, 20, 24, 27, 40, 90])
@pytest.mark.parametrize("group,dim", [(2, 64), (8, 128), (12, 256), (24, 64)])
def test_scores_of_any_size(torch, sv, capacity, power, group, dim):
    """Scores that lie 2^power and more apart, to both sides: from 2^12 on, e^-4096 apart, the output is the value of
    the largest one's token."""
    lens = [700, 40, 3]
    s = Setup8(torch, sv, lens, 1, dim, 16, 4, seed=power + dim, scales=(-40, 40), capacity=capacity)
    q = torch.zeros((len(lens), group, dim), dtype=s.dt, device="cuda")
    q[:, :, 0] = 1.0
    q[:, 1, 0] = -1.0
    s.scales[0].fill_(1.0)
    for b, n in enumerate(lens):
        p, at = places(s, b)
        s.k[p, 0, at, 0] = e4m3(torch, torch.randint(-15, 16, (n,), device="cuda", generator=s.g).float())
        for i, x in ((n // 2, -16.0), (n // 3, 16.0)):
            s.k[p[i], 0, at[i], 0] = e4m3(torch, torch.tensor(x, device="cuda"))
    out, lse = sv.attend_decode(s.cache, q, scale=2.0 ** power, return_lse=True)
    if power < 12:    # scales 2^80 apart outweigh e^-16
        got = worst(s, q, out, lse, 2.0 ** power)
        assert max(got) <= 1, got
        return
    k, v = s.values()
    u = torch.finfo(s.dt).eps / 2      # 2^-8: bf16's step is 2^-7
    for b, n in enumerate(lens):
        p, at = (x.cpu().numpy() for x in places(s, b))
        score, value = k[p, 0, at, 0], v[p, 0, at]
        # (in three tokens the places of -16 and 16 are one: the other's largest is one of those drawn, or several alike)
        for heads, best, sign in (([0] + list(range(2, group)), score.max(), 1.0), ([1], score.min(), -1.0)):
            picked = value[score == best]
            want, size = picked.mean(axis=0), np.abs(picked).mean(axis=0)
            assert np.all(np.abs(f64(out[b, heads]) - want) <= u * np.abs(want) + 2.0 ** -18 * size)
            top = sign * best * 2.0 ** power + np.log(len(picked))
            assert np.all(np.abs(f64(lse[b, heads]) - top) <= 2.0 ** -21 * abs(top))
