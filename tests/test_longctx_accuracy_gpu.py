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
        tol = rel * w["absv"] + u * np.abs(w["out"]) + small
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
