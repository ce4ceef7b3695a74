"""Attention whose output is the tail of its softmax, against the float64 oracle.

Tolerances count roundings (u = eps / 2 of the type) as in test_serving_gpu.py: scores are fp32 sums, a
probability is two 16-bit terms and off by 2^-17 (bf16) or 2^-21 (fp16) relative.  fp16 has no step
below 2^-24: probabilities enter the product scaled by at least 2^13 over the running maximum, so one
is also off by up to 2^-25 2^-13 = 2^-38 of the largest.
"""
import numpy as np
import pytest

from oracle import serving_oracle as SO
from tests.test_serving_gpu import Setup, f64, sv, torch  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("depth", [0, 8, 14, 16, 17, 18, 20])
@pytest.mark.parametrize("lens,kv_heads,dim,group", [([200] * 80, 8, 64, 1), ([3000, 200, 33], 2, 128, 8), ([700], 1, 256, 12),
                                                     ([1000], 1, 64, 24)])
def test_attention_sink(torch, sv, dtype, depth, lens, kv_heads, dim, group):
    """The first token takes nearly all the weight and has a value of 0; the others lie `depth` nats below it."""
    s = Setup(torch, sv, lens, kv_heads, dim, 16, "head", dtype, seed=depth)
    q = torch.zeros((len(lens), kv_heads * group, dim), dtype=s.dt, device="cuda")
    q[:, :, 0] = 1.0
    s.k[:, :, :, 0] = s.k[:, :, :, 0] * 0.25
    s.v.copy_((1000 * (1 + 0.25 * s.v.float())).to(s.dt))
    first = s.table[:, 0].long()
    s.k[first, :, 0, 0], s.v[first, :, 0] = float(depth), 0.0
    out, lse = sv.attend_decode(s.cache, q, scale=1.0, return_lse=True)
    want = SO.attend(f64(q), f64(s.k), f64(s.v), s.table.cpu().numpy(), lens, 1.0)
    u, bf = torch.finfo(s.dt).eps / 2, dtype == "bfloat16"
    got = f64(out)
    for i, w in enumerate(want):
        b, h = divmod(i, kv_heads)
        n = lens[b]
        mine = got[b, h * group:(h + 1) * group]
        delta = (dim / 16 + 16 + 4) * 2.0 ** -24 * w["absqk"]
        rel = 2 * delta + 2.0 ** -20 + (2.0 ** -17 if bf else 2.0 ** -21) + (n / 64 + 64) * 2.0 ** -24
        tol = rel * w["absv"] + u * np.abs(w["out"]) + (0 if bf else 2.0 ** -38 * w["vsum"] / w["floor"]) + 2.0 ** -25
        err = np.abs(mine - w["out"])
        assert np.all(err <= tol), (i, float((err / tol).max()), float((err / np.abs(w["out"])).max()))
