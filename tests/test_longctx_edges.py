"""Calls of the operators for long contexts at the ends of what their arguments allow, without a GPU."""
import os
import subprocess
import sys

from .test_serving_boundary import ROOT, mw   # noqa: F401  (mw: the fixture)

READS = """
import ctypes
from tests import test_longctx_boundary as t
from bit_quantized_sparse_gb300 import moe_w4 as mw
ref, c = ctypes.byref, t.cache8(mw, n_seqs=0)
print(*(f(ref(x), ref(t.tokens(mw, n=n)), None) for n in (3, 0) for f, x in ((mw.moe_w4_kv8_read, c), (mw.moe_w4_kv_read, c.c))))
"""


def test_rows_of_a_cache_of_no_sequences_are_written(mw):   # noqa: F811
    """Their zeros need a launch: without a GPU that is an error, not success; no rows need none."""
    got = subprocess.run([sys.executable, "-c", READS], cwd=ROOT, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""},
                         capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
    assert got.stdout.split() == ["-4", "-4", "0", "0"]
