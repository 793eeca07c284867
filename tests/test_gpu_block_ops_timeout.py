"""Waits of the operators around the linears that run out, by arrivals which the test build of the library withholds
(libnvfp4_testhooks.so, compiled with NVFP4_TEST_HOOKS): the call reports the timeout, its copies have landed and its TMEM is free
when it ends, and the next ordinary call gives its usual bits.  Nothing is faulted or hung: every wait has the limit set
here."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = r"""
import ctypes, sys
sys.path.insert(0, {root!r})
import torch
from epilogue_gemm_nvfp4_b200 import binding as B
from epilogue_gemm_nvfp4_b200 import build as BLD

B.LIB_PATH = BLD.TEST_LIB
lib = B.load()
lib.nvfp4_test_withhold_arrivals.argtypes = [ctypes.c_int32]
lib.nvfp4_test_withhold_arrivals.restype = None
torch.cuda.set_device(0)
torch.manual_seed(0)

def check(name, call):
    ref = call()
    clean = B.get_device_error()
    lib.nvfp4_test_withhold_arrivals(1)
    call()
    timed_out = B.get_device_error()
    lib.nvfp4_test_withhold_arrivals(0)
    again = call()
    after = B.get_device_error()
    torch.cuda.synchronize()
    print("RESULT", name, clean, timed_out, after, int(torch.equal(again, ref)), flush=True)
"""


def run(tmp_path, body, names):
    script = tmp_path / "child.py"
    script.write_text(HEAD.format(root=ROOT) + body)
    env = dict(os.environ, NVFP4_WAIT_TIMEOUT_MS="100")
    res = subprocess.run([sys.executable, str(script)], env=env, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    from epilogue_gemm_nvfp4_b200 import binding as B
    results = [line.split()[1:] for line in res.stdout.splitlines() if line.startswith("RESULT")]
    assert [r[0] for r in results] == names, res.stdout + res.stderr
    for name, clean, timed_out, after, same in results:
        assert int(clean) == B.OK, (name, clean)
        assert int(timed_out) == B.ERR_DEVICE_TIMEOUT, (name, timed_out)
        assert int(after) == B.OK, (name, after)
        assert same == "1", name


W4A16 = r"""
# one chunk of K per unit and at least three units per CTA on up to 160 SMs, fewer than its ring's stages: all loads are out before
# the wait for the third accumulator (of two; the second of one for 32 rows)
w = B.quantize(torch.randn(256 * 160 * 3, 256, device="cuda").bfloat16())
for M in (1, 3, 12, 32):   # digits made in the product kernel's own CTAs, and by a kernel before it
    x = torch.randn(M, 256, device="cuda").bfloat16()
    check(f"rows{M}", lambda: B.w4a16_linear(x, w))
"""


def test_few_row_linear_reports_a_wait_that_runs_out(tmp_path):
    run(tmp_path, W4A16, ["rows1", "rows3", "rows12", "rows32"])


ATTENTION = r"""
lens = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
for D in (64, 128, 256):
    # tiles, alone and split over a cluster; pieces of two tiles, more than one per CTA or pair; keys whose loads are all out at
    # once and keys that go round the ring; lengths that end inside a tile (V rows cleared), and none
    for name, B_, Mq, Mk, H, n in (("tile", 1, 64, 128, 1, None), ("split", 1, 3, 1300, 2, None), ("pieces", 2, 3000, 128, 8, None),
                                   ("ring", 2, 3000, 900, 8, (900, 333)), ("none", 3, 2000, 200, 8, (0, 200, 7))):
        q, k, v = r(B_, Mq, H, D), r(B_, Mk, H, D), r(B_, Mk, H, D)
        n = n and lens(*n)
        check(f"{name}{D}", lambda: B.cross_attention(q, k, v, kv_lens=n))
"""


def test_attention_reports_a_wait_that_runs_out(tmp_path):
    run(tmp_path, ATTENTION, [f"{name}{D}" for D in (64, 128, 256) for name in ("tile", "split", "pieces", "ring", "none")])
