"""Operators around the linears whose first call in a process is made under graph capture, and two captured graphs whose replays
overlap.  The first runs in a child process: nothing of the library has been called before."""
import os
import subprocess
import sys

import pytest
import torch

from epilogue_gemm_nvfp4_b200 import binding as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import torch
from epilogue_gemm_nvfp4_b200 import binding as B

r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
N, K = 640, 4608
w = B.QTensor(torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda"),
              torch.randint(0, 127, (-(-N // 128) * (K // 64) * 512,), dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"), N, K)
cos = torch.rand(50, 64, device="cuda")
calls = {{
    "w1": (lambda x: B.w4a16_linear(x, w), r(1, K)), "w7": (lambda x: B.w4a16_linear(x, w), r(7, K)),
    "w32": (lambda x: B.w4a16_linear(x, w), r(32, K)),
    "rope": (lambda x: B.qk_norm_rope(x, x, cos, cos, gamma_q=x[0, 0], gamma_k=x[1, 0]), r(50, 3, 128)),
    "few64": (lambda x: B.cross_attention(x, x, x), r(1, 200, 2, 64)), "few256": (lambda x: B.cross_attention(x, x, x), r(1, 200, 2, 256)),
    "many64": (lambda x: B.cross_attention(x, x, x), r(2, 1500, 16, 64)), "many128": (lambda x: B.cross_attention(x, x, x), r(2, 1500, 16, 128)),
    "many256": (lambda x: B.cross_attention(x, x, x), r(2, 1500, 16, 256)),
}}
torch.cuda.synchronize()
for name, (f, x) in calls.items():
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(x)
    x.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    want = f(x)
    same = all(torch.equal(a, b) for a, b in zip(out, want)) if isinstance(out, tuple) else torch.equal(out, want)
    print("RESULT", name, int(same), B.get_device_error(), flush=True)
"""

NAMES = ["w1", "w7", "w32", "rope", "few64", "few256", "many64", "many128", "many256"]


def test_first_call_under_capture(tmp_path):
    script = tmp_path / "child.py"
    script.write_text(CHILD.format(root=ROOT))
    res = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    results = [line.split()[1:] for line in res.stdout.splitlines() if line.startswith("RESULT")]
    assert [r[0] for r in results] == NAMES and all(r[1] == "1" and int(r[2]) == B.OK for r in results), res.stdout


def test_two_graphs_replayed_at_once():
    """Each graph has workspaces of its own; replays of both on two streams keep their bits."""
    r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    w = B.quantize(r(4608, 4608))
    pos = torch.randint(-1, 40, (900,), device="cuda", dtype=torch.int32)
    cos = torch.rand(40, 32, device="cuda")

    def block(x, q):
        y = B.w4a16_linear(x, w, silu_input=True)
        k, _ = B.qk_norm_rope(q, None, cos, cos, positions=pos, gamma_q=y[0, :128])
        return y, k, B.cross_attention(k[None], q[None], q[None]), B.w4a16_linear(y, w)
    inputs = [(r(5, 4608), r(900, 6, 128)) for _ in range(2)]
    want = [block(*i) for i in inputs]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, i in zip(graphs, inputs):
        with torch.cuda.graph(g):
            outs.append(block(*i))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    B.check_device_error()
