"""A call's result is that of its own launch, not of an earlier call that
failed on the host. In a process of its own: the failing call ends a capture."""
import os
import subprocess
import sys

import pytest

from helpers import need_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = r"""
import torch, invariant_gemm_gb300 as ig, synth
u8, b16 = torch.uint8, torch.bfloat16
x = torch.randn(16, 1024, device="cuda").to(b16)
w = torch.randn(64, 1024, device="cuda").to(b16)
new = lambda v: (torch.empty(v.shape[0], 512, dtype=u8, device="cuda"),
                 torch.empty(ig.mx4_scale_bytes(v.shape[0], 1024), dtype=u8, device="cuda"))
xq, wq, one = new(x), new(w), torch.ones(1024, dtype=b16, device="cuda")
y, n = torch.empty(16, 64, device="cuda"), torch.empty_like(x)
ws = ig.mx4_workspace()
p = synth.make_problem(16, 1024, 512, 16, L=2, seed=1, device="cuda")
lora = {}
for name, kw in dict(fused={}, two=dict(flags=ig.FLAG_UNFUSED), tree=dict(mode=ig.MODE_DET_TREE),
                     fma=dict(path=ig.PATH_FMA)).items():
    sh = ig.make_shape(p.M, p.K, p.N, p.r, num_adapters=p.L, split_k=4, **kw)
    lora[name] = (sh, ig.workspace(sh))
z = torch.empty(p.slices, p.M, p.r, device="cuda")

calls = [lambda: ig.mx4_quantize(x, *xq), lambda: ig.mx4_quantize(w, *wq),
         lambda: ig.mx4_dequantize(*xq, x), lambda: ig.block_norm(x, None, None, one, n_out=n),
         lambda: ig.mx4_gemm(*xq, *wq, y, ws)]
calls += [lambda a=a: ig.lora_apply(a[0], p.x, p.y, p.idx, p.A, p.B, p.scale, z, a[1])
          for a in lora.values()]
for c in calls:
    c()
torch.cuda.synchronize()
for i, c in enumerate(calls):
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        failed = ig.check_status(ws)         # a stream that is captured cannot be waited for
        try:
            graph.capture_end()
        except RuntimeError:
            pass
    assert failed == -5, failed
    c()                                      # raises where the old error is taken for its own
    torch.cuda.synchronize()
print("all", len(calls))
"""


@pytest.mark.gpu
def test_an_earlier_failure_is_not_reported_again():
    need_gpu()
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "all 9" in r.stdout
