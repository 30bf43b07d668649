"""The first call of a process made inside a graph capture: what the calls look up once
(opt-ins, resident clusters, the tensor maps' encoder) is looked up there too."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
import combine_topk_idx_gb300 as ep
from tests.ops_harness import routing
g = torch.Generator().manual_seed(1)
def normal(*s):
    return torch.randn(*s, generator=g).bfloat16().cuda()
what = {what!r}
rows = {rows}
x, w, gy = normal(rows, 256), normal(512, 256), normal(rows, 512)
torch.cuda.synchronize()
if what == "clip":
    call = lambda: ep.ep_clip_grads([x], 1.0, out=[out])
    out = torch.zeros_like(x)
elif what == "layout":
    h = ep.ep_layout(ep.make_config(rows, 2, 4, 1, 256, rows, 8, do_expand=True,
                                    do_cpu_sync=False), routing(rows, 2, 4, 3).cuda())
    gy, x = normal(h.rows_alloc, 512), normal(h.rows_alloc, 256)
    out = torch.zeros(4, 512, 256, device="cuda")
    call = lambda: ep.ep_ffn_weight_grad(h, gy, x, out)
else:
    out = torch.zeros(rows, 256, dtype=torch.bfloat16, device="cuda")
    call = lambda: ep.ep_ffn_gated(None, x, w, act=out)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = out.clone()
out.zero_()
call()
torch.cuda.synchronize()
assert got.any() and torch.equal(got, out)
print("the same")
"""


@pytest.mark.parametrize("what,rows", [("gated", 30), ("gated", 2000), ("layout", 700),
                                       ("clip", 40), ("clip", 20000)])
def test_first_call_captured(what, rows):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(what=what, rows=rows)], cwd=ROOT,
                       capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]
