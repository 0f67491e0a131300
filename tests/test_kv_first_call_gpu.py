"""A handle's first shaped attention, which loads its kernels, under capture: a process of its own, in which nothing has loaded
them before."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

PROGRAM = """
import torch
import hybrid_draft_tree_gb300 as g
eight, shape = {eight}, dict({shape})
gen = torch.Generator(device="cuda").manual_seed(3)
kv = g.GraftKV(g.graft_kv_default_config(8, 2, {dim}, 16, 40, 2, 5, cache="e4m3" if eight else None))
cache = torch.randn((40, 2, 16, {dim}), generator=gen, device="cuda").to(torch.float8_e4m3fn if eight else torch.bfloat16)
q = torch.randn((10, 8 * {dim}), generator=gen, device="cuda").to(torch.bfloat16)
table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
ctx = torch.tensor([300, 7], dtype=torch.int32, device="cuda")
if shape.pop("alibi", 0):
    shape["slopes"] = torch.full((8,), 0.25, device="cuda")
outs = [torch.zeros_like(q) for _ in range(2)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    kv.attend(2, 5, q, cache, cache, table, ctx, 300, outs[0], **shape)
graph.replay()
kv.attend(2, 5, q, cache, cache, table, ctx, 300, outs[1], **shape)
assert kv.sync() == 0 and torch.equal(*outs) and outs[0].abs().sum() > 0 and torch.isfinite(outs[0]).all()
print("right")
"""


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("shape", ["window=50", "softcap=5.0", "softcap=1e6", "alibi=1, window=9", ""])
def test_the_first_shaped_call_may_be_captured(cuda_ok, eight, shape):
    run = subprocess.run([sys.executable, "-c", PROGRAM.format(eight=eight, shape=shape, dim=64 if "=5" in shape else 128)],
                         capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.strip() == "right", run.stderr[-2000:]
