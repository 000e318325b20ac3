"""The losses at the output head in CUDA graphs: fp32 steps that follow their inputs, and a
process whose first call of all is captured."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.block_common import status_ok  # noqa: E402
from tests.loss_common import bounds, check, device, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import orthogonal_reparameterized_packed_gb300 as poetx
    poetx.load_library()
    return poetx


# products on the CUDA cores and on the tensor cores, one block and several
@pytest.mark.parametrize("tau", [None, 2.0])
@pytest.mark.parametrize("T,d,V,block", [(100, 72, 500, None), (515, 512, 3001, None),
                                         (515, 512, 3001, 256)])
def test_fp32_steps_follow_their_inputs(px, T, d, V, block, tau):
    from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
    K = 1 if tau is None else 5
    kw = dict(dtype="f32", backward=True, weight_grad=True, block_tokens=block)
    h = (PoetxCrossEntropy(d, V, T, **kw) if tau is None else
         PoetxDistill(d, V, T, top=K, temperature=tau, **kw))
    c = make(T, d, V, K, "f32", seed=0)
    x, W, rest = c["x"][0].clone(), c["W"][0].clone(), device(c, tau is not None)
    h.step(x, W, *rest)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.step(x, W, *rest)
    # some tokens count; none does; a value that the tensor cores do not take, and then not
    for seed, ignored, tiny in ((1, 0.3, False), (2, 1.0, False), (3, 0.0, True), (4, 0.1, False)):
        n = make(T, d, V, K, "f32", seed=seed, ignored=ignored)
        if tiny:
            t = n["W"][0].clone()
            t[7, :5] = 1e-36
            n["W"] = (t, t.double().cpu().numpy())
        x.copy_(n["x"][0])
        W.copy_(n["W"][0])
        for a, b in zip(rest, device(n, tau is not None)):
            a.copy_(b)
        graph.replay()
        status_ok(px)
        want, bound = bounds(n, tau or 1.0, None, n["s"] if tau else np.zeros(n["idx"].shape))
        check((h.loss, h.total, h.dx, h.dW), want, bound)


FIRST = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import orthogonal_reparameterized_packed_gb300 as px
from orthogonal_reparameterized_packed_gb300.loss import PoetxCrossEntropy, PoetxDistill
for dtype in ("bf16", "f32"):
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((515, 512), generator=g, device="cuda").to(t)
    W = (torch.randn((3001, 512), generator=g, device="cuda") / 16).to(t)
    y = torch.randint(0, 3001, (515,), generator=g, device="cuda")
    i = torch.randint(0, 3001, (515, 4), generator=g, device="cuda")
    s = torch.randn((515, 4), generator=g, device="cuda")
    kw = dict(dtype=dtype, backward=True, weight_grad=True)
    ce, kd = PoetxCrossEntropy(512, 3001, 515, **kw), PoetxDistill(512, 3001, 515, top=4, **kw)
    few = PoetxCrossEntropy(512, 3001, 8, dtype=dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ce.step(x, W, y)
        kd.step(x, W, i, s)
        few.forward(x[:8], W, y[:8])
    graph.replay()
    torch.cuda.synchronize()
    outs = [v.clone() for v in (ce.loss, ce.dx, ce.dW, kd.loss, kd.dx, kd.dW, few.loss)]
    ce.step(x, W, y)
    kd.step(x, W, i, s)
    few.forward(x[:8], W, y[:8])
    torch.cuda.synchronize()
    for a, b in zip(outs, (ce.loss, ce.dx, ce.dW, kd.loss, kd.dx, kd.dW, few.loss)):
        assert a.isfinite().all() and a.any() and torch.equal(a, b)
assert px.poetx_device_status() == 0
print("captured first")
"""


def test_the_first_call_of_a_process_is_captured(px):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST, root], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
