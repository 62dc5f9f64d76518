"""What a refused position bias leaves behind, in the layer and in the stack; the stack's bias on a stream of the
caller's; the exchange of the shared table's gradient."""
import os
import subprocess
import sys

import pytest
import torch

import transformer_layer_pre_b200 as tlp
from transformer_layer_pre_b200 import Layer
from transformer_layer_pre_b200.dp import gradient_shapes

pytestmark = pytest.mark.gpu
TL_ENOMEM = 2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _weights(h, f, g, dtype=torch.float16):
    return {n: (0.1 * torch.randn(s, generator=g, device="cuda")).to(dtype) for n, s in gradient_shapes(h, f).items()}


CHILD = """
import torch
import transformer_layer_pre_b200 as tlp
from test_gpu_position_bias_state import _weights, TL_ENOMEM
g = torch.Generator(device="cuda").manual_seed(3)
wt = _weights(64, 64, g)
x = torch.randn(1, 304, 64, generator=g, device="cuda").half()
small, large = (torch.randn(n, 1, generator=g, device="cuda").half() for n in (4, 256))
layer = tlp.Layer(1, 304, 64, 1, 64, dtype=torch.float16)
layer.set_position_bias(small, 100)
before = layer.forward(x, None, wt).clone()
plain = tlp.Layer(1, 304, 64, 1, 64, dtype=torch.float16).forward(x, None, wt)
torch.cuda.synchronize()
status = None
graph = torch.cuda.CUDAGraph()
try:
    with torch.cuda.graph(graph):          # an allocation is an error while a stream is captured
        try:
            layer.set_position_bias(large, 100)
        except tlp.TlError as e:
            status = e.status
except Exception:
    pass                                   # the capture is broken off
torch.cuda.synchronize()
after = layer.forward(x, None, wt)
torch.cuda.synchronize()
assert status == TL_ENOMEM, status
assert not torch.equal(before, plain) and torch.equal(before, after)
layer.set_position_bias(large, 100)
assert not torch.equal(before, layer.forward(x, None, wt))
tlp.device_check()
print("kept")
"""


def test_a_failed_allocation_keeps_the_bias():
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, env=env, cwd=ROOT)
    assert r.returncode == 0 and "kept" in r.stdout, r.stdout + r.stderr


def test_a_table_on_another_device_than_the_current_one(monkeypatch):
    """The layer works on the current device (its own, or an error); a table elsewhere is no table of it."""
    layer = Layer(1, 16, 64, 1, 64, dtype=torch.float16)
    try:
        table = torch.zeros(32, 1, dtype=torch.float16, device="cuda")
        layer.set_position_bias(table)
        other = table.get_device() + 1
        monkeypatch.setattr(torch.cuda, "current_device", lambda: other)
        with pytest.raises(tlp.TlError, match="device"):
            layer.set_position_bias(table)
    finally:
        monkeypatch.undo()
        layer.close()


def test_stack_on_a_stream_of_the_callers_with_an_exchange():
    """Forward, backward and clipping on an explicit stream, with a stand-in collective that adds an identical rank: the
    bits of the step on the current stream, the table's gradient exchanged last and after it was written."""
    from transformer_layer_pre_b200.dp import GradExchanger
    from transformer_layer_pre_b200.stack import EncoderStack
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(2, 200, 128, generator=g, device="cuda").half() for _ in range(2))
    wts = [_weights(128, 256, g) for _ in range(2)]
    table = torch.randn(32, 2, generator=g, device="cuda").half()
    st = EncoderStack(2, 2, 200, 128, 2, 256, dtype=torch.float16)
    seen = []

    def identical_rank(t):
        torch.cuda._sleep(20_000_000)            # a slow collective
        seen.append(t.clone())
        t.add_(t)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (y, dx, norm, st.position_bias_grad, *(f.flat for f in st.grads))]

    try:
        st.set_position_bias(table)
        y = st.forward(x, None, wts)
        dx, _ = st.backward(dy, wts)
        unclipped = st.position_bias_grad.clone()
        norm = st.clip_grad_norm(0.5)
        want = results()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        for _ in range(2):
            y = st.forward(x, None, wts, stream=stream)
            dx, _ = st.backward(dy, wts, exchange=GradExchanger(allreduce=identical_rank, world=2), stream=stream)
            norm = st.clip_grad_norm(0.5, stream=stream)
            assert all(torch.equal(a, b) for a, b in zip(results(), want))
        assert len(seen) == 6 and torch.equal(seen[2], unclipped) and torch.equal(seen[5], unclipped)
        tlp.device_check()
    finally:
        st.close()
