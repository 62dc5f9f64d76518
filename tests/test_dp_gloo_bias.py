"""Data-parallel exchange of a stack with a shared position bias, two gloo ranks on the CPU: every layer's gradients and
the table's are averaged, in the same order on both ranks, with a layer skipped."""
import os
import socket

import torch
import torch.distributed as dist
import torch.multiprocessing as mp


class _AddingLayer:
    """Writes rank-dependent gradients, adds to the shared table's as the layer's backward does."""

    def __init__(self, batch, seq, hidden, heads, ffn=0, *rest, **options):
        self.ffn = ffn

    def set_position_bias(self, table, max_distance=128, dtable=None, accumulate=False):
        self.dtable = dtable

    def forward(self, x, mask, weights, y=None, stream=None):
        return x

    def backward(self, x, dy, weights, grads=None, dx=None, stream=None):
        for t in grads.values():
            t.fill_(weights + dist.get_rank())
        self.dtable.add_(weights * 100 + 2 * dist.get_rank())
        return dy, grads


def _worker(rank, port, q):
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path[:0] = [root, os.path.join(root, "tests")]
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE="2")
    dist.init_process_group("gloo", rank=rank, world_size=2)
    try:
        from transformer_layer_pre_b200 import stack as module
        module.Layer = _AddingLayer
        st = module.EncoderStack(3, 2, 16, 64, 4, 64, device="cpu", share_scratch=False)
        st.set_position_bias(torch.zeros(32, 4))
        x = torch.zeros(2, 16, 64)
        got = []
        for _ in range(2):                       # the second step begins at zero again
            st.forward(x, None, [1.0, 2.0, 3.0], keep=[True, False, True])
            st.backward(x, [1.0, 2.0, 3.0], exchange=True)
            got.append((st.position_bias_grad.clone(), [float(g["w1"][0, 0]) for g in st.grads]))
        ok = all(bool((t == 100 + 300 + 2 * 2 * 0.5).all()) and g == [1.5, 0.0, 3.5] for t, g in got)
        q.put((rank, ok, [float(t[0, 0]) for t, _ in got], [g for _, g in got]))
    finally:
        dist.destroy_process_group()


def test_table_gradient_is_averaged_with_the_layers():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_worker, args=(r, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    res = [q.get(timeout=120) for _ in procs]
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    assert all(r[1] for r in res), res
