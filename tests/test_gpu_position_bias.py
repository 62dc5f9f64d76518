"""The layer and the stack with a learned relative position bias, against the
same layer written in float64 and differentiated by autograd, within the
parity bars of the plain layer (parity.py): float32 max error 1e-5 of the
largest value, 16-bit relative Frobenius error 1e-2; and the whole training
step: forward, backward, gradient clipping."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref
import transformer_layer_pre_b200 as tlp
from parity import REL_FROB, REL_MAX_F32, TORCH_DT
from transformer_layer_pre_b200 import WEIGHT_NAMES, Layer
from transformer_layer_pre_b200.stack import EncoderStack
from transformer_layer_pre_b200.synthetic import Workload, make_inputs, with_random_affine

pytestmark = pytest.mark.gpu
TL_EUNSUPPORTED, TL_ESTATE, TL_EINVAL = 6, 3, 1

CASES = [
    Workload("bias-f32", 2, 24, 64, 4, 136, "f32", 0.0, 0.0, lengths=(9, 24)),
    Workload("bias-post-f32", 2, 72, 96, 3, 200, "f32", 0.0, 0.0, pre_layer_norm=False),
    Workload("bias-f16", 3, 136, 192, 3, 520, "f16", 0.0, 0.0, lengths=(40, 136)),
    Workload("bias-post-bf16", 2, 264, 128, 2, 256, "bf16", 0.0, 0.0, pre_layer_norm=False, lengths=(130, 264)),
    Workload("bias-d128-f16", 2, 200, 256, 2, 512, "f16", 0.0, 0.0, lengths=(1, 200)),
    Workload("bias-d32-bf16", 2, 40, 128, 4, 256, "bf16", 0.0, 0.0),
]


def _norm(x, g, b, eps=1e-12):
    m = x.mean(-1, keepdim=True)
    v = ((x - m) ** 2).mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(v + eps) * g + b


def _layer64(w, wt, x, mask, table, distance):
    b, s, h = x.shape
    d = h // w.heads
    bias = table.t()[:, ref.bucket_matrix(s, table.shape[0], distance, x.device)]

    def attention(y):
        q, k, v = (t.view(b, s, w.heads, d).transpose(1, 2) for t in (y @ wt["wqkv"].t() + wt["bqkv"]).split(h, -1))
        z = q @ k.transpose(2, 3) / math.sqrt(d) + bias
        if mask is not None:
            z = z + mask[:, None, None]
        return (torch.softmax(z, -1) @ v).transpose(1, 2).reshape(b, s, h) @ wt["wo"].t() + wt["bo"]

    def ffn(y):
        u = y @ wt["w1"].t() + wt["b1"]
        return (u * 0.5 * (1 + torch.erf(u / math.sqrt(2)))) @ wt["w2"].t() + wt["b2"]

    if w.pre_layer_norm:
        x = x + attention(_norm(x, wt["ln1_g"], wt["ln1_b"]))
        return x + ffn(_norm(x, wt["ln2_g"], wt["ln2_b"]))
    x = _norm(x + attention(x), wt["ln1_g"], wt["ln1_b"])
    return _norm(x + ffn(x), wt["ln2_g"], wt["ln2_b"])


def _close(name, got, want, dtype):
    got, want = got.double().cpu(), want.detach().cpu()
    if dtype == "f32":
        assert float((got - want).abs().max()) <= REL_MAX_F32 * float(want.abs().max()), name
    else:
        assert float((got - want).norm()) <= REL_FROB * float(want.norm()), name


def _setup(w, buckets=16, seed=5):
    inp = with_random_affine(make_inputs(w))
    dev = torch.device("cuda", 0)
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn(buckets, w.heads, generator=g, device=dev).to(TORCH_DT[w.dtype])
    wts = [{n: t.to(dev) for n, t in l.items()} for l in inp.weights]
    mask = None if inp.mask is None else inp.mask.to(dev)
    return inp, dev, table, wts, mask


@pytest.mark.parametrize("w", CASES, ids=lambda w: w.name)
def test_layer_with_a_position_bias(w):
    inp, dev, table, wts, mask = _setup(w)
    x, dy = inp.x.to(dev), inp.dy.to(dev)
    dtable = torch.full((16, w.heads), 3.0, device=dev)
    layer = Layer(w.batch, w.seq, w.hidden, w.heads, w.ffn, 0.0, 0.0, w.pre_layer_norm, w.seed, dtype=TORCH_DT[w.dtype])
    try:
        plain = layer.forward(x, mask, wts[0]).clone()
        layer.set_position_bias(table, 40, dtable)
        with pytest.raises(tlp.TlError) as e:      # the plain forward's activations are gone
            layer.backward(x, dy, wts[0])
        assert e.value.status == TL_ESTATE
        y = layer.forward(x, mask, wts[0])
        dx, grads = layer.backward(x, dy, wts[0])
        first = dtable.clone()
        layer.set_position_bias(table, 40, dtable, accumulate=True)
        layer.forward(x, mask, wts[0])
        layer.backward(x, dy, wts[0])
        tlp.device_check()
        layer.set_position_bias(None)
        assert torch.equal(layer.forward(x, mask, wts[0]), plain)
        layer.set_position_bias(table, 40)          # no gradient wanted
        layer.forward(x, mask, wts[0])
        dx2, _ = layer.backward(x, dy, wts[0])
        assert torch.equal(dx, dx2)
    finally:
        layer.close()
    p64 = {n: t.double().requires_grad_() for n, t in wts[0].items()}
    x64, t64 = x.double().requires_grad_(), table.double().requires_grad_()
    y64 = _layer64(w, p64, x64, None if mask is None else mask.double(), t64, 40)
    y64.backward(dy.double())
    _close("y", y, y64, w.dtype)
    _close("dx", dx, x64.grad, w.dtype)
    for n in WEIGHT_NAMES:
        _close(n, grads[n], p64[n].grad, w.dtype)
    _close("dtable", first, t64.grad, w.dtype)
    assert float((dtable - 2 * first).abs().max()) <= 2.0 ** -22 * float(first.abs().max())
    assert not torch.equal(plain, y)


def test_stack_step_with_bias_and_clipping():
    """Shared table over the layers, one skipped; then clipping over everything that ran."""
    w = Workload("bias-stack-f16", 2, 72, 128, 2, 256, "f16", 0.0, 0.0, lengths=(30, 72), layers=3)
    inp, dev, table, wts, mask = _setup(w, buckets=32)
    keep = [True, False, True]
    x, dy = inp.x.to(dev), inp.dy.to(dev)
    st = EncoderStack(3, w.batch, w.seq, w.hidden, w.heads, w.ffn, 0.0, 0.0, True, w.seed, dtype=torch.float16)
    try:
        assert st.position_bias_grad is None
        st.set_position_bias(table)
        out = []
        for _ in range(2):                       # the table's gradient is overwritten, not added to
            y = st.forward(x, mask, wts, keep=keep)
            dx, grads = st.backward(dy, wts)
            out.append((y.clone(), dx.clone(), st.position_bias_grad.clone()))
        assert all(torch.equal(a, b) for a, b in zip(*out))
        flat = [g.flat.clone() for g in st.grads]
        ran = [flat[0], flat[2], st.position_bias_grad.clone()]
        total = math.sqrt(sum(float(t.double().square().sum()) for t in ran))
        norm = st.clip_grad_norm(0.5 * total)
        assert abs(float(norm) - total) <= 2.0 ** -23 * total
        after = [st.grads[0].flat, st.grads[2].flat, st.position_bias_grad]
        for a, b in zip(after, ran):
            assert float((a - 0.5 * b).abs().max()) <= 2.0 ** -20 * float(b.abs().max())
        assert torch.equal(st.grads[1].flat, flat[1])
        assert float(st.clip_grad_norm(2 * total)) <= 0.5 * total * (1 + 2.0 ** -20)
        st.set_position_bias(None)
        assert st.position_bias_grad is None
    finally:
        st.close()
    p64 = [{n: t.double().requires_grad_() for n, t in l.items()} for l in wts]
    x64, t64 = x.double().requires_grad_(), table.double().requires_grad_()
    h = x64
    for l in (0, 2):
        h = _layer64(w, p64[l], h, mask.double(), t64, 128)
    h.backward(dy.double())
    _close("y", out[0][0], h, "f16")
    _close("dx", out[0][1], x64.grad, "f16")
    _close("dtable", out[0][2], t64.grad, "f16")
    for l, f in ((0, flat[0]), (2, flat[2])):
        want = torch.cat([p64[l][n].grad.reshape(-1) for n in WEIGHT_NAMES])
        got = torch.cat([st.grads[l][n].reshape(-1) for n in WEIGHT_NAMES])
        _close(f"grads[{l}]", 2 * got, want, "f16")


def test_captured_training_step_follows_its_inputs():
    """Two layers' forward, backward and clipping in a graph, replayed on other inputs."""
    w = Workload("bias-graph-bf16", 2, 136, 128, 2, 256, "bf16", 0.0, 0.0, layers=2)
    inp, dev, table, wts, mask = _setup(w, buckets=32)
    g = torch.Generator(device="cuda").manual_seed(1)
    st = EncoderStack(2, w.batch, w.seq, w.hidden, w.heads, w.ffn, dtype=torch.bfloat16)
    try:
        st.set_position_bias(table)
        x, dy = inp.x.to(dev).clone(), inp.dy.to(dev).clone()

        def step():
            y = st.forward(x, mask, wts)
            dx, _ = st.backward(dy, wts)
            return y, dx, st.clip_grad_norm(0.1)

        def results():
            torch.cuda.synchronize()
            return [t.clone() for t in (*out, st.grads[0].flat, st.grads[1].flat, st.position_bias_grad, )]

        sets = [[torch.randn(x.shape, generator=g, device=dev).bfloat16() for _ in range(2)] for _ in range(2)]
        want = []
        for a, b in sets:
            x.copy_(a)
            dy.copy_(b)
            out = step()
            want.append(results())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for (a, b), ref_ in list(zip(sets, want)) * 2:
            x.copy_(a)
            dy.copy_(b)
            graph.replay()
            assert all(torch.equal(i, j) for i, j in zip(results(), ref_))
        del graph
    finally:
        st.close()


def test_dropout_and_bad_tables_are_refused():
    dev = torch.device("cuda", 0)
    x = torch.zeros(1, 16, 64, dtype=torch.float16, device=dev)
    wt = {n: torch.zeros(s, dtype=torch.float16, device=dev) for n, s in tlp_shapes().items()}
    table = torch.zeros(32, 1, dtype=torch.float16, device=dev)
    layer = Layer(1, 16, 64, 1, 64, attn_dropout=0.1, dtype=torch.float16)
    try:
        layer.set_position_bias(table)
        with pytest.raises(tlp.TlError) as e:
            layer.forward(x, None, wt)
        assert e.value.status == TL_EUNSUPPORTED
        for bad in (table.float(), table[:31], table[:2], torch.zeros(32, 2, dtype=torch.float16, device=dev), table.cpu()):
            with pytest.raises(tlp.TlError):
                layer.set_position_bias(bad)
        with pytest.raises(tlp.TlError):
            layer.set_position_bias(table, 8)
        with pytest.raises(tlp.TlError):
            layer.set_position_bias(table, dtable=torch.zeros(32, 1, dtype=torch.float16, device=dev))
    finally:
        layer.close()
    infer = Layer(1, 16, 64, 1, 64, attn_dropout=0.1, dtype=torch.float16, training=False)
    try:
        infer.set_position_bias(table)
        infer.forward(x, None, wt)
        torch.cuda.synchronize()
    finally:
        infer.close()


def tlp_shapes():
    from transformer_layer_pre_b200.dp import gradient_shapes
    return gradient_shapes(64, 64)
