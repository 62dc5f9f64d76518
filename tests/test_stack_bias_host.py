"""The stack's bookkeeping of a shared position bias, on the CPU, with layers that only note the bias they were given
and refuse one where they are told to."""
import pytest
import torch

import transformer_layer_pre_b200 as tlp
from transformer_layer_pre_b200 import stack as stack_module
from transformer_layer_pre_b200.stack import EncoderStack


class _NotingLayer:
    refuses = False
    held = None

    def __init__(self, batch, seq, hidden, heads, ffn=0, *rest, **options):
        self.ffn = ffn

    def set_position_bias(self, table, max_distance=128, dtable=None, accumulate=False):
        if self.refuses and table is not None:
            raise tlp.TlError(2, "refused")
        self.held = None if table is None else (table, max_distance, dtable)

    def close(self):
        pass


@pytest.fixture
def stack(monkeypatch):
    monkeypatch.setattr(stack_module, "Layer", _NotingLayer)
    return EncoderStack(3, 2, 16, 64, 4, 64, device="cpu", share_scratch=False)


@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("earlier", [False, True])
def test_a_refused_table_leaves_the_earlier_one(stack, at, earlier):
    first = torch.zeros(32, 4)
    if earlier:
        stack.set_position_bias(first, 100)
    before = stack.position_bias_grad
    stack.layers[at].refuses = True
    with pytest.raises(tlp.TlError):
        stack.set_position_bias(torch.zeros(64, 4))
    assert stack.position_bias_grad is before
    if earlier:
        assert all(t is first and m == 100 and g is before for t, m, g in [layer.held for layer in stack.layers])
    else:
        assert before is None and [layer.held for layer in stack.layers] == [None, None, None]


def test_layers_share_the_gradient_that_the_stack_returns(stack):
    table = torch.zeros(32, 4)
    stack.set_position_bias(table, 100)
    assert stack.position_bias_grad.shape == table.shape and stack.position_bias_grad.dtype == torch.float32
    assert all(t is table and m == 100 and g is stack.position_bias_grad for t, m, g in [layer.held for layer in stack.layers])
    stack.set_position_bias(None)
    assert stack.position_bias_grad is None and [layer.held for layer in stack.layers] == [None, None, None]
