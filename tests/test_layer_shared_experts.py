"""Whose activations the shared expert tensors hold: a backward of a forward that is gone, and a checkpoint that
holds another one or none, are refused before anything is launched.  The library's calls are stood in for; CPU only."""
import pytest

from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import layer

SIZE = (8, 64, 8, 2, 64, "bf16", "cpu")
GATE = layer.GroupGate()


class Calls:
    """The binding's constants, and calls that are noted and do nothing."""

    def __init__(self):
        self.made, self.fails = [], None

    def __getattr__(self, name):
        if name.startswith("MOE_") or name == "moe_workspace_bytes":
            return getattr(L, name)

        def call(*args, **kw):
            if name == self.fails:
                raise L.MoEError(name, L.MOE_ERR_CUDA, "stood in for")
            self.made.append(name)
        return call


@pytest.fixture
def calls(monkeypatch):
    from token_dispatch_gb300 import build
    build.build()
    c = Calls()
    monkeypatch.setattr(layer, "L", c)
    return c


def forward(b):
    layer.moe_forward(b, None, None, None, None, None, None)


def backward(b):
    layer.moe_train_backward(b, None, None, None, None, None, None)


def block_forward(m, **kw):
    layer.moe_block_forward(m, None, None, None, None, GATE, None, None, None, **kw)


def block_backward(m, **kw):
    layer.moe_block_backward(m, None, None, None, GATE, None, None, None, None, **kw)


def refused(calls, f, *args, **kw):
    n = len(calls.made)
    with pytest.raises(ValueError):
        f(*args, **kw)
    assert len(calls.made) == n


def test_layers_that_share_expert_tensors(calls):
    one = layer.MoEBuffers(*SIZE, train=True)
    two = layer.MoEBuffers(*SIZE, train=True, experts=one)
    refused(calls, backward, one)  # no forward yet
    forward(one)
    backward(one)
    backward(one)  # a backward leaves what it reads
    forward(two)
    refused(calls, backward, one)
    backward(two)
    forward(one)
    backward(one)
    refused(calls, backward, two)


def test_a_layer_by_itself_asks_nothing(calls):
    b = layer.MoEBuffers(*SIZE, train=True)
    backward(b)  # its forward may have been launched call by call


def test_layer_and_block_on_shared_tensors(calls):
    block = layer.MoEBlockBuffers(*SIZE, train=True)
    other = layer.MoEBuffers(*SIZE, train=True, experts=block.moe)
    ck = layer.ExpertCheckpoint(block.moe)
    block_forward(block)
    block_backward(block)
    block_forward(block, ckpt=ck)
    forward(other)
    refused(calls, block_backward, block)
    refused(calls, ck.save, block.moe)  # the tensors are the other's now
    block_backward(block, ckpt=ck)
    block_backward(block)  # restored
    refused(calls, backward, other)
    forward(block.moe)  # the layer's own call in the block's buffers: the block's norms are of the forward before
    refused(calls, block_backward, block)
    refused(calls, block_backward, block, ckpt=ck)


def test_checkpoints_of_nothing_and_of_another_forward(calls):
    one = layer.MoEBlockBuffers(*SIZE, train=True)
    two = layer.MoEBlockBuffers(*SIZE, train=True, experts=one.moe)
    a, b = layer.ExpertCheckpoint(one.moe), layer.ExpertCheckpoint(two.moe)
    block_forward(one)
    refused(calls, a.restore, one.moe)  # never saved
    refused(calls, block_backward, one, ckpt=a)
    block_forward(one, ckpt=a)
    block_forward(two, ckpt=b)
    refused(calls, block_backward, one, ckpt=b)
    block_backward(two, ckpt=b)
    block_backward(one, ckpt=a)
    block_forward(one)  # a second batch, not saved
    refused(calls, block_backward, one, ckpt=a)
    block_backward(one)


@pytest.mark.parametrize("at", ["moe_route_group", "moe_dispatch", "moe_expert_ffn_ex"])
def test_a_forward_that_ended_early(calls, at):
    one = layer.MoEBlockBuffers(*SIZE, train=True)
    two = layer.MoEBlockBuffers(*SIZE, train=True, experts=one.moe)
    block_forward(one)
    calls.fails = at
    with pytest.raises(L.MoEError):
        block_forward(two)
    calls.fails = None
    refused(calls, block_backward, one)
    refused(calls, block_backward, two)


def test_a_checkpoint_that_was_not_finished(calls):
    one = layer.MoEBlockBuffers(*SIZE, train=True)
    ck = layer.ExpertCheckpoint(one.moe)
    block_forward(one, ckpt=ck)
    calls.fails = "moe_ckpt_pack"
    with pytest.raises(L.MoEError):
        block_forward(one, ckpt=ck)
    calls.fails = None
    refused(calls, block_backward, one, ckpt=ck)
    block_forward(one, ckpt=ck)
    calls.fails = "moe_ckpt_unpack"
    with pytest.raises(L.MoEError):
        block_backward(one, ckpt=ck)
    calls.fails = None
    refused(calls, block_backward, one)
    block_backward(one, ckpt=ck)
