"""Calls of the layer that are refused are refused before anything is launched or changed.  The library's calls are stood in
for; CPU only."""
import torch

from token_dispatch_gb300 import layer
from tests.test_layer_shared_experts import SIZE, calls, refused  # noqa: F401

T, H, E, K, Hp = SIZE[:5]


def test_mod_forward_refuses_packed_experts_before_it_selects(calls):  # noqa: F811
    m = layer.MoDBuffers(2, 16, 4, *SIZE[1:])
    w4 = layer.ExpertsW4(E, H, Hp, "cpu")
    before = m.moe.forward
    for w in ((layer.ExpertsW4(E, H, Hp + 8, "cpu"), None, None), (w4, torch.zeros(1), None), (w4, None, torch.zeros(1))):
        refused(calls, layer.mod_forward, m, None, None, None, *w)
    assert m.moe.forward is before
    layer.mod_forward(m, None, None, None, w4, None, None)
    assert "moe_expert_ffn_w4" in calls.made
