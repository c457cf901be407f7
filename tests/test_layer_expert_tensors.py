"""What the layer refuses of 4-bit experts and of the momentum step, before anything is launched, and which calls it
makes.  The library's calls are stood in for; CPU only."""
import pytest
import torch

from token_dispatch_gb300 import layer
from tests.test_layer_shared_experts import GATE, SIZE, calls, refused  # noqa: F401

T, H, E, K, Hp = SIZE[:5]


def test_forwards_take_packed_experts(calls):  # noqa: F811
    w4 = layer.ExpertsW4(E, H, Hp, "cpu", group=32)
    assert w4.q_gate.shape == (E, Hp, 16) and w4.s_gate.shape == (E, Hp, 4) and w4.q_down.shape == (E, H, 16)
    b = layer.MoEBuffers(*SIZE, backward=False)
    layer.moe_forward(b, None, None, None, w4, None, None)
    assert "moe_expert_ffn_w4" in calls.made and "moe_expert_ffn_ex" not in calls.made
    m = layer.MoEBlockBuffers(*SIZE)
    calls.made.clear()
    layer.moe_block_forward(m, None, None, None, None, GATE, w4, None, None)
    assert calls.made.count("moe_expert_ffn_w4") == 1 and "moe_expert_ffn_ex" not in calls.made


def test_packed_experts_are_refused_where_they_do_not_fit(calls):  # noqa: F811
    w4 = layer.ExpertsW4(E, H, Hp, "cpu")
    t = torch.zeros(1)
    cases = [(layer.MoEBuffers(*SIZE, train=True), w4, None, None), (layer.MoEBuffers(*SIZE), w4, t, None),
             (layer.MoEBuffers(*SIZE), w4, None, t),
             (layer.MoEBuffers(*SIZE), layer.ExpertsW4(E, H, Hp + 8, "cpu"), None, None),
             (layer.MoEBuffers(*SIZE[:5], "f32", "cpu"), w4, None, None)]
    for b, *w in cases:
        before = b.forward
        refused(calls, layer.moe_forward, b, None, None, None, *w)
        assert b.forward is before  # the last forward is still there
    m = layer.MoEBlockBuffers(*SIZE, train=True)
    refused(calls, layer.moe_block_forward, m, None, None, None, None, GATE, w4, None, None)
    with pytest.raises(ValueError):
        layer.ExpertsW4(E, H, Hp, "cpu", group=16)
    refused(calls, w4.pack, torch.zeros(1, dtype=torch.float16), t, t)


def test_momentum_step_calls_and_refusals(calls):  # noqa: F811
    b = layer.MoEBuffers(*SIZE, train=True)
    muon = layer.ExpertMuon(b)
    assert muon.m_gate.shape == b.dw_gate.shape and not muon.m_down.any()
    w = torch.zeros(E, H, Hp)
    muon.step(b, w, w, w, 1e-3)
    assert calls.made == ["moe_muon_step"] * 3
    refused(calls, muon.step, layer.MoEBuffers(T, H, E, K, Hp + 8, "bf16", "cpu", train=True), w, w, w, 1e-3)
    refused(calls, muon.step, b, w.half(), w, w, 1e-3)
    with pytest.raises(ValueError):
        layer.ExpertMuon(layer.MoEBuffers(*SIZE))
