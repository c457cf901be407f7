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


def bad_tensors(dtypes):
    """Expert tensors that a call cannot take: of another type, too small, with strides, on another device, and not aligned."""
    other = next(t for t in (torch.float16, torch.float64) if t not in dtypes)
    yield torch.zeros(E, H, Hp, dtype=other)
    if len(dtypes) == 2:  # the tensors themselves, which cannot be left out
        yield None
    for t in dtypes:
        yield torch.zeros(E, H, Hp - 1, dtype=t)
        yield torch.zeros(E, Hp, H, dtype=t).transpose(1, 2) if H != Hp else torch.zeros(E, H, 2 * Hp, dtype=t)[..., ::2]
        yield torch.zeros(E, H, Hp, dtype=t, device="meta")
        yield torch.zeros(E * H * Hp + 1, dtype=t)[1:].view(E, H, Hp)


def test_momentum_step_refuses_before_it_updates(calls):  # noqa: F811
    """A second or third tensor that does not fit must not leave the first one updated."""
    b = layer.MoEBuffers(*SIZE, train=True)
    muon = layer.ExpertMuon(b)
    w = torch.zeros(E, H, Hp)
    low = torch.zeros(E, H, Hp, dtype=torch.bfloat16)
    for bad in bad_tensors((torch.float32, torch.bfloat16)):
        for at in range(3):
            refused(calls, muon.step, b, *(bad if k == at else w for k in range(3)), 1e-3)
    for bad in bad_tensors((torch.bfloat16,)):
        for at in range(3):
            refused(calls, muon.step, b, w, w, w, 1e-3, low=tuple(bad if k == at else low for k in range(3)))
    refused(calls, muon.step, b, w, w, w, 1e-3, low=(low, low))
    muon.step(b, w, low, w, 1e-3, low=(low, None, None))
    assert calls.made == ["moe_muon_step"] * 3


def test_packing_refuses_before_it_writes(calls):  # noqa: F811
    w4 = layer.ExpertsW4(E, H, Hp, "cpu")
    w = torch.zeros(E, H, Hp)
    for bad in bad_tensors((torch.float32, torch.bfloat16)):
        for at in range(3):
            refused(calls, w4.pack, *(bad if k == at else w for k in range(3)))
            refused(calls, w4.unpack, *(bad if k == at else w for k in range(3)))
    w4.pack(w, w.bfloat16(), w).unpack(w, w, w)
    assert calls.made == ["moe_w4_pack"] * 3 + ["moe_w4_unpack"] * 3
